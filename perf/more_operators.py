"""Cases of a transformer layer's projections in 16 bits: the gated feed-forward (both projections,
the activation and the product), its gradients, and a shared projection with the low-rank adapters
of many requests beside it.

  gated        pre = x W_in^T (tokens x 2 hidden: the gate's columns, then the other projection's);
               h = act(gate) * up
  gated_grad   from dh: dpre = [dh * up * act'(gate) | dh * act(gate)];
               dx = dpre W_in, dW_in = dpre^T x
  block_grad   the same behind y = h W_out^T, from dy: dh = dy W_out, h = act(gate) * up;
               dx, dW_in as above, dW_out = dy^T h
  adapters     y_i = x_i W^T + scale_s (x_i A_s^T) B_s^T, s = index_i the adapter of row i's
               request; rows whose index is negative have none

act: silu g / (1 + e^-g); gelu g Phi(g); gelu_tanh g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a decode step through a wide feed-forward: the weights' bytes.
        dict(name="gated_token", op="gated", tokens=1, width=8192, hidden=28672, type="bf16",
             act="silu", save=False),
        # A few tokens through a small layer: latency alone.
        dict(name="gated_few", op="gated", tokens=7, width=1024, hidden=2816, type="bf16",
             act="silu", save=False),
        # An odd batch of a training step, which keeps the projections for its backward pass.
        dict(name="gated_ragged", op="gated", tokens=333, width=2200, hidden=1000, type="f16",
             act="gelu", save=True),
        # A long prompt through the wide layer: the tensor cores' rate.
        dict(name="gated_prompt", op="gated", tokens=4096, width=8192, hidden=28672, type="bf16",
             act="silu", save=False),
        # The gradient where the second projection runs elsewhere (in 8 bits, say).
        dict(name="gated_grad", op="gated_grad", tokens=4096, width=8192, hidden=8192, type="bf16",
             act="silu"),
        # The same for an odd batch of a small layer.
        dict(name="gated_grad_ragged", op="gated_grad", tokens=777, width=1000, hidden=2200,
             type="f16", act="gelu_tanh"),
        # The whole block's gradient in a training step.
        dict(name="block_grad", op="block_grad", tokens=4096, width=8192, hidden=8192, type="bf16",
             act="silu"),
        # The same for a small model's layer.
        dict(name="block_grad_small", op="block_grad", tokens=512, width=1024, hidden=2816,
             type="bf16", act="silu"),
        # One token of one request with its adapter: the shared weights' bytes.
        dict(name="adapters_token", op="adapters", tokens=1, inner=8192, outer=8192, adapters=16,
             rank=16, type="bf16", order="mixed"),
        # A decode batch, nearly every row with an adapter of its own.
        dict(name="adapters_decode", op="adapters", tokens=64, inner=8192, outer=8192, adapters=64,
             rank=16, type="bf16", order="mixed"),
        # An odd batch of rows in any order over a few adapters of a small rank.
        dict(name="adapters_ragged", op="adapters", tokens=333, inner=2200, outer=1000, adapters=5,
             rank=8, type="f16", order="mixed"),
        # Prompts of several requests one behind the other.
        dict(name="adapters_prompt", op="adapters", tokens=8192, inner=8192, outer=8192,
             adapters=8, rank=64, type="bf16", order="segments"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(("gated", "gated_grad", "block_grad", "adapters"))
    kind = rng.choice(("bf16", "f16"))
    if op == "adapters":
        return dict(op=op, tokens=_log(rng, 1, 8192), inner=_eights(rng, 64, 8192),
                    outer=_eights(rng, 64, 8192), adapters=_log(rng, 1, 64),
                    rank=8 * rng.choice((1, 2, 3, 4, 6, 8, 16)), type=kind,
                    order=rng.choice(("mixed", "segments")))
    c = dict(op=op, tokens=_log(rng, 1, 4096), width=_eights(rng, 64, 8192),
             hidden=_eights(rng, 64, 28672 if op == "gated" else 8192), type=kind,
             act=rng.choice(("silu", "gelu", "gelu_tanh")))
    if op == "gated":
        c["save"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "adapters":
        t, k, n, r = c["tokens"], c["inner"], c["outer"], c["rank"]
        used = min(c["adapters"], t)
        return dict(bytes=2 * (t * k + n * k + t * n + used * r * (k + n)) + 4 * (t + used),
                    flops=2 * t * n * k + 2 * t * r * (k + n))
    t, d, f = c["tokens"], c["width"], c["hidden"]
    if c["op"] == "gated":
        return dict(bytes=2 * (t * d + 2 * f * d + t * f * (3 if c["save"] else 1)),
                    flops=4 * t * d * f)
    if c["op"] == "gated_grad":  # dh, pre, x and W_in read; dx and dW_in written
        return dict(bytes=2 * (3 * t * f + 2 * t * d + 4 * f * d), flops=8 * t * d * f)
    # dy, pre, x, W_in and W_out read; dx, dW_in and dW_out written
    return dict(bytes=2 * (2 * t * f + 3 * t * d + 6 * f * d), flops=12 * t * d * f)


# ------------------------------------------------------------------ inputs
def _normal(gen, kind, *shape, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda")
    return x.mul_(scale).to(TYPES[kind])


def _activations(gen, kind, rows, cols):
    """Normal values whose channels differ in size, a few of them by much, as behind a norm."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    chan = torch.exp(0.3 * torch.randn(cols, generator=gen, device="cuda"))
    big = torch.rand(cols, generator=gen, device="cuda") < 0.002
    return x.mul_(torch.where(big, 8.0 * chan, chan)).to(TYPES[kind])


def _index(gen, c):
    """The adapter of each row; about one request in ten has none."""
    t, s = c["tokens"], c["adapters"]
    if c["order"] == "mixed":
        i = torch.randint(0, s, (t,), generator=gen, device="cuda")
        none = torch.rand(t, generator=gen, device="cuda") < 0.1
    else:  # requests one behind the other, of lengths of all sizes
        ends = torch.rand(t, generator=gen, device="cuda") < max(1.0 / 700, 3.0 / t)
        request = ends.long().cumsum(0)
        pick = torch.randint(0, s, (t + 1,), generator=gen, device="cuda")
        i = pick[request]
        none = (torch.rand(t + 1, generator=gen, device="cuda") < 0.1)[request]
    if t <= 8:
        none = none & False  # so few rows all have one: a call without any is the plain product
    return torch.where(none, torch.full_like(i, -1), i).int()


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda").manual_seed(int(seed))
    kind = c["type"]
    s = dict(case=c)
    if c["op"] == "adapters":
        t, k, n, a, r = c["tokens"], c["inner"], c["outer"], c["adapters"], c["rank"]
        s["x"] = _activations(gen, kind, t, k)
        s["w"] = _normal(gen, kind, n, k, scale=k ** -0.5)
        s["a"] = _normal(gen, kind, a, r, k, scale=k ** -0.5)
        s["b"] = _normal(gen, kind, a, n, r, scale=0.3 * r ** -0.5)
        s["scale"] = 0.5 + torch.rand(a, generator=gen, device="cuda")
        s["index"] = _index(gen, c)
    else:
        t, d, f = c["tokens"], c["width"], c["hidden"]
        s["x"] = _activations(gen, kind, t, d)
        s["w_in"] = _normal(gen, kind, 2 * f, d, scale=d ** -0.5)
        if c["op"] != "gated":  # what the forward pass kept
            s["pre"] = (s["x"] @ s["w_in"].t()).contiguous()
        if c["op"] == "gated_grad":
            s["dh"] = _normal(gen, kind, t, f, scale=1e-2)
        elif c["op"] == "block_grad":
            s["w_out"] = _normal(gen, kind, d, f, scale=f ** -0.5)
            s["dy"] = _normal(gen, kind, t, d, scale=1e-2)
    if own:  # the handle that a program keeps for its calls
        from stream_decomposition_abft_gb300 import layers
        s["workspace"] = layers.workspace("cuda")
    return s


# ------------------------------------------------------------------ the plain form
def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), \
        0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3.0 * 0.044715 * g * g)


def _plain(s):
    c = s["case"]
    kind = TYPES[c["type"]]
    x = s["x"].float()
    if c["op"] == "adapters":
        n_ad, r, k = s["a"].shape
        t = x @ s["a"].float().view(n_ad * r, k).t()
        mine = s["index"].long()[:, None] == torch.arange(n_ad, device=x.device)[None, :]
        t = torch.where(mine[:, :, None], t.view(-1, n_ad, r) * s["scale"][None, :, None],
                        t.new_zeros(()))
        up = s["b"].float().permute(0, 2, 1).reshape(n_ad * r, -1)
        return (x @ s["w"].float().t() + t.view(-1, n_ad * r) @ up).to(kind)
    f = c["hidden"]
    if c["op"] == "gated":
        pre = x @ s["w_in"].float().t()
        h = (_act(pre[:, :f], c["act"])[0] * pre[:, f:]).to(kind)
        return dict(h=h, pre=pre.to(kind)) if c["save"] else h
    gate, up = s["pre"][:, :f].float(), s["pre"][:, f:].float()
    a, da = _act(gate, c["act"])
    dh = s["dh"].float() if c["op"] == "gated_grad" else s["dy"].float() @ s["w_out"].float()
    dpre = torch.cat((dh * up * da, dh * a), 1)
    out = dict(dx=(dpre @ s["w_in"].float()).to(kind), dw_in=(dpre.t() @ x).to(kind))
    if c["op"] == "block_grad":
        out["dw_out"] = (s["dy"].float().t() @ (a * up)).to(kind)
    return out


# ------------------------------------------------------------------ the framework's operators
def _framework(s):
    from stream_decomposition_abft_gb300 import layers
    c, ws = s["case"], s["workspace"]
    if c["op"] == "adapters":
        return layers.linear(s["x"], s["w"], layers.Adapters(s["a"], s["b"], s["scale"]),
                             s["index"], workspace=ws)
    if c["op"] == "gated":
        if not c["save"]:
            return layers.gated(s["x"], s["w_in"], c["act"], workspace=ws)
        h, pre = layers.gated(s["x"], s["w_in"], c["act"], save=True, workspace=ws)
        return dict(h=h, pre=pre)
    if c["op"] == "gated_grad":
        dx, dw = layers.gated_backward(s["dh"], s["x"], s["w_in"], s["pre"], c["act"],
                                       workspace=ws)
        return dict(dx=dx, dw_in=dw)
    dx, dw_in, dw_out = layers.feed_forward_backward(s["dy"], s["x"], s["w_in"], s["w_out"],
                                                     s["pre"], c["act"], workspace=ws)
    return dict(dx=dx, dw_in=dw_in, dw_out=dw_out)


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * torch.special.erfc(-g / 2.0 ** 0.5)
    return g / (1.0 + torch.exp(-2.0 * (2.0 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    x = s["x"].double()
    if c["op"] == "adapters":
        y = x @ s["w"].double().t()
        for i in range(c["adapters"]):
            rows = torch.nonzero(s["index"] == i)[:, 0]
            low = x[rows] @ s["a"][i].double().t() @ s["b"][i].double().t()
            y[rows] += s["scale"][i].double() * low
        return y
    if c["op"] == "gated":
        gate, up = (x @ w.double().t() for w in s["w_in"].chunk(2))
        h = _exact_act(gate, c["act"]) * up
        return dict(h=h, pre=torch.cat((gate, up), 1)) if c["save"] else h
    # The derivative of act from the definition by automatic differentiation.
    gate, up = (p.double().detach().requires_grad_() for p in s["pre"].chunk(2, 1))
    h = _exact_act(gate, c["act"]) * up
    dh = s["dh"].double() if c["op"] == "gated_grad" else \
        torch.einsum("td,df->tf", s["dy"].double(), s["w_out"].double())
    dgate, dup = torch.autograd.grad(h, (gate, up), dh)
    w_gate, w_up = (w.double() for w in s["w_in"].chunk(2))
    out = dict(dx=dgate @ w_gate + dup @ w_up,
               dw_in=torch.cat((dgate.t() @ x, dup.t() @ x)))
    if c["op"] == "block_grad":
        out["dw_out"] = s["dy"].double().t() @ h.detach()
    return out
