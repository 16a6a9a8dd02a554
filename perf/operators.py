"""Measured cases of the operators around the distillation loss: the cached top-K teacher built from teacher
logits, the embedding table tied to the output head with its gradient, and activations saved in 8 bits, alone
and as what an RMS norm's backward pass reads.

``run`` computes a case in plain torch (``own`` false) or through the package's entry points (``own`` true)."""
import math

import torch

own = False

BLOCK = 32  # columns that share one exponent in the 8-bit form
EPS = 1e-6


def listed():
    return [
        # one position of a teacher's output, as it is cached token by token while the teacher generates
        dict(name="topk_one_row", op="topk", T=1, V=32000, K=100, dtype="bf16", form=0, masked=False),
        # one chunk of rows of a 32K-token document over the large vocabulary
        dict(name="topk_chunk", op="topk", T=2048, V=201088, K=100, dtype="bf16", form=0, masked=False),
        # packed documents (a quarter of the rows masked), truncated log-probabilities, a long cache per row
        dict(name="topk_masked_f32", op="topk", T=301, V=50021, K=1000, dtype="f32", form=1, masked=True),
        # embedding of the tokens of one generation step
        dict(name="embed_step", op="embed", T=16, V=32000, d=2048, dtype="bf16", padded=False),
        # embedding of a 32K-token document
        dict(name="embed_document", op="embed", T=32768, V=201088, d=2880, dtype="bf16", padded=True),
        # gradient of a short prompt, added to the head's
        dict(name="embed_grad_prompt", op="embed_grad", T=200, V=32000, d=2048, dtype="bf16", grad="f32", add=True,
             padded=False),
        # gradient of a 32K-token document, added to the fp32 gradient of the tied head
        dict(name="embed_grad_tied", op="embed_grad", T=32768, V=201088, d=2880, dtype="bf16", grad="f32", add=True,
             padded=True),
        # gradient of an untied table, written whole in bf16; odd sizes
        dict(name="embed_grad_table", op="embed_grad", T=4099, V=32003, d=1000, dtype="f32", grad="bf16", add=False,
             padded=True),
        # the hidden states of one layer at 128K tokens, saved and restored
        dict(name="save_131072", op="save", T=131072, d=2880, dtype="bf16"),
        # a few rows in fp32
        dict(name="save_odd_f32", op="save", T=77, d=1000, dtype="f32"),
        # a training step of the norm before the head: 32K tokens
        dict(name="norm_document", op="norm", T=32768, d=2880, dtype="bf16"),
        # a training step of a small model on a short sequence
        dict(name="norm_short", op="norm", T=257, d=520, dtype="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "embed", "embed_grad", "save", "norm"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "topk":
        V = _log_uniform(rng, 1000, 210000)
        T = _log_uniform(rng, 1, max(1, min(8192, 100_000_000 // V)))
        return dict(op=op, T=T, V=V, K=_log_uniform(rng, 1, min(1024, V)), dtype=dtype, form=rng.choice([0, 1]),
                    masked=rng.random() < 0.5)
    d = 8 * _log_uniform(rng, 8, 1024)
    T = _log_uniform(rng, 1, min(65536, 60_000_000 // d))
    if op in ("save", "norm"):
        return dict(op=op, T=T, d=d, dtype=dtype)
    V = _log_uniform(rng, 500, min(210000, 200_000_000 // d))
    case = dict(op=op, T=T, V=V, d=d, dtype=dtype, padded=rng.random() < 0.5)
    if op == "embed_grad":
        case["grad"] = rng.choice(["bf16", "f32"])
        case["add"] = case["grad"] == "f32" and rng.random() < 0.6
    return case


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _zipf(V):
    """Cumulative word frequencies: token r drawn with weight 1 / (r + 2.7)."""
    w = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
    return torch.cumsum(w / w.sum(), 0)


def _scale(case):
    return math.sqrt(case["d"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, dt = case["T"], _dtype(case["dtype"])

    def normal(*shape, dtype=dt, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)

    s = dict(case=case)
    if case["op"] == "topk":
        s["logits"] = normal(T, case["V"], std=3.0)
        s["mask"] = (torch.rand(T, device="cuda", generator=g) >= 0.25) if case["masked"] else None
        return s
    d = case["d"]
    if case["op"] in ("embed", "embed_grad"):
        u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
        tokens = torch.searchsorted(_zipf(case["V"]).cuda(), u).clamp_(max=case["V"] - 1)
        if case["padded"]:  # an eighth of the positions pads the batch
            tokens = torch.where(torch.rand(T, device="cuda", generator=g) < 0.125, -1, tokens)
        s["tokens"] = tokens
    if case["op"] == "embed":
        s["W"] = normal(case["V"], d, std=d ** -0.5)
    elif case["op"] == "embed_grad":
        s["dY"] = normal(T, d)
        s["dW"] = normal(case["V"], d, dtype=_dtype(case["grad"])) if case["add"] else None
    else:
        # hidden states: columns of different size, as residual streams have them
        s["x"] = (normal(T, d, dtype=torch.float32) * torch.exp(normal(d, dtype=torch.float32, std=0.5))).to(dt)
        if case["op"] == "norm":
            s["x"].requires_grad_(True)
            s["weight"] = (1.0 + normal(d, dtype=torch.float32, std=0.1)).to(dt).requires_grad_(True)
            s["dY"] = normal(T, d)
    return s


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import chunked_kl_loss_amd as ckl
        if op == "topk":
            return ckl.teacher_topk(state["logits"], case["K"], mask=state["mask"], teacher_form=case["form"])
        if op == "embed":
            return ckl.embedding(state["W"], state["tokens"], scale=_scale(case))
        if op == "embed_grad":
            return ckl.embedding_backward(state["dY"], state["tokens"], case["V"], scale=_scale(case),
                                          dw_dtype=_dtype(case["grad"]), add_to=state["dW"])
        if op == "save":
            codes, exps = ckl.act_encode(state["x"])
            return ckl.act_decode(codes, exps, dtype=state["x"].dtype)
        y = ckl.rms_norm_8bit(state["x"], state["weight"], eps=EPS)
        dx, dweight = torch.autograd.grad(y, (state["x"], state["weight"]), state["dY"])
        return y, dx, dweight
    if op == "topk":
        return _plain_topk(state, case)
    if op == "embed":
        return _plain_embed(state, case)
    if op == "embed_grad":
        return _plain_embed_grad(state, case)
    if op == "save":
        return _plain_restored(state["x"]).to(state["x"].dtype)
    return _plain_norm(state)


# ------------------------------------------------------------ plain forms --
def _plain_topk(state, case):
    z, K, mask = state["logits"].float(), case["K"], state["mask"]
    values, idx = torch.sort(z, dim=1, descending=True, stable=True)
    values, idx = values[:, :K], idx[:, :K].to(torch.int32)
    top = values[:, :1]
    lse = (top + torch.log(torch.exp(z - top).sum(dim=1, keepdim=True)))
    if case["form"] == 1:
        values = values - lse
    lse = lse[:, 0]
    if mask is not None:
        keep = mask[:, None]
        idx = torch.where(keep, idx, torch.arange(K, device=idx.device, dtype=torch.int32))
        values = torch.where(keep, values, 0.0)
        lse = torch.where(mask, lse, 0.0)
    return idx.contiguous(), values.contiguous(), lse


def _plain_embed(state, case):
    W, tokens = state["W"], state["tokens"]
    inside = (tokens >= 0) & (tokens < W.shape[0])
    rows = W[torch.where(inside, tokens, 0)].float() * _scale(case)
    return torch.where(inside[:, None], rows, 0.0).to(W.dtype)


def _plain_embed_grad(state, case):
    dY, tokens, dW = state["dY"], state["tokens"], state["dW"]
    inside = (tokens >= 0) & (tokens < case["V"])
    rows = torch.where(inside[:, None], dY.float() * _scale(case), 0.0)
    if dW is None:
        dW = torch.zeros(case["V"], case["d"], dtype=torch.float32, device=dY.device)
    dW.index_add_(0, torch.where(inside, tokens, 0), rows)
    return dW.to(_dtype(case["grad"]))


def _plain_restored(x):
    """x as 8 bits hold it: blocks of 32 columns share the power of two that brings their largest magnitude
    below 127.5; each value is rounded to a whole number of it."""
    T, d = x.shape
    pad = -d % BLOCK
    b = torch.cat([x.float(), x.new_zeros(T, pad, dtype=torch.float32)], dim=1).view(T, -1, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    _, e = torch.frexp(top)  # top = m 2^e with m in [0.5, 1)
    step = torch.ldexp(torch.ones_like(top), e - 7)
    step = torch.where(top >= 127.5 * step, 2.0 * step, step).clamp(min=2.0 ** -126)
    return (torch.round(b / step) * step).view(T, -1)[:, :d].contiguous()


def _plain_norm(state):
    x, w, dY = state["x"].detach(), state["weight"].detach(), state["dY"]
    x32, w32, g = x.float(), w.float(), dY.float()
    r = torch.rsqrt((x32 * x32).mean(dim=1, keepdim=True) + EPS)
    y = (x32 * r * w32).to(x.dtype)
    xs = _plain_restored(x)
    gw = g * w32
    c = (gw * xs).mean(dim=1, keepdim=True) * r * r
    dx = (r * (gw - xs * c)).to(x.dtype)
    dweight = (g * xs * r).sum(dim=0).to(w.dtype)
    return y, dx, dweight


# ------------------------------------------------------ 64-bit definitions --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "topk":
        z = s["logits"].double()
        values = torch.topk(z, case["K"], dim=1).values
        lse = torch.logsumexp(z, dim=1)
        if case["form"] == 1:
            values = values - lse[:, None]
        if s["mask"] is not None:
            values[~s["mask"]] = 0.0
            lse[~s["mask"]] = 0.0
        return None, values, lse
    if case["op"] == "embed":
        t, W = s["tokens"], s["W"]
        out = torch.zeros(t.shape[0], W.shape[1], dtype=torch.float64, device="cuda")
        at = ((t >= 0) & (t < W.shape[0])).nonzero()[:, 0]
        out[at] = W.double()[t[at]] * math.sqrt(case["d"])
        return out
    if case["op"] == "embed_grad":
        t = s["tokens"]
        at = ((t >= 0) & (t < case["V"])).nonzero()[:, 0]
        total = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
        total.index_add_(0, t[at], s["dY"][at].double())
        total *= math.sqrt(case["d"])
        return total if s["dW"] is None else total + s["dW"].double()
    x = s["x"].detach().double()
    T, d = x.shape
    held = torch.empty_like(x)
    for c in range(0, d, BLOCK):
        block = x[:, c:c + BLOCK]
        top = block.abs().max(dim=1, keepdim=True).values.clamp(min=1e-300)
        e = torch.floor(torch.log2(top / 127.5)) + 1.0  # smallest e with top < 127.5 * 2^e
        step = torch.exp2(e.clamp(min=-126.0))
        held[:, c:c + BLOCK] = torch.round(block / step) * step
    if case["op"] == "save":
        return held
    w, g = s["weight"].detach().double(), s["dY"].double()
    inv = 1.0 / torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / d + EPS)
    n = held * inv  # the normalised rows that the backward pass works with
    y = x * inv * w
    gw = g * w
    dx = inv * (gw - n * ((gw * n).sum(dim=1, keepdim=True) / d))
    return y, dx, (g * n).sum(dim=0)


# ------------------------------------------------------------------- work --
def work(case):
    T, e = case["T"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "topk":
        rows = T * (0.75 if case["masked"] else 1.0)
        n = rows * case["V"]
        # one comparison, one exponential and one addition an element
        return {"bytes": n * e + T * (case["K"] * 8 + 4), "flops": 3 * n}
    d = case["d"]
    if case["op"] in ("save", "norm"):
        held = T * d + T * -(-d // BLOCK)
        if case["op"] == "save":  # read x, write the 8-bit form, read it, write the restored x
            return {"bytes": 2 * T * d * e + 2 * held, "flops": 4 * T * d}
        # forward: read x, write y and the 8-bit form; backward: read dY and the 8-bit form, write dx
        return {"bytes": 4 * T * d * e + 2 * held + 2 * d * e, "flops": 16 * T * d}
    p = torch.diff(_zipf(case["V"]), prepend=torch.zeros(1, dtype=torch.float64))
    n = T * (0.875 if case["padded"] else 1.0)
    rows = float((1.0 - (1.0 - p) ** n).sum())  # distinct tokens to be expected
    if case["op"] == "embed":
        return {"bytes": rows * d * e + T * d * e + T * 8, "flops": T * d}
    ge = 2 if case["grad"] == "bf16" else 4
    out = 2 * rows * d * ge if case["add"] else case["V"] * d * ge
    return {"bytes": n * d * e + out + T * 8, "flops": 2 * n * d}
