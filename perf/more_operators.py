"""Measured cases of the operators between a model's last block and its training signal: log probabilities of given
tokens with entropy and top alternatives (from logits, and from hidden states and the output head), dropout from a
counter-based generator, and the RMS norm with the residual's addition, also with its output in 8 bits.

``run`` computes a case in plain torch (``own`` false) or through the package's entry points (``own`` true)."""
import math

import torch

own = False

BLOCK = 32  # columns that share one exponent in the int8 form
EPS = 1e-6


def listed():
    return [
        # the tokens that a batch of sixteen sequences has just sampled, with twenty alternatives each
        dict(name="logprobs_step", op="logprobs", T=16, V=32000, top=20, dtype="bf16", masked=False, train=False),
        # one chunk of a packed document scored over the large vocabulary
        dict(name="logprobs_chunk", op="logprobs", T=2048, V=201088, top=5, dtype="bf16", masked=True, train=False),
        # a policy-gradient step with an entropy bonus on logits in fp32; odd vocabulary
        dict(name="logprobs_grad_f32", op="logprobs", T=509, V=50021, top=0, dtype="f32", masked=False, train=True),
        # eight sampled tokens scored from their hidden states
        dict(name="head_step", op="head", T=8, V=201088, d=2880, dtype="bf16", masked=False, train=False),
        # cross entropy on one chunk of rows of the large vocabulary, both gradients
        dict(name="head_train", op="head", T=2048, V=201088, d=2880, dtype="bf16", masked=False, train=True),
        # a small model in fp32, packed documents, odd sizes
        dict(name="head_odd_f32", op="head", T=301, V=5003, d=520, dtype="f32", masked=True, train=True),
        # a branch's output at 32K tokens, forward and backward
        dict(name="dropout_document", op="dropout", T=32768, d=2880, dtype="bf16", p=0.1),
        # a small activation whose size is no multiple of anything
        dict(name="dropout_odd_f32", op="dropout", T=77, d=1003, dtype="f32", p=0.25),
        # a training step of the norm behind a branch with dropout: 32K tokens
        dict(name="addnorm_document", op="addnorm", T=32768, d=2880, dtype="bf16", residual="bf16", p=0.1),
        # a short sequence of a small model that keeps its residual stream in fp32
        dict(name="addnorm_short", op="addnorm", T=257, d=520, dtype="bf16", residual="f32", p=0.0),
        # one generation step into a product in 8 bits
        dict(name="quant_step_e4m3", op="quant", T=16, d=2880, dtype="bf16", residual="bf16", form="e4m3"),
        # a long prompt, into blocks of 32 columns with a power of two each
        dict(name="quant_prompt_int8", op="quant", T=65536, d=2880, dtype="bf16", residual="bf16", form="int8"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "head", "dropout", "addnorm", "quant"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "logprobs":
        V = _log_uniform(rng, 1000, 210000)
        T = _log_uniform(rng, 1, max(1, min(8192, 100_000_000 // V)))
        return dict(op=op, T=T, V=V, top=rng.choice([0, _log_uniform(rng, 1, 200)]), dtype=dtype,
                    masked=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "head":
        d = 8 * _log_uniform(rng, 8, 512)
        V = _log_uniform(rng, 500, 210000)
        most = 1_000_000_000_000 if dtype == "bf16" else 50_000_000_000
        T = _log_uniform(rng, 1, max(1, min(8192, 200_000_000 // V, most // (V * d))))
        return dict(op=op, T=T, V=V, d=d, dtype=dtype, masked=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "dropout":
        d = _log_uniform(rng, 1, 9000)
        T = _log_uniform(rng, 1, min(65536, 60_000_000 // d))
        return dict(op=op, T=T, d=d, dtype=dtype, p=round(rng.uniform(0.01, 0.6), 3))
    d = 8 * _log_uniform(rng, 8, 1024)
    T = _log_uniform(rng, 1, min(65536, 60_000_000 // d))
    residual = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    case = dict(op=op, T=T, d=d, dtype=dtype, residual=residual)
    if op == "addnorm":
        case["p"] = rng.choice([0.0, round(rng.uniform(0.01, 0.5), 3)])
    else:
        case["form"] = rng.choice(["int8", "e4m3"])
    return case


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, dt = case["T"], _dtype(case["dtype"])

    def normal(*shape, dtype=dt, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)

    s = dict(case=case)
    if case["op"] in ("logprobs", "head"):
        V = case["V"]
        s["tokens"] = tokens = torch.randint(0, V, (T,), device="cuda", generator=g)
        s["mask"] = (torch.rand(T, device="cuda", generator=g) >= 0.25) if case["masked"] else None
        if case["train"]:  # a weight for each token, and a small bonus on the entropy, of a mean over the rows
            s["dlogprob"] = normal(T, dtype=torch.float32, std=1.0 / T)
            s["dentropy"] = torch.full((T,), -0.01 / T, dtype=torch.float32, device="cuda")
        # the given tokens are likely ones: some are almost sure, some are one among many
        lift = normal(T, dtype=torch.float32, std=5.0) + 8.0
        if case["op"] == "logprobs":
            z = normal(T, V, dtype=torch.float32, std=3.0)
            z[torch.arange(T, device="cuda"), tokens] += lift
            s["logits"] = z.to(dt).requires_grad_(case["train"])
            return s
        d = case["d"]
        W = normal(V, d, dtype=torch.float32, std=d ** -0.5)
        H = normal(T, d, dtype=torch.float32, std=2.0) + lift[:, None] * W[tokens]
        s["H"] = H.to(dt).requires_grad_(case["train"])
        s["W"] = W.to(dt).requires_grad_(case["train"])
        return s
    d = case["d"]
    # hidden states: columns of different size, as residual streams have them
    size = torch.exp(normal(d, dtype=torch.float32, std=0.5))
    if case["op"] == "dropout":
        s["x"] = (normal(T, d, dtype=torch.float32) * size).to(dt).requires_grad_(True)
        s["dy"] = normal(T, d)
        s["seed"], s["offset"] = 1234567 + seed, 3
        return s
    train = case["op"] == "addnorm"
    rt = _dtype(case["residual"])
    s["x"] = (normal(T, d, dtype=torch.float32, std=0.3) * size).to(dt).requires_grad_(train)
    s["residual"] = (normal(T, d, dtype=torch.float32) * size).to(rt).requires_grad_(train)
    s["weight"] = (1.0 + normal(d, dtype=torch.float32, std=0.1)).to(dt).requires_grad_(train)
    if train:
        s["dy"], s["dh"] = normal(T, d), normal(T, d, dtype=rt)
        s["seed"], s["offset"] = 7654321 + seed, 5
    return s


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(state, case)
    if op == "logprobs":
        return _plain_logprobs(state, case)
    if op == "head":
        return _plain_head(state, case)
    if op == "dropout":
        x, keep = state["x"].detach(), _plain_keep(case, state)
        scale = _keep_scale(case["p"])
        return tuple(torch.where(keep, t.float() * scale, 0.0).to(t.dtype) for t in (x, state["dy"]))
    if op == "addnorm":
        return _plain_addnorm(state, case)
    return _plain_quant(state, case)


def _own(state, case):
    import chunked_kl_loss_amd as ckl
    op = case["op"]
    if op == "logprobs":
        logprob, entropy, top_idx, top_logprob = ckl.token_logprobs(state["logits"], state["tokens"], top=case["top"],
                                                                    mask=state["mask"])
        out = (logprob.detach(), entropy.detach(), top_idx, top_logprob)
        if case["train"]:
            out += torch.autograd.grad((logprob, entropy), (state["logits"],), (state["dlogprob"], state["dentropy"]))
        return out
    if op == "head":
        logprob, entropy = ckl.head_logprobs(state["H"], state["W"], state["tokens"], mask=state["mask"])
        out = (logprob.detach(), entropy.detach())
        if case["train"]:
            out += torch.autograd.grad((logprob, entropy), (state["H"], state["W"]),
                                       (state["dlogprob"], state["dentropy"]))
        return out
    if op == "dropout":
        y = ckl.dropout(state["x"], case["p"], seed=state["seed"], offset=state["offset"])
        return (y.detach(),) + torch.autograd.grad(y, (state["x"],), state["dy"])
    if op == "addnorm":
        y, h = ckl.add_rms_norm(state["x"], state["residual"], state["weight"], eps=EPS, p=case["p"],
                                seed=state["seed"], offset=state["offset"])
        grads = torch.autograd.grad((y, h), (state["x"], state["residual"], state["weight"]),
                                    (state["dy"], state["dh"]))
        return (y.detach(), h.detach()) + grads
    codes, scales, h = ckl.add_norm_quant(state["x"], state["residual"], state["weight"], eps=EPS, form=case["form"])
    if case["form"] == "int8":
        return ckl.act_decode(codes, scales), h
    return (codes.float() * scales[:, None]).to(torch.bfloat16), h


# ------------------------------------------------------------ plain forms --
def _plain_rows(z, tokens):
    """Log probabilities, those of the tokens, and the entropies of rows of logits in fp32."""
    m = z.amax(dim=1, keepdim=True)
    logq = z - (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True)))
    entropy = -(torch.exp(logq) * logq).sum(dim=1)
    return logq, torch.gather(logq, 1, tokens[:, None])[:, 0], entropy


def _plain_dz(logq, entropy, state):
    """Gradient of the logits."""
    a, b = state["dlogprob"][:, None], state["dentropy"][:, None]
    if state["mask"] is not None:
        a, b = a * state["mask"][:, None], b * state["mask"][:, None]
    dz = -torch.exp(logq) * (a + b * (logq + entropy[:, None]))
    dz[torch.arange(dz.shape[0], device=dz.device), state["tokens"]] += a[:, 0]
    return dz


def _keep_rows(mask, *rows):
    return rows if mask is None else tuple(torch.where(mask, r, 0.0) for r in rows)


def _plain_logprobs(state, case):
    z, mask, top = state["logits"].detach().float(), state["mask"], case["top"]
    logq, logprob, entropy = _plain_rows(z, state["tokens"])
    if top:
        values, idx = torch.sort(z, dim=1, descending=True, stable=True)
        idx = idx[:, :top].to(torch.int32)
        values = torch.gather(logq, 1, idx.long())
    else:
        idx, values = z.new_zeros(z.shape[0], 0, dtype=torch.int32), z.new_zeros(z.shape[0], 0)
    if mask is not None:
        idx = torch.where(mask[:, None], idx, torch.arange(top, device=idx.device, dtype=torch.int32))
        values = torch.where(mask[:, None], values, 0.0)
    out = _keep_rows(mask, logprob, entropy) + (idx.contiguous(), values)
    if case["train"]:
        out += (_plain_dz(logq, entropy, state).to(state["logits"].dtype),)
    return out


def _plain_head(state, case):
    H, W = state["H"].detach().float(), state["W"].detach().float()
    logq, logprob, entropy = _plain_rows(H @ W.t(), state["tokens"])
    out = tuple(_keep_rows(state["mask"], logprob, entropy))
    if case["train"]:
        dz = _plain_dz(logq, entropy, state)
        out += ((dz @ W).to(state["H"].dtype), (dz.t() @ H).to(state["W"].dtype))
    return out


def _threshold(p):
    return round(p * 65536)


def _keep_scale(p):
    return 65536.0 / (65536 - _threshold(p))


def _plain_keep(case, state):
    """Which elements are kept: sixteen bits each of Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
    "Parallel random numbers: as easy as 1, 2, 3", 2011), one counter for eight consecutive elements."""
    n = case["T"] * case["d"]
    low = 0xFFFFFFFF
    c0 = torch.arange((n + 7) // 8, dtype=torch.int64, device="cuda")
    c1 = c0 >> 32
    c0 = c0 & low
    c2 = torch.full_like(c0, state["offset"] & low)
    c3 = torch.full_like(c0, state["offset"] >> 32)
    k0, k1 = state["seed"] & low, state["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (products past 2^63 wrap; their 64 bits are what is wanted)
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], dim=1)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(-1)[:n]
    return (bits >= _threshold(case["p"])).view(case["T"], case["d"])


def _plain_h(state, case):
    x = state["x"].detach().float()
    if case.get("p"):
        x = torch.where(_plain_keep(case, state), x * _keep_scale(case["p"]), 0.0)
    h = (state["residual"].detach().float() + x).to(state["residual"].dtype)
    h32 = h.float()
    return h, h32, torch.rsqrt((h32 * h32).mean(dim=1, keepdim=True) + EPS)


def _plain_addnorm(state, case):
    h, h32, r = _plain_h(state, case)
    w, dy = state["weight"].detach(), state["dy"].float()
    n, gw = h32 * r, dy * w.float()
    y = (n * w.float()).to(state["x"].dtype)
    dres = state["dh"].float() + r * (gw - n * (gw * n).mean(dim=1, keepdim=True))
    dx = dres
    if case["p"]:
        dx = torch.where(_plain_keep(case, state), dres * _keep_scale(case["p"]), 0.0)
    return y, h, dx.to(state["x"].dtype), dres.to(h.dtype), (dy * n).sum(dim=0).to(w.dtype)


def _plain_quant(state, case):
    """What the 8 bits stand for, as a bf16 product reads them, and h."""
    h, h32, r = _plain_h(state, case)
    y = h32 * r * state["weight"].float()
    T, d = y.shape
    if case["form"] == "e4m3":  # one scale a row: the largest magnitude becomes 448
        scale = (y.abs().amax(dim=1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
        q = (y / scale).clamp(-448.0, 448.0)
        # three bits behind the first; below 2^-6 steps of 2^-9
        _, e = torch.frexp(q)
        step = torch.ldexp(torch.ones_like(q), (e - 4).clamp(min=-9))
        return (torch.round(q / step) * step * scale).to(torch.bfloat16), h
    pad = -d % BLOCK
    b = torch.cat([y, y.new_zeros(T, pad)], dim=1).view(T, -1, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    _, e = torch.frexp(top)  # top = m 2^e with m in [0.5, 1)
    step = torch.ldexp(torch.ones_like(top), e - 7)
    step = torch.where(top >= 127.5 * step, 2.0 * step, step).clamp(min=2.0 ** -126)
    return (torch.round(b / step) * step).view(T, -1)[:, :d].to(torch.bfloat16), h


# ------------------------------------------------------ 64-bit definitions --
def _exact_rows(z, s, case, top):
    """From logits in 64 bits: outputs per row and, for training, the logits' gradient."""
    T = z.shape[0]
    at = torch.arange(T, device="cuda")
    lse = torch.logsumexp(z, dim=1)
    logprob = z[at, s["tokens"]] - lse
    q = torch.exp(z - lse[:, None])
    entropy = lse - (q * z).sum(dim=1)
    values = torch.topk(z, top, dim=1).values - lse[:, None] if top else None
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    dz = None
    if case["train"]:
        a = s["dlogprob"].double() * keep
        b = s["dentropy"].double() * keep
        # d entropy / d z_v = -q_v (log q_v + entropy)
        dz = q * (-a - b * (entropy - lse))[:, None]
        dz -= q * z * b[:, None]
        dz[at, s["tokens"]] += a
    logprob[~keep], entropy[~keep] = 0.0, 0.0
    if values is not None:
        values[~keep] = 0.0
    return logprob, entropy, values, dz


def _exact_keep(case, s):
    """The kept elements again, with products taken in 16-bit halves and both multiplications side by side."""
    n = case["T"] * case["d"]
    c = torch.arange(-(-n // 8), dtype=torch.int64, device="cuda")
    even = torch.stack([c % 2 ** 32, torch.full_like(c, s["offset"] % 2 ** 32)])  # the words that are multiplied
    odd = torch.stack([c // 2 ** 32, torch.full_like(c, s["offset"] // 2 ** 32)])
    mult = [0xD2511F53, 0xCD9E8D57]
    weyl = [0x9E3779B9, 0xBB67AE85]
    for i in range(10):
        low, high = torch.empty_like(even), torch.empty_like(even)
        for j in range(2):
            lo = even[j] * (mult[j] % 65536)  # below 2^48
            hi = even[j] * (mult[j] // 65536) + lo // 65536  # below 2^49
            low[j] = (hi % 65536) * 65536 + lo % 65536
            high[j] = hi // 65536
        key = [(s["seed"] // 2 ** (32 * j) + i * weyl[j]) % 2 ** 32 for j in range(2)]
        even = torch.stack([high[1] ^ odd[0] ^ key[0], high[0] ^ odd[1] ^ key[1]])
        odd = torch.stack([low[1], low[0]])
    bits = torch.empty(c.shape[0], 8, dtype=torch.int64, device="cuda")
    for k, word in enumerate((even[0], odd[0], even[1], odd[1])):
        bits[:, 2 * k], bits[:, 2 * k + 1] = word % 65536, word // 65536
    return (bits.flatten()[:n] >= round(case["p"] * 65536)).view(case["T"], case["d"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        logprob, entropy, values, dz = _exact_rows(s["logits"].detach().double(), s, case, case["top"])
        if values is None:
            values = torch.zeros(case["T"], 0, dtype=torch.float64, device="cuda")
        return (logprob, entropy, None, values) + ((dz,) if case["train"] else ())
    if op == "head":
        H, W = s["H"].detach().double(), s["W"].detach().double()
        logprob, entropy, _, dz = _exact_rows(torch.matmul(H, W.t()), s, case, 0)
        return (logprob, entropy) + ((torch.matmul(dz, W), torch.matmul(dz.t(), H)) if case["train"] else ())
    if op == "dropout":
        factor = _exact_keep(case, s) * (1.0 / (1.0 - round(case["p"] * 65536) / 65536))
        return s["x"].detach().double() * factor, s["dy"].double() * factor
    x, res = s["x"].detach().double(), s["residual"].detach()
    factor = 1.0
    if case.get("p"):
        factor = _exact_keep(case, s) * (1.0 / (1.0 - round(case["p"] * 65536) / 65536))
    h = (res.double() + x * factor).to(res.dtype).double()
    inv = 1.0 / torch.sqrt(h.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS)
    n, w = h * inv, s["weight"].detach().double()
    y = n * w
    if op == "addnorm":
        dy = s["dy"].double()
        gw = dy * w
        total = s["dh"].double() + inv * (gw - n * ((gw * n).sum(dim=1, keepdim=True) / case["d"]))
        return y, h, total * factor, total, (dy * n).sum(dim=0)
    if case["form"] == "e4m3":
        scale = y.abs().max(dim=1, keepdim=True).values / 448.0
        v = y / scale
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3.0)
        return (v / step).round() * step * scale, h
    held = torch.empty_like(y)
    for c in range(0, case["d"], BLOCK):
        block = y[:, c:c + BLOCK]
        top = block.abs().max(dim=1, keepdim=True).values.clamp(min=1e-300)
        e = torch.floor(torch.log2(top / 127.5)) + 1.0  # smallest e with top < 127.5 * 2^e
        step = torch.exp2(e.clamp(min=-126.0))
        held[:, c:c + BLOCK] = torch.round(block / step) * step
    return held, h


# ------------------------------------------------------------------- work --
def work(case):
    T, e = case["T"], 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("logprobs", "head"):
        V, rows = case["V"], T * (0.75 if case["masked"] else 1.0)
        small = T * (8 + 8 + case.get("top", 0) * 8) + (T * 8 if case["train"] else 0)
        if op == "logprobs":
            # one exponential, three additions and products an element, and as much again for the gradient
            return {"bytes": rows * V * e + (T * V * e if case["train"] else 0) + small,
                    "flops": rows * V * (8 if case["train"] else 4)}
        d = case["d"]
        states = (T + V) * d * e
        return {"bytes": states * (2 if case["train"] else 1) + small,
                "flops": rows * V * (2 * d * (3 if case["train"] else 1) + 4)}
    d = case["d"]
    n = T * d
    if op == "dropout":
        return {"bytes": 4 * n * e, "flops": 4 * n}
    re = 2 if case["residual"] == "bf16" else 4
    if op == "quant":
        scales = T * (-(-d // BLOCK) if case["form"] == "int8" else 4)
        return {"bytes": n * (e + 2 * re + 1) + scales + d * e, "flops": 8 * n}
    # forward: read x and the residual, write h and y; backward: read dy, dh and h, write the residual's gradient and x's
    return {"bytes": n * (e + 2 * re + e) + n * (e + 3 * re + (e if case["p"] or e != re else 0)) + 2 * d * e,
            "flops": 20 * n}
