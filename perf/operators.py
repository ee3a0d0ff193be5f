"""The training operators around the sketched linear layers, as measured workloads.

Three operators and their gradients: layer norm (forward; backward with the
reduction of the weight's gradient), the softmax cross entropy of a linear head
over a large vocabulary (forward; backward), and an AdamW step over many
tensors (states in 32 bits; states in 8 bits).

``run`` computes each in plain 32-bit torch operations, or, where ``own`` is
true, through this package's entry points.  ``exact`` is the definition in 64
bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# AdamW: hyperparameters, the step (from 0) that the calls make, and the tags of
# the Philox streams that round weights, first moments and second moments.
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, SEED = 3e-4, 0.9, 0.999, 1e-8, 0.1, 99, 1234
TAG_W, TAG_M, TAG_U = 0, 3, 4
BLOCK = 256   # values of an 8-bit state that share a scale
ALIGN = 256   # each tensor starts at a multiple of this many values in the flat buffers


def listed():
    return [
        # one decoding-sized batch through a norm: a call's latency
        {"name": "norm_fwd_8x2048", "op": "norm_fwd", "T": 8, "k": 2048, "x": "bf16", "w": "fp32", "beta": True},
        # a whole step's tokens through a block's norm
        {"name": "norm_fwd_32768x4096", "op": "norm_fwd", "T": 32768, "k": 4096, "x": "bf16", "w": "fp32", "beta": True},
        # fp32 activations of an odd width, a ragged number of tokens
        {"name": "norm_bwd_1021x1001_fp32", "op": "norm_bwd", "T": 1021, "k": 1001, "x": "fp32", "w": "fp32", "beta": True},
        # a whole step's tokens back through a block's norm, BF16 weights
        {"name": "norm_bwd_32768x4096", "op": "norm_bwd", "T": 32768, "k": 4096, "x": "bf16", "w": "bf16", "beta": True},
        # scoring a few tokens: the head's weights are read once
        {"name": "ce_fwd_16x2048x32768", "op": "ce_fwd", "T": 16, "k": 2048, "V": 32768},
        # two microbatches' tokens over a large vocabulary
        {"name": "ce_fwd_8192x4096x131072", "op": "ce_fwd", "T": 8192, "k": 4096, "V": 131072},
        # a ragged batch over a vocabulary of odd size, gradients of both sides
        {"name": "ce_bwd_1000x2048x32771", "op": "ce_bwd", "T": 1000, "k": 2048, "V": 32771, "dw": True},
        # a microbatch's tokens, gradients of both sides
        {"name": "ce_bwd_4096x4096x65536", "op": "ce_bwd", "T": 4096, "k": 4096, "V": 65536, "dw": True},
        # the norm weights and biases of a 28-block stack: many small tensors
        {"name": "adam32_114x2048", "op": "adam", "states": 32, "tensors": 114, "total": 114 * 2048, "w": "bf16", "g": "fp32"},
        # an embedding table and a dense head
        {"name": "adam32_2x134M", "op": "adam", "states": 32, "tensors": 2, "total": 2 * 32768 * 4096, "w": "bf16", "g": "bf16"},
        # tensors of odd sizes, fp32 weights and gradients
        {"name": "adam8_37x1M_fp32", "op": "adam", "states": 8, "tensors": 37, "total": 1000003, "w": "fp32", "g": "fp32"},
        # the same table and head with small states
        {"name": "adam8_2x134M", "op": "adam", "states": 8, "tensors": 2, "total": 2 * 32768 * 4096, "w": "bf16", "g": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ce_fwd", "ce_bwd", "adam", "adam"])
    if op.startswith("norm"):
        k = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            k = max(64, k // 8 * 8)
        T = min(_log(rng, 1, 32768), 32768 * 4096 // k)
        return {"op": op, "T": T, "k": k, "x": rng.choice(["bf16", "bf16", "fp32"]), "w": rng.choice(["bf16", "fp32"]),
                "beta": rng.random() < 0.7}
    if op.startswith("ce"):
        most = 8192 * 4096 * 131072 if op == "ce_fwd" else 4096 * 4096 * 65536
        k = _log(rng, 64, 4096) // 8 * 8
        V = _log(rng, 1000, 131072 if op == "ce_fwd" else 65536)
        T = max(1, min(_log(rng, 1, 8192 if op == "ce_fwd" else 4096), most // (k * V)))
        case = {"op": op, "T": T, "k": k, "V": V}
        if op == "ce_bwd":
            case["dw"] = rng.random() < 0.7
        return case
    tensors = _log(rng, 1, 200)
    return {"op": "adam", "states": rng.choice([8, 32]), "tensors": tensors,
            "total": max(tensors, _log(rng, 1000, 200_000_000)), "w": rng.choice(["bf16", "fp32"]),
            "g": rng.choice(["bf16", "fp32"])}


def _normal(gen, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=gen, device=DEV) * std + mean


# ---- inputs -------------------------------------------------------------------

def _norm_inputs(case, gen):
    T, k = case["T"], case["k"]
    dx, dw = DTYPES[case["x"]], DTYPES[case["w"]]
    # activations of a residual stream: rows of unequal size with an offset
    size = torch.exp(_normal(gen, T, 1, std=0.5))
    s = {"X": (_normal(gen, T, k) * size + 0.1 * _normal(gen, T, 1)).to(dx),
         "gamma": _normal(gen, k, std=0.1, mean=1.0).to(dw),
         "beta": _normal(gen, k, std=0.1).to(dw) if case["beta"] else None}
    if case["op"] == "norm_bwd":
        s["dY"] = _normal(gen, T, k, std=1e-3).to(dx)
    return s


def _norm_stats(X):
    x = X.float()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _pieces(V, T):
    """Vocabulary ranges whose T x piece logits take a gigabyte at most in 32 bits."""
    step = max(1024, (1 << 28) // T)
    return [(v, min(V, v + step)) for v in range(0, V, step)]


def _ce_inputs(case, gen):
    T, k, V = case["T"], case["k"], case["V"]
    W = _normal(gen, V, k, std=0.02).to(torch.bfloat16)
    targets = torch.randint(0, V, (T,), generator=gen, device=DEV)
    # hidden states that lean towards their target, as a trained model's do: its logit is raised by up to 8
    lean = torch.rand(T, 1, generator=gen, device=DEV) * 8.0 / (k * 0.02 ** 2)
    X = (_normal(gen, T, k) + lean * W[targets].float()).to(torch.bfloat16)
    targets = torch.where(torch.rand(T, generator=gen, device=DEV) < 0.1, torch.full_like(targets, -100), targets)
    s = {"X": X, "W": W, "targets": targets, "scale": 0.9}
    if case["op"] == "ce_bwd":
        parts = [torch.logsumexp(s["scale"] * (X.float() @ W[a:b].float().t()), 1) for a, b in _pieces(V, T)]
        s["lse"] = torch.logsumexp(torch.stack(parts), 0)
        s["g"] = _normal(gen, T, std=0.5, mean=1.0) / T   # a token's weight in the loss: advantages over a batch
    return s


def _sizes(case):
    """Sizes of the tensors: `total` values spread unevenly, each at least one."""
    n, total = case["tensors"], case["total"]
    if total % n == 0 and total // n % ALIGN == 0:
        return [total // n] * n
    weight = [1.0 + (7 * i) % 11 for i in range(n)]
    sizes = [max(1, int(total * w / sum(weight))) for w in weight]
    sizes[0] = max(1, sizes[0] + total - sum(sizes))
    return sizes


def _adam_inputs(case, gen):
    sizes = _sizes(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + ALIGN - 1) // ALIGN * ALIGN
    held = torch.zeros(at, dtype=torch.bool, device=DEV)
    for a, n in zip(starts, sizes):
        held[a:a + n] = True
    # per-value gradient sizes over three orders of magnitude, as in a trained model
    size = torch.exp(_normal(gen, at, std=1.5) - 8.0)
    s = {"sizes": sizes, "starts": starts,
         "w": torch.where(held, _normal(gen, at, std=0.02), 0.0).to(DTYPES[case["w"]]),
         "g": torch.where(held, _normal(gen, at) * size, 0.0).to(DTYPES[case["g"]])}
    m = torch.where(held, 0.3 * _normal(gen, at) * size, 0.0)
    u = torch.where(held, size * torch.exp(_normal(gen, at, std=0.2)), 0.0)
    del size, held
    if case["states"] == 32:
        s["m"], s["v"] = m, u.square()
    else:
        s["m"], s["m_scale"] = _quantize(m)
        s["u"], s["u_scale"] = _quantize(u)
    return s


def _quantize(x):
    """Values as 8-bit floats times a scale for each block, to nearest: where the inputs' states come from."""
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1) / 448.0
    q = (b / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-448.0, 448.0)
    return q.view(-1).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"norm": _norm_inputs, "ce": _ce_inputs, "adam": _adam_inputs}[op.split("_")[0]](case, gen)
    s["case"] = case
    if own:
        _buffers(s, case)
    return s


def _buffers(s, case):
    """The output buffers, and for AdamW the optimizer object, that a program keeps from step to step."""
    import rank_gradient_sketching_philox_gb300 as rgs
    op = case["op"]
    if op.startswith("norm"):
        T, k = case["T"], case["k"]
        s["Y"] = torch.empty_like(s["X"])
        if op == "norm_fwd":
            s["mean"], s["rstd"] = (torch.empty(T, device=DEV) for _ in range(2))
        else:
            s["mean"], s["rstd"] = _norm_stats(s["X"])
            s["dgamma"] = torch.empty(k, device=DEV)
            s["dbeta"] = torch.empty(k, device=DEV) if case["beta"] else None
    elif op == "ce_fwd":
        s["loss"], s["lse"] = (torch.empty(case["T"], device=DEV) for _ in range(2))
    elif op == "ce_bwd":
        s["dX"] = torch.empty_like(s["X"])
        s["dW"] = torch.empty_like(s["W"]) if case["dw"] else None
    else:
        def parts(name, per=1):
            return [s[name][a // per:a // per + -(-n // per)] for a, n in zip(s["starts"], s["sizes"])]
        if case["states"] == 32:
            state = {"m": parts("m"), "v": parts("v")}
        else:
            state = {"m": parts("m"), "u": parts("u"), "m_scale": parts("m_scale", BLOCK), "u_scale": parts("u_scale", BLOCK)}
        s["opt"] = rgs.AdamW(parts("w"), parts("g"), state_bits=case["states"], state=state, betas=(BETA1, BETA2),
                             eps=ADAM_EPS, weight_decay=DECAY, seed=SEED)


# ---- the plain forms ------------------------------------------------------------

def _norm_fwd(s):
    x = s["X"].float()
    mean, rstd = _norm_stats(x)
    y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    return {"y": y.to(s["X"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(s):
    x, dy = s["X"].float(), s["dY"].float()
    mean, rstd = _norm_stats(x)
    xh = (x - mean[:, None]) * rstd[:, None]
    dxh = dy * s["gamma"].float()
    dx = rstd[:, None] * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
    out = {"dx": dx.to(s["X"].dtype), "dgamma": (dy * xh).sum(0)}
    if s["beta"] is not None:
        out["dbeta"] = dy.sum(0)
    return out


def _ce_fwd(s):
    logits = s["X"].float() @ s["W"].float().t()
    logits *= s["scale"]
    top = logits.amax(1)
    kept = s["targets"] >= 0
    hit = logits[torch.arange(len(top), device=DEV), s["targets"].clamp(min=0)]
    logits -= top[:, None]
    lse = top + torch.log(logits.exp_().sum(1))
    return {"loss": torch.where(kept, lse - hit, 0.0), "lse": lse}


def _ce_bwd(s):
    x, w = s["X"].float(), s["W"].float()
    d = x @ w.t()
    d *= s["scale"]
    d -= s["lse"][:, None]
    d.exp_()
    d[torch.arange(len(x), device=DEV), s["targets"].clamp(min=0)] -= 1.0
    d *= torch.where(s["targets"] >= 0, s["g"] * s["scale"], 0.0)[:, None]
    out = {"dx": (d @ w).to(torch.bfloat16)}
    if s["case"]["dw"]:
        out["dw"] = (d.t() @ x).to(torch.bfloat16)
    return out


def _mul_wide(a, b):
    """High and low 32 bits of a * b, for int64 tensors a below 2^32 and a number b below 2^32."""
    low = (a & 0xFFFF) * b
    high = (a >> 16) * b + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _random16(s, tag):
    """16 random bits for each value: value e of tensor `layer` takes 16-bit lane e % 8 of the tensor's
    Philox4x32-10 block e // 8."""
    at = torch.arange(len(s["w"]) // 8, dtype=torch.int64, device=DEV)
    first = torch.tensor(s["starts"], dtype=torch.int64, device=DEV) // 8
    layer = torch.searchsorted(first, at, right=True) - 1
    c0, c1, c2, c3 = at - first[layer], torch.full_like(at, STEP), layer, torch.full_like(at, tag)
    k0, k1 = SEED & 0xFFFFFFFF, SEED >> 32
    for _ in range(10):
        (h0, l0), (h1, l1) = _mul_wide(c0, 0xD2511F53), _mul_wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1).to(torch.int32)


def _round_bf16(x, r):
    """x to BF16, up with the probability of the dropped bits: 16 random bits are added below the kept ones."""
    return (((x.view(torch.int32) + r) >> 16) << 16).view(torch.float32).to(torch.bfloat16)


def _round_e4m3(y, r):
    """y in [0, 448] to E4M3 the same way; below 2^-6 its steps are 2^-9, as those of y + 2^-6 are."""
    small = y < 2.0 ** -6
    bits = torch.where(small, y + 2.0 ** -6, y).view(torch.int32)
    return ((bits + (r << 4)) >> 20) - torch.where(small, 968, 960)


def _hold8(x, random, q, scale, least):
    """Put x into the 8-bit values q and their blocks' scales; what is not zero gets a code of `least` at least."""
    top = x.abs().view(-1, BLOCK).amax(1)
    scale.copy_(top / 448.0)
    inv = torch.where(top > 0, 448.0 / top, 0.0).repeat_interleave(BLOCK)
    code = _round_e4m3((x.abs() * inv).clamp(max=448.0), random)
    code = torch.where(x != 0, code.clamp(min=least), code)
    q.view(torch.uint8).copy_(torch.where(x < 0, code | 0x80, code))


def _adam(s):
    c1 = LR / (1.0 - BETA1 ** (STEP + 1))
    c2 = 1.0 / math.sqrt(1.0 - BETA2 ** (STEP + 1))
    eight = "u" in s
    w, g, m = s["w"], s["g"].float(), s["m"].float()
    if eight:
        m = m * s["m_scale"].repeat_interleave(BLOCK)
        v = (s["u"].float() * s["u_scale"].repeat_interleave(BLOCK)).square()
    else:
        v = s["v"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    u = torch.sqrt(v)
    new = w.float() * (1.0 - LR * DECAY) - c1 * m / (u * c2 + ADAM_EPS)
    w.copy_(_round_bf16(new, _random16(s, TAG_W)) if w.dtype == torch.bfloat16 else new)
    if eight:
        _hold8(m, _random16(s, TAG_M), s["m"], s["m_scale"], 0)
        _hold8(u, _random16(s, TAG_U), s["u"], s["u_scale"], 1)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adam_out(s)


def _adam_out(s):
    return {name: s[name] for name in ("w", "m", "v", "u", "m_scale", "u_scale") if name in s}


PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd, "adam": _adam}


# ---- the framework's calls -------------------------------------------------------

def _run_own(s):
    import rank_gradient_sketching_philox_gb300 as rgs
    op = s["case"]["op"]
    if op == "norm_fwd":
        rgs.layer_norm_forward(s["X"], s["gamma"], s["beta"], s["Y"], s["mean"], s["rstd"], eps=EPS)
        return {"y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        rgs.layer_norm_backward(s["dY"], s["X"], s["gamma"], s["mean"], s["rstd"], s["Y"], s["dgamma"], s["dbeta"],
                                overwrite=True)
        out = {"dx": s["Y"], "dgamma": s["dgamma"]}
        if s["dbeta"] is not None:
            out["dbeta"] = s["dbeta"]
        return out
    if op == "ce_fwd":
        rgs.cross_entropy_forward(s["X"], s["W"], s["targets"], s["loss"], s["lse"], scale=s["scale"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "ce_bwd":
        rgs.cross_entropy_backward(s["X"], s["W"], s["targets"], s["lse"], s["g"], dX=s["dX"], dW=s["dW"],
                                   overwrite=True, scale=s["scale"])
        out = {"dx": s["dX"]}
        if s["dW"] is not None:
            out["dw"] = s["dW"]
        return out
    s["opt"].step(lr=LR, step=STEP)
    return _adam_out(s)


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op.startswith("norm"):
        T, k, e, w = case["T"], case["k"], size[case["x"]], size[case["w"]]
        if op == "norm_fwd":
            return {"bytes": 2 * T * k * e + 8 * T + k * w * (2 if case["beta"] else 1), "flops": 8 * T * k}
        return {"bytes": 3 * T * k * e + 8 * T + k * w + 4 * k * (2 if case["beta"] else 1), "flops": 14 * T * k}
    if op.startswith("ce"):
        T, k, V = case["T"], case["k"], case["V"]
        if op == "ce_fwd":
            return {"bytes": 2 * k * (T + V) + 16 * T, "flops": 2 * T * k * V}
        out = T + V if case["dw"] else T
        return {"bytes": 2 * k * (T + V) + 2 * k * out + 16 * T, "flops": (6 if case["dw"] else 4) * T * k * V}
    n = case["total"]
    state = 16 if case["states"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * size[case["w"]] + size[case["g"]] + state), "flops": 16 * n}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    global own
    keep, own = own, False
    s = prepare(case, seed)
    own = keep
    return {"norm_fwd": _norm_fwd64, "norm_bwd": _norm_bwd64, "ce_fwd": _ce_fwd64, "ce_bwd": _ce_bwd64,
            "adam": _adam64}[case["op"]](s)


def _standard64(X):
    x = X.double()
    k = x.shape[1]
    mean = x.sum(1) / k
    x.sub_(mean[:, None])
    rstd = ((x * x).sum(1) / k + EPS).pow(-0.5)
    return x.mul_(rstd[:, None]), mean, rstd


def _norm_fwd64(s):
    xh, mean, rstd = _standard64(s["X"])
    xh.mul_(s["gamma"].double())
    if s["beta"] is not None:
        xh.add_(s["beta"].double())
    return {"y": xh, "mean": mean, "rstd": rstd}


def _norm_bwd64(s):
    xh, _, rstd = _standard64(s["X"])
    dy = s["dY"].double()
    out = {"dgamma": torch.einsum("tk,tk->k", dy, xh)}
    if s["beta"] is not None:
        out["dbeta"] = dy.sum(0)
    k = xh.shape[1]
    dy.mul_(s["gamma"].double())
    a = torch.einsum("tk->t", dy) / k
    b = torch.einsum("tk,tk->t", dy, xh) / k
    out["dx"] = dy.sub_(a[:, None]).sub_(xh.mul_(b[:, None])).mul_(rstd[:, None])
    return out


def _ce_logits64(s, a, b):
    return (s["X"].double() @ s["W"][a:b].double().t()).mul_(s["scale"])


def _ce_fwd64(s):
    T, V = len(s["X"]), len(s["W"])
    total = torch.full((T,), -math.inf, dtype=torch.float64, device=DEV)
    hit = torch.zeros(T, dtype=torch.float64, device=DEV)
    for a, b in _pieces(V, T):
        logits = _ce_logits64(s, a, b)
        total = torch.logaddexp(total, torch.logsumexp(logits, 1))
        here = ((s["targets"] >= a) & (s["targets"] < b)).nonzero()[:, 0]
        hit[here] = logits[here, s["targets"][here] - a]
    return {"loss": (total - hit).masked_fill(s["targets"] < 0, 0.0), "lse": total}


def _ce_bwd64(s):
    T, V = len(s["X"]), len(s["W"])
    x = s["X"].double()
    weight = (s["g"].double() * s["scale"]).masked_fill(s["targets"] < 0, 0.0)
    dx, dw = torch.zeros_like(x), []
    for a, b in _pieces(V, T):
        d = torch.exp(_ce_logits64(s, a, b).sub_(s["lse"].double()[:, None]))
        here = ((s["targets"] >= a) & (s["targets"] < b)).nonzero()[:, 0]
        d[here, s["targets"][here] - a] -= 1.0
        d.mul_(weight[:, None])
        dx.addmm_(d, s["W"][a:b].double())
        if s["case"]["dw"]:
            dw.append(d.t() @ x)
    out = {"dx": dx}
    if dw:
        out["dw"] = torch.cat(dw)
    return out


def _adam64(s):
    """The updated weights and states before any rounding; 8-bit values in units of their blocks' scales."""
    out = {name: t.double() for name, t in _adam_out(s).items()}
    t = STEP + 1
    wide = lambda scale: scale.double().view(-1, 1).expand(-1, BLOCK).reshape(-1)  # noqa: E731
    g = s["g"].double()
    eight = "u" in s
    m = out["m"] * wide(s["m_scale"]) if eight else out["m"]
    v = (out["u"] * wide(s["u_scale"])) ** 2 if eight else out["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g ** 2 * (1 - BETA2)
    step = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    out["w"] = out["w"] - LR * (step + DECAY * out["w"])
    if not eight:
        out["m"], out["v"] = m, v
        return out
    for name, x in (("m", m), ("u", v.sqrt())):
        scale = x.abs().view(-1, BLOCK).amax(1) / 448.0
        out[name] = x / wide(torch.where(scale > 0, scale, 1.0))
        out[name + "_scale"] = scale
    return out
