"""The 8-bit forward path of the sketched linear layers, and gradient clipping, as measured workloads.

Four operators: the root-mean-square norm of a residual stream (forward with the
residual's addition and an output in 8 bits; backward), the rounding of a matrix
to 8 bits with a scale for each block of 128, the matrix product of two such
matrices (a layer's output, or its input's gradient), and the global norm of many
gradients with their clipping.

``run`` computes each in plain 32-bit torch operations, or, where ``own`` is
true, through this package's entry points.  ``exact`` is the definition in 64
bits.  8-bit values are E4M3: a value is its code times its block's scale, the
block's largest magnitude over 448.  Codes are returned as the numbers that they
are, in units of the scales beside them.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 128        # values, or rows and columns of a weight, that share a scale
TOP = 448.0        # the largest E4M3 value
LEAST = 2.0 ** -126  # the smallest scale
MAX_NORM = 1.0
ALIGN = 256        # each gradient starts at a multiple of this many values in the flat buffer
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
MOST_PRODUCT = 8192 * 12288 * 4096


def listed():
    return [
        # a decoding batch through a block's norm: a call's latency
        {"name": "rms_fwd_8x2048", "op": "rms_fwd", "T": 8, "k": 2048, "x": "bf16", "w": "bf16", "res": True, "y": True, "q": False},
        # a step's tokens through a block's norm: BF16 for the projected inputs, 8 bits for the layers' products
        {"name": "rms_fwd_32768x4096_q", "op": "rms_fwd", "T": 32768, "k": 4096, "x": "bf16", "w": "bf16", "res": True, "y": True, "q": True},
        # fp32 activations of an odd width, a ragged number of tokens
        {"name": "rms_bwd_1021x1001_fp32", "op": "rms_bwd", "T": 1021, "k": 1001, "x": "fp32", "w": "fp32", "res": True},
        # a step's tokens back through a block's norm, joining the residual's gradient
        {"name": "rms_bwd_32768x4096", "op": "rms_bwd", "T": 32768, "k": 4096, "x": "bf16", "w": "bf16", "res": True},
        # one layer's weights after their update, for the product and its gradient
        {"name": "quant_w_6144x2048", "op": "quant", "T": 6144, "k": 2048, "x": "bf16", "rows": 128, "t": True},
        # a microbatch's output derivatives of the widest layer
        {"name": "quant_d_4096x12288", "op": "quant", "T": 4096, "k": 12288, "x": "bf16", "rows": 1, "t": False},
        # a decoding batch through a square layer: its weights are read once
        {"name": "mm8_16x4096x4096", "op": "mm8", "T": 16, "N": 4096, "k": 4096, "out": "bf16"},
        # a short prompt through a layer of odd sizes, fp32 output
        {"name": "mm8_301x1027x2100_fp32", "op": "mm8", "T": 301, "N": 1027, "k": 2100, "out": "fp32"},
        # a microbatch's derivatives back through the widest layer
        {"name": "mm8_4096x4096x12288", "op": "mm8", "T": 4096, "N": 4096, "k": 12288, "out": "bf16"},
        # two microbatches through the widest layer
        {"name": "mm8_8192x12288x4096", "op": "mm8", "T": 8192, "N": 12288, "k": 4096, "out": "bf16"},
        # the norm weights of a stack: many small gradients, their norm and the scale that AdamW takes
        {"name": "gnorm_114x2048", "op": "gnorm", "tensors": 114, "total": 114 * 2048, "g": "fp32", "clip": False},
        # an embedding table's and a dense head's gradients, clipped
        {"name": "gclip_2x134M", "op": "gnorm", "tensors": 2, "total": 2 * 32768 * 4096, "g": "bf16", "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width, most often a multiple of 8."""
    k = _log(rng, lo, hi)
    return max(lo, k // 8 * 8) if rng.random() < 0.7 else k


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "quant", "mm8", "mm8", "gnorm"])
    x = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("rms"):
        k = _width(rng, 64, 16384)
        case = {"op": op, "T": min(_log(rng, 1, 32768), 32768 * 2048 // k), "k": k, "x": x,
                "w": rng.choice(["bf16", "fp32"]), "res": rng.random() < 0.7}
        if op == "rms_fwd":
            case["q"] = rng.random() < 0.6
            case["y"] = not case["q"] or rng.random() < 0.5
        return case
    if op == "quant":
        k = _width(rng, 64, 16384)
        rows = rng.choice([1, 128])
        return {"op": op, "T": min(_log(rng, 1, 16384), 32768 * 2048 // k), "k": k, "x": x, "rows": rows,
                "t": rows == 128 and rng.random() < 0.5}
    if op == "mm8":
        k, N = _width(rng, 64, 16384), _width(rng, 64, 16384)
        return {"op": op, "T": max(1, min(_log(rng, 1, 16384), MOST_PRODUCT // 2 // (k * N))), "N": N, "k": k,
                "out": rng.choice(["bf16", "bf16", "fp32"])}
    tensors = _log(rng, 1, 200)
    return {"op": "gnorm", "tensors": tensors, "total": max(tensors, _log(rng, 1000, 200_000_000)),
            "g": rng.choice(["bf16", "fp32"]), "clip": rng.random() < 0.5}


def _normal(gen, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=gen, device=DEV) * std + mean


def _up(n, m):
    return (n + m - 1) // m * m


def _rows_of(T, k, dtype, multiple):
    """An uninitialised T x k matrix whose rows start `multiple` values apart, as the products want them."""
    return torch.empty(T, _up(k, multiple), dtype=dtype, device=DEV)[:, :k]


# ---- inputs -------------------------------------------------------------------

def _stream(gen, T, k):
    """A residual stream: rows of unequal size, a few channels much larger than the others."""
    size = torch.exp(_normal(gen, T, 1, std=0.5))
    channel = torch.where(torch.rand(k, generator=gen, device=DEV) < 0.01, 20.0, 1.0)
    return _normal(gen, T, k) * size * channel


def _rms_inputs(case, gen):
    T, k = case["T"], case["k"]
    dx, dw = DTYPES[case["x"]], DTYPES[case["w"]]
    s = {"X": _stream(gen, T, k).to(dx), "gamma": _normal(gen, k, std=0.1, mean=1.0).to(dw)}
    if case["op"] == "rms_fwd":
        s["R"] = _normal(gen, T, k, std=0.5).to(dx) if case["res"] else None   # a block's output
    else:
        s["dY"] = _normal(gen, T, k, std=1e-3).to(dx)
        s["dS"] = _normal(gen, T, k, std=1e-3).to(dx) if case["res"] else None   # the stream's gradient from above
        s["rstd"] = 1.0 / torch.sqrt(s["X"].float().square().mean(1) + EPS)
    return s


def _quant_inputs(case, gen):
    T, k = case["T"], case["k"]
    if case["rows"] == 1:   # output derivatives: a few tokens with large ones
        heavy = torch.where(torch.rand(T, 1, generator=gen, device=DEV) < 0.05, 10.0, 1.0)
        x = _normal(gen, T, k, std=1e-3) * heavy
    else:
        x = _normal(gen, T, k, std=0.02)
    return {"X": x.to(DTYPES[case["x"]])}


def _mm8_inputs(case, gen):
    T, N, k = case["T"], case["N"], case["k"]
    a, sa = _quantize(_stream(gen, T, k), 1)
    b, sb = _quantize(_normal(gen, N, k, std=0.02), BLOCK)
    s = {"A": _rows_of(T, k, torch.float8_e4m3fn, 16), "a_scale": sa, "B": _rows_of(N, k, torch.float8_e4m3fn, 16),
         "b_scale": sb}
    s["A"].copy_(a)
    s["B"].copy_(b)
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


def _gnorm_inputs(case, gen):
    sizes = _sizes(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += _up(n, ALIGN)
    # per-value sizes over three orders of magnitude, as in a trained model
    flat = (_normal(gen, at) * torch.exp(_normal(gen, at, std=1.5) - 8.0)).to(DTYPES[case["g"]])
    for a, n in zip(starts, sizes):
        flat[a + n:a + _up(n, ALIGN)] = 0.0
    return {"flat": flat, "starts": starts, "sizes": sizes}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"rms": _rms_inputs, "quant": _quant_inputs, "mm8": _mm8_inputs,
         "gnorm": _gnorm_inputs}[case["op"].split("_")[0]](case, gen)
    s["case"] = case
    if own:
        _buffers(s, case)
    return s


def _buffers(s, case):
    """The output buffers, and for the norm of the gradients the table of them, that a program keeps from step to step."""
    import rank_gradient_sketching_philox_gb300 as rgs
    op, f32, f8 = case["op"], torch.float32, torch.float8_e4m3fn
    if op == "gnorm":
        def parts(flat):
            return [flat[a:a + n] for a, n in zip(s["starts"], s["sizes"])]
        s["out"] = torch.zeros_like(s["flat"]) if case["clip"] else None
        s["clip"] = rgs.GradClip(parts(s["flat"]), MAX_NORM, outs=parts(s["out"]) if case["clip"] else None)
        return
    T, k = case["T"], case["k"]
    if op == "mm8":
        s["Y"] = _rows_of(T, case["N"], DTYPES[case["out"]], 8)
        return
    if op == "rms_bwd":
        s["dX"], s["dgamma"] = torch.empty_like(s["X"]), torch.empty(k, device=DEV)
        return
    groups = (k + BLOCK - 1) // BLOCK
    if op == "rms_fwd":
        s["S"] = torch.empty_like(s["X"]) if case["res"] else None
        s["Y"] = torch.empty_like(s["X"]) if case["y"] else None
        s["rstd"] = torch.empty(T, dtype=f32, device=DEV)
        s["Q"] = _rows_of(T, k, f8, 16) if case["q"] else None
        s["scale"] = torch.empty(T, groups, dtype=f32, device=DEV) if case["q"] else None
    else:
        s["Q"] = _rows_of(T, k, f8, 16)
        s["scale"] = torch.empty((T + case["rows"] - 1) // case["rows"], groups, dtype=f32, device=DEV)
        s["Qt"] = _rows_of(k, T, f8, 16) if case["t"] else None


# ---- the plain forms ------------------------------------------------------------

def _blocks(x, rows):
    """x with zeros behind its last row and column, as (row blocks, rows, column blocks, 128)."""
    T, k = x.shape
    full = torch.zeros(_up(T, rows), _up(k, BLOCK), dtype=x.dtype, device=x.device)
    full[:T, :k] = x
    return full.view(-1, rows, _up(k, BLOCK) // BLOCK, BLOCK)


def _quantize(x, rows):
    """(codes, scales) of an fp32 matrix: each block of `rows` rows and 128 columns in units of its largest magnitude over 448."""
    b = _blocks(x, rows)
    scale = (b.abs().amax((1, 3)) / TOP).clamp(min=LEAST)
    code = (b / scale[:, None, :, None]).clamp(-TOP, TOP).view(-1, b.shape[2] * BLOCK)
    return code[:x.shape[0], :x.shape[1]].to(torch.float8_e4m3fn), scale


def _rms_fwd(s):
    case = s["case"]
    x = s["X"].float()
    if s["R"] is not None:
        x = x + s["R"].float()
    rstd = 1.0 / torch.sqrt(x.square().mean(1) + EPS)
    y = x * rstd[:, None] * s["gamma"].float()
    out = {"rstd": rstd}
    if s["R"] is not None:
        out["s"] = x.to(s["X"].dtype)
    if case["y"]:
        out["y"] = y.to(s["X"].dtype)
    if case["q"]:
        out["q"], out["scale"] = _quantize(y, 1)
    return out


def _rms_bwd(s):
    xh, dy = s["X"].float() * s["rstd"][:, None], s["dY"].float()
    dxh = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (dxh - xh * (dxh * xh).mean(1, keepdim=True))
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    return {"dx": dx.to(s["X"].dtype), "dgamma": (dy * xh).sum(0)}


def _quant(s):
    q, scale = _quantize(s["X"].float(), s["case"]["rows"])
    out = {"q": q, "scale": scale}
    if s["case"]["t"]:
        out["qt"] = q.t().contiguous()
    return out


def _values(q, scale, rows, dtype):
    """The numbers that codes and their blocks' scales stand for."""
    wide = scale.to(dtype).repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return wide.mul_(q.to(dtype))


def _mm8(s):
    a, b = _values(s["A"], s["a_scale"], 1, torch.float32), _values(s["B"], s["b_scale"], BLOCK, torch.float32)
    return {"y": (a @ b.t()).to(DTYPES[s["case"]["out"]])}


def _gnorm(s):
    parts = s["flat"].view(-1, ALIGN).float()   # a long sum: parts in 32 bits, their sum in 64
    norm = parts.square().sum(1).double().sum(0, keepdim=True).sqrt()
    scale = torch.where(norm <= MAX_NORM, 1.0, MAX_NORM / norm).float()
    out = {"norm": norm.float(), "scale": scale}
    if s["case"]["clip"]:
        out["g"] = (parts * scale).view(-1).to(s["flat"].dtype)
    return out


PLAIN = {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "quant": _quant, "mm8": _mm8, "gnorm": _gnorm}


# ---- the framework's calls -------------------------------------------------------

def _run_own(s):
    import rank_gradient_sketching_philox_gb300 as rgs
    case = s["case"]
    op = case["op"]
    if op == "rms_fwd":
        rgs.rms_norm_forward(s["X"], s["gamma"], s["rstd"], R=s["R"], S=s["S"], Y=s["Y"], Q=s["Q"], scale=s["scale"], eps=EPS)
        out = {"rstd": s["rstd"]}
        if s["S"] is not None:
            out["s"] = s["S"]
        if s["Y"] is not None:
            out["y"] = s["Y"]
        if s["Q"] is not None:
            out["q"], out["scale"] = s["Q"], s["scale"]
        return out
    if op == "rms_bwd":
        rgs.rms_norm_backward(s["dY"], s["X"], s["gamma"], s["rstd"], dS=s["dS"], dX=s["dX"], dgamma=s["dgamma"], overwrite=True)
        return {"dx": s["dX"], "dgamma": s["dgamma"]}
    if op == "quant":
        rgs.quantize_blocks(s["X"], s["Q"], s["scale"], rows=case["rows"], Qt=s["Qt"])
        out = {"q": s["Q"], "scale": s["scale"]}
        if s["Qt"] is not None:
            out["qt"] = s["Qt"]
        return out
    if op == "mm8":
        rgs.matmul_blocks(s["A"], s["a_scale"], s["B"], s["b_scale"], s["Y"])
        return {"y": s["Y"]}
    s["clip"].step()
    out = {"norm": s["clip"].norm, "scale": s["clip"].scale}
    if s["out"] is not None:
        out["g"] = s["out"]
    return out


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "gnorm":
        n, e = case["total"], size[case["g"]]
        return {"bytes": n * e * (2 if case["clip"] else 1), "flops": n * (3 if case["clip"] else 2)}
    T, k = case["T"], case["k"]
    groups = (k + BLOCK - 1) // BLOCK
    if op == "mm8":
        N = case["N"]
        return {"bytes": T * k + N * k + T * N * size[case["out"]] + 4 * groups * (T + (N + BLOCK - 1) // BLOCK),
                "flops": 2 * T * N * k}
    e = size[case["x"]]
    if op == "rms_fwd":
        moved = e * (1 + 2 * case["res"] + case["y"]) + case["q"]
        return {"bytes": T * k * moved + 4 * T + 4 * T * groups * case["q"] + k * size[case["w"]], "flops": 6 * T * k}
    if op == "rms_bwd":
        return {"bytes": T * k * e * (3 + case["res"]) + 4 * T + k * (size[case["w"]] + 4), "flops": 11 * T * k}
    return {"bytes": T * k * (e + 1 + case["t"]) + 4 * groups * ((T + case["rows"] - 1) // case["rows"]), "flops": 3 * T * k}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    global own
    keep, own = own, False
    s = prepare(case, seed)
    own = keep
    return {"rms_fwd": _rms_fwd64, "rms_bwd": _rms_bwd64, "quant": _quant64, "mm8": _mm8_64, "gnorm": _gnorm64}[case["op"]](s)


def _codes64(y, rows):
    """Values in units of their blocks' scales before any rounding, and the scales."""
    T, k = y.shape
    q = torch.empty_like(y)
    scale = torch.empty((T + rows - 1) // rows, (k + BLOCK - 1) // BLOCK, dtype=torch.float64, device=DEV)
    for c in range(scale.shape[1]):
        part = y[:, c * BLOCK:(c + 1) * BLOCK]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.stack([t.amax() for t in top.split(rows)])
        scale[:, c] = (top / TOP).clamp(min=LEAST)
        q[:, c * BLOCK:(c + 1) * BLOCK] = part / scale[:, c].repeat_interleave(rows)[:T, None]
    return q, scale


def _rms_fwd64(s):
    x = s["X"].double()
    if s["R"] is not None:
        x = x + s["R"].double()
    rstd = (torch.einsum("tk,tk->t", x, x) / x.shape[1] + EPS).pow(-0.5)
    out = {"rstd": rstd}
    if s["R"] is not None:
        out["s"] = x.clone()
    y = x.mul_(rstd[:, None]).mul_(s["gamma"].double())
    if s["case"]["y"]:
        out["y"] = y
    if s["case"]["q"]:
        out["q"], out["scale"] = _codes64(y, 1)
    return out


def _rms_bwd64(s):
    rstd = s["rstd"].double()[:, None]
    xh = s["X"].double().mul_(rstd)
    dy = s["dY"].double()
    out = {"dgamma": torch.einsum("tk,tk->k", dy, xh)}
    dy.mul_(s["gamma"].double())
    c = torch.einsum("tk,tk->t", dy, xh) / xh.shape[1]
    dx = dy.sub_(xh.mul_(c[:, None])).mul_(rstd)
    if s["dS"] is not None:
        dx.add_(s["dS"].double())
    out["dx"] = dx
    return out


def _quant64(s):
    q, scale = _codes64(s["X"].double(), s["case"]["rows"])
    out = {"q": q, "scale": scale}
    if s["case"]["t"]:
        out["qt"] = q.t().contiguous()
    return out


def _mm8_64(s):
    T, N = s["A"].shape[0], s["B"].shape[0]
    y = torch.zeros(T, N, dtype=torch.float64, device=DEV)
    for c in range(s["a_scale"].shape[1]):
        cols = slice(c * BLOCK, (c + 1) * BLOCK)
        a = s["A"][:, cols].double() * s["a_scale"][:, c, None].double()
        b = s["B"][:, cols].double() * s["b_scale"][:, c].double().repeat_interleave(BLOCK)[:N, None]
        y.addmm_(a, b.t())
    return {"y": y}


def _gnorm64(s):
    norm = torch.linalg.vector_norm(s["flat"], dtype=torch.float64).view(1)
    scale = (MAX_NORM / norm).clamp(max=1.0)
    out = {"norm": norm, "scale": scale}
    if s["case"]["clip"]:
        out["g"] = s["flat"].double() * scale
    return out
