"""Measured cases of the operators around 8-bit floating point matrices and
their training: the norm with the residual's addition (rms_norm, rms_train with
its gradient), the activations' codes with a scale per block of 128 (quant_fp8),
the product with a matrix of such codes (gemm_fp8), and the global norm of the
gradients with their clipping (clip_grads).

With `own` false, run() computes an operator from elementary torch operations
in 32 bits, rounded once at the end; with `own` true it makes the library's
calls.  Either way one run() is one pass as a program makes it, on inputs that
prepare() draws from the seed.
"""
import math

import torch

own = False

BLOCK = 128                 # columns (and rows of a matrix) that share a scale
CODE_MAX = 448.0            # the largest finite e4m3 value
SMALLEST_MAX = 2.0 ** -100  # a block's largest value counts as at least this
EPS = 1e-5
F8 = torch.float8_e4m3fn


def listed():
    return [
        # the smallest projection of an 8B-shape block, one token: launch and latency bound
        dict(name="gemm_fp8 k_proj 1 token", op="gemm_fp8", rows=1024, cols=4096, tokens=1, out="bf16"),
        # its widest projection for a small batch of sequences: bound by reading the matrix
        dict(name="gemm_fp8 gate_proj 16 tokens", op="gemm_fp8", rows=14336, cols=4096, tokens=16, out="bf16"),
        # odd sizes: rows and tokens not in tiles, a short last block, results kept in 32 bits
        dict(name="gemm_fp8 odd 333 tokens", op="gemm_fp8", rows=1003, cols=2096, tokens=333, out="f32"),
        # a 70B-shape block's gate projection over a long prefill: bound by the matrix cores
        dict(name="gemm_fp8 70B prefill", op="gemm_fp8", rows=28672, cols=8192, tokens=8192, out="bf16"),
        # before a projection, one token: launch and latency bound
        dict(name="rms_norm 1 token fp8", op="rms_norm", tokens=1, dim=4096, residual=True, out="fp8"),
        # a 70B-shape model's prefill
        dict(name="rms_norm prefill fp8", op="rms_norm", tokens=8192, dim=8192, residual=True, out="fp8"),
        # a small model's training step, every size odd
        dict(name="rms_train odd", op="rms_train", tokens=515, dim=1160, residual=True),
        # a large batch's
        dict(name="rms_train batch", op="rms_train", tokens=16384, dim=4096, residual=True),
        # attention's output before its projection, a few tokens, a short last block
        dict(name="quant_fp8 odd 37 tokens", op="quant_fp8", tokens=37, dim=1168, gated=False),
        # the gated activation before a 70B-shape down projection, a long prefill
        dict(name="quant_fp8 70B gated prefill", op="quant_fp8", tokens=8192, dim=28672, gated=True),
        # a tiny model's gradients in 32 bits, odd sizes: launch and latency bound
        dict(name="clip_grads small odd", op="clip_grads", layers=2, dim=131, kv=35, ffn=347, kind="f32",
             max_norm=1.0),
        # four 8B-shape blocks' gradients
        dict(name="clip_grads 8B blocks", op="clip_grads", layers=4, dim=4096, kv=1024, ffn=14336, kind="bf16",
             max_norm=1.0),
    ]


def _size(rng, lo, hi, mult=1):
    """A whole number from lo to hi, uniform in its logarithm, a multiple of mult."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(("gemm_fp8", "gemm_fp8", "gemm_fp8", "rms_norm", "rms_train", "quant_fp8", "clip_grads"))
    if op == "gemm_fp8":
        rows, cols = _size(rng, 64, 28672), _size(rng, 256, 28672, 16)
        most = min(8192, 28672 * 8192 * 8192 // (rows * cols))
        return dict(op=op, rows=rows, cols=cols, tokens=_size(rng, 1, most), out=rng.choice(("bf16", "f32")))
    if op == "rms_norm":
        dim = _size(rng, 256, 16384, 16)
        return dict(op=op, tokens=_size(rng, 1, 8192 * 8192 // dim), dim=dim, residual=rng.random() < 0.5,
                    out=rng.choice(("bf16", "fp8")))
    if op == "rms_train":
        dim = _size(rng, 256, 8192, 8)
        return dict(op=op, tokens=_size(rng, 1, 16384 * 4096 // dim), dim=dim, residual=rng.random() < 0.5)
    if op == "quant_fp8":
        gated, dim = rng.random() < 0.5, _size(rng, 256, 28672, 16)
        return dict(op=op, tokens=_size(rng, 1, 8192 * 28672 // dim), dim=dim, gated=gated)
    dim = _size(rng, 64, 4096)
    return dict(op=op, layers=rng.randint(1, 4), dim=dim, kv=max(1, dim // rng.randint(1, 8)),
                ffn=_size(rng, dim, 3 * dim), kind=rng.choice(("bf16", "f32")), max_norm=rng.choice((1.0, 1.0, 1e6)))


def _blocks(n):
    return -(-n // BLOCK)


def _per_column(scales, cols):
    """One value per block to one per column."""
    return scales.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def _amax(y):
    """Each row's largest magnitude per block of columns."""
    rows, cols = y.shape
    padded = torch.nn.functional.pad(y, (0, _blocks(cols) * BLOCK - cols))
    return padded.abs().reshape(rows, -1, BLOCK).amax(dim=2)


def _quantised(y):
    """Codes and scales of a matrix's rows."""
    scales = _amax(y).clamp_min(SMALLEST_MAX) / CODE_MAX
    return (y / _per_column(scales, y.shape[1])).to(F8), scales


def _matrix_codes(g, rows, cols):
    """A matrix of normal weights as e4m3 codes with a scale per block of 128 x 128."""
    w = torch.randn(rows, cols, generator=g, device="cuda").mul_(0.02)
    top = torch.nn.functional.pad(_amax(w), (0, 0, 0, _blocks(rows) * BLOCK - rows))
    scales = top.reshape(_blocks(rows), BLOCK, -1).amax(dim=1) / CODE_MAX
    wide = _per_column(scales, cols).repeat_interleave(BLOCK, dim=0)[:rows]
    return w.div_(wide).to(F8), scales.contiguous()


def _activations(g, tokens, dim):
    """Normal values with a few columns that are much larger, as hidden states have them."""
    x = torch.randn(tokens, dim, generator=g, device="cuda")
    x *= torch.where(torch.rand(dim, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _gradient_shapes(case):
    d, kv, f = case["dim"], case["kv"], case["ffn"]
    return [(d, d), (kv, d), (kv, d), (d, d), (f, d), (f, d), (d, f), (d,), (d,)] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, bf16 = case["op"], torch.bfloat16
    s = dict(case)
    if op == "clip_grads":
        # matrices in the case's type, the norms' weights always in 32 bits
        kind = bf16 if case["kind"] == "bf16" else torch.float32
        s["grads"] = [torch.randn(shape, generator=g, device="cuda").mul_(0.01).to(kind if len(shape) == 2 else
                                                                                  torch.float32)
                      for shape in _gradient_shapes(case)]
        s["outs"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda")
        return s
    tokens = case["tokens"]
    if op == "gemm_fp8":
        rows, cols = case["rows"], case["cols"]
        s["codes"], s["scales"] = _matrix_codes(g, rows, cols)
        s["x_codes"], s["x_scales"] = _quantised(_activations(g, tokens, cols).float())
        s["y"] = torch.empty(tokens, rows, device="cuda", dtype=bf16 if case["out"] == "bf16" else torch.float32)
        return s
    dim = case["dim"]
    s["x"] = _activations(g, tokens, 2 * dim if op == "quant_fp8" and case["gated"] else dim)
    if op == "quant_fp8" or (op == "rms_norm" and case["out"] == "fp8"):
        s["y_codes"] = torch.empty(tokens, dim, device="cuda", dtype=F8)
        s["y_scales"] = torch.empty(tokens, _blocks(dim), device="cuda")
    if op == "quant_fp8":
        return s
    s["weight"] = (torch.randn(dim, generator=g, device="cuda") * 0.1 + 1.0).to(bf16)
    s["residual_in"] = s["sum"] = None
    if case["residual"]:
        s["residual_in"] = torch.randn(tokens, dim, generator=g, device="cuda").mul_(2.0).to(bf16)
        s["sum"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
    if op == "rms_train" or case["out"] == "bf16":
        s["y"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
    if op == "rms_train":
        s["rstd"] = torch.empty(tokens, device="cuda")
        s["dy"] = torch.randn(tokens, dim, generator=g, device="cuda").mul_(0.01).to(bf16)
        s["dsum"] = torch.randn(tokens, dim, generator=g, device="cuda").mul_(0.01).to(bf16)
        s["dh"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
        s["dweight"] = torch.empty(dim, device="cuda")
    return s


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ---- the plain forms ------------------------------------------------------------

def _plain_gemm_fp8(s):
    rows, cols = s["rows"], s["cols"]
    w = s["codes"].float() * _per_column(s["scales"], cols).repeat_interleave(BLOCK, dim=0)[:rows]
    x = s["x_codes"].float() * _per_column(s["x_scales"], cols)
    return (x @ w.t()).to(s["y"].dtype)


def _plain_norm(s):
    """(h, rstd, y in 32 bits): the norm is of the sum as it is stored."""
    h = s["x"] if s["residual_in"] is None else (s["x"].float() + s["residual_in"].float()).to(torch.bfloat16)
    wide = h.float()
    rstd = torch.rsqrt(wide.square().mean(dim=1, keepdim=True) + EPS)
    return h, rstd, wide * rstd * s["weight"].float()


def _plain_rms_norm(s):
    h, _, y = _plain_norm(s)
    out = dict(sum=h) if s["residual"] else {}
    if s["out"] == "bf16":
        return dict(out, y=y.to(torch.bfloat16))
    codes, scales = _quantised(y)
    return dict(out, codes=codes, scales=scales)


def _plain_rms_train(s):
    h, rstd, y = _plain_norm(s)
    dy, unit = s["dy"].float(), h.float() * rstd
    g = dy * s["weight"].float()
    dh = s["dsum"].float() + rstd * (g - unit * (g * unit).mean(dim=1, keepdim=True))
    out = dict(y=y.to(torch.bfloat16), dh=dh.to(torch.bfloat16), dweight=(dy * unit).sum(dim=0))
    return dict(out, sum=h) if s["residual"] else out


def _plain_quant_fp8(s):
    y = s["x"].float()
    if s["gated"]:
        gate, up = y[:, :s["dim"]], y[:, s["dim"]:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    codes, scales = _quantised(y)
    return dict(codes=codes, scales=scales)


def _plain_clip_grads(s):
    squares = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]])
    norm = squares.sum().sqrt()
    factor = torch.where((norm > s["max_norm"]) & torch.isfinite(norm), s["max_norm"] / norm, 1.0).float()
    return dict(norm=norm.float().reshape(1), grads=[(t.float() * factor).to(t.dtype) for t in s["grads"]])


_PLAIN = dict(gemm_fp8=_plain_gemm_fp8, rms_norm=_plain_rms_norm, rms_train=_plain_rms_train,
              quant_fp8=_plain_quant_fp8, clip_grads=_plain_clip_grads)


# ---- the library's calls --------------------------------------------------------

def _workspace(s, nbytes):
    """The caller's scratch memory, which a program keeps from call to call."""
    if "work" not in s:
        s["work"] = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device="cuda")
    return s["work"], s["work"].numel()


def _own(s):
    from lossless_entropy_coded_amd import wc

    op = s["op"]
    if op == "clip_grads":
        if "list" not in s:   # the handle of the gradients, which a program keeps with them
            s["list"] = wc.GradList(s["grads"], s["outs"])
        work, nbytes = _workspace(s, lambda: wc.clip_grads_work_bytes(s["list"]))
        wc.clip_grads_async(s["list"], s["max_norm"], s["norm"], work, nbytes)
        return dict(norm=s["norm"], grads=s["outs"])
    tokens = s["tokens"]
    if op == "gemm_fp8":
        if "matrix" not in s:   # the handle of the matrix, which a program keeps with it
            s["matrix"] = wc.Fp8Matrix(s["codes"], s["scales"], s["rows"], s["cols"])
        work, nbytes = _workspace(s, lambda: wc.gemm_fp8_work_bytes(s["matrix"], tokens))
        wc.gemm_fp8_async(s["matrix"], s["x_codes"], s["x_scales"], tokens, s["y"], work, nbytes, out=s["out"])
        return s["y"]
    dim = s["dim"]
    if op == "quant_fp8":
        wc.quant_fp8_async(s["x"], tokens, dim, s["y_codes"], s["y_scales"], gated=s["gated"])
        return dict(codes=s["y_codes"], scales=s["y_scales"])
    into = dict(residual_dev=s["residual_in"], sum_dev=s["sum"])
    out = dict(sum=s["sum"]) if s["residual"] else {}
    if op == "rms_norm" and s["out"] == "fp8":
        wc.rms_norm_async(s["x"], s["weight"], tokens, dim, EPS, codes_dev=s["y_codes"], scales_dev=s["y_scales"],
                          **into)
        return dict(out, codes=s["y_codes"], scales=s["y_scales"])
    if op == "rms_norm":
        wc.rms_norm_async(s["x"], s["weight"], tokens, dim, EPS, y_dev=s["y"], **into)
        return dict(out, y=s["y"])
    wc.rms_norm_async(s["x"], s["weight"], tokens, dim, EPS, y_dev=s["y"], rstd_dev=s["rstd"], **into)
    work, nbytes = _workspace(s, lambda: wc.rms_norm_grad_work_bytes(tokens, dim))
    wc.rms_norm_grad_async(s["dy"], s["sum"] if s["residual"] else s["x"], s["weight"], s["rstd"], tokens, dim,
                           s["dh"], s["dweight"], work, nbytes, dsum_dev=s["dsum"])
    return dict(out, y=s["y"], dh=s["dh"], dweight=s["dweight"])


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    op = case["op"]
    if op == "clip_grads":
        size = 2 if case["kind"] == "bf16" else 4
        values = [math.prod(shape) for shape in _gradient_shapes(case)]
        wide = [n * (size if len(shape) == 2 else 4) for n, shape in zip(values, _gradient_shapes(case))]
        return dict(bytes=2 * sum(wide) + 4, flops=3 * sum(values))
    tokens = case["tokens"]
    if op == "gemm_fp8":
        rows, cols = case["rows"], case["cols"]
        scales = 4 * _blocks(cols) * (tokens + _blocks(rows))
        return dict(bytes=cols * (rows + tokens) + scales + (2 if case["out"] == "bf16" else 4) * rows * tokens,
                    flops=2 * rows * cols * tokens)
    dim = case["dim"]
    values, codes = tokens * dim, tokens * (dim + 4 * _blocks(dim))
    if op == "quant_fp8":
        return dict(bytes=values * (4 if case["gated"] else 2) + codes, flops=values * (8 if case["gated"] else 3))
    sums = 4 * values if case["residual"] else 0      # the residual in, the sum out
    if op == "rms_norm":
        return dict(bytes=2 * values + sums + 2 * dim + (codes if case["out"] == "fp8" else 2 * values),
                    flops=6 * values)
    # forward: x, the residual, the sum, y; gradient: dy, dsum, dh, and the sum once more
    return dict(bytes=2 * values + sums + 2 * values + 8 * values + 6 * dim, flops=18 * values)


# ---- the definitions in 64 bits -------------------------------------------------

def _codes64(y):
    """(code values before their rounding, scales): y over the scale of its block."""
    rows, cols = y.shape
    at = torch.arange(cols, device="cuda") // BLOCK
    top = torch.zeros(rows, _blocks(cols), dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, at.expand(rows, cols), y.abs(), "amax")
    scales = torch.maximum(top, torch.full_like(top, SMALLEST_MAX)) / CODE_MAX
    return y / scales[:, at], scales


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip_grads":
        norm = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in s["grads"]:
            flat = t.double().flatten()
            norm += torch.dot(flat, flat)
        norm = norm.sqrt()
        clips = math.isfinite(float(norm)) and float(norm) > case["max_norm"]
        return dict(norm=norm.reshape(1),
                    grads=[t.double() * case["max_norm"] / norm if clips else t.double() for t in s["grads"]])
    if op == "gemm_fp8":
        down = torch.arange(case["rows"], device="cuda") // BLOCK
        across = torch.arange(case["cols"], device="cuda") // BLOCK
        w = s["codes"].double().mul_(s["scales"].double()[down][:, across])
        x = s["x_codes"].double().mul_(s["x_scales"].double()[:, across])
        return torch.mm(w, x.t()).t()
    if op == "quant_fp8":
        y = s["x"].double()
        if case["gated"]:
            y = y[:, :case["dim"]] * torch.sigmoid(y[:, :case["dim"]]) * y[:, case["dim"]:]
        codes, scales = _codes64(y)
        return dict(codes=codes, scales=scales)
    h = s["x"].double()
    if case["residual"]:
        h = (h + s["residual_in"].double()).to(torch.bfloat16).double()   # the norm is of the sum as it is stored
    unit = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["dim"] + EPS)
    weight = s["weight"].double()
    out = dict(sum=h) if case["residual"] else {}
    if op == "rms_norm":
        if case["out"] == "bf16":
            return dict(out, y=unit * weight)
        codes, scales = _codes64(unit * weight)
        return dict(out, codes=codes, scales=scales)
    g, dy = s["dy"].double() * weight, s["dy"].double()
    rstd = torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["dim"] + EPS).reciprocal()
    along = (g * unit).sum(dim=1, keepdim=True) / case["dim"]
    return dict(out, y=unit * weight, dh=s["dsum"].double() + (g - unit * along) * rstd, dweight=(dy * unit).sum(dim=0))
