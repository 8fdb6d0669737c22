"""Measured cases of the operators that consume decoded tensors: 4-bit
matrix-vector products (gemv_q4), embedding lookup (embed, embed_q4) with its
gradient (embed_grad), and the vocabulary product's softmax cross entropy
(ce_loss) with its gradients (ce_train).

With `own` false, run() computes an operator from elementary torch operations
in 32 bits, rounded once at the end; with `own` true it makes the library's
calls.  Either way one run() is one pass as a program makes it, on inputs that
prepare() draws from the seed.
"""
import math

import torch

own = False

WEIGHT_SIGMA = 1.5          # spread of 4-bit codes in units of the scale (the int4 code-plane workload's)


def listed():
    return [
        # the smallest projection of an 8B-shape block, one token: launch and latency bound
        dict(name="gemv_q4 k_proj 1 token", op="gemv_q4", rows=1024, cols=4096, vecs=1, group=128, zeros=False),
        # its widest projection, one token: the ordinary serving step
        dict(name="gemv_q4 gate_proj 1 token", op="gemv_q4", rows=14336, cols=4096, vecs=1, group=128, zeros=False),
        # a 70B-shape block's down projection, eight tokens verified at once, finer groups with zero points
        dict(name="gemv_q4 70B down_proj 8 tokens", op="gemv_q4", rows=8192, cols=28672, vecs=8, group=64,
             zeros=True),
        # odd sizes: rows not in tiles, rows of codes that start off 16-byte boundaries, a short last group
        dict(name="gemv_q4 odd 5 tokens", op="gemv_q4", rows=1003, cols=2088, vecs=5, group=32, zeros=True),
        # the next token of one sequence: a single row of a large table
        dict(name="embed 1 token", op="embed", vocab=131072, dim=4096, tokens=1, scale=1.0, pads=False),
        # a prefill's tokens from a 4-bit table, scaled by sqrt(dim)
        dict(name="embed_q4 prefill", op="embed_q4", vocab=131072, dim=4096, tokens=8192, group=128, zeros=True,
             scale=64.0, pads=False),
        # a training batch's gradient in 32 bits, token frequencies falling as 1 / rank
        dict(name="embed_grad batch f32", op="embed_grad", vocab=32768, dim=4096, tokens=16384, scale=1.0,
             out="f32", pads=False),
        # a padded batch's, odd sizes, rounded to bf16
        dict(name="embed_grad padded bf16", op="embed_grad", vocab=50021, dim=1160, tokens=4099, scale=34.0,
             out="bf16", pads=True),
        # scoring a few tokens against the whole vocabulary: bound by reading the matrix
        dict(name="ce_loss 16 tokens", op="ce_loss", vocab=131072, dim=4096, tokens=16, pads=False),
        # perplexity over a long text, odd vocabulary, a masked prompt
        dict(name="ce_loss perplexity", op="ce_loss", vocab=50021, dim=4096, tokens=2048, pads=True),
        # a small model's training step, every size odd
        dict(name="ce_train odd", op="ce_train", vocab=32003, dim=1160, tokens=515, pads=True),
        # a large one's: a full batch, the largest vocabulary
        dict(name="ce_train batch", op="ce_train", vocab=131072, dim=4096, tokens=4096, pads=False),
    ]


def _size(rng, lo, hi, mult=1):
    """A whole number from lo to hi, uniform in its logarithm, a multiple of mult."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(("gemv_q4", "gemv_q4", "embed", "embed_q4", "embed_grad", "ce_loss", "ce_train"))
    pads, zeros = rng.random() < 0.5, rng.random() < 0.5
    if op == "gemv_q4":
        return dict(op=op, rows=_size(rng, 64, 28672), cols=_size(rng, 256, 28672, 8), vecs=rng.randint(1, 16),
                    group=rng.choice((32, 64, 128)), zeros=zeros)
    case = dict(op=op, vocab=_size(rng, 1000, 131072), dim=_size(rng, 256, 4096, 8), pads=pads)
    if op == "embed":
        return dict(case, tokens=_size(rng, 1, 65536), scale=rng.choice((1.0, 11.5)))
    if op == "embed_q4":
        return dict(case, tokens=_size(rng, 1, 65536), group=rng.choice((32, 64, 128)), zeros=zeros,
                    scale=rng.choice((1.0, 45.25)))
    if op == "embed_grad":
        return dict(case, tokens=_size(rng, 1, 65536), out=rng.choice(("f32", "bf16")),
                    scale=rng.choice((1.0, 11.5)))
    return dict(case, tokens=_size(rng, 1, 4096))


def _codes(g, rows, cols):
    q = torch.randn(rows, cols, generator=g, device="cuda").mul_(WEIGHT_SIGMA).round_().clamp_(-8, 7).add_(8)
    q = q.to(torch.uint8)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()


def _q4(g, rows, cols, group, zeros):
    groups = -(-cols // group)
    scales = torch.rand(rows, groups, generator=g, device="cuda").add_(0.5).mul_(0.02 / WEIGHT_SIGMA)
    z = torch.randint(6, 11, (rows, groups), generator=g, device="cuda").to(torch.uint8) if zeros else None
    return dict(codes=_codes(g, rows, cols), scales=scales.to(torch.bfloat16), zeros=z)


def _ids(g, vocab, tokens, pads):
    """Token ids whose frequency falls as 1 / rank; with pads, the last part of the batch (and one id in 16) is -1."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(vocab)).long().sub_(1).clamp_(0, vocab - 1)
    if pads:
        ids[tokens - tokens // 8:] = -1
        ids[torch.rand(tokens, generator=g, device="cuda") < 1 / 16] = -1
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, bf16 = case["op"], torch.bfloat16
    s = dict(case)
    if op == "gemv_q4":
        s.update(_q4(g, case["rows"], case["cols"], case["group"], case["zeros"]))
        s["x"] = torch.randn(case["vecs"], case["cols"], generator=g, device="cuda").to(bf16)
        s["y"] = torch.empty(case["vecs"], case["rows"], device="cuda")
        return s
    vocab, dim, tokens = case["vocab"], case["dim"], case["tokens"]
    s["ids"] = _ids(g, vocab, tokens, case["pads"])
    if op == "embed":
        s["table"] = torch.randn(vocab, dim, generator=g, device="cuda", dtype=bf16)
        s["rows_out"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
    elif op == "embed_q4":
        s.update(_q4(g, vocab, dim, case["group"], case["zeros"]))
        s["rows_out"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
    elif op == "embed_grad":
        s["drows"] = torch.randn(tokens, dim, generator=g, device="cuda").mul_(0.01).to(bf16)
        s["dtable"] = torch.empty(vocab, dim, device="cuda", dtype=torch.float32 if case["out"] == "f32" else bf16)
    else:
        s["h"] = torch.randn(tokens, dim, generator=g, device="cuda").to(bf16)
        s["W"] = torch.randn(vocab, dim, generator=g, device="cuda", dtype=bf16).mul_(2.0 / math.sqrt(dim))
        s["loss"] = torch.empty(tokens, device="cuda")
        s["lse"] = torch.empty(tokens, device="cuda")
        if op == "ce_train":                     # the mean loss's gradient, with a weight for each token
            s["dloss"] = (torch.rand(tokens, generator=g, device="cuda") + 0.5) / tokens
            s["dh"] = torch.empty(tokens, dim, device="cuda", dtype=bf16)
            s["dW"] = torch.empty(vocab, dim, device="cuda", dtype=bf16)
    return s


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ---- the plain forms ------------------------------------------------------------

def _unpack(s, rows=None):
    """The matrix (or some of its rows) in 32 bits: scale * (code - zero point)."""
    codes, scales, zeros = s["codes"], s["scales"], s["zeros"]
    if rows is not None:
        codes, scales = codes[rows], scales[rows]
        zeros = None if zeros is None else zeros[rows]
    q = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1).float()
    cols, group = q.shape[1], s["group"]
    wide = lambda t: t.float().repeat_interleave(group, dim=1)[:, :cols]  # noqa: E731
    return wide(scales) * (q - (8.0 if zeros is None else wide(zeros)))


def _plain_gemv_q4(s):
    return s["x"].float() @ _unpack(s).t()


def _rows_of(s, vocab):
    ids = s["ids"]
    fits = (ids >= 0) & (ids < vocab)
    return torch.where(fits, ids, 0), fits


def _plain_embed(s):
    ids, fits = _rows_of(s, s["vocab"])
    rows = s["table"][ids].float() * s["scale"]
    return torch.where(fits[:, None], rows, 0.0).to(torch.bfloat16)


def _plain_embed_q4(s):
    ids, fits = _rows_of(s, s["vocab"])
    rows = _unpack(s, ids) * s["scale"]
    return torch.where(fits[:, None], rows, 0.0).to(torch.bfloat16)


def _plain_embed_grad(s):
    ids, fits = _rows_of(s, s["vocab"])
    rows = torch.where(fits[:, None], s["drows"].float(), 0.0)
    total = torch.zeros(s["vocab"], s["dim"], device="cuda").index_add_(0, ids, rows)
    return (total * s["scale"]).to(s["dtable"].dtype)


def _plain_ce_loss(s):
    ids, fits = _rows_of(s, s["vocab"])
    logits = s["h"].float() @ s["W"].float().t()
    top = logits.amax(dim=1, keepdim=True)
    lse = (top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True))).squeeze(1)
    own_logit = logits.gather(1, ids[:, None]).squeeze(1)
    return dict(loss=torch.where(fits, lse - own_logit, 0.0), lse=lse)


def _plain_ce_train(s):
    ids, fits = _rows_of(s, s["vocab"])
    h, W = s["h"].float(), s["W"].float()
    logits = h @ W.t()
    top = logits.amax(dim=1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True))
    loss = torch.where(fits, (lse - logits.gather(1, ids[:, None])).squeeze(1), 0.0)
    d = torch.exp(logits - lse)
    d.scatter_add_(1, ids[:, None], torch.full_like(lse, -1.0))
    d *= torch.where(fits, s["dloss"], 0.0)[:, None]
    return dict(loss=loss, lse=lse.squeeze(1), dh=(d @ W).to(torch.bfloat16), dW=(d.t() @ h).to(torch.bfloat16))


_PLAIN = dict(gemv_q4=_plain_gemv_q4, embed=_plain_embed, embed_q4=_plain_embed_q4, embed_grad=_plain_embed_grad,
              ce_loss=_plain_ce_loss, ce_train=_plain_ce_train)


# ---- the library's calls --------------------------------------------------------

def _matrix(wc, s, rows, cols):
    """The handle of a 4-bit matrix, which a program keeps with the matrix."""
    if "matrix" not in s:
        s["matrix"] = wc.Q4Matrix(s["codes"], s["scales"], rows, cols, s["group"], zeros=s["zeros"])
    return s["matrix"]


def _workspace(s, nbytes):
    """The caller's scratch memory, which a program keeps from call to call."""
    if "work" not in s:
        s["work"] = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device="cuda")
    return s["work"], s["work"].numel()


def _own(s):
    from lossless_entropy_coded_amd import wc

    op = s["op"]
    if op == "gemv_q4":
        wc.gemv_q4_async(_matrix(wc, s, s["rows"], s["cols"]), s["x"], s["vecs"], s["y"])
        return s["y"]
    vocab, dim, tokens = s["vocab"], s["dim"], s["tokens"]
    if op == "embed":
        wc.embed_async(s["table"], vocab, dim, s["ids"], tokens, s["rows_out"], scale=s["scale"])
        return s["rows_out"]
    if op == "embed_q4":
        wc.embed_q4_async(_matrix(wc, s, vocab, dim), s["ids"], tokens, s["rows_out"], scale=s["scale"])
        return s["rows_out"]
    if op == "embed_grad":
        work, nbytes = _workspace(s, lambda: wc.embed_grad_work_bytes(tokens, dim))
        wc.embed_grad_async(s["drows"], s["ids"], tokens, s["dtable"], vocab, dim, work, nbytes, out=s["out"],
                            scale=s["scale"])
        return s["dtable"]
    train = op == "ce_train"
    work, nbytes = _workspace(s, lambda: wc.ce_work_bytes(tokens, vocab, dim, grad=train))
    wc.ce_loss_async(s["h"], s["W"], s["ids"], tokens, vocab, dim, s["loss"], s["lse"], work, nbytes)
    if not train:
        return dict(loss=s["loss"], lse=s["lse"])
    wc.ce_grad_async(s["h"], s["W"], s["ids"], tokens, vocab, dim, s["lse"], s["dloss"], s["dh"], s["dW"], work,
                     nbytes)
    return dict(loss=s["loss"], lse=s["lse"], dh=s["dh"], dW=s["dW"])


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    op = case["op"]
    if op == "gemv_q4":
        rows, cols, vecs = case["rows"], case["cols"], case["vecs"]
        per_group = 2 + bool(case["zeros"])
        weights = rows * cols // 2 + rows * -(-cols // case["group"]) * per_group
        return dict(bytes=weights + 2 * vecs * cols + 4 * vecs * rows, flops=2 * rows * cols * vecs)
    vocab, dim, tokens = case["vocab"], case["dim"], case["tokens"]
    if op == "embed":
        return dict(bytes=tokens * (8 + 4 * dim), flops=tokens * dim)
    if op == "embed_q4":
        row = dim // 2 + -(-dim // case["group"]) * (2 + bool(case["zeros"]))
        return dict(bytes=tokens * (8 + row + 2 * dim), flops=2 * tokens * dim)
    if op == "embed_grad":
        out = vocab * dim * (4 if case["out"] == "f32" else 2)
        return dict(bytes=tokens * (8 + 2 * dim) + out, flops=tokens * dim)
    inputs = 2 * dim * (tokens + vocab) + 8 * tokens
    product = 2 * tokens * vocab * dim
    if op == "ce_loss":
        return dict(bytes=inputs + 8 * tokens, flops=product)
    return dict(bytes=inputs + 2 * dim * (tokens + vocab) + 12 * tokens, flops=3 * product)


# ---- the definitions in 64 bits -------------------------------------------------

def _weights64(s):
    """scale * (code - zero point), one column parity at a time."""
    codes, group = s["codes"], s["group"]
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    at = torch.arange(cols, device="cuda") // group
    w = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    w[:, 0::2] = (codes % 16).double()
    w[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    w -= 8.0 if s["zeros"] is None else s["zeros"].double()[:, at]
    return w.mul_(s["scales"].double()[:, at])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemv_q4":
        return (_weights64(s) @ s["x"].double().t()).t()
    ids, vocab = s["ids"], case["vocab"]
    valid = torch.nonzero((ids >= 0) & (ids < vocab)).squeeze(1)
    if op in ("embed", "embed_q4"):
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        if op == "embed_q4":
            picked = {k: s[k] if s[k] is None else s[k].index_select(0, ids[valid])
                      for k in ("codes", "scales", "zeros")}
            rows = _weights64(dict(picked, group=case["group"]))
        else:
            rows = s["table"].index_select(0, ids[valid]).double()
        out[valid] = rows * case["scale"]
        return out
    if op == "embed_grad":
        total = torch.zeros(vocab, case["dim"], dtype=torch.float64, device="cuda")
        order = valid[torch.argsort(ids[valid], stable=True)]
        total.index_put_((ids[order],), s["drows"][order].double(), accumulate=True)
        return total * case["scale"]
    # cross entropy, a piece of the tokens at a time
    W = s["W"].double()
    loss = torch.zeros(case["tokens"], dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    train = op == "ce_train"
    if train:
        dW = torch.zeros_like(W)
        dh = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    for t0 in range(0, case["tokens"], 1024):
        part = slice(t0, min(t0 + 1024, case["tokens"]))
        h = s["h"][part].double()
        z = h @ W.t()
        lse[part] = torch.logsumexp(z, dim=1)
        has = torch.nonzero((ids[part] >= 0) & (ids[part] < vocab)).squeeze(1)
        to = ids[part][has]
        loss[t0 + has] = lse[part][has] - z[has, to]
        if train:
            p = torch.zeros_like(z)
            p[has] = torch.softmax(z[has], dim=1)
            p[has, to] -= 1
            p *= s["dloss"][part].double()[:, None]
            dh[part] = p @ W
            dW += p.t() @ h
    if not train:
        return dict(loss=loss, lse=lse)
    return dict(loss=loss, lse=lse, dh=dh, dW=dW)
