"""GPU tests of the matrix-vector products with 4-bit weights and group scales."""
import numpy as np
import pytest
import torch

from gpu_util import log, to_device_aligned
from operator_ref import q4_case, q4_tolerance, within

pytestmark = pytest.mark.gpu
GUARD = 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _run(wc, matrix, x, **kw):
    vecs, rows = x.shape[0], matrix.rows
    y = torch.full((vecs * rows + GUARD,), float("nan"), device="cuda")
    wc.gemv_q4_async(matrix, x, vecs, y, **kw)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[vecs * rows:]).all()), "wrote past y"
    return y[:vecs * rows].reshape(vecs, rows)


SHAPES = [(1, 8, 1, 32, False), (3, 24, 2, 32, True), (16, 32, 1, 32, False), (17, 40, 4, 64, True),
          (31, 128, 1, 128, False), (33, 256, 3, 64, True), (48, 1160, 3, 64, True), (40, 2048, 7, 128, True),
          (64, 4096, 1, 128, False), (100, 4096, 16, 128, True), (100, 4096, 9, 32, False),
          (5, 8200, 16, 96, True), (36, 6144, 5, 256, True), (20, 28672, 1, 65536, False),
          (20, 28672, 4, 64, True), (1003, 2088, 5, 32, True), (1024, 4096, 1, 128, True), (4097, 512, 2, 128, False)]


@pytest.mark.parametrize("rows,cols,vecs,group,zeros", SHAPES)
def test_products(wc, rows, cols, vecs, group, zeros):
    codes, scales, z, w = q4_case(rows, cols, group, zeros, rows + cols)
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(vecs, cols, generator=g).to(torch.bfloat16)
    log(f"case: gemv_q4 {rows}x{cols} vecs {vecs} group {group} zeros {zeros}")
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    y = _run(wc, matrix, x.cuda())
    assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))
    again = _run(wc, matrix, x.cuda())
    assert torch.equal(y.view(torch.int32), again.view(torch.int32)), "two runs differ"


@pytest.mark.parametrize("vecs", range(1, 17))
def test_vectors_do_not_depend_on_each_other(wc, vecs):
    """Every vector's products within the bound, whatever stands beside it."""
    rows, cols, group = 37, 1056, 32
    codes, scales, z, w = q4_case(rows, cols, group, True, 5)
    g = torch.Generator().manual_seed(vecs)
    x = torch.randn(vecs, cols, generator=g).to(torch.bfloat16)
    x[vecs - 1] *= 1e6
    log(f"case: gemv_q4 {vecs} vectors of different size")
    y = _run(wc, wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z), x.cuda())
    assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False), (128, True)])
@pytest.mark.parametrize("vecs", [1, 6])
def test_values_of_x(wc, group, zeros, vecs):
    """Zeros, subnormals, one outlier among small values, and magnitudes from 2^-120 to 2^120."""
    rows, cols = 48, 1024
    codes, scales, z, w = q4_case(rows, cols, group, zeros, 11)
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    g = torch.Generator().manual_seed(3)
    n = torch.randn(vecs, cols, generator=g)
    outlier = n.clone()
    outlier[:, 5] = 3e4
    for what, x in (("zeros", torch.zeros(vecs, cols)), ("outlier", outlier), ("2^100", n * 2.0 ** 100),
                    ("2^-90", n * 2.0 ** -90), ("mixed", n * torch.exp2(torch.randint(-40, 41, (1, cols),
                                                                                        generator=g).float()))):
        x = x.to(torch.bfloat16)
        log(f"case: gemv_q4 x {what}, group {group}, vecs {vecs}")
        y = _run(wc, matrix, x.cuda())
        assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double())), what


def test_infinities_and_nans(wc):
    """x with non-finite values gives what IEEE sums of scale * (code - zero) * x give."""
    rows, cols, group = 40, 512, 64
    codes, scales, z, w = q4_case(rows, cols, group, True, 2)
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    for what, places in (("inf", {7: float("inf")}), ("-inf", {300: float("-inf")}), ("nan", {511: float("nan")}),
                         ("inf in two blocks", {0: float("inf"), 400: float("inf")})):
        for vecs in (1, 5):
            x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(1))
            for c, v in places.items():
                x[vecs - 1, c] = v
            x = x.to(torch.bfloat16)
            log(f"case: gemv_q4 x with {what}, vecs {vecs}")
            y = _run(wc, matrix, x.cuda()).cpu().double()
            ref = torch.stack([(w * v).sum(dim=1) for v in x.double()])
            fin = torch.isfinite(ref)
            assert torch.equal(torch.isnan(y), torch.isnan(ref)), what
            assert torch.equal(y[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)]), what
            tol = q4_tolerance(w, torch.nan_to_num(x.double(), 0.0, 0.0, 0.0))
            assert bool(((y - ref).abs()[fin] <= tol[fin]).all()), what


def test_extreme_zero_points(wc):
    """Zero points are bytes: 0, 15 and 255 too."""
    rows, cols, group = 24, 256, 32
    codes, scales, z, _ = q4_case(rows, cols, group, True, 9)
    z = torch.tensor([0, 15, 255], dtype=torch.uint8)[torch.arange(rows * 8) % 3].reshape(rows, 8).cuda()
    q = torch.stack((codes & 15, codes >> 4), dim=2).reshape(rows, cols).cpu().double()
    at = torch.arange(cols) // group
    w = scales.cpu().double()[:, at] * (q - z.cpu().double()[:, at])
    for vecs in (1, 8):
        x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(vecs)).to(torch.bfloat16)
        log(f"case: gemv_q4 zero points 0, 15, 255, vecs {vecs}")
        y = _run(wc, wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z), x.cuda())
        assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))


def test_empty_calls_write_nothing(wc):
    codes, scales, _, _ = q4_case(16, 64, 32, False, 1)
    y = torch.full((16,), float("nan"), device="cuda")
    x = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    wc.gemv_q4_async(wc.Q4Matrix(codes, scales, 16, 64, 32), x, 0, y)
    wc.gemv_q4_async(wc.Q4Matrix(codes, scales, 0, 64, 32), x, 1, y)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y).all())


def test_decoded_code_plane(wc):
    """An int4 code plane through its container, decoded and multiplied in place: the bits of the plain plane's."""
    from lossless_entropy_coded_amd.synth import make_code_workload
    wl = make_code_workload("int4_codes_8b", scale_rows=48)
    blob = wc.encode_u8_host(wl.tensors())
    with wc.Plan(blob) as plan:
        _, dblob = to_device_aligned(blob)
        plane = torch.empty(plan.n_elems, dtype=torch.uint8, device="cuda")
        wc.decode_u8_async(plan, dblob, plane)
        for k, (rows, half) in enumerate(wl.shapes):
            cols, off = 2 * half, plan.tensor_offsets[k]
            codes = plane[off:off + rows * half]
            g = torch.Generator().manual_seed(k)
            scales = (torch.rand(rows, cols // 128, generator=g) * 0.02).to(torch.bfloat16)
            x = torch.randn(1, cols, generator=g).to(torch.bfloat16)
            log(f"case: gemv_q4 on decoded plane {wl.names[k]} {rows}x{cols}")
            y = _run(wc, wc.Q4Matrix(codes, scales.cuda(), rows, cols, 128), x.cuda())
            raw = torch.from_numpy(np.ascontiguousarray(wl.tensors()[k])).cuda()
            y2 = _run(wc, wc.Q4Matrix(raw, scales.cuda(), rows, cols, 128), x.cuda())
            assert torch.equal(y.view(torch.int32), y2.view(torch.int32))
            b = raw.cpu().long().reshape(rows, half)
            q = torch.stack((b & 15, b >> 4), dim=2).reshape(rows, cols).double()
            w = (q - 8) * scales.double().repeat_interleave(128, dim=1)
            assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))


def test_side_stream_and_graph(wc):
    """On another stream, and captured and replayed with new x between the replays."""
    rows, cols, vecs = 200, 2048, 3
    codes, scales, z, w = q4_case(rows, cols, 128, True, 4)
    matrix = wc.Q4Matrix(codes, scales, rows, cols, 128, zeros=z)
    xs = [torch.randn(vecs, cols, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in range(3)]
    eager = [_run(wc, matrix, x.cuda()) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    log("case: gemv_q4 on a side stream")
    y = _run(wc, matrix, xs[0].cuda(), stream=side)
    assert torch.equal(y, eager[0])
    x, y = xs[0].cuda(), torch.empty(vecs, rows, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.gemv_q4_async(matrix, x, vecs, y)
    log("case: gemv_q4 captured, three replays")
    for i in (1, 2, 0):
        x.copy_(xs[i])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])


@pytest.mark.parametrize("vecs", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("cols", [128, 1152, 4096])
def test_scales_off_their_alignment(wc, cols, vecs):
    """Groups of 32 with scales and zero points that start off 8-byte places: the bits of aligned ones."""
    rows, group = 21, 32
    codes, scales, z, w = q4_case(rows, cols, group, True, cols)
    x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(vecs)).to(torch.bfloat16)
    groups = cols // group
    shifted = torch.empty(rows * groups + 1, dtype=torch.bfloat16, device="cuda")[1:].reshape(rows, groups)
    shifted_z = torch.empty(rows * groups + 3, dtype=torch.uint8, device="cuda")[3:].reshape(rows, groups)
    shifted.copy_(scales), shifted_z.copy_(z)
    log(f"case: gemv_q4 {rows}x{cols} group 32 vecs {vecs}, aligned and shifted scales")
    y = _run(wc, wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z), x.cuda())
    assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))
    y2 = _run(wc, wc.Q4Matrix(codes, shifted, rows, cols, group, zeros=shifted_z), x.cuda())
    assert torch.equal(y.view(torch.int32), y2.view(torch.int32))


@pytest.mark.parametrize("vecs", [1, 2, 5, 16])
@pytest.mark.parametrize("cols", [8, 104, 112, 120, 1144, 2024, 4088])
def test_columns_end_just_before_a_step(wc, cols, vecs):
    """The last workgroup has one row, so that its codes end where a step's uniform offset may already be past them."""
    rows, group = 17, 64
    codes, scales, z, w = q4_case(rows, cols, group, True, cols)
    x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(vecs)).to(torch.bfloat16)
    log(f"case: gemv_q4 {rows}x{cols}, {vecs} vectors, the last step a few columns short")
    y = _run(wc, wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z), x.cuda())
    assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double()))


@pytest.mark.parametrize("group", [4096, 1 << 20, 0xFFFFFFE0])
def test_one_scale_per_row_whatever_the_group(wc, group):
    rows, cols = 40, 1152
    codes, scales, z, w = q4_case(rows, cols, group, True, 3)
    x = torch.randn(2, cols, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    log(f"case: gemv_q4 and lookup, group {group}")
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    assert within(_run(wc, matrix, x.cuda()), x.double() @ w.t(), q4_tolerance(w, x.double()))
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    wc.embed_q4_async(matrix, torch.arange(rows, device="cuda"), rows, out)
    # scale (8 bits) times code less zero point (5 bits) is exact in fp32, so out is w rounded once
    assert torch.equal(out.cpu(), w.to(torch.bfloat16))
