"""fp8_matmul against the same product in 64 bits.

Tolerance, per element: the products of two FP8 values are exact in FP32, so
an FP32 result has the roundings of its sums only.  A K of 128 B elements is
128 additions in each of B blocks, one rounding of the combined scale, one
fused multiply-add a block, and at most 16 additions of K splits: with each
step off by at most one unit (2^-23, twice a rounding, since the matrix
instruction may cut off instead of rounding) of the sum of magnitudes,
    |out - exact| <= (128 + B + 20) 2^-23 sum |terms| + half a step of out's type
(half its smallest subnormal where out is that small).  For BF16 and FP16
results the FP8 matrix instruction keeps, of the products of 16 consecutive k,
only what lies within 13 binades of the largest one's exponents (2^E with 2^E
<= the largest product): each product p of a group loses at most
    min(|p|, 2^-13 max |p| of the group),
whose sum is added to the bound."""
import pytest
import torch

import loss_scaling_fp8_amd as gs

pytestmark = pytest.mark.gpu

B1, B128 = gs.FP8_BLOCK_1x128, gs.FP8_BLOCK_128x128
E4M3, E5M2 = gs.FP8_E4M3, gs.FP8_E5M2
TORCH8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


def _operand(rows, k, fmt, gran, seed, dev):
    """Random finite codes (every finite code of the format occurs) and scales
    spread over 2^-12 .. 2^2."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, k), generator=g, dtype=torch.uint8)
    mag = codes & 0x7F
    top = 0x7E if fmt == E4M3 else 0x7B
    codes = torch.where(mag > top, codes & 0x83, codes)
    shape = gs.scale_shape(rows, k, gran)
    scales = torch.exp2(torch.rand(shape, generator=g) * 14 - 12) * (1 + torch.rand(shape, generator=g))
    return codes.to(dev), scales.to(dev)


def _values(codes, scales, fmt, gran):
    v = codes.cpu().view(TORCH8[fmt]).double()
    s = scales.cpu().double().repeat_interleave(128, 1)
    if gran == B128:
        s = s.repeat_interleave(128, 0)
    return v * s


def _cut(va, vb, dev):
    """Sum over the groups of 16 of min(|p|, 2^-13 max |p|), [m, n]."""
    m, k = va.shape
    n = vb.shape[0]
    a, b = va.abs().float().to(dev), vb.abs().float().to(dev)
    total = torch.zeros(m, n, dtype=torch.float64, device=dev)
    step = max(1, (1 << 26) // (16 * n))
    for r in range(0, m, step):
        for g in range(0, k, 16):
            p = a[r:r + step, None, g:g + 16] * b[None, :, g:g + 16]
            total[r:r + step] += torch.minimum(p, p.amax(-1, keepdim=True) * 2.0 ** -13).sum(-1)
    return total.cpu() * (1 + 2.0 ** -20)            # these sums are FP32


def _check(out, exact, absum, kblocks, base=None, cut=None):
    o = out.cpu().double()
    want = exact if base is None else exact + base
    tol = (128 + kblocks + 20) * 2.0 ** -23 * absum
    if cut is not None:
        tol = tol + cut
    if base is not None:
        tol = tol + 2.0 ** -24 * (absum + base.abs())
    tol = tol + HALF_STEP[out.dtype] * (want.abs() + tol) + TINY[out.dtype]
    bad = (o - want).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((o - want).abs() / tol).max()))


def _run(m, n, k, dev, a_fmt=E4M3, b_fmt=E4M3, a_gran=B1, b_gran=B128, dtype=torch.bfloat16,
         accumulate=False, seed=0):
    """One product between guard bands, checked; returns out."""
    a, sa = _operand(m, k, a_fmt, a_gran, 2 * seed + 1, dev)
    b, sb = _operand(n, k, b_fmt, b_gran, 2 * seed + 2, dev)
    va, vb = _values(a, sa, a_fmt, a_gran), _values(b, sb, b_fmt, b_gran)
    exact, absum = va @ vb.t(), va.abs() @ vb.abs().t()
    cut = _cut(va, vb, dev) if dtype != torch.float32 else None
    if dtype == torch.float16:                       # keep inside FP16's range
        f = 2.0 ** -torch.ceil(torch.log2(exact.abs().max() / 30000))
        sa, exact, absum, cut = sa * float(f), exact * f, absum * f, cut * f
    guard = 1024
    flat = torch.full((m * n + 2 * guard,), 7.0, dtype=dtype, device=dev)
    out = flat[guard:guard + m * n].view(m, n)
    base = None
    if accumulate:
        base = torch.randn(m, n, generator=torch.Generator().manual_seed(seed)) * float(exact.abs().mean())
        out.copy_(base)
        base = base.double()
    ws_bytes = gs.fp8_matmul_workspace_size(m, n, k)
    ws = torch.full((ws_bytes + 64,), 0xFF, dtype=torch.uint8, device=dev)    # NaN bits
    r = gs.fp8_matmul(a, sa, a_fmt, a_gran, b, sb, b_fmt, b_gran, out=out, accumulate=accumulate,
                      workspace=ws)
    assert r is out
    torch.cuda.synchronize()
    assert bool((flat[:guard] == 7).all()) and bool((flat[guard + m * n:] == 7).all())
    assert bool((ws[ws_bytes:] == 0xFF).all())
    _check(out, exact, absum, k // 128, base, cut)
    return out


# few rows; one row of tiles; K splits; ragged tiles; enough tiles for the largest
SHAPES = [(1, 128, 128), (1, 1024, 4096), (3, 128, 384), (16, 256, 1152), (17, 128, 256),
          (32, 384, 640), (33, 128, 2048), (64, 256, 896), (65, 128, 128), (100, 256, 1024),
          (128, 128, 128), (129, 384, 640), (128, 128, 4096), (333, 512, 4608), (257, 1024, 256)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes_weight_blocks(m, n, k, dev):
    _run(m, n, k, dev, seed=m + n)


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 17, 256), (5, 1000, 384), (40, 77, 1152),
                                   (64, 15, 128), (65, 1, 128), (66, 130, 256), (200, 333, 2048),
                                   (513, 255, 640), (70, 31, 8192)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_odd_sizes_row_blocks(m, n, k, dtype, dev):
    _run(m, n, k, dev, b_gran=B1, dtype=dtype, seed=m)


@pytest.mark.parametrize("a_fmt", [E4M3, E5M2])
@pytest.mark.parametrize("b_fmt", [E4M3, E5M2])
@pytest.mark.parametrize("a_gran", [B1, B128])
@pytest.mark.parametrize("b_gran", [B1, B128])
def test_formats_and_granularities(a_fmt, b_fmt, a_gran, b_gran, dev):
    """Both formats and granularities on either side, through each kernel."""
    for m, n, k in ((128, 256, 512), (256, 128, 4096)) + (((16, 128, 384),) if a_gran == B1 else ()):
        _run(m, n, k, dev, a_fmt, b_fmt, a_gran, b_gran, torch.float32, seed=7)


@pytest.mark.parametrize("a_fmt", [E4M3, E5M2])
@pytest.mark.parametrize("b_gran", [B1, B128])
def test_large_tiles(a_fmt, b_gran, dev):
    """Enough 256x256 tiles to fill the GPU, the last ones ragged."""
    n = 3712 if b_gran == B128 else 3701
    _run(4001, n, 384, dev, a_fmt, E4M3, B1, b_gran, torch.float32, seed=3)
    _run(4001, n, 128, dev, a_fmt, E4M3, B1, b_gran, torch.bfloat16, seed=4)


@pytest.mark.parametrize("a_fmt", [E4M3, E5M2])
@pytest.mark.parametrize("b_fmt", [E4M3, E5M2])
@pytest.mark.parametrize("m,n,k,b_gran,dtype", [
    (4001, 2949, 384, B1, torch.float32),            # 256x192 tiles
    (3900, 4001, 128, B1, torch.float32),            # 256x128
    (3900, 3968, 256, B128, torch.float32),
    (3841, 4001, 640, B1, torch.bfloat16),           # 256x256
    (4001, 3968, 128, B128, torch.float16)])
def test_large_tiles_of_each_kind(a_fmt, b_fmt, m, n, k, b_gran, dtype, dev):
    _run(m, n, k, dev, a_fmt, b_fmt, B1, b_gran, dtype, seed=13)


def test_accumulate_large_tiles(dev):
    _run(4001, 2949, 256, dev, E5M2, E4M3, B1, B1, torch.float32, accumulate=True, seed=14)


@pytest.mark.parametrize("m,n,k", [(1, 130, 256), (64, 128, 640), (130, 129, 128), (100, 70, 4096),
                                   (4001, 3701, 256)])
def test_accumulate(m, n, k, dev):
    _run(m, n, k, dev, E5M2, E4M3, B1, B1, torch.float32, accumulate=True, seed=9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_longest_k(dtype, dev):
    """k = 2^22, zero but for blocks at both ends and in the middle: zeros add
    nothing, so the tolerance is that of those blocks."""
    m, n, k = 65, 128, 1 << 22
    used = [0, 1, 9999, 16383, 16384, 32766, 32767]
    a, sa = _operand(m, 128 * len(used), E4M3, B1, 15, dev)
    b, sb = _operand(n, 128 * len(used), E4M3, B128, 16, dev)
    va, vb = _values(a, sa, E4M3, B1), _values(b, sb, E4M3, B128)
    la, lb = (torch.zeros(r, k, dtype=torch.uint8, device=dev) for r in (m, n))
    lsa, lsb = torch.ones(m, k // 128, device=dev), torch.ones(n // 128, k // 128, device=dev)
    for i, kb in enumerate(used):
        la[:, 128 * kb:128 * kb + 128] = a[:, 128 * i:128 * i + 128]
        lb[:, 128 * kb:128 * kb + 128] = b[:, 128 * i:128 * i + 128]
        lsa[:, kb], lsb[:, kb] = sa[:, i], sb.view(n // 128, -1)[:, i]
    out = gs.fp8_matmul(la, lsa, E4M3, B1, lb, lsb, E4M3, B128, out_dtype=dtype)
    _check(out, va @ vb.t(), va.abs() @ vb.abs().t(), len(used),
           cut=_cut(va, vb, dev) if dtype != torch.float32 else None)


def test_empty(dev):
    a, sa = _operand(4, 128, E4M3, B1, 1, dev)
    z, zs = a[:, :0].contiguous(), sa[:, :0].contiguous()
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        out = torch.full((4, 4), 3.0, dtype=dtype, device=dev)
        gs.fp8_matmul(z, zs, E4M3, B1, z, zs, E4M3, B1, out=out)
        assert bool((out == 0).all())
    out = torch.full((4, 4), 3.0, device=dev)
    gs.fp8_matmul(z, zs, E4M3, B1, z, zs, E4M3, B1, out=out, accumulate=True)
    assert bool((out == 3).all())
    e = a[:0]
    assert gs.fp8_matmul(e, sa[:0], E4M3, B1, a, sa, E4M3, B1).shape == (0, 4)
    assert gs.fp8_matmul(a, sa, E4M3, B1, e, sa[:0], E4M3, B1).shape == (4, 0)


@pytest.mark.parametrize("m,n", [(5, 128), (128, 256)])
def test_special_values(m, n, dev):
    """NaN codes of both formats, E5M2 infinities, zeros, and scales that are
    0, infinite or NaN: the result is NaN or infinite exactly where the 64-bit
    result is, and the other elements are unaffected."""
    k = 512
    a, sa = _operand(m, k, E5M2, B1, 31, dev)
    b, sb = _operand(n, k, E4M3, B1, 32, dev)
    sb[4, 1] = 0.0
    a[0, 3] = 0x7C                                   # +Inf
    a[1, 130] = 0xFD                                 # NaN
    a[2, 200] = 0xFC                                 # -Inf
    b[9, 7] = 0x7F                                   # NaN
    b[:, 3] = torch.where((b[:, 3] & 0x7F) == 0, 0x38, b[:, 3])
    b[11, 3] = 0                                     # Inf * 0
    sa[3, 2] = float("inf")
    sa[4, 0] = float("nan")
    va, vb = _values(a, sa, E5M2, B1), _values(b, sb, E4M3, B1)
    out = gs.fp8_matmul(a, sa, E5M2, B1, b, sb, E4M3, B1, out_dtype=torch.float32).cpu().double()
    # the block sums times the combined scale, as the product is defined
    exact = torch.zeros(m, n, dtype=torch.float64)
    for kb in range(k // 128):
        cols = slice(128 * kb, 128 * kb + 128)
        ca = a.cpu().view(TORCH8[E5M2]).double()[:, cols]
        cb = b.cpu().view(TORCH8[E4M3]).double()[:, cols]
        prod = (ca[:, None, :] * cb[None, :, :]).sum(-1)
        exact += prod * (sa.cpu().double()[:, kb, None] * sb.cpu().double()[None, :, kb])
    assert torch.equal(torch.isnan(out), torch.isnan(exact))
    inf = torch.isinf(exact)
    assert int(inf.sum()) > 0 and torch.equal(out[inf], exact[inf])
    fine = torch.isfinite(exact)
    rows = slice(5, m) if m > 5 else slice(0, 0)
    absum = va.abs() @ vb.abs().t()
    ok = (out - exact).abs() <= (128 + 4 + 20) * 2.0 ** -23 * absum * 1.0001
    assert bool(ok[rows][fine[rows]].all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k,b_gran", [(5, 128, 512, B1), (130, 256, 2048, B128),
                                          (130, 255, 384, B1), (3841, 4001, 256, B1),
                                          (3841, 3968, 256, B128)])
def test_special_values_16_bit(m, n, k, b_gran, dtype, dev):
    """The same in 16 bits, whose products take the FP8 instruction: through
    few rows, K splits and both sizes of tiles."""
    a, sa = _operand(m, k, E5M2, B1, 33, dev)
    b, sb = _operand(n, k, E4M3, b_gran, 34, dev)
    b[:, 3] = torch.where((b[:, 3] & 0x7F) == 0, 0x38, b[:, 3])
    b[11, 3] = 0                                     # for Inf * 0
    va, vb = _values(a, sa, E5M2, B1), _values(b, sb, E4M3, b_gran)
    if dtype == torch.float16:                       # keep the finite ones inside FP16's range
        f = float(2.0 ** -torch.ceil(torch.log2((va.abs() @ vb.abs().t()).max() / 30000)))
        sa = sa * f
        va = va * f
    absum, cut = va.abs() @ vb.abs().t(), _cut(va, vb, dev)
    b[9, 7] = 0x7F                                   # NaN
    a[0, 3] = 0x7C                                   # +Inf
    a[1, 130] = 0xFD                                 # NaN
    a[2, 200] = 0xFC                                 # -Inf
    out = gs.fp8_matmul(a, sa, E5M2, B1, b, sb, E4M3, b_gran, out_dtype=dtype).cpu().double()
    exact = torch.zeros(m, n, dtype=torch.float64)
    sa64, sb64 = sa.cpu().double(), sb.cpu().double()
    if b_gran == B128:
        sb64 = sb64.repeat_interleave(128, 0)
    for kb in range(k // 128):
        cols = slice(128 * kb, 128 * kb + 128)
        ca = a.cpu().view(TORCH8[E5M2]).double()[:, cols]
        cb = b.cpu().view(TORCH8[E4M3]).double()[:, cols]
        prod = ca @ cb.t()
        if kb <= 1:                                  # the rows with specials, product by product
            prod[:3] = (ca[:3, None, :] * cb[None, :, :]).sum(-1)
        prod[:, 9] = (ca * cb[9]).sum(-1)
        exact += prod * (sa64[:, kb, None] * sb64[None, :, kb])
    assert torch.equal(torch.isnan(out), torch.isnan(exact))
    inf = torch.isinf(exact)
    assert int(inf.sum()) > 0 and torch.equal(out[inf], exact[inf])
    fine = torch.isfinite(exact)
    fine[:3] = False
    tol = (128 + k // 128 + 20) * 2.0 ** -23 * absum + cut
    tol = tol + HALF_STEP[dtype] * (exact.abs() + tol) + TINY[dtype]
    assert bool(((out - exact).abs() <= tol)[fine].all())


def test_fp16_overflow_raises_the_flag(dev):
    """A weight gradient past FP16's range becomes an infinity that the
    unscale finds."""
    a = torch.full((128, 128), 0x7E, dtype=torch.uint8, device=dev)          # 448
    s = torch.ones(128, 1, device=dev)
    out = gs.fp8_matmul(a, s, E4M3, B1, a, s, E4M3, B1, out_dtype=torch.float16)
    assert bool(torch.isinf(out).all())
    found = torch.zeros(1, dtype=torch.int32, device=dev)
    gs.gs_unscale_check([out], [torch.empty(128, 128, device=dev)], torch.ones(1, device=dev), found)
    assert int(found) == 1


@pytest.mark.parametrize("m,n,k", [(7, 128, 1024), (333, 512, 4608), (4001, 3712, 256)])
def test_equal_calls_give_equal_bits(m, n, k, dev):
    a, sa = _operand(m, k, E4M3, B1, 41, dev)
    b, sb = _operand(n, k, E4M3, B128, 42, dev)
    first = gs.fp8_matmul(a, sa, E4M3, B1, b, sb, E4M3, B128, out_dtype=torch.float32)
    for _ in range(3):
        again = gs.fp8_matmul(a, sa, E4M3, B1, b, sb, E4M3, B128, out_dtype=torch.float32)
        assert torch.equal(first, again)


def test_streams_and_graph(dev):
    """Another stream; two captured graphs with workspaces of their own,
    replayed several times with eager work between, inputs changed between."""
    shapes = [(333, 512, 4608), (20, 256, 1024)]
    ops, graphs = [], []
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    for i, (m, n, k) in enumerate(shapes):
        a, sa = _operand(m, k, E4M3, B1, 50 + i, dev)
        b, sb = _operand(n, k, E4M3, B128, 60 + i, dev)
        out = torch.empty(m, n, device=dev)
        ws = torch.empty(max(16, gs.fp8_matmul_workspace_size(m, n, k)), dtype=torch.uint8, device=dev)
        ops.append((a, sa, b, sb, out, ws))
    torch.cuda.synchronize()
    eager = lambda o: gs.fp8_matmul(o[0], o[1], E4M3, B1, o[2], o[3], E4M3, B128,   # noqa: E731
                                    out_dtype=torch.float32)
    for a, sa, b, sb, out, ws in ops:
        gs.fp8_matmul(a, sa, E4M3, B1, b, sb, E4M3, B128, out=out, workspace=ws, stream=side)
    side.synchronize()
    for o in ops:
        assert torch.equal(o[4], eager(o))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gs.fp8_matmul(o[0], o[1], E4M3, B1, o[2], o[3], E4M3, B128, out=o[4], workspace=o[5])
        graphs.append(g)
    for trial in range(4):
        for i, (o, g) in enumerate(zip(ops, graphs)):
            new, _ = _operand(*o[0].shape, E4M3, B1, 70 + 10 * trial + i, dev)
            o[0].copy_(new)
            o[4].zero_()
            g.replay()
        torch.cuda.synchronize()
        for o in ops:
            assert torch.equal(o[4], eager(o)), trial


def test_refusals(dev):
    a, sa = _operand(16, 256, E4M3, B1, 1, dev)
    b, sb = _operand(128, 256, E4M3, B128, 2, dev)
    ok = lambda **kw: gs.fp8_matmul(a, sa, E4M3, B1, b, sb, E4M3, B128, **kw)       # noqa: E731
    out = torch.full((16, 128), 5.0, device=dev)
    with pytest.raises(ValueError, match="columns"):
        gs.fp8_matmul(a[:, :128].contiguous(), sa, E4M3, B1, b, sb, E4M3, B128)
    with pytest.raises(ValueError, match="contiguous"):
        gs.fp8_matmul(a[:, :128], sa, E4M3, B1, b, sb, E4M3, B128)
    with pytest.raises(ValueError, match="a_scales holds"):
        gs.fp8_matmul(a, sa[:15], E4M3, B1, b, sb, E4M3, B128)
    with pytest.raises(ValueError, match="out holds"):
        ok(out=out[:15])
    with pytest.raises(ValueError, match="blocks"):
        gs.fp8_matmul(a, sa, E4M3, gs.FP8_PER_TENSOR, b, sb, E4M3, B128)
    with pytest.raises(TypeError, match="a must be"):
        gs.fp8_matmul(a.float(), sa, E4M3, B1, b, sb, E4M3, B128)
    with pytest.raises(TypeError, match="accumulate"):
        ok(out=out.bfloat16(), accumulate=True)
    with pytest.raises(ValueError, match="accumulate"):
        ok(accumulate=True)
    with pytest.raises(TypeError, match="out is"):
        ok(out=out, out_dtype=torch.bfloat16)
    with pytest.raises(gs.GSError, match="SHAPE"):
        gs.fp8_matmul(a, sa, E4M3, B128, b, sb, E4M3, B128)
    big = torch.zeros(333, 18432, dtype=torch.uint8, device=dev)
    bs = torch.ones(333, 144, device=dev)
    if gs.fp8_matmul_workspace_size(333, 128, 18432):
        w = torch.zeros(128, 18432, dtype=torch.uint8, device=dev)
        with pytest.raises(ValueError, match="workspace holds"):
            gs.fp8_matmul(big, bs, E4M3, B1, w, torch.ones(1, 144, device=dev), E4M3, B128,
                          workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert bool((out == 5).all())
