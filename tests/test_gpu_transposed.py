"""fp8_quantize_transposed, bit for bit against the CPU oracle's fp8_quantize
of the transposed (zero-padded) matrix, and against the oracle of the matrix
itself for the codes that come with it."""
import numpy as np
import pytest
import torch

import loss_scaling_fp8_amd as gs
import oracle

pytestmark = pytest.mark.gpu

B1, B128 = gs.FP8_BLOCK_1x128, gs.FP8_BLOCK_128x128


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


def _data(rows, cols, dtype, seed, special):
    """Host bits (uint16 BF16 / float32) of normal values over many binades;
    special: NaN, infinities, zeros of both signs and an all-zero column and
    row among them."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-12, 6, (rows, cols)))).astype(np.float32)
    if special and x.size:
        flat = x.reshape(-1)
        at = rng.integers(0, flat.size, max(8, flat.size // 40))
        flat[at] = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-30, -3e38],
                                       dtype=np.float32), at.size)
        x[:, cols // 2] = 0.0
        x[rows // 2] = -0.0
    if dtype == "f32":
        return x
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def _to_dev(h, dev):
    if h.dtype == np.uint16:
        return torch.from_numpy(h.view(np.int16)).view(torch.bfloat16).to(dev)
    return torch.from_numpy(h).to(dev)


def _padded_t(h):
    t = np.zeros((h.shape[1], -(-h.shape[0] // 128) * 128), dtype=h.dtype)
    t[:, :h.shape[0]] = h.T
    return np.ascontiguousarray(t)


def _same_scales(got, want):
    return np.array_equal(got.cpu().numpy().reshape(-1).view(np.uint32), want.reshape(-1).view(np.uint32))


def _check(rows, cols, dtype, fmt, gran, both, dev, special=True, seed=0):
    h = _data(rows, cols, dtype, 1000 * seed + rows + cols, special)
    x = _to_dev(h, dev)
    (c_r, c_c), s_shape = gs.transposed_shapes(rows, cols, gran)
    guard = 256
    flat = torch.full((c_r * c_c + 2 * guard,), 0xAA, dtype=torch.uint8, device=dev)
    codes_t = flat[guard:guard + c_r * c_c].view(c_r, c_c)
    sflat = torch.full((s_shape[0] * s_shape[1] + 16,), -5.0, device=dev)
    scales_t = sflat[8:8 + s_shape[0] * s_shape[1]].view(s_shape)
    nf = torch.zeros(1, dtype=torch.int32, device=dev)
    out = gs.fp8_quantize_transposed(x, fmt, gran, both=both, codes_t=codes_t, scales_t=scales_t,
                                     nonfinite=nf)
    torch.cuda.synchronize()
    rc, rs, rnf = oracle.quantize(_padded_t(h), fmt, gran)
    assert np.array_equal(codes_t.cpu().numpy(), rc.reshape(c_r, c_c))
    assert _same_scales(scales_t, rs)
    assert int(nf) == rnf
    assert bool((flat[:guard] == 0xAA).all()) and bool((flat[guard + c_r * c_c:] == 0xAA).all())
    assert bool((sflat[:8] == -5).all()) and bool((sflat[8 + s_shape[0] * s_shape[1]:] == -5).all())
    if both:
        rc, rs, _ = oracle.quantize(h, fmt, gran)
        assert np.array_equal(out[2].cpu().numpy(), rc.reshape(rows, cols))
        assert _same_scales(out[3], rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [gs.FP8_E4M3, gs.FP8_E5M2])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (5, 7), (127, 130), (128, 128), (129, 33),
                                       (300, 1000), (640, 264), (1003, 76)])
def test_any_shape(rows, cols, fmt, dtype, dev):
    _check(rows, cols, dtype, fmt, B1, False, dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [gs.FP8_E4M3, gs.FP8_E5M2])
@pytest.mark.parametrize("rows,cols", [(1, 128), (77, 256), (128, 384), (385, 640)])
def test_both(rows, cols, fmt, dtype, dev):
    _check(rows, cols, dtype, fmt, B1, True, dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [gs.FP8_E4M3, gs.FP8_E5M2])
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 640), (384, 128)])
def test_tiles(rows, cols, both, fmt, dtype, dev):
    _check(rows, cols, dtype, fmt, B128, both, dev)


def test_clean_input_leaves_the_flag(dev):
    for gran in (B1, B128):
        _check(256, 256, "bf16", gs.FP8_E4M3, gran, True, dev, special=False)


def test_full_size(dev):
    """The activations' full shape, on the GPU against the row-major cast of
    the transposed tensor (itself pinned to the oracle)."""
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(16384, 7168, device=dev, generator=g).bfloat16()
    ct, st, c, s = gs.fp8_quantize_transposed(x, gs.FP8_E4M3, B1, both=True)
    xt = x.t().contiguous()
    wc, ws = gs.fp8_quantize(xt, gs.FP8_E4M3, B1)
    assert torch.equal(ct, wc) and torch.equal(st, ws)
    wc, ws = gs.fp8_quantize(x, gs.FP8_E4M3, B1)
    assert torch.equal(c, wc) and torch.equal(s, ws)


def test_graph_and_stream(dev):
    x = torch.randn(300, 256, device=dev)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    out = gs.fp8_quantize_transposed(x, gs.FP8_E5M2, B1, both=True, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.fp8_quantize_transposed(x, gs.FP8_E5M2, B1, codes_t=out[0], scales_t=out[1], codes=out[2],
                                   scales=out[3])
    for _ in range(3):
        x.copy_(torch.randn(300, 256, device=dev))
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, gs.fp8_quantize_transposed(x, gs.FP8_E5M2, B1, both=True)):
            assert torch.equal(a, b)


def test_refusals(dev):
    x = torch.ones(256, 256, dtype=torch.bfloat16, device=dev)
    q = gs.fp8_quantize_transposed
    with pytest.raises(ValueError, match="contiguous"):
        q(x.t()[:, ::2], gs.FP8_E4M3, B1)
    with pytest.raises(ValueError, match="codes_t holds"):
        q(x[:129], gs.FP8_E4M3, B1, codes_t=torch.empty(256, 129, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="scales_t holds"):
        q(x, gs.FP8_E4M3, B1, scales_t=torch.empty(256, 1, device=dev))
    with pytest.raises(ValueError, match="blocks"):
        q(x, gs.FP8_E4M3, gs.FP8_PER_TENSOR)
    with pytest.raises(gs.GSError, match="SHAPE"):
        q(x[:, :100].contiguous(), gs.FP8_E4M3, B1, both=True,
          scales=torch.empty(256, 2, device=dev))
    with pytest.raises(gs.GSError, match="SHAPE"):
        q(x[:100], gs.FP8_E4M3, B128, scales_t=torch.empty(2, 2, device=dev))
    with pytest.raises(TypeError):
        q(x.half(), gs.FP8_E4M3, B1)
    assert q(x[:0], gs.FP8_E4M3, B1)[0].shape == (256, 0)
