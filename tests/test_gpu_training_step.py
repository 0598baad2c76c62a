"""The operators together, as a mixed-precision step uses them: a linear
layer's forward and both backward products from FP8 casts, the unscale with
its norm, AdamW on the FP32 weights, the loss-scale update, and the new
weights' cast for the next step."""
import numpy as np
import pytest
import torch

import adamw_reference as ref
import loss_scaling_fp8_amd as gs

pytestmark = pytest.mark.gpu

B1, B128, E4M3, E5M2 = gs.FP8_BLOCK_1x128, gs.FP8_BLOCK_128x128, gs.FP8_E4M3, gs.FP8_E5M2


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("bits", [32, 8])
def test_linear_layer_steps(bits, dev):
    """Five steps on a ragged batch; the loss scale overflows the FP16 weight
    gradient in one of them, which is skipped.  Every product is near the
    64-bit product of the unquantized operands.  An element off by at most a
    fraction e of itself makes a product's norm off by about e / sqrt(3) for
    each operand; E4M3's e is 2^-4 and E5M2's 2^-3, so two E4M3 operands give
    at most 0.054 and E4M3 with E5M2 0.084."""
    T, C, O = 333, 512, 384
    gen = torch.Generator().manual_seed(3)
    W = (torch.randn(O, C, generator=gen) * 0.05).to(dev)
    W16 = W.bfloat16()
    dW = torch.empty(O, C, dtype=torch.float16, device=dev)
    g32 = torch.empty(O, C, device=dev)
    if bits == 8:
        m, v = (torch.zeros(O, C, dtype=torch.uint8, device=dev) for _ in range(2))
        ms, vs = (torch.zeros(O * C // 128, device=dev) for _ in range(2))
        plan = gs.gs_adamw_plan([W], [g32], [m], [v], [ms], [vs], [W16], 0.1)
    else:
        m, v = torch.zeros(O, C, device=dev), torch.zeros(O, C, device=dev)
        plan = gs.gs_adamw_plan([W], [g32], [m], [v], copies=[W16], weight_decays=0.1)
    scale = torch.tensor([1024.0], device=dev)
    tracker = torch.zeros(1, dtype=torch.int32, device=dev)
    found = torch.zeros(1, dtype=torch.int32, device=dev)
    skips = torch.zeros(1, dtype=torch.int64, device=dev)
    lr, step = torch.tensor([1e-3], device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    norm_sq = torch.zeros(1, dtype=torch.float64, device=dev)
    for it in range(5):
        x = torch.randn(T, C, generator=gen).to(dev).bfloat16()
        dy = (torch.randn(T, O, generator=gen) * 1e-2).to(dev)
        S = float(scale)
        dy_s = (dy * S).bfloat16() if it != 2 else (dy * 2.0 ** 24).bfloat16()
        xt, xts, xc, xs = gs.fp8_quantize_transposed(x, E4M3, B1, both=True)
        dt, dts, dc, ds = gs.fp8_quantize_transposed(dy_s, E5M2, B1, both=True)
        wt, wts, wc, wsc = gs.fp8_quantize_transposed(W16, E4M3, B128, both=True)
        y = gs.fp8_matmul(xc, xs, E4M3, B1, wc, wsc, E4M3, B128)
        dx = gs.fp8_matmul(dc, ds, E5M2, B1, wt, wts, E4M3, B128)
        gs.fp8_matmul(dt, dts, E5M2, B1, xt, xts, E4M3, B1, out=dW)
        x64, w64, d64 = x.double().cpu(), W16.double().cpu(), dy_s.double().cpu()
        assert _rel(y.cpu(), x64 @ w64.t()) < 0.054
        assert _rel(dx.cpu(), d64 @ w64) < 0.084
        if it != 2:
            assert _rel(dW.cpu(), d64.t() @ x64) < 0.084
        before = (W.clone(), m.clone(), v.clone(), W16.clone())
        sumsq = torch.zeros(2, dtype=torch.int64, device=dev)
        gs.gs_unscale_check_sumsq([dW], [g32], scale, found, sumsq, norm_sq)
        gs.gs_adamw_step(plan, lr, step, beta2=0.95, found_inf=found, norm_sq=norm_sq, max_norm=1.0,
                         seed=9)
        gs.gs_update_scale(scale, tracker, found, 2.0, 0.5, 3, skips)
        torch.cuda.synchronize()
        after = (W, m, v, W16)
        if it == 2:
            assert float(scale) == 512.0 and int(skips) == 1 and int(step) == 2
            assert all(torch.equal(a, b) for a, b in zip(after, before))
            continue
        t = int(step)
        assert t == (it + 1 if it < 2 else it) and torch.equal(W16, W.bfloat16())
        if bits == 32:
            want = ref.update32(before[0].cpu().numpy(), g32.cpu().numpy(), before[1].cpu().numpy(),
                                before[2].cpu().numpy(), 0.1, float(lr), t, 0.9, 0.95, 1e-8,
                                norm_sq=float(norm_sq), max_norm=1.0)
            for got, w in zip((W, m, v), want):
                assert np.array_equal(got.cpu().numpy().view(np.int32), w.view(np.int32))
        assert not torch.equal(W, before[0])


def test_weight_gradient_accumulates_micro_batches(dev):
    """Two micro-batches into one FP32 gradient equal one product over both,
    up to the sums' rounding (tolerance as in test_gpu_matmul.py)."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(512, 256, generator=gen).to(dev).bfloat16()
    dy = torch.randn(512, 384, generator=gen).to(dev).bfloat16()
    whole = None
    total = torch.zeros(384, 256, device=dev)
    parts = []
    for rows in (slice(0, 512), slice(0, 256), slice(256, 512)):
        xt, xs = gs.fp8_quantize_transposed(x[rows].contiguous(), E4M3, B1)
        dt, ds = gs.fp8_quantize_transposed(dy[rows].contiguous(), E5M2, B1)
        if whole is None:
            whole = gs.fp8_matmul(dt, ds, E5M2, B1, xt, xs, E4M3, B1, out_dtype=torch.float32)
            va = gs.fp8_dequantize(dt, E5M2, B1, ds).double().abs().cpu()
            vb = gs.fp8_dequantize(xt, E4M3, B1, xs).double().abs().cpu()
            absum = va @ vb.t()
        else:
            parts.append((dt, xt))
            gs.fp8_matmul(dt, ds, E5M2, B1, xt, xs, E4M3, B1, out=total, accumulate=True)
    tol = 3 * (128 + 4 + 20) * 2.0 ** -23 * absum
    assert bool(((total - whole).double().abs().cpu() <= tol).all())


def test_several_streams(dev):
    """Products, casts and steps on three streams at once, each with its own
    tensors, equal the same calls one after the other."""
    def work(seed):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(200, 256, generator=gen).to(dev)
        w = torch.randn(384, 256, generator=gen).to(dev)
        st = [torch.randn(5000, generator=gen).to(dev) for _ in range(3)] + [torch.zeros(5000, device=dev)]
        plan = gs.gs_adamw_plan([st[0]], [st[1]], [st[2]], [st[3]])
        out = torch.empty(200, 384, device=dev)
        return x, w, st, plan, out, torch.tensor([1e-3], device=dev), torch.zeros(
            1, dtype=torch.int32, device=dev)

    def go(s, stream=None):
        x, w, st, plan, out, lr, step = s
        xc, xs = gs.fp8_quantize(x, E4M3, B1, stream=stream)
        wc, ws = gs.fp8_quantize(w, E4M3, B128, stream=stream)
        for _ in range(3):
            gs.fp8_matmul(xc, xs, E4M3, B1, wc, ws, E4M3, B128, out=out, stream=stream)
            gs.gs_adamw_step(plan, lr, step, stream=stream)
        return xc, xs, wc, ws
    serial, several = [work(i) for i in range(3)], [work(i) for i in range(3)]
    for s in serial:
        go(s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=dev) for _ in several]
    kept = []
    for s, st in zip(several, streams):
        with torch.cuda.stream(st):
            kept.append(go(s))
    torch.cuda.synchronize()
    for a, b in zip(serial, several):
        assert torch.equal(a[4], b[4]) and all(torch.equal(x, y) for x, y in zip(a[2], b[2]))


def test_own_memory_on_another_stream(dev):
    """What a call allocates for another stream (workspace, outputs) is not
    memory that the current stream still uses, nor given back to it early: a
    long chain of calls on a side stream, with the current stream allocating
    and overwriting memory meanwhile."""
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(333, 4608, generator=gen).to(dev)
    w = torch.randn(512, 4608, generator=gen).to(dev)
    xc, xs = gs.fp8_quantize(x, E4M3, B1)
    wc, ws = gs.fp8_quantize(w, E4M3, B128)
    assert gs.fp8_matmul_workspace_size(333, 512, 4608) > 0
    want = gs.fp8_matmul(xc, xs, E4M3, B1, wc, ws, E4M3, B128, out_dtype=torch.float32)
    want_t = gs.fp8_quantize_transposed(x, E4M3, B1)
    side = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        outs = []
        for _ in range(20):
            outs.append((gs.fp8_matmul(xc, xs, E4M3, B1, wc, ws, E4M3, B128, out_dtype=torch.float32,
                                       stream=handle),
                         gs.fp8_quantize_transposed(x, E4M3, B1, stream=handle)))
            for numel in (333 * 512, 333 * 512 * 2, 4608 * 384):
                torch.empty(numel, device=dev).fill_(float("nan"))
        side.synchronize()
        for o, t in outs:
            assert torch.equal(o, want)
            assert all(torch.equal(a, b) for a, b in zip(t, want_t))
        torch.cuda.synchronize()
