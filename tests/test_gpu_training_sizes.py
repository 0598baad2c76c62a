"""The training operators past 2^32 elements: operands, results, both casts and
a tensor of an optimizer step whose last elements lie past a 32-bit offset."""
import numpy as np
import pytest
import torch

import adamw_reference as ref
import loss_scaling_fp8_amd as gs
import test_gpu_matmul as products

pytestmark = pytest.mark.gpu

B1, B128, E4M3 = gs.FP8_BLOCK_1x128, gs.FP8_BLOCK_128x128, gs.FP8_E4M3
F = np.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def _big_codes(rows, k, dev):
    """Any finite E4M3 codes, and scales of 1x128 blocks."""
    gen = torch.Generator(device=dev).manual_seed(rows)
    c = torch.randint(0, 256, (rows, k), dtype=torch.uint8, device=dev, generator=gen)
    c[(c & 0x7F) == 0x7F] = 0
    return c, torch.rand(rows, k // 128, device=dev, generator=gen) + 0.5


def _check_part(out, a, sa, b, sb, b_gran, dev):
    va, vb = products._values(a, sa, E4M3, B1), products._values(b, sb, E4M3, b_gran)
    products._check(out, va @ vb.t(), va.abs() @ vb.abs().t(), a.shape[1] // 128,
                    cut=products._cut(va, vb, dev) if out.dtype != torch.float32 else None)


def test_result_past_32_bits(dev):
    m, n, k = 65700, 65664, 128
    a, sa = _big_codes(m, k, dev)
    b, sb = products._operand(n, k, E4M3, B128, 5, dev)
    out = gs.fp8_matmul(a, sa, E4M3, B1, b, sb, E4M3, B128)
    assert out.numel() > 1 << 32
    for rows in (slice(0, 4), slice(32766, 32770), slice(m - 4, m)):
        _check_part(out[rows], a[rows].contiguous(), sa[rows].contiguous(), b, sb, B128, dev)


@pytest.mark.parametrize("big", ["a", "b"])
def test_operand_past_32_bits(big, dev):
    rows, k = 524416, 8320
    c, s = _big_codes(rows, k, dev)
    assert c.numel() > 1 << 32
    o, so = products._operand(128 if big == "a" else 2, k, E4M3, B1, 6, dev)
    if big == "a":
        out = gs.fp8_matmul(c, s, E4M3, B1, o, so, E4M3, B1)
    else:
        out = gs.fp8_matmul(o, so, E4M3, B1, c, s, E4M3, B1, out_dtype=torch.float32)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        cp, sp = c[part].contiguous(), s[part].contiguous()
        if big == "a":
            _check_part(out[part], cp, sp, o, so, B1, dev)
        else:
            _check_part(out[:, part], o, so, cp, sp, B1, dev)


@pytest.mark.parametrize("gran", [B1, B128])
def test_transposed_past_32_bits(gran, dev):
    rows, cols = 65792, 65664
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    x.normal_(generator=torch.Generator(device=dev).manual_seed(2))
    assert x.numel() > 1 << 32
    ct, st, c, s = gs.fp8_quantize_transposed(x, E4M3, gran, both=True)
    for lo in (0, 32768, cols - 128):
        want, wscales = gs.fp8_quantize(x[:, lo:lo + 128].t().contiguous(), E4M3, gran)
        assert torch.equal(ct[lo:lo + 128], want)
        per = 128 if gran == B1 else 1
        at = lo if gran == B1 else lo // 128
        assert torch.equal(st.view(-1, rows // 128)[at:at + per], wscales.view(per, -1))
    for lo in (0, rows - 128):
        want, wscales = gs.fp8_quantize(x[lo:lo + 128].contiguous(), E4M3, gran)
        assert torch.equal(c[lo:lo + 128], want)
        per = 128 if gran == B1 else 1
        at = lo if gran == B1 else lo // 128
        assert torch.equal(s.view(-1, cols // 128)[at:at + per], wscales.view(per, -1))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_32_bits(bits, dev):
    """The elements around offset 2^32 and the ragged end, bit for bit."""
    n = (1 << 32) + 5000
    first = (1 << 32) - 1280
    w = n - first
    rng = np.random.default_rng(bits)
    p = torch.zeros(n, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    hp, hg = rng.standard_normal(w).astype(F), torch.from_numpy(rng.standard_normal(w).astype(F)).bfloat16()
    hm, hv = rng.standard_normal(w).astype(F), rng.random(w).astype(F)
    p[first:].copy_(torch.from_numpy(hp))
    g[first:].copy_(hg)
    step, lr = torch.zeros(1, dtype=torch.int32, device=dev), torch.tensor([1e-2], device=dev)
    if bits == 8:
        nb = -(-n // 128)
        h16 = rng.integers(0, 1 << 16, w).astype(np.uint64)
        (cm, sm), (cv, sv) = ref.encode(hm, h16, False), ref.encode(np.sqrt(hv), h16, True)
        m, v = (torch.zeros(n, dtype=torch.uint8, device=dev) for _ in range(2))
        ms, vs = (torch.zeros(nb, device=dev) for _ in range(2))
        for t, h in ((m, cm), (v, cv), (ms, sm), (vs, sv)):
            t[t.numel() - h.size:].copy_(torch.from_numpy(h))
        hm, r = ref.decode(cm, sm, w), ref.decode(cv, sv, w)
        hv = r * r
        plan = gs.gs_adamw_plan([p], [g], [m], [v], [ms], [vs], weight_decays=0.1)
    else:
        m, v = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
        m[first:].copy_(torch.from_numpy(hm))
        v[first:].copy_(torch.from_numpy(hv))
        plan = gs.gs_adamw_plan([p], [g], [m], [v], weight_decays=0.1)
    gs.gs_adamw_step(plan, lr, step, beta2=0.95, seed=11)
    p1, m1, v1, r1 = ref.update32(hp, hg.float().numpy(), hm, hv, 0.1, float(lr), 1, 0.9, 0.95, 1e-8)
    torch.cuda.synchronize()
    assert np.array_equal(p[first:].cpu().numpy().view(np.int32), p1.view(np.int32))
    assert not bool(p[:first].any())
    if bits == 8:
        hs = ref.hashes(w, 0, 11, 1, first)
        for t, ts, (codes, scales) in ((m, ms, ref.encode(m1, hs & np.uint64(0xFFFF), False)),
                                       (v, vs, ref.encode(r1, hs >> np.uint64(16), True))):
            assert np.array_equal(t[first:].cpu().numpy(), codes)
            assert np.array_equal(ts[first // 128:].cpu().numpy().view(np.int32), scales.view(np.int32))
    else:
        assert np.array_equal(m[first:].cpu().numpy().view(np.int32), m1.view(np.int32))
        assert np.array_equal(v[first:].cpu().numpy().view(np.int32), v1.view(np.int32))
