"""The AdamW reference on the CPU: its FP32 form is near its 64-bit form, its
rounding by chance is unbiased, and E4M3 states follow FP32 states."""
import numpy as np
import torch

import adamw_reference as ref

F = np.float32


def test_codes_are_the_format():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, ref.CODES)


def test_update32_is_update64():
    """Both operands of every sum have the same few roundings: m and v of same
    sign terms within 4 steps of 2^-24, p within the size of its change."""
    rng = np.random.default_rng(1)
    n = 20000
    p, g, m = (rng.standard_normal(n).astype(F) for _ in range(3))
    v = rng.random(n).astype(F) + F(0.01)
    args = (0.1, 3e-3, 7, 0.9, 0.95, 1e-8, F(1024.0), 50.0, 5.0)
    p32, m32, v32, _ = ref.update32(p, g, m, v, *args)
    p64, m64, v64 = ref.update64(p, g, m, v, *args)
    assert np.all(np.abs(v32 - v64) <= 6 * 2.0 ** -24 * v64)
    assert np.all(np.abs(m32 - m64) <= 6 * 2.0 ** -24 * (np.abs(m) + np.abs(g)))
    assert np.all(np.abs(p32 - p64) <= 4 * 2.0 ** -24 * np.abs(p) + 20 * 2.0 ** -24 * np.abs(p64 - p) + 1e-9)


def test_rounding_is_unbiased():
    """The mean of many roundings of one value: of x for m, of x^2 for r; the
    standard error of 400000 draws of a step of 2^-3 is below 2e-4 of it."""
    n = 128 * 3200
    h = ref.hashes(n, 3, 99, 5)
    for value in (1.03, 100.0, 447.9, 0.0051, 2.0 ** -11):
        x = np.full(n, value, dtype=F)
        x[::128] = F(448.0)                       # scale 1
        keep = np.arange(n) % 128 != 0
        c, s = ref.encode(x, h & np.uint64(0xFFFF), False)
        got = ref.decode(c, s, n)[keep].astype(np.float64)
        se = 6 * got.std() / np.sqrt(keep.sum()) + 1e-5 * value
        assert np.all(s == 1) and abs(got.mean() - value) <= se
        c, s = ref.encode(x, h >> np.uint64(16), True)
        got = ref.decode(c, s, n)[keep].astype(np.float64) ** 2
        if value >= 2.0 ** -9:                    # below, r is never stored as 0
            se = 6 * got.std() / np.sqrt(keep.sum()) + 1e-5 * value ** 2
            assert abs(got.mean() - float(F(value)) ** 2) <= se
        else:
            assert np.all(got == 2.0 ** -18)


def test_e4m3_states_follow_fp32_states():
    """1500 steps on gradients whose size drifts by 30 within each group:
    r = sqrt(v) from E4M3 states stays near that of FP32 states (a quarter off
    on average; rounding to nearest loses most of the drift), without bias in
    v over the elements."""
    rng = np.random.default_rng(2)
    n, b1, b2 = 1024, 0.9, 0.999
    m = m32 = np.zeros(n, F)
    v = v32 = np.zeros(n, F)
    cm, sm = ref.encode(m, np.zeros(n, np.uint64), False)
    cv, sv = ref.encode(v, np.zeros(n, np.uint64), True)
    grow = np.exp(rng.uniform(-1.7, 1.7, n))
    p = np.zeros(n, F)
    for t in range(1, 1501):
        g = (rng.standard_normal(n) * grow ** (t / 1500)).astype(F)
        h = ref.hashes(n, 0, 1, t)
        _, m32, v32, _ = ref.update32(p, g, m32, v32, 0, 1e-3, t, b1, b2, 1e-8)
        _, m, _, r = ref.update32(p, g, ref.decode(cm, sm, n), ref.decode(cv, sv, n) ** 2, 0, 1e-3, t,
                                  b1, b2, 1e-8)
        cm, sm = ref.encode(m, h & np.uint64(0xFFFF), False)
        cv, sv = ref.encode(r, h >> np.uint64(16), True)
    v8 = ref.decode(cv, sv, n).astype(np.float64) ** 2
    ratio = v8 / v32
    assert abs(ratio.mean() - 1) < 6 * ratio.std() / np.sqrt(n)
    assert np.abs(np.sqrt(ratio) - 1).mean() < 0.25
