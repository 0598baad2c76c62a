"""Workloads of the training operators that stand next to the FP8 casts and
the loss scaling: the block-scaled FP8 matrix product, the transposing block
quantizer that makes its backward operands, and the multi-tensor AdamW step
with FP32 or FP8 states.

run() computes them in plain FP32 torch operations, or, where `own` is set,
through the package's entry points; exact() computes the same results in 64
bits from the definitions.  Inputs come from a seed and are made on the GPU.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MAX = {"e4m3": 448.0, "e5m2": 57344.0}
FLOOR = 1e-12


# ------------------------------------------------------------------ cases
def _matmul(name, m, n, k, pair, out, accumulate=False, a_fmt="e4m3", b_fmt="e4m3"):
    """pair: granularities of a and b.  "act-weight": a 1x128 blocks, b
    128x128 blocks; "act-act": both 1x128."""
    return {"name": name, "op": "matmul", "m": m, "n": n, "k": k, "pair": pair, "out": out,
            "accumulate": accumulate, "a_fmt": a_fmt, "b_fmt": b_fmt}


def _transposed(name, rows, cols, dtype, fmt, gran, both):
    return {"name": name, "op": "transposed", "rows": rows, "cols": cols, "dtype": dtype,
            "fmt": fmt, "gran": gran, "both": both}


def _adamw(name, tensors, total, bits, grad, copy, scaled=False, shards=0):
    """A list of `tensors` tensors with `total` elements in all, or (shards >
    0) one rank's share of the Llama-3-8B list cut into that many."""
    return {"name": name, "op": "adamw", "tensors": tensors, "total": total, "bits": bits,
            "grad": grad, "copy": copy, "scaled": scaled, "shards": shards}


def listed():
    return [
        # one token through the key projection of a Llama-3-8B layer: latency
        _matmul("token 1x1024x4096", 1, 1024, 4096, "act-weight", "bf16"),
        # a decode batch through the largest weight of the block benchmark
        _matmul("decode 16x18432x7168", 16, 18432, 7168, "act-weight", "bf16"),
        # a ragged prefill chunk: few row tiles, a long K
        _matmul("chunk 333x7168x18432", 333, 7168, 18432, "act-weight", "bf16"),
        # forward of a training batch, the block benchmark's own shapes
        _matmul("forward 16384x18432x7168", 16384, 18432, 7168, "act-weight", "bf16"),
        # gradient of the input: E5M2 gradients against the transposed weight, ragged rows
        _matmul("dgrad 4099x7168x18432", 4099, 7168, 18432, "act-weight", "bf16", a_fmt="e5m2"),
        # gradient of the weight, added to the FP32 gradient of earlier micro-batches
        _matmul("wgrad 14336x4096x8192", 14336, 4096, 8192, "act-act", "f32", True, a_fmt="e5m2"),
        # activations for the forward pass and, transposed, for the weight's gradient
        _transposed("transpose 16384x7168", 16384, 7168, "bf16", "e4m3", "1x128", True),
        # FP32 gradients of a ragged batch, transposed only
        _transposed("transpose 1003x4160", 1003, 4160, "f32", "e5m2", "1x128", False),
        # a small model's list, where launches count
        _adamw("adamw 1M", 16, 1 << 20, 32, "f32", "bf16"),
        # one of 16 ranks' share of the Llama-3-8B list, FP32 states
        _adamw("adamw llama/16", 0, 0, 32, "f32", "bf16", shards=16),
        # FP8 states, a mid-sized list of odd lengths, FP16 gradients that still carry the loss scale
        _adamw("adamw8 20M", 63, 20_000_003, 8, "f16", "f16", scaled=True),
        # FP8 states, one of 32 ranks' share of the Llama-3-8B list
        _adamw("adamw8 llama/32", 0, 0, 8, "f32", "bf16", shards=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("matmul", "matmul", "matmul", "transposed", "adamw", "adamw"))
    if op == "matmul":
        kind = rng.choice(("forward", "dgrad", "wgrad"))
        m = _log_int(rng, 1, 16384)
        if kind == "wgrad":
            m, n = _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        else:
            n = 128 * _log_int(rng, 1, 144)
        k = 128 * _log_int(rng, 1, 144)
        while m * n * k > 2_000_000_000_000:
            m = (m + 1) // 2
        out = rng.choice(("f32", "f16")) if kind == "wgrad" else rng.choice(("bf16", "f32"))
        c = _matmul("", m, n, k, "act-act" if kind == "wgrad" else "act-weight", out,
                    out == "f32" and kind == "wgrad" and rng.random() < 0.5,
                    a_fmt="e4m3" if kind == "forward" else "e5m2")
    elif op == "transposed":
        gran = rng.choice(("1x128", "1x128", "128x128"))
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 1, 18432)
        both = gran == "128x128" or rng.random() < 0.5
        if both:
            cols = max(128, cols // 128 * 128)
        if gran == "128x128":
            rows = max(128, rows // 128 * 128)
        while rows * cols > 16384 * 7168:
            rows = max(128, rows // 256 * 128) if gran == "128x128" else rows // 2
        c = _transposed("", rows, cols, rng.choice(("bf16", "f32")), rng.choice(("e4m3", "e5m2")),
                        gran, both)
    else:
        total = _log_int(rng, 5000, 100_000_000)
        scaled = rng.random() < 0.5
        c = _adamw("", rng.randint(1, min(300, total // 1000)), total, rng.choice((32, 8)),
                   "f16" if scaled else rng.choice(("f32", "bf16")),
                   rng.choice(("none", "bf16", "f16")), scaled)
    del c["name"]
    return c


def _llama_sizes():
    """The 291 tensors of the Llama-3-8B gradient list."""
    layer = [4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096,
             4096 * 14336, 4096, 4096]
    return [128256 * 4096] + layer * 32 + [4096, 128256 * 4096]


def _sizes(case):
    if case["shards"]:
        return [-(-n // case["shards"]) for n in _llama_sizes()]
    rng = random.Random(case["tensors"] * 1_000_003 + case["total"])
    weights = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    scale = (case["total"] - case["tensors"]) / sum(weights)
    sizes = [1 + int(w * scale) for w in weights]
    sizes[-1] += case["total"] - sum(sizes)
    return sizes


# ------------------------------------------------------------------ inputs
def _block_codes(x, gran, fmt):
    """FP8 codes (uint8) and scales of x at 1x128 or 128x128 granularity."""
    rows, cols = x.shape
    if gran == "1x128":
        b = x.view(rows, cols // 128, 128)
        amax = b.abs().amax(-1, keepdim=True)
    else:
        b = x.view(rows // 128, 128, cols // 128, 128)
        amax = b.abs().amax((1, 3), keepdim=True)
    s = _scale(amax, fmt)
    codes = (b / s).clamp(-MAX[fmt], MAX[fmt]).to(FP8[fmt]).view(torch.uint8).view(rows, cols)
    return codes, s.view(rows, -1) if gran == "1x128" else s.view(rows // 128, cols // 128)


def _scale(amax, fmt):
    """max(amax, 1e-12) / MAX as an FP32 quotient (torch multiplies by the
    reciprocal where a tensor is divided by a Python number)."""
    return amax.clamp_min(FLOOR) / torch.full_like(amax, MAX[fmt])


def _values(rows, cols, sigma, gen):
    """Normal values with a few large outliers, as activations and weights have."""
    x = torch.randn(rows, cols, device=DEV, generator=gen)
    far = torch.rand(rows, cols, device=DEV, generator=gen) < 1e-4
    return torch.where(far, x * 500.0, x).mul_(sigma)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        grad = case["a_fmt"] == "e5m2"
        st["a"], st["a_s"] = _block_codes(_values(m, k, 1e-3 if grad else 1.0, gen), "1x128",
                                          case["a_fmt"])
        st["b_gran"] = "1x128" if case["pair"] == "act-act" else "128x128"
        pad = -n % 128 if st["b_gran"] == "128x128" else 0
        b = _values(n + pad, k, 1.0 if case["pair"] == "act-act" else 0.02, gen)
        st["b"], st["b_s"] = _block_codes(b, st["b_gran"], case["b_fmt"])
        st["c"] = torch.zeros(m, n, dtype=TYPES[case["out"]], device=DEV)
        if case["accumulate"]:
            st["c"].copy_(torch.randn(m, n, device=DEV, generator=gen) * 1e-2)
        if own:
            import loss_scaling_fp8_amd as gs
            st["ws"] = torch.empty(gs.fp8_matmul_workspace_size(m, n, k), dtype=torch.uint8,
                                   device=DEV)
    elif case["op"] == "transposed":
        st["x"] = _values(case["rows"], case["cols"], 1.0, gen).to(TYPES[case["dtype"]])
    else:
        sizes = _sizes(case)
        # flat buffers with every tensor at a multiple of 128 elements
        places = [0]
        for n in sizes:
            places.append(places[-1] + -(-n // 128) * 128)
        total = places[-1]
        cut = lambda flat: [flat[o:o + n] for o, n in zip(places, sizes)]  # noqa: E731
        blocks = lambda flat: [flat[o // 128:(o + n + 127) // 128]  # noqa: E731
                               for o, n in zip(places, sizes)]
        S = 65536.0 if case["scaled"] else 1.0
        mag = torch.exp(torch.randn(total, device=DEV, generator=gen) - 7.0)
        g = (torch.randn(total, device=DEV, generator=gen) * mag * S).to(TYPES[case["grad"]])
        p = torch.randn(total, device=DEV, generator=gen) * 0.02
        # moments of an optimizer that has run for a while
        m = (torch.randn(total, device=DEV, generator=gen) * mag * 0.3)
        v = (torch.rand(total, device=DEV, generator=gen) + 0.5) * mag * mag
        del mag
        st["flat"] = {"p": p}
        st["g"] = cut(g)
        if case["bits"] == 8:
            for name, x in (("m", m), ("v", v.sqrt_())):
                b = x.view(-1, 128)
                s = _scale(b.abs().amax(-1, keepdim=True), "e4m3")
                st["flat"][name] = (b / s).clamp(-448.0, 448.0).to(FP8["e4m3"]).view(-1)
                st["flat"][name + "_s"] = s.view(-1)
                st[name + "_s"] = blocks(st["flat"][name + "_s"])
            del b, s, x
        else:
            st["flat"]["m"], st["flat"]["v"] = m, v
        del m, v
        if case["copy"] != "none":
            st["flat"]["copy"] = torch.zeros(total, dtype=TYPES[case["copy"]], device=DEV)
            st["copy_t"] = cut(st["flat"]["copy"])
        st["p"] = cut(st["flat"]["p"])
        codes = lambda t: t.view(torch.uint8) if case["bits"] == 8 else t  # noqa: E731
        st["m"], st["v"] = cut(codes(st["flat"]["m"])), cut(codes(st["flat"]["v"]))
        # no decay for the short tensors (norms, biases)
        st["wd"] = [0.1 if n > 8192 else 0.0 for n in sizes]
        st["lr"] = torch.tensor([3e-4], device=DEV)
        st["step"] = torch.tensor([41], dtype=torch.int32, device=DEV)
        st["found"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        st["scale"] = torch.tensor([S], device=DEV)
        norm = torch.stack([t.double().square().sum() for t in st["g"]]).sum() / (S * S)
        st["norm_sq"] = norm.view(1)
        st["max_norm"] = 0.7 * math.sqrt(float(norm))
        st["hyper"] = (0.9, 0.95, 1e-8)
        st["seed"] = seed & 0xFFFFFFFF
        if own:
            import loss_scaling_fp8_amd as gs
            st["plan"] = gs.gs_adamw_plan(st["p"], st["g"], st["m"], st["v"],
                                          exp_avg_scales=st.get("m_s"),
                                          exp_avg_sq_scales=st.get("v_s"),
                                          copies=st.get("copy_t"), weight_decays=st["wd"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if st["op"] == "matmul":
        return _run_matmul(st)
    if st["op"] == "transposed":
        return _run_transposed(st)
    return _run_adamw(st)


def _decode(codes, scales, gran, fmt, dtype=torch.float32):
    """The values that codes [rows, cols] stand for."""
    rows, cols = codes.shape
    v = codes.view(FP8[fmt]).to(dtype)
    s = scales.to(dtype)
    if gran == "1x128":
        return (v.view(rows, cols // 128, 128) * s.view(rows, cols // 128, 1)).view(rows, cols)
    v = v.view(rows // 128, 128, cols // 128, 128)
    return (v * s.view(rows // 128, 1, cols // 128, 1)).view(rows, cols)


def _run_matmul(st):
    if own:
        import loss_scaling_fp8_amd as gs
        fmt = {"e4m3": gs.FP8_E4M3, "e5m2": gs.FP8_E5M2}
        gran = {"1x128": gs.FP8_BLOCK_1x128, "128x128": gs.FP8_BLOCK_128x128}
        return gs.fp8_matmul(st["a"], st["a_s"], fmt[st["a_fmt"]], gs.FP8_BLOCK_1x128, st["b"],
                             st["b_s"], fmt[st["b_fmt"]], gran[st["b_gran"]], out=st["c"],
                             accumulate=st["accumulate"], workspace=st["ws"])
    a = _decode(st["a"], st["a_s"], "1x128", st["a_fmt"])
    b = _decode(st["b"], st["b_s"], st["b_gran"], st["b_fmt"])
    c = a @ b.t()
    st["c"].copy_(st["c"] + c if st["accumulate"] else c)
    return st["c"]


def _to_fp8(y, fmt):
    return y.clamp(-MAX[fmt], MAX[fmt]).to(FP8[fmt])


def _padded(x):
    """x with its rows padded with zeros to a multiple of 128."""
    pad = -x.shape[0] % 128
    return torch.cat([x, x.new_zeros(pad, x.shape[1])]) if pad else x


def _run_transposed(st):
    if own:
        import loss_scaling_fp8_amd as gs
        fmt = {"e4m3": gs.FP8_E4M3, "e5m2": gs.FP8_E5M2}[st["fmt"]]
        gran = {"1x128": gs.FP8_BLOCK_1x128, "128x128": gs.FP8_BLOCK_128x128}[st["gran"]]
        out = gs.fp8_quantize_transposed(st["x"], fmt, gran, both=st["both"])
        # codes as the FP8 values that they are
        return [t.view(FP8[st["fmt"]]) if t.dtype == torch.uint8 else t for t in out]
    fmt = st["fmt"]
    x = _padded(st["x"].float())
    rows, cols = x.shape
    if st["gran"] == "1x128":
        b = x.view(rows // 128, 128, cols)
        s = _scale(b.abs().amax(1, keepdim=True), fmt)
        codes_t = _to_fp8(b / s, fmt).view(rows, cols).t().contiguous()
        out = [codes_t, s.view(rows // 128, cols).t().contiguous()]
        if st["both"]:
            x = st["x"].float()
            b = x.view(x.shape[0], cols // 128, 128)
            s = _scale(b.abs().amax(-1, keepdim=True), fmt)
            out += [_to_fp8(b / s, fmt).view(x.shape), s.view(x.shape[0], cols // 128)]
        return out
    b = x.view(rows // 128, 128, cols // 128, 128)
    s = _scale(b.abs().amax((1, 3), keepdim=True), fmt)
    codes = _to_fp8(b / s, fmt).view(rows, cols)
    s = s.view(rows // 128, cols // 128)
    out = [codes.t().contiguous(), s.t().contiguous()]
    return out + [codes, s] if st["both"] else out


def _mix32(x):
    """A 32-bit integer hash (lowbias32) of int64 values in [0, 2^32)."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _hash(n, index, seed, t):
    """32 random bits for each of a tensor's n elements (n < 2^32)."""
    key = _mix32(_mix32(_mix32(torch.tensor(seed, device=DEV)) ^ t.long()) ^ index)
    return _mix32(torch.arange(n, device=DEV) ^ _mix32(key))


def _quantum(y):
    """Spacing of the E4M3 values at |y| <= 448: 2^(max(floor(log2 |y|), -6) - 3)."""
    e = torch.frexp(y)[1] - 1
    e = torch.where(y == 0, -6, e).clamp_min(-6)
    return torch.ldexp(torch.ones_like(y), e - 3)


def _blocks(x):
    """x [n] as rows of 128, the last one padded with zeros."""
    pad = -x.numel() % 128
    return (torch.cat([x, x.new_zeros(pad)]) if pad else x).view(-1, 128)


def _store8(x, scales, codes, u, squared):
    """Rounds x [n] >= the block scales to E4M3 by chance: up when the
    fraction towards the next value (of x, or of x^2 where `squared`) is
    above u; a positive value never becomes 0 where `squared`."""
    n = x.numel()
    b = _blocks(x)
    s = _scale(b.abs().amax(-1, keepdim=True), "e4m3")
    y = (b.abs() / s).clamp_max(448.0).view(-1)[:n]
    q = _quantum(y)
    y0 = torch.floor(y / q) * q
    if squared:
        up = (y - y0) * (y + y0) > u * (q * (y0 + y0 + q))
        y = torch.where(up, y0 + q, y0)
        y = torch.where((y == 0) & (x > 0), q, y)
    else:
        up = (y - y0) > u * q
        y = torch.where(up, y0 + q, y0)
    codes.copy_(torch.copysign(y, x).to(FP8["e4m3"]).view(torch.uint8))
    scales.copy_(s.view(-1))


def _load8(codes, scales):
    v = _blocks(codes.view(FP8["e4m3"]).float())
    return (v * scales.view(-1, 1)).view(-1)[:codes.numel()]


def _adamw_tensor(st, i, t, mul, size, rbc2):
    b1, b2, eps = st["hyper"]
    p, g = st["p"][i], st["g"][i].float() * mul
    bits8 = st["bits"] == 8
    if bits8:
        m = _load8(st["m"][i], st["m_s"][i])
        v = _load8(st["v"][i], st["v_s"][i]).square()
    else:
        m, v = st["m"][i], st["v"][i]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = v.sqrt()
    lrwd = st["lr"] * st["wd"][i]
    p.copy_(p * (1.0 - lrwd) - (m / (r * rbc2 + eps)) * size)
    if bits8:
        h = _hash(p.numel(), i, st["seed"], t)
        _store8(m, st["m_s"][i], st["m"][i], ((h & 0xFFFF) * 2 + 1).float() * 2.0 ** -17, False)
        _store8(r, st["v_s"][i], st["v"][i], ((h >> 16) * 2 + 1).float() * 2.0 ** -17, True)
    else:
        st["m"][i].copy_(m)
        st["v"][i].copy_(v)
    if st["copy"] != "none":
        st["copy_t"][i].copy_(p)


def _run_adamw(st):
    b1, b2, eps = st["hyper"]
    if own:
        import loss_scaling_fp8_amd as gs
        gs.gs_adamw_step(st["plan"], st["lr"], st["step"], beta1=b1, beta2=b2, eps=eps,
                         scale=st["scale"] if st["scaled"] else None, found_inf=st["found"],
                         norm_sq=st["norm_sq"], max_norm=st["max_norm"], seed=st["seed"])
        return {**st["flat"], "step": st["step"]}
    t = st["step"] + 1
    coef = (st["max_norm"] / (st["norm_sq"].sqrt() + 1e-6)).clamp_max(1.0)
    mul = ((1.0 / st["scale"]).double() * coef).float()
    size = (st["lr"].double() / (1.0 - torch.pow(b1, t.double()))).float()
    rbc2 = (1.0 / (1.0 - torch.pow(b2, t.double())).sqrt()).float()
    [_adamw_tensor(st, i, t, mul, size, rbc2) for i in range(len(st["p"]))]
    st["step"].add_(1)
    return {**st["flat"], "step": st["step"]}


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["out"] == "f32" else 2
        scales = m * (k // 128) + (n if case["pair"] == "act-act" else -(-n // 128)) * (k // 128)
        return {"bytes": m * k + n * k + 4 * scales + m * n * size * (2 if case["accumulate"] else 1),
                "flops": 2 * m * n * k}
    if case["op"] == "transposed":
        rows, cols = case["rows"], case["cols"]
        pad = -(-rows // 128) * 128
        size = 4 if case["dtype"] == "f32" else 2
        per = 128 if case["gran"] == "1x128" else 16384
        b = rows * cols * size + pad * cols * (1 + 4 / per)
        if case["both"]:
            b += rows * cols * (1 + 4 / per)
        return {"bytes": int(b), "flops": 4 * rows * cols}
    n = sum(_sizes(case))
    state = 4 * 4 if case["bits"] == 32 else 4 * (1 + 4 / 128)
    b = 8 + (4 if case["grad"] == "f32" else 2) + state + (0 if case["copy"] == "none" else 2)
    return {"bytes": int(n * b), "flops": 16 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "matmul":
        return _exact_matmul(st)
    if case["op"] == "transposed":
        return _exact_transposed(st)
    return _exact_adamw(st)


def _exact_matmul(st):
    k = st["k"]
    a = st["a"].view(FP8[st["a_fmt"]]).double()
    a *= st["a_s"].double().repeat_interleave(128, 1)
    b = st["b"].view(FP8[st["b_fmt"]]).double()
    if st["b_gran"] == "128x128":
        b *= st["b_s"].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        b *= st["b_s"].double().repeat_interleave(128, 1)
    assert a.shape[1] == b.shape[1] == k
    out = torch.mm(a, b.t().contiguous())
    return out + st["c"].double() if st["accumulate"] else out


def _round_fp8(y, fmt):
    """The FP8 value nearest to y (64 bits), ties to even, past the maximum
    the maximum."""
    frac, low = (3, -6) if fmt == "e4m3" else (2, -14)
    y = y.clamp(-MAX[fmt], MAX[fmt])
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** (low - 8))))
    q = torch.pow(2.0, e.clamp_min(low) - frac)
    return torch.round(y / q) * q


def _exact_transposed(st):
    """From the cast's definition: scales and quotients are FP32 values (the
    64-bit quotient of two FP32 values, rounded to FP32, is the FP32
    quotient)."""
    top, fmt = MAX[st["fmt"]], st["fmt"]
    x = st["x"].double()

    def of(t, axis0, axis1):
        """codes and scales of t with blocks of axis0 x axis1"""
        r, c = t.shape
        b = t.reshape(r // axis0, axis0, c // axis1, axis1)
        amax = b.abs().amax((1, 3)).float().clamp_min(FLOOR).double()
        s = (amax / top).float().double()
        y = (b / s[:, None, :, None]).float().double()
        return _round_fp8(y, fmt).reshape(r, c), s

    xt = _padded(x).t().contiguous()
    blocks = (1, 128) if st["gran"] == "1x128" else (128, 128)
    codes_t, s_t = of(xt, *blocks)
    out = [codes_t, s_t]
    if st["both"]:
        codes, s = of(x, *blocks)
        out += [codes, s]
    return out


def _exact_adamw(st):
    b1, b2, eps = st["hyper"]
    t = int(st["step"]) + 1
    lr, S = float(st["lr"]), float(st["scale"])
    coef = min(1.0, st["max_norm"] / (math.sqrt(float(st["norm_sq"])) + 1e-6))
    out = {k: (x.double() if x.dtype.is_floating_point else x) for k, x in st["flat"].items()}
    place = 0
    for i, (p, g) in enumerate(zip(st["p"], st["g"])):
        n = p.numel()
        at, nb = slice(place, place + n), -(-n // 128)
        sc = slice(place // 128, place // 128 + nb)
        spread = lambda s: s.double().repeat_interleave(128)[:n]  # noqa: E731
        m, v = out["m"][at], out["v"][at]
        if st["bits"] == 8:
            m = m * spread(st["m_s"][i])
            v = (v * spread(st["v_s"][i])) ** 2
        d = g.double() * (coef / S)
        m = b1 * m + (1 - b1) * d
        v = b2 * v + (1 - b2) * d * d
        new = out["p"][at] * (1 - lr * st["wd"][i])
        new -= lr / (1 - b1 ** t) * m / (v.sqrt() / math.sqrt(1 - b2 ** t) + eps)
        out["p"][at] = new
        if "copy" in out:
            out["copy"][at] = new
        if st["bits"] == 8:
            key = _mix32(_mix32(_mix32(torch.tensor(st["seed"], device=DEV)) ^ t) ^ i)
            h = _mix32(torch.arange(n, device=DEV) ^ _mix32(key))
            for name, x, bits in (("m", m, h & 0xFFFF), ("v", v.sqrt(), h >> 16)):
                rows = torch.nn.functional.pad(x, (0, nb * 128 - n)).view(nb, 128)
                s = rows.abs().amax(1).clamp_min(FLOOR) / 448.0
                y = x.abs() / s.repeat_interleave(128)[:n]
                y = y.clamp_max(448.0)
                e = torch.floor(torch.log2(y.clamp_min(2.0 ** -6)))
                q = torch.pow(2.0, e - 3)
                low = torch.floor(y / q) * q
                f = (y - low) / q if name == "m" else (y * y - low * low) / ((low + q) ** 2 - low * low)
                r = torch.where(f > (bits.double() + 0.5) / 65536, low + q, low)
                if name == "v":
                    r = torch.where((r == 0) & (x > 0), q, r)
                out[name][at] = torch.copysign(r, x)
                out[name + "_s"][sc] = s
        else:
            out["m"][at], out["v"][at] = m, v
        place += nb * 128
    out["step"] = torch.tensor([float(t)])
    return out
