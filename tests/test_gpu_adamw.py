"""gs_adamw_step bit for bit against the numpy reference of its definition
(adamw_reference.py), which the CPU tests hold to the 64-bit update."""
import numpy as np
import pytest
import torch

import adamw_reference as ref
import loss_scaling_fp8_amd as gs

pytestmark = pytest.mark.gpu

F = np.float32
GRADS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


def _bits(t):
    t = t.detach().cpu().contiguous()
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()]).numpy()


class Case:
    """A list of tensors on the device and the same list in the reference."""

    def __init__(self, sizes, dev, bits=32, grad="f32", copy=None, offset=0, seed=0, S=1.0, wd=None,
                 grads=None):
        rng = np.random.default_rng(seed)
        self.sizes, self.bits, self.copy = sizes, bits, copy
        self.wd = wd if wd is not None else [0.1 if i % 2 else 0.0 for i in range(len(sizes))]

        def place(h):                            # `offset` elements into an allocation
            t = torch.empty(h.size + offset + 8, dtype=torch.from_numpy(h).dtype, device=dev)
            t = t[offset:offset + h.size]
            t.copy_(torch.from_numpy(h))
            return t
        self.p, self.g, self.m, self.v, self.ms, self.vs, self.c = ([] for _ in range(7))
        self.h = []
        for i, n in enumerate(sizes):
            mag = np.exp(rng.standard_normal(n) * 1.5 - 4)
            p = rng.standard_normal(n).astype(F)
            gt = torch.from_numpy((rng.standard_normal(n) * mag * S).astype(F)).to(GRADS[grad])
            if grads is not None:
                gt = grads[i].to(GRADS[grad])
            m = (rng.standard_normal(n) * mag).astype(F)
            v = (rng.random(n) * mag * mag).astype(F)
            host = {"p": p, "g": gt.float().numpy(), "m": m, "v": v}
            if bits == 8:
                h16 = rng.integers(0, 1 << 16, n).astype(np.uint64)
                host["m"], host["ms"] = ref.encode(m, h16, False)
                host["v"], host["vs"] = ref.encode(np.sqrt(v), h16, True)
                self.ms.append(place(host["ms"]))
                self.vs.append(place(host["vs"]))
            self.h.append(host)
            self.p.append(place(p))
            self.m.append(place(host["m"]))
            self.v.append(place(host["v"]))
            g = torch.empty(n + offset + 8, dtype=GRADS[grad], device=dev)[offset:offset + n]
            g.copy_(gt)
            self.g.append(g)
            if copy:
                c = torch.zeros(n + offset + 8, dtype=GRADS[copy], device=dev)[offset:offset + n]
                self.c.append(c)
        self.plan = gs.gs_adamw_plan(self.p, self.g, self.m, self.v, self.ms if bits == 8 else None,
                                     self.vs if bits == 8 else None, self.c if copy else None, self.wd)
        self.lr = torch.tensor([2e-3], device=dev)
        self.step = torch.zeros(1, dtype=torch.int32, device=dev)
        self.t = 0

    def run(self, beta1=0.9, beta2=0.95, eps=1e-8, **kw):
        gs.gs_adamw_step(self.plan, self.lr, self.step, beta1=beta1, beta2=beta2, eps=eps, **kw)

    def reference(self, beta1=0.9, beta2=0.95, eps=1e-8, seed=0, **kw):
        self.t += 1
        lr = float(self.lr)
        for i, h in enumerate(self.h):
            n = h["p"].size
            m, v = h["m"], h["v"]
            if self.bits == 8:
                m, r = ref.decode(m, h["ms"], n), ref.decode(v, h["vs"], n)
                v = r * r
            h["p"], m, v, r = ref.update32(h["p"], h["g"], m, v, self.wd[i], lr, self.t, beta1, beta2,
                                           eps, **kw)
            if self.bits == 8:
                hs = ref.hashes(n, i, seed, self.t)
                h["m"], h["ms"] = ref.encode(m, hs & np.uint64(0xFFFF), False)
                h["v"], h["vs"] = ref.encode(r, hs >> np.uint64(16), True)
            else:
                h["m"], h["v"] = m, v

    def check(self):
        torch.cuda.synchronize()
        assert int(self.step) == self.t
        for i, h in enumerate(self.h):
            lists = [("p", self.p), ("m", self.m), ("v", self.v)]
            if self.bits == 8:
                lists += [("ms", self.ms), ("vs", self.vs)]
            for name, ts in lists:
                got, want = _bits(ts[i]), h[name].view(np.int32 if h[name].dtype == F else np.uint8)
                nan = np.isnan(h[name]) if h[name].dtype == F else np.zeros(got.shape, bool)
                same = (got == want) | (nan & np.isnan(ts[i].cpu().float().numpy()))
                assert same.all(), (name, i, np.flatnonzero(~same)[:5], int((~same).sum()))
            if self.copy:
                want = torch.from_numpy(h["p"]).to(GRADS[self.copy])
                assert torch.equal(self.c[i].cpu().view(torch.int16), want.view(torch.int16)), i


SIZES = [1, 2048, 127, 0, 128, 129, 4096, 5000, 2049, 7]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("copy", [None, "bf16", "f16"])
def test_types(bits, grad, copy, dev):
    """Sizes around the group, lane and chunk borders; three steps."""
    c = Case(SIZES, dev, bits, grad, copy, seed=bits)
    for _ in range(3):
        c.run(seed=5)
        c.reference(seed=5)
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_unaligned(bits, offset, dev):
    """Tensors that begin off a 16-byte border take the element-wise path."""
    c = Case([5000, 33, 2048], dev, bits, "bf16", "bf16", offset=offset, seed=3)
    for _ in range(2):
        c.run()
        c.reference()
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_scale_and_clip(bits, dev):
    """Gradients that carry S, clipped by the norm of what the unscale saw;
    a norm below the limit changes nothing."""
    S = 1024.0
    c = Case([3000, 129], dev, bits, "f16", "bf16", S=S, seed=4)
    scale = torch.tensor([S], device=dev)
    sumsq = torch.zeros(2, dtype=torch.int64, device=dev)
    norm_sq = torch.zeros(1, dtype=torch.float64, device=dev)
    found = torch.zeros(1, dtype=torch.int32, device=dev)
    gs.gs_unscale_check_sumsq(c.g, [torch.empty(n, device=dev) for n in c.sizes], scale, found, sumsq,
                              norm_sq)
    for max_norm in (0.5 * float(norm_sq) ** 0.5, 2.0 * float(norm_sq) ** 0.5):
        kw = dict(max_norm=max_norm)
        c.run(scale=scale, found_inf=found, norm_sq=norm_sq, seed=77, **kw)
        c.reference(scale=F(S), norm_sq=float(norm_sq), seed=77, **kw)
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_found_inf_leaves_everything(bits, dev):
    c = Case([3000, 129], dev, bits, "f32", "bf16", seed=6)
    found = torch.ones(1, dtype=torch.int32, device=dev)
    c.run(found_inf=found)
    torch.cuda.synchronize()
    assert int(found) == 1
    copies, c.copy = c.copy, None
    c.check()                                        # as at the start
    assert all(bool((t == 0).all()) for t in c.c)
    c.copy = copies
    found.zero_()
    c.run(found_inf=found)
    c.reference()
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [(0.0, 0.0, 1e-8), (0.9, 0.999, 0.0), (0.5, 0.0, 1e-3)])
def test_hyperparameters(bits, hyper, dev):
    c = Case([700, 2048], dev, bits, seed=8, wd=[0.3, 0.0])
    for _ in range(2):
        c.run(*hyper)
        c.reference(*hyper)
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_gradients(bits, dev):
    """Zeros, the smallest and largest values, groups of zeros only, and
    (without the flag) NaN and infinities, which stay in their elements."""
    n = 1024
    g = torch.randn(n, generator=torch.Generator().manual_seed(1))
    g[:128] = 0
    g[128:256] = 1e-30
    g[256] = 3e18
    g[300] = -1e-44
    g[400] = float("nan")
    g[500] = float("inf")
    g[600] = float("-inf")
    c = Case([n], dev, bits, "f32", seed=9, grads=[g])
    for _ in range(2):
        c.run()
        c.reference()
    c.check()


def test_seed_step_and_tensor_choose_the_rounding(dev):
    codes = []
    for seed, sizes in ((1, [4096, 4096]), (2, [4096, 4096]), (1, [4096, 4096])):
        c = Case(sizes, dev, 8, seed=10)
        c.run(seed=seed)
        codes.append([_bits(t).copy() for t in c.m + c.v])
    assert all(np.array_equal(a, b) for a, b in zip(codes[0], codes[2]))
    assert not any(np.array_equal(a, b) for a, b in zip(codes[0], codes[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_and_stream(bits, dev):
    """A captured step replayed: the step count, the learning rate and the
    flag are read on the device each time."""
    c = Case([5000, 300, 2048], dev, bits, "bf16", "bf16", seed=11)
    found = torch.zeros(1, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    gs.gs_adamw_step(c.plan, c.lr, c.step, beta1=0.9, beta2=0.95, found_inf=found, seed=3, stream=side)
    side.synchronize()
    c.reference(seed=3)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(found_inf=found, seed=3)
    for i in range(4):
        found.fill_(1 if i == 2 else 0)
        c.lr.fill_(2e-3 / (i + 1))
        g.replay()
        torch.cuda.synchronize()
        if i != 2:
            c.reference(seed=3)
        c.check()


def test_mismatched_plan_changes_nothing(dev):
    """The C entry point called with other kinds than the plan's."""
    c = Case([3000], dev, 32, "f32", seed=12)
    for kw in (dict(grad_dtype=gs.GS_F16), dict(state_bits=8), dict(copy_dtype=gs.GS_F16)):
        old = {k: getattr(c.plan, k) for k in kw}
        c.plan.__dict__.update(kw)
        c.run()
        c.plan.__dict__.update(old)
        c.check()
    c.run()
    c.reference()
    c.check()


def test_many_tensors(dev):
    """291 tensors, most of odd lengths, in one call."""
    rng = np.random.default_rng(13)
    sizes = [int(n) for n in rng.integers(1, 9000, 291)]
    for bits in (32, 8):
        c = Case(sizes, dev, bits, "f16", "f16", seed=14)
        c.run(seed=1)
        c.reference(seed=1)
        c.check()


def test_refusals(dev):
    f = [torch.zeros(300, device=dev) for _ in range(4)]
    u = [torch.zeros(300, dtype=torch.uint8, device=dev) for _ in range(2)]
    s = [torch.zeros(3, device=dev) for _ in range(2)]
    plan = gs.gs_adamw_plan
    with pytest.raises(gs.GSError, match="ARG"):
        plan([f[0]], [f[1]], [f[2]], [f[2]])                     # m is v
    with pytest.raises(gs.GSError, match="ARG"):
        plan([f[0], f[0]], [f[1], f[1]], [f[2], f[2]], [f[3], f[3]])
    with pytest.raises(TypeError, match="exp_avgs"):
        plan([f[0]], [f[1]], [u[0]], [u[1]])
    with pytest.raises(ValueError, match="both lists"):
        plan([f[0]], [f[1]], [u[0]], [u[1]], exp_avg_scales=[s[0]])
    with pytest.raises(ValueError, match="exp_avg_sq_scales"):
        plan([f[0]], [f[1]], [u[0]], [u[1]], [s[0]], [s[1][:2]])
    with pytest.raises(ValueError, match="grads"):
        plan([f[0]], [f[1][:299]], [f[2]], [f[3]])
    with pytest.raises(TypeError, match="grads"):
        plan([f[0]], [f[1].double()], [f[2]], [f[3]])
    with pytest.raises(TypeError, match="copies"):
        plan([f[0]], [f[1]], [f[2]], [f[3]], copies=[torch.zeros(300, device=dev)])
    with pytest.raises(ValueError, match="contiguous"):
        plan([torch.zeros(600, device=dev)[::2]], [f[1]], [f[2]], [f[3]])
    with pytest.raises(ValueError, match="weight_decays"):
        plan([f[0]], [f[1]], [f[2]], [f[3]], weight_decays=[0.1, 0.1])
    good = plan([f[0]], [f[1]], [f[2]], [f[3]])
    lr, step = torch.tensor([1e-3], device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    with pytest.raises(TypeError, match="step"):
        gs.gs_adamw_step(good, lr, step.long())
    with pytest.raises(gs.GSError, match="ARG"):
        gs.gs_adamw_step(good, lr, step, beta1=1.0)
    with pytest.raises(gs.GSError, match="ARG"):
        gs.gs_adamw_step(good, lr, step, norm_sq=torch.ones(1, dtype=torch.float64, device=dev))
    torch.cuda.synchronize()
    assert int(step) == 0 and all(bool((t == 0).all()) for t in f)
