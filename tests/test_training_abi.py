"""CPU checks of include/gs/training.h: it compiles as C, the library exports
what it declares, every argument error is returned on the host with its
documented status, the AdamW plan's layout and overlap check, and the Python
binding refuses host tensors."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import loss_scaling_fp8_amd as gs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gs", "training.h")
FAKE = 1 << 40          # an aligned, never-dereferenced "device" address


def test_header_declares_the_exports():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:gs_status|size_t)\s+([a-z][a-z0-9_]*)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(gs.TRAINING_EXPORTS)
    for name in names:
        assert hasattr(gs.lib(), name), name
        assert callable(getattr(gs, name)), name


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_is_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "gs/training.h"\nint main(void) { return fp8_matmul_workspace_size(0, 0, 0) != 0; }\n')
    libdir = os.path.dirname(gs.LIB_PATH)
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe, "-L" + libdir,
                    "-l:libgsfp8.so", "-Wl,-rpath," + libdir], check=True)
    subprocess.run([exe], check=True, timeout=60)


# ------------------------------------------------------------------ fp8_matmul
def _matmul(**kw):
    a = dict(a=FAKE, af=0, ag=1, sa=FAKE, b=FAKE, bf=0, bg=2, sb=FAKE, m=4, n=128, k=256,
             od=gs.GS_BF16, acc=0, out=FAKE, ws=None, wsb=0)
    a.update(kw)
    return gs.lib().fp8_matmul(a["a"], a["af"], a["ag"], a["sa"], a["b"], a["bf"], a["bg"], a["sb"],
                               a["m"], a["n"], a["k"], a["od"], a["acc"], a["out"], a["ws"],
                               a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(od=4), -4), (dict(od=0), -4), (dict(acc=2), -5), (dict(acc=1), -4),
    (dict(acc=1, od=gs.GS_F16), -4), (dict(af=2), -5), (dict(bf=-1), -5), (dict(ag=0), -5),
    (dict(bg=3), -5), (dict(m=-1), -2), (dict(n=-1), -2), (dict(k=-128), -2),
    (dict(k=(1 << 22) + 128), -2), (dict(m=(1 << 31) + 1), -2),
    (dict(m=1 << 31, n=128, k=128), -2),
    (dict(m=1 << 30, k=1 << 20), -2), (dict(m=1 << 31, n=1 << 31, k=128), -2),
    (dict(k=200), -3), (dict(n=100), -3), (dict(ag=2), -3), (dict(a=None), -1), (dict(sb=None), -1),
    (dict(out=None), -1), (dict(a=FAKE + 8), -6), (dict(b=FAKE + 1), -6), (dict(sa=FAKE + 2), -6),
    (dict(out=FAKE + 8), -6),
    (dict(m=0), 0), (dict(n=0), 0), (dict(m=0, a=None, sa=None, out=None), 0),
    (dict(k=0, a=None, b=None, sa=None, sb=None, acc=1, od=gs.GS_F32), 0),
])
def test_matmul_argument_errors(kw, code):
    assert _matmul(**kw) == code


def test_matmul_workspace():
    size = gs.fp8_matmul_workspace_size
    assert size(1, 1024, 4096) == size(0, 128, 128) == size(128, 128, 0) == size(-1, 5, 128) == 0
    split = [(m, n, k) for m in (65, 128, 333, 512) for n in (128, 1024, 7168)
             for k in (4096, 18432) if size(m, n, k)]
    assert split
    for m, n, k in split:
        need = size(m, n, k)
        assert need % (4 * m * n) == 0
        assert _matmul(m=m, n=n, k=k, wsb=need) == -7
        assert _matmul(m=m, n=n, k=k, ws=FAKE, wsb=need - 1) == -7
        assert _matmul(m=m, n=n, k=k, ws=FAKE + 4, wsb=need) == -6


# ------------------------------------------------------------------ transposing cast
def _transposed(**kw):
    a = dict(x=FAKE, dt=gs.GS_BF16, r=256, c=128, f=0, g=1, ct=FAKE, st=FAKE, cd=None, s=None, nf=None)
    a.update(kw)
    return gs.lib().fp8_quantize_transposed(a["x"], a["dt"], a["r"], a["c"], a["f"], a["g"], a["ct"],
                                            a["st"], a["cd"], a["s"], a["nf"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=1), -4), (dict(f=2), -5), (dict(g=0), -5), (dict(g=3), -5), (dict(r=-1), -2),
    (dict(c=1 << 32), -2), (dict(g=2, r=100), -3), (dict(g=2, c=100), -3),
    (dict(c=100, cd=FAKE, s=FAKE), -3), (dict(x=None), -1), (dict(ct=None), -1), (dict(st=None), -1),
    (dict(cd=FAKE), -1), (dict(s=FAKE), -1), (dict(x=FAKE + 8), -6), (dict(ct=FAKE + 8), -6),
    (dict(cd=FAKE + 8, s=FAKE), -6), (dict(st=FAKE + 2), -6), (dict(nf=FAKE + 1), -6),
    (dict(r=0, x=None, ct=None, st=None), 0), (dict(c=0, x=None, ct=None, st=None), 0),
])
def test_transposed_argument_errors(kw, code):
    assert _transposed(**kw) == code


# ------------------------------------------------------------------ AdamW
def _plan(n=1, numels=(300,), grad=gs.GS_F32, bits=32, copy=0, size=None, host=None, **kw):
    """gs_adamw_plan on made-up addresses 1 GiB apart: (status, plan bytes)."""
    at = {name: [FAKE + ((8 * j + i) << 34) for i in range(max(n, 1))]
          for j, name in enumerate(("p", "g", "m", "v", "ms", "vs", "c"))}
    for name, v in kw.items():
        if name in at:
            at[name] = v
    arr = {k: None if v is None else (ctypes.c_void_p * max(n, 1))(*v) for k, v in at.items()}
    nums = (ctypes.c_int64 * max(n, 1))(*numels)
    wd = (ctypes.c_float * max(n, 1))(*kw.get("wd", [0.1] * max(n, 1)))
    need = gs.gs_adamw_plan_size(list(numels)[:n])
    host = torch.full((max(need, 64),), 0xAB, dtype=torch.uint8) if host is None else host
    st = gs.lib().gs_adamw_plan(
        n, arr["p"], arr["g"], grad, arr["m"], arr["v"], bits, arr["ms"] if bits == 8 else None,
        arr["vs"] if bits == 8 else None, arr["c"] if copy else None, copy, nums, wd,
        host.data_ptr(), need if size is None else size)
    return st, host


def test_plan_size_and_layout():
    assert gs.gs_adamw_plan_size([]) == 64
    assert gs.gs_adamw_plan_size([0, 1, 1024, 1025]) == 64 + 4 * 80 + 8 * (0 + 1 + 1 + 2)
    assert gs.gs_adamw_plan_size([-1]) == 0
    numels = (5, 0, 2049)
    st, host = _plan(3, numels, grad=gs.GS_F16, bits=8, copy=gs.GS_BF16)
    assert st == 0
    raw = bytes(host.numpy())
    assert struct.unpack_from("<iq", raw, 4)[0] == 3 and struct.unpack_from("<q", raw, 8)[0] == 4
    for i, numel in enumerate(numels):
        entry = struct.unpack_from("<7QqfIQ", raw, 64 + 80 * i)
        assert entry[7] == numel and abs(entry[8] - 0.1) < 1e-8 and entry[9] == 0
        want = tuple(FAKE + ((8 * j + i) << 34) for j in range(7)) if numel else (0,) * 7
        assert entry[:7] == want
    chunks = [struct.unpack_from("<II", raw, 64 + 240 + 8 * k) for k in range(4)]
    assert chunks == [(0, 0), (2, 0), (2, 1), (2, 2)]


@pytest.mark.parametrize("kw,code", [
    (dict(grad=4), -4), (dict(copy=gs.GS_F32), -4), (dict(bits=16), -5), (dict(numels=(-1,)), -2),
    (dict(p=None), -1), (dict(g=None), -1), (dict(bits=8, ms=None), -1), (dict(p=[None]), -1),
    (dict(copy=gs.GS_F16, c=[None]), -1), (dict(p=[FAKE + 2]), -6),
    (dict(g=[FAKE + 1], grad=gs.GS_BF16), -6), (dict(m=[FAKE + 2]), -6),
    (dict(bits=8, ms=[FAKE + 2]), -6), (dict(copy=gs.GS_F16, c=[FAKE + 1]), -6),
    (dict(wd=[-0.1]), -5), (dict(wd=[float("nan")]), -5), (dict(wd=[float("inf")]), -5),
    (dict(size=150), -7),
    # what is written overlaps something: m and v, the gradient's last bytes, another tensor
    (dict(m=[FAKE], v=[FAKE]), -5), (dict(p=[FAKE], g=[FAKE + 1196]), -5),
    (dict(n=2, numels=(300, 300), p=[FAKE, FAKE]), -5),
    (dict(n=2, numels=(300, 300), p=[FAKE, FAKE + 1196]), -5),
    (dict(bits=8, ms=[FAKE], vs=[FAKE + 8]), -5),
    # adjacent tensors, shared gradients and empty tensors are no overlap
    (dict(n=2, numels=(300, 300), p=[FAKE, FAKE + 1200]), 0),
    (dict(n=2, numels=(300, 300), g=[FAKE + (1 << 39), FAKE + (1 << 39)]), 0),
    (dict(n=2, numels=(300, 0), p=[FAKE, None]), 0), (dict(n=0, numels=()), 0),
])
def test_plan_argument_errors(kw, code):
    assert _plan(**kw)[0] == code


def test_step_argument_errors():
    args = dict(plan=FAKE, bytes=64 + 80 + 8, n=1, g=gs.GS_F32, bits=32, c=0, lr=FAKE, step=FAKE,
                b1=0.9, b2=0.99, eps=1e-8, s=None, f=None, ns=None, mn=0.0)

    def call(**kw):
        a = dict(args, **kw)
        return gs.lib().gs_adamw_step(a["plan"], a["bytes"], a["n"], a["g"], a["bits"], a["c"],
                                      a["lr"], a["step"], a["b1"], a["b2"], a["eps"], a["s"], a["f"],
                                      a["ns"], a["mn"], 0, None)
    nan, inf = float("nan"), float("inf")
    for kw, code in [(dict(g=7), -4), (dict(c=3), -4), (dict(bits=4), -5), (dict(n=-1), -2),
                     (dict(plan=None), -1), (dict(lr=None), -1), (dict(step=None), -1),
                     (dict(plan=FAKE + 8), -6), (dict(lr=FAKE + 2), -6), (dict(step=FAKE + 1), -6),
                     (dict(s=FAKE + 2), -6), (dict(f=FAKE + 2), -6), (dict(ns=FAKE + 4, mn=1.0), -6),
                     (dict(b1=1.0), -5), (dict(b1=-0.1), -5), (dict(b2=nan), -5), (dict(eps=-1.0), -5),
                     (dict(eps=inf), -5), (dict(ns=FAKE), -5), (dict(ns=FAKE, mn=inf), -5),
                     (dict(bytes=100), -7), (dict(bytes=64 + 80 + 4), -7)]:
        assert call(**kw) == code, kw


# ------------------------------------------------------------------ the binding, on the CPU
def test_host_tensors_are_refused():
    codes, sc = torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4, 1)
    f = torch.zeros(8)
    calls = [
        lambda: gs.fp8_matmul(codes, sc, 0, gs.FP8_BLOCK_1x128, codes, sc, 0, gs.FP8_BLOCK_1x128),
        lambda: gs.fp8_quantize_transposed(torch.zeros(4, 8), 0, gs.FP8_BLOCK_1x128),
        lambda: gs.gs_adamw_plan([f], [f], [f], [f]),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(TypeError, match="gs_adamw_plan"):
        gs.gs_adamw_step(None, f, f)
    with pytest.raises(ValueError, match="empty"):
        gs.gs_adamw_plan([], [], [], [])


def test_transposed_shapes():
    assert gs.transposed_shapes(1, 5, gs.FP8_BLOCK_1x128) == ((5, 128), (5, 1))
    assert gs.transposed_shapes(257, 64, gs.FP8_BLOCK_1x128) == ((64, 384), (64, 3))
    assert gs.transposed_shapes(256, 384, gs.FP8_BLOCK_128x128) == ((384, 256), (3, 2))
