"""The training operators' grid-stride paths: the transposing cast and AdamW
through the library built with tiny grid caps
(tests/c/_build/libgsfp8_capped_grid.so), so that each workgroup strides over
many tiles or chunks, which in the real build only lists of more than 10^9
elements need."""
import os

import pytest
import torch

import loss_scaling_fp8_amd as gs
import test_gpu_adamw as adamw_cases
import test_gpu_transposed as transposed_cases

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CAPPED = os.path.join(ROOT, "tests", "c", "_build", "libgsfp8_capped_grid.so")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


@pytest.fixture
def capped():
    """The binding's calls go to the capped-grid library for one test."""
    assert os.path.exists(CAPPED), "%s is not built (run __graft_entry__.build())" % CAPPED
    old_path, old_lib = gs.LIB_PATH, gs._lib
    gs.LIB_PATH, gs._lib = CAPPED, None
    try:
        yield gs.lib()
    finally:
        gs.LIB_PATH, gs._lib = old_path, old_lib


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad,copy", [("f32", "bf16"), ("f16", None)])
def test_adamw_strided(bits, grad, copy, dev, capped):
    c = adamw_cases.Case([20000, 1, 5000, 0, 1024, 130], dev, bits, grad, copy, seed=20)
    for _ in range(2):
        c.run(seed=8)
        c.reference(seed=8)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_transposed_strided(dtype, dev, capped):
    transposed_cases._check(1003, 584, dtype, gs.FP8_E4M3, gs.FP8_BLOCK_1x128, False, dev)
    transposed_cases._check(700, 640, dtype, gs.FP8_E5M2, gs.FP8_BLOCK_1x128, True, dev)
    transposed_cases._check(512, 768, dtype, gs.FP8_E4M3, gs.FP8_BLOCK_128x128, True, dev)
