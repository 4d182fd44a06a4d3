"""The norm of rows of 1032 to 1536 columns: teams of three waves, one a block in
the forward and two in the backward pass, in one block and in many."""
import pytest
import torch

import test_gpu_rows as rows

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1032), (5, 1032), (8, 1280), (9, 1536), (700, 1032), (1100, 1536)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [rows.BF16, rows.F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", ["layer", "layer_nobeta", "rms"])
@pytest.mark.parametrize("T,m", SHAPES)
def test_norm_forward(T, m, norm, dtype):
    rows.test_norm_forward(T, m, norm, dtype)


@pytest.mark.parametrize("dtype", [rows.BF16, rows.F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("T,m", SHAPES)
def test_norm_backward(T, m, layer, dtype):
    rows.test_norm_backward(T, m, layer, dtype)
