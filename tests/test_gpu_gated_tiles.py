"""Every kernel of the gated feed-forward block, on sizes that select it (test_gated_choice.py), with
experts of none and of several row blocks, against the 64-bit definitions (bounds as in
test_gpu_gated_ffn.py)."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

from _gated_tiles import CASES, offsets
from _gpu import log
from test_gpu_gated_ffn import BF16, F32, check_backward, check_forward, inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def make(name):
    bf16, rows, m, p, E = CASES[name]
    dtype, k = BF16 if bf16 else F32, 2
    T = (rows + k - 1) // k
    g = torch.Generator(device="cuda").manual_seed(rows + m + p)
    r = lambda *s, scale=1.0, shift=0.0: inside((torch.randn(*s, generator=g, device="cuda") * scale + shift).to(dtype))  # noqa: E731
    return {"T": T, "k": k, "E": E, "m": m, "p": p, "rows": rows, "dtype": dtype, "x": r(T, m, shift=0.3),
            "wg": r(E, m, p, scale=m**-0.5), "wu": r(E, m, p, scale=m**-0.5), "wd": r(E, p, m, scale=p**-0.5),
            "gate": r(rows, p, scale=1.5), "up": r(rows, p, scale=1.5), "dy": r(rows, m),
            "offsets": torch.tensor(offsets(rows, E), dtype=torch.int32, device="cuda"),
            "perm": torch.randperm(T * k, generator=g, device="cuda")[:rows].to(torch.int32)}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    log(f"gated forward {name}")
    check_forward(make(name))


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    log(f"gated backward {name}")
    check_backward(make(name))
