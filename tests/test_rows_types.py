"""The row operators' binding refuses tensors whose elements are not what the
call reads or writes there.  CPU only: the tensors are stand-ins and the
library is one that records the call."""
import pytest
import torch

import mixture_experts_layer_gemv_amd as M

BF16, F32, I32, I8, I16, F16 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.int16, torch.float16
VALUES = {M.MOE_F32: F32, M.MOE_BF16: BF16}


class Tensor:
    """As much of a contiguous GPU tensor as the binding looks at."""

    def __init__(self, dtype):
        self.dtype, self.itemsize, self.nbytes, self.shape, self.device = dtype, dtype.itemsize, 1 << 40, (1,), "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x7F0000000000


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return M.MOE_OK

        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(M, "lib", lambda: L)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return L


# {call: (the types of its tensors, in order), the call on those tensors}; a, b: value types
OPERATORS = {
    "moe_norm_forward": (lambda a, b: (a, F32, F32, a, F32, F32), lambda t, a, b: M.moe_norm_forward(
        t[0], a, M.MOE_NORM_LAYER, t[1], t[2], 1e-5, 4, 64, t[3], t[4], t[5], stream=0)),
    "moe_norm_backward": (lambda a, b: (a, a, F32, F32, F32, a, F32, F32), lambda t, a, b: M.moe_norm_backward(
        t[0], t[1], a, M.MOE_NORM_LAYER, t[2], t[3], t[4], 4, 64, t[5], t[6], t[7], Tensor(torch.uint8), 4096, stream=0)),
    "moe_permute_rows": (lambda a, b: (a, I32, a), lambda t, a, b: M.moe_permute_rows(
        t[0], a, t[1], 4, 64, 2, 8, t[2], stream=0)),
    "moe_permute_rows_backward": (lambda a, b: (a, I32, b), lambda t, a, b: M.moe_permute_rows_backward(
        t[0], a, t[1], 4, 64, 2, 8, t[2], b, stream=0)),
    "moe_combine_rows": (lambda a, b: (a, I32, F32, b), lambda t, a, b: M.moe_combine_rows(
        t[0], a, t[1], t[2], 4, 64, 2, 8, t[3], b, stream=0)),
    "moe_combine_rows_backward": (lambda a, b: (a, b, I32, F32, b, F32), lambda t, a, b: M.moe_combine_rows_backward(
        t[0], a, t[1], b, t[2], t[3], 4, 64, 2, 8, t[4], t[5], stream=0)),
    "moe_quantize_codes_i8": (lambda a, b: (BF16, I8, F32), lambda t, a, b: M.moe_quantize_codes_i8(
        t[0], 4, 64, t[1], t[2], stream=0)),
    "moe_matmul_i8": (lambda a, b: (I8, F32, I8, F32, I32, I32, b), lambda t, a, b: M.moe_matmul_i8(
        t[0], t[1], t[2], t[3], t[4], t[5], 4, 2, 8, 64, 64, 2, t[6], b, stream=0)),
}
# what each element type could be taken for, of the same size or smaller
WRONG = {BF16: (F16, F32, torch.uint8, torch.int64), F32: (BF16, I32, torch.float64), I32: (F32, torch.int64, torch.uint8),
         I8: (torch.uint8, BF16, torch.bool)}


@pytest.mark.parametrize("fn", OPERATORS)
@pytest.mark.parametrize("b", VALUES, ids=["f32", "bf16"])
@pytest.mark.parametrize("a", VALUES, ids=["f32", "bf16"])
def test_wrong_elements_are_refused(fn, a, b, library):
    types, call = OPERATORS[fn]
    types = types(VALUES[a], VALUES[b])
    call([Tensor(d) for d in types], a, b)
    assert library.calls == 1
    # bf16 bit patterns in 16-bit integers are bf16
    call([Tensor(I16 if d == BF16 else d) for d in types], a, b)
    assert library.calls == 2
    for i, d in enumerate(types):
        for wrong in WRONG[d]:
            t = [Tensor(w if i == j else e) for j, e in enumerate(types) for w in [wrong]]
            with pytest.raises(M.MoeError) as ei:
                call(t, a, b)
            assert ei.value.status == M.MOE_ERR_INVALID_ARG and str(wrong) in ei.value.message, (fn, i, wrong)
    assert library.calls == 2


def test_pointers_and_unknown_value_types_reach_the_call(library):
    """Plain pointers carry no type; a value type that the operators do not take is the call's to refuse."""
    p = 0x7F0000000000
    M.moe_permute_rows(p, M.MOE_BF16, p, 4, 64, 2, 8, p, stream=0)
    M.moe_permute_rows(Tensor(F32), 7, Tensor(I32), 4, 64, 2, 8, Tensor(F32), stream=0)
    assert library.calls == 2
