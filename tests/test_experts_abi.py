"""CPU checks of the expert operators' C ABI and binding: refusals before anything touches the device."""
import ctypes

import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex

L = moe.lib()
F = 1 << 30  # 16-byte aligned, never-dereferenced addresses, far enough apart not to overlap
A, B_, C_, D_, E_, G_ = (F * i for i in range(1, 7))
OK, INV, UNS = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
BF, E4 = moe.DT_BF16, moe.DT_E4M3

# name: valid arguments by position (the stream last)
CALLS = {
    "moe_dispatch": [A, BF, 8, 4, 64, B_, 32, C_, None],
    "moe_combine": [A, BF, 8, 4, 64, B_, 32, C_, D_, None],
    "moe_combine_backward": [A, B_, BF, 8, 4, 64, C_, 32, D_, E_, G_, None],
    "moe_quantize_rows": [A, BF, 8, 64, E4, B_, C_, None],
    "moe_dispatch_quantize": [A, BF, 8, 4, 64, B_, 32, E4, C_, D_, None],
    "moe_quantize_blocks": [A, BF, 2, 64, 64, E4, B_, C_, None],
    "moe_quantize_columns": [A, BF, 8, 64, B_, 4, E4, C_, D_, None],
    "moe_activation": [A, BF, 0, 8, 64, B_, None],
    "moe_activation_quantize": [A, BF, 0, 8, 64, E4, B_, C_, None],
    "moe_activation_backward": [A, B_, BF, 0, 8, 64, C_, None],
    "moe_product": [A, B_, E4, C_, D_, 8, 64, 64, E_, 4, BF, G_, None],
    "moe_product_activation": [A, B_, E4, C_, D_, 8, 64, 64, E_, 4, 0, E4, G_, F * 7, None],
    "moe_product_input_grad": [A, B_, E4, C_, D_, 8, 64, 64, E_, 4, BF, G_, None],
    "moe_product_weight_grad": [A, B_, E4, C_, D_, E4, 4, 64, 64, E_, 4, BF, 0, G_, None],
}
# (name, argument position, bad value, status)
BAD = [
    ("moe_dispatch", 1, 2, INV), ("moe_dispatch", 2, -1, INV), ("moe_dispatch", 3, 0, INV), ("moe_dispatch", 3, 33, UNS),
    ("moe_dispatch", 4, 60, INV), ("moe_dispatch", 4, 0, INV), ("moe_dispatch", 4, (1 << 20) + 8, UNS),
    ("moe_dispatch", 6, -1, INV), ("moe_dispatch", 6, 1 << 20, UNS), ("moe_dispatch", 2, 1 << 18, UNS),
    ("moe_combine", 4, 4, INV), ("moe_combine", 7, C_ + 4, INV), ("moe_combine", 0, None, INV),
    ("moe_combine_backward", 2, 3, INV), ("moe_combine_backward", 8, None, INV),
    ("moe_quantize_rows", 4, 0, INV), ("moe_quantize_rows", 4, 4, INV), ("moe_quantize_rows", 3, 72, INV),
    ("moe_quantize_rows", 2, -1, INV), ("moe_dispatch_quantize", 4, 72, INV), ("moe_dispatch_quantize", 7, BF, INV),
    ("moe_quantize_blocks", 3, 24, INV), ("moe_quantize_blocks", 4, 24, INV), ("moe_quantize_blocks", 2, -1, INV),
    # 2^30 matrices of 64 x 64 are 2^30 blocks, which a launch can have, but their 2^43 bytes reach the output
    ("moe_quantize_blocks", 2, 1 << 30, INV),
    ("moe_quantize_columns", 4, None, INV), ("moe_quantize_columns", 5, 0, INV), ("moe_quantize_columns", 5, 2000, UNS),
    ("moe_quantize_columns", 2, 1 << 20, UNS), ("moe_activation", 2, 2, INV), ("moe_activation", 4, 12, INV),
    ("moe_activation_quantize", 4, 72, INV), ("moe_activation_quantize", 5, 1, INV),
    ("moe_activation_backward", 3, -1, INV), ("moe_product", 2, BF, INV), ("moe_product", 6, 72, INV),
    ("moe_product", 7, 72, INV), ("moe_product", 8, None, INV), ("moe_product", 8, E_ + 4, INV),
    ("moe_product", 9, 0, INV), ("moe_product", 9, 1025, UNS), ("moe_product", 10, E4, INV),
    ("moe_product", 5, -1, INV), ("moe_product", 5, 1 << 20, UNS), ("moe_product", 6, 1 << 21, UNS),
    ("moe_product_activation", 10, 2, INV), ("moe_product_activation", 11, BF, INV),
    ("moe_product_activation", 13, None, INV), ("moe_product_input_grad", 10, 2, INV),
    ("moe_product_weight_grad", 5, 1, INV), ("moe_product_weight_grad", 6, -1, INV),
    ("moe_product_weight_grad", 6, 1 << 20, UNS), ("moe_product_weight_grad", 11, 2, INV),
    ("moe_product_weight_grad", 12, 2, INV), ("moe_product_weight_grad", 13, None, INV),
]


@pytest.mark.parametrize("name,at,value,status", BAD)
def test_bad_arguments_are_refused(name, at, value, status):
    args = list(CALLS[name])
    args[at] = value
    assert getattr(L, name)(*args) == status


@pytest.mark.parametrize("name", sorted(CALLS))
def test_missing_or_misaligned_pointers_are_refused(name):
    args = CALLS[name]
    for at, v in enumerate(args):
        if isinstance(v, int) and v >= F:
            for bad in (None, v + 8):
                if bad is None and name in ("moe_combine",) and at == 7:
                    continue  # combine's weights may be missing
                a = list(args)
                a[at] = bad
                assert getattr(L, name)(*a) == INV, (at, bad)


@pytest.mark.parametrize("name,src,dst", [
    ("moe_dispatch", 0, 7), ("moe_combine", 0, 8), ("moe_combine_backward", 0, 9), ("moe_combine_backward", 1, 9),
    ("moe_quantize_rows", 0, 5), ("moe_dispatch_quantize", 0, 8), ("moe_quantize_blocks", 0, 6),
    ("moe_quantize_columns", 0, 7), ("moe_activation", 0, 5), ("moe_activation_quantize", 0, 6),
    ("moe_activation_backward", 0, 6), ("moe_activation_backward", 1, 6), ("moe_product", 0, 11), ("moe_product", 3, 11),
    ("moe_product_activation", 0, 12), ("moe_product_input_grad", 3, 11), ("moe_product_weight_grad", 0, 13),
    ("moe_product_weight_grad", 3, 13)])
def test_outputs_must_not_overlap_inputs(name, src, dst):
    args = list(CALLS[name])
    args[dst] = args[src] + 64
    assert getattr(L, name)(*args) == INV


@pytest.mark.parametrize("name,zero", [
    ("moe_dispatch", 2), ("moe_dispatch", 6), ("moe_combine", 2), ("moe_combine_backward", 3), ("moe_quantize_rows", 2),
    ("moe_dispatch_quantize", 2), ("moe_dispatch_quantize", 6), ("moe_quantize_blocks", 2), ("moe_quantize_columns", 2),
    ("moe_activation", 3), ("moe_activation_quantize", 3), ("moe_activation_backward", 4), ("moe_product", 5),
    ("moe_product_activation", 5), ("moe_product_input_grad", 5)])
def test_no_rows_is_a_noop_without_buffers(name, zero):
    args = [None if isinstance(v, int) and v >= F else v for v in CALLS[name]]
    args[zero] = 0
    if name in ("moe_product", "moe_product_activation", "moe_product_input_grad"):
        args[8] = E_  # offsets are checked with the sizes
    if name == "moe_quantize_columns":
        args[4] = E_
    assert getattr(L, name)(*args) == OK


def test_weight_gradient_without_rows_adds_nothing():
    args = list(CALLS["moe_product_weight_grad"])
    args[6], args[12] = 0, 1
    assert L.moe_product_weight_grad(*args) == OK


def test_column_blocks_hold_every_split():
    assert L.moe_column_blocks(0, 4) == 0
    assert L.moe_column_blocks(1, 4) == 1
    for P, E in ((127, 3), (128, 3), (1000, 7), (5, 64)):
        most = 0
        for cut in range(P + 1):  # two experts share the rows, the others get one each where there are enough
            rest = [1] * min(E - 2, P - cut) if E > 2 else []
            counts = [cut, P - cut - len(rest)] + rest
            most = max(most, sum(-(-n // 128) for n in counts))
        assert most <= L.moe_column_blocks(P, E)


def test_error_word_needs_a_place():
    assert L.moe_product_get_error(None, None) == INV


def test_binding_refuses_host_tensors_and_other_objects():
    x, inv = torch.zeros(4, 64), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: ex.dispatch(x, inv), lambda: ex.quantize_rows(x), lambda: ex.activation(x, "swiglu"),
                 lambda: ex.dispatch(None, inv), lambda: ex.combine(x, inv, x), lambda: ex.quantize_blocks([1.0])):
        with pytest.raises(ValueError):
            call()
