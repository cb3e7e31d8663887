"""CPU checks: every output of an expert operator that shares memory with any input, or with another output, is
refused before anything touches the device."""
import pytest

from tests.test_experts_abi import CALLS, F, INV, L

# name: (positions of the inputs, positions of the outputs) in CALLS
BUFFERS = {
    "moe_dispatch": ((0, 5), (7,)),
    "moe_combine": ((0, 5, 7), (8,)),
    "moe_combine_backward": ((0, 1, 6, 8), (9, 10)),
    "moe_quantize_rows": ((0,), (5, 6)),
    "moe_dispatch_quantize": ((0, 5), (8, 9)),
    "moe_quantize_blocks": ((0,), (6, 7)),
    "moe_quantize_columns": ((0, 4), (7, 8)),
    "moe_activation": ((0,), (5,)),
    "moe_activation_quantize": ((0,), (6, 7)),
    "moe_activation_backward": ((0, 1), (6,)),
    "moe_product": ((0, 1, 3, 4, 8), (11,)),
    "moe_product_activation": ((0, 1, 3, 4, 8), (12, 13)),
    "moe_product_input_grad": ((0, 1, 3, 4, 8), (11,)),
    "moe_product_weight_grad": ((0, 1, 3, 4, 9), (13,)),
}
PAIRS = [(n, i, o) for n, (ins, outs) in BUFFERS.items() for i in ins + outs for o in outs if i != o]


def test_every_buffer_is_named():
    assert set(BUFFERS) == set(CALLS)
    for name, (ins, outs) in BUFFERS.items():
        assert sorted(ins + outs) == [i for i, v in enumerate(CALLS[name]) if isinstance(v, int) and v >= F]


@pytest.mark.parametrize("name,other,out", PAIRS)
def test_shared_memory_is_refused(name, other, out):
    args = list(CALLS[name])
    args[out] = args[other]
    assert getattr(L, name)(*args) == INV


# the last 16 bytes of a buffer: (name, its position, its size in bytes with CALLS' arguments, output position)
ENDS = [
    ("moe_dispatch", 5, 8 * 4 * 4, 7), ("moe_combine", 7, 8 * 4 * 4, 8), ("moe_combine_backward", 8, 8 * 4 * 4, 9),
    ("moe_combine_backward", 10, 8 * 4 * 4, 9), ("moe_quantize_rows", 6, 8 * 4, 5),
    ("moe_dispatch_quantize", 9, 32 * 4, 8), ("moe_quantize_blocks", 0, 2 * 64 * 64 * 2, 7),
    ("moe_quantize_columns", 8, 4 * 64 * 4, 7), ("moe_activation_quantize", 0, 8 * 128 * 2, 7),
    ("moe_product", 1, 8 * 4, 11), ("moe_product", 4, 4 * 4, 11), ("moe_product_activation", 4, 4 * 4, 13),
    ("moe_product_input_grad", 1, 8 * 4, 11), ("moe_product_weight_grad", 1, 4 * 64 * 4, 13),
    ("moe_product_weight_grad", 4, 4 * 64 * 4, 13)]


@pytest.mark.parametrize("name,other,size,out", ENDS)
def test_shared_ends_are_refused(name, other, size, out):
    args = list(CALLS[name])
    args[out] = args[other] + size - 16
    assert getattr(L, name)(*args) == INV

