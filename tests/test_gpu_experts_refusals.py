"""Arguments that the expert operators' binding refuses, each with the error that it promises: ValueError for a wrong
type, shape, device or layout, MoEError for what the library does not take."""
import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def d():
    g = T.gen(1)
    x = torch.randn((8, 256), generator=g, device="cuda").to(BF)
    off = T.offsets([3, 5])
    return {"x": x, "inv": torch.arange(16, dtype=torch.int32, device="cuda"), "off": off, "q": ex.quantize_rows(x),
            "c": ex.quantize_columns(x, off), "w": ex.quantize_blocks(torch.randn((2, 128, 256), generator=g, device="cuda"))}


WRONG = {
    "offsets a list": lambda d: ex.quantize_columns(d["x"], [0, 8]),
    "offsets a number": lambda d: ex.quantize_columns(d["x"], 8),
    "offsets empty": lambda d: ex.quantize_columns(d["x"], d["off"][:0]),
    "weight gradient's offsets a list": lambda d: ex.product_weight_grad(*d["c"], *d["c"], [0, 3, 8]),
    "weight gradient's offsets two-dimensional": lambda d: ex.product_weight_grad(*d["c"], *d["c"], d["off"][None]),
    "product's offsets a list": lambda d: ex.product(*d["q"], *d["w"], [0, 3, 8]),
    "weights a number": lambda d: ex.combine(d["x"], d["inv"], torch.ones((), device="cuda")),
    "weights a row": lambda d: ex.combine(d["x"], d["inv"], torch.ones(16, device="cuda")),
    "weights of three dimensions": lambda d: ex.combine(d["x"], d["inv"], torch.ones((8, 2, 1), device="cuda")),
    "rows a fraction": lambda d: ex.dispatch(d["x"], d["inv"], 16.0),
    "rows a text": lambda d: ex.dispatch_quantize(d["x"], d["inv"], "16"),
    "M a fraction": lambda d: ex.dispatch_backward(d["x"], d["inv"], 8.0),
    "M no number": lambda d: ex.dispatch_backward(d["x"], d["inv"], None),
    "out a number": lambda d: ex.quantize_rows(d["x"], out=3),
    "out three tensors": lambda d: ex.quantize_rows(d["x"], out=(*d["q"], d["x"])),
    "act a list": lambda d: ex.activation(d["x"], ["swiglu"]),
    "dtype a list": lambda d: ex.quantize_rows(d["x"], [T.E4]),
    "dtype a text": lambda d: ex.quantize_rows(d["x"], "e4m3"),
    "stream a list": lambda d: ex.quantize_rows(d["x"], stream=[]),
    "stream a text": lambda d: ex.quantize_rows(d["x"], stream="s"),
}


@pytest.mark.parametrize("what", sorted(WRONG))
def test_wrong_types_and_shapes_raise_value_error(d, what):
    with pytest.raises(ValueError):
        WRONG[what](d)


LIMITS = {
    "rows negative": (INV, lambda d: ex.dispatch(d["x"], d["inv"], -1)),
    "rows negative, 8 bits": (INV, lambda d: ex.dispatch_quantize(d["x"], d["inv"], -1)),
    "M negative": (INV, lambda d: ex.dispatch_backward(d["x"], d["inv"], -8)),
    "rows past the limit": (UNS, lambda d: ex.dispatch(d["x"], d["inv"], ex.MAX_ROWS + 1)),
    # 2^32 + 16 would be 16 in the library's 32 bits
    "rows past 32 bits": (UNS, lambda d: ex.dispatch(d["x"], d["inv"], 2 ** 32 + 16)),
    "rows over tokens": (INV, lambda d: ex.dispatch(d["x"], d["inv"][:8], out=d["x"])),
    "scales over rows": (INV, lambda d: ex.quantize_rows(d["x"], out=(
        d["q"][0], d["x"].view(-1)[:32].view(F32).view(8, 2)))),
}


@pytest.mark.parametrize("what", sorted(LIMITS))
def test_what_the_library_does_not_take_raises_moe_error(d, what):
    status, call = LIMITS[what]
    with pytest.raises(moe.MoEError) as e:
        call(d)
    assert e.value.status == status


def test_sizes_past_32_bits_are_refused():
    """2^32 + 8 rows would be eight in the library's 32 bits."""
    y = torch.empty((2 ** 32 + 8, 1), dtype=BF, device="cuda")
    for call in (lambda: ex.activation(y, "relu2"), lambda: ex.quantize_rows(y),
                 lambda: ex.activation_quantize(y, "relu2"), lambda: ex.quantize_columns(y),
                 lambda: ex.activation_backward(y, y, "relu2")):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == UNS
    del y
    torch.cuda.empty_cache()


def test_refused_calls_leave_the_device_as_it_was(d):
    assert torch.equal(ex.dispatch(d["x"], d["inv"]), d["x"].repeat(2, 1)) and ex.get_error() == 0
