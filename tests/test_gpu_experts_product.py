"""The grouped 8-bit product, its gradients and the fused activation against 64 bits."""
import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

COUNTS = [[1], [0, 1, 0], [127, 129, 0, 300, 5], [16] * 8, [0] * 30 + [700] + [0] * 9]
SHAPES = [(16, 16), (128, 128), (272, 400), (1024, 2048), (640, 2560), (1856, 144)]


def _ids(c):
    return f"{len(c)}x{sum(c)}"


def _weights(E, N, C, g):
    return ex.quantize_blocks(T.randn((E, N, C), g, scale=C ** -0.5))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=_ids)
def test_product(counts, N, C, fp8, out):
    g = T.gen(N + C)
    P, E = sum(counts), len(counts)
    xq, xs = ex.quantize_rows(T.randn((P, C), g), fp8)
    wq, ws = _weights(E, N, C, g)
    got = ex.product(xq, xs, wq, ws, T.offsets(counts), out)
    x, w = T.rows_value(xq, xs), T.weights_value(wq, ws)
    want = T.grouped(x, w, counts, True)
    tol = T.sum_bound(T.grouped(x.abs(), w.abs(), counts, True), -(-C // 128)) + want.abs() * T.HALF[out] * 1.01
    T.assert_within(got, want, tol)
    assert ex.get_error() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=_ids)
def test_product_input_grad(counts, N, C, fp8, out):
    g = T.gen(N + C + 1)
    P, E = sum(counts), len(counts)
    dq, ds = ex.quantize_rows(T.randn((P, N), g, scale=1e-3), fp8)
    wq, ws = _weights(E, N, C, g)
    got = ex.product_input_grad(dq, ds, wq, ws, T.offsets(counts), out)
    d, w = T.rows_value(dq, ds), T.weights_value(wq, ws)
    want = T.grouped(d, w, counts, False)
    tol = T.sum_bound(T.grouped(d.abs(), w.abs(), counts, False), -(-N // 128)) + want.abs() * T.HALF[out] * 1.01
    T.assert_within(got, want, tol)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("f1,f2", [(T.E4, T.E4), (T.E5, T.E4), (T.E4, T.E5)])
@pytest.mark.parametrize("N,C", [(16, 16), (272, 400), (640, 1040), (144, 1856)])
@pytest.mark.parametrize("counts", COUNTS + [[0, 0]], ids=_ids)
def test_product_weight_grad(counts, N, C, f1, f2, out, accumulate):
    g = T.gen(N + C + 2)
    P, E, off = sum(counts), len(counts), T.offsets(counts)
    dy, x = T.randn((P, N), g, scale=1e-3), T.randn((P, C), g)
    dq, ds = ex.quantize_columns(dy, off, f1)
    xq, xs = ex.quantize_columns(x, off, f2)
    dw = torch.randn((E, N, C), generator=g, device="cuda").to(out)
    before = dw.double() if accumulate else torch.zeros((E, N, C), dtype=torch.float64, device="cuda")
    ex.product_weight_grad(dq, ds, xq, xs, off, out, out=dw, accumulate=accumulate)
    want, mag, r = before.clone(), before.abs(), 0
    for e, n in enumerate(counts):
        for _ in range(-(-n // 128)):
            a = dq[r * 128:r * 128 + 128].double() * ds[r].double()
            b = xq[r * 128:r * 128 + 128].double() * xs[r].double()
            want[e] += a.t() @ b
            mag[e] += a.abs().t() @ b.abs()
            r += 1
    T.assert_within(dw, want, T.sum_bound(mag, max(-(-n // 128) for n in counts) + 1) +
                    want.abs() * T.HALF[out] * 1.01)


@pytest.mark.parametrize("h8", [T.E4, T.E5])
@pytest.mark.parametrize("name", ["swiglu", "relu2"])
@pytest.mark.parametrize("I,C", [(16, 16), (128, 256), (640, 2560), (400, 272), (1856, 144)])
@pytest.mark.parametrize("counts", COUNTS, ids=_ids)
def test_product_activation(counts, I, C, name, h8):
    g = T.gen(I + C + 3)
    P, E = sum(counts), len(counts)
    N = 2 * I if name == "swiglu" else I
    xq, xs = ex.quantize_rows(T.randn((P, C), g))
    wq, ws = _weights(E, N, C, g)
    q, s = ex.product_activation(xq, xs, wq, ws, T.offsets(counts), name, h8)
    x, w = T.rows_value(xq, xs), T.weights_value(wq, ws)
    y, ty = T.grouped(x, w, counts, True), T.sum_bound(T.grouped(x.abs(), w.abs(), counts, True), -(-C // 128))
    h = T.act(y, name)
    if name == "swiglu":  # |silu'| <= 1.1; the activation's own error as in the unfused form
        gt, up = y.chunk(2, 1)
        tg, tu = ty.chunk(2, 1)
        tol = 1.1 * tg * (up.abs() + tu) + gt.abs() * torch.sigmoid(gt) * tu + \
            h.abs() * (2 + 1.173 * gt.abs() + 4) * 2.0 ** -23
    else:
        tol = 2 * y.abs() * ty + ty * ty + h.abs() * 2.0 ** -23
    amax = torch.nn.functional.pad(h.abs(), (0, -I % 128)).view(P, -1, 128).amax(2)
    tmax = torch.nn.functional.pad(tol, (0, -I % 128)).view(P, -1, 128).amax(2)
    T.assert_within(s, amax / T.FMAX[h8], (tmax + amax * 2.0 ** -24) / T.FMAX[h8] * 1.01, "scales")
    sc = s.double().repeat_interleave(128, 1)[:, :I]
    T.assert_within(q.double() * sc, h, (h.abs() + tol) * T.HALF[h8] * 1.001 + sc * T.TINY[h8] + tol +
                    h.abs() * 2.0 ** -22, "values")


def test_rows_behind_the_last_expert_are_left():
    g = T.gen(9)
    xq, xs = ex.quantize_rows(T.randn((300, 256), g))
    wq, ws = _weights(2, 256, 256, g)
    off = torch.tensor([0, 100, 170], dtype=torch.int32, device="cuda")
    for f, n in ((ex.product, 256), (ex.product_input_grad, 256)):
        out = torch.full((300, n), 7.0, dtype=BF, device="cuda")
        f(xq, xs, wq, ws, off, out=out)
        assert (out[170:] == 7.0).all()
        assert torch.equal(out[:170], f(xq[:170].contiguous(), xs[:170].contiguous(), wq, ws, off))
    q, s = torch.zeros((300, 128), dtype=torch.uint8, device="cuda").view(T.E4), torch.full((300, 1), 7.0, device="cuda")
    ex.product_activation(xq, xs, wq, ws, off, "swiglu", out=(q, s))
    assert (q[170:].view(torch.uint8) == 0).all() and (s[170:] == 7.0).all() and (s[:170] != 7.0).all()


def test_nan_and_infinite_rows_stay_in_their_rows():
    g = T.gen(10)
    x = T.randn((200, 256), g)
    clean = ex.product(*ex.quantize_rows(x), *_weights(1, 384, 256, T.gen(11)))
    x[5, 3], x[77, 200], x[199, 0] = float("nan"), float("inf"), float("-inf")
    got = ex.product(*ex.quantize_rows(x), *_weights(1, 384, 256, T.gen(11)))
    bad = torch.zeros(200, dtype=torch.bool, device="cuda")
    bad[[5, 77, 199]] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])


def test_offsets_outside_the_rows_are_clamped():
    """Offsets a caller got wrong read and write no row outside the buffers."""
    g = T.gen(12)
    xq, xs = ex.quantize_rows(T.randn((64, 128), g))
    wq, ws = _weights(3, 128, 128, g)
    off = torch.tensor([-5, 40, 1 << 30, 20], dtype=torch.int32, device="cuda")
    out = ex.product(xq, xs, wq, ws, off)
    good = ex.product(xq, xs, wq, ws, torch.tensor([0, 40, 64, 64], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, good)
