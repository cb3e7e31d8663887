"""The grouped products where every kernel variant is met: many tiles per block, 32- and 64-row tiles, narrow and
wide tiles of the weight gradient, 1024 experts; against 64 bits, and the same bits run to run."""
import pytest
import torch

from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# 30 and 50 rows an expert take 64-row tiles (50: SwiGLU only); the long lists have several tiles for each of
# the 148 blocks, with empty experts and ragged ends among them
MANY = [[30] * 8, [50] * 6, [70, 0, 20, 33, 64, 65, 1], [(37 * i) % 230 for i in range(40)], [(5 * i) % 40 for i in range(64)],
        [1500, 900], [1] * 1024]


def _ids(c):
    return f"{len(c)}x{sum(c)}"


def _operands(counts, N, C, seed):
    g = T.gen(seed)
    P, E = sum(counts), len(counts)
    w = ex.quantize_blocks(T.randn((E, N, C), g, scale=C ** -0.5))
    return g, P, w, T.offsets(counts)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("counts", MANY, ids=_ids)
def test_products(counts, out):
    N, C = (1040, 528) if len(counts) < 100 else (144, 272)
    g, P, w, off = _operands(counts, N, C, 31)
    wv = T.weights_value(*w)
    for f, cols, transposed, depth in ((ex.product, C, True, C), (ex.product_input_grad, N, False, N)):
        q = ex.quantize_rows(T.randn((P, cols), g))
        got = f(*q, *w, off, out)
        v = T.rows_value(*q)
        want = T.grouped(v, wv, counts, transposed)
        tol = T.sum_bound(T.grouped(v.abs(), wv.abs(), counts, transposed), -(-depth // 128)) + \
            want.abs() * T.HALF[out] * 1.01
        T.assert_within(got, want, tol, f.__name__)
        assert torch.equal(got, f(*q, *w, off, out))
    assert ex.get_error() == 0


@pytest.mark.parametrize("name", ["swiglu", "relu2"])
@pytest.mark.parametrize("counts", MANY, ids=_ids)
def test_fused_activation(counts, name):
    """Against the product and the activation one after the other, both in FP32 here: the same values up to the
    rounding of the sums, so the 8-bit values are at most one step apart, and equal but for a few."""
    I, C = (528, 656) if len(counts) < 100 else (80, 272)
    g, P, w, off = _operands(counts, 2 * I if name == "swiglu" else I, C, 32)
    q = ex.quantize_rows(T.randn((P, C), g))
    hq, hs = ex.product_activation(*q, *w, off, name)
    aq, as_ = ex.activation_quantize(ex.product(*q, *w, off, F32), name)
    # Both sum the same blocks in FP32; their order of rounding differs by at most the sums' bound, which the
    # activation passes on; held to 2^-10 of the row's largest value in its block of 128 features.
    sc, sa = (s.double().repeat_interleave(128, 1)[:, :I] for s in (hs, as_))
    T.assert_within(hs, as_, as_.double() * 2.0 ** -10, "scales")
    step = (hq.double() * sc).abs() * 2 * T.HALF[T.E4] * 1.01 + 2 * sa * T.TINY[T.E4]
    T.assert_within(hq.double() * sc, aq.double() * sa, step + sa * 448 * 2.0 ** -10, "values")
    assert (hq.view(torch.uint8) != aq.view(torch.uint8)).float().mean() < 0.02
    again = ex.product_activation(*q, *w, off, name)
    assert torch.equal(hq.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(hs, again[1])


@pytest.mark.parametrize("out,accumulate", [(F32, False), (F32, True), (BF, False), (BF, True)])
@pytest.mark.parametrize("counts", MANY, ids=_ids)
def test_weight_gradient(counts, out, accumulate):
    N, C = (656, 528) if len(counts) < 100 else (144, 272)
    g = T.gen(33)
    P, E, off = sum(counts), len(counts), T.offsets(counts)
    d, x = ex.quantize_columns(T.randn((P, N), g, scale=1e-2), off, T.E5), ex.quantize_columns(T.randn((P, C), g), off)
    dw = torch.randn((E, N, C), generator=g, device="cuda").to(out)
    want = dw.double() if accumulate else torch.zeros((E, N, C), dtype=torch.float64, device="cuda")
    mag = want.abs()
    ex.product_weight_grad(*d, *x, off, out, out=dw, accumulate=accumulate)
    b = 0
    for e, n in enumerate(counts):
        k = -(-n // 128)
        a = (d[0][b * 128:(b + k) * 128].double().view(k, 128, N) * d[1][b:b + k, None].double()).flatten(0, 1)
        v = (x[0][b * 128:(b + k) * 128].double().view(k, 128, C) * x[1][b:b + k, None].double()).flatten(0, 1)
        want[e] += a.t() @ v
        mag[e] += a.abs().t() @ v.abs()
        b += k
    T.assert_within(dw, want, T.sum_bound(mag, max(-(-n // 128) for n in counts) + 1) +
                    want.abs() * T.HALF[out] * 1.01)
    assert ex.get_error() == 0


@pytest.mark.parametrize("P", [1, 127, 128, 256, 300])
def test_one_expert_without_offsets(P):
    """All blocks are the expert's then, the one that P leaves empty too: what lay in the buffers before
    (here NaN) must not reach the weight gradient."""
    N, C = 144, 272
    g = T.gen(P)
    dy, x = T.randn((P, N), g, BF), T.randn((P, C), g, BF)
    B = ex.column_blocks(P, 1)

    def room(cols):
        return (torch.full((B * 128, cols), 0x7f, dtype=torch.uint8, device="cuda").view(T.E4),
                torch.full((B, cols), float("nan"), device="cuda"))

    d, xq = ex.quantize_columns(dy, out=room(N)), ex.quantize_columns(x, out=room(C))
    dw = ex.product_weight_grad(*d, *xq)
    off = T.offsets([P])
    want = ex.product_weight_grad(*ex.quantize_columns(dy, off, out=room(N)), *ex.quantize_columns(x, off, out=room(C)), off)
    assert torch.equal(dw, want) and not dw.isnan().any()
    w = ex.quantize_blocks(T.randn((1, N, C), g))
    q = ex.quantize_rows(x)
    assert torch.equal(ex.product(*q, *w), ex.product(*q, *w, off))
    assert torch.equal(ex.product_input_grad(*ex.quantize_rows(dy), *w), ex.product_input_grad(*ex.quantize_rows(dy), *w, off))
    a, b = ex.product_activation(*q, *w, act="relu2"), ex.product_activation(*q, *w, off, "relu2")
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("E", [1, 2, 31, 257, 1000, 1024])
def test_any_offsets_give_disjoint_rows(E):
    """Offsets that are no prefix sums act as their running maximum, clamped to the rows there are."""
    g = T.gen(E)
    P, N, C = 500, 32, 144
    raw = torch.randint(-200, 900, (E + 1,), generator=g, device="cuda")
    raw[::3] = torch.randint(0, P, raw[::3].shape, generator=g, device="cuda")
    raw = (raw // max(1, 8 - E)).int() if E < 8 else raw.int()
    good = raw.clamp(0, P).long().cummax(0).values.int()
    w = ex.quantize_blocks(T.randn((E, N, C), g))
    q = ex.quantize_rows(T.randn((P, C), g))
    a, b = (torch.full((P, N), 7.0, dtype=BF, device="cuda") for _ in range(2))
    ex.product(*q, *w, raw, out=a)
    ex.product(*q, *w, good, out=b)
    assert torch.equal(a, b) and (a[:int(good[0])] == 7.0).all() and (a[int(good[-1]):] == 7.0).all()
    x, dy = T.randn((P, C), g), T.randn((P, N), g)
    B = ex.column_blocks(P, E)

    def columns(t, off):
        out = torch.zeros((B * 128, t.shape[1]), dtype=torch.uint8, device="cuda").view(T.E4), \
            torch.zeros((B, t.shape[1]), device="cuda")
        return ex.quantize_columns(t, off, out=out)

    for t in (x, dy):
        c, d = columns(t, raw), columns(t, good)
        assert torch.equal(c[0].view(torch.uint8), d[0].view(torch.uint8)) and torch.equal(c[1], d[1])
    assert torch.equal(ex.product_weight_grad(*columns(dy, raw), *columns(x, raw), raw),
                       ex.product_weight_grad(*columns(dy, good), *columns(x, good), good))
    assert ex.get_error() == 0
