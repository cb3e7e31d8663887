"""The products at the ends of the range in which the product of two scales keeps FP32's precision: blocks whose
largest magnitudes multiply to between 2^-94 and 2^145."""
import pytest
import torch

from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
F32 = torch.float32
COUNTS = [40, 0, 130, 6]

# powers of two of the rows and of the weights (or of x): values of both are normal, so a block's largest is near 1
# to 4 times that; the sums stay in FP32's normal range, and so do the operands
SIZES = [(-40, -50), (-80, -10), (-10, -80), (55, 55), (-90, 90), (100, 10)]


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("a,b", SIZES)
def test_products_of_small_and_large_values(a, b, few):
    counts = COUNTS if not few else [3, 0, 9, 1]
    N, C, P, E, g = 144, 272, sum(counts), len(counts), T.gen(a + 200)
    off = T.offsets(counts)
    x = torch.randn((P, C), generator=g, device="cuda") * 2.0 ** a
    w = torch.randn((E, N, C), generator=g, device="cuda") * 2.0 ** b
    wq, xq = ex.quantize_blocks(w), ex.quantize_rows(x)
    v, wv = T.rows_value(*xq), T.weights_value(*wq)
    got, want = ex.product(*xq, *wq, off, F32), T.grouped(v, wv, counts, True)
    T.assert_within(got, want, T.sum_bound(T.grouped(v.abs(), wv.abs(), counts, True), 3) + want.abs() * 2.0 ** -24)
    dy = torch.randn((P, N), generator=g, device="cuda") * 2.0 ** b
    d, q = ex.quantize_columns(dy, off), ex.quantize_columns(x, off)
    dw = ex.product_weight_grad(*d, *q, off)
    r = 0
    for e, n in enumerate(counts):
        k = -(-n // 128)
        p = (d[0][r * 128:(r + k) * 128].double().view(k, 128, N) * d[1][r:r + k, None].double()).flatten(0, 1)
        t = (q[0][r * 128:(r + k) * 128].double().view(k, 128, C) * q[1][r:r + k, None].double()).flatten(0, 1)
        want = p.t() @ t
        T.assert_within(dw[e], want, T.sum_bound(p.abs().t() @ t.abs(), k + 1) + want.abs() * 2.0 ** -24)
        r += k
