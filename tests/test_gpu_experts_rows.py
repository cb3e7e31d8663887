"""Tokens sorted by expert and back with their gradients, the 8-bit quantisers and the
activation, against plain forms: copies and roundings exactly, sums in 64 bits."""
import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# M tokens, K slots, H features, P rows kept of the M K slots
SLOTS = [(1, 1, 8, 1), (1, 1, 16, 0), (1, 8, 2048, 8), (3, 2, 24, 5), (5, 32, 264, 160), (257, 10, 2560, 2570),
         (300, 3, 1000, 1), (2047, 6, 2688, 12000), (4096, 8, 128, 32768), (64, 4, 20000, 200)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,H,P", SLOTS)
def test_dispatch_copies_rows_and_leaves_the_rest(M, K, H, P, dtype):
    g = T.gen(M + H)
    x, inv = T.randn((M, H), g, dtype), T.slots(M, K, P, g)
    out = torch.full((P + 3, H), 7.0, dtype=dtype, device="cuda")
    want = out.clone()
    src = torch.nonzero((inv >= 0) & (inv < P)).view(-1)
    inv2 = torch.where(inv >= P, inv + 3, inv)  # out has three more rows; dropped slots stay outside
    want[inv[src].long()] = x[src % M]
    got = ex.dispatch(x, inv2, P + 3, out=out)
    assert got is out and torch.equal(got, want)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,H,P", SLOTS)
def test_combine(M, K, H, P, dtype, weighted):
    g = T.gen(M + H + 1)
    ys, inv = T.randn((P, H), g, dtype), T.slots(M, K, P, g)
    w = torch.randn((M, K), generator=g, device="cuda")
    kept = ((inv >= 0) & (inv < P)).view(K, M)
    w = torch.where(kept.t(), w, torch.full_like(w, float("nan"))).contiguous()  # a dropped slot's weight is not used
    rows = torch.zeros((K, M, H), dtype=torch.float64, device="cuda")
    rows[kept] = ys[inv.view(K, M)[kept].long()].double()
    terms = rows * torch.where(kept.t(), w, 0).t().double()[:, :, None] if weighted else rows
    got = ex.combine(ys, inv, w) if weighted else ex.dispatch_backward(ys, inv, M)
    want = terms.sum(0)
    # one rounding of the running sum a slot, and one to the type
    T.assert_within(got, want, terms.abs().sum(0) * (K + 1) * 2.0 ** -24 + want.abs() * T.HALF[dtype] * 1.01)
    again = ex.combine(ys, inv, w) if weighted else ex.dispatch_backward(ys, inv, M)
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,H,P", SLOTS)
def test_combine_backward(M, K, H, P, dtype):
    g = T.gen(M + H + 2)
    dy, ys, inv = T.randn((M, H), g, dtype), T.randn((P, H), g, dtype), T.slots(M, K, P, g)
    w = torch.randn((M, K), generator=g, device="cuda")
    out = torch.full((P, H), 7.0, dtype=dtype, device="cuda"), torch.full((M, K), 7.0, device="cuda")
    dys, dw = ex.combine_backward(dy, ys, inv, w, out=out)
    want, wdw, tol = torch.full((P, H), 7.0, dtype=dtype, device="cuda"), torch.zeros_like(w).double(), \
        torch.zeros_like(w).double()
    for k in range(K):
        m = torch.nonzero((inv[k * M:k * M + M] >= 0) & (inv[k * M:k * M + M] < P)).view(-1)
        p = inv[k * M:k * M + M][m].long()
        want[p] = (w[m, k][:, None] * dy[m].float()).to(dtype)
        prod = dy[m].double() * ys[p].double()
        wdw[m, k], tol[m, k] = prod.sum(1), prod.abs().sum(1)
    assert torch.equal(dys, want)
    # a lane adds H / 32 products in turn (rounded up to its chunks), the lanes five times
    T.assert_within(dw, wdw, tol * (H / 32 + 16 + 5) * 2.0 ** -24)


def test_gradients_match_differences():
    """combine is linear in the rows and in the weights, so a difference is its gradient up to rounding."""
    g = T.gen(3)
    M, K, H = 37, 4, 128
    P = M * K - 9
    inv = T.slots(M, K, P, g)
    ys, w, dy = T.randn((P, H), g), torch.rand((M, K), generator=g, device="cuda"), T.randn((M, H), g)
    dys, dw = ex.combine_backward(dy, ys, inv, w, out=(torch.zeros_like(ys), torch.empty_like(w)))
    d_ys, d_w = T.randn((P, H), g), torch.randn((M, K), generator=g, device="cuda")
    f = lambda a, b: (ex.combine(a, inv, b).double() * dy.double()).sum()  # noqa: E731
    base, size = f(ys, w), (ex.combine(ys.abs(), inv, w).double() * dy.abs().double()).sum()
    for diff, grad, s in ((f(ys + d_ys, w) - base, (dys.double() * d_ys.double()).sum(), d_ys.abs().max()),
                          (f(ys, w + d_w) - base, (dw.double() * d_w.double()).sum(), d_w.abs().max())):
        assert abs(diff - grad) <= 40 * 2.0 ** -24 * size * (2 + s)


QUANT = [(1, 16), (1, 2048), (3, 144), (130, 1856), (1000, 112), (77, 2688), (2048, 512)]


def _special(x):
    """Zeros, the smallest and largest values, infinities and NaN in some blocks."""
    x = x.clone()
    R, C = x.shape
    x[0, :min(C, 128)] = 0
    if R > 2:
        x[1, :] = 1e-38
        x[1, 0] = 1e-36
        x[2, -1] = 3e38
    if R > 70:
        x[5, 3], x[6, 5], x[7, 1] = float("nan"), float("inf"), float("-inf")
        x[9, C - 1], x[9, C - 2] = float("inf"), float("nan")
    return x


def _same8(got, want):
    got, want = got.cpu(), want.cpu()
    a, b = got.float(), want.float()
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(got.view(torch.uint8)[~a.isnan()], want.view(torch.uint8)[~a.isnan()])


def _same32(got, want):
    assert torch.equal(got.cpu().nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C", QUANT)
def test_quantize_rows(R, C, dtype, fp8):
    x = _special(T.randn((R, C), T.gen(R + C)).float()).to(dtype)
    q, s = ex.quantize_rows(x, fp8)
    wq, ws = T.quant_rows(x, fp8)
    _same8(q, wq)
    _same32(s, ws)


@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,H,P", [(1, 8, 2048, 8), (1, 1, 16, 0), (5, 32, 272, 150), (2047, 6, 2688, 12000),
                                     (300, 3, 1008, 900)])
def test_dispatch_quantize(M, K, H, P, dtype, fp8):
    g = T.gen(M + H + 5)
    x, inv = T.randn((M, H), g, dtype), T.slots(M, K, P, g)
    q, s = ex.dispatch_quantize(x, inv, P, fp8)
    assert q.shape == (P, H) and s.shape == (P, -(-H // 128))
    src = torch.zeros(P, dtype=torch.long)
    at = torch.nonzero((inv >= 0) & (inv < P)).view(-1)
    src[inv[at].long().cpu()] = at.cpu()
    wq, ws = T.quant_rows(x, fp8)
    _same8(q, wq.view(torch.uint8)[src % M].view(fp8))
    _same32(s, ws[src % M])


@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,N,C", [(1, 16, 16), (3, 128, 256), (2, 1856, 144), (5, 272, 2688)])
def test_quantize_blocks(E, N, C, dtype, fp8):
    w = T.randn((E, N, C), T.gen(E + N))
    w[0, :128, :128] = 0
    w[-1, -1, -1] = 1e6
    if E > 1:
        w[0, 5, C - 1] = float("nan")
    w = w.to(dtype)
    q, s = ex.quantize_blocks(w, fp8)
    wq, ws = T.quant_blocks(w, fp8)
    _same8(q, wq)
    _same32(s, ws)


COUNTS = [[1], [0, 1, 0], [128, 128], [127, 129, 0, 300, 5], [0] * 40 + [513] + [0] * 23, [3] * 300, [1] * 1024]


@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}experts{sum(c)}rows")
@pytest.mark.parametrize("C", [16, 400])
def test_quantize_columns(counts, C, dtype, fp8):
    P = sum(counts)
    x = _special(T.randn((P, C), T.gen(P + C)).float()).to(dtype)
    B = ex.column_blocks(P, len(counts))
    q = torch.full((B * 128, C), 0x55, dtype=torch.uint8, device="cuda").view(fp8)
    s = torch.full((B, C), 7.0, device="cuda")
    ex.quantize_columns(x, T.offsets(counts), fp8, out=(q, s))
    wq, ws = T.quant_columns(x, counts, fp8)
    n = len(ws)
    assert n <= B
    _same8(q[:n * 128], wq)
    _same32(s[:n], ws)
    assert (q[n * 128:].view(torch.uint8) == 0x55).all() and (s[n:] == 7.0).all()
    if len(counts) == 1:  # one expert needs no offsets
        q2, s2 = ex.quantize_columns(x, None, fp8)
        _same8(q2[:n * 128], wq)


def _act_tolerance(y, h, name, dtype):
    """SwiGLU takes one __expf (off by 2 + 1.173 |g| units of 2^-23), a sum, a quotient and a product."""
    if name == "relu2":
        return h.abs() * (T.HALF[dtype] * 1.01 + 2.0 ** -23)
    g = y[:, :y.shape[1] // 2].double().abs()
    return h.abs() * (T.HALF[dtype] * 1.01 + (2 + 1.173 * g + 3) * 2.0 ** -23) + 2.0 ** -120


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["swiglu", "relu2"])
@pytest.mark.parametrize("P,I", [(1, 8), (3, 136), (700, 1856), (4100, 512)])
def test_activation_and_its_gradient(P, I, name, dtype):
    g = T.gen(P + I)
    y = T.randn((P, 2 * I if name == "swiglu" else I), g, dtype)
    y[0, :4] = torch.tensor([0.0, -0.0, 80.0, -80.0])
    dh = T.randn((P, I), g, dtype)
    h = T.act(y.double(), name)
    T.assert_within(ex.activation(y, name), h, _act_tolerance(y, h, name, dtype))
    yd = y.double().requires_grad_()
    T.act(yd, name).backward(dh.double())
    want = yd.grad
    got = ex.activation_backward(y, dh, name)
    rel = T.HALF[dtype] * 1.01
    if name == "relu2":
        tol = want.abs() * (rel + 2.0 ** -22)
    else:
        gd, ud = y.double().chunk(2, 1)
        sg = torch.sigmoid(gd)
        err = (2 + 1.173 * gd.abs() + 4) * 2.0 ** -23  # of the sigmoid, and the products after it
        # dg = dh u (sg + g sg (1 - sg)): the sum's terms may cancel; 1 - sg carries sg's error
        tg = (dh.double() * ud).abs() * (sg + (gd * sg).abs() * (1 + sg / (1 - sg).clamp(min=2.0 ** -24))
                                         .clamp(max=1e9) * (1 - sg) + (gd * sg).abs() * 2.0 ** -1) * err * 2
        tu = (dh.double() * gd * sg).abs() * err
        # Below g = -ln(FLT_MAX) = -88.7, e^-g is infinite in FP32 and sg is 0 where it is below 1 / FLT_MAX = 2^-128:
        # sg is off by less than 2^-127 there, dg by that times |dh u| (1 + |g|) and du by that times |dh g|.
        tg = tg + (dh.double() * ud).abs() * (1 + gd.abs()) * 2.0 ** -127
        tu = tu + (dh.double() * gd).abs() * 2.0 ** -127
        tol = want.abs() * rel + torch.cat([tg, tu], 1) + 2.0 ** -120
    T.assert_within(got, want, tol)


def test_activation_keeps_nan():
    y = torch.tensor([[float("nan"), 1.0, -2.0, 3.0, 0.0, -0.0, 2.0, float("inf")]], device="cuda")
    h = ex.activation(y, "relu2")
    assert h[0, 0].isnan() and h[0, 1:].tolist() == [1.0, 0.0, 9.0, 0.0, 0.0, 4.0, float("inf")]
    z = torch.ones((1, 16), device="cuda")
    z[0, 0], z[0, 9] = float("nan"), float("nan")
    h = ex.activation(z, "swiglu")
    assert h[0, 0].isnan() and h[0, 1].isnan() and not h[0, 2:].isnan().any()


@pytest.mark.parametrize("fp8", [T.E4, T.E5])
@pytest.mark.parametrize("name", ["swiglu", "relu2"])
@pytest.mark.parametrize("P,I,dtype", [(1, 16, F32), (300, 1856, BF), (5, 640, BF), (2000, 144, F32)])
def test_activation_quantize(P, I, name, fp8, dtype):
    y = T.randn((P, 2 * I if name == "swiglu" else I), T.gen(P * I), dtype)
    q, s = ex.activation_quantize(y, name, fp8)
    h = T.act(y.double(), name)
    tol = _act_tolerance(y, h, name, F32)
    amax = torch.nn.functional.pad(h.abs(), (0, -I % 128)).view(P, -1, 128).amax(2)
    tmax = torch.nn.functional.pad(tol, (0, -I % 128)).view(P, -1, 128).amax(2)
    T.assert_within(s, amax / T.FMAX[fp8], (tmax + amax * 2.0 ** -24) / T.FMAX[fp8] * 1.01, "scales")
    sc = s.double().repeat_interleave(128, 1)[:, :I]
    # half a step of the 8-bit type, of the value as the kernel has it; its factor and product are rounded
    T.assert_within(q.double() * sc, h, (h.abs() + tol) * T.HALF[fp8] * 1.001 + sc * T.TINY[fp8] + tol +
                    h.abs() * 2.0 ** -22)
