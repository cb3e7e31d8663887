"""Weight gradients where fewer rows were kept than the offsets name (a capacity limit): what lies in buffers
that nobody wrote (here NaN) must not reach them."""
import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# P rows that are there, and the rows that the offsets give each expert
LIMITS = [(100, [100, 200]), (100, [300]), (1, [0, 5, 5]), (200, [90, 90, 90]), (1000, [200] * 8), (128, [128, 128]),
          (129, [1, 300, 0, 7]), (700, [3] * 300), (513, [0] * 40 + [513] + [0] * 22 + [1]), (640, [640, 0, 0])]


def _ids(c):
    return f"{c[0]}of{sum(c[1])}"


def _nan_room(B, cols, fp8):
    return (torch.full((B * 128, cols), 0x7f, dtype=torch.uint8, device="cuda").view(fp8),
            torch.full((B, cols), float("nan"), device="cuda"))


def _kept(P, counts):
    """Rows of each expert that are there."""
    out, r = [], 0
    for n in counts:
        out.append(max(0, min(r + n, P) - r))
        r += n
    return out


def _want(dy, x, kept, f1, f2, E, N, C):
    """The gradient in 64 bits from the plain quantiser's blocks of the rows that are there."""
    (dq, ds), (xq, xs) = T.quant_columns(dy, kept, f1), T.quant_columns(x, kept, f2)
    want = torch.zeros((E, N, C), dtype=torch.float64)
    mag, b = torch.zeros_like(want), 0
    for e, n in enumerate(kept):
        for _ in range(-(-n // 128)):
            r = slice(b * 128, b * 128 + 128)
            p, q = dq[r].double() * ds[b].double(), xq[r].double() * xs[b].double()
            want[e] += p.t() @ q
            mag[e] += p.abs().t() @ q.abs()
            b += 1
    return want.cuda(), mag.cuda()


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("f1", [T.E4, T.E5])
@pytest.mark.parametrize("limit", LIMITS, ids=_ids)
def test_weight_gradient_of_the_rows_that_are_there(limit, f1, out):
    P, counts = limit
    E, N, C = len(counts), 144, 272
    g = T.gen(P + E)
    dy, x, off = T.randn((P, N), g, BF, 1e-2), T.randn((P, C), g, BF), T.offsets(counts)
    B = ex.column_blocks(P, E)
    d = ex.quantize_columns(dy, off, f1, out=_nan_room(B, N, f1))
    q = ex.quantize_columns(x, off, out=_nan_room(B, C, T.E4))
    kept = _kept(P, counts)
    want, mag = _want(dy, x, kept, f1, T.E4, E, N, C)
    tol = T.sum_bound(mag, max(-(-n // 128) for n in kept) + 1) + want.abs() * T.HALF[out] * 1.01
    dw = ex.product_weight_grad(*d, *q, off, out)
    T.assert_within(dw, want, tol)
    # The same offsets, clamped by the caller, give the same bits.
    good = off.clamp(max=P)
    again = ex.product_weight_grad(*ex.quantize_columns(dy, good, f1, out=_nan_room(B, N, f1)),
                                   *ex.quantize_columns(x, good, out=_nan_room(B, C, T.E4)), good, out)
    assert torch.equal(dw, again)
    # Added to what is there: nothing for an expert whose rows are all missing.
    acc = torch.full((E, N, C), 0.5, dtype=out, device="cuda")
    ex.product_weight_grad(*d, *q, off, out, out=acc, accumulate=True)
    T.assert_within(acc, want + 0.5, T.sum_bound(mag + 0.5, max(-(-n // 128) for n in kept) + 2) +
                    (want + 0.5).abs() * T.HALF[out] * 1.01)
    for e, n in enumerate(kept):
        if n == 0:
            assert (dw[e] == 0).all() and (acc[e] == 0.5).all()
    assert ex.get_error() == 0


@pytest.mark.parametrize("limit", LIMITS, ids=_ids)
def test_blocks_of_missing_rows_are_zeros(limit):
    """The blocks of the rows that are there as without a limit; those that the offsets name besides, as far as
    there is room, zeros; the ones behind them left."""
    P, counts = limit
    E, C = len(counts), 48
    x, off = T.randn((P, C), T.gen(P), BF), T.offsets(counts)
    B = ex.column_blocks(P, E)
    q, s = torch.full((B * 128, C), 0x55, dtype=torch.uint8, device="cuda").view(T.E4), \
        torch.full((B, C), 7.0, device="cuda")
    ex.quantize_columns(x, off, out=(q, s))
    wq, ws = T.quant_columns(x, _kept(P, counts), T.E4)
    n = len(ws)
    assert torch.equal(q[:n * 128].cpu().view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s[:n].cpu(), ws)
    top = off.long().clamp(max=B * 128)
    named = min(B, int(((top[1:] - top[:-1] + 127) // 128).sum()))
    assert named >= n
    assert (q[n * 128:named * 128].view(torch.uint8) == 0).all() and (s[n:named] == 0).all()
    assert (q[named * 128:].view(torch.uint8) == 0x55).all() and (s[named:] == 7.0).all()


def test_training_step_with_a_row_limit():
    """Offsets as moe.permute writes them, fewer rows than slots: every gradient of the kept rows."""
    M, H, I, E, K, R = 120, 256, 144, 6, 3, 250
    g = T.gen(22)
    x = torch.randn((M, H), generator=g, device="cuda").to(BF)
    ids = torch.rand((M, E), generator=g, device="cuda").topk(K, 1).indices.int()
    dy = torch.randn((M, H), generator=g, device="cuda").to(BF)
    rw = torch.rand((M, K), generator=g, device="cuda")
    w = ex.quantize_blocks(torch.randn((E, I, H), generator=g, device="cuda") * H ** -0.5)
    offsets, perm, inv = moe.permute(ids, E)
    counts = (offsets[1:] - offsets[:-1]).tolist()
    kept = _kept(R, counts)
    xs = ex.dispatch(x, inv, R)
    assert torch.equal(xs, x[perm[:R].long() % M])
    ys = ex.product(*ex.quantize_rows(xs), *w, offsets)
    assert ys.shape == (R, I)
    dys = T.randn((R, I), g, BF, 1e-2)
    B = ex.column_blocks(R, E)
    d = ex.quantize_columns(dys, offsets, out=_nan_room(B, I, T.E4))
    q = ex.quantize_columns(xs, offsets, out=_nan_room(B, H, T.E4))
    dw = ex.product_weight_grad(*d, *q, offsets)
    want, mag = _want(dys, xs, kept, T.E4, T.E4, E, I, H)
    T.assert_within(dw, want, T.sum_bound(mag, max(-(-n // 128) for n in kept) + 1) + want.abs() * T.HALF[F32] * 1.01)
    dxs = ex.product_input_grad(*ex.quantize_rows(dys), *w, offsets)
    assert not dxs.isnan().any() and not ex.dispatch_backward(dxs, inv, M).isnan().any()
    y = torch.zeros((R, H), dtype=BF, device="cuda")
    drows, drw = ex.combine_backward(dy, y, inv, rw)
    slot = perm.long()
    assert torch.equal(drows, (rw[slot[:R] % M, slot[:R] // M][:, None] * dy[slot[:R] % M].float()).to(BF))
    assert (drw == 0).all()


@pytest.mark.parametrize("P", [1, 128, 256, 300])
def test_blocks_without_rows_and_without_offsets_are_zeros(P):
    B = ex.column_blocks(P, 1)
    q, s = ex.quantize_columns(T.randn((P, 48), T.gen(P), BF), out=_nan_room(B, 48, T.E4))
    n = -(-P // 128)
    assert (s[:n] > 0).all() and (s[n:] == 0).all() and (q[P:].view(torch.uint8) == 0).all()
