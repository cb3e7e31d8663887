"""Runs of the expert operators as they are used: a served layer, a training step, other streams, captured
graphs, long buffers; and the binding's refusals."""
import pytest
import torch

import mixture_experts_layer_35_b200.moe as moe
from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _layer(M, H, I, E, K, act, seed):
    g = T.gen(seed)
    n = 2 * I if act == "swiglu" else I
    return {"x": torch.randn((M, H), generator=g, device="cuda").to(BF),
            "logits": torch.randn((M, E), generator=g, device="cuda"),
            "w1": ex.quantize_blocks(torch.randn((E, n, H), generator=g, device="cuda") * H ** -0.5),
            "w2": ex.quantize_blocks(torch.randn((E, H, I), generator=g, device="cuda") * I ** -0.5),
            "g": g}


def _serve(d, K, E, act, stream=None):
    w, ids, _ = moe.router_topk(d["logits"], K, stream=stream)
    offsets, perm, inv = moe.permute(ids, E, ws=d.get("ws"), stream=stream)
    xq, xs = ex.dispatch_quantize(d["x"], inv, stream=stream)
    hq, hs = ex.product_activation(xq, xs, *d["w1"], offsets, act, stream=stream)
    return ex.combine(ex.product(hq, hs, *d["w2"], offsets, stream=stream), inv, w, stream=stream)


def _serve_exact(d, K, E, act):
    """The same layer in 64 bits, with the 8-bit rows and weights as the operators' definition gives them."""
    s = torch.sigmoid(d["logits"].double())
    w, ids = s.topk(K, dim=1)
    w = w / w.sum(1, keepdim=True)
    x = T.rows_value(*(t.cuda() for t in T.quant_rows(d["x"], T.E4)))
    w1, w2 = T.weights_value(*d["w1"]), T.weights_value(*d["w2"])
    y = torch.zeros_like(x)
    for e in range(E):
        m, k = torch.nonzero(ids == e, as_tuple=True)
        if len(m):
            h = T.act(x[m] @ w1[e].t(), act)
            h = T.rows_value(*(t.cuda() for t in T.quant_rows(h.float(), T.E4)))
            y.index_add_(0, m, (h @ w2[e].t()) * w[m, k][:, None])
    return y


# bf16 outputs and intermediate rows, and 8-bit activations that may round the other way at a border:
# each of the K rows is off by half a BF16 step, and where an activation's 8-bit value moves by a step
# (2^-3 of it), by that share of its part of the sum.  Held to 2^-7 of the row's largest value.
SERVE = [(1, 256, 128, 8, 2, "swiglu"), (33, 512, 208, 16, 4, "swiglu"), (700, 256, 400, 5, 3, "relu2"),
         (64, 1024, 640, 64, 8, "swiglu")]


@pytest.mark.parametrize("M,H,I,E,K,act", SERVE)
def test_served_layer(M, H, I, E, K, act):
    d = _layer(M, H, I, E, K, act, M + E)
    y = _serve(d, K, E, act).double()
    want = _serve_exact(d, K, E, act)
    T.assert_within(y, want, want.abs().amax(1, keepdim=True) * 2.0 ** -7)
    assert ex.get_error() == 0


def test_training_step_gradients():
    """An expert layer's step in 8 bits: every gradient against the formula in 64 bits on the operands that
    the step's products really had."""
    M, H, I, E, K = 300, 256, 144, 7, 3
    g = T.gen(21)
    x = torch.randn((M, H), generator=g, device="cuda").to(BF)
    ids = torch.rand((M, E), generator=g, device="cuda").topk(K, 1).indices.int()
    rw = torch.rand((M, K), generator=g, device="cuda")
    w1 = ex.quantize_blocks(torch.randn((E, 2 * I, H), generator=g, device="cuda") * H ** -0.5)
    w2 = ex.quantize_blocks(torch.randn((E, H, I), generator=g, device="cuda") * I ** -0.5)
    dy = torch.randn((M, H), generator=g, device="cuda").to(BF)
    offsets, perm, inv = moe.permute(ids, E)
    counts = (offsets[1:] - offsets[:-1]).tolist()
    # forward
    xs = ex.dispatch(x, inv)
    xr = ex.quantize_rows(xs)
    y1 = ex.product(*xr, *w1, offsets)
    hr = ex.activation_quantize(y1, "swiglu")
    ys = ex.product(*hr, *w2, offsets)
    ex.combine(ys, inv, rw)
    # backward
    dys, drw = ex.combine_backward(dy, ys, inv, rw)
    dyr = ex.quantize_rows(dys, T.E5)
    dh = ex.product_input_grad(*dyr, *w2, offsets)
    dw2 = ex.product_weight_grad(*ex.quantize_columns(dys, offsets, T.E5),
                                 *ex.quantize_columns(ex.activation(y1, "swiglu"), offsets), offsets)
    dy1 = ex.activation_backward(y1, dh, "swiglu")
    dw1 = ex.product_weight_grad(*ex.quantize_columns(dy1, offsets), *ex.quantize_columns(xs, offsets), offsets)
    dxs = ex.product_input_grad(*ex.quantize_rows(dy1), *w1, offsets)
    dx = ex.dispatch_backward(dxs, inv, M)
    # the formula in 64 bits, from the unquantised rows
    w1v, w2v = T.weights_value(*w1), T.weights_value(*w2)
    xd, rd = x.double().requires_grad_(), rw.double().requires_grad_()
    w1d, w2d = w1v.clone().requires_grad_(), w2v.clone().requires_grad_()
    rows = torch.zeros((M * K, H), dtype=torch.float64, device="cuda")
    tok = (perm.long() % M)
    xsd = xd[tok]
    ysd = T.grouped(T.act(T.grouped(xsd, w1d, counts, True), "swiglu"), w2d, counts, True)
    yd = torch.zeros((M, H), dtype=torch.float64, device="cuda").index_add(
        0, tok, ysd * rd[tok, perm.long() // M][:, None])
    yd.backward(dy.double())
    # Every 8-bit operand is off by up to 2^-4 (e4m3) or 2^-3 (e5m2) of its values; independent errors of that
    # size (root mean square 0.6 of half a step) through the chain leave each gradient within 15 % in norm.
    for name, got, want in (("dx", dx, xd.grad), ("dweights", drw, rd.grad), ("dw1", dw1, w1d.grad),
                            ("dw2", dw2, w2d.grad)):
        off = (got.double() - want).norm() / want.norm()
        assert off <= 0.15, f"{name}: {off:.3f}"


def test_other_stream_and_external_handle():
    M, H, I, E, K, act = 200, 256, 128, 6, 2, "swiglu"
    d = _layer(M, H, I, E, K, act, 5)
    want = _serve(d, K, E, act)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = ex.quantize_rows(d["x"], stream=s)
    b = ex.quantize_rows(d["x"], stream=s.cuda_stream)
    with torch.cuda.stream(s):
        y = _serve(d, K, E, act)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_two_streams_at_once():
    E, act = 8, "swiglu"
    ds = [_layer(150, 512, 256, E, 3, act, s) for s in (1, 2)]
    want = [_serve(d, 3, E, act) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_serve(ds[i], 3, E, act))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_captured_graphs_replay_with_new_inputs():
    """Two graphs of the same operators, replayed in turn, on inputs changed in place."""
    E, K, act = 8, 3, "relu2"
    ds = [_layer(90, 256, 272, E, K, act, s) for s in (3, 4)]
    graphs, outs = [], []
    for d in ds:
        d["ws"] = torch.zeros(moe.permute_workspace_size(90, K, E), dtype=torch.uint8, device="cuda")
        _serve(d, K, E, act)
    torch.cuda.synchronize()
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = _serve(d, K, E, act)
        graphs.append(g)
        outs.append(y)
    for turn in range(3):
        for i, d in enumerate(ds):
            d["x"].copy_(torch.randn(d["x"].shape, generator=d["g"], device="cuda"))
            d["logits"].copy_(torch.randn(d["logits"].shape, generator=d["g"], device="cuda"))
        for g in graphs:
            g.replay()
        for i, d in enumerate(ds):
            assert torch.equal(outs[i], _serve(d, K, E, act)), (turn, i)


def test_backward_operators_in_a_graph():
    counts = [100, 0, 33]
    off = T.offsets(counts)
    g = T.gen(8)
    dy, x = T.randn((133, 144), g, BF), T.randn((133, 272), g, BF)
    w = ex.quantize_blocks(T.randn((3, 144, 272), g))
    dw = torch.zeros((3, 144, 272), device="cuda")

    def step():
        d, xq = ex.quantize_columns(dy, off, T.E5), ex.quantize_columns(x, off)
        ex.product_weight_grad(*d, *xq, off, out=dw, accumulate=True)
        return ex.product_input_grad(*ex.quantize_rows(dy), *w, off)

    one = step().clone()
    first = dw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = step()
    dw.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, one) and torch.equal(dw, first)
    graph.replay()
    assert torch.equal(dw, first + first)


def test_rows_past_two_billion_elements():
    """More than 2^31 elements in the sorted rows, and in a product's output."""
    M, K, H = 65536, 8, 4112
    g = T.gen(2)
    x = torch.randn((M, H), generator=g, device="cuda").to(BF)
    inv = torch.randperm(M * K, generator=g, device="cuda").int()
    xs = ex.dispatch(x, inv)
    at = torch.tensor([0, 1, M * K // 2, M * K - 2, M * K - 1, 123457], device="cuda")
    src = torch.empty(M * K, dtype=torch.long, device="cuda")
    src[inv.long()] = torch.arange(M * K, device="cuda")
    assert torch.equal(xs[at], x[src[at] % M])
    y = ex.combine(xs, inv, torch.full((M, K), 0.125, device="cuda"))
    assert torch.equal(y, x)  # eight times an eighth of the same row, exact
    del xs, y
    xq, s = ex.quantize_rows(x[:, :128].contiguous().repeat(K, 1))
    w = ex.quantize_blocks(torch.randn((1, H, 128), generator=g, device="cuda"))
    out = ex.product(xq, s, *w)
    want = T.rows_value(xq[at], s[at]) @ T.weights_value(*w)[0].t()
    T.assert_within(out[at], want, want.abs() * T.HALF[BF] * 1.01 + T.sum_bound(
        T.rows_value(xq[at], s[at]).abs() @ T.weights_value(*w)[0].abs().t(), 1))


def test_binding_refusals():
    g = T.gen(1)
    x = torch.randn((8, 256), generator=g, device="cuda").to(BF)
    inv = torch.arange(16, dtype=torch.int32, device="cuda")
    w = ex.quantize_blocks(torch.randn((2, 128, 256), generator=g, device="cuda"))
    q = ex.quantize_rows(x)
    off = T.offsets([3, 5])
    bad = [
        lambda: ex.dispatch(x.half(), inv), lambda: ex.dispatch(x.t(), inv), lambda: ex.dispatch(x[0], inv),
        lambda: ex.dispatch(x, inv.long()), lambda: ex.dispatch(x, inv[:9]), lambda: ex.dispatch(x, inv.cpu()),
        lambda: ex.dispatch(x, inv, out=torch.empty((16, 256), device="cuda")),
        lambda: ex.dispatch(x[:0], inv), lambda: ex.combine(x, inv, torch.ones((8, 3), device="cuda")),
        lambda: ex.combine(x, inv, torch.ones((8, 2), device="cuda").half()),
        lambda: ex.combine_backward(x, x.float(), inv, torch.ones((8, 2), device="cuda")),
        lambda: ex.quantize_rows(x, torch.int8), lambda: ex.quantize_rows(x, out=(q[0],)),
        lambda: ex.quantize_rows(x, out=(q[0], q[1].half())), lambda: ex.quantize_columns(x, off.long()),
        lambda: ex.activation(x, "gelu"), lambda: ex.activation(x[:, :255].contiguous(), "swiglu"),
        lambda: ex.activation_backward(x, x, "swiglu"), lambda: ex.product(*q, *w),
        lambda: ex.product(*q, *w, off[:2]), lambda: ex.product(q[0], q[1][:, :1].contiguous(), *w, off),
        lambda: ex.product(q[0].view(torch.uint8), q[1], *w, off), lambda: ex.product(*q, *w, off, torch.float16),
        lambda: ex.product(*q, w[0].transpose(1, 2), w[1], off), lambda: ex.product_input_grad(*q, *w, off),
        lambda: ex.product(*q, w[0].view(torch.uint8).view(T.E5), w[1], off),
        lambda: ex.product_weight_grad(*ex.quantize_columns(x, off), *ex.quantize_columns(x, off), off, accumulate=True),
        lambda: ex.product_weight_grad(*q, *q, off),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: ex.quantize_rows(x[:, :24].contiguous()),  # the library's own limits
                 lambda: ex.dispatch(x[:, 4:12].contiguous()[:, :4].contiguous(), inv),
                 lambda: ex.dispatch(x, inv, -1)):
        with pytest.raises((moe.MoEError, RuntimeError)):
            call()
    assert torch.equal(ex.dispatch(x, inv), ex.dispatch(x, inv))  # the device is as it was


def test_empty_inputs():
    e = torch.empty((0, 256), dtype=BF, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ex.dispatch(e, none).shape == (0, 256)
    assert ex.combine(e, none, torch.empty((0, 2), device="cuda")).shape == (0, 256)
    q = ex.quantize_rows(e)
    w = ex.quantize_blocks(torch.ones((2, 128, 256), device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ex.product(*q, *w, off).shape == (0, 128)
    assert ex.product_activation(*q, *w, off, "swiglu")[0].shape == (0, 64)
    c = ex.quantize_columns(e, off)
    dw = ex.product_weight_grad(*c, *c, off)
    assert dw.shape == (2, 256, 256) and (dw == 0).all()
    x = torch.ones((4, 256), dtype=BF, device="cuda")
    drop = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    assert (ex.combine(e, drop, torch.ones((4, 2), device="cuda")) == 0).all()  # every slot dropped
    assert ex.dispatch(x, drop, 0).shape == (0, 256)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_on_another_device():
    x = torch.randn((64, 256), device="cuda:1")
    q, s = ex.quantize_rows(x)
    assert q.device == x.device and torch.cuda.current_device() == 0
    wq, ws = T.quant_rows(x, T.E4)
    assert torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s.cpu(), ws)
