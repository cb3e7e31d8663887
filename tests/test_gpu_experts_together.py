"""Expert operators at once: first calls from many threads, and captured graphs whose branches fork and join."""
import subprocess
import sys

import pytest
import torch

from mixture_experts_layer_35_b200 import experts as ex
from tests import _experts as T

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# A process of its own, so that the threads' calls are the library's first ones.
THREADS = """
import threading, torch
from mixture_experts_layer_35_b200 import experts as ex
w = torch.randint(0, 120, (4, 128, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
ws = torch.ones((4, 1, 2), device="cuda")
x = torch.randint(0, 120, (64, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
xs = torch.ones((64, 2), device="cuda")
off = torch.tensor([0, 10, 20, 30, 64], dtype=torch.int32, device="cuda")
streams = [torch.cuda.Stream() for _ in range(16)]
torch.cuda.synchronize()
start, got = threading.Barrier(16), [None] * 16
def call(i):
    start.wait()
    try:
        got[i] = ex.product(x, xs, w, ws, off, stream=streams[i])
    except Exception as e:
        got[i] = e
ts = [threading.Thread(target=call, args=(i,)) for i in range(16)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
bad = [g for g in got if isinstance(g, Exception)]
assert not bad, bad
assert all(torch.equal(g, got[0]) for g in got)
assert ex.get_error() == 0
"""


@pytest.mark.parametrize("turn", range(3))
def test_first_calls_from_many_threads(turn):
    r = subprocess.run([sys.executable, "-c", THREADS], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_branches_that_fork_and_join_in_a_graph():
    """Both gradients of a product in branches of their own, joined by the optimiser's read; replayed on new
    inputs, with a second graph of the same operators in between."""
    counts, N, C = [70, 0, 33, 140], 144, 272
    off, P, E = T.offsets(counts), sum(counts), len(counts)
    sides = []
    for seed in (1, 2):
        g = T.gen(seed)
        d = {"dy": T.randn((P, N), g, BF), "x": T.randn((P, C), g, BF), "g": g,
             "w": ex.quantize_blocks(T.randn((E, N, C), g)), "dw": torch.zeros((E, N, C), device="cuda")}
        sides.append(d)

    def step(d, side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            c = ex.quantize_columns(d["dy"], off, T.E5)
        q = ex.quantize_columns(d["x"], off)
        dx = ex.product_input_grad(*ex.quantize_rows(d["dy"]), *d["w"], off)
        main.wait_stream(side)
        ex.product_weight_grad(*c, *q, off, out=d["dw"])
        return dx, dx.float().sum(0)

    side = torch.cuda.Stream()
    for d in sides:
        step(d, side)
    torch.cuda.synchronize()
    graphs = []
    for d in sides:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(d, side)
        graphs.append((graph, out))
    for turn in range(4):
        for d in sides:
            d["dy"].copy_(T.randn((P, N), d["g"], BF))
            d["x"].copy_(T.randn((P, C), d["g"], BF))
            d["dw"].fill_(float("nan"))
        for graph, _ in graphs:
            graph.replay()
        got = [(d["dw"].clone(), graph[1][0].clone()) for d, graph in zip(sides, graphs)]
        for d, (dw, dx) in zip(sides, got):
            want, _ = step(d, side)
            torch.cuda.synchronize()
            assert torch.equal(dw, d["dw"]) and torch.equal(dx, want), turn
    assert ex.get_error() == 0
