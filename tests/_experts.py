"""Plain 64-bit forms of the expert operators for their tests, and the inputs' helpers."""
import numpy as np
import torch

from mixture_experts_layer_35_b200 import experts as ex

B = ex.BLOCK
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
FMAX = {E4: 448.0, E5: 57344.0}
# Half a step, relative to the value: finfo.eps / 2.  BF16 stores 7 bits of the significand, so its steps at 1
# are 2^-7 and half of one is 2^-8 (FP32: 23 bits, 2^-24; e4m3: 3 bits, 2^-4; e5m2: 2 bits, 2^-3).
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32, E4, E5)}
TINY = {E4: 2.0 ** -10, E5: 2.0 ** -17}  # half the smallest step of the 8-bit types


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=torch.float32, scale=1.0):
    """Normal values, rows of different sizes."""
    t = torch.randn(shape, generator=g, device="cuda")
    if len(shape) == 2 and shape[0]:
        t = t * torch.exp(torch.randn((shape[0], 1), generator=g, device="cuda"))
    return (t * scale).to(dtype)


def slots(M, K, P, g):
    """inv [K * M]: P of the slots get distinct rows, the others are dropped (negative, or past the end)."""
    at = torch.randperm(M * K, generator=g, device="cuda")
    inv = torch.where(torch.rand(M * K, generator=g, device="cuda") < 0.5, -1 - at, P + at).int()
    inv[at[:P]] = torch.randperm(P, generator=g, device="cuda").int()
    return inv


def offsets(counts):
    off = np.zeros(len(counts) + 1, np.int32)
    off[1:] = np.cumsum(counts)
    return torch.from_numpy(off).cuda()


def scale_factor(amax, dtype):
    """FP32 scale and factor of blocks whose largest magnitudes are ``amax`` (on the CPU)."""
    a = amax.clamp(min=2.0 ** -96)
    top = torch.full_like(a, FMAX[dtype])
    return a / top, top / a


def quant_rows(x, dtype):
    x = x.cpu().float()
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % B)).view(R, -1, B)
    s, f = scale_factor(b.abs().amax(2), dtype)
    return (b * f[:, :, None]).reshape(R, -1)[:, :C].to(dtype), s


def quant_blocks(w, dtype):
    w = w.cpu().float()
    E, N, C = w.shape
    p = torch.nn.functional.pad(w, (0, -C % B, 0, -N % B)).view(E, -(-N // B), B, -(-C // B), B)
    s, f = scale_factor(p.abs().amax((2, 4)), dtype)
    q = (p * f[:, :, None, :, None]).view(E, -(-N // B) * B, -(-C // B) * B)[:, :N, :C]
    return q.to(dtype), s


def quant_columns(x, counts, dtype):
    """The blocks that are written, in order."""
    x, qs, ss, r = x.cpu().float(), [], [], 0
    for n in counts:
        for i in range(0, n, B):
            t = torch.zeros((B, x.shape[1]))
            t[:min(B, n - i)] = x[r + i:r + min(n, i + B)]
            s, f = scale_factor(t.abs().amax(0), dtype)
            qs.append((t * f).to(dtype))
            ss.append(s)
        r += n
    return torch.cat(qs), torch.stack(ss)


def rows_value(q, s):
    return q.double() * s.double().repeat_interleave(B, 1)[:, :q.shape[1]]


def weights_value(q, s):
    s = s.double().repeat_interleave(B, 1)[:, :q.shape[1]]
    return q.double() * s.repeat_interleave(B, 2)[:, :, :q.shape[2]]


def grouped(x, w, counts, transposed):
    """Each row times its expert's matrix, in 64 bits: x w^T (transposed) or x w."""
    out, r = [], 0
    for e, n in enumerate(counts):
        out.append(x[r:r + n] @ (w[e].t() if transposed else w[e]))
        r += n
    return torch.cat(out)


def act(y, name):
    if name == "relu2":
        return torch.where(y > 0, y * y, torch.zeros_like(y))
    g, u = y.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def sum_bound(abs_sum, blocks):
    """Error of a product's FP32 sum: a block of 128 takes four tensor-core steps, each
    aligning 33 addends (32 products and the sum so far) to the largest and keeping at least 24
    bits of it, so each is off by at most 2^-23 of the sum of magnitudes; the scale's
    product, one fused multiply-add a block."""
    return abs_sum * (4 * 33 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24)


def assert_within(got, want, tol, what=""):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = int(torch.argmax(bad.reshape(-1).int()))
        t = torch.as_tensor(tol, device=got.device, dtype=torch.float64).expand_as(got).reshape(-1)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                             f"{got.reshape(-1)[i].item()!r} for {want.reshape(-1)[i].item()!r}, tolerance {t[i].item():.3g}")
