"""Row-by-row float64 recurrences of the prompt operators, and their inputs, for the tests."""
import math

import torch

D = 128


def unit(gen, *shape):
    x = torch.randn(*shape, generator=gen)
    return x / x.norm(dim=-1, keepdim=True)


def linear_inputs(seed, R, Hk, H, dtype=torch.float32, g_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    q, k = unit(gen, R, Hk, D).to(dtype), unit(gen, R, Hk, D).to(dtype)
    v = torch.randn(R, H, D, generator=gen).to(dtype)
    g = -g_scale * torch.rand(R, H, generator=gen)
    return q, k, v, g


def kda_inputs(seed, R, H, dtype=torch.float32, g_scale=5.0):
    gen = torch.Generator().manual_seed(seed)
    q, k = unit(gen, R, H, D).to(dtype), unit(gen, R, H, D).to(dtype)
    v = torch.randn(R, H, D, generator=gen).to(dtype)
    g = (-g_scale * torch.rand(R, H, D, generator=gen)).to(dtype)
    beta = torch.sigmoid(torch.randn(R, H, generator=gen)).to(dtype)
    return q, k, v, g, beta


def states(seed, B, H, scale=0.3):
    gen = torch.Generator().manual_seed(seed + 1000)
    return scale * torch.randn(B, H, D, D, generator=gen)


def linear_rows(S, q, k, v, g):
    """One sequence: S [H][D][D], rows [n][..]; returns (o, S) in float64."""
    S = S.double().clone()
    H, Hk = v.shape[1], q.shape[1]
    q, k = (x.double().repeat_interleave(H // Hk, dim=1) for x in (q, k))
    v, g = v.double(), g.double()
    o = torch.zeros(v.shape, dtype=torch.float64)
    for t in range(v.shape[0]):
        S = S * torch.exp(g[t].clamp(max=0.0))[:, None, None] + k[t, :, :, None] * v[t, :, None, :]
        o[t] = (S * q[t, :, :, None]).sum(1) / math.sqrt(D)
    return o, S


def kda_rows(S, q, k, v, g, beta):
    S = S.double().clone()
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    o = torch.zeros(v.shape, dtype=torch.float64)
    for t in range(v.shape[0]):
        S = S * torch.exp(g[t].clamp(-5.0, 0.0))[:, :, None]
        e = beta[t][:, None] * (v[t] - (S * k[t, :, :, None]).sum(1))
        S = S + k[t, :, :, None] * e[:, None, :]
        o[t] = (S * q[t, :, :, None]).sum(1) / math.sqrt(D)
    return o, S


def packed(rows, S, lens, *xs):
    """`rows` over every sequence of a packed batch; S [B][H][D][D]."""
    o = torch.zeros(xs[2].shape, dtype=torch.float64)
    S = S.double().clone()
    first = 0
    for b, n in enumerate(lens):
        part = slice(first, first + n)
        if n:
            o[part], S[b] = rows(S[b], *(x[part] for x in xs))
        first += n
    return o, S


def offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


def tolerance(rows):
    """Relative 2-norm error of f32 outputs.  An output passes through at most 256 + rows roundings
    of 2^-24 that count (the 128-key sums of the update and of the output, and one decay and one add
    a row; the delta rule's step has norm at most 1, so it carries errors without growth).  They are
    independent, so their root mean square adds: 8 of them leave room for the exponentials' last
    places and for every sum's own order."""
    return 8 * math.sqrt(256 + rows) * 2.0 ** -24


def relative(x, want):
    x, want = x.detach().cpu().double(), want.double()
    assert torch.isfinite(x).all()
    norm = want.norm()
    return float((x - want).norm() / norm) if norm else float((x - want).norm())
