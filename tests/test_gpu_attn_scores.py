"""kda_attn_rows with finite scores of any size: where the scores of a row are so large that f32 holds them
in steps of a power of two and more, the largest still takes the whole weight, equal ones share it, and the
other rows and heads keep their bits."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.cache_ref import D, make_cache

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
SCALE = 1.0 / math.sqrt(D)


def _call(q, k, v, table, length, window=0, sinks=0):
    n, H, _ = q.shape
    o = torch.full_like(q, 7.0)
    work = kda.attn_workspace(n, 1, H, k.shape[2])
    work.fill_(0xFF)
    kda.kda_attn_rows(q, k, v, table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, n], dtype=torch.int32, device="cuda"), o, window=window, sinks=sinks, work=work)
    torch.cuda.synchronize()
    return o


def _by_position(pages, table, length):
    at = torch.arange(length)
    return pages.cpu()[table.cpu()[0, at // pages.shape[1]].long(), at % pages.shape[1]]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n,H,length,page", [(1, 2, 300, 64), (1, 2, 100, 16), (15, 8, 5000, 64), (15, 40, 333, 16),
                                             (200, 2, 700, 64), (60, 3, 129, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_scores_of_any_finite_size(dt, n, H, length, page, window, sinks):
    gen = torch.Generator().manual_seed(n + length)
    k, v, table = make_cache(gen, [length], page, 1, dt)
    # one channel makes the scores: a power of two a row and head, up to 2^113 either way, times a key's 1 .. 2 in
    # steps of 2^-7 (exact in f32, for either type), so that two scores are equal or 2^-8 of themselves apart
    k.zero_()
    k[..., 0] = 1 + torch.randint(0, 128, k.shape[:3], generator=gen).to(dt).cuda() / 128
    sizes = torch.tensor([20, 30, 36, 45, 70, 113])[torch.randint(0, 6, (n, H), generator=gen)].double()
    signs = torch.randint(0, 2, (n, H), generator=gen).double() * 2 - 1
    q = torch.zeros(n, H, D, dtype=dt)
    q[..., 0] = (signs * 2.0**sizes).to(dt)
    o = _call(q.cuda(), k, v, table, length, window, sinks).double().cpu()
    K, V = _by_position(k, table, length).double()[:, 0, 0], _by_position(v, table, length).double()[:, 0]
    for r in range(n):
        p = length - n + r
        j = torch.arange(p + 1)
        if window:
            j = j[(j > p - window) | (j < sinks)]
        for h in range(H):
            x = K[j] * float(q[r, h, 0]) * SCALE
            # the nearest other score is 2^20 / 128 / 11.4 = 724 below the largest at least: all others weigh
            # less than 2^-1000, and the largest ones the same
            top = j[x == x.max()]
            want = V[top].mean(0)
            # sums of as many values as share it, their quotient, and the rounding to the result's type.  Below 2^24 the
            # same weight of the largest is a power of 2 near 0 (c s - m in one operation), 1 within half a step of m: it
            # is not 1 then, and bf16 rounds it by 2^-8 of itself
            size = V[top].abs().mean(0)
            bound = (len(top) + 4) * 2.0**-24 * size
            if dt == torch.bfloat16:
                bound = bound + (2.0**-8 * size if sizes[r, h] < 24 else 0.0)
                bound = bound + 2.0**-8 * (want.abs() + bound)
            assert ((o[r, h] - want).abs() <= bound).all(), (r, h, float(sizes[r, h]), float(signs[r, h]), len(top))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n,H,length", [(1, 8, 300), (15, 8, 2000), (200, 4, 500)])
def test_a_head_of_large_scores_leaves_the_others_their_bits(dt, n, H, length):
    gen = torch.Generator().manual_seed(n)
    k, v, table = make_cache(gen, [length], 64, 1, dt)
    q = torch.randn(n, H, D, generator=gen).to(dt).cuda()
    clean = _call(q, k, v, table, length)
    for size in (1e12, 1e30):
        x = q.clone()
        x[n // 2, 1] *= size
        o = _call(x, k, v, table, length)
        assert torch.isfinite(o).all() and not torch.equal(o[n // 2, 1], clean[n // 2, 1])
        o[n // 2, 1] = clean[n // 2, 1]
        assert torch.equal(o, clean)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("length", [100, 400, 6000])
def test_scores_that_grow_and_shrink_along_the_keys(dt, length):
    """The maximum passes from small to large, from large negative to small, and stays, tile by tile."""
    gen = torch.Generator().manual_seed(length)
    k, v, table = make_cache(gen, [length], 64, 1, dt)
    V = _by_position(v, table, length)[:, 0]
    q = torch.zeros(1, 2, D, dtype=dt)
    q[0, :, 0] = 1.0
    rising = torch.linspace(0, 100, length).exp2()
    for keys, win in ((rising, length - 1), (rising.flip(0), 0), (-rising, 0), (-rising.flip(0), length - 1),
                      (torch.where(torch.arange(length) == length // 2, 500.0, -1e30), length // 2),
                      (torch.where(torch.arange(length) == 1, -1e20, -1e30), 1)):
        keys = keys.to(dt)
        at = torch.arange(length)
        k.zero_()
        k[table[0].cpu()[at // 64].long().cuda(), (at % 64).cuda(), 0, 0] = keys.cuda()
        o = _call(q.cuda(), k, v, table, length).cpu()
        x = keys.double() * SCALE
        w = torch.softmax(x, 0)
        assert int(w.argmax()) == win
        want = (w[:, None] * V.double()).sum(0)
        size = (w[:, None] * V.double().abs()).sum(0)
        # where two scores are near the largest these are below 40: 3 half steps of 40 in base 2 each, twice, and the sums
        near = x[w > 1e-12].abs().max() if float(w.max()) < 0.999999 else 0.0
        bound = (2 * 3 * 1.5 * float(near) + 2 * (length + 64) + 8) * 2.0**-24 * size + 1e-11
        if dt == torch.bfloat16:
            bound = bound + 2.0**-8 * size + 2.0**-8 * (want.abs() + 2.0**-8 * size)
        assert ((o[0].double() - want).abs() <= bound).all()
