"""kda_attn_rows over caches that are divided among workgroups, and by kernels that divide nothing: every stretch of
keys takes part once, under the maxima of its own share (tests/split_ref.py), and whole tiles of long pages."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.cache_ref import D, attn_bound, make_cache
from tests.split_ref import bound, keys_and_values, off, result

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]


def _ends(news):
    ends = [0]
    for n in news:
        ends.append(ends[-1] + n)
    return ends


def _call(q, k, v, table, lens, offsets, scale, window=0, sinks=0):
    o = torch.full_like(q, 7.0)
    work = kda.attn_workspace(q.shape[0], len(lens), q.shape[1], k.shape[2])
    work.fill_(0xFF)
    kda.kda_attn_rows(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      torch.tensor(offsets, dtype=torch.int32, device="cuda"), o, scale=scale, window=window, sinks=sinks,
                      work=work)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("even", [True, False])
@pytest.mark.parametrize("news,lens,H,Hk,page", [
    ([1], [40000], 1, 1, 256),                    # hundreds of shares of one column, joined by four waves
    ([1], [5000], 8, 8, 16),
    ([15], [40000], 8, 1, 256),
    ([15], [20011], 16, 4, 32),
    ([1, 1, 1, 1], [20011, 5, 700, 9000], 64, 8, 64),
    ([15, 2, 9], [5000, 129, 12000], 8, 2, 64),
    ([100, 7], [3000, 5000], 4, 1, 128),
    ([1] * 40, [700 + 31 * i for i in range(40)], 8, 1, 64),   # few shares a sequence, joined by a wave
    ([1] * 60, [700 + 31 * i for i in range(60)], 8, 1, 32),   # so for f32 too
])
def test_every_share_of_the_keys_is_joined_once(dt, even, news, lens, H, Hk, page):
    gen = torch.Generator().manual_seed(sum(lens))
    k, v, table = make_cache(gen, lens, page, Hk, dt)
    k.zero_()
    v.zero_()
    offsets, rows = _ends(news), sum(news)
    factors = torch.tensor([1.0, -1.0, 0.5, -0.5])[torch.randint(0, 4, (rows, H), generator=gen)]
    q = torch.zeros(rows, H, D, dtype=dt)
    q[..., 0] = factors.to(dt)
    plain = []
    for b, length in enumerate(lens):
        scores, channel = keys_and_values(length, gen, even)
        at = torch.arange(length)
        place = table[b].cpu()[at // page].long().cuda(), (at % page).cuda()
        k[place[0], place[1], :, 0] = scores.to(dt).cuda()[:, None]
        v[place[0], place[1], :, channel.cuda()] = 1.0
        plain.append((scores, channel))
    o = _call(q.cuda(), k, v, table, lens, offsets, 1.0).double().cpu()
    for b, length in enumerate(lens):
        scores, channel = plain[b]
        for r in range(offsets[b], offsets[b + 1]):
            sees = length - (offsets[b + 1] - r) + 1
            rel = bound(sees, dt, even)
            for factor in (1.0, -1.0, 0.5, -0.5):
                heads = (factors[r] == factor).nonzero()[:, 0]
                want = result(scores[:sees], channel[:sees], factor, torch.ones(sees, dtype=torch.float64))
                assert len(heads) == 0 or not off(o[r, heads], want, rel), (b, r, factor)


def _plain(q, k, v, table, lens, offsets, scale, window, sinks):
    """o in 64 bits with the sizes that attn_bound takes, a head at a time on the GPU."""
    R, H, _ = q.shape
    page, Hk = k.shape[1], k.shape[2]
    out, size, count, dot = (torch.zeros(R, H, D, dtype=torch.float64), torch.zeros(R, H, D, dtype=torch.float64),
                             torch.zeros(R, dtype=torch.float64), torch.zeros(R, H, dtype=torch.float64))
    for b, length in enumerate(lens):
        first, last = offsets[b], offsets[b + 1]
        j = torch.arange(length, device="cuda")
        p = torch.arange(length - (last - first), length, device="cuda")[:, None]
        sees = (j <= p) & ((j > p - window) | (j < sinks) if window else torch.ones_like(j <= p))
        count[first:last] = sees.sum(1).cpu()
        at = table[b, j // page].long(), j % page
        for h in range(H):
            K, V = (x[at[0], at[1], h // (H // Hk)].double() for x in (k, v))
            Q = q[first:last, h].double()
            x = (Q @ K.T.contiguous()) * scale
            w = torch.softmax(x.masked_fill(~sees, -math.inf), 1)
            out[first:last, h] = (w @ V).cpu()
            size[first:last, h] = (w @ V.abs()).cpu()
            dot[first:last, h] = ((Q.abs() @ K.abs().T.contiguous()) * scale).masked_fill(~sees, 0.0).amax(1).cpu()
    return out, size, count, dot


# Tiles of columns that fill the chip by themselves, so that no key is split, with pages of whole tiles: bf16, f32 of
# many columns (the wide kernel) and of few (the narrow one).
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
@pytest.mark.parametrize("dt,news,lens,H,Hk,page", [
    (torch.bfloat16, [300, 1, 130], [700, 40, 130], 128, 128, 64),
    (torch.bfloat16, [500], [500], 128, 64, 128),
    (torch.bfloat16, [1100], [1100], 64, 8, 64),
    (torch.float32, [300, 1, 130], [700, 40, 130], 128, 128, 32),
    (torch.float32, [500], [500], 128, 64, 64),
    (torch.float32, [60] * 6, [60, 200, 333, 61, 128, 64], 128, 128, 64),
    (torch.float32, [15] * 20, [400 + 7 * i for i in range(20)], 192, 64, 256),
])
def test_nothing_split_over_pages_of_whole_tiles(dt, news, lens, H, Hk, page, window, sinks):
    gen = torch.Generator().manual_seed(sum(news))
    k, v, table = make_cache(gen, lens, page, Hk, dt)
    q = torch.randn(sum(news), H, D, generator=gen).to(dt).cuda()
    scale, offsets = 1.0 / math.sqrt(D), _ends(news)
    o = _call(q, k, v, table, lens, offsets, scale, window, sinks)
    want, size, count, dot = _plain(q, k, v, table, lens, offsets, scale, window, sinks)
    assert ((o.double().cpu() - want).abs() <= attn_bound(want, size, count, dot, dt)).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nothing_split_spoiled_values_reach_only_rows_that_see_them(dt, bad):
    """Whole tiles and tiles of the diagonal, without splits."""
    gen = torch.Generator().manual_seed(3)
    n, length, H = 400, 500, 128
    k, v, table = make_cache(gen, [length], 64, H, dt)
    q = torch.randn(n, H, D, generator=gen).to(dt).cuda()
    clean = _call(q, k, v, table, [length], [0, n], 0.1)
    for j in (length - 1, length - 130, length - n, 20):
        spoiled = v.clone()
        spoiled[int(table[0, j // 64]), j % 64, 5, 77] = bad
        o = _call(q, k, spoiled, table, [length], [0, n], 0.1)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[max(0, j - (length - n)):, 5, 77] = True
        assert not torch.isfinite(o[hit]).any() and torch.equal(o[~hit], clean[~hit])
