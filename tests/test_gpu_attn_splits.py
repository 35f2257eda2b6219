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
