"""kda_attn_rows and kda_cache_append against plain forms in 64 bits: one token, verify rows and chunks
over paged caches of every layout, windows, first tokens, pages that are missing, rows that see nothing,
and values that are not finite where no row sees them."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.cache_ref import D, attn_bound, attn_ref, make_cache

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(D)
TYPES = [torch.float32, torch.bfloat16]


def _ends(news):
    ends = [0]
    for n in news:
        ends.append(ends[-1] + n)
    return ends


def _call(q, k, v, table, lens, offsets, o, window=0, sinks=0, scale=None, work=None, stream=None):
    if work is None:
        work = kda.attn_workspace(q.shape[0], len(lens), q.shape[1], k.shape[2])
        work.fill_(0xFF)   # any state: all NaN
    kda.kda_attn_rows(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      torch.tensor(offsets, dtype=torch.int32, device="cuda"), o, scale=scale, window=window,
                      sinks=sinks, work=work, stream=stream)


def _check(q, k, v, table, lens, offsets, o, before, window=0, sinks=0, scale=SCALE):
    torch.cuda.synchronize()
    want, size, count, dot = attn_ref(q, k, v, table, lens, offsets, before, scale, window, sinks)
    got = o.double().cpu()
    err = (got - want).abs()
    bound = attn_bound(want, size, count, dot, o.dtype)
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()), float(bound[bad].min()), bad.nonzero()[:4].tolist())


def _run(dt, news, lens, H, Hk, page, window=0, sinks=0, layout="rows", extra=0, seed=1, edit=None, scale=None):
    gen = torch.Generator().manual_seed(seed)
    offsets = _ends(news)
    R = offsets[-1] + extra
    k, v, table = make_cache(gen, lens, page, Hk, dt, layout)
    rows = torch.randn(R, H + 2 * Hk, D, generator=gen).to(dt).cuda()
    q = rows[:, :H]
    if edit:
        edit(q, k, v, table)
    o = torch.full((R, H, D), 7.0, dtype=dt, device="cuda")
    before = o.clone()
    _call(q, k, v, table, lens, offsets, o, window, sinks, scale)
    _check(q, k, v, table, lens, offsets, o, before, window, sinks, SCALE if scale is None else scale)
    return o


CASES = [
    # news, lens, H, Hk, page
    ([1], [1], 1, 1, 16),
    ([1], [2], 8, 1, 16),
    ([1], [31], 4, 4, 1),
    ([1], [300], 8, 1, 16),
    ([1], [1500], 3, 1, 64),
    ([1, 1, 1], [700, 1, 33], 16, 2, 32),
    ([15], [900], 8, 1, 64),
    ([15], [15], 8, 2, 16),
    ([15, 0, 3, 8], [260, 5, 3, 777], 6, 2, 32),
    ([70], [70], 4, 1, 16),
    ([130, 1, 33], [400, 65, 33], 6, 2, 128),
    ([257], [257], 5, 5, 256),
    ([2], [200], 40, 1, 64),       # more query heads to a key head than a wave has columns
    ([9], [100], 130, 1, 64),      # and than four waves have
    ([100], [1300], 8, 1, 64),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_attn_rows(dt, case):
    _run(dt, *case)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (64, 64), (100, 3), (333, 70), (5000, 9), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("case", [([1, 1], [900, 40], 8, 1, 16), ([15, 4], [700, 65], 4, 2, 32), ([90], [500], 4, 1, 64)])
def test_attn_window(dt, window, sinks, case):
    _run(dt, *case, window=window, sinks=sinks)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["heads", "pages", "mixed"])
def test_attn_layouts(dt, layout):
    _run(dt, [4, 60], [300, 99], 6, 3, 32, layout=layout)
    _run(dt, [1, 1], [300, 99], 6, 3, 16, layout=layout)


@pytest.mark.parametrize("dt", TYPES)
def test_attn_rows_without_keys_and_rows_left_out(dt):
    # five rows but two positions: three rows lie below zero and give 0; rows behind the last stay
    o = _run(dt, [5, 2], [2, 40], 4, 2, 16, extra=3)
    assert (o[:3] == 0).all() and (o[7:] == 7).all()
    o = _run(dt, [3, 40], [0, 20], 4, 2, 16)
    assert (o[:3] == 0).all()
    assert (_run(dt, [2], [-9], 4, 2, 16) == 0).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("news", [[1, 1], [15, 15], [80, 3]])
def test_attn_missing_pages(dt, news):
    def edit(q, k, v, table):
        table[0, 2] = -1
        table[0, 5] = k.shape[0]            # one past the last page
        table[0, 7:9] = 2**31 - 1
        table[1, :] = -1                    # nothing at all
        table[1, -1] = -(2**31)
    o = _run(dt, news, [400, 90], 4, 2, 16, edit=edit)
    assert (o[news[0]:] == 0).all()
    _run(dt, news, [400, 90], 4, 2, 16, edit=edit, window=50, sinks=40)


@pytest.mark.parametrize("dt", TYPES)
def test_attn_lengths_behind_the_table(dt):
    gen = torch.Generator().manual_seed(3)
    k, v, table = make_cache(gen, [100], 16, 2, dt)   # 7 pages and one more entry: 128 places
    table[0, 7] = 1
    q = torch.randn(3, 4, D, generator=gen).to(dt).cuda()
    for length in (126, 129, 140, 2**31 - 1):
        for window in (0, 20):
            o = torch.full((3, 4, D), 7.0, dtype=dt, device="cuda")
            _call(q, k, v, table, [length], [0, 3], o, window)
            if length < 2**20:
                _check(q, k, v, table, [length], [0, 3], o, o, window)
            elif window:
                assert (o == 0).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("news,lens,window,sinks", [([1], [333], 0, 0), ([1], [333], 40, 5), ([15], [333], 0, 0),
                                                    ([15], [333], 40, 5), ([120], [333], 0, 0), ([120], [333], 40, 5)])
def test_attn_what_no_row_sees_has_no_effect(dt, bad, news, lens, window, sinks):
    n, length = news[0], lens[0]

    def edit(q, k, v, table):
        place = {int(e): i for i, e in enumerate(table[0].tolist()) if e >= 0}
        for page in range(k.shape[0]):
            for r in range(16):
                j = place.get(page, 10**6) * 16 + r
                low = length - n - window + 1 if window else 0
                if j >= length or sinks <= j < low:
                    k[page, r] = bad
                    v[page, r] = bad
    _run(dt, news, lens, 4, 2, 16, window, sinks, edit=edit)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n,length,window,sinks", [(15, 200, 0, 0), (100, 170, 0, 0), (15, 200, 30, 4), (100, 170, 30, 4)])
def test_attn_spoiled_rows_reach_only_those_that_see_them(dt, bad, n, length, window, sinks):
    gen = torch.Generator().manual_seed(9)
    k, v, table = make_cache(gen, [length], 16, 2, dt)
    q = torch.randn(n, 4, D, generator=gen).to(dt).cuda()
    clean = torch.empty(n, 4, D, dtype=dt, device="cuda")
    _call(q, k, v, table, [length], [0, n], clean, window, sinks)
    at = lambda j: (int(table[0, j // 16]), j % 16)  # noqa: E731
    for j in (length - 1, length - n // 2, length - n, length - n - 20, 2):
        spoiled = v.clone()
        spoiled[at(j)[0], at(j)[1], 1, 77] = bad
        o = torch.empty_like(clean)
        _call(q, k, spoiled, table, [length], [0, n], o, window, sinks)
        p = torch.arange(length - n, length, device="cuda")
        sees = (j <= p) & ((j > p - window) | (j < sinks) if window else torch.ones_like(p, dtype=torch.bool))
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[sees, 2:, 77] = True
        assert not torch.isfinite(o[hit]).any()
        assert torch.equal(o[~hit], clean[~hit])
        keys = k.clone()
        keys[at(j)[0], at(j)[1], 0, 5] = math.nan
        _call(q, keys, v, table, [length], [0, n], o, window, sinks)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[sees, :2] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n", [1, 15, 90])
def test_attn_a_query_that_is_not_finite_spoils_its_row_and_head_alone(dt, n):
    gen = torch.Generator().manual_seed(n)
    k, v, table = make_cache(gen, [300], 16, 2, dt)
    q = torch.randn(n, 4, D, generator=gen).to(dt).cuda()
    clean, o = (torch.empty(n, 4, D, dtype=dt, device="cuda") for _ in range(2))
    _call(q, k, v, table, [300], [0, n], clean)
    for bad in (math.nan, math.inf):
        x = q.clone()
        x[n // 2, 2, 9] = bad
        _call(x, k, v, table, [300], [0, n], o)
        hit = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
        hit[n // 2, 2] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


def test_binding_refuses_what_it_sees_of_device_tensors():
    gen = torch.Generator().manual_seed(1)
    k, v, table = make_cache(gen, [20, 30], 16, 2, torch.float32)
    lens = torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    q, o, new = (torch.zeros(5, h, D, device="cuda") for h in (4, 4, 2))
    work = kda.attn_workspace(5, 2, 4, 2)

    def attn(q=q, k=k, v=v, table=table, lens=lens, offsets=offsets, o=o, **kw):
        kda.kda_attn_rows(q, k, v, table, lens, offsets, o, work=work, **kw)

    def append(new_k=new, new_v=new, k=k, v=v, table=table, lens=lens, offsets=offsets):
        kda.kda_cache_append(new_k, new_v, k, v, table, lens, offsets)

    attn()
    append()
    for call in (attn, append):
        for kw in (dict(k=k[0]), dict(k=k[:2]), dict(v=v.transpose(1, 2).contiguous().transpose(1, 2)), dict(k=k[..., :64]),
                   dict(k=k.repeat_interleave(2, 3)[..., ::2], v=v.repeat_interleave(2, 3)[..., ::2]), dict(k=k.cpu()),
                   dict(table=table[0]), dict(table=table[:, ::2]), dict(table=table.cpu()), dict(lens=lens[:1]),
                   dict(offsets=offsets[:2])):
            with pytest.raises((ValueError, kda.KdaError)):
                call(**kw)
        for kw in (dict(k=k.bfloat16(), v=v.bfloat16()), dict(table=table.long()), dict(lens=lens.long()), dict(offsets=offsets.long())):
            with pytest.raises(TypeError):
                call(**kw)
    with pytest.raises(TypeError):
        attn(q=q.half(), o=o.half(), k=k.half(), v=v.half())
    for kw in (dict(o=o[:4]), dict(q=q[:, :, ::2]), dict(q=q[:, :3], o=o[:, :3].contiguous()), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(o=torch.zeros(5, 8, D, device="cuda")[:, ::2]), dict(window=-1), dict(sinks=1), dict(scale=0.0), dict(window=2**31)):
        with pytest.raises((ValueError, kda.KdaError)):
            attn(**kw)
    for kw in (dict(new_v=new[:4]), dict(new_k=torch.zeros(5, 2, 2 * D, device="cuda")[..., ::2]), dict(new_k=k.view(-1, 2, D)[:5])):
        with pytest.raises((ValueError, kda.KdaError)):
            append(**kw)


@pytest.mark.parametrize("dt", TYPES)
def test_attn_scores_of_any_size(dt):
    # weights that underflow but for one key, a score of -inf, scores that only the maximum keeps finite
    gen = torch.Generator().manual_seed(4)
    k, v, table = make_cache(gen, [200], 16, 1, dt)
    for news in (1, 40):
        q = (torch.randn(news, 2, D, generator=gen) * 1e4).to(dt).cuda()
        o = torch.empty(news, 2, D, dtype=dt, device="cuda")
        _call(q, k, v, table, [200], [0, news], o)
        torch.cuda.synchronize()
        want, *_ = attn_ref(q, k, v, table, [200], [0, news], o, SCALE)
        # the scores are some 1e4 apart: nearly every weight is 0 or 1, whatever their roundings
        assert torch.isfinite(o).all()
        assert ((o.double().cpu() - want).abs() < 0.02 * (want.abs() + 1)).double().mean() > 0.99
        q = torch.zeros(news, 2, D, dtype=dt, device="cuda")
        q[..., 0] = 3e38
        keys = k.clone()
        keys[..., 0] = 1.0
        dead = torch.arange(0, 200, 3).tolist()
        for j in dead:
            keys[int(table[0, j // 16]), j % 16, 0, 0] = -3e38      # -inf after the product
        _call(q, keys, v, table, [200], [0, news], o, scale=1e-38)
        torch.cuda.synchronize()
        for r in range(news):
            p = 200 - news + r
            alive = [j for j in range(p + 1) if j % 3]
            V = torch.stack([v[int(table[0, j // 16]), j % 16, 0] for j in alive]).double().cpu()
            x = torch.stack([keys[int(table[0, j // 16]), j % 16, 0, 0] for j in alive]).double().cpu()
            w = torch.softmax(float(q[r, 0, 0]) * x * 1e-38, 0)
            err = (o[r].double().cpu() - w @ V).abs().max()
            assert err <= (2.0**-6 if dt == torch.bfloat16 else 1e-4)


def test_attn_scale_and_offsets_table():
    _run(torch.float32, [3, 40], [77, 90], 4, 2, 16, scale=0.5)
    gen = torch.Generator().manual_seed(6)
    lens = [50, 60, 70, 30]
    k, v, table = make_cache(gen, lens, 16, 2, torch.float32)
    for offsets in ([2, 5, 5, 9, 12], [0, 10, 5, 7, 12], [-3, 4, 99, 99, 99], [9, 3, 1, 12, 2], [12, 12, 12, 12, 12]):
        q = torch.randn(12, 4, D, generator=gen).cuda()
        o = torch.full((12, 4, D), 7.0, device="cuda")
        before = o.clone()
        _call(q, k, v, table, lens, offsets, o)
        _check(q, k, v, table, lens, offsets, o, before)


@pytest.mark.parametrize("B", [65, 200, 700])
def test_attn_many_sequences(B):
    gen = torch.Generator().manual_seed(B)
    news = [int(x) for x in torch.randint(0, 3, (B,), generator=gen)]
    news[3] = 40
    lens = [n + int(x) for n, x in zip(news, torch.randint(0, 90, (B,), generator=gen))]
    _run(torch.bfloat16, news, lens, 4, 1, 16)
    _run(torch.float32, news, lens, 2, 2, 16, window=20, sinks=2)


@pytest.mark.parametrize("dt", TYPES)
def test_attn_long_cache_split_many_times(dt):
    # one head, one row: hundreds of splits are joined
    gen = torch.Generator().manual_seed(8)
    for n, H in ((1, 1), (15, 8)):
        length = 40000
        k, v, table = make_cache(gen, [length], 256, 1, dt)
        q = torch.randn(n, H, D, generator=gen).to(dt).cuda()
        o = torch.empty(n, H, D, dtype=dt, device="cuda")
        _call(q, k, v, table, [length], [0, n], o)
        _check(q[-1:], k, v, table, [length], [0, 1], o[-1:], o[-1:])
        # and the first row, which sees n - 1 keys fewer
        _check(q[:1], k, v, table, [length - n + 1], [0, 1], o[:1], o[:1])


def test_attn_a_cache_of_more_than_4_gib():
    # rows on both sides of 2^31 elements and 2^32 bytes
    page, Hk = 4096, 64
    pages = 2**32 // (page * Hk * D) + 3
    k = torch.zeros(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator().manual_seed(5)
    want = [0, pages // 2, pages - 1]
    for i in want:
        k[i, :20] = torch.randn(20, Hk, D, generator=gen).cuda()
        v[i, :20] = torch.randn(20, Hk, D, generator=gen).cuda()
    table = torch.tensor([[i] for i in want], dtype=torch.int32, device="cuda")
    q = torch.randn(3, Hk, D, generator=gen).to(torch.bfloat16).cuda()
    o = torch.empty(3, Hk, D, dtype=torch.bfloat16, device="cuda")
    _call(q, k, v, table, [20, 11, 17], [0, 1, 2, 3], o)
    small = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    sk, sv = (torch.stack([x[i, :32] for i in want]) for x in (k, v))
    _check(q, sk, sv, small, [20, 11, 17], [0, 1, 2, 3], o, o)
    new = torch.randn(1, Hk, D, generator=gen).to(torch.bfloat16).cuda()
    kda.kda_cache_append(new, new, k, v, table[2:], torch.tensor([31], dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[pages - 1, 30], new[0]) and torch.equal(v[pages - 1, 30], new[0])


@pytest.mark.parametrize("news,lens,H,Hk", [([1, 1], [700, 90], 8, 1), ([15], [900], 8, 1), ([300], [300], 4, 4)])
def test_attn_same_bits_every_time_on_any_stream_and_in_a_graph(news, lens, H, Hk):
    gen = torch.Generator().manual_seed(2)
    k, v, table = make_cache(gen, lens, 32, Hk, torch.bfloat16)
    R = sum(news)
    q = torch.randn(R, H, D, generator=gen).to(torch.bfloat16).cuda()
    args = (k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.tensor(_ends(news), dtype=torch.int32, device="cuda"))
    work = kda.attn_workspace(R, len(news), H, Hk)
    first = torch.empty(R, H, D, dtype=torch.bfloat16, device="cuda")
    kda.kda_attn_rows(q, *args, first, work=work)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = torch.zeros_like(first)
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_attn_rows(q, *args, o, work=work, stream=side)
    side.synchronize()
    assert torch.equal(o, first)
    graph = torch.cuda.CUDAGraph()
    o.zero_()
    with torch.cuda.graph(graph):
        kda.kda_attn_rows(q, *args, o, work=work)
    for i in range(4):
        o.zero_()
        work.fill_(0xFF if i & 1 else 0)
        q.neg_() if i else None
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(first)
        kda.kda_attn_rows(q, *args, want, work=kda.attn_workspace(R, len(news), H, Hk))
        assert torch.equal(o, want)
    # lengths that shrink on the device (a rollback) between replays
    args[3].sub_(3)
    graph.replay()
    want = torch.empty_like(first)
    kda.kda_attn_rows(q, *args, want, work=kda.attn_workspace(R, len(news), H, Hk))
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def _append_ref(k, pages, table, lens, offsets):
    want = pages.clone()
    page, R, upto = pages.shape[1], k.shape[0], 0
    for b in range(len(lens)):
        first = max(upto, min(max(offsets[b], 0), R))
        last = min(max(offsets[b + 1], first), R)
        upto = first
        for r in range(first, last):
            p = max(lens[b], 0) - (last - r)
            if 0 <= p < table.shape[1] * page and 0 <= int(table[b, p // page]) < pages.shape[0]:
                want[int(table[b, p // page]), p % page] = k[r]
    return want


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["rows", "heads", "pages", "mixed"])
@pytest.mark.parametrize("news,lens,Hk,page", [([1], [1], 1, 16), ([15], [40], 1, 16), ([3, 0, 90, 1], [5, 9, 333, 64], 5, 32),
                                               ([300], [290], 2, 1), ([7, 7], [-5, 20], 70, 8)])
def test_append(dt, layout, news, lens, Hk, page):
    gen = torch.Generator().manual_seed(7)
    k_pages, v_pages, table = make_cache(gen, [max(n, 0) for n in lens], page, Hk, dt, layout)
    if len(news) == 4:
        table[2, 9], table[2, 10] = -1, k_pages.shape[0]
    offsets = _ends(news)
    rows = torch.randn(offsets[-1] + 2, 2 * Hk + 3, D, generator=gen).to(dt).cuda()
    k, v = rows[:, :Hk], rows[:, Hk + 3:]
    want = [_append_ref(x, y, table, lens, offsets) for x, y in ((k, k_pages), (v, v_pages))]
    kda.kda_cache_append(k, v, k_pages, v_pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(k_pages, want[0]) and torch.equal(v_pages, want[1])


def test_append_moves_bits_and_reads_any_offsets_table():
    gen = torch.Generator().manual_seed(11)
    lens = [50, 60, 70, 30]
    for offsets in ([2, 5, 5, 9, 12], [0, 10, 5, 7, 12], [-3, 4, 99, 99, 99], [9, 3, 1, 12, 2]):
        k_pages, v_pages, table = make_cache(gen, lens, 16, 2, torch.float32)
        k = torch.randn(12, 2, D, generator=gen).cuda()
        k.view(torch.int32)[3, 1, :4] = torch.tensor([0x7FC00001, -1, 0x7F800000, 1], dtype=torch.int32, device="cuda")
        want = [_append_ref(k, y, table, lens, offsets) for y in (k_pages, v_pages)]
        kda.kda_cache_append(k, k, k_pages, v_pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        for got, x in ((k_pages, want[0]), (v_pages, want[1])):
            assert torch.equal(got.view(torch.int32), x.view(torch.int32))


def test_attn_and_append_without_rows():
    gen = torch.Generator().manual_seed(1)
    k, v, table = make_cache(gen, [20], 16, 2, torch.float32)
    none = torch.empty(0, 2, D, device="cuda")
    lens, offsets = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    before = k.clone()
    kda.kda_cache_append(none, none, k, v, table, lens, offsets)
    kda.kda_attn_rows(none, k, v, table, lens, offsets, none, work=kda.attn_workspace(0, 1, 2, 2))
    torch.cuda.synchronize()
    assert torch.equal(k, before)


def test_append_refuses_more_rows_than_a_c_int_counts():
    # 2^32 rows of one row in memory: as a C int they would be none at all
    gen = torch.Generator().manual_seed(1)
    k, v, table = make_cache(gen, [20], 16, 2, torch.float32)
    rows = torch.zeros(1, 2, D, device="cuda").expand(2**32, 2, D)
    lens, offsets = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(kda.KdaError):
        kda.kda_cache_append(rows, rows, k, v, table, lens, offsets)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n", [1, 15, 120])
def test_attn_a_score_of_minus_infinity_has_no_weight_but_its_value_is_seen(dt, bad, n):
    gen = torch.Generator().manual_seed(n)
    length, dead = 333, [3, 200, 332]
    k, v, table = make_cache(gen, [length], 16, 1, dt)
    q = torch.randn(n, 2, D, generator=gen).to(dt).cuda()
    q[..., 0] = 1.0
    for j in dead:
        k[int(table[0, j // 16]), j % 16, 0, 0] = -math.inf
    k_finite = torch.where(torch.isinf(k), 0.0, k)
    o, spoiled = (torch.empty(n, 2, D, dtype=dt, device="cuda") for _ in range(2))
    _call(q, k, v, table, [length], [0, n], o)
    torch.cuda.synchronize()
    p = torch.arange(length - n, length)
    # the same as if the keys' pages were not there: a cache of pages of one row, these keys' entries -1
    rows_k, rows_v = (x.reshape(-1, 1, 1, D) for x in (k_finite, v))
    rows = torch.full((1, length), -1, dtype=torch.int32)
    for j in range(length):
        if j not in dead:
            rows[0, j] = int(table[0, j // 16]) * 16 + j % 16
    _check(q, rows_k, rows_v, rows.cuda(), [length], [0, n], o, o)
    for j in dead:
        w = v.clone()
        w[int(table[0, j // 16]), j % 16, 0, 77] = bad
        _call(q, k, w, table, [length], [0, n], spoiled)
        hit = torch.zeros(n, 2, D, dtype=torch.bool)
        hit[p >= j, :, 77] = True
        assert not torch.isfinite(spoiled[hit.cuda()]).any() and torch.equal(spoiled[~hit.cuda()], o[~hit.cuda()])
