"""kda_accept_sampled against a plain form in 64 bits: the accepted counts, the drawn tokens and the
drafts' probabilities, over ragged sessions, masked and odd vocabularies, temperatures, drafts with and
without probabilities, and rows that have no distribution."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.cache_ref import accept_ref

pytestmark = pytest.mark.gpu

NO_TOKEN = 0xFFFFFFFF


def _inputs(rows, V, dt, seed, masked=False, drafted=True, pad=0, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    offsets = [0]
    for n in rows:
        offsets.append(offsets[-1] + n)
    R = offsets[-1] + 2
    x = torch.randn(R, V + pad, generator=gen) * spread
    if masked:
        kept = torch.rand(R, V + pad, generator=gen) < 0.2
        kept[:, 7 % V] = True
        x.masked_fill_(~kept, -math.inf)
    x = x.to(dt).cuda()
    probs = torch.softmax(x[:, :V].float() + 0.7 * torch.randn(R, V, generator=gen).cuda(), 1)
    drafts = torch.multinomial(probs.cpu(), 1, generator=gen)[:, 0].to(torch.int32).cuda()
    u = torch.rand(R, generator=gen).cuda()
    return x[:, :V], offsets, drafts, u, probs if drafted else None


def _call(x, offsets, drafts, u, probs=None, temp=None, want_p=True, work=None):
    R, V = x.shape
    B = len(offsets) - 1
    out = torch.full((B, 2), -5, dtype=torch.int32, device="cuda")
    p = torch.full((R,), 9.0, device="cuda") if want_p else None
    if work is None:
        work = kda.accept_sampled_workspace(R, B, V)
        work.fill_(0xFF)
    kda.kda_accept_sampled(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), drafts, u, out,
                           probs=probs, temp=temp, p_draft=p, work=work)
    torch.cuda.synchronize()
    return out, p


def _check(x, offsets, drafts, u, probs=None, temp=None):
    out, p = _call(x, offsets, drafts, u, probs, temp)
    want, p_want, margin = accept_ref(x, offsets, drafts, u, probs, temp)
    for b, w in enumerate(want):
        got = tuple(int(y) & NO_TOKEN for y in out[b])
        if w is None:
            assert got == (-5 & NO_TOKEN,) * 2
        else:
            assert got == w, (b, got, w, margin[b])   # (the distance to the nearest border)
    for r in range(x.shape[0]):
        if r not in p_want:
            assert float(p[r]) == 9.0
        elif math.isnan(p_want[r]):
            assert math.isnan(float(p[r]))
        else:
            # the sum's exponentials are good to 2 half steps of their own (2^-24) and of an argument
            # of at most 150 in base 2; the rest is f64, rounded once
            assert abs(float(p[r]) - p_want[r]) <= 160 * 2.0**-24 * p_want[r] + 1e-38
    return out


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 5001, 33333])
@pytest.mark.parametrize("drafted", [True, False])
def test_sampled(dt, V, drafted):
    x, offsets, drafts, u, probs = _inputs([1, 15, 0, 3, 8, 2], V, dt, V, drafted=drafted)
    _check(x, offsets, drafts, u, probs)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", [False, True])
def test_sampled_strides_masks_and_temperatures(dt, masked):
    x, offsets, drafts, u, probs = _inputs([4, 15, 1, 9], 4099, dt, 5, masked=masked, pad=6)
    wide = torch.zeros(probs.shape[0], 4110, device="cuda")
    wide[:, 3:3 + 4099] = probs
    temp = torch.tensor([0.3, 1.0, 2.5, 0.9], device="cuda")
    _check(x, offsets, drafts, u, wide[:, 3:3 + 4099], temp)
    _check(x, offsets, drafts, u, None, temp)


def test_sampled_one_session_of_many_rows_and_many_sessions():
    x, offsets, drafts, u, probs = _inputs([70], 300, torch.float32, 1)
    u[:60] *= 0.05
    _check(x, offsets, drafts, u, probs)
    x, offsets, drafts, u, probs = _inputs([1 + i % 4 for i in range(150)], 200, torch.bfloat16, 2)
    _check(x, offsets, drafts, u, probs)


def test_sampled_offsets_table():
    x, _, drafts, u, probs = _inputs([10], 500, torch.float32, 3)
    for offsets in ([2, 5, 5, 9, 12], [0, 10, 5, 7, 12], [-3, 4, 99, 99, 99], [9, 3, 1, 12, 2]):
        _check(x, offsets, drafts, u, probs)


def test_sampled_rows_without_a_distribution():
    x, offsets, drafts, u, probs = _inputs([3, 3, 3, 1, 4], 2000, torch.float32, 4)
    u[:] = 0.0                      # every draft that can be is accepted
    x[1, 77] = math.nan
    x[3] = -math.inf
    x[8, 5] = math.inf
    x[9, :] = math.nan
    drafts[11] = 2000               # no token
    drafts[12] = -1
    out = _check(x, offsets, drafts, u, probs)
    assert [int(y) for y in out[:, 0]] == [1, 0, 2, 0, 1]
    assert [int(y) for y in out[:4, 1]] == [-1, -1, -1, -1] and int(out[4, 1]) >= 0
    for temp in ([1.0, 0.0, -1.0, math.nan, math.inf], [1e-29, 1e-31, 3e38, 1e-40, 1e30]):
        _check(x, offsets, drafts, u, probs, torch.tensor(temp, device="cuda"))


def test_sampled_borders():
    V = 1000
    x = torch.zeros(3, V, device="cuda")            # p = 1/1000 each
    u = torch.tensor([0.5, 0.5, 0.25049], device="cuda")
    drafts = torch.tensor([3, 4, 0], dtype=torch.int32, device="cuda")
    # q = p: u < 1 accepts, and the bonus token is the one that holds u
    out, p = _call(x, [0, 3], drafts, u, torch.full((3, V), 1.0 / V, device="cuda"))
    assert out.tolist() == [[2, 250]]
    # u q = p exactly does not accept
    x = torch.zeros(2, 4, device="cuda")
    q = torch.tensor([[0.5, 0.5, 0.0, 0.0]] * 2, device="cuda")
    u = torch.tensor([0.5, 0.75], device="cuda")
    drafts = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    assert _call(x, [0, 2], drafts, u, q)[0].tolist() == [[0, 3]]     # weights 0 0 1/4 1/4: half of them is passed at 3
    # u = 0 takes the first token with weight, u = 1 (outside of the range) the last
    x = torch.tensor([[-math.inf, 0.0, 0.0, -math.inf]], device="cuda")
    for value, token in ((0.0, 1), (1.0, 2)):
        got, _ = _call(x, [0, 1], drafts[:1], torch.tensor([value], device="cuda"))
        assert got.tolist() == [[0, token]]
    # nothing is left of p - q: p itself
    x = torch.tensor([[0.0, -math.inf], [0.0, 0.0]], device="cuda")
    q = torch.tensor([[1.0, 0.0], [0.0, 0.0]], device="cuda")
    u = torch.tensor([1.0, 0.3], device="cuda")     # 1 q < p fails: a row that rejects where p = q
    assert _call(x, [0, 2], torch.zeros(2, dtype=torch.int32, device="cuda"), u, q)[0].tolist() == [[0, 0]]


def test_sampled_draws_follow_the_target():
    # accept and residual together give the target's distribution, whatever the drafter: 40,000 sessions
    V, n = 8, 4000
    gen = torch.Generator().manual_seed(12)
    p = torch.softmax(torch.randn(V, generator=gen), 0)
    q = torch.softmax(torch.randn(V, generator=gen), 0)
    x = p.log().repeat(2 * n, 1).cuda()
    seen = torch.zeros(V)
    for i in range(10):
        drafts = torch.multinomial(q, 2 * n, replacement=True, generator=gen).to(torch.int32)
        u = torch.rand(2 * n, generator=gen).cuda()
        out, _ = _call(x, list(range(0, 2 * n + 1, 2)), drafts.cuda(), u, q.repeat(2 * n, 1).cuda(), want_p=False)
        out = out.cpu()
        first = torch.where(out[:, 0] > 0, drafts[::2], out[:, 1])
        seen += torch.bincount(first.long(), minlength=V)
    # a count's standard deviation is sqrt(N p (1 - p)) <= 100; six of them
    assert (seen - 10 * n * p).abs().max() < 600


def test_sampled_same_bits_every_time_and_in_a_graph():
    x, offsets, drafts, u, probs = _inputs([5, 15, 2], 20011, torch.bfloat16, 6)
    R, B = x.shape[0], 3
    work = kda.accept_sampled_workspace(R, B, 20011)
    ends = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    p = torch.zeros(R, device="cuda")
    kda.kda_accept_sampled(x, ends, drafts, u, out, probs=probs, p_draft=p, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_accept_sampled(x, ends, drafts, u, out, probs=probs, p_draft=p, work=work)
    for i in range(4):
        u.copy_(torch.rand(R, generator=torch.Generator().manual_seed(i)))
        out.zero_()
        p.zero_()
        work.fill_(0xFF if i & 1 else 0)
        graph.replay()
        torch.cuda.synchronize()
        got, got_p = out.clone(), p.clone()
        want, want_p = _call(x, offsets, drafts, u, probs)
        assert torch.equal(got, want)
        live = want_p != 9.0
        assert torch.equal(got_p[live], want_p[live])


def test_sampled_without_rows():
    out = torch.full((2, 2), 3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 50, device="cuda")
    kda.kda_accept_sampled(none, torch.zeros(3, dtype=torch.int32, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda"), out)
    torch.cuda.synchronize()
    assert (out == 3).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sampled_rounds_of_fewer_rows_share_the_largest_ones_workspace(dt):
    V, B = 20011, 64
    work = kda.accept_sampled_workspace(B * 8, B, V)
    for rows in ([8] * B, [8] * 63 + [7], [8, 6] * 32, [1] * B, [9, 1, 0, 15, 3], [7], [1], [2, 2, 2]):
        x, offsets, drafts, u, probs = _inputs(rows, V, dt, sum(rows))
        n = offsets[-1]
        x, drafts, u, probs = x[:n], drafts[:n], u[:n], probs[:n]
        want, want_p = _call(x, offsets, drafts, u, probs)
        work.fill_(0xFF)
        got, got_p = _call(x, offsets, drafts, u, probs, work=work)
        assert torch.equal(got, want) and torch.equal(got_p, want_p)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 600])
def test_sampled_probabilities_of_unlikely_drafts(dt, V):
    """A draft far behind the likeliest token, at any temperature: p down to f32's smallest numbers."""
    gen = torch.Generator().manual_seed(V)
    B = 64
    temp = 0.4 + 2 * torch.rand(B, generator=gen)
    x = torch.randn(2 * B, V, generator=gen)
    drafts = torch.randint(0, V, (2 * B,), generator=gen)
    x[torch.arange(2 * B), drafts] = -(60 + 20 * torch.rand(2 * B, generator=gen)) * temp.repeat_interleave(2)
    x, temp = x.to(dt).cuda(), temp.cuda()
    offsets = list(range(0, 2 * B + 1, 2))
    _, p = _call(x, offsets, drafts.to(torch.int32).cuda(), torch.rand(2 * B, generator=gen).cuda(), temp=temp)
    _, want, _ = accept_ref(x, offsets, drafts, torch.zeros(2 * B), temp=temp)
    for r, w in want.items():
        assert w > 2.0**-126
        # half steps of f32 (2^-24): the sum's exponentials, 3 (ln V + 6 ln 2) of their arguments in the mean (three
        # roundings each; the reference that they are taken from may lag by 6 in base 2), 2 of their own,
        # 10 of the additions of 32 of them; the quotient is f64 and rounded once
        assert abs(float(p[r]) - w) <= (3 * (math.log(V) + 6 * math.log(2)) + 13) * 2.0**-24 * w, (r, float(p[r]) / w - 1)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [262144, 262145, 300007, 600011])
def test_sampled_vocabularies_whose_pieces_are_several_chunks(dt, V):
    """Rows are summed in 64 pieces at most and searched 4,096 tokens at a time: tokens on both sides of the borders of
    pieces and chunks, each drawn by a number in the middle of its share; rows that live in one chunk alone."""
    gen = torch.Generator().manual_seed(V)
    each = -(-V // min(64, -(-V // 4096)))
    live = set()
    for piece in (0, 1, 31, (V - 1) // each):
        begin, end = piece * each, min(piece * each + each, V)
        live |= {begin, begin + 1, begin + 4095, begin + 4096, begin + 4097, begin + 8191, begin + 8192, end - 1} & set(range(begin, end))
    live = sorted(live)
    near = [v for v in live if each <= v < each + 4096]
    rows = []   # (tokens alive, the one that is drawn)
    rows += [(live, v) for v in live]
    rows += [(near, v) for v in near]
    rows += [([v], v) for v in live[::5]]
    x = torch.full((len(rows), V), -math.inf)
    for r, (some, _) in enumerate(rows):
        x[r, some] = torch.randn(len(some), generator=gen)
    x = x.to(dt)
    p = torch.softmax(x.double(), 1)

    def middle(weights, v):   # of v's share: some 0.1 % of the whole at least, against 1e-5 that the sums are off by
        c = torch.cumsum(weights, 0)
        share = weights[v] / c[-1]
        assert share > 1e-3
        return float((c[v] - weights[v] / 2) / c[-1])

    drawn = [v for _, v in rows]
    u = torch.tensor([middle(p[r], v) for r, v in enumerate(drawn)], dtype=torch.float32)
    # a session a row: the token of the row
    out, _ = _call(x.cuda(), list(range(len(rows) + 1)), torch.zeros(len(rows), dtype=torch.int32, device="cuda"), u.cuda(), want_p=False)
    assert out.tolist() == [[0, v] for v in drawn]
    # sessions of two rows whose draft is rejected: without it, and with what p leaves of q
    two = x.repeat_interleave(2, 0)
    offsets = list(range(0, 2 * len(rows) + 1, 2))
    drafts, left = [], torch.zeros(2 * len(rows), V)
    u_two, u_left = torch.full((2 * len(rows),), 0.999999), torch.full((2 * len(rows),), 0.999999)
    for r, (some, v) in enumerate(rows):
        d = some[0] if some[0] != v else some[-1]       # (a row of one token: nothing is left, p itself)
        drafts += [d, d]
        w = p[r].clone()
        if len(some) > 1:
            w[d] = 0.0
        u_two[2 * r + 1] = middle(w, v)
        # q takes a half of each other token's share and all of the draft's and more
        left[2 * r] = (p[r] / 2).float()
        left[2 * r, d] = 1.0
        w = (p[r] - left[2 * r].double()).clamp(min=0.0)
        if len(some) == 1:
            w = p[r]
        u_left[2 * r + 1] = middle(w, v)
    drafts = torch.tensor(drafts, dtype=torch.int32, device="cuda")
    for probs, numbers in ((None, u_two), (left.cuda(), u_left)):
        out, _ = _call(two.cuda(), offsets, drafts, numbers.cuda(), probs, want_p=False)
        # (where one token lives, p = 1 at the draft: accepted, and drawn again)
        assert out.tolist() == [[int(len(some) == 1), v] for some, v in rows]
