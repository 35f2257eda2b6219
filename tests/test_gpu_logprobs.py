"""kda_logprobs on the GPU against float64 softmax statistics and a stable sort."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda

pytestmark = pytest.mark.gpu

NONE = -1   # KDA_NO_TOKEN read as int32
inf = float("inf")


def _call(x, tokens, n, work=None, stream=None, outs=None):
    t, V = x.shape
    if outs is None:
        outs = (torch.full((t,), 7.0, device="cuda"), torch.full((t,), 7.0, device="cuda"),
                torch.full((t, n), 7, dtype=torch.int32, device="cuda"), torch.full((t, n), 7.0, device="cuda"))
    lp, ent, ids, top = outs
    kda.kda_logprobs(x, tokens, lp, ent, *((ids, top) if n else (None, None)),
                     work=kda.logprobs_workspace(t, V, n) if work is None else work, stream=stream)
    return outs


def _want(x, tokens, n):
    """By the definition, in float64, row by row on the CPU."""
    x = x.double()
    t, V = x.shape
    lp, ent = torch.full((t,), math.nan, dtype=torch.float64), torch.full((t,), math.nan, dtype=torch.float64)
    ids = torch.full((t, n), NONE, dtype=torch.int32)
    top = torch.full((t, n), math.nan, dtype=torch.float64)
    for r in range(t):
        tok = int(tokens[r])
        ok = 0 <= tok < V
        if not (x[r] < inf).all():
            continue
        if (x[r] == -inf).all():
            lp[r], ent[r], top[r] = (-inf if ok else math.nan), 0.0, -inf
            continue
        y = x[r] - x[r].max()                     # first, or a row near the type's lowest value loses it
        y = y - y.exp().sum().log()
        p = y.exp()
        lp[r] = y[tok] if ok else math.nan
        ent[r] = -torch.xlogy(p, p).sum()
        order = torch.sort(x[r], descending=True, stable=True).indices[:n]
        there = x[r][order] > -inf
        top[r, :len(order)] = torch.where(there, y[order], -inf)
        top[r, len(order):] = -inf
        ids[r, :len(order)] = torch.where(there, order, NONE).to(torch.int32)
    # past f32's range an output is -inf
    return lp.float().double(), ent, ids, top.float().double()


def _near(got, want, tol):
    got, want = got.cpu().double(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    fine = want.isfinite()
    rest = ~fine & ~want.isnan()
    assert torch.equal(got[rest], want[rest])
    assert ((got - want).abs()[fine] <= tol[fine] if torch.is_tensor(tol) else
            (got - want).abs()[fine] <= tol).all()


def _compare(got, want, V):
    """z sums V exponentials (2 last places each) through at most V/256 + 32 adds in a row, so log z
    is off by (V/256 + 36) 2^-24 and a place of its own; x - m and the last subtraction round once
    each; the entropy's second sum is off by as much relative to itself."""
    lp, ent, ids, top = got
    z = V / 256 + 40
    _near(lp, want[0], 2.0 ** -24 * (z + 2 * want[0].abs().nan_to_num(0, 0, 0) + 2 * math.log(V + 1)))
    _near(ent, want[1], 2.0 ** -24 * (z * (1 + want[1].abs().nan_to_num(0) + math.log(V + 1))))
    if ids.shape[1]:
        assert torch.equal(ids.cpu(), want[2])
        _near(top, want[3], 2.0 ** -24 * (z + 2 * want[3].abs().nan_to_num(0, 0, 0) + 2 * math.log(V + 1)))


def _logits(seed, t, V, dtype, scale=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = (scale * torch.randn(t, V, generator=gen)).to(dtype)
    return x, torch.randint(0, V, (t,), generator=gen, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("t,V,n", [(1, 1, 0), (1, 1, 1), (2, 3, 5), (3, 63, 32), (4, 64, 1), (15, 65, 20),
                                   (1, 1000, 32), (5, 4095, 7), (2, 4097, 32), (15, 32768, 20),
                                   (1, 50001, 5), (3, 150000, 32), (300, 2050, 3), (600, 300, 0)])
def test_logprobs_sizes(dtype, t, V, n):
    x, tok = _logits(t * V + n, t, V, dtype)
    _compare(_call(x.cuda(), tok.cuda(), n), _want(x, tok, n), V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("t", [2, 700])
def test_logprobs_ties_take_the_lowest_index(dtype, t):
    V = 9001
    x, tok = _logits(1, t, V, dtype)
    x = x.round()
    x[0] = 2.0                       # all equal: 0, 1, 2, ...
    x[1] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    _compare(_call(x.cuda(), tok.cuda(), 32), _want(x, tok, 32), V)


@pytest.mark.parametrize("t", [2, 600])
@pytest.mark.parametrize("order", ["rising", "falling", "late"])
def test_logprobs_sorted_rows(order, t):
    # every next value is among the best so far, or none is, or all of the best come last
    V = 20011
    x = torch.linspace(-40, 10, V).expand(t, V).clone()
    if order == "falling":
        x = x.flip(1).contiguous()
    if order == "late":
        x = torch.full((t, V), -5.0)
        x[:, -40:] = torch.arange(40).float()
    tok = torch.full((t,), V - 1, dtype=torch.int32)
    _compare(_call(x.cuda(), tok.cuda(), 32), _want(x, tok, 32), V)


@pytest.mark.parametrize("t_more", [0, 700])
@pytest.mark.parametrize("V", [70, 5000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_logprobs_special_rows(dtype, V, t_more):
    t = 14
    x, tok = _logits(2, t + t_more, V, dtype)
    low = torch.finfo(dtype).min
    x[0] = -inf                                   # nothing left
    x[1, 1:] = -inf                               # one token left
    x[2, 10:] = -inf                              # fewer than the alternatives asked for
    x[3, V // 2] = math.nan
    x[4, V - 1] = inf
    x[5] = math.nan
    x[6, 3:] = low                                # masked by the type's lowest value
    x[7] = low
    x[8, 5] = torch.finfo(dtype).max              # a value that others overflow against
    x[8, 6] = low
    x[9] = 0.0                                    # uniform
    x[10, ::2] = -inf
    x[11, 0] = 80.0                               # one certain token
    x[12, V - 1] = inf
    x[12, 0] = math.nan
    x[13, V - 1] = 60.0
    tok[1], tok[2], tok[6], tok[8], tok[10], tok[11] = 5, 3, V - 1, 6, 0, 0
    tok[9] = V                                    # no such token
    tok[13] = NONE
    _compare(_call(x.cuda(), tok.cuda(), 20), _want(x, tok, 20), V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("t", [3, 520])
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (8, 3), (0, 8), (4, 12)])
def test_logprobs_row_strides_and_alignment(dtype, t, offset, pad):
    V = 3001
    gen = torch.Generator().manual_seed(offset + pad)
    flat = (3 * torch.randn(offset + t * (V + pad), generator=gen)).to(dtype)
    for r in range(t):                            # what lies between the rows must not count
        flat[offset + r * (V + pad) + V:offset + (r + 1) * (V + pad)] = math.nan
    x = flat.cuda()[offset:].view(t, V + pad)[:, :V]
    tok = torch.randint(0, V, (t,), generator=gen, dtype=torch.int32)
    _compare(_call(x, tok.cuda(), 9), _want(x.cpu(), tok, 9), V)


def test_logprobs_outputs_are_optional():
    x, tok = _logits(3, 4, 777, torch.float32)
    x, tok = x.cuda(), tok.cuda()
    lp, ent, ids, top = _call(x, tok, 5)
    a, b = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    kda.kda_logprobs(x, tok, lp=a, work=kda.logprobs_workspace(4, 777, 0))
    kda.kda_logprobs(x, entropy=b, work=kda.logprobs_workspace(4, 777, 0))
    c, d = torch.empty_like(ids), torch.empty_like(top)
    kda.kda_logprobs(x, top_ids=c, top_lp=d, work=kda.logprobs_workspace(4, 777, 5))
    for u, w in ((a, lp), (b, ent), (c, ids), (d, top)):
        assert torch.equal(u, w)


def test_logprobs_rows_past_32_bit_offsets():
    V, ld, t = 500, 1 << 28, 9                    # the last row starts at element 2^31
    x = torch.empty((t - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((t, V), (ld, 1))
    y, tok = _logits(4, t, V, torch.bfloat16)
    x.copy_(y)
    _compare(_call(x, tok.cuda(), 6), _want(y, tok, 6), V)


@pytest.mark.parametrize("t,V", [(3, 30001), (600, 500)])
def test_logprobs_graph_replays_and_two_streams(t, V):
    n = 11
    xs = [_logits(5 + i, t, V, torch.float32) for i in range(2)]
    xs = [(x.cuda(), tok.cuda()) for x, tok in xs]
    work = [kda.logprobs_workspace(t, V, n) for _ in xs]
    outs = [_call(x, tok, n, work[i]) for i, (x, tok) in enumerate(xs)]
    torch.cuda.synchronize()
    want = [[y.clone() for y in o] for o in outs]
    graphs = []
    for i, (x, tok) in enumerate(xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(x, tok, n, work[i], outs=outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    for rep in range(4):
        for o in outs:
            for y in o:
                y.fill_(rep)
        torch.cuda.synchronize()
        for i, (x, tok) in enumerate(xs):
            if rep % 2:
                _call(x, tok, n, work[i], streams[i], outs[i])
            else:
                graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for u, y in zip(o, w):
                assert torch.equal(u, y), rep
