"""kda_prompt, kda_linear_prompt and kda_linear_step on the GPU against float64 recurrences."""
import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests import prompt_ref as ref

pytestmark = pytest.mark.gpu

D = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# lengths around one row, the chunk edges, several chunks, empty sequences in every place
LENS = [[1], [2], [15, 16, 17], [0, 1, 0], [31, 32, 33], [63, 0, 64, 65], [127, 129], [200, 3, 1, 0],
        [511, 513], [0, 0]]


def _pointers(S):
    return kda.state_table(S.unsqueeze(0))


def _cuda(*xs):
    return [x.cuda() for x in xs]


def _linear(S, lens, xs, o=None, off=None, ptrs=None, work=None, stream=None):
    R, H = xs[2].shape[:2]
    B = S.shape[0]
    off = ref.offsets(lens).cuda() if off is None else off
    work = kda.linear_workspace(R, B, H) if work is None else work
    kda.kda_linear_prompt(_pointers(S) if ptrs is None else ptrs, off, *xs, o=o, work=work, stream=stream)


def _kda(S, lens, xs, o=None, off=None, ptrs=None, work=None, stream=None):
    R, H = xs[2].shape[:2]
    B = S.shape[0]
    off = ref.offsets(lens).cuda() if off is None else off
    work = kda.prompt_workspace(R, B, H) if work is None else work
    kda.kda_prompt(_pointers(S) if ptrs is None else ptrs, off, *xs, o=o, work=work, stream=stream)


def _inputs(op, seed, R, H, dtype=torch.float32, Hk=None, g_scale=None):
    if op == "linear":
        return ref.linear_inputs(seed, R, Hk or H, H, dtype, 1.0 if g_scale is None else g_scale)
    return ref.kda_inputs(seed, R, H, dtype, 5.0 if g_scale is None else g_scale)


CALL = {"linear": _linear, "kda": _kda}
ROWS = {"linear": ref.linear_rows, "kda": ref.kda_rows}


def _check(op, lens, xs, S0):
    R = sum(lens)
    want_o, want_S = ref.packed(ROWS[op], S0, lens, *xs)
    S = S0.cuda()
    o = torch.full(xs[2].shape, 7.0, device="cuda")
    CALL[op](S, lens, _cuda(*xs), o)
    torch.cuda.synchronize()
    tol = ref.tolerance(max(lens))
    if R:
        assert ref.relative(o, want_o) <= tol
    for b, n in enumerate(lens):
        if n:
            assert ref.relative(S[b], want_S[b]) <= tol, b
        else:
            assert torch.equal(S[b].cpu(), S0[b])
    # the state alone, and the same bits again
    S2 = S0.cuda()
    CALL[op](S2, lens, _cuda(*xs), None)
    assert torch.equal(S, S2)


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt_lengths(op, dtype, lens):
    xs = _inputs(op, len(lens) + sum(lens), sum(lens), 3, DTYPES[dtype])
    _check(op, lens, xs, ref.states(5, len(lens), 3))


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [1, 2, 8])
def test_prompt_long(op, dtype, H):
    lens = [1300, 77]
    xs = _inputs(op, H, sum(lens), H, DTYPES[dtype], g_scale=0.05)
    _check(op, lens, xs, ref.states(6, 2, H))


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("lens,H,g_scale", [([2100, 0, 600], 2, 0.02), ([2048], 16, 5.0), ([5, 2600], 1, 0.5),
                                            ([513, 512, 511, 544], 4, 0.01), ([2560], 3, 0.0)], ids=str)
def test_prompt_in_parts(op, lens, H, g_scale):
    # few heads and long sequences: parts side by side, chained by their transitions
    xs = _inputs(op, H + len(lens), sum(lens), H, torch.bfloat16, g_scale=g_scale)
    _check(op, lens, xs, ref.states(23, len(lens), H))


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 4), (2, 4), (3, 6), (5, 5)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_linear_prompt_shared_key_heads(Hk, H, dtype):
    lens = [70, 1, 129]
    xs = _inputs("linear", Hk + H, sum(lens), H, DTYPES[dtype], Hk)
    _check("linear", lens, xs, ref.states(7, 3, H))


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("g", [0.0, -0.001, -5.0, -30.0, 3.0])
def test_prompt_constant_gates(op, g):
    # no decay, almost none, the KDA bound, far past it, and a gate that would grow the state
    lens = [130, 33]
    xs = list(_inputs(op, 11, sum(lens), 2))
    xs[3] = torch.full_like(xs[3], g)
    _check(op, lens, xs, ref.states(8, 2, 2))


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_gates_that_differ_by_row_and_channel(op):
    # rows of no decay between rows of the strongest, so that a chunk's running sums lose what
    # follows if they are not taken apart
    lens = [150]
    xs = list(_inputs(op, 12, 150, 2))
    strong = torch.zeros(150, dtype=torch.bool)
    strong[::7] = True
    xs[3] = torch.where(strong.view(-1, *[1] * (xs[3].dim() - 1)), torch.full_like(xs[3], -5.0),
                        xs[3] * 1e-3)
    _check(op, lens, xs, ref.states(9, 1, 2))


def test_linear_prompt_restarts_at_minus_infinity():
    lens = [100, 65]
    xs = list(_inputs("linear", 13, sum(lens), 2))
    for t, g in ((0, -float("inf")), (17, -1e30), (18, -float("inf")), (64, -200.0), (99, -3.0e38),
                 (100, -104.5), (164, -float("inf"))):
        xs[3][t] = g
    _check("linear", lens, xs, ref.states(10, 2, 2))


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_kda_prompt_beta_ends(beta):
    lens = [90]
    xs = list(_inputs("kda", 14, 90, 2, g_scale=0.2))
    xs[4] = torch.full_like(xs[4], beta)
    _check("kda", lens, xs, ref.states(11, 1, 2))


def test_kda_prompt_repeated_key():
    # the same key in every row: the triangular system is as far from the identity as it gets
    lens = [96]
    xs = list(_inputs("kda", 15, 96, 2, g_scale=0.02))
    xs[1] = xs[1][:1].expand_as(xs[1]).contiguous()
    xs[4] = torch.full_like(xs[4], 1.0)
    _check("kda", lens, xs, ref.states(12, 1, 2))


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_prompt_scales_with_the_state_and_values(op, scale):
    # both operators are linear in (state, v): a power of two comes out exactly
    lens = [70, 20]
    xs = list(_inputs(op, 16, 90, 2))
    S0 = ref.states(13, 2, 2)
    got = []
    for f in (1.0, scale):
        S, ys = (S0 * f).cuda(), list(xs)
        ys[2] = xs[2] * f
        o = torch.empty(xs[2].shape, device="cuda")
        CALL[op](S, lens, _cuda(*ys), o)
        got.append((o / f, S / f))
    assert ref.relative(got[1][0], got[0][0].cpu()) <= 2.0 ** -20
    assert ref.relative(got[1][1], got[0][1].cpu()) <= 2.0 ** -20


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_columns_of_very_different_size(op):
    # value columns never meet: powers of two by column come out to the bit
    lens = [100, 33]
    xs = list(_inputs(op, 27, 133, 2, g_scale=0.3))
    S0 = ref.states(28, 2, 2)
    scale = torch.exp2((torch.arange(D) * 7 % 61 - 30).float())
    got = []
    for f in (torch.ones(D), scale):
        S, ys = (S0 * f).cuda(), list(xs)
        ys[2] = xs[2] * f
        o = torch.empty(xs[2].shape, device="cuda")
        CALL[op](S, lens, _cuda(*ys), o)
        got.append((o.cpu() / f, S.cpu() / f))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_rows_of_very_different_size(op):
    # rows of v over 2^16, beta of 0 in the largest, a state far above what the rows add
    lens = [96]
    xs = list(_inputs(op, 29, 96, 2, g_scale=0.3))
    size = torch.exp2((torch.arange(96) * 5 % 17).float())
    xs[2] = xs[2] * size[:, None, None]
    if op == "kda":
        xs[4] = torch.where(size[:, None] > 2.0 ** 15, torch.zeros(()), xs[4])
    _check(op, lens, xs, ref.states(30, 1, 2, 1000.0))


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_leaves_rows_outside_its_sequences(op):
    # rows before, between and behind the sequences, and a sequence with no state
    R, H = 120, 2
    xs = _inputs(op, 17, R, H)
    off = torch.tensor([5, 40, 40, 73, 100], dtype=torch.int32)
    S0 = ref.states(14, 4, H)
    S = S0.cuda()
    ptrs = _pointers(S)
    ptrs[2] = 0
    o = torch.full((R, H, D), 7.0, device="cuda")
    CALL[op](S, None, _cuda(*xs), o, off=off.cuda(), ptrs=ptrs)
    o, S = o.cpu(), S.cpu()
    for a, b in ((0, 5), (40, 73), (100, R)):
        assert (o[a:b] == 7.0).all()
    for b in (1, 2):
        assert torch.equal(S[b], S0[b])
    for b, (lo, hi) in ((0, (5, 40)), (3, (73, 100))):
        want_o, want_S = ROWS[op](S0[b], *(x[lo:hi] for x in xs))
        assert ref.relative(o[lo:hi], want_o) <= ref.tolerance(hi - lo)
        assert ref.relative(S[b], want_S) <= ref.tolerance(hi - lo)


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_reads_bad_offsets_as_clamped(op):
    R, H = 50, 1
    xs = _inputs(op, 18, R, H)
    off = torch.tensor([-9, 20, 10, 2000000000], dtype=torch.int32)   # read with a running maximum: 0..20, none, 20..50
    S0 = ref.states(15, 3, H)
    S = S0.cuda()
    CALL[op](S, None, _cuda(*xs), None, off=off.cuda())
    for b, (lo, hi) in ((0, (0, 20)), (2, (20, 50))):
        _, want = ROWS[op](S0[b], *(x[lo:hi] for x in xs))
        assert ref.relative(S[b], want) <= ref.tolerance(hi - lo)
    assert torch.equal(S[1].cpu(), S0[1])


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_does_not_depend_on_its_neighbours(op):
    lens = [130, 40]
    xs = _inputs(op, 19, 170, 2)
    S0 = ref.states(16, 2, 2)
    S = S0.cuda()
    CALL[op](S, lens, _cuda(*xs), None)
    for b, part in ((0, slice(0, 130)), (1, slice(130, 170))):
        alone = S0[b:b + 1].cuda()
        CALL[op](alone, [lens[b]], _cuda(*(x[part].contiguous() for x in xs)), None)
        assert torch.equal(alone[0], S[b])


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_rows_past_32_bit_offsets(op):
    # the sequence lies behind 2^31 elements of q, k, v (and o)
    H, n = 64, 40
    R = (2 ** 31) // (H * D) + 100
    xs = _inputs(op, 20, n, H, torch.bfloat16)
    S0 = ref.states(17, 1, H)
    want_o, want_S = ROWS[op](S0[0], *xs)
    big = []
    for x in xs:
        y = torch.empty(R, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[R - n:] = x.cuda()
        big.append(y)
    o = torch.empty(R, H, D, device="cuda")
    S = S0.cuda()
    CALL[op](S, None, big, o, off=torch.tensor([R - n, R], dtype=torch.int32, device="cuda"))
    assert ref.relative(o[R - n:], want_o) <= ref.tolerance(n)
    assert ref.relative(S[0], want_S[0:]) <= ref.tolerance(n)


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_sequence_across_a_full_workspace(op):
    # 581 slots of prepared chunks, of which the workspace holds 574: the second sequence's
    # chunks (slots 572..576) are walked in two turns, the third's in the last
    H, R, cuts = 64, 18500, [0, 18300, 18450, 18500]
    xs = _inputs(op, 25, R - cuts[1], H, torch.bfloat16, g_scale=0.1)
    S0 = ref.states(26, 3, H)
    big = []
    for x in xs:
        y = torch.zeros(R, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[cuts[1]:] = x.cuda()
        big.append(y)
    S = S0.cuda()
    ptrs = _pointers(S)
    ptrs[0] = 0
    o = torch.full((R, H, D), 7.0, device="cuda")
    CALL[op](S, None, big, o, off=torch.tensor(cuts, dtype=torch.int32, device="cuda"), ptrs=ptrs)
    assert torch.equal(S[0].cpu(), S0[0])
    assert (o[:cuts[1]] == 7.0).all()
    for b in (1, 2):
        part = slice(cuts[b] - cuts[1], cuts[b + 1] - cuts[1])
        want_o, want_S = ROWS[op](S0[b], *(x[part] for x in xs))
        tol = ref.tolerance(cuts[b + 1] - cuts[b])
        assert ref.relative(o[cuts[b]:cuts[b + 1]], want_o) <= tol
        assert ref.relative(S[b], want_S) <= tol


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("B", [64, 65, 300, 4096])
def test_prompt_many_short_sequences(op, B):
    lens = [(7 * i) % 5 if i % 64 < 50 else 0 for i in range(B)]
    lens[B // 2] = 70
    xs = _inputs(op, 21, sum(lens), 1)
    _check(op, lens, xs, ref.states(18, B, 1))


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_prompt_long_tables_with_bad_entries(op):
    # 200 entries, some far out or falling: as if by the running maximum
    B, R = 200, 900
    gen = torch.Generator().manual_seed(24)
    off = torch.sort(torch.randint(0, R + 1, (B + 1,), generator=gen)).values.to(torch.int32)
    off[3], off[70], off[150], off[199] = -5, 0, 2 ** 31 - 1, -2 ** 31
    read = torch.cummax(off.clamp(0, R), 0).values.tolist()
    xs = _inputs(op, 25, R, 1)
    S0 = ref.states(26, B, 1)
    S = S0.cuda()
    o = torch.full((R, 1, D), 7.0, device="cuda")
    CALL[op](S, None, _cuda(*xs), o, off=off.cuda())
    for b in range(B):
        lo, hi = read[b], read[b + 1]
        if lo == hi:
            assert torch.equal(S[b].cpu(), S0[b]), b
        else:
            want_o, want_S = ROWS[op](S0[b], *(x[lo:hi] for x in xs))
            assert ref.relative(S[b], want_S) <= ref.tolerance(hi - lo), b
            assert ref.relative(o[lo:hi], want_o) <= ref.tolerance(hi - lo), b


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("lens", [[[150, 20], [64, 300]], [[2100, 20], [7, 2300]]], ids=["chunks", "parts"])
def test_prompt_graph_replays_and_two_streams(op, lens):
    """A captured call replays to the eager bits, and two calls on two streams with a
    workspace each do not disturb each other."""
    H = 4
    xs = [_cuda(*_inputs(op, 22 + i, sum(n), H, torch.bfloat16)) for i, n in enumerate(lens)]
    S0 = [ref.states(19 + i, 2, H).cuda() for i in range(2)]
    S = [x.clone() for x in S0]
    o = [torch.zeros(sum(n), H, D, device="cuda") for n in lens]
    off = [ref.offsets(n).cuda() for n in lens]
    ptrs = [_pointers(x) for x in S]
    space = kda.linear_workspace if op == "linear" else kda.prompt_workspace
    work = [space(sum(n), 2, H) for n in lens]

    def call(i, stream=None):
        CALL[op](S[i], None, xs[i], o[i], off=off[i], ptrs=ptrs[i], work=work[i], stream=stream)

    want = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        want.append((S[i].clone(), o[i].clone()))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(4):
        for i in range(2):
            S[i].copy_(S0[i])
            o[i].fill_(float(rep))
        torch.cuda.synchronize()
        for i in range(2):
            if rep % 2:
                call(i, streams[i])
            else:
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(S[i], want[i][0]) and torch.equal(o[i], want[i][1]), (rep, i)


# ------------------------------------------------------------------ single tokens


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("L,B,Hk,H", [(1, 1, 1, 1), (1, 1, 8, 8), (3, 5, 2, 6), (2, 40, 1, 3)])
def test_linear_step(dtype, L, B, Hk, H):
    n = L * B
    xs = ref.linear_inputs(30 + n, n, Hk, H, DTYPES[dtype])
    S0 = ref.states(31, n, H)
    want_o, want_S = ref.packed(ref.linear_rows, S0, [1] * n, *xs)
    S = S0.cuda()
    o = torch.empty(L, B, H, D, device="cuda")
    ys = [x.view(L, B, *x.shape[1:]).contiguous().cuda() for x in xs]
    kda.kda_linear_step(kda.state_table(S.view(L, B, H, D, D)), *ys, o=o)
    assert ref.relative(o.view(n, H, D), want_o) <= ref.tolerance(1)
    assert ref.relative(S, want_S) <= ref.tolerance(1)
    S2 = S0.cuda()
    kda.kda_linear_step(kda.state_table(S2.view(L, B, H, D, D)), *ys)
    assert torch.equal(S, S2)


def test_linear_step_leaves_out_sessions_without_a_state():
    xs = [x.view(1, 3, *x.shape[1:]).cuda() for x in ref.linear_inputs(40, 3, 2, 2)]
    S0 = ref.states(41, 3, 2).cuda()
    S = S0.clone()
    ptrs = _pointers(S)
    ptrs[1] = 0
    o = torch.full((1, 3, 2, D), 7.0, device="cuda")
    kda.kda_linear_step(ptrs, *xs, o=o)
    assert torch.equal(S[1], S0[1]) and (o[0, 1] == 7.0).all()
    assert not torch.equal(S[0], S0[0]) and not (o[0, 2] == 7.0).any()


@pytest.mark.parametrize("g", [0.0, 2.0, -200.0, -float("inf")])
def test_linear_step_gates(g):
    xs = list(ref.linear_inputs(42, 1, 1, 1))
    xs[3] = torch.full_like(xs[3], g)
    S0 = ref.states(43, 1, 1)
    want_o, want_S = ref.packed(ref.linear_rows, S0, [1], *xs)
    S = S0.cuda()
    o = torch.empty(1, 1, 1, D, device="cuda")
    kda.kda_linear_step(_pointers(S), *(x.view(1, 1, *x.shape[1:]).cuda() for x in xs), o=o)
    assert ref.relative(o.view(1, 1, D), want_o) <= ref.tolerance(1)
    assert ref.relative(S, want_S) <= ref.tolerance(1)


# ------------------------------------------------------------------ together


def test_linear_prompt_then_steps_equals_the_whole_prompt():
    n, H, extra = 100, 4, 5
    xs = ref.linear_inputs(50, n + extra, 2, H, torch.bfloat16)
    S0 = torch.zeros(1, H, D, D)
    want_o, want_S = ref.packed(ref.linear_rows, S0, [n + extra], *xs)
    S = S0.cuda()
    o = torch.empty(n, H, D, device="cuda")
    _linear(S, [n], _cuda(*(x[:n].contiguous() for x in xs)), o)
    assert ref.relative(o, want_o[:n]) <= ref.tolerance(n)
    for t in range(n, n + extra):
        step = torch.empty(1, 1, H, D, device="cuda")
        kda.kda_linear_step(_pointers(S), *(x[t].view(1, 1, *x.shape[1:]).cuda() for x in xs), o=step)
        assert ref.relative(step.view(1, H, D), want_o[t:t + 1]) <= ref.tolerance(n + extra)
    assert ref.relative(S, want_S) <= ref.tolerance(n + extra)


def test_prompt_then_verify_round_accept_and_log_probabilities():
    """A session as it is served: prompt, verify rows against the state it left, the accept,
    the log probabilities of the committed tokens, and the rollback."""
    n, T, H, V = 90, 6, 4, 5000
    xs = ref.kda_inputs(60, n + T, H, torch.bfloat16, 1.0)
    S0 = torch.zeros(1, H, D, D)
    want_o, _ = ref.packed(ref.kda_rows, S0, [n + T], *xs)
    S = S0.cuda()
    _kda(S, [n], _cuda(*(x[:n].contiguous() for x in xs)))
    rows = [x[n:].unsqueeze(0).contiguous().cuda() for x in xs]
    after, o = torch.empty_like(S), torch.empty(1, T, H, D, device="cuda")
    kda.kda_scan_rows(S, after, *rows, o=o)
    assert ref.relative(o[0], want_o[n:]) <= ref.tolerance(n + T)

    gen = torch.Generator().manual_seed(61)
    logits = 3 * torch.randn(T, V, generator=gen)
    best = logits.argmax(1)
    drafts = best[:T - 1].to(torch.int32)
    drafts[3] = (drafts[3] + 1) % V
    vam, out2 = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    x = logits.cuda()
    kda.kda_accept_greedy(x, drafts.cuda(), vam, out2, kda.accept_workspace())
    lp, ent = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ids, top = torch.empty(T, 3, dtype=torch.int32, device="cuda"), torch.empty(T, 3, device="cuda")
    kda.kda_logprobs(x, vam, lp, ent, ids, top, kda.logprobs_workspace(T, V, 3))
    torch.cuda.synchronize()
    assert int(out2[0]) == 3 and torch.equal(ids[:, 0], vam) and torch.equal(top[:, 0], lp)
    want = torch.log_softmax(logits.double(), 1).gather(1, best[:, None])[:, 0]
    assert (lp.cpu().double() - want).abs().max() <= 2.0 ** -24 * (V / 256 + 80)

    keep = int(out2[0]) + 1
    back = torch.empty_like(S)
    kda.kda_replay(S, back, *rows, keep=keep)
    _, want_S = ref.packed(ref.kda_rows, S0, [n + keep], *(x[:n + keep] for x in xs))
    assert ref.relative(back, want_S) <= ref.tolerance(n + T)
