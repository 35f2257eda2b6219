"""A NaN or an infinity in a row of a prompt reaches that row and later ones of its own sequence
and head, as in the row program, and nothing else: every other output and state is the bits of the
same call with a finite value in its place."""
import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests import prompt_ref as ref

pytestmark = pytest.mark.gpu

D = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": -float("inf")}
H = 2


def _run(op, lens, xs, S0):
    R = sum(lens)
    S, o = S0.cuda(), torch.full(xs[2].shape, 7.0, device="cuda")
    ptrs, off = kda.state_table(S.unsqueeze(0)), ref.offsets(lens).cuda()
    xs = [x.cuda() for x in xs]
    if op == "linear":
        kda.kda_linear_prompt(ptrs, off, *xs, o=o, work=kda.linear_workspace(R, len(lens), H))
    else:
        kda.kda_prompt(ptrs, off, *xs, o=o, work=kda.prompt_workspace(R, len(lens), H))
    return o.cpu(), S.cpu()


def _check(op, lens, xs, S0, change, reached_o, reached_S):
    """change(xs, S0) puts the bad values in; reached_o [R][H][D] and reached_S [B][H][D][D] are true
    where they arrive.  There nothing is finite; elsewhere nothing changes."""
    want_o, want_S = _run(op, lens, xs, S0)
    xs, S0 = [x.clone() for x in xs], S0.clone()
    change(xs, S0)
    o, S = _run(op, lens, xs, S0)
    assert not o[reached_o].isfinite().any()
    assert torch.equal(o[~reached_o], want_o[~reached_o])
    assert not S[reached_S].isfinite().any()
    assert torch.equal(S[~reached_S], want_S[~reached_S])


def _inputs(op, lens, dtype):
    R = sum(lens)
    xs = ref.linear_inputs(90, R, H, H, dtype, 0.1) if op == "linear" else ref.kda_inputs(90, R, H, dtype, 0.1)
    return list(xs), ref.states(91, len(lens), H), torch.zeros(R, H, D, dtype=torch.bool), \
        torch.zeros(len(lens), H, D, D, dtype=torch.bool)


# one sequence of several chunks behind another; parts of 512 rows with the bad row in the first
LENS = [[20, 100, 40], [3, 2300, 5]]


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("row", [0, 13, 31, 32, 77])
def test_values(op, dtype, lens, bad, row):
    # one channel of v: that channel's outputs from the row on, and its column of the state
    xs, S0, at_o, at_S = _inputs(op, lens, DTYPES[dtype])
    t, end = lens[0] + row, lens[0] + lens[1]
    at_o[t:end, 1, 37] = True
    at_S[1, 1, :, 37] = True

    def change(xs, S0):
        xs[2][t, 1, 37] = BAD[bad]

    _check(op, lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_values_of_many_channels(op, dtype):
    # other rows for other channels of one chunk, two in one channel, the last row of a sequence
    lens = [70, 90]
    xs, S0, at_o, at_S = _inputs(op, lens, DTYPES[dtype])
    places = [(40, 0, "nan"), (45, 0, "inf"), (33, 16, "-inf"), (63, 17, "nan"), (32, 127, "inf"), (69, 64, "nan")]
    for t, c, _ in places:
        at_o[t:70, 0, c] = True
        at_S[0, 0, :, c] = True

    def change(xs, S0):
        for t, c, bad in places:
            xs[2][t, 0, c] = BAD[bad]

    _check(op, lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("row", [0, 13, 31, 32, 77])
def test_queries(op, dtype, bad, row):
    # one row's outputs
    lens = [20, 100, 40]
    xs, S0, at_o, at_S = _inputs(op, lens, DTYPES[dtype])
    at_o[20 + row, 1] = True

    def change(xs, S0):
        xs[0][20 + row, 1, 99] = BAD[bad]

    _check(op, lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("row", [0, 13, 31, 32, 77])
def test_linear_keys(dtype, row):
    # all outputs from the row on; the key's row of the state
    lens = [20, 100, 40]
    xs, S0, at_o, at_S = _inputs("linear", lens, DTYPES[dtype])
    at_o[20 + row:120, 1] = True
    at_S[1, 1, 99] = True

    def change(xs, S0):
        xs[1][20 + row, 1, 99] = BAD["nan"]

    _check("linear", lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("op", ["linear", "kda"])
def test_states(op):
    # a channel of one state
    lens = [20, 100, 40]
    xs, S0, at_o, at_S = _inputs(op, lens, torch.float32)
    at_o[20:120, 1, 5] = True
    at_S[1, 1, :, 5] = True

    def change(xs, S0):
        S0[1, 1, :, 5] = BAD["nan"]

    _check(op, lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("row", [0, 13, 31, 32, 77])
def test_linear_gates(lens, row):
    # a NaN decay: the head's outputs from the row on and its state
    xs, S0, at_o, at_S = _inputs("linear", lens, torch.float32)
    t, end = lens[0] + row, lens[0] + lens[1]
    at_o[t:end, 1] = True
    at_S[1, 1] = True

    def change(xs, S0):
        xs[3][t, 1] = BAD["nan"]

    _check("linear", lens, xs, S0, change, at_o, at_S)


@pytest.mark.parametrize("which,bad", [("g", "nan"), ("v", "inf"), ("q", "nan"), ("k", "nan")])
def test_linear_step(which, bad):
    xs = [x.view(1, 3, *x.shape[1:]).cuda() for x in ref.linear_inputs(92, 3, H, H)]
    S0 = ref.states(93, 3, H).cuda()

    def step(xs):
        S, o = S0.clone(), torch.full((1, 3, H, D), 7.0, device="cuda")
        kda.kda_linear_step(kda.state_table(S.unsqueeze(0)), *xs, o=o)
        return o[0], S

    want_o, want_S = step(xs)
    at_o, at_S = torch.zeros_like(want_o, dtype=torch.bool), torch.zeros_like(want_S, dtype=torch.bool)
    ys = [x.clone() for x in xs]
    i = "qkvg".index(which)
    if which == "g":
        ys[i][0, 1, 1] = BAD[bad]
    else:
        ys[i][0, 1, 1, 9] = BAD[bad]
    if which == "v":
        at_o[1, 1, 9] = True
        at_S[1, 1, :, 9] = True
    else:
        at_o[1, 1] = True
    if which == "k":
        at_S[1, 1, 9] = True
    if which == "g":
        at_S[1, 1] = True
    o, S = step(ys)
    assert not o[at_o].isfinite().any() and torch.equal(o[~at_o], want_o[~at_o])
    assert not S[at_S].isfinite().any() and torch.equal(S[~at_S], want_S[~at_S])


@pytest.mark.parametrize("which", ["k", "beta"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("row", [0, 13, 31, 32, 77])
def test_kda_keys_and_strengths(which, dtype, lens, bad, row):
    # a delta of every channel, so all of the head's outputs from the row on and its whole state
    xs, S0, at_o, at_S = _inputs("kda", lens, DTYPES[dtype])
    t, end = lens[0] + row, lens[0] + lens[1]
    at_o[t:end, 1] = True
    at_S[1, 1] = True

    def change(xs, S0):
        if which == "k":
            xs[1][t, 1, 99] = BAD[bad]
        else:
            xs[4][t, 1] = BAD[bad]

    _check("kda", lens, xs, S0, change, at_o, at_S)


def test_kda_several_at_once():
    # a query before and behind the first bad key of a chunk, and values in two channels
    lens = [64, 33]
    xs, S0, at_o, at_S = _inputs("kda", lens, torch.float32)
    at_o[34, 0] = at_o[40:64, 0] = True
    at_o[35:, 0, 3] = at_o[38:, 0, 100] = True
    at_o[64:] = False
    at_S[0, 0] = True

    def change(xs, S0):
        xs[0][34, 0, 1] = xs[0][50, 0, 2] = BAD["nan"]
        xs[1][40, 0, 7] = xs[1][45, 0, 8] = BAD["inf"]
        xs[2][35, 0, 3], xs[2][38, 0, 100], xs[2][60, 0, 3] = BAD["inf"], BAD["nan"], BAD["nan"]

    _check("kda", lens, xs, S0, change, at_o, at_S)


def test_kda_nan_gates_count_as_the_lowest():
    lens = [70]
    xs, S0, _, _ = _inputs("kda", lens, torch.float32)
    xs[3][5, 0, 3] = xs[3][40, 1, 100] = -5.0
    want = _run("kda", lens, xs, S0)
    rows = [x[:10].unsqueeze(0).cuda() for x in xs]
    scan = torch.empty(1, H, D, D, device="cuda")
    kda.kda_scan_rows(S0.cuda(), scan, *rows)
    xs[3][5, 0, 3] = xs[3][40, 1, 100] = BAD["nan"]
    got = _run("kda", lens, xs, S0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rows[3][0, 5, 0, 3] = BAD["nan"]
    again = torch.empty_like(scan)
    kda.kda_scan_rows(S0.cuda(), again, *rows)
    assert torch.equal(scan, again)
