"""kda_prompt and kda_linear_prompt row by row: every row's output and every column of the state
against float64, each relative to itself.  One norm over a whole output is blind to rows that are
small beside the others: late rows of a chunk whose state has decayed and that add little to it."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests import prompt_ref as ref

pytestmark = pytest.mark.gpu

D = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# below this a row's outputs come near the end of float32's range, where its values lose bits
SMALLEST = 2.0 ** -100


def _call(op, S, lens, xs, o):
    R, H = xs[2].shape[:2]
    ptrs, off = kda.state_table(S.unsqueeze(0)), ref.offsets(lens).cuda()
    if op == "linear":
        kda.kda_linear_prompt(ptrs, off, *xs, o=o, work=kda.linear_workspace(R, len(lens), H))
    else:
        kda.kda_prompt(ptrs, off, *xs, o=o, work=kda.prompt_workspace(R, len(lens), H))


def _sizes(rows, S, lens, xs):
    """What the rounding errors of a row's outputs are relative to, [R][H].  Output j is the sum of
    128 products q_c S_cj, each off by its own share of itself, independently: the sum's error has
    the size of the root of their squares, which can be far above the sum where q happens to be at
    right angles to what the state holds (behind one large row the state is nearly k v^T, and q.k
    can be anything below the root of the squares of q_c k_c)."""
    size, first = [], 0
    for b, n in enumerate(lens):
        s = S[b].double()
        for t in range(first, first + n):
            _, s = rows(s, *(x[t:t + 1] for x in xs))
            q = xs[0][t].double()
            q = q.repeat_interleave(s.shape[0] // q.shape[0], dim=0)
            size.append((q[:, :, None] * s).norm(dim=(1, 2)) / math.sqrt(D))
        first += n
    return torch.stack(size)


def _worst(got, want, dim, size=None):
    """The largest 2-norm error along dim, relative to the values (or to size, if that is larger),
    of what is not too small for it."""
    assert torch.isfinite(got).all()
    size = want.norm(dim=dim) if size is None else torch.maximum(size, want.norm(dim=dim))
    there = size > SMALLEST
    return torch.where(there, (got - want).norm(dim=dim) / size.clamp(min=SMALLEST), 0.0), there


def _check(op, lens, xs, S0, row, rest):
    """row: 2^-24 that a row's error may grow by with every row of its sequence; rest: what comes
    once."""
    rows = {"linear": ref.linear_rows, "kda": ref.kda_rows}[op]
    want_o, want_S = ref.packed(rows, S0, lens, *xs)
    size = _sizes(rows, S0, lens, xs)
    S, o = S0.cuda(), torch.full(xs[2].shape, 7.0, device="cuda")
    _call(op, S, lens, [x.cuda() for x in xs], o)
    at = torch.cat([torch.arange(n) for n in lens])
    err, there = _worst(o.cpu().double(), want_o, -1, size)                 # [R][H]
    assert there.any()
    assert bool((err <= 2.0 ** -24 * (row * (at[:, None] + 1) + rest)).all()), (float(err.max()), int(err.argmax()))
    err, there = _worst(S.cpu().double(), want_S, -2)                       # by column: [B][H][D]
    tol = torch.tensor([2.0 ** -24 * (row * n + rest) for n in lens])
    assert bool((err <= tol[:, None, None]).all()), float(err.max())


# Tolerances, in 2^-24.  A row's decay is an exponential good to one last place (2) and one product
# (1): 3 a row, in one direction where every gate is the same.  Beside it each output passes through
# a few operands of 22 bits (4 each) and f32 sums whose roundings are independent: 16 for an output
# of the decayed state alone, 64 where the deltas (their system, their own operands and sums) come in.
ROW, STATE_ONLY, DELTAS = 3, 16, 64


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("g", [0.0, -0.6, -1.0, -2.5, -5.0])
def test_kda_rows_that_add_nothing(dtype, g):
    # beta of 0: each output is the decayed state's alone
    lens = [64, 33]
    xs = list(ref.kda_inputs(70, 97, 2, DTYPES[dtype]))
    xs[3], xs[4] = torch.full_like(xs[3], g), torch.zeros_like(xs[4])
    _check("kda", lens, xs, ref.states(71, 2, 2), ROW, STATE_ONLY)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("g", [-0.6, -1.0, -2.5])
def test_kda_rows_without_values(dtype, g):
    # v of 0: the deltas take from the state only, and decay with it
    lens = [40, 64]
    xs = list(ref.kda_inputs(72, 104, 2, DTYPES[dtype]))
    xs[2], xs[3] = torch.zeros_like(xs[2]), torch.full_like(xs[3], g)
    _check("kda", lens, xs, ref.states(73, 2, 2), ROW, DELTAS)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("what", ["beta", "v"])
def test_kda_late_rows_that_add_nothing(dtype, what):
    # the second half of each chunk leaves what the first half wrote to decay
    lens = [96, 64]
    xs = list(ref.kda_inputs(74, 160, 2, DTYPES[dtype]))
    xs[3] = torch.full_like(xs[3], -1.0)
    at = torch.cat([torch.arange(n) for n in lens]) % 32 >= 16
    if what == "beta":
        xs[4] = torch.where(at[:, None], torch.zeros_like(xs[4]), xs[4])
    else:
        xs[2] = torch.where(at[:, None, None], torch.zeros_like(xs[2]), xs[2])
    _check("kda", lens, xs, ref.states(75, 2, 2), ROW, DELTAS)


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("g", [0.0, -0.6, -2.5])
def test_values_of_any_size(op, g):
    # rows of v of 2^-20 .. 2^20 in no order
    lens = [100]
    xs = list(ref.kda_inputs(76, 100, 2) if op == "kda" else ref.linear_inputs(76, 100, 2, 2))
    xs[2] = xs[2] * torch.exp2((torch.arange(100) * 7 % 41 - 20).float())[:, None, None]
    xs[3] = torch.full_like(xs[3], g)
    _check(op, lens, xs, ref.states(77, 1, 2), ROW, DELTAS)


@pytest.mark.parametrize("g", [-0.6, -2.5, -20.0])
def test_linear_rows_that_add_nothing(g):
    lens = [64, 33]
    xs = list(ref.linear_inputs(78, 97, 2, 2))
    xs[2], xs[3] = torch.zeros_like(xs[2]), torch.full_like(xs[3], g)
    _check("linear", lens, xs, ref.states(79, 2, 2), ROW, STATE_ONLY)


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens,H", [([130, 33, 1], 3), ([2100, 64], 2)], ids=str)
def test_rows_of_plain_prompts(op, dtype, lens, H):
    # gates as a model has them; few heads and long sequences run in parts
    R = sum(lens)
    xs = list(ref.kda_inputs(80, R, H, DTYPES[dtype]) if op == "kda" else ref.linear_inputs(80, R, H, H, DTYPES[dtype]))
    gen = torch.Generator().manual_seed(81)
    g = -torch.nn.functional.softplus(2.0 * torch.randn(xs[3].shape, generator=gen))
    xs[3] = g.clamp(-5.0, 0.0).to(xs[3].dtype)
    # random gates: what a row's error brings with it decays within a few rows
    _check(op, lens, xs, ref.states(82, len(lens), H), 0, DELTAS)


def test_small_states():
    # a state near the end of float32's range, and nothing added
    xs = list(ref.kda_inputs(83, 40, 2, g_scale=0.1))
    xs[4] = torch.zeros_like(xs[4])
    S0 = ref.states(84, 1, 2) * 2.0 ** -90
    _check("kda", [40], xs, S0, ROW, STATE_ONLY)
    assert math.isclose(SMALLEST, 2.0 ** -100)
