"""The prompts and the linear step to the precision that their operands' words allow."""
import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests import prompt_ref as ref
from tests.prompt_words import BOUND

pytestmark = pytest.mark.gpu

D = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _softplus_gates(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    return -torch.nn.functional.softplus(2.0 * torch.randn(shape, generator=gen))


@pytest.mark.parametrize("op", ["linear", "kda"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens,H", [([1], 2), ([33, 150], 2), ([700, 64], 3), ([2300], 2)], ids=str)
@pytest.mark.parametrize("gates", ["plain", "slow"])
def test_prompts(op, dtype, lens, H, gates):
    R, B = sum(lens), len(lens)
    if op == "linear":
        xs = list(ref.linear_inputs(110, R, H, H, DTYPES[dtype], 0.02))
        if gates == "plain":
            xs[3] = _softplus_gates(xs[3].shape, 111)
    else:
        xs = list(ref.kda_inputs(110, R, H, DTYPES[dtype], 0.02))
        if gates == "plain":
            xs[3] = _softplus_gates(xs[3].shape, 111).clamp(-5.0, 0.0).to(DTYPES[dtype])
    S0 = ref.states(112, B, H)
    want_o, want_S = ref.packed({"linear": ref.linear_rows, "kda": ref.kda_rows}[op], S0, lens, *xs)
    S, o = S0.cuda(), torch.empty(R, H, D, device="cuda")
    ptrs, off, ys = kda.state_table(S.unsqueeze(0)), ref.offsets(lens).cuda(), [x.cuda() for x in xs]
    if op == "linear":
        kda.kda_linear_prompt(ptrs, off, *ys, o=o, work=kda.linear_workspace(R, B, H))
    else:
        kda.kda_prompt(ptrs, off, *ys, o=o, work=kda.prompt_workspace(R, B, H))
    assert ref.relative(o, want_o) <= BOUND
    assert ref.relative(S, want_S) <= BOUND


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_linear_step(dtype):
    n, H = 40, 4
    xs = ref.linear_inputs(113, n, 2, H, DTYPES[dtype])
    S0 = ref.states(114, n, H)
    want_o, want_S = ref.packed(ref.linear_rows, S0, [1] * n, *xs)
    S, o = S0.cuda(), torch.empty(1, n, H, D, device="cuda")
    kda.kda_linear_step(kda.state_table(S.unsqueeze(0)), *(x.unsqueeze(0).cuda() for x in xs), o=o)
    assert ref.relative(o[0], want_o) <= BOUND
    assert ref.relative(S, want_S) <= BOUND
