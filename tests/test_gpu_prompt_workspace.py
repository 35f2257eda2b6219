"""The prompts' workspaces: calls stay within the bytes they ask for, whatever their sequences are."""
import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests import prompt_ref as ref

pytestmark = pytest.mark.gpu

D = 128
GUARD = 1 << 20


def _guarded(n):
    whole = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    return whole[:n], whole[n:]


# sequences of several parts of 512 rows between short, empty and one-part ones; more of them than
# R / 512 (places by twice the rows), and fewer (places by slots)
@pytest.mark.parametrize("lens", [[1, 513, 0, 1, 2, 1030, 3, 512, 5, 600], [513, 513, 513], [700] + [1] * 30 + [2000],
                                  [511, 1025, 514], [0, 0, 1540, 0], [3] * 200 + [513]], ids=lambda x: str(x[:4]))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_linear_prompt_of_long_and_short_sequences(lens, dtype):
    R, B, H = sum(lens), len(lens), 2
    xs = ref.linear_inputs(100 + B, R, H, H, dtype, 0.02)
    S0 = ref.states(101, B, H)
    want_o, want_S = ref.packed(ref.linear_rows, S0, lens, *xs)
    S, o = S0.cuda(), torch.empty(R, H, D, device="cuda")
    work, guard = _guarded(kda.linear_workspace(R, B, H).numel())
    kda.kda_linear_prompt(kda.state_table(S.unsqueeze(0)), ref.offsets(lens).cuda(), *(x.cuda() for x in xs), o=o,
                          work=work)
    tol = ref.tolerance(max(lens))
    assert ref.relative(o, want_o) <= tol
    for b, n in enumerate(lens):
        if n:
            assert ref.relative(S[b], want_S[b]) <= tol, b
        else:
            assert torch.equal(S[b].cpu(), S0[b]), b
    assert bool((guard == 0x5A).all())


def test_linear_prompt_of_many_sequences_of_many_heads():
    # 64 GiB by one place for each sequence; 33 MiB by two for each 512 rows
    R, B, H = 513, 4096, 256
    n = kda.linear_workspace(R, B, H).numel()
    assert n < 1 << 26
    xs = [x.cuda() for x in ref.linear_inputs(102, R, 1, H, torch.bfloat16, 0.1)]
    off = torch.full((B + 1,), R, dtype=torch.int32)
    off[:2], off[2:7] = torch.tensor([0, 3]), torch.tensor([10, 11, 12, 400, 500])
    S = torch.zeros(6, H, D, D, device="cuda")
    ptrs = torch.zeros(B, dtype=torch.int64)
    ptrs[:6] = torch.tensor([S[i].data_ptr() for i in range(6)])
    o = torch.empty(R, H, D, device="cuda")
    kda.kda_linear_prompt(ptrs.cuda(), off.cuda(), *xs, o=o, work=torch.empty(n, dtype=torch.uint8, device="cuda"))
    edges = off.tolist()
    for b in range(6):
        alone = torch.zeros(1, H, D, D, device="cuda")
        part = [x[edges[b]:edges[b + 1]].contiguous() for x in xs]
        o1 = torch.empty(edges[b + 1] - edges[b], H, D, device="cuda")
        one = torch.tensor([0, o1.shape[0]], dtype=torch.int32, device="cuda")
        kda.kda_linear_prompt(kda.state_table(alone.unsqueeze(0)), one, *part, o=o1)
        assert torch.equal(alone[0], S[b]) and torch.equal(o[edges[b]:edges[b + 1]], o1), b
