"""Verify rounds of a hybrid layer pair as a serving loop runs them, with nothing read back in between: the
new rows' keys and values into the paged cache, attention over it, the KDA rows of the fused round, the
sampled accept over logits of both outputs, and the rollback of both: the state by the accepted count on
the device, the cache by its length.  Two sessions; every round's outputs and the committed rows are checked
against plain forms in 64 bits and against the row scan."""
import math

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.cache_ref import D, accept_ref, attn_bound, attn_ref, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rounds_with_rollback(dt):
    B, T, H, Hk, HS, V, rounds, page = 2, 6, 4, 2, 2, 700, 4, 16
    gen = torch.Generator().manual_seed(31)
    start = [37, 5]                                     # rows cached before
    k_pages, v_pages, table = make_cache(gen, [n + rounds * T for n in start], page, Hk, dt)
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    head = (torch.randn(H * D + HS * D, V, generator=gen) * 0.2).cuda()
    attn_work = kda.attn_workspace(B * T, B, H, Hk)
    accept_work = kda.accept_sampled_workspace(B * T, B, V)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    snap = [torch.randn(1, HS, D, D, generator=gen).mul_(0.1).cuda() for _ in range(B)]
    first_state = [s.clone() for s in snap]
    prev, out_prev = [None] * B, None
    log = []
    for r in range(rounds):
        rows = torch.randn(B * T, H + 2 * Hk, D, generator=gen).to(dt).cuda()
        q, k, v = rows.split([H, Hk, Hk], dim=1)
        lens += T                                       # the round's rows, drafts among them
        kda.kda_cache_append(k, v, k_pages, v_pages, table, lens, ends)
        o = torch.empty(B * T, H, D, dtype=dt, device="cuda")
        kda.kda_attn_rows(q, k_pages, v_pages, table, lens, ends, o, work=attn_work)
        states, o_kda, ins = [], [], []
        for b in range(B):
            x = [unit(torch.randn(1, T, HS, D, generator=gen)).cuda(), unit(torch.randn(1, T, HS, D, generator=gen)).cuda(),
                 torch.randn(1, T, HS, D, generator=gen).cuda(), -torch.rand(1, T, HS, D, generator=gen).cuda(),
                 torch.rand(1, T, HS, generator=gen).cuda()]
            nxt, ok, e = torch.empty_like(snap[b]), torch.empty(1, T, HS, D, device="cuda"), torch.empty(1, T, HS, D, device="cuda")
            keep = 0 if prev[b] is None else out_prev[b]
            kda.kda_verify_round(snap[b], nxt, prev[b], keep, *x, ok, e=e)
            prev[b] = (x[1], None, x[3], None, e)
            states.append(nxt)
            o_kda.append(ok[0].reshape(T, HS * D))
            ins.append(x)
        logits = torch.cat([o.float().reshape(B * T, -1), torch.cat(o_kda)], 1) @ head
        probs = torch.softmax(logits + torch.randn(B * T, V, generator=gen).cuda(), 1)
        drafts = torch.multinomial(probs.cpu(), 1, generator=gen)[:, 0].to(torch.int32).cuda()
        u = torch.rand(B * T, generator=gen).cuda()
        out = torch.empty(B, 2, dtype=torch.int32, device="cuda")
        kda.kda_accept_sampled(logits.to(dt), ends, drafts, u, out, probs=probs, work=accept_work)
        log.append((q.clone(), k.clone(), v.clone(), o, lens.clone(), ins, states, logits.to(dt), drafts, u, probs, out))
        lens -= T - 1 - out[:, 0]                       # the rollback of the cache: keep = j + 1 rows
        snap, out_prev = states, out
    torch.cuda.synchronize()

    # the same by plain forms: the committed rows only
    kept_len, committed = list(start), [first_state[b].clone() for b in range(B)]
    fresh_k, fresh_v = k_pages.clone(), v_pages.clone()
    for b in range(B):                                  # behind the rows cached before: from the log
        for j in range(start[b], table.shape[1] * page):
            entry = int(table[b, j // page])
            if entry >= 0:
                fresh_k[entry, j % page] = math.nan
                fresh_v[entry, j % page] = math.nan
    some, all_kept = False, True
    for q, k, v, o, lens_r, ins, states, logits, drafts, u, probs, out in log:
        assert lens_r.tolist() == [n + T for n in kept_len]
        for b in range(B):
            for i in range(T):
                p = kept_len[b] + i
                fresh_k[int(table[b, p // page]), p % page] = k[b * T + i]
                fresh_v[int(table[b, p // page]), p % page] = v[b * T + i]
        want, size, count, dot = attn_ref(q, fresh_k, fresh_v, table, lens_r.tolist(), [0, T, 2 * T], o, 1 / math.sqrt(D))
        assert ((o.double().cpu() - want).abs() <= attn_bound(want, size, count, dot, dt)).all()
        ref, _, _ = accept_ref(logits, [0, T, 2 * T], drafts, u, probs)
        assert [tuple(x) for x in out.tolist()] == ref
        for b in range(B):
            assert torch.equal(states[b], committed[b])     # the round's snapshot: the rows kept so far
            keep = ref[b][0] + 1
            some, all_kept = some or keep > 1, all_kept and keep == T
            step = torch.empty_like(committed[b])
            kda.kda_scan_rows(committed[b], step, *[x[:, :keep].contiguous() for x in ins[b]])
            committed[b] = step
            kept_len[b] += keep
    assert some and not all_kept                            # drafts were accepted, and others not
