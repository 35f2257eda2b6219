"""Measured cases of the prompt, single-token and log-probability operators.

Four kinds of case:
  linear_prompt  linear attention with one decay for each head, prompts packed row after row
  linear_step    the same layers, one token of each session, states updated in place
  kda_prompt     the KDA delta rule over packed prompts, states updated in place
  logprobs       log probabilities of given tokens, entropy and top alternatives of logits rows

With `own` false, run() computes them in elementary torch operations in 32 bits; with `own`
true it calls the library.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
GATE_LO = -5.0
NO_TOKEN = -1   # the library's 0xFFFFFFFF, read as int32


def listed():
    return [
        # one user's prompt through a layer of 64 heads
        {"name": "linear_prompt_4096x64_bf16", "op": "linear_prompt", "lens": "4096", "Hk": 64, "H": 64,
         "dtype": "bf16"},
        # an admission batch: prompts of mixed lengths (one of a single row, one empty), 4 value
        # heads to a key head
        {"name": "linear_prompt_ragged_bf16", "op": "linear_prompt", "lens": "1,777,0,64,2049,130,513",
         "Hk": 8, "H": 32, "dtype": "bf16"},
        # a long document on one tensor-parallel rank's share of 8 heads, f32 projections
        {"name": "linear_prompt_16384x8_f32", "op": "linear_prompt", "lens": "16384", "Hk": 8, "H": 8,
         "dtype": "f32"},
        # the smallest call: one session, one layer, one rank's 8 heads
        {"name": "linear_step_1x1x8_f32", "op": "linear_step", "L": 1, "B": 1, "Hk": 8, "H": 8, "dtype": "f32"},
        # a decode step of 15 sessions over 34 layers of 64 heads
        {"name": "linear_step_34x15x64_bf16", "op": "linear_step", "L": 34, "B": 15, "Hk": 16, "H": 64,
         "dtype": "bf16"},
        # one user's prompt through a KDA layer of 64 heads
        {"name": "kda_prompt_4096x64_bf16", "op": "kda_prompt", "lens": "4096", "H": 64, "dtype": "bf16"},
        # an admission batch, f32 projections (what the row ops give)
        {"name": "kda_prompt_ragged_f32", "op": "kda_prompt", "lens": "300,1,95,1500,0,33,640,17", "H": 32,
         "dtype": "f32"},
        # a long document on one tensor-parallel rank's share of 8 heads
        {"name": "kda_prompt_8192x8_bf16", "op": "kda_prompt", "lens": "8192", "H": 8, "dtype": "bf16"},
        # a short turn appended to a session: latency counts
        {"name": "kda_prompt_45x8_f32", "op": "kda_prompt", "lens": "45", "H": 8, "dtype": "f32"},
        # one verify round's 15 rows of a 150,000-entry vocabulary
        {"name": "logprobs_15x150000_f32", "op": "logprobs", "t": 15, "V": 150000, "n": 20, "masked": False,
         "dtype": "f32"},
        # one sampled token under a grammar that masks most of an odd vocabulary
        {"name": "logprobs_1x50001_bf16", "op": "logprobs", "t": 1, "V": 50001, "n": 5, "masked": True,
         "dtype": "bf16"},
        # scoring the rows of a prompt
        {"name": "logprobs_2048x150000_bf16", "op": "logprobs", "t": 2048, "V": 150000, "n": 8, "masked": False,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _lens(rng, total):
    lens, left = [], total
    for _ in range(rng.randint(1, 9)):
        if left <= 0:
            break
        n = _log_int(rng, 1, left)
        lens.append(n)
        left -= n
    if rng.random() < 0.3:
        lens.insert(rng.randint(0, len(lens)), 0)
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["linear_prompt", "linear_step", "kda_prompt", "logprobs"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "logprobs":
        V = _log_int(rng, 1000, 200000)
        t = _log_int(rng, 1, max(1, min(2048, 2048 * 150000 // V // (2 if dtype == "f32" else 1))))
        return {"op": op, "t": t, "V": V, "n": rng.randint(0, 32), "masked": rng.random() < 0.4, "dtype": dtype}
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    H = Hk * rng.choice([1, 2, 3, 4])
    if op == "linear_step":
        L = rng.randint(1, 34)
        B = _log_int(rng, 1, max(1, min(96, 34 * 15 * 64 // (L * H))))
        return {"op": op, "L": L, "B": B, "Hk": Hk, "H": H, "dtype": dtype}
    rows = _log_int(rng, 1, min(16384 if op == "linear_prompt" else 8192, 4096 * 64 // H // (2 if dtype == "f32" else 1)))
    case = {"op": op, "lens": _lens(rng, rows), "H": H, "dtype": dtype}
    if op == "linear_prompt":
        case["Hk"] = Hk
    return case


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    if case["op"] == "logprobs":
        t, V = case["t"], case["V"]
        logits = normal(t, V).mul_(3.0)
        if case["masked"]:
            kept = torch.rand(t, V, generator=gen, device="cuda") < 0.2
            kept[:, 7 % V] = True
            logits.masked_fill_(~kept, -math.inf)
        tokens = torch.randint(0, V, (t,), generator=gen, device="cuda", dtype=torch.int32)
        f = dict(dtype=torch.float32, device="cuda")
        return {"case": dict(case), "logits": logits.to(dt), "tokens": tokens, "lp": torch.empty(t, **f),
                "entropy": torch.empty(t, **f), "top_lp": torch.empty(t, case["n"], **f),
                "top_ids": torch.empty(t, case["n"], dtype=torch.int32, device="cuda")}

    H = case["H"]
    if case["op"] == "linear_step":
        L, B, Hk = case["L"], case["B"], case["Hk"]
        lead, n_states = (L, B), L * B
    else:
        lens = _lengths(case)
        R, B, Hk = sum(lens), len(lens), case.get("Hk", H)
        lead, n_states = (R,), B
    state = {"case": dict(case)}
    state["S"] = normal(n_states, H, D, D).mul_(0.1)
    base = state["S"].data_ptr()
    state["s_ptrs"] = torch.tensor([base + i * H * D * D * 4 for i in range(n_states)], dtype=torch.int64,
                                   device="cuda")
    state["q"], state["k"] = unit(*lead, Hk, D), unit(*lead, Hk, D)
    state["v"] = normal(*lead, H, D).to(dt)
    state["o"] = torch.empty(*lead, H, D, device="cuda")
    if case["op"] == "kda_prompt":
        state["g"] = (-torch.nn.functional.softplus(2.0 * normal(*lead, H, D))).clamp_(GATE_LO, 0.0).to(dt)
        state["beta"] = torch.sigmoid(normal(*lead, H)).to(dt)
    else:
        # a slope for each head, from slow to fast, times a gate of each row
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
        state["g"] = -slope * torch.nn.functional.softplus(normal(*lead, H))
    if case["op"] != "linear_step":
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        state["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    return state


def _chunks_of(lens, chunk):
    """Row numbers [N][chunk] of the chunks of all sequences, which of them exist, the sequences
    from longest to shortest, and how many of those still have rows at each step.  The chunks of
    one step lie together, in the sequences' order."""
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    length = torch.tensor(lens, device="cuda")
    first = (torch.cumsum(length, 0) - length)[order]
    at = torch.arange(-(-max(lens) // chunk) * chunk, device="cuda").view(-1, 1, chunk)
    there = at < length[order][:, None]                       # [steps][B][chunk]
    rows = torch.where(there, first[:, None] + at, 0)
    some = there[..., 0]
    alive = [sum(n > i * chunk for n in lens) for i in range(at.shape[0])]
    return rows[some], there[some], torch.tensor(order, device="cuda"), alive


def _gather(x, rows, there):
    """Packed [R][H][...] to [N][H][C][...] in 32 bits, zero where no row is."""
    y = x[rows].float()
    return (y * there.view(*there.shape, *([1] * (y.dim() - 2)))).transpose(1, 2)


def _linear_prompt_plain(s):
    case = s["case"]
    H, Hk, C = case["H"], case["Hk"], 64
    rows, there, order, alive = _chunks_of(_lengths(case), C)
    q, k, v, g = (_gather(s[n], rows, there) for n in ("q", "k", "v", "g"))
    q, k = (x.repeat_interleave(H // Hk, dim=1) for x in (q, k))                    # [N][H][C][D]
    G = g.clamp(max=0.0).double().cumsum(2)                                         # [N][H][C]
    tri = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(tri, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    o = ((q @ k.transpose(-1, -2)) * decay) @ v
    q_in = q * G.exp().float()[..., None]
    k_out = k * (G[..., -1:] - G).exp().float()[..., None]
    added = k_out.transpose(-1, -2) @ v                                             # [N][H][D][D]
    kept = G[..., -1].exp().float()[..., None, None]
    S, n = s["S"][order], 0
    for a in alive:
        o[n:n + a] += q_in[n:n + a] @ S[:a]
        S[:a] = kept[n:n + a] * S[:a] + added[n:n + a]
        n += a
    s["o"][rows[there]] = (o * SCALE).transpose(1, 2)[there]
    s["S"][order] = S
    return s["o"], s["S"]


def _linear_step_plain(s):
    case = s["case"]
    H, Hk = case["H"], case["Hk"]
    q, k = (s[n].float().repeat_interleave(H // Hk, dim=2) for n in ("q", "k"))
    S = s["S"].view(case["L"], case["B"], H, D, D)
    S.mul_(s["g"].clamp(max=0.0).exp()[..., None, None]).add_(k[..., :, None] * s["v"].float()[..., None, :])
    torch.mul((q[..., None, :] @ S)[..., 0, :], SCALE, out=s["o"])
    return s["o"], s["S"]


def _kda_prompt_plain(s):
    case, C = s["case"], 16
    rows, there, order, alive = _chunks_of(_lengths(case), C)
    q, k, v, g, beta = (_gather(s[n], rows, there) for n in ("q", "k", "v", "g", "beta"))
    G = g.clamp(GATE_LO, 0.0).double().cumsum(2)                                    # [N][H][C][D]
    tri = torch.ones(C, C, device="cuda").tril()
    between = k[..., None, :, :] * (G[..., :, None, :] - G[..., None, :, :]).clamp(max=0.0).exp().float()
    A = (k[..., :, None, :] * between).sum(-1) * tri.tril(-1)
    P = (q[..., :, None, :] * between).sum(-1) * tri
    del between
    X = -beta[..., None] * A
    eye = torch.eye(C, device="cuda")
    X2 = X @ X
    X4 = X2 @ X2
    M = (eye + X) @ (eye + X2) @ (eye + X4) @ (eye + X4 @ X4) * beta[..., None, :]
    q_in, k_in = q * G.exp().float(), k * G.exp().float()
    k_out = (k * (G[..., -1:, :] - G).exp().float()).transpose(-1, -2)
    kept = G[..., -1, :].exp().float()[..., None]
    S, o, n = s["S"][order], torch.empty_like(v), 0
    for a in alive:
        m = slice(n, n + a)
        E = M[m] @ (v[m] - k_in[m] @ S[:a])
        o[m] = q_in[m] @ S[:a] + P[m] @ E
        S[:a] = kept[m] * S[:a] + k_out[m] @ E
        n += a
    s["o"][rows[there]] = (o * SCALE).transpose(1, 2)[there]
    s["S"][order] = S
    return s["o"], s["S"]


def _logprobs_plain(s):
    x, n, V = s["logits"].float(), s["case"]["n"], s["case"]["V"]
    m = x.max(dim=1, keepdim=True).values
    y = x - m
    p = y.exp()
    z = p.sum(1, keepdim=True)
    log_z = z.log()
    lp = (y.gather(1, s["tokens"].long()[:, None]) - log_z)[:, 0]
    entropy = (log_z - torch.where(p > 0, p * y, 0.0).sum(1, keepdim=True) / z)[:, 0]
    del p
    bits = (x + 0.0).view(torch.int32)   # x + 0: one zero
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (key << 32) + torch.arange(V - 1, -1, -1, device="cuda")
    ids = V - 1 - (key.topk(n, dim=1).values & 0xFFFFFFFF)
    top_lp = y.gather(1, ids) - log_z
    ids = torch.where(top_lp == -math.inf, NO_TOKEN, ids)
    return lp, entropy, ids.to(torch.int32), top_lp


def _own(s):
    import gated_delta_rule_rows_amd as kda

    case, op = s["case"], s["case"]["op"]
    if op == "logprobs":
        if "work" not in s:
            s["work"] = kda.logprobs_workspace(case["t"], case["V"], case["n"])
        kda.kda_logprobs(s["logits"], s["tokens"], s["lp"], s["entropy"], s["top_ids"], s["top_lp"], s["work"])
        return s["lp"], s["entropy"], s["top_ids"], s["top_lp"]
    if op == "linear_step":
        kda.kda_linear_step(s["s_ptrs"], s["q"], s["k"], s["v"], s["g"], s["o"])
        return s["o"], s["S"]
    R, B, H = s["o"].shape[0], s["S"].shape[0], case["H"]
    if op == "linear_prompt":
        if "work" not in s:
            s["work"] = kda.linear_workspace(R, B, H)
        kda.kda_linear_prompt(s["s_ptrs"], s["offsets"], s["q"], s["k"], s["v"], s["g"], s["o"], s["work"])
    else:
        if "work" not in s:
            s["work"] = kda.prompt_workspace(R, B, H)
        kda.kda_prompt(s["s_ptrs"], s["offsets"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["work"])
    return s["o"], s["S"]


def run(state):
    if own:
        return _own(state)
    return {"linear_prompt": _linear_prompt_plain, "linear_step": _linear_step_plain,
            "kda_prompt": _kda_prompt_plain, "logprobs": _logprobs_plain}[state["case"]["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        t, V, n = case["t"], case["V"], case["n"]
        return {"bytes": t * V * es + t * (4 + 8 + 8 * n), "flops": 6 * t * V}
    H = case["H"]
    if case["op"] == "kda_prompt":
        rows, states, Hk = sum(_lengths(case)) * H, sum(n > 0 for n in _lengths(case)) * H, H
        gates, flops = (D + 1) * es, 7 * D * D
    else:
        one = case["op"] == "linear_step"
        n = case["L"] * case["B"] if one else sum(_lengths(case))
        rows, Hk = n * H, case["Hk"]
        states = rows if one else sum(n > 0 for n in _lengths(case)) * H
        gates, flops = 4, 5 * D * D
    return {"bytes": rows * (D * es + D * 4 + gates) + 2 * rows * Hk // H * D * es + 8 * states * D * D,
            "flops": rows * flops}


def _exact_rows(S, q, k, v, decay, beta, there):
    """The recurrence row by row in 64 bits over padded rows [B][T][H][..]; decay [B][T][H][D or 1]."""
    o = torch.zeros_like(v)
    for t in range(q.shape[1]):
        kt, vt = k[:, t], v[:, t]
        new = S * decay[:, t, :, :, None]
        e = vt if beta is None else beta[:, t, :, None] * (vt - (new * kt[..., None]).sum(2))
        new = new + kt[..., None] * e[:, :, None, :]
        S = torch.where(there[:, t, None, None, None], new, S)
        o[:, t] = (new * q[:, t][..., None]).sum(2)
    return o / math.sqrt(128), S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        lp, entropy, ids, top = [], [], [], []
        for x, token in zip(s["logits"].split(256), s["tokens"].split(256)):
            x = x.double()
            logp = x - torch.logsumexp(x, 1, keepdim=True)
            p = torch.softmax(x, 1)
            lp.append(logp.gather(1, token.long()[:, None])[:, 0])
            entropy.append(-torch.xlogy(p, p).sum(1))
            order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["n"]]
            best = logp.gather(1, order)
            top.append(best)
            ids.append(torch.where(best == -math.inf, NO_TOKEN, order).to(torch.int32))
        return torch.cat(lp), torch.cat(entropy), torch.cat(ids), torch.cat(top)
    H = case["H"]
    if case["op"] == "linear_step":
        pack = {n: s[n].reshape(-1, 1, *s[n].shape[2:]).double() for n in ("q", "k", "v", "g")}
        q, k = (pack[n].repeat_interleave(H // case["Hk"], dim=2) for n in ("q", "k"))
        there = torch.ones(q.shape[0], 1, dtype=torch.bool, device="cuda")
        os, Ss = [], []
        for at in torch.arange(q.shape[0], device="cuda").split(64):
            o, S = _exact_rows(s["S"][at].double(), q[at], k[at], pack["v"][at],
                               torch.exp(pack["g"][at].clamp(max=0.0))[..., None], None, there[at])
            os.append(o)
            Ss.append(S)
        return torch.cat(os).view(s["o"].shape), torch.cat(Ss)
    lens = _lengths(case)
    first = 0
    T = max(lens)
    there = torch.zeros(len(lens), T, dtype=torch.bool, device="cuda")
    pack = {n: torch.zeros(len(lens), T, *s[n].shape[1:], dtype=torch.float64, device="cuda")
            for n in ("q", "k", "v", "g", "beta") if n in s}
    for b, n in enumerate(lens):
        there[b, :n] = True
        for x in pack:
            pack[x][b, :n] = s[x][first:first + n].double()
        first += n
    if case["op"] == "linear_prompt":
        pack["q"], pack["k"] = (pack[n].repeat_interleave(H // case["Hk"], dim=2) for n in ("q", "k"))
        decay = torch.exp(pack["g"].clamp(max=0.0))[..., None]
    else:
        decay = torch.exp(pack["g"].clamp(GATE_LO, 0.0))
    o, S = _exact_rows(s["S"].double(), pack["q"], pack["k"], pack["v"], decay, pack.get("beta"), there)
    return o[there], S
