"""Measured cases of the attention rows over a paged cache, of the cache's filling and of the sampled accept.

Three kinds of case:
  attn     attention of new rows (one token, a verify round, a prompt's chunk) over a paged cache,
           with or without a sliding window and first tokens that stay visible
  append   the new rows' keys and values, written to their places in the cache
  accept   drafted tokens verified against the target's probabilities from given random numbers

With `own` false, run() computes them in elementary torch operations in 32 bits (probabilities next to
a border in 64); with `own` true it calls the library.
"""
import math

import torch

own = False

D = 128


def listed():
    return [
        # the smallest call: one token of one session on one tensor-parallel rank's 8 heads
        {"name": "attn_step_1x8_bf16", "op": "attn", "news": "1", "lens": "300", "Hk": 1, "H": 8, "page": 16,
         "window": 0, "sinks": 0, "dtype": "bf16"},
        # a decode step of 15 sessions of mixed lengths, 8 query heads to a key head
        {"name": "attn_step_15x64_bf16", "op": "attn", "news": ",".join(["1"] * 15),
         "lens": "16384,1,777,4096,12000,64,2049,8191,513,16001,300,9000,5000,130,7003", "Hk": 8, "H": 64,
         "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # the 15 rows of one session's verify round behind a long document
        {"name": "attn_verify_15x64_bf16", "op": "attn", "news": "15", "lens": "65536", "Hk": 8, "H": 64,
         "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # verify rounds of 8 sessions in a layer with a window and 4 first tokens, a key head for each head
        {"name": "attn_verify_window_f32", "op": "attn", "news": "15,8,1,15,3,15,11,15",
         "lens": "9000,515,70,20000,3,4097,16000,1030", "Hk": 16, "H": 16, "page": 32, "window": 1024,
         "sinks": 4, "dtype": "f32"},
        # one user's prompt
        {"name": "attn_prompt_4096x64_bf16", "op": "attn", "news": "4096", "lens": "4096", "Hk": 8, "H": 64,
         "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # chunks of prompts (one of a single row) behind what is cached already, odd lengths and heads
        {"name": "attn_chunk_ragged_bf16", "op": "attn", "news": "512,1,777,130", "lens": "8192,300,2049,4000",
         "Hk": 4, "H": 12, "page": 128, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a verify round's keys and values of one session on one rank: latency
        {"name": "append_15x1_f32", "op": "append", "news": "15", "lens": "1000", "Hk": 1, "H": 8, "page": 16,
         "dtype": "f32"},
        # an admission batch
        {"name": "append_prompts_bf16", "op": "append", "news": "4096,1,777,0,2049,8192,513",
         "lens": "4096,300,1777,64,2049,8192,9000", "Hk": 8, "H": 64, "page": 64, "dtype": "bf16"},
        # one session's verify round of 14 drafts
        {"name": "accept_1x15x150000_f32", "op": "accept", "rows": "15", "V": 150000, "drafted": True,
         "masked": False, "temp": False, "dtype": "f32"},
        # verify rounds of 64 sessions, each with its temperature
        {"name": "accept_64x8x150000_bf16", "op": "accept", "rows": ",".join(["8"] * 64), "V": 150000,
         "drafted": True, "masked": False, "temp": True, "dtype": "bf16"},
        # a token for each of 15 sessions without drafts, under grammars that mask most of an odd vocabulary
        {"name": "accept_15x1x50001_bf16", "op": "accept", "rows": ",".join(["1"] * 15), "V": 50001,
         "drafted": False, "masked": True, "temp": True, "dtype": "bf16"},
        # drafts copied from the prompt (no draft probabilities), rounds of mixed lengths
        {"name": "accept_ragged_50001_f32", "op": "accept", "rows": "15,3,1,0,9,12,15,2", "V": 50001,
         "drafted": False, "masked": False, "temp": False, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "accept"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "accept":
        V = _log_int(rng, 1000, 200000)
        most = max(1, min(512, 512 * 150000 // V // (2 if dtype == "f32" else 1)))
        rows, left = [], _log_int(rng, 1, most)
        while left > 0 and len(rows) < 64:
            rows.append(min(left, rng.randint(1, 15)))
            left -= rows[-1]
        return {"op": op, "rows": ",".join(map(str, rows)), "V": V, "drafted": rng.random() < 0.5,
                "masked": rng.random() < 0.4, "temp": rng.random() < 0.5, "dtype": dtype}
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "Hk": Hk, "H": H, "page": rng.choice([16, 32, 64, 128, 256]), "dtype": dtype}
    if op == "append":
        B = rng.randint(1, 15)
        news = [_log_int(rng, 1, 16384 // B) for _ in range(B)]
        lens = [n + rng.randint(0, 2000) for n in news]
    else:
        kind = rng.choice(["step", "verify", "chunk"])
        B = rng.randint(1, 32 if kind == "step" else 15 if kind == "verify" else 5)
        most = 1 if kind == "step" else 15 if kind == "verify" else 4096
        top = _log_int(rng, 16, min(65536, 1500000 // (B * Hk)))
        most = max(1, min(most, top, 4096 * 64 * 4096 // (B * H * top) // (2 if dtype == "f32" else 1)))
        news = [_log_int(rng, 1, most) for _ in range(B)]
        lens = [_log_int(rng, n, max(n, top)) for n in news]
        windowed = rng.random() < 0.4
        case["window"] = _log_int(rng, 1, 4096) if windowed else 0
        case["sinks"] = rng.choice([0, 1, 4, 64]) if windowed else 0
    return {**case, "news": ",".join(map(str, news)), "lens": ",".join(map(str, lens))}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ends(lens):
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    state = {"case": dict(case)}
    if case["op"] == "accept":
        rows, V = _ints(case["rows"]), case["V"]
        R, B = sum(rows), len(rows)
        logits = normal(R, V).mul_(3.0)
        if case["masked"]:
            kept = torch.rand(R, V, generator=gen, device="cuda") < 0.2
            kept[:, 7 % V] = True
            logits.masked_fill_(~kept, -math.inf)
        # a drafter that is somewhat off the target draws the drafts
        probs = torch.softmax(logits + 0.7 * normal(R, V), 1)
        drafts = torch.multinomial(probs, 1, generator=gen)[:, 0]
        state["logits"] = logits.to(dt)
        state["drafts"] = drafts.to(torch.int32)
        state["probs"] = probs if case["drafted"] else None
        state["u"] = torch.rand(R, generator=gen, device="cuda")
        state["temp"] = 0.5 + torch.rand(B, generator=gen, device="cuda") if case["temp"] else None
        state["offsets"] = _ends(rows)
        state["p_draft"] = torch.zeros(R, device="cuda")
        state["out"] = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
        return state

    news, lens, page = _ints(case["news"]), _ints(case["lens"]), case["page"]
    R, B, H, Hk = sum(news), len(news), case["H"], case["Hk"]
    rows = normal(R, H + 2 * Hk, D).to(dt)   # what one projection of a layer gives
    state["q"], state["k"], state["v"] = rows.split([H, Hk, Hk], dim=1)
    used = [-(-n // page) for n in lens]
    free = torch.randperm(sum(used) + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = free[at:at + n]
        at += n
    state["table"] = table
    state["k_pages"], state["v_pages"] = (normal(sum(used) + 3, page, Hk, D).to(dt) for _ in range(2))
    state["offsets"] = _ends(news)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "attn":
        state["o"] = torch.empty(R, H, D, dtype=dt, device="cuda")
    return state


def _places(s):
    """For each new row its sequence, its number there and its position."""
    offsets, lens = s["offsets"].long(), s["lens"].long()
    news = offsets[1:] - offsets[:-1]
    row = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(offsets, row, right=True) - 1
    i = row - offsets[b]
    return b, i, lens[b] - news[b] + i


def _append_plain(s):
    b, _, p = _places(s)
    page = s["k_pages"].shape[1]
    at = s["table"][b, p // page].long(), p % page
    s["k_pages"][at] = s["k"]
    s["v_pages"][at] = s["v"]
    return s["k_pages"], s["v_pages"]


def _attn_plain(s):
    case = s["case"]
    H, Hk, page = case["H"], case["Hk"], case["page"]
    news, lens = _ints(case["news"]), _ints(case["lens"])
    B, n, L, G = len(news), max(news), max(lens), H // Hk
    b, i, p = _places(s)
    keys = torch.arange(L, device="cuda")
    pages = s["table"][:, keys // page].clamp(min=0).long()                         # [B][L]
    K = s["k_pages"][pages, keys % page].float().permute(0, 2, 3, 1)                # [B][Hk][D][L]
    V = s["v_pages"][pages, keys % page].float().transpose(1, 2)                    # [B][Hk][L][D]
    q = torch.zeros(B, n, H, D, device="cuda")
    at = torch.full((B, n), -1, dtype=torch.long, device="cuda")
    q[b, i], at[b, i] = s["q"].float(), p
    q = q.view(B, n, Hk, G, D).transpose(1, 2).reshape(B, Hk, n * G, D)
    seen = keys <= at[..., None]                                                    # [B][n][L]
    if case["window"]:
        seen &= (keys > at[..., None] - case["window"]) | (keys < case["sinks"])
    x = (q @ K).mul_(1.0 / math.sqrt(D)).view(B, Hk, n, G, L)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, n * G, L) @ V).view(B, Hk, n, G, D) / torch.where(z > 0, z, 1.0)
    s["o"].copy_(o.transpose(1, 2).reshape(B, n, H, D)[b, i])
    return s["o"]


def _accept_plain(s):
    offsets, x = s["offsets"].long(), s["logits"].float()
    R, V = x.shape
    rows = offsets[1:] - offsets[:-1]
    row = torch.arange(R, device="cuda")
    b = torch.searchsorted(offsets, row, right=True) - 1
    x = (x - x.amax(1, keepdim=True)).double()
    if s["temp"] is not None:
        x = x / s["temp"].double()[b, None]
    p = x.exp_()
    p /= p.sum(1, keepdim=True)
    drafts, u = s["drafts"].long()[:, None], s["u"].double()
    p_draft = p.gather(1, drafts)[:, 0]
    q_draft = 1.0 if s["probs"] is None else s["probs"].gather(1, drafts)[:, 0].double()
    last = row == offsets[b + 1] - 1
    stops = last | ~(u * q_draft < p_draft)
    first = torch.full_like(rows, R).scatter_reduce(0, b, torch.where(stops, row, R), "amin")
    some = rows > 0
    at = first[some]
    w, full = p[at], last[at]
    q = torch.zeros_like(w).scatter_(1, drafts[at], 2.0) if s["probs"] is None else s["probs"][at].double()
    left = (w - q).clamp(min=0.0)
    w = torch.where(full[:, None] | (left.sum(1, keepdim=True) <= 0), w, left)
    c = w.cumsum(1)
    token = (c <= u[offsets[1:][some] - 1][:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    s["out"][some] = torch.stack([at - offsets[:-1][some], token], 1).to(torch.int32)
    s["p_draft"].copy_(torch.where(last, 0.0, p_draft))
    return s["out"], s["p_draft"]


def _own(s):
    import gated_delta_rule_rows_amd as kda

    case, op = s["case"], s["case"]["op"]
    if op == "append":
        kda.kda_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["offsets"])
        return s["k_pages"], s["v_pages"]
    if op == "attn":
        if "work" not in s:
            s["work"] = kda.attn_workspace(s["q"].shape[0], s["lens"].shape[0], case["H"], case["Hk"])
        kda.kda_attn_rows(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["offsets"], s["o"],
                          window=case["window"], sinks=case["sinks"], work=s["work"])
        return s["o"]
    if "work" not in s:
        s["work"] = kda.accept_sampled_workspace(s["logits"].shape[0], s["out"].shape[0], s["logits"].shape[1])
    kda.kda_accept_sampled(s["logits"], s["offsets"], s["drafts"], s["u"], s["out"], probs=s["probs"],
                           temp=s["temp"], p_draft=s["p_draft"], work=s["work"])
    return s["out"], s["p_draft"]


def run(state):
    if own:
        return _own(state)
    return {"attn": _attn_plain, "append": _append_plain, "accept": _accept_plain}[state["case"]["op"]](state)


def _seen(case):
    """Of all sequences: the (row, key) pairs that see each other, and the keys that any row sees."""
    pairs = keys = 0
    W, S = case["window"], case["sinks"]
    for n, length in zip(_ints(case["news"]), _ints(case["lens"])):
        for p in range(length - n, length):
            pairs += p + 1 if not W or p < W else W + min(S, p + 1 - W)
        low = max(0, length - n - W + 1) if W else 0
        keys += length - low + min(S, low) if n else 0
    return pairs, keys


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "accept":
        rows, V = _ints(case["rows"]), case["V"]
        R, B = sum(rows), sum(n > 0 for n in rows)
        return {"bytes": R * (V * es + 12) + B * (V * 4 * case["drafted"] + 8), "flops": 4 * R * V}
    R = sum(_ints(case["news"]))
    if case["op"] == "append":
        return {"bytes": 4 * R * case["Hk"] * D * es, "flops": 0}
    pairs, keys = _seen(case)
    return {"bytes": 2 * R * case["H"] * D * es + 2 * keys * case["Hk"] * D * es,
            "flops": 4 * D * case["H"] * pairs}


def _exact_attn(s):
    case = s["case"]
    G, page, W, S = case["H"] // case["Hk"], case["page"], case["window"], case["sinks"]
    out, first = [], 0
    for b, (n, length) in enumerate(zip(_ints(case["news"]), _ints(case["lens"]))):
        j = torch.arange(length, device="cuda")
        p = torch.arange(length - n, length, device="cuda")[:, None]
        seen = j <= p
        if W:
            seen = seen & ((j > p - W) | (j < S))
        rows = [s["table"][b, j // page].long(), j % page]
        heads = []
        for h in range(case["H"]):
            K, V = (s[x][rows[0], rows[1], h // G].double() for x in ("k_pages", "v_pages"))
            x = s["q"][first:first + n, h].double() @ K.T.contiguous() / math.sqrt(128)
            heads.append(torch.softmax(x.masked_fill(~seen, -math.inf), 1) @ V)
        out.append(torch.stack(heads, 1))
        first += n
    return torch.cat(out)


def _exact_accept(s):
    out, got = [], s["p_draft"].double()
    first = 0
    for b, n in enumerate(_ints(s["case"]["rows"])):
        if n == 0:
            out.append([0, 0])
            continue
        x = s["logits"][first:first + n].double()
        if s["temp"] is not None:
            x = x / s["temp"][b].double()
        p = torch.softmax(x, 1)
        d, u = s["drafts"][first:first + n].tolist(), s["u"][first:first + n].double()
        j = n - 1
        for i in range(n - 1):
            got[first + i] = p[i, d[i]]
            q = 1.0 if s["probs"] is None else s["probs"][first + i, d[i]].double()
            if j == n - 1 and not u[i] * q < p[i, d[i]]:
                j = i
        w = p[j].clone()
        if j < n - 1 and s["probs"] is None:
            w[d[j]] = 0.0
        elif j < n - 1:
            w = (w - s["probs"][first + j].double()).clamp(min=0.0)
        if not w.sum() > 0:
            w = p[j]
        c = torch.cumsum(w, 0)
        out.append([j, int(torch.searchsorted(c, u[-1:] * c[-1], right=True).clamp(max=len(c) - 1))])
        first += n
    return torch.tensor(out, dtype=torch.int32, device="cuda"), got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "accept":
        return _exact_accept(s)
    first = 0
    for b, (n, length) in enumerate(zip(_ints(case["news"]), _ints(case["lens"]))):
        p = torch.arange(length - n, length, device="cuda")
        at = s["table"][b, p // case["page"]].long() * case["page"] + p % case["page"]
        for pages, rows in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
            pages.view(-1, *pages.shape[2:]).index_copy_(0, at, rows[first:first + n].contiguous())
        first += n
    return s["k_pages"], s["v_pages"]
