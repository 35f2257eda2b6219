"""Plain forms in 64 bits of the paged cache's attention and of the sampled accept, written from their
definitions, and the inputs of their tests."""
import math

import torch

D = 128


def make_cache(gen, lens, page, Hk, dt, layout="rows", spare=3, device="cuda"):
    """k_pages and v_pages of random values, their table (a random order of the pages, -1 behind a
    sequence's last), with room for each length."""
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    x = torch.randn(2, pages, page, Hk, D, generator=gen).to(dt).to(device)
    if layout == "rows":           # [page][row][head]
        k, v = x[0].contiguous(), x[1].contiguous()
    elif layout == "heads":        # [page][head][row]
        k, v = (y.transpose(1, 2).contiguous().transpose(1, 2) for y in x)
    elif layout == "pages":        # keys and values in one buffer, page by page
        both = x.transpose(0, 1).contiguous()
        k, v = both[:, 0], both[:, 1]
    else:                          # row by row
        both = x.permute(1, 2, 0, 3, 4).contiguous()
        k, v = both[:, :, 0], both[:, :, 1]
    return k, v, table.to(device)


def seen_keys(p, length_cap, page, entries, pages, window, sinks):
    """The positions that a row at position p sees."""
    got = []
    for j in range(min(p + 1, length_cap)):
        if not 0 <= entries[j // page] < pages:
            continue
        if window == 0 or j > p - window or j < sinks:
            got.append(j)
    return got


def attn_ref(q, k_pages, v_pages, table, lens, offsets, o, scale, window=0, sinks=0):
    """o (64 bits, starting from the o given) and, for each value, the sum of |weight * value|, the
    number of keys and the largest sum of |q k| times the scale."""
    R, H, _ = q.shape
    pages, page, Hk, _ = k_pages.shape
    k64, v64, q64 = k_pages.double().cpu(), v_pages.double().cpu(), q.double().cpu()
    out = o.double().cpu().clone()
    size = torch.zeros(R, H, D, dtype=torch.float64)
    count = torch.zeros(R, dtype=torch.float64)
    dot = torch.zeros(R, H, dtype=torch.float64)
    upto = 0
    for b in range(len(lens)):
        first = max(upto, min(max(offsets[b], 0), R))
        last = min(max(offsets[b + 1], first), R)
        upto = first
        entries = table[b].tolist()
        for r in range(first, last):
            p = max(lens[b], 0) - (last - r)
            j = seen_keys(p, len(entries) * page, page, entries, pages, window, sinks)
            count[r] = len(j)
            if not j:
                out[r] = 0.0
                continue
            at = torch.tensor([entries[x // page] for x in j]), torch.tensor([x % page for x in j])
            K = k64[at].repeat_interleave(H // Hk, dim=1)      # [keys][H][D]
            V = v64[at].repeat_interleave(H // Hk, dim=1)
            x = (K * q64[r]).sum(-1) * scale                   # [keys][H]
            w = torch.softmax(x, 0)
            out[r] = (w[..., None] * V).sum(0)
            size[r] = (w[..., None] * V.abs()).sum(0)
            dot[r] = (K.abs() * q64[r].abs()).sum(-1).amax(0) * scale
    return out, size, count, dot


def attn_bound(out, size, count, dot, dt):
    """How far a result may be off.  A score's 128 products and their sums are off by 130 half steps of
    f32 (2^-24) of the sum of |q k| at most, times 1.5 for the scale and the conversion to base 2, whose
    products are rounded too; the weight's exponential by 4 half steps more; both sides of the quotient
    carry that (2x), and the sums over the keys a half step a key and of each of up to 64 moves to a new maximum.
    bf16: each weight is off by half a step of 2^-8 and the result by another."""
    h = 2.0 ** -24
    rel = 2 * (195 * h * dot[..., None] + 4 * h) + 2 * (count[:, None, None] + 64) * h
    err = rel * size + 4 * h * out.abs() + 1e-30
    if dt == torch.bfloat16:
        err = err + 2.0 ** -8 * size
        err = err + 2.0 ** -8 * (out.abs() + err)
    return err


def accept_ref(logits, offsets, drafts, u, probs=None, temp=None):
    """[(j, token) or None], p_draft ({row: p}) and the running sums that decided, in 64 bits."""
    R, V = logits.shape
    x64 = logits.double().cpu()
    out, p_draft, margin = [], {}, []
    upto = 0
    for b in range(len(offsets) - 1):
        first = max(upto, min(max(offsets[b], 0), R))
        last = min(max(offsets[b + 1], first), R)
        upto = first
        n = last - first
        if n == 0:
            out.append(None)
            margin.append(math.inf)
            continue
        t = 1.0 if temp is None else float(temp[b])
        good_t = t >= 1e-30 and math.isfinite(t)
        ps = []
        for r in range(first, last):
            x = x64[r]
            m = x.max()
            if not good_t or torch.isnan(x).any() or m == math.inf or m == -math.inf:
                ps.append(None)
            else:
                e = torch.exp((x - m) / t)
                ps.append(e / e.sum())
        gap = math.inf
        j = n - 1
        for i in range(n - 1):
            d = int(drafts[first + i]) & 0xFFFFFFFF
            p = math.nan if ps[i] is None else float(ps[i][d]) if d < V else 0.0
            p_draft[first + i] = p
            q = 1.0 if probs is None or d >= V else float(probs[first + i, d])
            if j == n - 1:
                if not math.isnan(p):
                    gap = min(gap, abs(float(u[first + i]) * q - p))
                if not float(u[first + i]) * q < p:
                    j = i
        if not good_t:
            j = 0
        p = ps[j]
        if p is None:
            out.append((j, 0xFFFFFFFF))
            margin.append(gap)
            continue
        w = p
        if j < n - 1:
            d = int(drafts[first + j]) & 0xFFFFFFFF
            if probs is None:
                w = p.clone()
                if d < V:
                    w[d] = 0.0
            else:
                w = (p - probs[first + j].double().cpu()).clamp(min=0.0)
            if not w.sum() > 0:
                w = p
        c = torch.cumsum(w, 0)
        place = float(u[last - 1]) * c[-1]
        hit = ((c > place) & (w > 0)).nonzero()
        token = int(hit[0]) if len(hit) else int((w > 0).nonzero()[-1])
        out.append((j, token))
        margin.append(min(gap, float((c - place).abs().min() / c[-1])))
    return out, p_draft, margin
