"""The operators on a paged key/value cache, case by case: what is run, on what inputs, and what each has to read, write and compute.

A cache holds the K and V rows of B sequences in pages: ``k_pages`` and ``v_pages`` are
[pages, page, Hkv, d], and entry i of a sequence's row of ``page_table`` names the page with its
slots [i * page, (i + 1) * page).  ``seq_lens`` counts a sequence's cached tokens, the new ones of
the call among them; the new tokens of all sequences are packed, ``cu`` holding the offsets.

    append  the new tokens' K (turned by RoPE) and V go into their slots;
    attend  the new tokens attend to the cached ones, causally, query heads in groups;
    weigh   the same, and what each cached token received is added to its running weight;
    evict   the tokens of the largest weights are kept, in order, on other pages.

``own`` chooses between the plain forms here and the framework's own calls.
"""

import math
import random

import torch

own = False

THETA = 500000.0
KINDS = ("append", "attend", "weigh", "evict")


# ------------------------------------------------------------------ cases
def case_of(name, kind, B, new, old, Hq, Hkv, d, page, shape, **more):
    """new, old: the range of a sequence's new and earlier tokens; shape: which lengths in it."""
    c = dict(kind=kind, B=B, new_lo=new[0], new_hi=new[1], old_lo=old[0], old_hi=old[1], Hq=Hq, Hkv=Hkv, d=d,
             page=page, shape=shape)
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a step of decoding for 64 requests: one row each, where the call itself is what costs
        case_of("append_step", "append", 64, (1, 1), (255, 8191), 32, 8, 128, 16, 1),
        # the keys and values of a whole 32K prompt
        case_of("append_prompt_32k", "append", 1, (32768, 32768), (0, 0), 32, 8, 128, 64, 2),
        # one request's next token early in its answer, in a small model: latency
        case_of("attend_one", "attend", 1, (1, 1), (516, 516), 8, 2, 128, 16, 3, lse=False),
        # a step of decoding for 64 requests of very different lengths
        case_of("attend_step_64", "attend", 64, (1, 1), (255, 16383), 32, 8, 128, 16, 4, lse=False),
        # one request's next token after a 128K prompt: a long axis and few rows
        case_of("attend_step_128k", "attend", 1, (1, 1), (131071, 131071), 32, 8, 128, 64, 5, lse=False),
        # the last part of a 32K prompt that is fed in parts
        case_of("attend_chunk_32k", "attend", 1, (2048, 2048), (30720, 30720), 32, 8, 128, 64, 6, lse=False),
        # a batch that mixes decoding with parts of prompts: ragged, seven heads to a group, narrow heads
        case_of("attend_mixed", "attend", 12, (1, 509), (0, 6001), 28, 4, 64, 32, 7, lse=True),
        # a whole 8K prompt: nothing was cached before
        case_of("attend_prompt_8k", "attend", 1, (8192, 8192), (0, 0), 32, 8, 128, 64, 8, lse=False),
        # a step of decoding that keeps account of what each head looked at
        case_of("weigh_step_16", "weigh", 16, (1, 1), (1023, 8191), 32, 8, 128, 16, 9, each=True),
        # the last 250 tokens of a 32K prompt weigh all the others, over all heads
        case_of("weigh_chunk_32k", "weigh", 1, (250, 250), (32518, 32518), 32, 8, 128, 64, 10, each=False),
        # after a 32K prompt: three tenths of its tokens stay, the last 64 among them
        case_of("evict_prompt_32k", "evict", 1, (0, 0), (32768, 32768), 32, 8, 128, 64, 11, each=False, keep=9830,
                sink=0, recent=64),
        # between steps of decoding, a budget for each head's own choice; some requests are still below it
        case_of("evict_heads_16", "evict", 16, (0, 0), (1500, 8200), 32, 8, 128, 16, 12, each=True, keep=2048, sink=4,
                recent=256),
    ]


def between(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2))) - 1)))


def draw(rng):
    kind = rng.choice(KINDS + ("attend", "weigh"))
    Hkv = rng.choice((1, 2, 4, 8))
    heads = dict(Hq=Hkv * rng.choice((1, 2, 4, 4, 5, 7, 8)), Hkv=Hkv, d=rng.choice((64, 128, 128)),
                 page=rng.choice((16, 32, 64, 128)), shape=rng.randrange(1 << 20))
    if kind == "append":
        B = between(rng, 1, 64)
        hi = between(rng, 1, 32768 // B)
        return case_of("", kind, B, (rng.choice((0, 1, hi)), hi), (0, between(rng, 1, 8192)), **heads)
    if kind == "evict":
        B = between(rng, 1, 32)
        hi = between(rng, 40, 32768 if B == 1 else 131072 // B)
        keep = max(8, int(hi * rng.uniform(0.1, 0.9)))
        return case_of("", kind, B, (0, 0), (hi // rng.randint(1, 9), hi), **heads, each=rng.random() < 0.5, keep=keep,
                       sink=rng.randint(0, 4), recent=between(rng, 0, keep - 4))
    # new tokens: one each, a few each, or parts of prompts; scores of all pairs stay below 2^31
    B = between(rng, 1, 64)
    new = between(rng, 1, rng.choice((1, 8, 2048)))
    most = max(64, min(131072 // B, (1 << 31) // (heads["Hq"] * B * new) - new))
    old = between(rng, 0, most)
    new_lo = rng.choice((0, 1, new))
    extra = dict(lse=rng.random() < 0.3) if kind == "attend" else dict(each=rng.random() < 0.5)
    return case_of("", kind, B, (new_lo, new), (rng.choice((0, old // 8, old)), old), **heads, **extra)


def lengths(case):
    """New and earlier tokens of each sequence; the first has the most of both."""
    r = random.Random(case["shape"])
    new = [between(r, case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    old = [between(r, case["old_lo"], case["old_hi"]) for _ in range(case["B"])]
    new[0], old[0] = case["new_hi"], case["old_hi"]
    return new, old


def work(case):
    new, old = lengths(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    row = Hkv * d * 2  # bytes of one token's K, or V
    T = sum(new)
    if case["kind"] == "append":
        return {"bytes": 4 * row * T + 4 * T, "flops": 3 * Hkv * d * T}
    if case["kind"] == "evict":
        kept = sum(min(n, case["keep"]) for n in old)
        heads = Hkv if case["each"] else 1
        return {"bytes": 4 * row * kept + 4 * heads * (sum(old) + 2 * kept), "flops": heads * sum(old)}
    cached = sum(n + o for n, o in zip(new, old) if n)
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    moved = 2 * row * cached + 4 * Hq * d * T + (4 * Hq * T if case.get("lse") else 0)
    if case["kind"] == "weigh":
        moved += 8 * (Hkv if case["each"] else 1) * cached
    return {"bytes": moved, "flops": 4 * Hq * d * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    new, old = lengths(case)
    total = [n + o for n, o in zip(new, old)]
    B, Hq, Hkv, d, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    T = sum(new)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def whole(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def tables(sizes, free):
        width = max(1, max(-(-n // page) for n in sizes))
        return whole([[free.pop() if i * page < n else -1 for i in range(width)] for n in sizes])

    def offsets(sizes):
        return [sum(sizes[:i]) for i in range(len(sizes) + 1)]

    kept = [min(n, case["keep"]) for n in total] if case["kind"] == "evict" else []
    n_pages = sum(-(-n // page) for n in total + kept) + 3
    free = list(range(n_pages))
    r.shuffle(free)
    s = dict(case=case, k_pages=normal(n_pages, page, Hkv, d), v_pages=normal(n_pages, page, Hkv, d),
             page_table=tables(total, free), seq_lens=whole(total), longest=max(total), most_new=max(new))
    if case["kind"] == "evict":
        heads = Hkv if case["each"] else 1
        # heavy-tailed, as attention is; the newest tokens have nothing yet
        w = torch.rand(B, heads, s["page_table"].shape[1] * page, generator=g, device="cuda").pow_(4)
        at = torch.arange(w.shape[2], device="cuda")
        w[(at >= s["seq_lens"][:, None, None] - min(8, case["recent"] + 1)).expand_as(w)] = 0
        s["weights"] = w
        s["dst_table"] = tables(kept, free)
        return s
    s["cu"] = whole(offsets(new))
    if case["kind"] == "append":
        # K and V as a projection leaves them: side by side in one row
        both = normal(T, 2 * Hkv, d)
        s["k_new"], s["v_new"] = both[:, :Hkv], both[:, Hkv:]
        first = [3 * o for o in old]  # original positions: tokens in between were skipped
        s["pos"] = whole([p + i for n, p in zip(new, first) for i in range(n)])
        return s
    s["q"] = normal(T, Hq, d) * 2
    if case["kind"] == "weigh":
        heads = Hkv if case["each"] else 1
        s["weights"] = torch.rand(B, heads, s["page_table"].shape[1] * page, generator=g, device="cuda")
        s["weights"] *= torch.arange(s["weights"].shape[2], device="cuda") < s["seq_lens"][:, None, None]
    return s


# ------------------------------------------------------------------ plain forms
def slots(table, page, at):
    """The flat cache slot of token `at` [B, ...] of each sequence."""
    b = torch.arange(table.shape[0], device=at.device).view(-1, *[1] * (at.dim() - 1))
    return table.clamp(min=0).long()[b, at // page] * page + at % page


def owners(cu, T):
    """For each packed new token its sequence and its place among that sequence's new tokens."""
    at = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu.long(), at, right=True) - 1
    return b, at - cu.long()[b]


def plain_append(s):
    k, v, cu, lens, table = s["k_new"], s["v_new"], s["cu"].long(), s["seq_lens"].long(), s["page_table"]
    T, Hkv, d = k.shape
    page = s["case"]["page"]
    b, i = owners(cu, T)
    at = lens[b] - (cu[b + 1] - cu[b]) + i
    slot = table.long()[b, at // page] * page + at % page
    turn = torch.arange(0, d, 2, device=k.device, dtype=torch.float64) / d
    angle = s["pos"].double()[:, None] * THETA ** -turn
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    lo, hi = k.float().chunk(2, dim=-1)
    s["k_pages"].view(-1, Hkv, d)[slot] = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1).bfloat16()
    s["v_pages"].view(-1, Hkv, d)[slot] = v
    return {"k": s["k_pages"], "v": s["v_pages"]}


def plain_attend(s):
    c, q, cu, lens = s["case"], s["q"], s["cu"].long(), s["seq_lens"].long()
    B, Hkv, d, page, L, N = c["B"], c["Hkv"], c["d"], c["page"], s["longest"], s["most_new"]
    G, T = c["Hq"] // Hkv, q.shape[0]
    b, i = owners(cu, T)
    at = torch.arange(L, device=q.device)
    slot = slots(s["page_table"], page, at.expand(B, L))
    there = at < lens[:, None]
    K = s["k_pages"].view(-1, Hkv, d)[slot].float().permute(0, 2, 1, 3)  # [B, Hkv, L, d]
    V = s["v_pages"].view(-1, Hkv, d)[slot].float().permute(0, 2, 1, 3)
    V = V.masked_fill(~there[:, None, :, None], 0)
    Q = q.new_zeros(B, N, Hkv, G, d, dtype=torch.float32)
    Q[b, i] = q.float().view(T, Hkv, G, d)
    Q = Q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, d)
    x = torch.matmul(Q, K.transpose(2, 3)).view(B, Hkv, G, N, L).mul_(d ** -0.5)
    n = cu[1:] - cu[:-1]
    place = torch.arange(N, device=q.device)
    sees = at <= (lens - n)[:, None, None] + place[:, None]  # [B, N, L]
    sees = sees & (place < n[:, None])[:, :, None]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0)
    x = x.sub_(top).exp_()
    all_ = x.sum(-1, keepdim=True)
    x.div_(all_.masked_fill(all_ == 0, 1))
    o = torch.matmul(x.view(B, Hkv, G * N, L), V).view(B, Hkv, G, N, d).permute(0, 3, 1, 2, 4)
    out = {"o": o[b, i].reshape(T, c["Hq"], d).bfloat16()}
    if c.get("lse"):
        out["lse"] = (top + all_.log())[..., 0].permute(0, 3, 1, 2)[b, i].reshape(T, c["Hq"])
    if c["kind"] == "weigh":
        got = x.sum((2, 3)) if c["each"] else x.sum((1, 2, 3))[:, None]
        out["weights"] = s["weights"].clone()
        out["weights"][:, :, :L] += got
    return out


def plain_evict(s):
    c, lens, w = s["case"], s["seq_lens"].long(), s["weights"]
    Hkv, d, page, keep = c["Hkv"], c["d"], c["page"], c["keep"]
    B, heads, cap = w.shape
    at = torch.arange(cap, device=w.device)
    n = lens[:, None, None]
    key = w.masked_fill((at < c["sink"]) | (at >= n - c["recent"]), math.inf).masked_fill(at >= n, -math.inf)
    width = s["dst_table"].shape[1] * page
    take = min(keep, cap)
    kept = key.sort(dim=-1, descending=True, stable=True)[1][..., :take].sort(-1)[0]  # [B, heads, take]
    new = lens.clamp(max=keep)
    t = torch.arange(take, device=w.device)
    valid = (t < new[:, None])[:, None].expand(B, heads, take)
    b = torch.arange(B, device=w.device)[:, None, None].expand_as(kept)
    src = slots(s["page_table"], page, kept)
    dst = slots(s["dst_table"], page, t.clamp(max=width - 1).expand(B, heads, take))
    h = torch.arange(heads, device=w.device)[:, None].expand_as(kept)
    out_w = w.new_zeros(B, heads, width)
    out_w[b[valid], h[valid], t.expand_as(kept)[valid]] = w.gather(-1, kept)[valid]
    # every head of a token, or the one that chose it
    to, of = (dst[valid], src[valid]) if not c["each"] else ((dst[valid], h[valid]), (src[valid], h[valid]))
    k, v = s["k_pages"].view(-1, Hkv, d), s["v_pages"].view(-1, Hkv, d)
    k[to], v[to] = k[of], v[of]
    idx = torch.full((B, heads, keep), -1, dtype=torch.int32, device=w.device)
    idx[..., :take] = torch.where(valid, kept, -1).int()
    return {"k": s["k_pages"], "v": s["v_pages"], "weights": out_w, "lens": new.int(), "kept": idx}


PLAIN = {"append": plain_append, "attend": plain_attend, "weigh": plain_attend, "evict": plain_evict}


def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["kind"]](s)
    import token_skipping_sparse_b200 as S
    if c["kind"] == "append":
        S.spts_cache_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["cu"],
                            pos=s["pos"], theta=THETA)
        return {"k": s["k_pages"], "v": s["v_pages"]}
    if c["kind"] == "evict":
        lens, weights, kept = S.spts_cache_evict(s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["weights"],
                                                 c["keep"], sink=c["sink"], recent=c["recent"], dst_table=s["dst_table"],
                                                 kept=True)
        return {"k": s["k_pages"], "v": s["v_pages"], "weights": weights, "lens": lens, "kept": kept}
    out = {}
    if c["kind"] == "weigh":
        out["weights"] = s["weights"].clone()
    got = S.spts_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["cu"],
                                 lse=c.get("lse", False), weights=out.get("weights"))
    if c.get("lse"):
        out["o"], out["lse"] = got
    else:
        out["o"] = got
    return out


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """Sequence by sequence and head by head, from the definitions."""
    s = prepare(case, seed)
    Hq, Hkv, d, page = (case[n] for n in ("Hq", "Hkv", "d", "page"))
    new, old = lengths(case)
    K, V = s["k_pages"].double(), s["v_pages"].double()
    table = s["page_table"].tolist()

    def rows(b, n):
        """The cache rows (page, place) of sequence b's first n tokens."""
        t = torch.arange(n, device="cuda")
        return torch.tensor(table[b], device="cuda")[t // page], t % page

    if case["kind"] == "append":
        first = 0
        for b, (n, o) in enumerate(zip(new, old)):
            p, at = rows(b, o + n)
            x = torch.view_as_complex(torch.stack(s["k_new"][first:first + n].double().chunk(2, -1), -1).contiguous())
            freq = torch.exp(-math.log(THETA) * torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
            angle = torch.outer(s["pos"][first:first + n].double(), freq)[:, None]
            y = x * torch.polar(torch.ones_like(angle), angle)
            K[p[o:], at[o:]] = torch.cat((y.real, y.imag), -1)
            V[p[o:], at[o:]] = s["v_new"][first:first + n].double()
            first += n
        return {"k": K, "v": V}

    if case["kind"] == "evict":
        w, width = s["weights"], s["dst_table"].shape[1] * page
        out_w = torch.zeros(*w.shape[:2], width, device="cuda", dtype=torch.float64)
        K0, V0 = K.clone(), V.clone()
        dst = s["dst_table"].tolist()
        for b, n in enumerate(old):
            p, at = rows(b, n)
            for h in range(w.shape[1]):
                got = w[b, h, :n].tolist()
                safe = set(range(min(n, case["sink"]))) | set(range(max(0, n - case["recent"]), n))
                order = sorted(range(n), key=lambda j: (j not in safe, -got[j], j))
                kept = torch.tensor(sorted(order[:case["keep"]]), device="cuda", dtype=torch.long)
                t = torch.arange(len(kept), device="cuda")
                to = torch.tensor(dst[b], device="cuda")[t // page], t % page
                some = slice(h, h + 1) if case["each"] else slice(None)
                K[to[0], to[1], some] = K0[p[kept], at[kept], some]
                V[to[0], to[1], some] = V0[p[kept], at[kept], some]
                out_w[b, h, :len(kept)] = w[b, h, kept].double()
        return {"k": K, "v": V, "weights": out_w, "lens": None, "kept": None}

    G = Hq // Hkv
    out = torch.zeros(sum(new), Hq, d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(sum(new), Hq, device="cuda", dtype=torch.float64)
    weights = s["weights"].double() if case["kind"] == "weigh" else None
    first = 0
    for b, (n, o) in enumerate(zip(new, old)):
        p, at = rows(b, o + n)
        sees = torch.arange(o + n, device="cuda") < o + 1 + torch.arange(n, device="cuda")[:, None]
        for h in range(Hq if n else 0):
            x = s["q"][first:first + n, h].double() @ K[p, at, h // G].T / math.sqrt(d)
            x = torch.where(sees, x, -math.inf)
            lse[first:first + n, h] = torch.logsumexp(x, -1)
            x = torch.exp(x - lse[first:first + n, h, None])
            out[first:first + n, h] = x @ V[p, at, h // G]
            if weights is not None:
                weights[b, h // G if case["each"] else 0, :o + n] += x.sum(0)
        first += n
    answer = {"o": out}
    if case.get("lse"):
        answer["lse"] = lse
    if weights is not None:
        answer["weights"] = weights
    return answer
