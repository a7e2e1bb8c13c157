"""The paged-cache operators as measured cases: what each pass computes, in
plain torch operations (`own` false) or through the library (`own` true).

Kinds of case:
  extend   block tables and slot maps from request lengths, then the roll-back
           of the same tokens (a speculative step whose draft is rejected), so
           that a pass leaves the free list and the lengths as they were
  append   new K/V rows written into the pages at the slots
  decode   attention of one new token per sequence over its pages; with
           K > 0 over K listed pages per (sequence, kv head)
  scores   per-page key bounds brought up to date, then the score of every page
  select   the K best-scored pages per (sequence, kv head)

A cache page holds `ps` tokens; pools are [pages, ps, Hkv, D].  Lengths belong
to the case (they fix the work), every value and page number to the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"


def _lib():
    import context_exact_attention_ring_b200 as ra
    return ra


def _cdiv(a, b):
    return -(-a // b)


def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _eb(case):
    return 4 if case["dtype"] == "fp32" else 2


def _loguniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(case):
    """The case's sequence lengths: log-uniform over [lo, hi], every seventh
    row of a batch of 7 or more an empty (padding) row."""
    rng = random.Random(case["lens_seed"])
    n = [_loguniform(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
    return [0 if case["B"] >= 7 and i % 7 == 6 else x for i, x in enumerate(n)]


def _news(case):
    rng = random.Random(case["lens_seed"] + 1)
    return [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]


def listed():
    return [
        # one decode step of a busy server with draft tokens: 256 requests, 1 to 4 tokens each (latency)
        dict(name="extend_step", kind="extend", B=256, ps=16, lo=1, hi=8000, new_lo=1, new_hi=4, lens_seed=1),
        # prompts admitted together: 1021 requests, about half a million new tokens
        dict(name="extend_prompts", kind="extend", B=1021, ps=16, lo=1, hi=2000, new_lo=1, new_hi=1024, lens_seed=2),
        # one new token for each of 64 requests, a float32 cache (latency)
        dict(name="append_step_fp32", kind="append", T=64, pad=5, Hq=32, Hkv=8, D=128, ps=16, dtype="fp32"),
        # a prompt chunk of 32k tokens written into its pages
        dict(name="append_prompt", kind="append", T=32768, pad=37, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16"),
        # one request, early in its answer (latency)
        dict(name="decode_one_short", kind="decode", B=1, Hq=8, Hkv=2, D=128, ps=16, lo=77, hi=77, lens_seed=3, K=0,
             dtype="bf16"),
        # an ordinary serving batch: ragged lengths, some rows padding
        dict(name="decode_batch", kind="decode", B=64, Hq=32, Hkv=8, D=128, ps=16, lo=64, hi=16000, lens_seed=4, K=0,
             dtype="bf16"),
        # float32 cache, 64-wide heads, five query heads to a kv head
        dict(name="decode_fp32_g5", kind="decode", B=24, Hq=40, Hkv=8, D=64, ps=32, lo=64, hi=9001, lens_seed=5, K=0,
             dtype="fp32"),
        # long contexts, 64k to 128k tokens each
        dict(name="decode_long", kind="decode", B=6, Hq=32, Hkv=8, D=128, ps=64, lo=65536, hi=131072, lens_seed=6, K=0,
             dtype="bf16"),
        # the same long contexts read through 128 selected pages of 32 tokens for each kv head
        dict(name="decode_selected", kind="decode", B=6, Hq=32, Hkv=8, D=128, ps=32, lo=65536, hi=131072, lens_seed=7,
             K=128, dtype="bf16"),
        # a decode step of short contexts: the newest page's bounds, then all scores, float32 (latency)
        dict(name="scores_step_fp32", kind="scores", B=5, Hq=8, Hkv=2, D=64, ps=16, lo=100, hi=5000, lens_seed=8,
             every=False, dtype="fp32"),
        # after long prompts: the bounds of every page, then all scores
        dict(name="scores_prompts", kind="scores", B=6, Hq=32, Hkv=8, D=128, ps=32, lo=65536, hi=131072, lens_seed=9,
             every=True, dtype="bf16"),
        # 128 of up to 4096 pages for each of 48 (sequence, kv head) pairs
        dict(name="select_long", kind="select", B=6, Hkv=8, ps=32, lo=65536, hi=131072, lens_seed=10, K=128),
    ]


def draw(rng):
    kind = rng.choice(["extend", "append", "decode", "decode", "decode", "scores", "select"])
    ps = rng.choice([8, 16, 32, 64, 128])
    seed = rng.randrange(1 << 20)
    if kind == "extend":
        B = _loguniform(rng, 1, 1021)
        return dict(kind=kind, B=B, ps=ps, lo=1, hi=_loguniform(rng, 2, 8000), new_lo=rng.choice([0, 1]),
                    new_hi=_loguniform(rng, 1, 1024), lens_seed=seed)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "append":
        return dict(kind=kind, T=_loguniform(rng, 1, 16384), pad=rng.randint(0, 40), Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps,
                    dtype=dtype)
    hi = _loguniform(rng, 2, 131072)
    lo = max(1, hi // rng.choice([1, 2, 16, 1000]))
    B = min(_loguniform(rng, 1, 256), max(1, 250000 // hi))
    if kind == "select":
        return dict(kind=kind, B=B, Hkv=Hkv, ps=ps, lo=lo, hi=hi, lens_seed=seed, K=_loguniform(rng, 3, 300))
    if kind == "scores":
        return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, lens_seed=seed,
                    every=rng.random() < 0.5, dtype=dtype)
    K = rng.choice([0, 0, _loguniform(rng, 3, 300)])
    return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, lens_seed=seed, K=K, dtype=dtype)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _tables(case, gen, lens, width):
    """A block table [B, width] of distinct random pages for the lengths and
    the number of pages of the pool; entries past a sequence's pages are 0."""
    need = [_cdiv(n, case["ps"]) for n in lens]
    total = sum(need)
    pages = total + 3
    perm = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)
    have = torch.tensor(need, device=DEV)
    start = have.cumsum(0) - have
    at = torch.arange(width, device=DEV)
    flat = (start[:, None] + at[None, :]).clamp(max=pages - 1)
    table = torch.where(at[None, :] < have[:, None], perm[flat], 0)
    return table.to(torch.int32).contiguous(), pages, perm


def _ints(v):
    return torch.tensor(v, device=DEV, dtype=torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, ps = case["kind"], case.get("ps")
    s = dict(case=case, ps=ps)
    if kind == "append":
        T, Hkv, D, dt = case["T"], case["Hkv"], case["D"], _dt(case)
        pages = _cdiv(T, ps) + 2
        # K and V rows as a projection leaves them: slices of one [T, Hq + 2 Hkv, D] tensor
        qkv = _normal(gen, (T + case["pad"], case["Hq"] + 2 * Hkv, D), dt)
        s["k_new"], s["v_new"] = qkv[:, case["Hq"]:case["Hq"] + Hkv], qkv[:, case["Hq"] + Hkv:]
        # consecutive tokens in consecutive rows of random pages, as a slot map lays them out; padding is -1
        order = torch.randperm(pages, generator=gen, device=DEV)
        t = torch.arange(T, device=DEV)
        slots = torch.full((T + case["pad"],), -1, device=DEV, dtype=torch.int32)
        slots[:T] = (order[t // ps] * ps + t % ps).to(torch.int32)
        s["slots"] = slots
        s["k_pool"] = torch.zeros((pages, ps, Hkv, D), device=DEV, dtype=dt)
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        return s
    lens = _lens(case)
    B = case["B"]
    s["lens"] = _ints(lens)
    if kind == "extend":
        news = _news(case)
        width = _cdiv(case["hi"] + case["new_hi"], ps)
        table, pages, perm = _tables(case, gen, lens, width)
        room = sum(_cdiv(a + b, ps) - _cdiv(a, ps) for a, b in zip(lens, news)) + 5
        s["table"], s["new"] = table, _ints(news)
        s["free"] = (pages + torch.randperm(room, generator=gen, device=DEV)).to(torch.int32)
        s["n_free"] = _ints([room])
        s["keep"] = s["lens"].clone()
        n_tokens = sum(news) + 16
        s["slots"] = torch.empty((n_tokens,), device=DEV, dtype=torch.int32)
        s["start"] = torch.empty((B,), device=DEV, dtype=torch.int32)
        s["cu"] = torch.empty((B + 1,), device=DEV, dtype=torch.int32)
        return s
    width = max(1, _cdiv(max(lens), ps))
    if kind == "select":
        s["scores"] = _normal(gen, (B, case["Hkv"], width), torch.float32) * 20
        # some scores alike, so that ties are met
        s["scores"] = torch.where(s["scores"] > 30, torch.full_like(s["scores"], 30.0), s["scores"])
        return s
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _dt(case)
    s["table"], pages, _ = _tables(case, gen, lens, width)
    s["k_pool"] = _normal(gen, (pages, ps, Hkv, D), dt)
    qkv = _normal(gen, (B, Hq + 2 * Hkv, D), dt)
    s["q"] = qkv[:, :Hq]                       # a slice of the projection's rows
    if kind == "decode":
        s["v_pool"] = _normal(gen, (pages, ps, Hkv, D), dt)
        s["scale"] = 1.0 / math.sqrt(D)
        K = case["K"]
        if K:
            # ascending random pages of each sequence, -1 past their number
            have = torch.tensor([_cdiv(n, ps) for n in lens], device=DEV)
            r = torch.rand((B, Hkv, width), generator=gen, device=DEV)
            r = torch.where(torch.arange(width, device=DEV) < have[:, None, None], r, 2.0)
            kk = min(K, width)
            pick = r.argsort(dim=-1)[..., :kk].sort(dim=-1).values
            big = torch.where(pick < have[:, None, None], pick, 1 << 30).sort(dim=-1).values
            sel = torch.full((B, Hkv, K), -1, device=DEV, dtype=torch.int32)
            sel[..., :kk] = torch.where(big < (1 << 30), big, -1).to(torch.int32)
            s["sel"] = sel
            s["n_sel"] = (sel >= 0).sum(-1).to(torch.int32)
        return s
    # bounds [pages, Hkv, 2, D]: those of the earlier pages are in place, the newest token's page is due
    s["start"] = None if case["every"] else (s["lens"] - 1).clamp(min=0)
    lo_hi = torch.stack([s["k_pool"].amin(1), s["k_pool"].amax(1)], dim=2)
    s["bounds"] = torch.zeros_like(lo_hi) if case["every"] else lo_hi.contiguous()
    s["scores"] = torch.empty((B, Hkv, width), device=DEV, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_extend(s):
    ps, table = s["ps"], s["table"].long()
    lens, new, free, n_free = s["lens"].long(), s["new"].long(), s["free"].long(), s["n_free"].long()
    B, width = table.shape
    n_tokens = s["slots"].numel()
    at = torch.arange(width, device=DEV)
    cu = torch.cat([torch.zeros(1, device=DEV, dtype=torch.long), new.cumsum(0)])
    old, full = (lens + ps - 1) // ps, (lens + new + ps - 1) // ps
    fits = (lens + new <= width * ps) & (cu[1:] <= n_tokens)
    need = torch.where(fits, full - old, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= n_free))
    # pages taken from the end of the free list, in order of sequence and page
    from_end = (upto - need)[:, None] + at[None, :] - old[:, None]
    mine = ok[:, None] & (at[None, :] >= old[:, None]) & (at[None, :] < full[:, None])
    taken = free[(n_free - 1 - from_end).clamp(0, free.numel() - 1)]
    table = torch.where(mine, taken, table)
    n_free = n_free - torch.where(ok, need, 0).sum()
    start = torch.where(ok, lens, -1)
    lens = lens + torch.where(ok, new, 0)
    t = torch.arange(n_tokens, device=DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    pos = start[b] + t - cu[b]
    live = (t < cu[-1]) & (start[b] >= 0)
    page = table[b, torch.where(live, pos, 0) // ps]
    slots = torch.where(live, page * ps + pos % ps, -1)
    # the roll-back: lengths down to keep, the pages back on the free list, last taken first
    keep = torch.minimum(s["keep"].long().clamp(min=0), lens)
    a, e = (keep + ps - 1) // ps, (lens + ps - 1) // ps
    gone = e - a
    upto = gone.cumsum(0)
    back = (at[None, :] >= a[:, None]) & (at[None, :] < e[:, None])
    to = n_free + upto[-1] - 1 - ((upto - gone)[:, None] + at[None, :] - a[:, None])
    more = torch.cat([free, torch.zeros(1, device=DEV, dtype=torch.long)])
    more[torch.where(back, to, free.numel())] = torch.where(back, table, 0)
    out = [slots, cu, start, table, keep, n_free + gone.sum(), more[:-1]]
    return [x.to(torch.int32) for x in out]


def _plain_append(s):
    k_pool, v_pool, slots = s["k_pool"], s["v_pool"], s["slots"].long()
    live = slots >= 0
    at = slots[live]
    k_pool.view(-1, *k_pool.shape[2:])[at] = s["k_new"][live]
    v_pool.view(-1, *v_pool.shape[2:])[at] = s["v_new"][live]
    return [k_pool, v_pool]


def _softmax_rows(q, k, v, live, scale):
    """q [..., G, D], k, v [..., S, D] float32, live [..., 1, S]: the rows'
    attention and the log of their sums; a row with no key is 0 and -inf."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = torch.where(live, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    some = total > 0
    o = torch.matmul(e, v) / torch.where(some, total, 1.0)
    return o, torch.where(some, m + torch.log(total), float("-inf"))[..., 0]


def _plain_decode(s):
    case, ps = s["case"], s["ps"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    lens, table = s["lens"].long(), s["table"].long()
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    off = torch.arange(ps, device=DEV)
    if case["K"]:
        sel = s["sel"].long()                                        # [B, Hkv, K]
        page = torch.gather(table[:, None, :].expand(-1, Hkv, -1), 2, sel.clamp(min=0))
        head = torch.arange(Hkv, device=DEV)[None, :, None]
        k, v = (p.permute(2, 0, 1, 3)[head, page].flatten(2, 3).float() for p in (s["k_pool"], s["v_pool"]))
        pos = (sel[..., None] * ps + off).flatten(2)                 # [B, Hkv, K ps]
        live = (pos >= 0) & (pos < lens[:, None, None]) & (sel >= 0).repeat_interleave(ps, dim=2)
        live = live[:, :, None, :]
    else:
        k, v = (p[table].flatten(1, 2).float().transpose(1, 2) for p in (s["k_pool"], s["v_pool"]))
        pos = torch.arange(k.shape[2], device=DEV)
        live = (pos[None, :] < lens[:, None])[:, None, None, :]
    o, lse = _softmax_rows(q, k, v, live, s["scale"])
    return [o.reshape(B, Hq, D).to(s["q"].dtype), lse.reshape(B, Hq)]


def _plain_scores(s):
    case, ps = s["case"], s["ps"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    lens, table, bounds = s["lens"].long(), s["table"].long(), s["bounds"]
    width = table.shape[1]
    have = (lens + ps - 1) // ps
    # bounds of the pages from start on
    first = torch.zeros_like(lens) if s["start"] is None else s["start"].long() // ps
    span = width if s["start"] is None else 1
    at = first[:, None] + torch.arange(span, device=DEV)
    due = at < have[:, None]
    page = torch.gather(table, 1, at.clamp(max=width - 1))
    rows = s["k_pool"][page]                                          # [B, span, ps, Hkv, D]
    live = (at[..., None] * ps + torch.arange(ps, device=DEV) < lens[:, None, None])[..., None, None]
    lo = torch.where(live, rows, float("inf")).amin(2)
    hi = torch.where(live, rows, float("-inf")).amax(2)
    bounds[page[due]] = torch.stack([lo, hi], dim=3)[due]
    # scores of all pages
    x = bounds[table].float()                                         # [B, width, Hkv, 2, D]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    up = torch.matmul(q.clamp(min=0), x[..., 1, :].permute(0, 2, 3, 1))
    down = torch.matmul(q.clamp(max=0), x[..., 0, :].permute(0, 2, 3, 1))
    score = (up + down).amax(2)
    valid = torch.arange(width, device=DEV)[None, :] < have[:, None]
    return [bounds, torch.where(valid[:, None, :], score, float("-inf"))]


def _plain_select(s):
    K, ps, x = s["case"]["K"], s["ps"], s["scores"]
    B, Hkv, width = x.shape
    have = (s["lens"].long() + ps - 1) // ps
    at = torch.arange(width, device=DEV)
    live = at[None, :] < have[:, None]
    must = live & ((at[None, :] < 1) | (at[None, :] >= have[:, None] - 1))     # the first page and the last
    x = torch.where(must[:, None, :], float("inf"), torch.where(live[:, None, :], x, float("-inf")))
    best = x.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    n = have.clamp(max=K)[:, None].expand(B, Hkv)
    best = torch.where(torch.arange(best.shape[-1], device=DEV) < n[..., None], best, width)
    best = best.sort(dim=-1).values
    sel = torch.full((B, Hkv, K), -1, device=DEV, dtype=torch.int32)
    sel[..., :best.shape[-1]] = torch.where(best < width, best, -1).to(torch.int32)
    return [sel, n.to(torch.int32).contiguous()]


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------
def _own(s):
    ra, kind, ps = _lib(), s["case"]["kind"], s["ps"]
    if kind == "extend":
        ra.ring_attn_page_extend(s["lens"], s["new"], s["table"], s["free"], s["n_free"], ps, slot_map=s["slots"],
                                 start_lens=s["start"], cu_new=s["cu"])
        ra.ring_attn_page_trim(s["lens"], s["keep"], s["table"], s["free"], s["n_free"], ps)
        return [s["slots"], s["cu"], s["start"], s["table"], s["lens"], s["n_free"], s["free"]]
    if kind == "append":
        ra.ring_attn_paged_append(s["k_pool"], s["v_pool"], s["k_new"], s["v_new"], s["slots"])
        return [s["k_pool"], s["v_pool"]]
    if kind == "decode":
        if "ws" not in s:
            s["ws"] = ra.decode_paged_workspace(s["case"]["D"])   # a program keeps one per stream
        out, lse = ra.ring_attn_decode_paged(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                             sel=s.get("sel"), n_sel=s.get("n_sel"), scale=s["scale"],
                                             workspace=s["ws"])
        return [out, lse]
    if kind == "scores":
        ra.ring_attn_page_bounds(s["k_pool"], s["table"], s["lens"], bounds=s["bounds"], start_lens=s["start"])
        ra.ring_attn_page_scores(s["q"], s["bounds"], s["table"], s["lens"], ps, scores=s["scores"])
        return [s["bounds"], s["scores"]]
    sel, n = ra.ring_attn_page_select(s["scores"], s["lens"], ps, s["case"]["K"], keep_first=1, keep_last=1)
    return [sel, n]


_PLAIN = dict(extend=_plain_extend, append=_plain_append, decode=_plain_decode, scores=_plain_scores,
              select=_plain_select)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------
def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    kind, ps = case["kind"], case["ps"]
    if kind == "append":
        row = case["Hkv"] * case["D"] * _eb(case)
        return {"bytes": 4 * case["T"] * row + 4 * (case["T"] + case["pad"]), "flops": 0}
    lens = _lens(case)
    B = case["B"]
    if kind == "extend":
        news = _news(case)
        taken = sum(_cdiv(a + b, ps) - _cdiv(a, ps) for a, b in zip(lens, news))
        # lengths in and out twice, new, keep, start, cu; slots; each page off the list, into the table and back
        return {"bytes": 4 * (8 * B + 1 + sum(news) + 16 + 4 * taken), "flops": 0}
    have = [_cdiv(n, ps) for n in lens]
    if kind == "select":
        n = sum(min(x, case["K"]) for x in have)
        return {"bytes": 4 * (case["Hkv"] * (sum(have) + n + B) + B), "flops": 0}
    Hq, Hkv, D, e = case["Hq"], case["Hkv"], case["D"], _eb(case)
    if kind == "scores":
        due = sum(lens) if case["every"] else sum((n - 1) % ps + 1 for n in lens if n)
        # a due page's bounds are written, and the other pages' read
        return {"bytes": Hkv * D * e * (due + 2 * sum(have)) + 4 * Hkv * sum(have) + 4 * (sum(have) + B)
                + B * Hq * D * e, "flops": 4 * Hq * D * sum(have)}
    if case["K"]:
        # K random pages of each; the last one, chosen or not, may be part filled: counted full
        keys = sum(min(n, min(x, case["K"]) * ps) for n, x in zip(lens, have))
    else:
        keys = sum(lens)
    return {"bytes": 2 * keys * Hkv * D * e + B * Hq * (2 * D * e + 4) + 4 * (sum(have) + B),
            "flops": 4 * keys * Hq * D}


# ---------------------------------------------------------------------------
def exact(case, seed):
    """The computed outputs in 64 bits, one sequence at a time from the
    definition; whole-number outputs have no such value."""
    kind, ps = case["kind"], case["ps"]
    if kind in ("extend", "select"):
        return None
    s = prepare(case, seed)
    if kind == "append":
        res = []
        for pool, rows in ((s["k_pool"], s["k_new"]), (s["v_pool"], s["v_new"])):
            x = torch.zeros((pool.shape[0] * ps,) + tuple(pool.shape[2:]), device=DEV, dtype=torch.float64)
            x.index_copy_(0, s["slots"][:case["T"]].long(), rows[:case["T"]].double())
            res.append(x.view(pool.shape))
        return res
    lens = s["lens"].tolist()
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    if kind == "decode":
        out = torch.zeros((case["B"], Hq, D), device=DEV, dtype=torch.float64)
        lse = torch.full((case["B"], Hq), float("-inf"), device=DEV, dtype=torch.float64)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = s["table"][b, :_cdiv(n, ps)].long()
            for h in range(Hkv):
                k, v = (p[:, :, h][pages].reshape(-1, D)[:n].double() for p in (s["k_pool"], s["v_pool"]))
                if case["K"]:
                    chosen = torch.zeros(pages.numel(), device=DEV, dtype=torch.bool)
                    chosen[s["sel"][b, h, :int(s["n_sel"][b, h])].long()] = True
                    rows = chosen.repeat_interleave(ps)[:n]
                    k, v = k[rows], v[rows]
                x = (s["q"][b, h * G:(h + 1) * G].double() @ k.T) * s["scale"]
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
        return [out, lse]
    width = s["table"].shape[1]
    bounds = s["bounds"].double()
    scores = torch.full((case["B"], Hkv, width), float("-inf"), device=DEV, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = s["table"][b, :_cdiv(n, ps)].long()
        p0 = 0 if case["every"] else (n - 1) // ps
        for h in range(Hkv):
            k = s["k_pool"][:, :, h][pages[p0:]].double()
            part = n - (pages.numel() - 1) * ps
            full, tail = k[:-1], k[-1, :part]
            bounds[pages[p0:-1], h, 0], bounds[pages[p0:-1], h, 1] = full.amin(1), full.amax(1)
            bounds[pages[-1], h, 0], bounds[pages[-1], h, 1] = tail.amin(0), tail.amax(0)
            x = bounds[pages, h]
            for g in range(G):
                q = s["q"][b, h * G + g].double()
                r = torch.maximum(q * x[:, 0], q * x[:, 1]).sum(-1)
                scores[b, h, :pages.numel()] = torch.maximum(scores[b, h, :pages.numel()], r)
    return [bounds, scores]
