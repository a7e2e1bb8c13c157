"""GPU tests of the paged-cache operators against plain 64-bit references:
block tables and slot maps, the paged append, the paged decode (all pages and
selected ones), page bounds, scores and selection."""
import math

import numpy as np
import pytest
import torch

import context_exact_attention_ring_b200 as ra
from tests import paged_ref as R
from tests.helpers import margin, need_cuda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ok():
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK


# ---------------------------------------------------------------- tables
def _tables(lens, ps, W, extra, seed):
    rng = np.random.default_rng(seed)
    need = [R.cdiv(min(max(n, 0), W * ps), ps) for n in lens]
    perm = rng.permutation(sum(need) + extra)
    table = np.full((len(lens), W), -7, dtype=np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:]


@pytest.mark.parametrize("ps", [8, 16, 1024])
@pytest.mark.parametrize("B,news,max_tokens", [
    (1, [0], 1), (1, [1], 1), (5, [3, 0, 17, 1, 40], 64), (5, [-4, 2000, 1, 1, 9], 5000), (6, [5, 5, 5, 5, 5, 5], 30),
    (6, [5, 40, 0, 3, 0, 1], 40),                        # tokens past the slot map; those without any are served
])
def test_extend_and_trim_small(ps, B, news, max_tokens):
    need_cuda()
    lens = [0, 1, ps, ps + 1, 3 * ps - 1, 5][:B]
    W = 4 + 2048 // ps
    table, free = _tables(lens, ps, W, 300, 7 * ps + B)
    ref = R.Tables(lens, table, free, len(free), ps)
    sl, tb, fr, nf = ints(lens), ints(table), ints(free), ints([len(free)])
    slots, start, cu = ra.ring_attn_page_extend(sl, ints(news), tb, fr, nf, ps, max_tokens=max_tokens)
    want = ref.extend(news, max_tokens)
    torch.cuda.synchronize()
    assert (slots.tolist(), start.tolist(), cu.tolist()) == want[:3]
    assert sl.tolist() == ref.lens and np.array_equal(tb.cpu().numpy(), ref.table) and nf.tolist() == [ref.n]
    assert fr.tolist() == ref.free
    assert ra.ring_attn_device_error()[0] == (ra.RING_ECAPACITY if want[3] else ra.RING_OK)
    # cutting the new tokens off restores lengths and free list
    before = list(free)
    ra.ring_attn_page_trim(sl, ints(lens), tb, fr, nf, ps)
    ref.trim(lens)
    ok()
    assert sl.tolist() == ref.lens == lens and nf.tolist() == [ref.n] == [len(before)] and fr.tolist() == before


@pytest.mark.parametrize("B,max_tokens,room", [(1500, 40000, 100000), (1500, 9000, 100000), (1030, 60000, 900), (3, 5000, 7)])
def test_extend_and_trim_many_sequences_and_shortage(B, max_tokens, room):
    # more sequences than a block has threads, more tokens than one launch writes, too few
    # free pages, too few token numbers, sequences beyond their table's width
    need_cuda()
    ps, W = 16, 40
    rng = np.random.default_rng(B + room)
    lens = [int(x) for x in rng.integers(0, 400, B)]
    news = [int(x) for x in rng.integers(-2, 30, B)]
    news[B // 2] = 600                                   # wider than the table
    table, free = _tables(lens, ps, W, 60000, 3)
    free = free[:room]
    ref = R.Tables(lens, table, free, len(free), ps)
    wide = ints(np.concatenate([table, np.full((B, 5), 99)], axis=1))
    tb = wide[:, :W]                                     # rows of a wider table
    sl, fr, nf = ints(lens), ints(free), ints([len(free)])
    slots, start, cu = ra.ring_attn_page_extend(sl, ints(news), tb, fr, nf, ps, max_tokens=max_tokens)
    w_slots, w_start, w_cu, short = ref.extend(news, max_tokens)
    assert short and ra.ring_attn_device_error()[0] == ra.RING_ECAPACITY
    assert slots.tolist() == w_slots and start.tolist() == w_start and cu.tolist() == w_cu
    assert sl.tolist() == ref.lens and nf.tolist() == [ref.n]
    assert np.array_equal(wide[:, :W].cpu().numpy(), ref.table) and (wide[:, W:] == 99).all()
    # end every third sequence, roll others back a little, and lengthen nobody
    keep = [0 if b % 3 == 0 else ref.lens[b] - 5 if b % 3 == 1 else 10 ** 6 for b in range(B)]
    over = ref.trim(keep)
    ra.ring_attn_page_trim(sl, ints(keep), tb, fr, nf, ps)
    assert ra.ring_attn_device_error()[0] == (ra.RING_ECAPACITY if over else ra.RING_OK)
    assert sl.tolist() == ref.lens and nf.tolist() == [ref.n] and fr.tolist() == ref.free


def test_extend_and_trim_long_sequences():
    # sequences of several hundred pages, moved by the whole block; a free list that is full again
    need_cuda()
    ps, W = 8, 4000
    lens, news = [5, 16000, 0, 77, 1], [9000, 1, 20000, 0, 6400]
    table, free = _tables(lens, ps, W, 4600, 9)
    ref = R.Tables(lens, table, free, len(free), ps)
    sl, tb, fr, nf = ints(lens), ints(table), ints(free), ints([len(free)])
    slots, start, cu = ra.ring_attn_page_extend(sl, ints(news), tb, fr, nf, ps, max_tokens=sum(news) + 3)
    w_slots, w_start, w_cu, short = ref.extend(news, sum(news) + 3)
    ok()
    assert not short and slots.tolist() == w_slots and start.tolist() == w_start and cu.tolist() == w_cu
    assert np.array_equal(tb.cpu().numpy(), ref.table) and nf.tolist() == [ref.n]
    keep = [0, 16001, 0, 0, 100]
    ref.trim(keep)
    ra.ring_attn_page_trim(sl, ints(keep), tb, fr, nf, ps)
    ok()
    assert sl.tolist() == ref.lens and nf.tolist() == [ref.n] and fr.tolist() == ref.free


# ---------------------------------------------------------------- append
def make_pools(layout, N, ps, Hkv, D, dtype, fill=None):
    """k, v pools [N, ps, Hkv, D] in the memory layout named."""
    def new(*shape):
        return torch.zeros(shape, device="cuda", dtype=dtype)
    if layout == "plain":
        k, v = new(N, ps, Hkv, D), new(N, ps, Hkv, D)
    elif layout == "kv_page":          # K and V of a page next to each other
        both = new(N, 2, ps, Hkv, D)
        k, v = both[:, 0], both[:, 1]
    elif layout == "heads_first":      # pages of [Hkv, ps, D]
        k, v = (new(N, Hkv, ps, D).transpose(1, 2) for _ in range(2))
    elif layout == "kv_token":         # K and V of a token next to each other
        both = new(N, ps, 2, Hkv, D)
        k, v = both[:, :, 0], both[:, :, 1]
    else:                              # the tokens of a page far apart
        k, v = (new(ps, N, Hkv, D).transpose(0, 1) for _ in range(2))
    if fill is not None:
        k.copy_(fill[0])
        v.copy_(fill[1])
    return k, v


LAYOUTS = ["plain", "kv_page", "heads_first", "kv_token", "tokens_apart"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,T,Hkv,D,ps", [("bf16", 1, 1, 64, 8), ("bf16", 333, 3, 128, 16), ("fp32", 70, 2, 64, 32),
                                             ("fp32", 129, 8, 128, 8)])
def test_append_writes_its_slots_and_nothing_else(layout, dtype, T, Hkv, D, ps):
    need_cuda()
    N = R.cdiv(T, ps) + 3
    g = torch.Generator(device="cuda").manual_seed(T)
    rows = torch.randn((T, 5 + 2 * Hkv, D), generator=g, device="cuda").to(DT[dtype])
    kn, vn = rows[:, 5:5 + Hkv], rows[:, 5 + Hkv:]      # slices of a fused projection
    k, v = make_pools(layout, N, ps, Hkv, D, DT[dtype])
    rng = np.random.default_rng(T)
    slots = rng.permutation(N * ps)[:T].astype(np.int64)
    bad = {0: -1, 3: N * ps, 5: 2 ** 31 - 1, 6: -2 ** 31}
    for i, s in bad.items():
        if i < T and T > 1:
            slots[i] = s
    kw, vw = torch.zeros((N * ps, Hkv, D), dtype=DT[dtype]), torch.zeros((N * ps, Hkv, D), dtype=DT[dtype])
    for t, s in enumerate(slots):
        if 0 <= s < N * ps:
            kw[s], vw[s] = kn[t].cpu(), vn[t].cpu()
    ra.ring_attn_paged_append(k, v, kn, vn, ints(slots))
    ok()
    assert torch.equal(k.cpu().reshape(kw.shape), kw) and torch.equal(v.cpu().reshape(vw.shape), vw)


# ---------------------------------------------------------------- decode
def make_cache(lens, ps, Hkv, D, dtype, seed, layout="plain", W=None, garbage=True):
    """Pools, table (int32 device) for the lengths; rows past a length hold NaN or Inf."""
    W = W or max(1, R.cdiv(max(max(lens), 1), ps))
    table, _ = _tables(lens, ps, W, 2, seed)
    N = sum(R.cdiv(min(max(n, 0), W * ps), ps) for n in lens) + 2
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((N, ps, Hkv, D), generator=g).to(DT[dtype])
    v = torch.randn((N, ps, Hkv, D), generator=g).to(DT[dtype])
    if garbage:
        used = torch.zeros((N, ps), dtype=torch.bool)
        for b, n in enumerate(lens):
            for lp in range(R.cdiv(min(max(n, 0), W * ps), ps)):
                used[table[b, lp], :max(0, min(ps, n - lp * ps))] = True
        k[~used] = float("nan")
        v[~used] = float("inf")
    return make_pools(layout, N, ps, Hkv, D, DT[dtype], fill=(k.cuda(), v.cuda())) + (ints(table),)


def queries(B, Hq, D, dtype, seed, strided=True):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((B, Hq + 3, D), generator=g).to(DT[dtype]).cuda()
    return rows[:, :Hq] if strided else rows[:, :Hq].contiguous()


def check_decode(out, lse, ref, D):
    t_out, t_lse = R.tolerances(ref, D, out.dtype)
    o, l = out.cpu().double(), lse.cpu().double()
    none = torch.isneginf(ref[1])
    assert torch.equal(torch.isneginf(l), none) and not o[none].any()
    if (~none).any():
        margin("out", ((o - ref[0]).abs() / t_out)[~none].max(), 1.0)
        margin("lse", ((l - ref[1]).abs() / t_lse)[~none].max(), 1.0)


LENS = [0, 1, 7, 8, 127, 128, 129, 255, 1000, 2049]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (4, 4, 64, 8), (10, 2, 128, 32), (7, 1, 64, 64), (16, 1, 128, 128),
                                         (20, 1, 64, 16), (9, 3, 128, 256), (32, 2, 128, 8), (6, 3, 64, 1024),
                                         (70, 2, 128, 16)])
def test_decode_against_64_bits(dtype, Hq, Hkv, D, ps):
    need_cuda()
    k, v, tb = make_cache(LENS, ps, Hkv, D, dtype, 11 + Hq)
    q = queries(len(LENS), Hq, D, dtype, 5)
    ws = ra.decode_paged_workspace(D)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(LENS), workspace=ws)
    ok()
    ref = R.decode(q, k, v, tb, LENS, 1 / math.sqrt(D))
    check_decode(out, lse, ref, D)
    # the counters are zero again: the same call gives the same bits
    out2, lse2 = ra.ring_attn_decode_paged(q, k, v, tb, ints(LENS), workspace=ws)
    ok()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    if dtype == "bf16":
        o32, l32 = ra.ring_attn_decode_paged(q, k, v, tb, ints(LENS), workspace=ws, out_dtype=torch.float32)
        ok()
        check_decode(o32, l32, ref, D)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_pool_layouts_and_scale(layout, dtype):
    need_cuda()
    lens = [300, 33, 0, 700]
    k, v, tb = make_cache(lens, 16, 3, 128, dtype, 3, layout)
    q = queries(4, 12, 128, dtype, 6)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), scale=0.3)
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 0.3), 128)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hkv,lens", [(1, 4, 1, [60000]), (1, 32, 8, [20011]), (2, 2, 2, [40000, 3]), (1, 1, 1, [1])])
def test_decode_one_long_sequence_is_split_and_joined(dtype, B, Hq, Hkv, lens):
    need_cuda()
    k, v, tb = make_cache(lens, 64, Hkv, 128, dtype, 17)
    q = queries(B, Hq, 128, dtype, 8)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens))
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / math.sqrt(128)), 128)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_many_ragged_sequences(dtype):
    # more rows than a block has threads, most of them short or empty; lengths outside the table are clamped
    need_cuda()
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 60, 700)]
    lens[50:150] = [0] * 100
    lens[13], lens[77] = 700, 300
    W = 44
    k, v, tb = make_cache(lens, 16, 1, 64, dtype, 23, W=W)
    q = queries(700, 2, 64, dtype, 9)
    asked = list(lens)
    asked[60] = -5
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(asked))
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / 8), 64)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ps", [8, 64, 256])
def test_decode_table_entries_outside_the_pool_are_absent(dtype, ps):
    need_cuda()
    lens = [5 * ps + 3, 2 * ps, ps]
    k, v, tb = make_cache(lens, ps, 2, 64, dtype, 29)
    tb[0, 1], tb[0, 5], tb[2, 0] = -1, k.shape[0], 2 ** 31 - 1      # a middle page, the last page, the only page
    q = queries(3, 4, 64, dtype, 2)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens))
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / 8), 64)
    # lengths beyond the table are clamped to it
    long = [10 ** 6, 2 * ps, 2 ** 31 - 1]
    W = tb.shape[1]
    out, lse = ra.ring_attn_decode_paged(q[:1], k, v, tb[:1, :4], ints(long[:1]))
    ok()
    check_decode(out, lse, R.decode(q[:1], k, v, tb[:1, :4], [4 * ps], 1 / 8), 64)
    assert W == 6


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,D,ps,K", [(8, 2, 128, 16, 9), (12, 2, 64, 32, 5), (4, 4, 128, 8, 40), (40, 2, 64, 256, 3)])
def test_decode_selected_pages(dtype, Hq, Hkv, D, ps, K):
    need_cuda()
    lens = [20 * ps + 3, ps - 1, 0, 33 * ps]
    k, v, tb = make_cache(lens, ps, Hkv, D, dtype, 31, garbage=True)
    q = queries(4, Hq, D, dtype, 12)
    rng = np.random.default_rng(K)
    sel = np.full((4, Hkv, K), -1, dtype=np.int64)
    n_sel = np.zeros((4, Hkv), dtype=np.int64)
    for b in range(4):
        for g in range(Hkv):
            have = R.cdiv(lens[b], ps)
            pick = sorted(rng.permutation(have)[:K])
            sel[b, g, :len(pick)] = pick
            n_sel[b, g] = len(pick)
    sel[0, 0, 0] = 20                                   # the partly filled last page, out of order
    sel[3, 0, 1] = sel[3, 0, 0]                          # a page twice counts twice
    sel[3, 1, :2] = [-3, 10 ** 6]                        # outside the sequence: ignored
    n_sel[0, 1] = 0                                      # one head of a sequence reads nothing
    sel[2, 0, :2], n_sel[2, 0] = [0, 1], 2               # pages listed of an empty sequence
    n_sel[3, Hkv - 1] = K + 100                          # clamped to K
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), sel=ints(sel), n_sel=ints(n_sel))
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / math.sqrt(D), sel, n_sel), D)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hkv", [(20, 3), (90, 3)])
def test_decode_selected_pages_of_many_sequences(dtype, B, Hkv):
    # more lists than a warp has lanes, and than a block has threads
    need_cuda()
    ps, K, D = 8, 30, 64
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 500, B)]
    k, v, tb = make_cache(lens, ps, Hkv, D, dtype, 43)
    q = queries(B, 2 * Hkv, D, dtype, 44)
    sel = np.full((B, Hkv, K), -1, dtype=np.int64)
    n_sel = np.zeros((B, Hkv), dtype=np.int64)
    for b in range(B):
        for g in range(Hkv):
            pick = sorted(rng.permutation(R.cdiv(lens[b], ps))[:rng.integers(0, K + 1)])
            sel[b, g, :len(pick)] = pick
            n_sel[b, g] = len(pick)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), sel=ints(sel), n_sel=ints(n_sel))
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / 8, sel, n_sel), D)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 24, 8), (64, 16, 1)])
@pytest.mark.parametrize("B", [33, 140])
def test_decode_batches_of_medium_lengths(D, Hq, Hkv, B):
    # runs of whole segments and parts of several tiles, more rows than a warp has lanes
    need_cuda()
    rng = np.random.default_rng(D + B)
    lens = [int(x) for x in rng.integers(1, 2500, B)]
    lens[5], lens[B - 1] = 0, 0
    k, v, tb = make_cache(lens, 16, Hkv, D, "bf16", 47)
    q = queries(B, Hq, D, "bf16", 48)
    ws = ra.decode_paged_workspace(D)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), workspace=ws)
    ok()
    check_decode(out, lse, R.decode(q, k, v, tb, lens, 1 / math.sqrt(D)), D)
    for _ in range(5):
        o2, l2 = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), workspace=ws)
    ok()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_nan_and_infinite_scores(dtype):
    # a valid NaN key makes its sequence NaN (as the formula does); large scores do not overflow
    need_cuda()
    lens = [200, 300, 400]
    k, v, tb = make_cache(lens, 16, 1, 64, dtype, 37)
    page = int(tb[1, 3])
    k[page, 5, 0, 7] = float("nan")
    q = queries(3, 2, 64, dtype, 3, strided=False)
    q[2] *= 300                                          # scores of several thousand
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens))
    ok()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    ref = R.decode(q, k, v, tb, lens, 1 / 8)
    keep = [0, 2]
    check_decode(out[keep], lse[keep], tuple(x[keep] for x in ref), 64)
    assert torch.isfinite(out[keep]).all()


# ---------------------------------------------------------------- bounds, scores, selection
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", [("bf16", 8, 2, 128, 16), ("fp32", 5, 1, 64, 8), ("bf16", 6, 3, 64, 128),
                                               ("fp32", 32, 2, 128, 64)])
def test_bounds_and_scores(layout, dtype, Hq, Hkv, D, ps):
    need_cuda()
    lens = [0, 1, ps, ps + 1, 9 * ps - 3]
    k, v, tb = make_cache(lens, ps, Hkv, D, dtype, 41, layout)
    tb[4, 2] = -1                                        # an absent page
    sent = torch.full((k.shape[0], Hkv, 2, D), 77.0, device="cuda", dtype=DT[dtype])
    for start in (None, [0, 0, ps - 1, ps, 7 * ps]):
        b = sent.clone()
        ra.ring_attn_page_bounds(k, tb, ints(lens), bounds=b, start_lens=None if start is None else ints(start))
        ok()
        want = sent.clone().cpu()
        for pg, x in R.bounds(k, tb, lens, start).items():
            want[pg] = x
        assert torch.equal(b.cpu(), want)
        if start is None:
            full = b
    q = queries(len(lens), Hq, D, dtype, 14)
    sc = ra.ring_attn_page_scores(q, full, tb, ints(lens), ps)
    ok()
    ref, mag = R.scores(q, full, tb, lens, ps)
    none = torch.isneginf(ref)
    assert torch.equal(torch.isneginf(sc.cpu()), none)
    # D products rounded once each and D float32 additions
    tol = (2 * D * 2.0 ** -24 * mag + 1e-30)[~none]
    margin("scores", ((sc.cpu().double() - ref)[~none].abs() / tol).max(), 1.0)
    # no key of a page scores above it
    for i, n in enumerate(lens):
        for lp in range(R.cdiv(n, ps)):
            pg = int(tb[i, lp])
            if pg < 0:
                continue
            x = torch.einsum("hgd,rhd->hgr", q[i].cpu().double().view(Hkv, Hq // Hkv, D),
                             k[pg, :min(ps, n - lp * ps)].cpu().double()).amax((1, 2))
            assert (x <= ref[i, :, lp] + 1e-9).all()


def test_bounds_keep_a_nan():
    need_cuda()
    k = torch.randn((2, 8, 1, 64), device="cuda").to(torch.bfloat16)
    k[1, 3, 0, 9] = float("nan")
    b = ra.ring_attn_page_bounds(k, ints([[0, 1]]), ints([12]))
    ok()
    assert torch.isnan(b[1, 0, :, 9]).all() and int(torch.isnan(b).sum()) == 2


@pytest.mark.parametrize("W,K,first,last", [(1, 1, 0, 1), (40, 7, 1, 1), (40, 40, 3, 2), (1025, 100, 1, 2), (5000, 33, 0, 0),
                                            (40000, 1000, 4, 4), (300, 299, 1, 1), (64, 3, 3, 0)])
def test_select(W, K, first, last):
    need_cuda()
    ps = 16
    lens = [W * ps, 0, max(1, W * ps - ps - 3), min(W, K) * ps, 3, 10 ** 8]
    g = torch.Generator(device="cuda").manual_seed(W)
    sc = torch.randn((len(lens), 2, W), generator=g, device="cuda") * 3
    sc[0, 1] = torch.round(sc[0, 1])                      # many ties
    sc[2, 0] = -1.25                                      # all alike
    sc[2, 1, ::3] = float("-inf")
    sc[0, 0, W // 2] = float("nan")
    sc[5, 0] = torch.where(sc[5, 0] > 0, 0.0, -0.0)       # zeros of both signs are alike
    sel, n = ra.ring_attn_page_select(sc, ints(lens), ps, K, keep_first=first, keep_last=last)
    ok()
    w_sel, w_n = R.select(sc, lens, ps, K, first, last)
    assert np.array_equal(n.cpu().numpy(), w_n)
    assert np.array_equal(sel.cpu().numpy(), w_sel)


# ---------------------------------------------------------------- addresses, streams, graphs
def test_offsets_beyond_32_bits():
    # pools of 2.2e9 elements (4.4 GB each); the tokens lie in the last pages and in the first
    need_cuda()
    ps, Hkv, D = 64, 4, 128
    N = 2 ** 31 // (ps * Hkv * D) + 3000
    k = torch.empty((N, ps, Hkv, D), device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    n = 5 * ps - 7
    pages = [N - 1, 0, N - 2, 3, N - 3]
    tb = ints([pages])
    g = torch.Generator(device="cuda").manual_seed(3)
    kn = torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    vn = torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    slots = ints([pages[t // ps] * ps + t % ps for t in range(n)])
    ra.ring_attn_paged_append(k, v, kn, vn, slots)
    q = queries(1, 8, D, "bf16", 4)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb, ints([n]))
    bnd = ra.ring_attn_page_bounds(k, tb, ints([n]))
    sc = ra.ring_attn_page_scores(q, bnd, tb, ints([n]), ps)
    ok()
    # the same tokens in a pool of five pages
    small = [(x.new_zeros((5, ps, Hkv, D))) for x in (k, v)]
    for x, new in zip(small, (kn, vn)):
        x.view(-1, Hkv, D)[:n] = new
        x.view(-1, Hkv, D)[n:] = float("nan")
    stb = ints([[0, 1, 2, 3, 4]])
    out2, lse2 = ra.ring_attn_decode_paged(q, *small, stb, ints([n]))
    bnd2 = ra.ring_attn_page_bounds(small[0], stb, ints([n]))
    sc2 = ra.ring_attn_page_scores(q, bnd2, stb, ints([n]), ps)
    ok()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(bnd[pages], bnd2) and torch.equal(sc, sc2)
    check_decode(out2, lse2, R.decode(q, *small, stb, [n], 1 / math.sqrt(D)), D)


def test_two_streams_with_a_workspace_each():
    need_cuda()
    cases = []
    for seed, lens in ((51, [3000, 20, 777, 6000]), (52, [100, 9000, 0, 5])):
        k, v, tb = make_cache(lens, 16, 2, 128, "bf16", seed)
        q = queries(4, 8, 128, "bf16", seed)
        cases.append((q, k, v, tb, ints(lens), ra.decode_paged_workspace(128), torch.cuda.Stream()))
    want = [ra.ring_attn_decode_paged(*c[:5], workspace=c[5]) for c in cases]
    ok()
    got = []
    for _ in range(20):
        for c in cases:
            c[6].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(c[6]):
                got.append(ra.ring_attn_decode_paged(*c[:5], workspace=c[5]))
    ok()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_one_workspace_serves_calls_of_all_kinds_in_turn():
    need_cuda()
    ws = ra.decode_paged_workspace(128)
    cases = []
    for i, (dtype, D, Hq, Hkv, lens) in enumerate((("bf16", 128, 8, 2, [5000, 1300]), ("bf16", 64, 16, 1, [9000]),
                                                   ("fp32", 64, 4, 2, [3000, 7]), ("fp32", 128, 3, 1, [4000]),
                                                   ("bf16", 64, 2, 2, [700, 800, 0]))):
        k, v, tb = make_cache(lens, 16, Hkv, D, dtype, 80 + i)
        q = queries(len(lens), Hq, D, dtype, 81 + i)
        cases.append((q, k, v, tb, lens, D))
    for turn in range(3):
        got = [ra.ring_attn_decode_paged(*c[:4], ints(c[4]), workspace=ws) for c in cases]
        ok()
        for (o, l), c in zip(got, cases):
            check_decode(o, l, R.decode(*c[:4], c[4], 1 / math.sqrt(c[5])), c[5])


def test_two_graphs_that_share_a_workspace_follow_the_lengths():
    # captured calls read lengths, tables and lists on the device; replayed in turn on one stream
    need_cuda()
    k, v, tb = make_cache([4000] * 3, 16, 2, 64, "bf16", 61, garbage=False)
    q = queries(3, 16, 64, "bf16", 62)
    sl = ints([10, 2000, 4000])
    sel = ints([[[0, 3, 9, 200], [1, 2, 100, 249]]] * 3)
    n_sel = ints([[4, 3]] * 3)
    ws = ra.decode_paged_workspace(64)
    outs = [(torch.empty((3, 16, 64), device="cuda", dtype=torch.bfloat16), torch.empty((3, 16), device="cuda"))
            for _ in range(2)]

    def dense():
        ra.ring_attn_decode_paged(q, k, v, tb, sl, out=outs[0][0], out_lse=outs[0][1], workspace=ws)

    def sparse():
        ra.ring_attn_decode_paged(q, k, v, tb, sl, sel=sel, n_sel=n_sel, out=outs[1][0], out_lse=outs[1][1], workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dense()
        sparse()
    torch.cuda.synchronize()
    graphs = []
    for f in (dense, sparse):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f()
        graphs.append(gr)
    for lens, ns in (([10, 2000, 4000], 4), ([0, 1, 3999], 2), ([4000, 129, 128], 3)):
        sl.copy_(ints(lens))
        n_sel.fill_(ns)
        for gr in graphs:
            gr.replay()
        ok()
        check_decode(*outs[0], R.decode(q, k, v, tb, lens, 1 / 8), 64)
        check_decode(*outs[1], R.decode(q, k, v, tb, lens, 1 / 8, sel.cpu(), n_sel.cpu()), 64)


# ---------------------------------------------------------------- the operators together
@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", [("bf16", 8, 2, 128, 16), ("fp32", 4, 1, 64, 32)])
def test_serving_loop(dtype, Hq, Hkv, D, ps):
    """Prompts of different lengths are admitted and decoded step by step through
    a paged cache; one request ends, its pages go to a new one; every step's
    attention (all pages, and the selected ones) is compared with 64-bit
    attention over the request's own keys, and the whole step is replayed from
    a graph."""
    need_cuda()
    dt, B, W, N = DT[dtype], 4, 40, 60
    gen = torch.Generator(device="cuda").manual_seed(71)
    k_pool, v_pool = make_pools("kv_page", N, ps, Hkv, D, dt)
    k_pool.fill_(float("nan"))                       # rows that no token was written to
    v_pool.fill_(float("nan"))
    bounds = torch.full((N, Hkv, 2, D), float("nan"), device="cuda", dtype=dt)
    table = torch.full((B, W), -1, device="cuda", dtype=torch.int32)
    free = torch.arange(N, device="cuda", dtype=torch.int32)
    n_free, lens = ints([N]), ints([0] * B)
    ws = ra.decode_paged_workspace(D)
    keys = [[] for _ in range(B)]                    # the tokens each request has, on the host
    K = 4

    def admit(news):
        T = sum(news)
        kv = torch.randn((T, 2 * Hkv, D), generator=gen, device="cuda").to(dt)
        slots, start, cu = ra.ring_attn_page_extend(lens, ints(news), table, free, n_free, ps, max_tokens=T)
        ra.ring_attn_paged_append(k_pool, v_pool, kv[:, :Hkv], kv[:, Hkv:], slots)
        ra.ring_attn_page_bounds(k_pool, table, lens, bounds=bounds, start_lens=start)
        at = 0
        for b, n in enumerate(news):
            keys[b].append(kv[at:at + n].double().cpu())
            at += n

    # one step's buffers: a graph replays on them
    qkv = torch.zeros((B, Hq + 2 * Hkv, D), device="cuda", dtype=dt)
    one, order = ints([1, 1, 0, 1]), ints([0, 1, 3, 3])
    slots, start, cu = torch.empty(B, device="cuda", dtype=torch.int32), torch.empty(B, device="cuda", dtype=torch.int32), \
        torch.empty(B + 1, device="cuda", dtype=torch.int32)
    outs = [(torch.empty((B, Hq, D), device="cuda", dtype=dt), torch.empty((B, Hq), device="cuda")) for _ in range(2)]
    scores = torch.empty((B, Hkv, W), device="cuda")
    sel, n_sel = torch.empty((B, Hkv, K), device="cuda", dtype=torch.int32), torch.empty((B, Hkv), device="cuda", dtype=torch.int32)

    def step():
        q, kn, vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        ra.ring_attn_page_extend(lens, one, table, free, n_free, ps, slot_map=slots, start_lens=start, cu_new=cu)
        # the tokens, packed; the slot past them is -1
        ra.ring_attn_paged_append(k_pool, v_pool, kn.index_select(0, order), vn.index_select(0, order), slots)
        ra.ring_attn_page_bounds(k_pool, table, lens, bounds=bounds, start_lens=start)
        ra.ring_attn_decode_paged(q, k_pool, v_pool, table, lens, out=outs[0][0], out_lse=outs[0][1], workspace=ws)
        ra.ring_attn_page_scores(q, bounds, table, lens, ps, scores=scores)
        ra.ring_attn_page_select(scores, lens, ps, K, keep_first=1, keep_last=1, sel=sel, n_sel=n_sel)
        ra.ring_attn_decode_paged(q, k_pool, v_pool, table, lens, sel=sel, n_sel=n_sel, out=outs[1][0],
                                  out_lse=outs[1][1], workspace=ws)

    def check():
        n = [sum(x.shape[0] for x in r) for r in keys]
        assert lens.tolist() == n
        # what the references gather through the table is the tokens themselves
        tbl = table.cpu().numpy()
        for b in range(B):
            own = torch.cat(keys[b]) if keys[b] else torch.zeros((0, 2 * Hkv, D), dtype=torch.float64)
            assert torch.equal(R.keys_of(k_pool.cpu(), tbl[b], n[b], ps), own[:, :Hkv])
            assert torch.equal(R.keys_of(v_pool.cpu(), tbl[b], n[b], ps), own[:, Hkv:])
        q = qkv[:, :Hq]
        check_decode(*outs[0], R.decode(q, k_pool, v_pool, table, n, 1 / math.sqrt(D)), D)
        check_decode(*outs[1], R.decode(q, k_pool, v_pool, table, n, 1 / math.sqrt(D), sel.cpu(), n_sel.cpu()), D)
        w_sel, w_n = R.select(scores, n, ps, K, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), w_sel) and np.array_equal(n_sel.cpu().numpy(), w_n)
        ref, mag = R.scores(q, bounds, table, n, ps)
        none = torch.isneginf(ref)
        assert torch.equal(torch.isneginf(scores.cpu()), none)
        assert ((scores.cpu().double() - ref)[~none].abs() <= 2 * D * 2.0 ** -24 * mag[~none] + 1e-30).all()

    def feed():
        new = torch.randn(qkv.shape, generator=gen, device="cuda").to(dt)
        qkv.copy_(new)
        for b in (0, 1, 3):
            keys[b].append(new[b:b + 1, Hq:].double().cpu())

    admit([5 * ps + 3, ps - 1, 0, 12 * ps])
    feed()
    step()                                             # eager
    ok()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(ps + 2):                            # over a page's end
        feed()
        graph.replay()
        if i in (0, 1, ps, ps + 1):
            ok()
            check()
    ok()
    # request 3 ends; its pages serve a new prompt, and request 1 is rolled back by 3 tokens
    before = int(n_free)
    keep = lens.clone()
    keep[3] = 0
    keep[1] -= 3
    ra.ring_attn_page_trim(lens, keep, table, free, n_free, ps)
    assert int(n_free) > before + 12
    keys[3] = []
    flat = torch.cat(keys[1])
    keys[1] = [flat[:-3]]
    admit([0, 2, 0, 20 * ps + 1])
    feed()
    graph.replay()
    ok()
    check()
    # pages in use and pages free are all pages, once each
    n = lens.tolist()
    used = [int(table[b, i]) for b in range(B) for i in range(R.cdiv(n[b], ps))]
    assert sorted(used + free[:int(n_free)].tolist()) == list(range(N))
