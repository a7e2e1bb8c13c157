"""GPU tests of the paged-cache operators as a program strings them together:
long tables, shards that are merged, captured steps on a shared workspace,
device memory."""
import math

import pytest
import torch

import context_exact_attention_ring_b200 as ra
from tests import paged_ref as R
from tests.helpers import margin, need_cuda
from tests.test_gpu_paged import check_decode, ints, make_cache, queries

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([6001 * 8 - 3], 16, 8, 128), ([9 * 8, 0, 5 * 8 + 1, 4000 * 8 + 5] + [17] * 36, 8, 8, 64)])
def test_bounds_and_scores_of_long_tables(dtype, lens, Hq, Hkv, D):
    # more columns and pages than the grids of the two kernels take at once
    need_cuda()
    ps, B = 8, len(lens)
    need = [R.cdiv(n, ps) for n in lens]
    W, N = max(need) + 3, sum(need) + 2
    g = torch.Generator(device="cuda").manual_seed(W)
    k = torch.randn((N, ps, Hkv, D), generator=g, device="cuda").to(dtype)
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    tb, at = torch.full((B, W), -1, device="cuda", dtype=torch.int32), 0
    for b, n in enumerate(need):
        tb[b, :n] = perm[at:at + n]
        at += n
    tb[lens.index(max(lens)), max(need) // 2] = -1
    q = torch.randn((B, Hq, D), generator=g, device="cuda").to(dtype)
    bnd = ra.ring_attn_page_bounds(k, tb, ints(lens), bounds=torch.full((N, Hkv, 2, D), 77.0, device="cuda", dtype=dtype))
    sc = ra.ring_attn_page_scores(q, bnd, tb, ints(lens), ps)
    ok()
    want = torch.full_like(bnd, 77.0)
    pos = torch.arange(ps, device="cuda")
    for b, n in enumerate(lens):
        ref, mag = torch.full((Hkv, W), -math.inf, device="cuda", dtype=torch.float64), torch.zeros((Hkv, W), device="cuda")
        pages = tb[b, :need[b]].long()
        here = pages >= 0
        rows = k[pages.clamp(min=0)].double()
        live = (torch.arange(need[b], device="cuda")[:, None] * ps + pos < n)[:, :, None, None]
        lo, hi = torch.where(live, rows, math.inf).amin(1), torch.where(live, rows, -math.inf).amax(1)
        want[pages[here]] = torch.stack([lo, hi], 2)[here].to(dtype)
        for h in range(Hq):
            x, j = q[b, h].double(), h // (Hq // Hkv)
            t = torch.maximum(x * lo[:, j], x * hi[:, j])
            r = torch.where(here, t.sum(-1), -math.inf)
            ref[j, :need[b]] = torch.maximum(ref[j, :need[b]], r)
            mag[j, :need[b]] = torch.maximum(mag[j, :need[b]], t.abs().sum(-1).float())
        none = torch.isneginf(ref)
        assert torch.equal(torch.isneginf(sc[b]), none)
        if not bool(none.all()):
            # D products rounded once each and D float32 additions
            margin("scores", ((sc[b].double() - ref).abs() / (2 * D * 2.0 ** -24 * mag + 1e-30))[~none].max(), 1.0)
    assert torch.equal(bnd, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 6)])
def test_shards_of_a_sequence_merge(dtype, D, Hq, Hkv):
    # each rank holds some of a sequence's pages; the float32 partial outputs and lse merge to the whole sequence's
    need_cuda()
    lens, ps, P = [3000, 16 * 40, 5, 0], 16, 3
    k, v, tb = make_cache(lens, ps, Hkv, D, dtype, 91)
    q = queries(len(lens), Hq, D, dtype, 92)
    whole, wl = ra.ring_attn_decode_paged(q, k, v, tb, ints(lens), out_dtype=torch.float32)
    parts = torch.empty((len(lens), Hq, P, D), device="cuda")
    plse = torch.empty((len(lens), Hq, P), device="cuda")
    for p in range(P):
        # rank p has the pages i with i % P == p: the table and length of its shard
        W = R.cdiv(tb.shape[1], P)
        mine, ml = torch.zeros((len(lens), W), device="cuda", dtype=torch.int32), []
        for b, n in enumerate(lens):
            pages = list(range(p, R.cdiv(n, ps), P))
            mine[b, :len(pages)] = tb[b, pages]
            ml.append(sum(min(ps, n - i * ps) for i in pages))
        parts[:, :, p], plse[:, :, p] = ra.ring_attn_decode_paged(q, k, v, mine, ints(ml), out_dtype=torch.float32)
    out, lse = ra.ring_attn_merge(parts, plse, dtype=torch.float32)
    ok()
    ref = R.decode(q, k, v, tb, lens, 1 / math.sqrt(D))
    check_decode(whole, wl, ref, D)
    check_decode(out, lse, ref, D)


def test_captured_calls_on_one_workspace_after_an_ordered_warm_up():
    # the workspace is zeroed on the stream that is current then: another stream waits for it before its first call
    need_cuda()
    lens = [10, 2000, 4000]
    k, v, tb = make_cache([4000] * 3, 16, 2, 64, "bf16", 61, garbage=False)
    q, sl = queries(3, 16, 64, "bf16", 62), ints(lens)
    sel, n_sel = ints([[[0, 3, 9, 200], [1, 2, 100, 249]]] * 3), ints([[4, 3]] * 3)
    ws = ra.decode_paged_workspace(64)
    outs = [(torch.empty((3, 16, 64), device="cuda", dtype=torch.bfloat16), torch.empty((3, 16), device="cuda"))
            for _ in range(2)]
    calls = [lambda i=i, kw=kw: ra.ring_attn_decode_paged(q, k, v, tb, sl, out=outs[i][0], out_lse=outs[i][1], workspace=ws,
                                                         **kw) for i, kw in enumerate((dict(), dict(sel=sel, n_sel=n_sel)))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for f in calls:
            f()
    torch.cuda.current_stream().wait_stream(side)
    for f in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for lens, ns in (([10, 2000, 4000], 4), ([0, 1, 3999], 2), ([4000, 129, 128], 3)):
        sl.copy_(ints(lens))
        n_sel.fill_(ns)
        for _ in range(3):
            for gr in graphs:
                gr.replay()
        ok()
        check_decode(*outs[0], R.decode(q, k, v, tb, lens, 1 / 8), 64)
        check_decode(*outs[1], R.decode(q, k, v, tb, lens, 1 / 8, sel.cpu(), n_sel.cpu()), 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_library_allocates_nothing(dtype):
    need_cuda()
    B, Hq, Hkv, D, ps, W, N, K = 4, 8, 2, 128, 16, 64, 300, 8
    k, v = (torch.zeros((N, ps, Hkv, D), device="cuda", dtype=dtype) for _ in range(2))
    rows = torch.zeros((B * 200, Hkv, D), device="cuda", dtype=dtype)
    q, out = (torch.zeros((B, Hq, D), device="cuda", dtype=dtype) for _ in range(2))
    lse, ws = torch.empty((B, Hq), device="cuda"), ra.decode_paged_workspace(D)
    tb, free, sl, nf = ints([[-1] * W] * B), ints(list(range(N))), ints([0] * B), ints([N])
    new, keep, slots, start, cu = ints([200] * B), ints([0] * B), ints([0] * B * 200), ints([0] * B), ints([0] * (B + 1))
    bnd = torch.zeros((N, Hkv, 2, D), device="cuda", dtype=dtype)
    sc = torch.empty((B, Hkv, W), device="cuda")
    sel, n_sel = ints([[[0] * K] * Hkv] * B), ints([[0] * Hkv] * B)

    def step():
        ra.ring_attn_page_extend(sl, new, tb, free, nf, ps, slot_map=slots, start_lens=start, cu_new=cu)
        ra.ring_attn_paged_append(k, v, rows, rows, slots)
        ra.ring_attn_page_bounds(k, tb, sl, bounds=bnd, start_lens=start)
        ra.ring_attn_page_scores(q, bnd, tb, sl, ps, scores=sc)
        ra.ring_attn_page_select(sc, sl, ps, K, sel=sel, n_sel=n_sel)
        ra.ring_attn_decode_paged(q, k, v, tb, sl, out=out, out_lse=lse, workspace=ws)
        ra.ring_attn_decode_paged(q, k, v, tb, sl, sel=sel, n_sel=n_sel, out=out, out_lse=lse, workspace=ws)
        ra.ring_attn_page_trim(sl, keep, tb, free, nf, ps)

    step()                 # loads the kernels
    ok()
    free_bytes, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(20):
        step()
    assert torch.cuda.memory_allocated() <= held
    ok()
    assert torch.cuda.mem_get_info()[0] >= free_bytes
