"""GPU tests of the paged-cache operators where their inputs mark something as
missing: absent pages, sequences that were not served, full lists, infinities."""
import math

import numpy as np
import pytest
import torch

import context_exact_attention_ring_b200 as ra
from tests import paged_ref as R
from tests.helpers import margin, need_cuda

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Present(R.Tables):
    """The reference tables, whose trim gives no absent page back."""

    def trim(self, keep):
        ps, back = self.ps, []
        for b, kp in enumerate(keep):
            old = min(max(self.lens[b], 0), self.table.shape[1] * ps)
            kp = min(max(int(kp), 0), old)
            pages = [int(x) for x in self.table[b, R.cdiv(kp, ps):R.cdiv(old, ps)]]
            back += [p for p in pages if 0 <= p <= (2 ** 31 - 1) // ps]
            self.lens[b] = kp
        back, room = back[::-1], len(self.free) - self.n
        for p in back[:room]:
            self.free[self.n] = p
            self.n += 1
        return len(back) > room


@pytest.mark.parametrize("B,hi,room,ps", [(1, 90, 400, 16), (7, 400, 300, 8), (300, 400, 9000, 16), (300, 400, None, 16),
                                          (2500, 400, 70000, 16), (2500, 400, 20000, 16), (9, 20000, 12000, 16),
                                          (9, 20000, None, 16), (6, 20000, 3000, 32)])
def test_trim_gives_no_absent_page_back(B, hi, room, ps):
    # few pages (one a thread) and many (a warp to a sequence, the block together), several chunks of sequences, a
    # list that has room for the pages only without the absent ones, or not even then
    need_cuda()
    rng = np.random.default_rng(B + (room or 0))
    W = R.cdiv(hi, ps) + 50
    lens = [int(x) for x in rng.integers(1, hi, B)]
    need = [R.cdiv(n, ps) for n in lens]
    perm = rng.permutation(sum(need) + 300)
    table, at = np.full((B, W), -9, dtype=np.int64), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        gone = rng.random(n) < (0.3 if b % 3 else 0.0)
        table[b, :n][gone] = rng.choice([-1, -2 ** 31, 2 ** 31 - 1], int(gone.sum()))
        at += n
    if B == 1:
        table[0, 1] = -1
    free = list(perm[at:])
    keep = [0 if b % 2 == 0 else n // 2 for b, n in enumerate(lens)]
    if room is None:                                     # as many as come back
        fit = Present(lens, table, free + [0] * sum(need), len(free), ps)
        fit.trim(keep)
        room = fit.n
    ref = Present(lens, table, (free + [0] * room)[:room], min(len(free), room), ps)
    sl, tb, fr, nf = ints(lens), ints(table), ints(ref.free), ints([ref.n])
    ra.ring_attn_page_trim(sl, ints(keep), tb, fr, nf, ps)
    over = ref.trim(keep)
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == (ra.RING_ECAPACITY if over else ra.RING_OK)
    assert sl.tolist() == ref.lens and nf.tolist() == [ref.n] and fr[:ref.n].tolist() == ref.free[:ref.n]
    # another sequence gets pages, all of them
    news = [0] * B
    news[0] = min(ref.n, 40) * ps
    slots, start, cu = ra.ring_attn_page_extend(sl, ints(news), tb, fr, nf, ps, max_tokens=sum(news))
    want = ref.extend(news, sum(news))
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK
    assert slots.tolist() == want[0] and min(want[0]) >= 0 and start.tolist() == want[1] and nf.tolist() == [ref.n]


def test_extend_reports_a_list_entry_that_is_no_page():
    need_cuda()
    for bad in (-1, 2 ** 31 - 1):
        sl, tb, nf = ints([0, 3]), ints([[-5] * 3, [4, -5, -5]]), ints([3])
        slots, start, cu = ra.ring_attn_page_extend(sl, ints([20, 5]), tb, ints([7, bad, 2]), nf, 16, max_tokens=25)
        torch.cuda.synchronize()
        assert ra.ring_attn_device_error()[0] == ra.RING_ECAPACITY
        assert slots.tolist() == [2 * 16 + i for i in range(16)] + [-1] * 4 + [4 * 16 + i for i in range(3, 8)]
        assert tb.tolist() == [[2, bad, -5], [4, -5, -5]] and nf.tolist() == [1] and sl.tolist() == [20, 8]


def test_slot_map_of_2_to_the_31_entries():
    # the last block's entries end where 32-bit numbers do (8.6 GB)
    need_cuda()
    T, ps = 2 ** 31 - 1, 1024
    slot_map = torch.full((T,), 7, device="cuda", dtype=torch.int32)
    lens, news = [0] * 70, [3] * 70
    tb, free = ints([[-1]] * 70), ints(list(range(100)))
    slots, start, cu = ra.ring_attn_page_extend(ints(lens), ints(news), tb, free, ints([100]), ps, slot_map=slot_map)
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK
    assert slots[:210].tolist() == [(99 - t // 3) * ps + t % 3 for t in range(210)]
    for at in range(210, T, 1 << 28):
        part = slots[at:at + (1 << 28)]
        assert int(part.min()) == int(part.max()) == -1, at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bounds_of_sequences_without_new_tokens_are_left(dtype):
    # start_lens as page_extend leaves it: -1 for a sequence that found no room; its keys are not looked at
    need_cuda()
    ps, Hkv, D, lens = 16, 2, 64, [40, 48, 5, 33]
    k = torch.randn((16, ps, Hkv, D), device="cuda").to(dtype)
    tb = ints([[0, 1, 2, 15], [3, 4, 5, 15], [6, 15, 15, 15], [7, 8, 9, 15]])
    sl, nf = ints(lens), ints([1])
    slots, start, cu = ra.ring_attn_page_extend(sl, ints([1, 1, 5, 40]), tb, ints([10]), nf, ps, max_tokens=47)
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_ECAPACITY and start.tolist() == [40, 48, 5, -1]
    bnd = torch.full((16, Hkv, 2, D), 77.0, device="cuda", dtype=dtype)
    ra.ring_attn_page_bounds(k, tb, sl, bounds=bnd, start_lens=start)
    torch.cuda.synchronize()
    want = torch.full_like(bnd, 77.0).cpu()
    for pg, x in R.bounds(k, tb[:3], sl[:3].tolist(), start[:3].tolist()).items():
        want[pg] = x
    assert torch.equal(bnd.cpu(), want)
    # any negative start is "nothing new"
    ra.ring_attn_page_bounds(k, tb, sl, bounds=bnd.fill_(77.0), start_lens=ints([-1, -2 ** 31, -1, -7]))
    torch.cuda.synchronize()
    assert (bnd == 77.0).all() and ra.ring_attn_device_error()[0] == ra.RING_OK


@pytest.mark.parametrize("full", ["extend", "trim", "kv_append"])
def test_an_expired_wait_is_reported_beside_a_full_list(full):
    # a lack of room is everyday business; it hides no wait that ran out, before it or after it
    need_cuda()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK

    def lack():
        if full == "extend":
            ra.ring_attn_page_extend(ints([0]), ints([5]), ints([[0]]), ints([0]), ints([0]), 16, max_tokens=5)
        elif full == "trim":
            ra.ring_attn_page_trim(ints([5]), ints([0]), ints([[0]]), ints([0]), ints([1]), 16)
        else:
            c, new = torch.zeros((1, 4, 1, 8), device="cuda"), torch.zeros((1, 2, 1, 8), device="cuda")
            ra.ring_attn_kv_append(c, c.clone(), new, new, ints([[4]]), ints([4]), 1, 4)

    for first, second in ((lack, lambda: ra.ring_attn_selftest_wait(1000)), (lambda: ra.ring_attn_selftest_wait(1000), lack)):
        first()
        second()
        st, where = ra.ring_attn_device_error()
        assert st == ra.RING_ETIMEOUT and where == 11
        assert ra.ring_attn_device_error()[0] == ra.RING_ECAPACITY
        assert ra.ring_attn_device_error() == (ra.RING_OK, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 1), (128, 16, 2), (128, 12, 1), (64, 2, 2)])
@pytest.mark.parametrize("lens", [[300, 200], [9000, 40, 700]])
def test_decode_infinite_values(dtype, D, Hq, Hkv, lens):
    # a valid key's infinite value makes its dims infinite in every head, both signs make them NaN; the rest is as without
    need_cuda()
    ps = 16
    W = R.cdiv(max(lens), ps)
    g = torch.Generator().manual_seed(D + Hq)
    N = sum(R.cdiv(n, ps) for n in lens)
    k, v = (torch.randn((N, ps, Hkv, D), generator=g).to(dtype).cuda() for _ in range(2))
    tb, at = torch.full((len(lens), W), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        tb[b, :R.cdiv(n, ps)] = torch.arange(at, at + R.cdiv(n, ps))
        at += R.cdiv(n, ps)
    q = torch.randn((len(lens), Hq, D), generator=g).to(dtype).cuda()
    pos, neg, both = 5, 9, D - 1
    last = R.cdiv(lens[0], ps) - 2
    bad = v.clone()
    bad[2, 3, :, pos], bad[2, 4, :, neg], bad[2, 5, :, both], bad[last, 0, :, both] = (
        float("inf"), -float("inf"), float("inf"), -float("inf"))
    for out_dtype in {dtype, torch.float32}:
        ws = ra.decode_paged_workspace(D)
        want, lse0 = ra.ring_attn_decode_paged(q, k, v, tb.cuda(), ints(lens), workspace=ws, out_dtype=out_dtype)
        out, lse = ra.ring_attn_decode_paged(q, k, bad, tb.cuda(), ints(lens), workspace=ws, out_dtype=out_dtype)
        torch.cuda.synchronize()
        assert ra.ring_attn_device_error()[0] == ra.RING_OK
        assert torch.isposinf(out[0, :, pos]).all() and torch.isneginf(out[0, :, neg]).all()
        assert torch.isnan(out[0, :, both]).all() and torch.equal(lse, lse0)
        rest = torch.ones(out.shape, dtype=torch.bool, device="cuda")
        rest[0, :, [pos, neg, both]] = False
        assert torch.equal(out[rest], want[rest])


@pytest.mark.parametrize("n,Hq,D,ramp", [(1000003, 2, 128, 0.0), (400001, 16, 64, 0.0), (300007, 4, 128, 24.0),
                                         (100000, 9, 64, 24.0), (130001, 1, 128, 24.0), (70000, 8, 64, 0.0)])
def test_decode_sums_of_many_keys_to_a_cta(n, Hq, D, ramp):
    # more sequences than CTAs, all on the same pages, so that a CTA adds up whole sequences; values of one sign, so
    # that sums which lose their last bits are off by as much as they lose.  With a ramp the scores grow along the
    # sequence, and the running maximum with them.
    need_cuda()
    ps, B = 64, 150
    N = R.cdiv(n, ps)
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn((N, ps, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    if ramp:
        k[..., 0] = torch.linspace(0, ramp, N * ps, device="cuda").view(N, ps, 1).to(torch.bfloat16)
    v = (0.5 + torch.rand((N, ps, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    q = torch.randn((B, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    q[..., 0] = 16.0 if ramp else q[..., 0]
    tb = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    out, lse = ra.ring_attn_decode_paged(q, k, v, tb.repeat(B, 1), ints([n] * B), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ra.ring_attn_device_error()[0] == ra.RING_OK
    scale = 1 / math.sqrt(D)
    kk, vv = (x[tb.long()].view(-1, D)[:n].double() for x in (k, v))
    for b in (0, 77, B - 1):
        x = q[b].double() @ kk.T * scale
        s = D * 2.0 ** -23 * float((q[b].double().abs() @ kk.abs().T).max() * scale)
        want, l = torch.softmax(x, -1) @ vv, torch.logsumexp(x, -1)
        # the scores' error s, in a weight and in the sum of all; the weights' second terms, 2^-16, and exponentials,
        # 2^-20; up to 16 tiles of 128 terms that drop a last bit each, 2^-23, and then sums that round: one per 16
        # tiles in the outputs, one per tile in the weights'
        tol = 2 * s + 2.0 ** -15 + 16 * 128 * 2.0 ** -23 + (n / 2048 + n / 128 + 20) * 2.0 ** -24
        margin("out", ((out[b].double() - want) / want).abs().max(), tol)
        margin("lse", (lse[b].double() - l).abs().max(), s + 2.0 ** -18 + (n / 128 + 20) * 2.0 ** -24 + 2.0 ** -21 * float(l.abs().max()))
