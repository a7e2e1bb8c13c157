"""Plain 64-bit references of the paged-cache operators, one element at a time
from their definitions (numpy / float64 torch on the host)."""
import numpy as np
import torch


def cdiv(a, b):
    return -(-a // b)


class Tables:
    """Block tables, lengths and the free list, as ring_attn_page_extend and
    ring_attn_page_trim define them."""

    def __init__(self, lens, table, free, n_free, ps):
        self.lens, self.table = [int(x) for x in lens], np.array(table, dtype=np.int64)
        self.free, self.n, self.ps = list(map(int, free)), int(n_free), ps

    def extend(self, news, max_tokens):
        W, ps = self.table.shape[1], self.ps
        slots, start, cu, asked, short = [-1] * max_tokens, [], [0], 0, False
        top = self.n
        for b, new in enumerate(news):
            new = max(0, int(new))
            cu.append(cu[-1] + new)
            old = min(max(self.lens[b], 0), W * ps)
            if old + new > W * ps or (new and cu[-1] > max_tokens):
                start.append(-1)
                short = True
                continue
            need = cdiv(old + new, ps) - cdiv(old, ps)
            asked += need
            if need and asked > top:
                start.append(-1)
                short = True
                continue
            for i in range(need):
                self.n -= 1
                self.table[b, cdiv(old, ps) + i] = self.free[self.n]
            start.append(old)
            self.lens[b] = old + new
            for t in range(new):
                pos = old + t
                slots[cu[b] + t] = self.table[b, pos // ps] * ps + pos % ps
        return slots, start, cu, short

    def trim(self, keep):
        W, ps = self.table.shape[1], self.ps
        back = []
        for b, kp in enumerate(keep):
            old = min(max(self.lens[b], 0), W * ps)
            kp = min(max(int(kp), 0), old)
            back += [int(self.table[b, i]) for i in range(cdiv(kp, ps), cdiv(old, ps))]
            self.lens[b] = kp
        back = back[::-1]
        room = len(self.free) - self.n
        for p in back[:room]:
            self.free[self.n] = p
            self.n += 1
        return len(back) > room


def keys_of(pool, table_row, n, ps, pages=None):
    """(values [m, Hkv, D] float64 of the valid keys, in order) of one sequence;
    pages: logical pages to read instead of all."""
    N = pool.shape[0]
    W = len(table_row)
    n = min(max(int(n), 0), W * ps)
    rows = []
    for lp in (range(cdiv(n, ps)) if pages is None else pages):
        if lp < 0 or lp >= W:
            continue
        valid = min(ps, n - lp * ps)
        pg = int(table_row[lp])
        if valid <= 0 or pg < 0 or pg >= N:
            continue
        rows.append(pool[pg, :valid])
    if not rows:
        return pool.new_zeros((0,) + tuple(pool.shape[2:]), dtype=torch.float64)
    return torch.cat(rows).double()


def decode(q, k_pool, v_pool, table, lens, scale, sel=None, n_sel=None):
    """out [B,Hq,D], lse [B,Hq], and for the tolerances spread = sum_j p_j |v_j|
    [B,Hq,D] and mag = max_j scale * sum_d |q_d k_jd| [B,Hq], n keys [B,Hq]."""
    q, k_pool, v_pool = q.cpu(), k_pool.cpu(), v_pool.cpu()
    table = table.cpu().numpy()
    B, Hq, D = q.shape
    ps, Hkv = k_pool.shape[1], k_pool.shape[2]
    G = Hq // Hkv
    out, spread = torch.zeros((B, Hq, D), dtype=torch.float64), torch.zeros((B, Hq, D), dtype=torch.float64)
    lse, mag = torch.full((B, Hq), float("-inf"), dtype=torch.float64), torch.zeros((B, Hq), dtype=torch.float64)
    count = torch.zeros((B, Hq))
    for b in range(B):
        for g in range(Hkv):
            pages = None
            if sel is not None:
                m = min(max(int(n_sel[b, g]), 0), sel.shape[2])
                pages = [int(x) for x in sel[b, g, :m]]
            k = keys_of(k_pool, table[b], lens[b], ps, pages)[:, g]
            v = keys_of(v_pool, table[b], lens[b], ps, pages)[:, g]
            if k.shape[0] == 0:
                continue
            h = slice(g * G, (g + 1) * G)
            x = (q[b, h].double() @ k.T) * scale
            p = torch.softmax(x, -1)
            out[b, h], lse[b, h] = p @ v, torch.logsumexp(x, -1)
            spread[b, h] = p @ v.abs()
            mag[b, h] = ((q[b, h].double().abs() @ k.abs().T) * scale).amax(-1)
            count[b, h] = k.shape[0]
    return out, lse, spread, mag, count


def tolerances(ref, D, out_dtype):
    """Largest allowed |out - ref| and |lse - ref|.

    A score is a float32 sum of D products (each exact, or rounded once for a
    float32 cache): off by at most s = D 2^-23 mag (an accumulation step of the
    tensor cores may drop a whole last bit, 2^-23).  A weight is then off by
    e^s in itself and in the sum it is divided by, 2 s together, plus the
    exponential's few units (2^-20) and, where the weights enter a bf16
    product as two bf16 terms, the second term's rounding (2^-16); summing
    n terms in float32 adds n 2^-23 at most.  All of it scales sum_j p_j |v_j|.
    The output is rounded once: half a step of its type relative to itself."""
    out, lse, spread, mag, count = ref
    s = D * 2.0 ** -23 * mag
    rel = 2 * s + 2.0 ** -15 + (count + 200) * 2.0 ** -23
    half = torch.finfo(out_dtype).eps / 2
    return half * out.abs() + (rel[..., None] * spread) * (1 + half) + 1e-30, s + 2.0 ** -18 + 2.0 ** -21 * lse.abs()


def bounds(k_pool, table, lens, start=None):
    """{page: [Hkv, 2, D]} of the pages that hold tokens from start on."""
    k_pool, table = k_pool.cpu(), table.cpu().numpy()
    ps = k_pool.shape[1]
    got = {}
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * ps)
        s0 = 0 if start is None else max(int(start[b]), 0)
        for lp in range(s0 // ps, cdiv(n, ps)):
            pg = int(table[b, lp])
            if 0 <= pg < k_pool.shape[0]:
                x = k_pool[pg, :min(ps, n - lp * ps)]
                got[pg] = torch.stack([x.amin(0), x.amax(0)], dim=1)
    return got


def scores(q, bnd, table, lens, ps):
    """scores [B,Hkv,W] and their magnitude sums (for the tolerance)."""
    q, bnd, table = q.cpu().double(), bnd.cpu().double(), table.cpu().numpy()
    B, Hq, D = q.shape
    N, Hkv = bnd.shape[:2]
    G, W = Hq // Hkv, table.shape[1]
    res = torch.full((B, Hkv, W), float("-inf"), dtype=torch.float64)
    mag = torch.zeros((B, Hkv, W), dtype=torch.float64)
    for b in range(B):
        for lp in range(cdiv(min(max(int(lens[b]), 0), W * ps), ps)):
            pg = int(table[b, lp])
            if not 0 <= pg < N:
                continue
            x = bnd[pg].repeat_interleave(G, dim=0)                    # [Hq, 2, D]
            t = torch.maximum(q[b] * x[:, 0], q[b] * x[:, 1])
            res[b, :, lp] = t.sum(-1).view(Hkv, G).amax(-1)
            mag[b, :, lp] = t.abs().sum(-1).view(Hkv, G).amax(-1)
    return res, mag


def select(scores_, lens, ps, K, first, last):
    x = scores_.cpu().numpy().astype(np.float64)
    B, Hkv, W = x.shape
    sel = np.full((B, Hkv, K), -1, dtype=np.int64)
    n = np.zeros((B, Hkv), dtype=np.int64)
    for b in range(B):
        have = cdiv(min(max(int(lens[b]), 0), W * ps), ps)
        for g in range(Hkv):
            def rank(i):
                must = i < first or i >= have - last
                v = x[b, g, i]
                return (0 if must else 1 if np.isnan(v) else 2, 0.0 if must or np.isnan(v) else -v, i)
            best = sorted(sorted(range(have), key=rank)[:K])
            sel[b, g, :len(best)] = best
            n[b, g] = len(best)
    return sel, n
