"""Inputs and 64-bit references for chunk attention and the 8-bit cache.

The references resolve every position through its block table and work in
fp64; they share no code with the library.  attention() also returns what the
tolerances are made of: A = sum_j p_j |v_j| (the rounding of each probability
counts against it), the largest sum of |q_d k_d| and the largest score.
"""
import math

import torch


def make_tables(lens, block, gen, spare=3):
    """Block tables [n, widest] (int32, CPU) over a shuffled pool, unused entries -1, and the pool's blocks."""
    need = [-(-n // block) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=gen, dtype=torch.int64).to(torch.int32)
    tables = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        tables[i, :k] = perm[at:at + k]
        at += k
    return tables, pool


def slots_of(table, n, block):
    pos = torch.arange(n)
    return table[pos // block].long() * block + pos % block


def used_rows(tables, lens, block, pool):
    """Mask [pool * block] of the slots that hold a position of some sequence."""
    used = torch.zeros(pool * block, dtype=torch.bool)
    for i, n in enumerate(lens):
        used[slots_of(tables[i], n, block)] = True
    return used


def attention(q, k, v, first_pos, scale):
    """q [n, H, D] at positions first_pos .. over k, v [L, Hk, D], causal, in
    fp64.  Returns (out, A, sum |q k|, largest |score|)."""
    n, H, D = q.shape
    L, Hk, _ = k.shape
    g = H // Hk
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    amount = torch.zeros_like(out)
    dots, top = 0.0, 0.0
    for r in range(n):
        seen = min(L, first_pos + r + 1)
        if seen <= 0:
            continue
        kk, vv = k[:seen].repeat_interleave(g, 1), v[:seen].repeat_interleave(g, 1)
        s = torch.einsum("hd,lhd->hl", q[r], kk) * scale
        p = torch.softmax(s, -1)
        out[r] = torch.einsum("hl,lhd->hd", p, vv)
        amount[r] = torch.einsum("hl,lhd->hd", p, vv.abs())
        dots = max(dots, float((torch.einsum("hd,lhd->hl", q[r].abs(), kk.abs()) * abs(scale)).max()))
        top = max(top, float(s.abs().max()))
    return out, amount, dots, top


def tolerance(dtype, out, amount, dots, top, keys, D, p_eps):
    """Bound on |computed - out|.  Scores: a dot product of D fp32 terms is off
    by at most D 2^-24 sum|q k|, the product with scale * log2(e) and the
    subtraction of the maximum by 2^-22 |score|, 2^x by 2^-22: together d, which
    changes a weight by a factor within exp(+-d) and the normalised weights by
    twice that.  A probability is rounded by p_eps (0 where it stays fp32),
    sums over the keys add keys 2^-24 in the worst order.  The output is
    rounded by half a step of its type."""
    d = D * 2.0 ** -24 * dots + 2.0 ** -22 * (2 * top + 2)
    return (2 * math.expm1(d) + p_eps + (keys + 64) * 2.0 ** -23) * amount + torch.finfo(dtype).eps / 2 * (out.abs() + amount * d) + 1e-30


class Chunk:
    """A pa_prefill call: tensors on the GPU and the reference's pieces on the CPU."""

    def __init__(self, q_lens, seq_lens, H, Hk, D, block, dtype, seed, layout="row", lead=0, tail=0, spare=3):
        from paged_kv_cache_150_gb300 import inputs

        gen = torch.Generator().manual_seed(seed)
        self.q_lens, self.seq_lens, self.block, self.scale = q_lens, seq_lens, block, 1.0 / math.sqrt(D)
        self.tables, pool = make_tables(seq_lens, block, gen, spare)
        k = torch.randn(pool * block, Hk, D, generator=gen).to(dtype)
        v = torch.randn(pool * block, Hk, D, generator=gen).to(dtype)
        stale = ~used_rows(self.tables, seq_lens, block, pool)
        k[stale] = math.nan  # slots of no sequence: nothing may come from them
        v[stale] = math.nan
        self.k, self.v = k, v
        self.lead = lead
        cu = [lead]
        for n in q_lens:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.q = torch.randn(cu[-1] + tail, H, D, generator=gen).to(dtype)
        kc, vc = k.view(pool, block, Hk, D), v.view(pool, block, Hk, D)
        if layout == "split":
            kc, vc = inputs.to_split_layout(kc, vc)
        self.dev = dict(q=self.q.cuda(), k_cache=kc.contiguous().cuda(), v_cache=vc.contiguous().cuda(),
                        block_tables=self.tables.cuda(), seq_lens=torch.tensor(seq_lens, dtype=torch.int32).cuda(),
                        cu_q_lens=torch.tensor(cu, dtype=torch.int32).cuda(), scale=self.scale)

    def reference(self, i):
        n, L = self.q_lens[i], self.seq_lens[i]
        rows = slots_of(self.tables[i], L, self.block)
        return attention(self.q[self.cu[i]:self.cu[i + 1]].cuda(), self.k[rows].cuda(), self.v[rows].cuda(), L - n,
                         self.scale)

    def check(self, out, p_eps):
        for i, n in enumerate(self.q_lens):
            if n == 0:
                continue
            ref, amount, dots, top = self.reference(i)
            got = out[self.cu[i]:self.cu[i + 1]].double()
            tol = tolerance(out.dtype, ref, amount, dots, top, self.seq_lens[i], ref.shape[-1], p_eps)
            err = (got - ref).abs()
            assert torch.isfinite(got).all(), "sequence %d has values that are not finite" % i
            worst = float((err / tol).max())
            assert worst <= 1.0, "sequence %d: error %.3g, %.2f of the bound" % (i, float(err.max()), worst)
