"""The tables, the block-scaled cache and cross attention together, as a serving
loop of an encoder-decoder model uses them: requests come and go, their blocks
come off the GPU's stack, prompts and single tokens are written and attended to,
and every token looks at its request's encoder states.  One decode step is
captured into a graph and replayed."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _block8 import BF, E4M3, Block8
from _chunks import attention, slots_of, tolerance

pytestmark = pytest.mark.gpu
H, HK, D, B, NB, R, W = 16, 4, 128, 16, 220, 6, 40
SCALE = 1.0 / math.sqrt(D)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Loop:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.tables = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
        self.lens, self.count = torch.zeros(R, dtype=torch.int32, device="cuda"), i32([NB])
        self.free = torch.randperm(NB, generator=self.g, device="cuda", dtype=torch.int32)
        self.codes = [torch.full((NB, B, HK, D), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        self.scales = [torch.full((NB, HK), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        # encoder states in a pool of their own
        self.enc_lens = i32([70, 1, 257, 128, 33, 16])
        self.enc_tables = torch.randperm(120, generator=self.g, device="cuda", dtype=torch.int32).view(R, 20).contiguous()
        self.enc = [self.rand(120, B, HK, D) for _ in range(2)]

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(BF)

    def state(self):
        return self.tables, self.lens, self.free, self.count

    def step(self, rows, new, q, k, v, max_tokens):
        bt, sl, cu, slots = pa.pa_extend_tables(*self.state(), new, B, max_tokens, rows=rows)
        pa.pa_write_blocks_fp8(k, v, bt, sl, cu, *self.codes, *self.scales)
        own = pa.pa_prefill_fp8(q, *self.codes, *self.scales, bt, sl, cu, SCALE)
        cross = pa.pa_cross(q, *self.enc, self.enc_tables[rows.long()], self.enc_lens[rows.long()], cu, SCALE)
        return bt, sl, cu, slots, own, cross

    def check(self, rows, bt, sl, cu, q, own, cross, p_own=2.0 ** -8, tail=0.0):
        vals = [Block8.decoded(c.view(torch.uint8).cpu(), s.cpu()).view(NB * B, HK, D) for c, s in zip(self.codes, self.scales)]
        for i, r in enumerate(rows):
            lo, hi, L = int(cu[i]), int(cu[i + 1]), int(sl[i])
            if lo == hi:
                continue
            at = slots_of(bt[i].cpu(), L, B)
            kk, vv = vals[0][at].cuda(), vals[1][at].cuda()
            ref, amount, dots, top = attention(q[lo:hi], kk, vv, L - (hi - lo), SCALE)
            tol = tolerance(BF, ref, amount, dots, top, L, D, p_own) + tail * L * float(vv.abs().max())
            assert float(((own[lo:hi].double() - ref).abs() / tol).max()) <= 1.0
            n = int(self.enc_lens[r])
            at = slots_of(self.enc_tables[r].cpu(), n, B).cuda()
            ref, amount, dots, top = attention(q[lo:hi], self.enc[0].view(-1, HK, D)[at], self.enc[1].view(-1, HK, D)[at], n, SCALE)
            tol = tolerance(BF, ref, amount, dots, top, n, D, 2.0 ** -8)
            assert float(((cross[lo:hi].double() - ref).abs() / tol).max()) <= 1.0


def test_requests_come_and_go():
    s = Loop(70)
    rng = np.random.default_rng(70)
    for step in range(8):
        rows = [int(r) for r in rng.permutation(R)[:rng.integers(1, R + 1)]]
        new = [int(x) for x in rng.choice([0, 1, 1, 5, 90], len(rows))]
        T = sum(new) + 3
        q, k, v = s.rand(T, H, D), s.rand(T, HK, D) * 2.0 ** float(rng.integers(-3, 4)), s.rand(T, HK, D)
        bt, sl, cu, slots, own, cross = s.step(i32(rows), i32(new), q, k, v, T)
        assert pa.pa_get_device_error(raise_on_error=False) == 0
        s.check(rows, bt, sl, cu, q, own, cross)
        # the slots name the rows that the write filled
        live = slots[:sum(new)].long()
        back = pa.pa_gather_cache_fp8(*s.codes, *s.scales, slots)
        assert bool((slots[sum(new):] == -1).all()) and torch.count_nonzero(back[0][sum(new):]) == 0
        scale = torch.exp2(s.scales[0][live // B].float() - 127)[..., None]
        # half a step of the codes (2^-4 of a normal value), or of the smallest ones (2^-10 of the scale)
        x = k[:sum(new)].float()
        assert bool(((back[0][:sum(new)].float() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * scale).all())
        gone = [r for r in range(R) if int(s.lens[r]) > 150]
        pa.pa_release_tables(*s.state(), i32(gone), B)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    used = int(((s.lens + B - 1) // B).sum())
    assert int(s.count) == NB - used
    held = [int(b) for r in range(R) for b in s.tables[r, :-(-int(s.lens[r]) // B)]]
    assert sorted(held + s.free[:NB - used].tolist()) == list(range(NB))  # every block in one place


def test_a_captured_decode_step():
    s = Loop(71)
    prompts = [30, 1, 64, 16, 47, 100]
    T = sum(prompts)
    rows = i32(list(range(R)))
    q, k, v = s.rand(T, H, D), s.rand(T, HK, D), s.rand(T, HK, D)
    s.step(rows, i32(prompts), q, k, v, T)
    one = i32([1] * R)
    q, k, v = s.rand(R, H, D), s.rand(R, HK, D), s.rand(R, HK, D)
    out = (torch.zeros(R, W, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda"),
           torch.zeros(R + 1, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda"))
    own, cross = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()

    def step():
        pa.pa_extend_tables(*s.state(), one, B, R, out=out)
        bt, sl, cu, _ = out
        pa.pa_write_blocks_fp8(k, v, bt, sl, cu, *s.codes, *s.scales)
        pa.pa_decode_fp8(q, *s.codes, *s.scales, bt, sl, SCALE, out=own)
        pa.pa_cross(q, *s.enc, s.enc_tables, s.enc_lens, cu, SCALE, out=cross)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        for x in (q, k, v):
            x.copy_(s.rand(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert out[1].tolist() == [n + i + 1 for n in prompts]
        if i in (0, 1, 16, 19):
            s.check(list(range(R)), out[0], out[1], out[2], q, own, cross, 2.0 ** -11, 2.0 ** -25)
    assert pa.pa_get_device_error(raise_on_error=False) == 0


FIRST_CALLS = """
import torch
import paged_kv_cache_150_gb300 as pa

g = torch.Generator(device="cuda").manual_seed(19)
bf = torch.bfloat16
i32 = dict(dtype=torch.int32, device="cuda")
nb, b, hk, d, h, width = 40, 16, 8, 128, 32, 10
tables, lens, count = torch.full((4, width), -1, **i32), torch.tensor([17, 0, 3, 0], **i32), torch.tensor([nb - 3], **i32)
tables[0, :2], tables[2, 0] = torch.tensor([39, 38], **i32), 37
free, rows, done, new = torch.arange(nb, **i32), torch.tensor([3, 0], **i32), torch.tensor([2], **i32), torch.tensor([100, 5], **i32)
kept = [x.clone() for x in (tables, lens, count, free)]
k, v = (torch.randn(105, hk, d, generator=g, device="cuda").to(bf) for _ in range(2))
q, one = torch.randn(105, h, d, generator=g, device="cuda").to(bf), torch.randn(2, h, d, generator=g, device="cuda").to(bf)
codes = [torch.zeros(nb, b, hk, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
scales = [torch.full((nb, hk), 120, dtype=torch.uint8, device="cuda") for _ in range(2)]
enc = [torch.randn(nb, b, hk, d, generator=g, device="cuda").to(bf) for _ in range(2)]
enc_tables, seen = torch.randperm(nb, generator=g, **i32).view(2, 20).contiguous(), torch.tensor([300, 77], **i32)
few, cu_few = torch.randn(7, h, d, generator=g, device="cuda").to(bf), torch.tensor([0, 3, 7], **i32)
batch = (torch.zeros(2, width, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(128, **i32))
outs = [torch.zeros_like(q) for _ in range(4)] + [torch.zeros_like(one), torch.zeros_like(few), torch.zeros_like(few)]


def step():
    pa.pa_release_tables(tables, lens, free, count, done, b)
    bt, sl, cu, _ = pa.pa_extend_tables(tables, lens, free, count, new, b, 128, rows=rows, out=batch)
    pa.pa_write_blocks_fp8(k, v, bt, sl, cu, *codes, *scales)
    pa.pa_prefill_fp8(q, *codes, *scales, bt, sl, cu, 0.1, out=outs[0], kernel="mma")
    pa.pa_prefill_fp8(q, *codes, *scales, bt, sl, cu, 0.1, out=outs[1], kernel="simt")
    pa.pa_cross(q, *enc, enc_tables, seen, cu, 0.1, out=outs[2])
    pa.pa_cross(q, *enc, enc_tables, seen, cu, 0.1, out=outs[3], kernel="simt")
    pa.pa_decode_fp8(one, *codes, *scales, bt, sl, 0.1, out=outs[4])
    pa.pa_prefill_fp8(few, *codes, *scales, bt, sl, cu_few, 0.1, out=outs[5])
    pa.pa_cross(few, *enc, enc_tables, seen, cu_few, 0.1, out=outs[6])


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
state = (tables, lens, count, free)
results = (*batch, *outs, *state, *[c.view(torch.uint8) for c in codes], *scales)
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in results]
for x, y in zip(state, kept):
    x.copy_(y)
for x in outs:
    x.zero_()
step()
assert pa.pa_get_device_error(raise_on_error=False) == 0
for x, y in zip(got, results):
    assert torch.equal(x, y) and torch.count_nonzero(x)
print("captured first")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured first" in done.stdout, done.stderr[-2000:]


def test_calls_on_two_streams_at_once():
    """Chunks over the 8-bit cache, cross attention and tables of two batches, each on a stream of its own."""
    a, b = Loop(81), Loop(82)
    new = {a: [30, 1, 64, 5, 47, 100], b: [7, 90, 2, 33, 1, 12]}
    rows, data = i32(list(range(R))), {}
    for s in (a, b):
        T = sum(new[s])
        data[s] = (i32(new[s]), s.rand(T, H, D), s.rand(T, HK, D), s.rand(T, HK, D), T)
    torch.cuda.synchronize()
    got = {}
    for s in (a, b):
        s.stream = torch.cuda.Stream()
    for s in (a, b):
        with torch.cuda.stream(s.stream):
            got[s] = s.step(rows, *data[s])
    torch.cuda.synchronize()
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    for s in (a, b):
        bt, sl, cu, _, own, cross = got[s]
        assert sl.tolist() == new[s]
        s.check(list(range(R)), bt, sl, cu, data[s][1], own, cross)
