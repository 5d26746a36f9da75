"""The block manager, both caches, chunk attention and decode together, as a
serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _chunks import attention, tolerance

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, HK, D, B = 32, 8, 128, 16
SCALE = 1.0 / math.sqrt(D)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def check(out, q, k, v, first_pos, p_eps):
    ref, amount, dots, top = attention(q, k, v, first_pos, SCALE)
    tol = tolerance(out.dtype, ref, amount, dots, top, k.shape[0], D, p_eps)
    assert float(((out.double() - ref).abs() / tol).max()) <= 1.0


def test_prompt_in_chunks_then_samples():
    """A prompt written and attended to chunk by chunk, a second one behind its
    cached prefix, then forked samples that copy on write, over the plain and
    the 8-bit cache at once."""
    g = torch.Generator(device="cuda").manual_seed(50)
    rng = np.random.default_rng(50)
    nb = 200
    bm = pa.BlockManager(nb, B, rng.permutation(nb).astype(np.int32))
    kc, vc = (torch.full((nb, B, HK, D), math.nan, dtype=BF, device="cuda") for _ in range(2))
    codes = [torch.full((nb, B, HK, D), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((nb, B, HK), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def rows(n):
        return tuple(torch.randn(n, h, D, generator=g, device="cuda").to(BF) for h in (H, HK, HK))

    def write(k, v, slots):
        slots = i32(slots)
        pa.pa_reshape_and_cache(k, v, slots, kc, vc)
        pa.pa_reshape_and_cache_fp8(k, v, slots, *codes, *scales)

    # a prompt of 300 tokens in chunks of 128, 128 and 44
    tokens = rng.integers(0, 1000, 300)
    seq, cached = bm.new_seq_cached(tokens)
    assert cached == 0
    q, k, v = rows(300)
    at = 0
    for n in (128, 128, 44):
        write(k[at:at + n], v[at:at + n], bm.slots(seq, at, n))
        tables, _ = bm.export([seq], 32)
        out = pa.pa_prefill(q[at:at + n].contiguous(), kc, vc, i32(tables), i32([at + n]), i32([0, n]), SCALE)
        check(out, q[at:at + n], k[:at + n], v[:at + n], at, 2.0 ** -8)
        at += n

    # another prompt shares 200 tokens: 12 full blocks are in the cache
    tokens2 = np.concatenate([tokens[:200], rng.integers(1000, 2000, 77)])
    seq2, cached2 = bm.new_seq_cached(tokens2)
    assert cached2 == 192
    n2 = len(tokens2) - cached2
    q2, k2, v2 = rows(n2)
    write(k2, v2, bm.slots(seq2, cached2, n2))
    tables, lens = bm.export([seq, seq2], 32)
    # both in one ragged batch: the first one's last 5 tokens again, the second one's suffix
    out = pa.pa_prefill(torch.cat([q[295:], q2]), kc, vc, i32(tables), i32(lens), i32([0, 5, 5 + n2]), SCALE)
    check(out[:5], q[295:], k, v, 295, 2.0 ** -8)
    kk2, vv2 = torch.cat([k[:192], k2]), torch.cat([v[:192], v2])
    check(out[5:], q2, kk2, vv2, 192, 2.0 ** -8)

    # three samples of the first prompt: the partly filled block is copied on write
    samples = [seq] + [bm.fork(seq) for _ in range(2)]
    hist = {s: (k, v) for s in samples}
    for step in range(3):
        qs, ks, vs = rows(3)
        slots, pairs = [], []
        for s in samples:
            slot, pair = bm.append_token(s)
            slots.append(slot)
            pairs += [pair] if pair else []
        if pairs:
            pa.pa_copy_blocks(kc, vc, i32(pairs))
            pa.pa_copy_blocks_fp8(*codes, *scales, i32(pairs))
        assert (len(pairs) == 2) == (step == 0)
        write(ks, vs, slots)
        for n, s in enumerate(samples):
            hist[s] = (torch.cat([hist[s][0], ks[n:n + 1]]), torch.cat([hist[s][1], vs[n:n + 1]]))
        tables, lens = bm.export(samples, 32)
        tables, lens = i32(tables), i32(lens)
        out = pa.pa_decode(qs, kc, vc, tables, lens, SCALE)
        same = pa.pa_prefill(qs, kc, vc, tables, lens, i32([0, 1, 2, 3]), SCALE)
        out8 = pa.pa_decode_fp8(qs, *codes, *scales, tables, lens, SCALE)
        for n, s in enumerate(samples):
            L = 301 + step
            check(out[n:n + 1], qs[n:n + 1], *hist[s], L - 1, 2.0 ** -8)
            check(same[n:n + 1], qs[n:n + 1], *hist[s], L - 1, 2.0 ** -8)
            # the 8-bit cache's own values, read back
            k8, v8 = pa.pa_gather_cache_fp8(*codes, *scales, i32(bm.slots(s, 0, L)), dtype=torch.float32)
            check(out8[n:n + 1], qs[n:n + 1], k8, v8, L - 1, 2.0 ** -10)
            # and they are within half a step of e4m3 of what was written (or of its smallest step)
            x = hist[s][0].float()
            unit = x.abs().amax(-1, keepdim=True) * 2.0 ** -16
            assert bool(((k8 - x).abs() <= x.abs() * 2.0 ** -4 + unit).all())
    # rows read back are a pool of their own: chunk attention over the 8-bit cache
    L = 303
    k8, v8 = pa.pa_gather_cache_fp8(*codes, *scales, i32(np.append(bm.slots(seq, 0, L), -1)))
    pool = [x.view(-1, B, HK, D) for x in (k8, v8)]
    out = pa.pa_prefill(q[:64].contiguous(), *pool, torch.arange(19, dtype=torch.int32, device="cuda")[None].contiguous(),
                        i32([L]), i32([0, 64]), SCALE)
    check(out, q[:64], k8[:L], v8[:L], L - 64, 2.0 ** -8)
    assert pa.pa_get_device_error(raise_on_error=False) == 0


FIRST_CALLS = """
import sys
import torch
import paged_kv_cache_150_gb300 as pa

g = torch.Generator(device="cuda").manual_seed(9)
bf = torch.bfloat16
i32 = dict(dtype=torch.int32, device="cuda")
nb, b, hk, d, h = 12, 16, 8, 128, 32
kc, vc = (torch.randn(nb, b, hk, d, generator=g, device="cuda").to(bf) for _ in range(2))
q, one = torch.randn(40, h, d, generator=g, device="cuda").to(bf), torch.randn(2, h, d, generator=g, device="cuda").to(bf)
codes = [torch.zeros(nb, b, hk, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
scales = [torch.full((nb, b, hk), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
back = [torch.empty(nb * b, hk, d, dtype=bf, device="cuda") for _ in range(2)]
slots, pairs = torch.arange(nb * b, **i32), torch.tensor([[2, 10], [3, 11]], **i32)
tables = torch.tensor([[4, 1, 0, 5], [11, 10, 9, 2]], **i32)
lens, cu = torch.tensor([60, 33], **i32), torch.tensor([0, 30, 40], **i32)
out, out32, out8 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(one)


def step():
    pa.pa_reshape_and_cache_fp8(kc.view(-1, hk, d), vc.view(-1, hk, d), slots, *codes, *scales)
    pa.pa_copy_blocks_fp8(*codes, *scales, pairs)
    pa.pa_decode_fp8(one, *codes, *scales, tables, lens, 0.1, out=out8)
    pa.pa_gather_cache_fp8(*codes, *scales, slots, k=back[0], v=back[1])
    pa.pa_prefill(q, kc, vc, tables, lens, cu, 0.1, out=out)
    pa.pa_prefill(q, kc, vc, tables, lens, cu, 0.1, out=out32, kernel="simt")


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (out, out32, out8, *back, *scales)]
for x in (out, out32, out8, *back):
    x.zero_()
step()
assert pa.pa_get_device_error(raise_on_error=False) == 0
for x, y in zip(got, (out, out32, out8, *back, *scales)):
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
