"""Chunk attention (pa_prefill) against fp64, over types, head layouts, block
sizes, lengths and splits; masks that leave a row empty, values that are not
finite in masked places, bad pages and offsets, streams and graphs."""
import math

import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _chunks import Chunk, tolerance

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
P_EPS = {BF: 2.0 ** -8, F32: 0.0}  # the tensor-core kernel rounds probabilities to bf16


def run(c, **kw):
    out = pa.pa_prefill(**c.dev, **kw)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    return out


RAGGED = ([5, 1, 0, 130, 64, 33, 7], [5, 300, 17, 130, 191, 1000, 129])
SHAPES = [
    # H, Hk, D, block, dtype
    (4, 4, 64, 4, F32), (32, 8, 128, 16, F32), (6, 2, 128, 16, F32), (4, 2, 256, 16, F32),
    (32, 8, 128, 16, BF), (8, 8, 128, 16, BF), (16, 2, 64, 32, BF), (12, 4, 128, 16, BF), (7, 1, 64, 64, BF),
    (8, 1, 128, 128, BF), (64, 1, 128, 16, BF), (8, 2, 128, 8, BF), (8, 2, 128, 24, BF), (8, 2, 128, 256, BF),
    (8, 2, 128, 5, BF), (4, 2, 256, 16, BF),
]


@pytest.mark.parametrize("H,Hk,D,block,dtype", SHAPES)
def test_ragged_chunks(H, Hk, D, block, dtype):
    c = Chunk(*RAGGED, H, Hk, D, block, dtype, seed=H * 1000 + D + block)
    c.check(run(c), P_EPS[dtype])


@pytest.mark.parametrize("dtype,D,block", [(F32, 64, 4), (F32, 128, 16), (BF, 128, 16), (BF, 64, 32)])
def test_split_layout(dtype, D, block):
    c = Chunk(*RAGGED, 8, 2, D, block, dtype, seed=11, layout="split")
    c.check(run(c), P_EPS[dtype])


@pytest.mark.parametrize("kernel", ["auto", "simt"])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 1000])
def test_any_split_count(kernel, splits):
    c = Chunk([3, 200, 1, 70], [3000, 200, 700, 1025], 8, 2, 128, 16, BF, seed=5)
    c.check(run(c, kernel=kernel, num_splits=splits), P_EPS[BF])


@pytest.mark.parametrize("kernel", ["auto", "simt"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_around_tile_edges(kernel, n):
    c = Chunk([n, 1, n, min(n, 3)], [n, n, n + 128, n + 1], 8, 2, 128, 16, BF, seed=n)
    c.check(run(c, kernel=kernel), P_EPS[BF])


def test_long_context_few_rows():
    c = Chunk([4, 1, 2], [20000, 9001, 127], 32, 8, 128, 16, BF, seed=9)
    c.check(run(c), P_EPS[BF])


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_large_scores_move_the_running_maximum(kernel):
    """Scores that grow along the sequence by far more than the slack of a lazy maximum."""
    c = Chunk([40, 9], [900, 400], 8, 2, 128, 16, BF, seed=3)
    ramp = torch.linspace(0.05, 12.0, c.k.shape[0]).view(-1, 1, 1)
    for i, L in enumerate(c.seq_lens):
        from _chunks import slots_of
        rows = slots_of(c.tables[i], L, 16)
        c.k[rows] = (c.k[rows].float() * ramp[:L]).to(BF)
    c.dev["k_cache"] = c.k.view(c.dev["k_cache"].shape).cuda()
    c.check(run(c, kernel=kernel), P_EPS[BF])


@pytest.mark.parametrize("dtype,kernel", [(BF, "auto"), (BF, "simt"), (F32, "auto")])
def test_rows_that_see_nothing_are_zero(dtype, kernel):
    """More new tokens than positions: the first rows stand before position 0."""
    c = Chunk([150, 9, 4], [20, 9, 0], 8, 2, 128, 16, dtype, seed=4)
    out = run(c, kernel=kernel)
    c.check(out, P_EPS[dtype])
    assert torch.count_nonzero(out[:130]) == 0 and torch.count_nonzero(out[159:163]) == 0


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_rows_of_no_sequence_stay(kernel):
    c = Chunk([5, 40], [70, 40], 8, 2, 128, 16, BF, seed=6, lead=3, tail=7)
    out = torch.full_like(c.dev["q"], 7.0)
    run(c, out=out, kernel=kernel)
    c.check(out, P_EPS[BF])
    assert bool((out[:3] == 7).all()) and bool((out[48:] == 7).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,kernel", [(BF, "auto"), (BF, "simt"), (F32, "auto")])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, kernel, value):
    """K and V of a chunk's later tokens are masked for its earlier rows."""
    c = Chunk([40, 200], [100, 200], 8, 2, 128, 16, dtype, seed=8)
    from _chunks import slots_of
    bad_pos = [80, 150]  # rows 0..19 and 0..149 do not see these
    for i, p in enumerate(bad_pos):
        row = slots_of(c.tables[i], c.seq_lens[i], 16)[p]
        c.v[row, 1, 5] = value
        c.k[row, 0, 3] = value
    dev = dict(c.dev, k_cache=c.k.view(c.dev["k_cache"].shape).cuda(), v_cache=c.v.view(c.dev["v_cache"].shape).cuda())
    out = pa.pa_prefill(**dev, kernel=kernel)
    clean = run(c, kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    assert torch.equal(out[:20], clean[:20]) and torch.equal(out[40:190], clean[40:190])
    # V's value reaches the rows that see it, in its head and element only
    assert not torch.isfinite(out[20:40, 4:, 5]).any() and not torch.isfinite(out[190:, 4:, 5]).any()
    assert torch.isfinite(out[20:40, 4:, :5]).all() and torch.isfinite(out[190:, 4:, 6:]).all()


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_same_bits_every_time(kernel):
    c = Chunk([3, 200, 1, 70], [5000, 200, 700, 1025], 32, 8, 128, 16, BF, seed=12)
    a = run(c, kernel=kernel)
    for _ in range(3):
        assert torch.equal(a, run(c, kernel=kernel))


def test_one_new_token_is_decode():
    c = Chunk([1] * 5, [1, 16, 17, 500, 3001], 32, 8, 128, 16, BF, seed=13)
    d = c.dev
    one = pa.pa_decode(d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["seq_lens"], c.scale)
    got = run(c)
    c.check(one, P_EPS[BF])
    c.check(got, P_EPS[BF])


@pytest.mark.parametrize("dtype,kernel", [(BF, "auto"), (BF, "simt"), (F32, "auto")])
def test_bad_pages_read_zeros_and_are_recorded(dtype, kernel):
    c = Chunk([30, 8], [200, 60], 8, 2, 128, 16, dtype, seed=14)
    tables = c.tables.clone()
    pool = c.dev["k_cache"].shape[0]
    zero = [(0, 3, pool), (0, 7, -5), (1, 0, 2 ** 31 - 1)]
    from _chunks import slots_of
    for i, b, x in zero:
        rows = slots_of(c.tables[i], c.seq_lens[i], 16)[b * 16:(b + 1) * 16]
        c.k[rows], c.v[rows] = 0, 0
        tables[i, b] = x
    out = pa.pa_prefill(**dict(c.dev, block_tables=tables.cuda()), kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    c.check(out, P_EPS[dtype])


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_bad_offsets_and_lengths(kernel):
    c = Chunk([30, 8], [200, 60], 8, 2, 128, 16, BF, seed=15)
    for cu in ([0, 39, 38], [-1, 30, 38], [0, 30, 39], [0, 2 ** 31 - 1, 38]):
        out = torch.full_like(c.dev["q"], 3.0)
        pa.pa_prefill(**dict(c.dev, cu_q_lens=torch.tensor(cu, dtype=torch.int32).cuda()), out=out, kernel=kernel)
        assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
        assert bool((out == 3).all())
    reach = c.tables.shape[1] * 16
    for bad in (-1, reach + 1, 2 ** 31 - 1):
        lens = torch.tensor([bad, 60], dtype=torch.int32).cuda()
        out = pa.pa_prefill(**dict(c.dev, seq_lens=lens), kernel=kernel)
        assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
        assert torch.count_nonzero(out[:30]) == 0
        ref, amount, dots, top = c.reference(1)
        assert float((out[30:].double() - ref).abs().max()) < 0.05


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_offsets_past_32_bits(kernel):
    """Blocks at the far end of a pool of more than 2^31 elements."""
    block, Hk, D, H = 16, 8, 128, 32
    pool = (2 ** 31 + 2 ** 28) // (block * Hk * D)
    c = Chunk([20], [100], H, Hk, D, block, BF, seed=16)
    need = c.tables.shape[1]
    far = torch.arange(pool - need, pool, dtype=torch.int32)
    caches = []
    for x in (c.k, c.v):
        big = torch.empty(pool, block, Hk, D, dtype=BF, device="cuda")
        big[far.long()] = x.view(-1, block, Hk, D)[c.tables[0].long()].cuda()
        caches.append(big)
    out = pa.pa_prefill(**dict(c.dev, k_cache=caches[0], v_cache=caches[1], block_tables=far[None].contiguous().cuda()),
                        kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    c.check(out, P_EPS[BF])


def test_side_stream_and_captured_graphs_that_share_a_workspace():
    a = Chunk([30, 100], [700, 100], 32, 8, 128, 16, BF, seed=17)
    b = Chunk([7, 64, 1], [90, 640, 2000], 32, 8, 128, 16, BF, seed=18)
    need = max(pa.pa_prefill_workspace_bytes(x.dev["k_cache"], x.dev["q"].shape[0], len(x.q_lens), 32) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x.dev["q"]) for x in (a, b)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x, o in zip((a, b), outs):
            pa.pa_prefill(**x.dev, out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    want = [o.clone() for o in outs]
    a.check(want[0], P_EPS[BF])
    b.check(want[1], P_EPS[BF])
    graphs = []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_prefill(**x.dev, out=o, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1, 0)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])


def test_empty_calls():
    c = Chunk([0, 0], [5, 9], 8, 2, 128, 16, BF, seed=19)
    assert pa.pa_prefill(**c.dev).shape == (0, 8, 128)
    e = dict(c.dev, q=torch.empty(3, 8, 128, dtype=BF, device="cuda"), seq_lens=c.dev["seq_lens"][:0],
             block_tables=c.dev["block_tables"][:0], cu_q_lens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    out = torch.full((3, 8, 128), 2.0, dtype=BF, device="cuda")
    pa.pa_prefill(**e, out=out)
    assert bool((out == 2).all())
    c = Chunk([0, 0], [5, 9], 8, 2, 128, 16, BF, seed=19, tail=2)
    out = torch.full((2, 8, 128), 2.0, dtype=BF, device="cuda")
    run(c, out=out)
    assert bool((out == 2).all())


def test_negative_and_zero_scale():
    for scale in (-0.2, 0.0):
        c = Chunk([30, 8], [200, 60], 8, 2, 128, 16, BF, seed=20)
        c.scale = c.dev["scale"] = scale
        c.check(run(c), P_EPS[BF])


def test_python_refusals():
    c = Chunk([30, 8], [200, 60], 8, 2, 128, 16, BF, seed=21)
    d = c.dev
    with pytest.raises(ValueError):
        pa.pa_prefill(**dict(d, q=d["q"][:, :, :64]))
    with pytest.raises(ValueError):
        pa.pa_prefill(**dict(d, q=d["q"].float()))
    with pytest.raises(ValueError):
        pa.pa_prefill(**dict(d, cu_q_lens=d["cu_q_lens"][:2]))
    with pytest.raises(TypeError):
        pa.pa_prefill(**dict(d, cu_q_lens=d["cu_q_lens"].long()))
    with pytest.raises(ValueError):
        pa.pa_prefill(**dict(d, q=d["q"].transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_prefill(**d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_prefill(**dict(d, q=torch.zeros(38, 7, 128, dtype=BF, device="cuda")))


@pytest.mark.parametrize("splits", [1, 3, 0])
def test_many_segments_per_cta_with_row_tiles_that_end_apart(splits):
    """Tiles whose first row tile needs a unit less than the second one (and
    finishes early), many in a row on every CTA."""
    lens = [64 + 37 * (i % 5) for i in range(40)]
    ctx = [90 + 61 * (i % 7) for i in range(40)]
    c = Chunk(lens, [a + b for a, b in zip(lens, ctx)], 32, 8, 128, 16, BF, seed=23)
    for _ in range(3):
        out = run(c, num_splits=splits)
    c.check(out, P_EPS[BF])


def check_some(c, out, which):
    """c.check for some of the sequences."""
    for i in which:
        if c.q_lens[i] == 0:
            continue
        ref, amount, dots, top = c.reference(i)
        tol = tolerance(out.dtype, ref, amount, dots, top, c.seq_lens[i], ref.shape[-1], P_EPS[out.dtype])
        err = (out[c.cu[i]:c.cu[i + 1]].double() - ref).abs()
        assert float((err / tol).max()) <= 1.0, i


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,longest", [(2049, 40), (2600, 9), (8300, 3)])
def test_more_sequences_and_tiles_than_shared_memory_lists(n, longest, dtype):
    # the work list keeps 2048 sequences and 8191 tiles in shared memory, more in the workspace
    lens = [1 + i * 7 % longest for i in range(n)]
    c = Chunk([min(L, (i * 5) % 3 + (n > 8000)) for i, L in enumerate(lens)], lens, 4, 2, 64, 8, dtype, seed=n)
    out = run(c)
    check_some(c, out, sorted({0, 1, 1023, 1024, 2047, 2048, n - 2, n - 1} | set(range(0, n, 97))))


@pytest.mark.parametrize("dtype,shift", [(BF, 2), (BF, 4), (F32, 2)])
def test_q_and_out_at_the_smallest_alignment(dtype, shift):
    c = Chunk([40, 1, 7], [300, 65, 7], 8, 2, 128, 16, dtype, seed=61)
    q, out = (torch.empty(c.q.numel() + shift, dtype=dtype, device="cuda")[shift:].view(c.q.shape) for _ in range(2))
    q.copy_(c.q)
    c.dev["q"] = q
    c.check(run(c, out=out), P_EPS[dtype])


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,kernel", [(BF, "mma"), (BF, "simt"), (F32, "simt")])
def test_a_query_row_that_is_not_finite_stays_alone(dtype, kernel, value):
    c = Chunk([150, 3], [400, 90], 8, 2, 128, 16, dtype, seed=62)
    clean = run(c, kernel=kernel)
    c.check(clean, P_EPS[dtype])
    c.dev["q"][17, 5, 3] = value
    out = run(c, kernel=kernel)
    assert torch.isnan(out[17, 5]).all()  # its scores hold NaN, or infinities of both signs
    out[17, 5] = clean[17, 5]
    c.check(out, P_EPS[dtype])


def test_two_calls_at_once():
    cs = [Chunk([700, 33], [2000, 5000], 32, 8, 128, 16, BF, seed=s) for s in (63, 64)]
    want = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pa.pa_prefill(**cs[i].dev))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def test_chunk_at_the_longest_reach():
    """The last two of 2^31 - 8 positions, through a table that names one block
    over and over: the last position's V is not finite, and the row before does not see it."""
    block, n = 8 * 127 * 113, 3 * 5 * 29 * 43
    L = block * n
    assert L == 2 ** 31 - 8
    k, v = torch.zeros(2, block, 1, 64, device="cuda"), torch.ones(2, block, 1, 64, device="cuda")
    v[1, -1] = math.nan
    table = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    i32 = dict(dtype=torch.int32, device="cuda")
    out = pa.pa_prefill(torch.ones(2, 1, 64, device="cuda"), k, v, table, torch.tensor([L], **i32),
                        torch.tensor([0, 2], **i32), 1.0)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    # every score is 0: the sums of a CTA are whole numbers below 2^24, the merge
    # rounds once for each of at most 2^10 pieces
    assert float((out[0].double() - 1).abs().max()) <= 2.0 ** -13
    assert torch.isnan(out[1]).all()


def test_tensor_core_chunk_at_the_longest_reach():
    """As above on the tensor cores, with two heads per KV head."""
    block, n = 8 * 127 * 113, 3 * 5 * 29 * 43
    k, v = torch.zeros(2, block, 1, 64, dtype=BF, device="cuda"), torch.ones(2, block, 1, 64, dtype=BF, device="cuda")
    v[1, -1] = math.nan
    table = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    i32 = dict(dtype=torch.int32, device="cuda")
    out = pa.pa_prefill(torch.ones(2, 2, 64, dtype=BF, device="cuda"), k, v, table, torch.tensor([block * n], **i32),
                        torch.tensor([0, 2], **i32), 1.0, kernel="mma")
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    assert float((out[0].double() - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -13
    assert torch.isnan(out[1]).all()


def with_odd_values(c, seed, share=0.6):
    """V values that are not finite at positions of the chunks' own tokens (and
    some before them), of every kind, in most chunks; returns the number placed."""
    from _chunks import slots_of
    g = torch.Generator().manual_seed(seed)
    Hk, D = c.v.shape[1:]
    kinds = [math.inf, -math.inf, math.nan]
    count = 0
    for i, (n, L) in enumerate(zip(c.q_lens, c.seq_lens)):
        if n == 0 or float(torch.rand(1, generator=g)) > share:
            continue
        rows = slots_of(c.tables[i], L, c.block)
        for _ in range(int(torch.randint(1, 7, (1,), generator=g))):
            pos = int(torch.randint(max(0, L - n - 2), L, (1,), generator=g))
            h, d, kind = (int(torch.randint(0, m, (1,), generator=g)) for m in (Hk, D, 3))
            c.v[rows[pos], h, d] = kinds[kind]
            count += 1
    c.dev["v_cache"] = c.v.view(c.dev["v_cache"].shape).cuda()
    return count


def check_odd(c, refs, out, p_eps):
    """out against fp64 (refs, of c.reference) where the sums hold infinities and NaN."""
    for i, (ref, amount, dots, top) in enumerate(refs):
        got = out[c.cu[i]:c.cu[i + 1]].double()
        fin = torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), i
        assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), i
        tol = tolerance(out.dtype, ref, amount, dots, top, c.seq_lens[i], ref.shape[-1], p_eps)
        assert float(((got - ref).abs() / tol)[fin].max()) <= 1.0, i


@pytest.mark.parametrize("H,Hk,D,block,dtype,kernel", [(8, 2, 128, 16, BF, "mma"), (4, 1, 64, 32, BF, "mma"),
                                                       (16, 1, 128, 8, BF, "mma"), (8, 2, 128, 16, BF, "simt"),
                                                       (4, 2, 64, 16, F32, "simt")])
def test_odd_values_in_chunk_after_chunk(H, Hk, D, block, dtype, kernel):
    """Many segments on a CTA, most of which hold values that are not finite, at
    positions that only some of their rows see, one row tile, both or neither."""
    q = [40, 200, 1, 64, 7, 300, 33, 129, 256, 2, 90, 65]
    ctx = [60, 0, 127, 700, 128, 30, 0, 255, 5, 900, 129, 62]
    for seed in (0, 1):
        c = Chunk(q, [a + b for a, b in zip(q, ctx)], H, Hk, D, block, dtype, seed=90 + seed)
        assert with_odd_values(c, seed) > 8
        refs = [c.reference(i) for i in range(len(q))]
        for splits in (1, 2, 3, 11, 0):
            out = run(c, kernel=kernel, num_splits=splits)
            check_odd(c, refs, out, P_EPS[BF] if kernel == "mma" else 0.0)
            for _ in range(3):
                assert torch.equal(run(c, kernel=kernel, num_splits=splits).view(torch.uint8), out.view(torch.uint8))


def test_roles_that_idle_for_longer_than_a_wait_may_last():
    """One CTA for 3 * 2^20 units (about 3 s) of sequences with a single new token, which the
    second row tile sits out, then a chunk of 200 that it takes part in."""
    block, n, seqs = 4096, 256, 384
    k, v = torch.zeros(1, block, 1, 64, dtype=BF, device="cuda"), torch.ones(1, block, 1, 64, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, cu = [block * n] * seqs + [200], list(range(seqs + 1)) + [seqs + 200]
    out = pa.pa_prefill(torch.ones(seqs + 200, 1, 64, dtype=BF, device="cuda"), k, v, torch.zeros(seqs + 1, n, **i32),
                        torch.tensor(lens, **i32), torch.tensor(cu, **i32), 1.0, kernel="mma", num_splits=1)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    assert bool((out == 1).all())  # every score is 0, every sum a whole number below 2^24


@pytest.mark.parametrize("H,Hk,D,block,dtype", SHAPES)
def test_ragged_chunks_on_the_cuda_cores(H, Hk, D, block, dtype):
    """fp32 probabilities: no allowance for their rounding."""
    c = Chunk(*RAGGED, H, Hk, D, block, dtype, seed=H * 1000 + D + block)
    c.check(run(c, kernel="simt"), 0.0)


@pytest.mark.parametrize("dtype,D,block", [(F32, 64, 4), (F32, 128, 16), (BF, 128, 16), (BF, 64, 32)])
def test_split_layout_on_the_cuda_cores(dtype, D, block):
    c = Chunk(*RAGGED, 8, 2, D, block, dtype, seed=11, layout="split")
    c.check(run(c), 0.0)


def on_tensor_cores(D, block, dtype):
    return dtype == BF and D in (64, 128) and block % 8 == 0


@pytest.mark.parametrize("H,Hk,D,block,dtype", SHAPES)
def test_which_kernel_a_call_takes(H, Hk, D, block, dtype):
    """auto is the tensor-core kernel, bit for bit, where that takes the call, and the CUDA cores' where not."""
    c = Chunk(*RAGGED, H, Hk, D, block, dtype, seed=101)
    out = run(c)
    if on_tensor_cores(D, block, dtype):
        assert torch.equal(out, run(c, kernel="mma")) and not torch.equal(out, run(c, kernel="simt"))
    else:
        assert torch.equal(out, run(c, kernel="simt"))
        with pytest.raises(pa.PagedAttentionError):
            run(c, kernel="mma")


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 1000])
def test_any_split_count_by_kernel(splits):
    c = Chunk([3, 200, 1, 70], [3000, 200, 700, 1025], 8, 2, 128, 16, BF, seed=5)
    c.check(run(c, kernel="mma", num_splits=splits), P_EPS[BF])
    c.check(run(c, kernel="simt", num_splits=splits), 0.0)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_around_tile_edges_by_kernel(n):
    c = Chunk([n, 1, n, min(n, 3)], [n, n, n + 128, n + 1], 8, 2, 128, 16, BF, seed=n)
    c.check(run(c, kernel="mma"), P_EPS[BF])
    c.check(run(c, kernel="simt"), 0.0)
