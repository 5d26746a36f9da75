"""The 8-bit cache with block scales: its write bit by bit against the rule worked
out in fp64, decode and chunk attention over it against fp64, its read-back and
block copy."""
import math

import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _block8 import BF, E4M3, Block8, code_values, write_rule
from _chunks import make_tables, slots_of

pytestmark = pytest.mark.gpu
F32 = torch.float32
P_MMA, P_SIMT = 2.0 ** -8, 0.0      # chunk kernels: P in bf16, in fp32
P_DECODE, TAIL = 2.0 ** -11, 2.0 ** -25  # decode's tensor-core kernel: P in fp16
BOUNDS = pa._lib.PA_ERR_DEVICE_BOUNDS


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def error():
    return pa.pa_get_device_error(raise_on_error=False)


# ------------------------------------------------------------------- write
class Write:
    """A pa_write_blocks_fp8 call over a pool of given codes and bytes."""

    def __init__(self, q_lens, seq_lens, Hk, D, block, dtype, seed, lead=0, tail=0, special=True, low=100, high=150):
        g = torch.Generator().manual_seed(seed)
        self.block, self.lens = block, seq_lens
        self.tables, self.pool = make_tables(seq_lens, block, g)
        self.cu = [lead]
        for n in q_lens:
            self.cu.append(self.cu[-1] + n)
        T = self.cu[-1] + tail
        self.x = []
        for _ in range(2):
            y = torch.randn(T, Hk, D, generator=g) * torch.exp2(torch.randint(-30, 30, (T, Hk, 1), generator=g).float())
            y = y.to(dtype)
            if special and y.numel() > 40:
                f = y.view(-1)
                f[1], f[5], f[7], f[11] = math.inf, -math.inf, math.nan, 0.0
                y[T // 2, -1] = 0
                y[-1, 0] = torch.finfo(dtype).tiny
                y[-1, -1, 0] = torch.finfo(dtype).max
            self.x.append(y)
        shape = (self.pool, block, Hk, D)
        self.codes = [torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8) for _ in range(2)]
        self.scales = [torch.randint(low, high, (self.pool, Hk), generator=g, dtype=torch.int32).to(torch.uint8)
                       for _ in range(2)]

    def run(self, tables=None, lens=None, cu=None, x=None):
        kc, vc = (c.cuda().view(E4M3) for c in self.codes)
        ks, vs = (s.cuda() for s in self.scales)
        x = x or [y.cuda() for y in self.x]
        pa.pa_write_blocks_fp8(*x, (self.tables if tables is None else tables).cuda(), i32(lens or self.lens),
                               i32(cu or self.cu), kc, vc, ks, vs)
        return (kc, ks), (vc, vs)

    def check(self, got, lens=None, tables=None):
        for x, codes, scales, (c, s) in zip(self.x, self.codes, self.scales, got):
            want, byte = write_rule(x, code_values()[codes.long()], scales, self.tables if tables is None else tables,
                                    lens or self.lens, self.cu, self.block, self.pool)
            val = code_values()[c.view(torch.uint8).cpu().long()]
            assert torch.equal(torch.isnan(val), torch.isnan(want))
            assert torch.equal(val.nan_to_num(), want.nan_to_num())
            assert torch.equal(s.cpu(), byte)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk,D,block", [(8, 128, 16), (2, 64, 32), (1, 128, 64), (3, 64, 4), (2, 256, 48), (2, 96, 16),
                                        (1, 1024, 8), (3, 7, 5), (2, 1, 3), (5, 33, 16), (1, 64, 256), (2, 8, 1)])
def test_write_bit_by_bit(Hk, D, block, dtype):
    q = [1, 1, 40, 0, 3, block, 2 * block + 1, 5]
    ctx = [0, block - 1, 7, 9, 2 * block, block, 3, 0]
    w = Write(q, [a + c for a, c in zip(q, ctx)], Hk, D, block, dtype, seed=Hk * D + block, lead=2, tail=3)
    got = w.run()
    assert error() == 0
    w.check(got)


@pytest.mark.parametrize("low,high", [(0, 12), (127, 128), (240, 256), (1, 248)])
def test_write_behind_bytes_of_every_size(low, high):
    """Blocks that hold earlier positions, whose bytes are smaller, larger, the same, and past the largest that a write makes."""
    n = 24
    w = Write([2] * n, [2 + i % 15 for i in range(n)], 4, 64, 16, F32, seed=low + 3, special=False, low=low, high=high)
    for x in w.x:
        x *= 1e-30 if high < 20 else 1.0
    w.check(w.run())
    assert error() == 0


def test_write_token_by_token_is_the_rule_applied_again():
    """A block that fills up one token per call: its byte never falls and its codes follow."""
    w = Write([1], [1], 2, 64, 8, BF, seed=5, special=False)
    g = torch.Generator().manual_seed(6)
    rows = [(torch.randn(20, 2, 64, generator=g) * torch.exp2(torch.arange(20) % 7 - 3.0).view(-1, 1, 1)).to(BF) for _ in range(2)]
    tables = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    kc, vc = (torch.zeros(4, 8, 2, 64, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.full((4, 2), 200, dtype=torch.uint8, device="cuda") for _ in range(2))
    state = [(torch.zeros(4, 8, 2, 64, dtype=torch.float64), torch.full((4, 2), 200, dtype=torch.uint8)) for _ in range(2)]
    for t in range(20):
        pa.pa_write_blocks_fp8(rows[0][t:t + 1].cuda(), rows[1][t:t + 1].cuda(), tables.cuda(), i32([t + 1]), i32([0, 1]),
                               kc, vc, ks, vs)
        for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
            state[i] = write_rule(rows[i][t:t + 1], *state[i], tables, [t + 1], [0, 1], 8, 4)
            assert torch.equal(code_values()[c.view(torch.uint8).cpu().long()], state[i][0])
            assert torch.equal(s.cpu(), state[i][1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_write_unaligned_rows(dtype):
    w = Write([9, 20], [12, 20], 2, 64, 16, dtype, seed=8)
    moved = []
    for y in w.x:
        buf = torch.zeros(y.numel() + 1, dtype=dtype, device="cuda")
        buf[1:] = y.cuda().flatten()
        moved.append(buf[1:].view(y.shape))
    w.check(w.run(x=moved))


def test_write_many_sequences_and_long_ones():
    """More offsets than shared memory holds; prompts of many blocks; heads whose rows need several warps."""
    n = 2500
    w = Write([1 + i % 3 for i in range(n)], [1 + i % 3 + i % 19 for i in range(n)], 1, 32, 8, BF, seed=9, special=False)
    w.check(w.run())
    w = Write([1500, 2], [1800, 700], 2, 128, 128, F32, seed=10)
    w.check(w.run())
    assert error() == 0


def test_write_refuses_bad_offsets_and_skips_bad_lengths_and_pages():
    w = Write([20, 8], [40, 30], 2, 64, 16, BF, seed=11)
    for cu in ([0, 29, 28], [-1, 20, 28], [0, 20, 29], [0, 2 ** 31 - 1, 28]):
        got = w.run(cu=cu)
        assert error() == BOUNDS
        for codes, scales, (c, s) in zip(w.codes, w.scales, got):
            assert torch.equal(c.view(torch.uint8).cpu(), codes) and torch.equal(s.cpu(), scales)
    reach = w.tables.shape[1] * 16
    for bad in (-1, 19, reach + 1, 2 ** 31 - 1):  # fewer positions than new tokens, more than the table's
        got = w.run(lens=[bad, 30])
        assert error() == BOUNDS
        only = Write([20, 8], [40, 30], 2, 64, 16, BF, seed=11)
        for x, codes, scales, (c, s) in zip(only.x, only.codes, only.scales, got):
            want, byte = write_rule(x[20:], code_values()[codes.long()], scales, w.tables[1:], [30], [0, 8], 16, w.pool)
            val = code_values()[c.view(torch.uint8).cpu().long()]
            assert torch.equal(val.nan_to_num(), want.nan_to_num()) and torch.equal(s.cpu(), byte)
    tables = w.tables.clone()
    tables[0, 1] = w.pool  # positions 20 .. 31 of sequence 0
    got = w.run(tables=tables)
    assert error() == BOUNDS
    lost = int(w.tables[0, 1])
    for x, codes, scales, (c, s) in zip(w.x, w.codes, w.scales, got):
        want, byte = write_rule(x, code_values()[codes.long()], scales, w.tables, w.lens, w.cu, 16, w.pool)
        want[lost], byte[lost] = code_values()[codes[lost].long()], scales[lost]
        val = code_values()[c.view(torch.uint8).cpu().long()]
        assert torch.equal(val.nan_to_num(), want.nan_to_num()) and torch.equal(s.cpu(), byte)


def test_write_past_32_bits():
    block, Hk, D = 16, 8, 128
    pool = (2 ** 31 + 2 ** 27) // (block * Hk * D)
    g = torch.Generator(device="cuda").manual_seed(12)
    kc, vc = (torch.zeros(pool, block, Hk, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros(pool, Hk, dtype=torch.uint8, device="cuda") for _ in range(2))
    far = torch.tensor([[pool - 1, pool - 3]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(20, Hk, D, generator=g, device="cuda").to(BF) for _ in range(2))
    pa.pa_write_blocks_fp8(k, v, far, i32([20]), i32([0, 20]), kc, vc, ks, vs)
    slots = slots_of(far[0].cpu(), 20, block).to(torch.int32).cuda()
    gk, gv = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots, dtype=F32)
    assert error() == 0
    for x, got in ((k, gk), (v, gv)):  # half a step of 3 bits behind the point, or of the smallest normal
        assert bool(((x.float() - got).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -17 * x.float().abs().max()).all())
    out = pa.pa_prefill_fp8(k.repeat_interleave(4, 1), kc, vc, ks, vs, far, i32([20]), i32([0, 20]), D ** -0.5)
    one = pa.pa_decode_fp8(k[19:].repeat_interleave(4, 1), kc, vc, ks, vs, far, i32([20]), D ** -0.5)
    assert error() == 0
    # P in bf16 and in fp16 over the same values, both rounded to bf16
    assert float((out[19:].float() - one.float()).abs().max()) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -8) * float(gv.abs().max())


# ------------------------------------------------- read-back and block copy
@pytest.mark.parametrize("Hk,D,block", [(8, 128, 16), (3, 96, 4), (2, 7, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_back(Hk, D, block, dtype):
    b = Block8([1], [3 * block], 1 * Hk, Hk, D, block, seed=20)
    pool = b.codes[0].shape[0]
    g = torch.Generator().manual_seed(21)
    slots = torch.randperm(pool * block, generator=g)[:2 * block + 3].to(torch.int32)
    slots[1] = -1
    got = pa.pa_gather_cache_fp8(b.dev["k_cache"], b.dev["v_cache"], b.dev["k_scale"], b.dev["v_scale"], slots.cuda(), dtype=dtype)
    assert error() == 0
    for val, x in zip(b.vals, got):
        want = val[slots.long()]
        want[1] = 0
        want = want.to(dtype)
        assert torch.equal(torch.isnan(x.cpu()), torch.isnan(want)) and torch.equal(x.cpu().nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("Hk,D,block", [(8, 128, 16), (3, 7, 5)])
def test_copy_blocks(Hk, D, block):
    b = Block8([1] * 6, [block] * 6, Hk, Hk, D, block, seed=22)
    args = [b.dev[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    want = [x.view(torch.uint8).clone() for x in args]
    pairs = [[0, 3], [4, 1], [0, 2]]
    for x in want:
        for s, d in pairs:
            x[d] = x[s]
    pa.pa_copy_blocks_fp8(*args, i32(pairs))
    assert error() == 0
    for x, y in zip(args, want):
        assert torch.equal(x.view(torch.uint8), y)


# ------------------------------------------------------------------- decode
SHAPES = [(32, 8, 128, 16), (8, 8, 128, 16), (16, 2, 64, 32), (12, 4, 128, 16), (8, 1, 128, 64), (7, 1, 64, 8),
          (8, 4, 128, 128), (6, 6, 128, 48), (10, 5, 64, 24), (64, 8, 128, 8), (8, 1, 64, 256)]
SLOW = [(8, 2, 128, 5), (8, 2, 256, 16), (4, 4, 64, 4)]  # CUDA cores
LENS = [1, 0, 15, 16, 17, 31, 33, 64, 65, 700, 129, 257]


@pytest.mark.parametrize("H,Hk,D,block", SHAPES)
def test_decode(H, Hk, D, block):
    b = Block8([1] * len(LENS), LENS, H, Hk, D, block, seed=H + D + block)
    out = pa.pa_decode_fp8(**b.decode_args(), kernel="mma")
    assert error() == 0
    b.check(out, P_DECODE, TAIL)
    assert torch.count_nonzero(out[1]) == 0
    assert torch.equal(out, pa.pa_decode_fp8(**b.decode_args()))


@pytest.mark.parametrize("H,Hk,D,block", SHAPES[:3] + SLOW)
def test_decode_on_the_cuda_cores(H, Hk, D, block):
    b = Block8([1] * len(LENS), LENS, H, Hk, D, block, seed=H + D + block)
    out = pa.pa_decode_fp8(**b.decode_args(), kernel="simt")
    assert error() == 0
    b.check(out, P_SIMT)


@pytest.mark.parametrize("splits", [1, 2, 5, 37, 900])
def test_decode_any_split_count(splits):
    b = Block8([1] * 4, [3000, 1, 900, 50], 32, 8, 128, 16, seed=40)
    b.check(pa.pa_decode_fp8(**b.decode_args(), num_splits=splits), P_DECODE, TAIL)


def test_decode_blocks_of_very_different_size():
    b = Block8([1] * 3, [700, 300, 2000], 32, 8, 128, 16, seed=41, spread=40)
    b.check(pa.pa_decode_fp8(**b.decode_args()), P_DECODE, TAIL)


@pytest.mark.parametrize("shift", [1, 2, 3, 4])
@pytest.mark.parametrize("H,Hk", [(32, 8), (8, 4), (4, 2), (3, 3)])
def test_decode_scales_at_any_alignment(H, Hk, shift):
    b = Block8([1] * 3, [70, 300, 9], H, Hk, 64, 16, seed=43)
    args = b.decode_args()
    for n in ("k_scale", "v_scale"):
        buf = torch.zeros(args[n].numel() + shift, dtype=torch.uint8, device="cuda")
        buf[shift:] = args[n].flatten()
        args[n] = buf[shift:].view(args[n].shape)
    b.check(pa.pa_decode_fp8(**args, kernel="mma"), P_DECODE, TAIL)
    assert error() == 0


# ------------------------------------------------------------------- chunks
@pytest.mark.parametrize("H,Hk,D,block", SHAPES)
def test_chunks(H, Hk, D, block):
    q = [1, 5, 0, 128, 33, 260, 2]
    lens = [1, 130, 9, 128, 700, 300, 1025]
    b = Block8(q, lens, H, Hk, D, block, seed=H + D + block + 1)
    out = pa.pa_prefill_fp8(**b.dev, kernel="mma")
    assert error() == 0
    b.check(out, P_MMA)
    assert torch.equal(out, pa.pa_prefill_fp8(**b.dev))


@pytest.mark.parametrize("H,Hk,D,block", SHAPES[:2] + SLOW)
def test_chunks_on_the_cuda_cores(H, Hk, D, block):
    b = Block8([1, 5, 0, 70, 33], [1, 130, 9, 70, 300], H, Hk, D, block, seed=H + D + block + 2)
    out = pa.pa_prefill_fp8(**b.dev, kernel="simt")
    assert error() == 0
    b.check(out, P_SIMT)


@pytest.mark.parametrize("splits", [1, 3, 40, 700])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks_any_split_count(D, splits):
    b = Block8([200, 3, 64], [900, 1500, 64], 16, 4, D, 16, seed=50)
    b.check(pa.pa_prefill_fp8(**b.dev, num_splits=splits, kernel="mma"), P_MMA)
    assert error() == 0


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 7, 13, 29])
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_chunks_per_cta(D, splits):
    """Tiles of a few rows, several to a CTA, cut at either end of its range; blocks of very different size."""
    b = Block8([3, 1, 8, 5, 2, 0, 7] * 3, [1000 - 41 * i for i in range(21)], 4, 2, D, 16, seed=80 + splits, spread=12)
    out = pa.pa_prefill_fp8(**b.dev, num_splits=splits, kernel="mma")
    assert error() == 0
    b.check(out, P_MMA)


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_chunks_over_blocks_of_very_different_size(kernel):
    b = Block8([33, 3, 150], [700, 300, 2000], 16, 4, 128, 16, seed=41, spread=40)
    b.check(pa.pa_prefill_fp8(**b.dev, kernel=kernel), P_MMA if kernel == "mma" else P_SIMT)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 257])
def test_chunk_lengths_around_tile_edges(n):
    b = Block8([n, 2], [n, 2 + n], 8, 2, 128, 16, seed=51 + n)
    b.check(pa.pa_prefill_fp8(**b.dev), P_MMA)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [0, 1, 5, 60])
def test_chunks_of_a_padded_batch(D, splits):
    """Sequences without tokens bring the mean chunk below a row tile: long chunks beside short ones in that form."""
    q, lens = [200, 260, 3, 0, 40, 129], [900, 300, 2000, 7, 40, 1300]
    b = Block8(q + [0] * 40, lens + [0, 17] * 20, 16, 4, D, 16, seed=90, spread=12)
    out = pa.pa_prefill_fp8(**b.dev, num_splits=splits, kernel="mma")
    assert error() == 0
    b.check(out, P_MMA)


@pytest.mark.parametrize("pad", [0, 40])
def test_nan_codes_in_long_chunks_of_a_padded_batch(pad):
    b = Block8([300, 5] + [0] * pad, [700, 300] + [0] * pad, 8, 2, 128, 16, seed=91)
    clean = pa.pa_prefill_fp8(**b.dev, kernel="mma")
    for i, p in enumerate([500, 297]):  # rows 0..99 and 0..1 do not see these
        row = int(slots_of(b.tables[i], b.seq_lens[i], 16)[p])
        b.dev["v_cache"].view(torch.uint8)[row // 16, row % 16, 1, 5] = 0x7f
    out = pa.pa_prefill_fp8(**b.dev, kernel="mma")
    assert error() == 0
    assert torch.equal(out[:100], clean[:100]) and torch.equal(out[300:302], clean[300:302])
    assert torch.isnan(out[100:300, 4:, 5]).all() and torch.isnan(out[302:, 4:, 5]).all()
    assert torch.equal(out[100:, :4], clean[100:, :4])


def test_chunk_of_long_context():
    b = Block8([4, 1, 2], [20000, 9001, 127], 32, 8, 128, 16, seed=52)
    b.check(pa.pa_prefill_fp8(**b.dev), P_MMA)


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_chunk_rows_that_see_nothing_and_rows_of_no_sequence(kernel):
    b = Block8([150, 9, 4], [20, 9, 0], 8, 2, 128, 16, seed=53, lead=3, tail=7)
    out = torch.full_like(b.dev["q"], 7.0)
    pa.pa_prefill_fp8(**b.dev, out=out, kernel=kernel)
    assert error() == 0
    b.check(out, P_MMA if kernel == "mma" else P_SIMT)
    assert torch.count_nonzero(out[3:133]) == 0 and torch.count_nonzero(out[162:166]) == 0
    assert bool((out[:3] == 7).all()) and bool((out[166:] == 7).all())


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_nan_codes_reach_only_the_rows_that_see_them(kernel):
    b = Block8([40, 200], [100, 200], 8, 2, 128, 16, seed=54)
    clean = pa.pa_prefill_fp8(**b.dev, kernel=kernel)
    for i, p in enumerate([80, 150]):  # rows 0..19 and 0..149 do not see these
        row = int(slots_of(b.tables[i], b.seq_lens[i], 16)[p])
        b.dev["v_cache"].view(torch.uint8)[row // 16, row % 16, 1, 5] = 0x7f
        b.dev["k_cache"].view(torch.uint8)[row // 16, row % 16, 0, 3] = 0xff
    out = pa.pa_prefill_fp8(**b.dev, kernel=kernel)
    assert error() == 0
    assert torch.equal(out[:20], clean[:20]) and torch.equal(out[40:190], clean[40:190])
    assert torch.isnan(out[20:40, 4:, 5]).all() and torch.isnan(out[190:, 4:, 5]).all()
    assert torch.isfinite(out[20:40, 4:, :5]).all() and torch.isfinite(out[190:, 4:, 6:]).all()
    assert torch.isnan(out[20:40, :4]).all() and torch.isnan(out[190:, :4]).all()


@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_the_nan_byte_makes_its_block_nan(kernel, which):
    """Byte 255 of a seen block and head: every value of it is NaN."""
    b = Block8([3, 1], [60, 20], 8, 2, 64, 16, seed=55)
    clean = pa.pa_prefill_fp8(**b.dev, kernel=kernel)
    b.dev[which][int(b.tables[0, 1]), 1] = 255
    out = pa.pa_prefill_fp8(**b.dev, kernel=kernel)
    assert torch.isnan(out[:3, 4:]).all()
    assert torch.equal(out[:, :4], clean[:, :4]) and torch.equal(out[3:], clean[3:])
    one = pa.pa_decode_fp8(**dict(b.decode_args(), q=b.dev["q"][2:].contiguous()), kernel=kernel)
    assert torch.isnan(one[0, 4:]).all() and torch.isfinite(one[:, :4]).all() and torch.isfinite(one[1]).all()


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_the_nan_byte_in_long_chunks(which):
    """As above for more rows than a row tile has: rows before the block's first position do not see it."""
    b = Block8([100], [170], 8, 2, 128, 16, seed=92)
    clean = pa.pa_prefill_fp8(**b.dev, kernel="mma")
    b.dev[which][int(b.tables[0, 9]), 1] = 255  # positions 144 .. 159, tokens from 74 on
    out = pa.pa_prefill_fp8(**b.dev, kernel="mma")
    assert error() == 0
    assert torch.isnan(out[74:, 4:]).all()
    assert torch.equal(out[:, :4], clean[:, :4]) and torch.equal(out[:74], clean[:74])


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_blocks_of_the_smallest_and_largest_bytes(kernel):
    """V of bytes 14 and 240 in one head each (K ordinary): the ends of what bf16 holds exactly."""
    b = Block8([6], [70], 2, 2, 64, 16, seed=56)
    pool = b.codes[1].shape[0]
    s = torch.tensor([[14, 240]], dtype=torch.uint8).expand(pool, 2).contiguous()
    b.dev["v_scale"].copy_(s)
    b.vals[1] = Block8.decoded(b.codes[1], s).view(pool * 16, 2, 64)
    out = pa.pa_prefill_fp8(**b.dev, kernel=kernel)
    for h in range(2):
        unit = 2.0 ** (113 if h else -113)
        r = slots_of(b.tables[0], 70, 16)
        from _chunks import attention, tolerance
        ref, amount, dots, top = attention(b.q[:, h:h + 1], b.vals[0][r][:, h:h + 1], b.vals[1][r][:, h:h + 1] / unit, 64, b.scale)
        tol = tolerance(BF, ref, amount, dots, top, 70, 64, P_MMA if kernel == "mma" else P_SIMT)
        assert bool(((out[:, h:h + 1].cpu().double() / unit - ref).abs() <= tol).all())


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_bad_pages_read_zeros_and_are_recorded(kernel):
    b = Block8([30, 8], [200, 60], 8, 2, 128, 16, seed=57)
    tables, pool = b.tables.clone(), b.codes[0].shape[0]
    for i, blk, x in [(0, 3, pool), (0, 7, -5), (1, 0, 2 ** 31 - 1)]:
        rows = slots_of(b.tables[i], b.seq_lens[i], 16)[blk * 16:(blk + 1) * 16]
        b.vals[0][rows], b.vals[1][rows] = 0, 0
        tables[i, blk] = x
    args = dict(b.dev, block_tables=tables.cuda())
    out = pa.pa_prefill_fp8(**args, kernel=kernel)
    assert error() == BOUNDS
    b.check(out, P_MMA if kernel == "mma" else P_SIMT)
    args = {k: v for k, v in args.items() if k != "cu_q_lens"}
    one = pa.pa_decode_fp8(**dict(args, q=b.dev["q"][[29, 37]].contiguous()), kernel=kernel)
    assert error() == BOUNDS
    assert float((one.float() - out[[29, 37]].float()).abs().max()) <= 3 * 2.0 ** -8 * float(b.vals[1][torch.isfinite(b.vals[1])].abs().max())


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_bad_offsets_and_lengths(kernel):
    b = Block8([30, 8], [200, 60], 8, 2, 128, 16, seed=58)
    for cu in ([0, 39, 38], [-1, 30, 38], [0, 30, 39]):
        out = torch.full_like(b.dev["q"], 3.0)
        pa.pa_prefill_fp8(**dict(b.dev, cu_q_lens=i32(cu)), out=out, kernel=kernel)
        assert error() == BOUNDS and bool((out == 3).all())
    out = pa.pa_prefill_fp8(**dict(b.dev, seq_lens=i32([2 ** 31 - 1, 60])), kernel=kernel)
    assert error() == BOUNDS and torch.count_nonzero(out[:30]) == 0
    b.q_lens[0] = 0
    b.cu[0] = 30
    b.check(out, P_MMA if kernel == "mma" else P_SIMT)


def test_negative_and_zero_scale():
    for scale in (-0.2, 0.0):
        b = Block8([30, 8], [200, 60], 8, 2, 128, 16, seed=59, spread=1)
        b.scale = b.dev["scale"] = scale
        b.check(pa.pa_prefill_fp8(**b.dev), P_SIMT)
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_prefill_fp8(**b.dev, kernel="mma")


def test_graphs_that_share_a_workspace_and_a_side_stream():
    a, b = Block8([30, 100], [700, 100], 32, 8, 128, 16, seed=60), Block8([7, 64, 1], [90, 640, 2000], 32, 8, 128, 16, seed=61)
    need = max(pa.pa_prefill_fp8_workspace_bytes(x.dev["k_cache"], x.dev["q"].shape[0], len(x.q_lens), 32) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x.dev["q"]) for x in (a, b)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x, o in zip((a, b), outs):
            pa.pa_prefill_fp8(**x.dev, out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    want = [o.clone() for o in outs]
    a.check(want[0], P_MMA)
    b.check(want[1], P_MMA)
    graphs = []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_prefill_fp8(**x.dev, out=o, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1, 0)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])


def test_two_calls_at_once():
    """Two streams with a workspace each, writes and chunks of their own pools."""
    jobs = [Block8([30, 100], [700, 100], 32, 8, 128, 16, seed=62), Block8([64] * 8, [640] * 8, 32, 8, 128, 16, seed=63)]
    want = [pa.pa_prefill_fp8(**b.dev) for b in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(4):
        for i, (b, s) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(s):
                got[i].append(pa.pa_prefill_fp8(**b.dev))
    torch.cuda.synchronize()
    assert error() == 0
    for w, g in zip(want, got):
        for x in g:
            assert torch.equal(x, w)


def test_empty_calls():
    b = Block8([0, 0], [5, 9], 8, 2, 128, 16, seed=64)
    assert pa.pa_prefill_fp8(**b.dev).shape == (0, 8, 128)
    before = [b.dev[n].view(torch.uint8).clone() for n in ("k_cache", "k_scale")]
    empty = torch.empty(0, 2, 128, dtype=BF, device="cuda")
    pa.pa_write_blocks_fp8(empty, empty, b.dev["block_tables"], b.dev["seq_lens"], b.dev["cu_q_lens"],
                           *[b.dev[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")])
    some = torch.ones(2, 2, 128, dtype=BF, device="cuda")  # rows of no sequence
    pa.pa_write_blocks_fp8(some, some, b.dev["block_tables"], b.dev["seq_lens"], b.dev["cu_q_lens"],
                           *[b.dev[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")])
    assert error() == 0
    for x, n in zip(before, ("k_cache", "k_scale")):
        assert torch.equal(x, b.dev[n].view(torch.uint8))


def test_python_refusals():
    b = Block8([30, 8], [200, 60], 8, 2, 128, 16, seed=65)
    d, one = b.dev, b.decode_args()
    k = torch.zeros(38, 2, 128, dtype=BF, device="cuda")
    caches = [d[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    write = (d["block_tables"], d["seq_lens"], d["cu_q_lens"], *caches)
    token = torch.zeros(caches[0].shape[:3], dtype=torch.uint8, device="cuda")
    for bad in (dict(d, q=d["q"].float()), dict(d, q=d["q"][:, :, :64].contiguous()), dict(d, block_tables=d["block_tables"][0]),
                dict(d, cu_q_lens=d["cu_q_lens"][:2]), dict(d, k_scale=token), dict(d, v_scale=d["v_scale"][:-1]),
                dict(d, k_scale=d["k_scale"].float()), dict(d, out=torch.empty(1, device="cuda")),
                dict(d, seq_lens=d["seq_lens"].long()), dict(d, q=d["q"].cpu()), dict(d, k_cache=d["k_cache"].view(torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            pa.pa_prefill_fp8(**bad)
    with pytest.raises(pa.PagedAttentionError):  # a scale per token
        pa.pa_prefill_fp8(**dict(d, k_scale=token, v_scale=token))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_prefill_fp8(**dict(d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_reshape_and_cache_fp8(k, k, i32(list(range(38))), *caches)
    with pytest.raises(ValueError):
        pa.pa_write_blocks_fp8(k, k, *write[:5], token, token)
    with pytest.raises(ValueError):
        pa.pa_write_blocks_fp8(k, k[:-1], *write)
    with pytest.raises(TypeError):
        pa.pa_write_blocks_fp8(k, k.float(), *write)
    with pytest.raises(TypeError):
        pa.pa_write_blocks_fp8(k.half(), k.half(), *write)
    with pytest.raises(ValueError):
        pa.pa_decode_fp8(**dict(one, q=d["q"][:2].contiguous(), v_scale=token))
