"""pa_write_blocks_fp8 at the ends of its ranges and next to other calls."""
import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _block8 import BF, E4M3, code_values, write_rule

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def error():
    return pa.pa_get_device_error(raise_on_error=False)


def values(codes):
    return code_values()[codes.view(torch.uint8).cpu().long()]


@pytest.mark.parametrize("pad", [0, 5])
def test_write_at_the_longest_reach(pad):
    """The last three of 2^31 - 1 positions in blocks of one token, with rows of a
    padded batch behind them: the numbers past the sequence's blocks name none."""
    L, Hk, D = 2 ** 31 - 1, 2, 64
    table = torch.zeros(1, L, dtype=torch.int32, device="cuda")
    table[0, -3:] = i32([3, 1, 4])
    g = torch.Generator().manual_seed(30 + pad)
    k, v = (torch.randn(3 + pad, Hk, D, generator=g).to(BF) for _ in range(2))
    old = [torch.randint(0, 120, (5, 1, Hk, D), generator=g, dtype=torch.int32).to(torch.uint8) for _ in range(2)]
    bytes_ = [torch.randint(100, 140, (5, Hk), generator=g, dtype=torch.int32).to(torch.uint8) for _ in range(2)]
    codes, scales = [x.cuda().view(E4M3) for x in old], [x.cuda() for x in bytes_]
    pa.pa_write_blocks_fp8(k.cuda(), v.cuda(), table, i32([L]), i32([0, 3]), *codes, *scales)
    assert error() == 0
    for x, c, s, c0, s0 in zip((k, v), codes, scales, old, bytes_):
        # the same three blocks of a sequence of three positions
        want, byte = write_rule(x[:3], code_values()[c0.long()], s0, [[3, 1, 4]], [3], [0, 3], 1, 5)
        assert torch.equal(values(c), want) and torch.equal(s.cpu(), byte)


def test_write_of_more_than_2_to_the_30_heads():
    """One position of 2^30 KV heads of one element: twice the heads pass 31 bits."""
    Hk, period = 2 ** 30, 2 ** 12
    g = torch.Generator().manual_seed(31)
    x = [(torch.randn(1, period, 1, generator=g) * torch.exp2(torch.randint(-40, 40, (1, period, 1), generator=g).float())).to(BF)
         for _ in range(2)]
    k, v = (y.cuda().repeat(1, Hk // period, 1) for y in x)
    codes = [torch.zeros(2, 1, Hk, 1, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.full((2, Hk), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pa.pa_write_blocks_fp8(k, v, i32([[1]]), i32([1]), i32([0, 1]), *codes, *scales)
    assert error() == 0
    for y, c, s in zip(x, codes, scales):
        want, byte = write_rule(y, torch.zeros(1, 1, period, 1, dtype=torch.float64), torch.zeros(1, period, dtype=torch.uint8),
                                [[0]], [1], [0, 1], 1, 1)
        first = c.view(torch.uint8)[1, 0, :period, 0]
        assert torch.equal(values(first), want[0, 0, :, 0])
        assert bool((c.view(torch.uint8)[1].view(-1, period) == first).all()) and torch.count_nonzero(c.view(torch.uint8)[0]) == 0
        assert bool((s[1].view(-1, period) == byte[0].cuda()).all()) and bool((s[0] == 9).all())


def growing_step(i, n, Hk, D, g):
    """A token for each of n requests, larger from step to step: exponents of partly filled blocks grow."""
    return [(torch.randn(n, Hk, D, generator=g, device="cuda") * 2.0 ** (i - 10)).to(BF) for _ in range(2)]


class Steps:
    """Requests of a token per step: tables, the 8-bit pool with block scales, an
    8-bit pool with a scale per token and a bf16 pool at the same slots, read back."""

    def __init__(self, n=300, Hk=3, D=64, B=16, steps=20):
        self.n, self.B = n, B
        W = -(-steps // B) + 1
        NB = n * W
        self.tables = torch.full((n, W), -1, dtype=torch.int32, device="cuda")
        self.lens, self.count = torch.zeros(n, dtype=torch.int32, device="cuda"), i32([NB])
        self.free = torch.arange(NB - 1, -1, -1, dtype=torch.int32, device="cuda")  # neighbours to neighbouring requests
        self.new = torch.ones(n, dtype=torch.int32, device="cuda")
        self.block = [torch.zeros(NB, B, Hk, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + \
                     [torch.zeros(NB, Hk, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.token = [torch.zeros(NB, B, Hk, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + \
                     [torch.zeros(NB, B, Hk, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.bf = [torch.zeros(NB, B, Hk, D, dtype=BF, device="cuda") for _ in range(2)]
        self.ws = torch.empty(pa.pa_tables_workspace_bytes(n, n), dtype=torch.uint8, device="cuda")
        self.q = torch.randn(n, Hk, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)

    def step(self, k, v, sync):
        """The step's calls, with nothing between them or one wait behind each; what they give."""
        bt, sl, cu, slots = pa.pa_extend_tables(self.tables, self.lens, self.free, self.count, self.new, self.B, self.n,
                                                workspace=self.ws)
        sync()
        pa.pa_write_blocks_fp8(k, v, bt, sl, cu, *self.block)
        sync()
        back = pa.pa_gather_cache_fp8(*self.block, slots)
        sync()
        slow = pa.pa_decode_fp8(self.q, *self.block, bt, sl, 0.125, kernel="simt")
        sync()
        pa.pa_reshape_and_cache_fp8(k, v, slots, *self.token)
        sync()
        back_t = pa.pa_gather_cache_fp8(*self.token, slots)
        sync()
        pa.pa_reshape_and_cache(*back_t, slots, *self.bf)
        sync()
        out = pa.pa_decode(self.q, *self.bf, bt, sl, 0.125)
        return (bt, sl, slots, slow, out) + back + back_t

    def state(self):
        return [x.view(torch.uint8) for x in self.block + self.token] + self.bf + [self.tables, self.lens, self.free]


def test_calls_behind_their_writers():
    """Each call reads what the one before it has just written, bit for bit as with a wait between them."""
    steps = 20
    a, b = Steps(steps=steps), Steps(steps=steps)
    g = torch.Generator(device="cuda").manual_seed(32)
    rows = [growing_step(i, a.n, 3, 64, g) for i in range(steps)]
    torch.cuda.synchronize()
    got = [a.step(*r, lambda: None) for r in rows]
    torch.cuda.synchronize()
    want = [b.step(*r, torch.cuda.synchronize) for r in rows]
    assert error() == 0
    for i, (x, y) in enumerate(zip(got, want)):
        for u, w in zip(x, y):
            assert torch.equal(u, w), "step %d" % i
    for u, w in zip(a.state(), b.state()):
        assert torch.equal(u, w)


def test_decode_takes_the_split_count_that_it_is_given():
    """One context of 100 units: 96 CTAs cut it into more pieces than 48 do, which
    shows in the last bits; left to itself the call takes 48 of a wave."""
    g = torch.Generator().manual_seed(33)
    codes = [torch.randint(0, 120, (100, 16, 8, 128), generator=g, dtype=torch.int32).to(torch.uint8).cuda().view(E4M3)
             for _ in range(2)]
    scales = [torch.randint(117, 121, (100, 8), generator=g, dtype=torch.int32).to(torch.uint8).cuda() for _ in range(2)]
    q = torch.randn(1, 32, 128, generator=g).to(BF).cuda()
    table = torch.randperm(100, generator=g).to(torch.int32).view(1, -1).cuda()
    out = {n: pa.pa_decode_fp8(q, *codes, *scales, table, i32([1600]), 0.05, kernel="mma", num_splits=n) for n in (0, 48, 96)}
    assert error() == 0
    assert not torch.equal(out[96], out[48])
    assert torch.equal(out[0], out[48])


def test_writes_on_two_streams_that_recode_what_their_blocks_hold():
    """A decode loop per stream, with a workspace that it keeps: each step's rows are
    larger, so the exponent of a partly filled block grows and its codes are rounded
    anew; codes, bytes and outputs bit for bit as one loop after the other gives them."""
    def loop(seed, n, Hk, D, B, steps=24):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = -(-steps // B)
        pool = [torch.zeros(n * W, B, Hk, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + \
               [torch.zeros(n * W, Hk, dtype=torch.uint8, device="cuda") for _ in range(2)]
        tables = torch.arange(n * W, dtype=torch.int32, device="cuda").view(W, n).t().contiguous()
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        lens = [torch.full((n,), i + 1, dtype=torch.int32, device="cuda") for i in range(steps)]
        rows = [growing_step(i, n, Hk, D, g) for i in range(steps)]
        q = torch.randn(n, 4 * Hk, D, generator=g, device="cuda").to(BF)
        ws = torch.empty(pa.pa_prefill_fp8_workspace_bytes(pool[0], n, n, 4 * Hk), dtype=torch.uint8, device="cuda")
        outs = [torch.zeros_like(q) for _ in range(steps)]

        def step(i):
            pa.pa_write_blocks_fp8(*rows[i], tables, lens[i], cu, *pool)
            pa.pa_prefill_fp8(q, *pool, tables, lens[i], cu, 0.125, out=outs[i], workspace=ws)
        return step, pool, outs

    shapes = [(34, 200, 8, 128, 16), (35, 150, 3, 64, 8)]
    runs = []
    for together in (False, True):
        loops = [loop(*s) for s in shapes]
        streams = [torch.cuda.Stream() for _ in loops]
        torch.cuda.synchronize()
        for i in range(24):
            for (step, _, _), s in zip(loops, streams):
                with torch.cuda.stream(s):
                    step(i)
                if not together:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert error() == 0
        runs.append([[x.view(torch.uint8) for x in pool] + outs for _, pool, outs in loops])
    for x, y in zip(*runs):
        for u, w in zip(x, y):
            assert torch.equal(u, w)
        assert int(x[2].min()) > 0 and torch.isfinite(x[-1]).all()
