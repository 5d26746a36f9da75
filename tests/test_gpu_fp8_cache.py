"""The 8-bit cache: write, read-back and block copy bit by bit against the rule
worked out in fp64, and decode attention over it against fp64."""
import math

import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _chunks import attention, make_tables, slots_of, tolerance, used_rows

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def code_values():
    """Values of the 256 e4m3 codes, from the format's definition."""
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        vals.append(-x if c > 127 else x)
    return torch.tensor(vals, dtype=torch.float64)


def rule(x):
    """(values of the codes, scale bytes) of rows x [t, hk, d], in fp64 on the CPU."""
    x = x.double()
    fin = torch.where(torch.isfinite(x), x.abs(), 0.0)
    top = fin.amax(-1)
    e = torch.full_like(top, -126.0)
    for step in range(-126, 120):  # raise e while the row does not fit
        e = torch.where(top > 448.0 * 2.0 ** step, torch.full_like(e, step + 1.0), e)
    y = x / torch.exp2(e).unsqueeze(-1)
    mag = y.abs()
    octave = torch.floor(torch.log2(mag.clamp(min=2.0 ** -12, max=448.0))).clamp(min=-6)
    unit = torch.exp2(octave - 3)
    r = torch.round(mag / unit) * unit  # half to even
    r = torch.where(torch.isinf(mag), torch.full_like(r, 448.0), r)
    return torch.where(torch.isnan(x), x, torch.copysign(r, y)), (e + 127).to(torch.uint8)


def pools(nb, bs, hk, d, fill=0x2b):
    codes = [torch.full((nb, bs, hk, d), fill, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.full((nb, bs, hk), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return codes + scales


def rows(shape, dtype, seed, special=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-40, 40, shape[:2], generator=g).float()).unsqueeze(-1)
    x = x.to(dtype)
    if special and x.numel() > 40:
        f = x.view(-1)
        f[1], f[5], f[7], f[11] = math.inf, -math.inf, math.nan, 0.0
        x[0, -1] = 0
        x[-1, 0] = torch.finfo(dtype).tiny  # clamps the exponent
        x[-1, -1, 0] = torch.finfo(dtype).max
    return x


SHAPES = [(7, 2, 64), (33, 8, 128), (5, 1, 256), (9, 3, 8), (6, 2, 96), (4, 2, 7), (3, 1, 1), (5, 2, 33), (3, 2, 1024),
          (200, 4, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hk,d", SHAPES)
def test_write_and_read_back_bit_by_bit(t, hk, d, dtype):
    bs = 4
    nb = t // bs + 3
    k, v = rows((t, hk, d), dtype, t), rows((t, hk, d), dtype, t + 1)
    g = torch.Generator().manual_seed(t + 2)
    slots = torch.randperm(nb * bs, generator=g)[:t].to(torch.int32)
    slots[t // 2] = -1
    kc, vc, ks, vs = pools(nb, bs, hk, d)
    pa.pa_reshape_and_cache_fp8(k.cuda(), v.cuda(), slots.cuda(), kc, vc, ks, vs)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    keep = slots >= 0
    at = slots[keep].long()
    vals = code_values()
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        want, byte = rule(x[keep])
        got = vals[codes.view(torch.uint8).cpu().view(-1, hk, d)[at].long()]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        assert torch.equal(scales.cpu().view(-1, hk)[at], byte)
        rest = torch.ones(nb * bs, dtype=torch.bool)
        rest[at] = False  # every other slot as it was
        assert bool((codes.view(torch.uint8).cpu().view(-1, hk, d)[rest] == 0x2b).all())
        assert bool((scales.cpu().view(-1, hk)[rest] == 99).all())
    for out_dt in (BF, F32):
        gk, gv = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots.cuda(), dtype=out_dt)
        assert pa.pa_get_device_error(raise_on_error=False) == 0
        for x, got in ((k, gk), (v, gv)):
            want, byte = rule(x[keep])
            want = (want * torch.exp2(byte.double() - 127).unsqueeze(-1)).to(out_dt)
            full = torch.zeros(t, hk, d, dtype=out_dt)
            full[keep] = want
            got = got.cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(full))
            assert torch.equal(got.nan_to_num(), full.nan_to_num())


def test_every_code_and_scale_byte_reads_back():
    hk, d, bs = 1, 256, 1
    kc, vc, ks, vs = pools(254, bs, hk, d)
    allc = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 256).expand(254, bs, hk, d).contiguous()
    kc.view(torch.uint8).copy_(allc)
    ks.copy_(torch.arange(1, 255, dtype=torch.uint8).view(254, 1, 1))
    slots = torch.arange(254, dtype=torch.int32, device="cuda")
    got = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots, dtype=F32)[0].cpu().view(254, 256)
    want = (code_values()[None] * torch.exp2(torch.arange(1, 255).double() - 127)[:, None]).float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(posinf=3e38), want.nan_to_num(posinf=3e38))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_rows(dtype):
    """k, v and the outputs start one element past a 16-byte boundary."""
    t, hk, d, bs = 9, 2, 64, 4
    k, v = rows((t, hk, d), dtype, 31), rows((t, hk, d), dtype, 32)
    kc, vc, ks, vs = pools(4, bs, hk, d)
    kd, vd = (torch.empty(t * hk * d + 1, dtype=dtype, device="cuda")[1:].view(t, hk, d) for _ in range(2))
    kd.copy_(k)
    vd.copy_(v)
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_fp8(kd, vd, slots, kc, vc, ks, vs)
    ref = pools(4, bs, hk, d)
    pa.pa_reshape_and_cache_fp8(k.cuda(), v.cuda(), slots, *ref)
    for a, b in zip((kc, vc, ks, vs), ref):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots, k=kd, v=vd)
    gk, gv = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots, dtype=dtype)
    assert torch.equal(kd.nan_to_num(), gk.nan_to_num()) and torch.equal(vd.nan_to_num(), gv.nan_to_num())
    assert pa.pa_get_device_error(raise_on_error=False) == 0


@pytest.mark.parametrize("d", [128, 33])
def test_slots_past_the_pool(d):
    hk, bs, nb = 2, 4, 3
    kc, vc, ks, vs = pools(nb, bs, hk, d)
    k = torch.ones(3, hk, d, dtype=BF, device="cuda")
    slots = torch.tensor([nb * bs, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_fp8(k, k, slots, kc, vc, ks, vs)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    assert int((ks != 99).sum()) == hk
    gk, gv = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    assert torch.count_nonzero(gk[0]) == 0 and torch.count_nonzero(gk[2]) == 0 and torch.equal(gk[1], k[1])


def test_write_and_read_rows_past_32_bits():
    """More than 2^31 codes in the pool and more than 2^31 elements in k and v."""
    hk, d, bs = 8, 128, 16
    t = (2 ** 31) // (hk * d) + 1000
    nb = -(-t // bs) + 1
    kc, vc, ks, vs = pools(nb, bs, hk, d)
    k = torch.zeros(t, hk, d, dtype=BF, device="cuda")
    k[-1000:] = torch.randn(1000, hk, d, device="cuda").to(BF)
    slots = torch.arange(t, dtype=torch.int32, device="cuda") + bs
    pa.pa_reshape_and_cache_fp8(k, k, slots, kc, vc, ks, vs)
    gk, gv = pa.pa_gather_cache_fp8(kc, vc, ks, vs, slots)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    want, byte = rule(k[-1000:].cpu())
    want = (want * torch.exp2(byte.double() - 127).unsqueeze(-1)).to(BF)
    assert torch.equal(gk[-1000:].cpu(), want) and torch.equal(gv[-1000:].cpu(), want)
    assert torch.count_nonzero(gk[:-1000]) == 0


@pytest.mark.parametrize("nb,bs,hk,d", [(12, 16, 8, 128), (9, 4, 2, 64), (8, 1, 1, 7), (8, 3, 1, 1)])
def test_copy_blocks(nb, bs, hk, d):
    g = torch.Generator().manual_seed(nb)
    kc, vc = (torch.randint(0, 256, (nb, bs, hk, d), generator=g).to(torch.uint8).cuda().view(E4M3) for _ in range(2))
    ks, vs = (torch.randint(1, 240, (nb, bs, hk), generator=g).to(torch.uint8).cuda() for _ in range(2))
    want = [x.view(torch.uint8).clone() for x in (kc, vc, ks, vs)]
    pairs = torch.tensor([[0, 5], [1, 6], [0, 7]], dtype=torch.int32)
    for w in want:
        w[pairs[:, 1].long()] = w[pairs[:, 0].long()]
    pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs.cuda())
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    for w, x in zip(want, (kc, vc, ks, vs)):
        assert torch.equal(w, x.view(torch.uint8))
    pa.pa_copy_blocks_fp8(kc, vc, ks, vs, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))


class Batch:
    """A pa_decode_fp8 call; stale slots hold NaN codes and the NaN scale byte."""

    def __init__(self, lens, H, Hk, D, block, seed, spread=6):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.block, self.scale = lens, block, 1.0 / math.sqrt(D)
        self.tables, pool = make_tables(lens, block, g)
        stale = ~used_rows(self.tables, lens, block, pool)
        self.vals, self.dev = [], {}
        for name in ("k", "v"):
            x = torch.randn(pool * block, Hk, D, generator=g)
            x *= torch.exp2(torch.randint(-spread, 3, (pool * block, Hk), generator=g).float()).unsqueeze(-1)
            cache, byte = x.to(BF), None
            c = torch.empty(pool, block, Hk, D, dtype=torch.uint8, device="cuda").view(E4M3)
            s = torch.empty(pool, block, Hk, dtype=torch.uint8, device="cuda")
            slots = torch.arange(pool * block, dtype=torch.int32, device="cuda")
            pa.pa_reshape_and_cache_fp8(cache.cuda(), cache.cuda(), slots, c, c.clone(), s, s.clone())
            c.view(torch.uint8).view(-1, Hk, D)[stale.cuda()] = 0x7f
            s.view(-1, Hk)[stale.cuda()] = 255
            codes = code_values()[c.view(torch.uint8).cpu().view(-1, Hk, D).long()]
            self.vals.append(codes * torch.exp2(s.cpu().view(-1, Hk).double() - 127).unsqueeze(-1))
            self.dev[name + "_cache"], self.dev[name + "_scale"] = c, s
        self.q = torch.randn(len(lens), H, D, generator=g).to(BF)
        self.dev.update(q=self.q.cuda(), block_tables=self.tables.cuda(), scale=self.scale,
                        seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())

    def check(self, out):
        # probabilities in fp16: 2^-11 each, or 2^-25 absolute of a weight of at least 1 (the largest score's)
        p_eps = 2.0 ** -11
        for i, L in enumerate(self.lens):
            r = slots_of(self.tables[i], L, self.block)
            k, v = self.vals[0][r].cuda(), self.vals[1][r].cuda()
            ref, amount, dots, top = attention(self.q[i:i + 1].cuda(), k, v, L - 1, self.scale)
            big = float(v.abs().max()) if L else 0.0
            tol = tolerance(BF, ref, amount, dots, top, L, ref.shape[-1], p_eps) + L * 2.0 ** -25 * big
            got = out[i:i + 1].double()
            assert torch.isfinite(got).all()
            assert float(((got - ref).abs() / tol).max()) <= 1.0, (i, L)


DECODE = [(32, 8, 128, 16), (8, 8, 128, 16), (16, 2, 64, 32), (12, 4, 128, 16), (8, 1, 128, 64), (7, 1, 64, 8),
          (8, 4, 128, 128), (6, 6, 128, 48), (8, 2, 128, 5), (8, 2, 256, 16), (4, 4, 64, 4), (4, 2, 64, 256)]


@pytest.mark.parametrize("kernel", ["auto", "simt"])
@pytest.mark.parametrize("H,Hk,D,block", DECODE)
def test_decode(H, Hk, D, block, kernel):
    b = Batch([1, 0, 15, 16, 17, 31, 33, 64, 65, 700, 129], H, Hk, D, block, seed=H + D + block)
    out = pa.pa_decode_fp8(**b.dev, kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    b.check(out)
    assert torch.count_nonzero(out[1]) == 0
    assert torch.equal(out, pa.pa_decode_fp8(**b.dev, kernel=kernel))


@pytest.mark.parametrize("H,Hk,D,block", [(32, 8, 128, 16), (64, 16, 64, 32), (6, 6, 128, 48), (8, 1, 128, 64)])
def test_decode_tensor_core_kernel_by_name(H, Hk, D, block):
    b = Batch([257, 40, 16, 3], H, Hk, D, block, seed=50)
    b.check(pa.pa_decode_fp8(**b.dev, kernel="mma"))
    assert pa.pa_get_device_error(raise_on_error=False) == 0


@pytest.mark.parametrize("H,Hk,D,block", [(8, 2, 256, 16), (8, 2, 128, 5), (7, 1, 64, 8)])
def test_decode_tensor_core_kernel_refusals(H, Hk, D, block):
    b = Batch([20], H, Hk, D, block, seed=51)
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_fp8(**b.dev, kernel="mma")


@pytest.mark.parametrize("kernel", ["auto", "simt"])
@pytest.mark.parametrize("splits", [1, 2, 5, 37, 900])
def test_decode_any_split_count(kernel, splits):
    b = Batch([3000, 1, 900, 50], 32, 8, 128, 16, seed=40)
    b.check(pa.pa_decode_fp8(**b.dev, num_splits=splits, kernel=kernel))


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_decode_over_rows_of_very_different_size(kernel):
    b = Batch([700, 300, 2000], 32, 8, 128, 16, seed=41, spread=40)
    b.check(pa.pa_decode_fp8(**b.dev, kernel=kernel))


@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_decode_bad_pages_and_lengths(kernel):
    b = Batch([200, 60], 8, 2, 128, 16, seed=42)
    tables = b.tables.clone()
    tables[0, 3], tables[1, 0] = b.dev["k_cache"].shape[0], -7
    for i, blk in ((0, 3), (1, 0)):
        r = slots_of(b.tables[i], b.lens[i], 16)[blk * 16:(blk + 1) * 16]
        for x in b.vals:
            x[r] = 0
    out = pa.pa_decode_fp8(**dict(b.dev, block_tables=tables.cuda()), kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    b.check(out)
    out = pa.pa_decode_fp8(**dict(b.dev, seq_lens=torch.tensor([200, 10 ** 6], dtype=torch.int32).cuda()), kernel=kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    assert torch.count_nonzero(out[1]) == 0


def test_decode_side_stream_and_graphs_that_share_a_workspace():
    a, b = Batch([200, 60, 3000], 32, 8, 128, 16, seed=43), Batch([7, 64], 32, 8, 128, 16, seed=44)
    need = max(pa.pa_decode_fp8_workspace_bytes(x.dev["k_cache"], len(x.lens), 32) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x.dev["q"]) for x in (a, b)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x, o in zip((a, b), outs):
            pa.pa_decode_fp8(**x.dev, out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    want = [o.clone() for o in outs]
    a.check(want[0])
    b.check(want[1])
    graphs = []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_fp8(**x.dev, out=o, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])


def test_python_refusals():
    b = Batch([20, 6], 8, 2, 128, 16, seed=45)
    d = b.dev
    with pytest.raises(TypeError):
        pa.pa_decode_fp8(**dict(d, q=d["q"].float()))
    with pytest.raises(TypeError):
        pa.pa_decode_fp8(**dict(d, k_cache=d["k_cache"].view(torch.uint8)))
    with pytest.raises(ValueError):
        pa.pa_decode_fp8(**dict(d, k_scale=d["k_scale"][:, :, :1]))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_fp8(**dict(d, q=torch.zeros(2, 32, 128, dtype=BF, device="cuda")))  # 16 heads per KV head
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_fp8(**d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    k = torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        pa.pa_reshape_and_cache_fp8(k, k, slots, d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"])
    with pytest.raises(ValueError):
        pa.pa_gather_cache_fp8(d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], slots, k=k)
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_fp8(k[:, :1].bfloat16(), k[:, :1].bfloat16(), slots, d["k_cache"], d["v_cache"],
                                    d["k_scale"], d["v_scale"])


@pytest.mark.parametrize("n,H,Hk,D,block", [(2049, 8, 4, 64, 8), (8300, 4, 2, 128, 16), (2600, 4, 2, 64, 5)])
def test_decode_more_sequences_than_shared_memory_lists(n, H, Hk, D, block):
    b = Batch([i * 7 % 20 for i in range(n)], H, Hk, D, block, seed=n)
    out = pa.pa_decode_fp8(**b.dev)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    some = sorted({0, 1, 2047, 2048, n - 1} | set(range(0, n, 53)))
    # the reference of a part of the batch: the same rows by another list
    part = Batch.__new__(Batch)
    part.__dict__.update(b.__dict__)
    part.lens, part.tables, part.q = [b.lens[i] for i in some], b.tables[some], b.q[some]
    part.check(out[some])


@pytest.mark.parametrize("which", ["k_scale", "v_scale", "q", "out"])
def test_decode_at_the_smallest_alignment(which):
    b = Batch([700, 3, 129], 32, 8, 128, 16, seed=71)
    kw = {}
    if which.endswith("scale"):
        x = b.dev[which]
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        y.copy_(x)
        b.dev[which] = y
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_decode_fp8(**b.dev, kernel="mma")
    else:
        y = torch.empty(b.q.numel() + 2, dtype=BF, device="cuda")[2:].view(b.q.shape)
        if which == "q":
            y.copy_(b.q)
            b.dev["q"] = y
        else:
            kw["out"] = y
    b.check(pa.pa_decode_fp8(**b.dev, **kw))
    assert pa.pa_get_device_error(raise_on_error=False) == 0


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_decode_a_query_row_that_is_not_finite_stays_alone(kernel, value):
    b = Batch([700, 300], 32, 8, 128, 16, seed=72)
    clean = pa.pa_decode_fp8(**b.dev, kernel=kernel)
    b.check(clean)
    b.dev["q"][0, 9, 3] = value
    out = pa.pa_decode_fp8(**b.dev, kernel=kernel)
    assert torch.isnan(out[0, 9]).all()
    out[0, 9] = clean[0, 9]
    b.check(out)


def test_decode_two_calls_at_once():
    bs = [Batch([3000, 900, 1], 32, 8, 128, 16, seed=s) for s in (73, 74)]
    want = [pa.pa_decode_fp8(**b.dev) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pa.pa_decode_fp8(**bs[i].dev))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


class Given(Batch):
    """One sequence with given rows k, v [L, Hk, D] (quantised by the library) and queries q [1, H, D]."""

    def __init__(self, k, v, q, scale, block, seed):
        g = torch.Generator().manual_seed(seed)
        L, Hk, D = k.shape
        self.lens, self.block, self.scale, self.q = [L], block, scale, q.to(BF)
        self.tables, pool = make_tables(self.lens, block, g)
        dev = pools(pool, block, Hk, D, fill=0x7f)
        dev[2].fill_(255)
        dev[3].fill_(255)
        rows_of = slots_of(self.tables[0], L, block)
        pa.pa_reshape_and_cache_fp8(k.to(BF).cuda(), v.to(BF).cuda(), rows_of.to(torch.int32).cuda(), *dev)
        self.dev = dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), dev), q=self.q.cuda(), scale=scale,
                        block_tables=self.tables.cuda(), seq_lens=torch.tensor(self.lens, dtype=torch.int32).cuda())
        self.rows_of = rows_of
        self.read()

    def read(self):
        """The values that the codes and scale bytes stand for."""
        self.vals = []
        for name in "kv":
            codes = code_values()[self.dev[name + "_cache"].view(torch.uint8).cpu().flatten(0, 1).long()]
            byte = self.dev[name + "_scale"].cpu().flatten(0, 1).double()
            self.vals.append(codes * torch.where(byte == 255, math.nan, torch.exp2(byte - 127)).unsqueeze(-1))

    def reference(self):
        k, v = (x[self.rows_of].cuda() for x in self.vals)
        return attention(self.q.cuda(), k, v, self.lens[0] - 1, self.scale) + (float(v.abs().max()),)


@pytest.mark.parametrize("H,Hk,D", [(8, 8, 64), (16, 8, 128), (8, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("below", [20.0, 22.5, 24.5, 25.25, 26.0])
@pytest.mark.parametrize("splits", [1, 0])
def test_decode_a_long_flat_tail_behind_one_large_weight(H, Hk, D, below, splits):
    """A weight of 1 and 65535 of 2^-below, whose V rows are as large and lie in
    other columns: the tail's sum must reach its columns as it reaches the
    softmax's sum."""
    L = 65536
    k, v, q = torch.zeros(L, Hk, D), torch.zeros(L, Hk, D), torch.zeros(1, H, D)
    whole = float(math.floor(below / 2) * 2)
    q[..., :2] = 1.0
    k[1:, :, 0], k[1:, :, 1] = -whole, whole - below  # e4m3 holds both beside each other
    v[0, :, 0] = 1.0
    v[1:, :, 1:] = 1.0
    b = Given(k, v, q, math.log(2.0), 16, seed=80)
    out = pa.pa_decode_fp8(**b.dev, kernel="mma", num_splits=splits).double()
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    ref, amount, dots, top, big = b.reference()
    # P's reference is 2^7, an fp16 subnormal is off by 2^-25: 2^-32 of the largest weight for each key
    tol = tolerance(BF, ref, amount, dots, top, L, D, 2.0 ** -11) + L * 2.0 ** -32 * big
    assert float(((out - ref).abs() / tol).max()) <= 1.0


def test_decode_values_of_every_size():
    """V rows of zeros, of the smallest scale byte that a write makes and of larger ones, alone and mixed."""
    L, Hk, D = 200, 8, 64
    g = torch.Generator().manual_seed(84)
    sizes = [0.0, 2.0 ** -126, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 112]
    for pick in ([0], [1], [5], [0, 1], [0, 3], [1, 5], [2, 4], [0, 1, 2, 3, 4, 5]):
        size = torch.tensor([sizes[i] for i in pick])[torch.randint(0, len(pick), (L, Hk, 1), generator=g)]
        b = Given(torch.randn(L, Hk, D, generator=g), torch.randn(L, Hk, D, generator=g).clamp(-3, 3) * size,
                  torch.randn(1, 16, D, generator=g), 0.125, 16, seed=85)
        ref, amount, dots, top, big = b.reference()
        tol = tolerance(BF, ref, amount, dots, top, L, D, 2.0 ** -11) + L * 2.0 ** -25 * big - 1e-30 + 2.0 ** -134
        for kernel in ("mma", "simt"):
            out = pa.pa_decode_fp8(**b.dev, kernel=kernel).double()
            assert float(((out - ref).abs() / tol).max()) <= 1.0, (pick, kernel)
    assert pa.pa_get_device_error(raise_on_error=False) == 0


@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_decode_a_seen_row_with_the_scale_byte_of_nan(kernel, which):
    """Byte 255 is NaN in E8M0: the heads that read such a row get NaN, no other does."""
    b = Batch([700, 300, 33, 1], 32, 8, 128, 16, seed=81)
    clean = pa.pa_decode_fp8(**b.dev, kernel=kernel)
    b.check(clean)
    want = clean.clone()
    for i, pos, h in ((0, 0, 1), (0, 699, 5), (1, 123, 0), (2, 32, 7), (3, 0, 2)):
        at = int(slots_of(b.tables[i], b.lens[i], 16)[pos])
        b.dev[which + "_scale"].view(-1, 8)[at, h] = 255
        want[i, 4 * h:4 * h + 4] = math.nan
    for splits in (0, 1, 7):
        out = pa.pa_decode_fp8(**b.dev, kernel=kernel, num_splits=splits)
        assert pa.pa_get_device_error(raise_on_error=False) == 0
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        tight = torch.nan_to_num(out.double() - want.double()).abs().max()
        assert float(tight) <= (0.0 if splits == 0 else 2.0 ** -7 * float(torch.nan_to_num(want).abs().max()))


@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_the_smallest_scale_byte(kernel, D):
    """Byte 0 stands for 2^-127: K rows of it behind large queries, V rows of it alone, both at once."""
    L, Hk, H = 300, 8, 16
    g = torch.Generator().manual_seed(82)
    q = torch.randn(1, H, D, generator=g) * 2.0 ** 118
    for small_k, small_v in ((True, False), (False, True), (True, True)):
        b = Given(torch.randn(L, Hk, D, generator=g), torch.randn(L, Hk, D, generator=g),
                  q if small_k else q * 2.0 ** -118, 1.0 / math.sqrt(D), 16, seed=83)
        for name, small in (("k", small_k), ("v", small_v)):
            if small:
                b.dev[name + "_scale"].view(-1, Hk)[b.rows_of.cuda()] = 0
        b.read()
        out = pa.pa_decode_fp8(**b.dev, kernel=kernel).double()
        assert pa.pa_get_device_error(raise_on_error=False) == 0
        ref, amount, dots, top, big = b.reference()
        # bf16 is off by up to 2^-134 where it has no more bits left (below 2^-126)
        tol = tolerance(BF, ref, amount, dots, top, L, D, 2.0 ** -11) + L * 2.0 ** -25 * big - 1e-30 + 2.0 ** -134
        assert float(((out - ref).abs() / tol).max()) <= 1.0
        assert float(ref.abs().max()) > 2.0 ** -126


@pytest.mark.parametrize("H,Hk,D,block", [(8, 1, 128, 16), (4, 2, 64, 8), (8, 2, 128, 48), (32, 8, 128, 16)])
@pytest.mark.parametrize("splits", [1, 3, 0])
def test_decode_bad_pages_in_every_box_of_a_stage(H, Hk, D, block, splits):
    """Bad entries at every place of a stage, one at a time, every other one and
    all of them; the codes that they would have named hold NaN."""
    lens = [block * n - 1 for n in range(1, 18)] + [block * 40] * 3
    b = Batch(lens, H, Hk, D, block, seed=86)
    tables, nb = b.tables.clone(), b.dev["k_cache"].shape[0]
    bad = [(n, n) for n in range(17)] + [(17, n) for n in range(40)] + [(18, n) for n in range(0, 40, 2)]
    bad += [(19, n) for n in range(1, 40, 3)]
    for i, n in bad:
        at = int(b.tables[i, n])
        for name in "kv":
            b.dev[name + "_cache"].view(torch.uint8)[at] = 0x7f
            b.dev[name + "_scale"][at] = 255
        rows_of = slots_of(b.tables[i], lens[i], block)[n * block:(n + 1) * block]
        for x in b.vals:
            x[rows_of] = 0
        tables[i, n] = (-1, nb, -2 ** 31, 2 ** 31 - 1)[n % 4]
    dev = dict(b.dev, block_tables=tables.cuda())
    out = pa.pa_decode_fp8(**dev, kernel="mma", num_splits=splits)
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    b.check(out)
    for _ in range(5):
        assert torch.equal(out, pa.pa_decode_fp8(**dev, kernel="mma", num_splits=splits))
    assert pa.pa_get_device_error(raise_on_error=False) == pa._lib.PA_ERR_DEVICE_BOUNDS
    assert torch.count_nonzero(out[17]) == 0


def test_decode_at_the_longest_reach():
    """2^31 - 8 positions through a table that names one block over and over."""
    block, n = 8 * 127 * 113, 3 * 5 * 29 * 43
    L = block * n
    assert L == 2 ** 31 - 8
    kc, vc, ks, vs = pools(1, block, 2, 64)
    ones = torch.ones(block, 2, 64, dtype=BF, device="cuda")
    pa.pa_reshape_and_cache_fp8(torch.zeros_like(ones), ones, torch.arange(block, dtype=torch.int32, device="cuda"), kc, vc,
                                ks, vs)
    out = pa.pa_decode_fp8(torch.ones(1, 8, 64, dtype=BF, device="cuda"), kc, vc, ks, vs,
                           torch.zeros(1, n, dtype=torch.int32, device="cuda"),
                           torch.tensor([L], dtype=torch.int32, device="cuda"), 1.0, kernel="mma")
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    # every score is 0: the sums of a CTA are whole numbers below 2^24 times a
    # power of two, the merge rounds once for each of at most 2^10 pieces
    assert float((out.double() - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -13


@pytest.mark.parametrize("H,Hk,D,block", DECODE)
def test_decode_on_the_cuda_cores(H, Hk, D, block):
    """fp32 probabilities: no allowance for their rounding."""
    b = Batch([1, 0, 15, 16, 17, 31, 33, 64, 65, 700, 129], H, Hk, D, block, seed=H + D + block)
    out = pa.pa_decode_fp8(**b.dev, kernel="simt")
    for i, L in enumerate(b.lens):
        at = slots_of(b.tables[i], L, block)
        ref, amount, dots, top = attention(b.q[i:i + 1].cuda(), b.vals[0][at].cuda(), b.vals[1][at].cuda(), L - 1, b.scale)
        tol = tolerance(BF, ref, amount, dots, top, L, D, 0.0)
        assert float(((out[i:i + 1].double() - ref).abs() / tol).max()) <= 1.0, (i, L)


@pytest.mark.parametrize("H,Hk,D,block", DECODE)
def test_which_kernel_a_decode_takes(H, Hk, D, block):
    b = Batch([300, 17, 1], H, Hk, D, block, seed=102)
    out = pa.pa_decode_fp8(**b.dev)
    step = math.gcd(block, 128 // max(n for n in (1, 2, 4, 8) if Hk % n == 0))
    if D <= 128 and block % 8 == 0 and step * Hk % 16 == 0:
        assert torch.equal(out, pa.pa_decode_fp8(**b.dev, kernel="mma"))
    else:
        assert torch.equal(out, pa.pa_decode_fp8(**b.dev, kernel="simt"))
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_decode_fp8(**b.dev, kernel="mma")


@pytest.mark.parametrize("D,block", [(64, 16), (128, 16), (256, 4)])
def test_fp32_chunk_attention_over_rows_read_back(D, block):
    """A chunk over a pool of rows read back in fp32: nothing is rounded to fewer bits on the way."""
    b = Batch([303], 8, 2, D, block, seed=103)
    rows_of = slots_of(b.tables[0], 303, block)
    n = -(-303 // block)
    slots = torch.cat([rows_of, torch.full((n * block - 303,), -1)]).to(torch.int32).cuda()
    k8, v8 = pa.pa_gather_cache_fp8(b.dev["k_cache"], b.dev["v_cache"], b.dev["k_scale"], b.dev["v_scale"], slots, dtype=F32)
    q = torch.randn(64, 8, D, generator=torch.Generator().manual_seed(104)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = pa.pa_prefill(q, k8.view(n, block, 2, D), v8.view(n, block, 2, D), torch.arange(n, **i32)[None].contiguous(),
                        torch.tensor([303], **i32), torch.tensor([0, 64], **i32), b.scale)
    assert pa.pa_get_device_error(raise_on_error=False) == 0
    ref, amount, dots, top = attention(q, b.vals[0][rows_of].cuda(), b.vals[1][rows_of].cuda(), 303 - 64, b.scale)
    tol = tolerance(F32, ref, amount, dots, top, 303, D, 0.0)
    assert float(((out.double() - ref).abs() / tol).max()) <= 1.0


@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0 ** -40, 8.0])
def test_decode_scales_of_every_sign_and_size(kernel, scale):
    b = Batch([700, 1, 40], 32, 8, 128, 16, seed=105)
    b.scale = b.dev["scale"] = scale
    b.check(pa.pa_decode_fp8(**b.dev, kernel=kernel))
    assert pa.pa_get_device_error(raise_on_error=False) == 0
