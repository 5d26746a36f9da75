"""Cross attention over paged encoder states against fp64."""
import math

import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from _chunks import Chunk, attention, slots_of, tolerance

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
BOUNDS = pa._lib.PA_ERR_DEVICE_BOUNDS


class Cross(Chunk):
    """seq_lens: the encoders' lengths."""

    def run(self, **kw):
        d = dict(self.dev)
        d["kv_lens"] = d.pop("seq_lens")
        d.update(kw)
        return pa.pa_cross(**d)

    def reference(self, i):
        L = self.seq_lens[i]
        rows = slots_of(self.tables[i], L, self.block)
        return attention(self.q[self.cu[i]:self.cu[i + 1]].cuda(), self.k[rows].cuda(), self.v[rows].cuda(), L, self.scale)


def p_eps(dtype, kernel):
    return 2.0 ** -8 if dtype == BF and kernel != "simt" else 0.0


def error():
    return pa.pa_get_device_error(raise_on_error=False)


SHAPES = [(32, 8, 128, 16), (16, 16, 64, 16), (8, 1, 128, 64), (12, 4, 64, 8), (6, 6, 128, 48), (64, 1, 64, 16), (5, 5, 128, 24)]
SLOW = [(4, 4, 64, 4), (8, 2, 256, 16), (4, 2, 128, 5)]
Q, L = [1, 5, 0, 128, 33, 260, 2, 70], [700, 1, 9, 128, 129, 300, 0, 257]


@pytest.mark.parametrize("H,Hk,D,block", SHAPES)
def test_tensor_cores(H, Hk, D, block):
    c = Cross(Q, L, H, Hk, D, block, BF, seed=H + D + block)
    out = c.run(kernel="mma")
    assert error() == 0
    c.check(out, p_eps(BF, "mma"))
    assert torch.count_nonzero(out[c.cu[6]:c.cu[7]]) == 0  # no encoder state
    assert torch.equal(out, c.run())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk,D,block", SHAPES[:3] + SLOW)
def test_cuda_cores(H, Hk, D, block, dtype):
    c = Cross([1, 5, 0, 70, 33, 2], [200, 1, 9, 128, 65, 0], H, Hk, D, block, dtype, seed=H + D + block)
    out = c.run(kernel="simt")
    assert error() == 0
    c.check(out, p_eps(dtype, "simt"))


@pytest.mark.parametrize("dtype,layout,D", [(BF, "split", 128), (F32, "split", 64), (F32, "row", 128)])
def test_layouts(dtype, layout, D):
    c = Cross([9, 3], [100, 40], 8, 2, D, 16, dtype, seed=4, layout=layout)
    c.check(c.run(), p_eps(dtype, "simt" if layout == "split" else "auto"))


@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("splits", [1, 3, 40, 900])
def test_any_split_count(kernel, splits):
    c = Cross([200, 3, 64], [900, 1500, 64], 16, 4, 64, 16, BF, seed=5)
    c.check(c.run(num_splits=splits, kernel=kernel), p_eps(BF, kernel))


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 7, 13, 29])
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_tiles_per_cta(D, splits):
    """Tiles of a few rows, several to a CTA, cut at either end of its range."""
    c = Cross([3, 1, 8, 5, 2, 0, 7] * 3, [1000 - 41 * i for i in range(21)], 4, 2, D, 16, BF, seed=70 + splits)
    out = c.run(num_splits=splits, kernel="mma")
    assert error() == 0
    c.check(out, p_eps(BF, "mma"))


@pytest.mark.parametrize("splits", [0, 1, 4, 6, 30])
@pytest.mark.parametrize("kernel", ["mma", "simt"])
@pytest.mark.parametrize("Hk", [1, 3, 10, 12, 20])
def test_numbers_of_heads_and_ctas(Hk, kernel, splits):
    """The order of heads and tiles depends on the CTAs that a head has: none, some, with and without a common divisor."""
    c = Cross([5, 300, 1, 0, 140, 33], [200, 500, 129, 64, 0, 1000], Hk, Hk, 64, 16, BF, seed=90 + Hk)
    out = c.run(num_splits=splits, kernel=kernel)
    assert error() == 0
    c.check(out, p_eps(BF, kernel))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384])
def test_encoder_lengths_around_unit_edges(n):
    c = Cross([3, 300], [n, n], 8, 2, 128, 16, BF, seed=60 + n)
    c.check(c.run(), p_eps(BF, "mma"))


def test_one_token_is_decode():
    c = Cross([1] * 5, [1, 16, 0, 500, 3001], 32, 8, 128, 16, BF, seed=7)
    d = c.dev
    one = pa.pa_decode(d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["seq_lens"], c.scale)
    c.check(one, 2.0 ** -8)
    c.check(c.run(), p_eps(BF, "mma"))


def test_more_tokens_than_states_and_the_last_token_is_the_causal_one():
    """The last token of a causal chunk sees every position: the same output, bit for bit."""
    c = Cross([150, 40], [20, 700], 8, 2, 128, 16, BF, seed=8)
    out = c.run()
    c.check(out, p_eps(BF, "mma"))
    causal = pa.pa_prefill(**c.dev, kernel="simt")
    full = c.run(kernel="simt")
    assert torch.equal(causal[[149, 189]], full[[149, 189]])


@pytest.mark.parametrize("dtype,kernel", [(BF, "mma"), (BF, "simt"), (F32, "auto")])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_values_that_are_not_finite(dtype, kernel, value):
    """Stale slots hold NaN already; a seen one reaches every token of its sequence, in its head and column only."""
    c = Cross([40, 20], [100, 130], 8, 2, 128, 16, dtype, seed=9)
    clean = c.run(kernel=kernel)
    row = int(slots_of(c.tables[0], 100, 16)[99])
    c.v[row, 1, 5] = value
    out = c.run(kernel=kernel, v_cache=c.v.view(c.dev["v_cache"].shape).cuda())
    assert error() == 0
    assert not torch.isfinite(out[:40, 4:, 5]).any()
    keep = torch.ones(8, 128, dtype=torch.bool, device="cuda")
    keep[4:, 5] = False
    assert torch.equal(out[:40][:, keep], clean[:40][:, keep]) and torch.equal(out[40:], clean[40:])


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_rows_of_no_sequence_stay(kernel):
    c = Cross([5, 40], [70, 40], 8, 2, 128, 16, BF, seed=10, lead=3, tail=7)
    out = torch.full_like(c.dev["q"], 7.0)
    c.run(out=out, kernel=kernel)
    c.check(out, p_eps(BF, kernel))
    assert bool((out[:3] == 7).all()) and bool((out[48:] == 7).all())


@pytest.mark.parametrize("kernel", ["mma", "simt"])
def test_bad_pages_lengths_and_offsets(kernel):
    c = Cross([30, 8], [200, 60], 8, 2, 128, 16, BF, seed=11)
    tables = c.tables.clone()
    tables[0, 3] = c.dev["k_cache"].shape[0]
    rows = slots_of(c.tables[0], 200, 16)[48:64]
    c.k[rows], c.v[rows] = 0, 0
    out = c.run(block_tables=tables.cuda(), kernel=kernel)
    assert error() == BOUNDS
    c.check(out, p_eps(BF, kernel))
    for cu in ([0, 39, 38], [-1, 30, 38], [0, 30, 39]):
        out = torch.full_like(c.dev["q"], 3.0)
        c.run(cu_q_lens=torch.tensor(cu, dtype=torch.int32).cuda(), out=out, kernel=kernel)
        assert error() == BOUNDS and bool((out == 3).all())
    for bad in (-1, c.tables.shape[1] * 16 + 1, 2 ** 31 - 1):
        out = c.run(kv_lens=torch.tensor([bad, 60], dtype=torch.int32).cuda(), kernel=kernel)
        assert error() == BOUNDS and torch.count_nonzero(out[:30]) == 0


def test_graphs_that_share_a_workspace():
    a, b = Cross([30, 100], [700, 100], 32, 8, 128, 16, BF, seed=12), Cross([7, 64, 1], [90, 640, 2000], 32, 8, 128, 16, BF, seed=13)
    need = max(pa.pa_cross_workspace_bytes(x.dev["k_cache"], x.dev["q"].shape[0], len(x.q_lens), 32) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x.dev["q"]) for x in (a, b)]
    want, graphs = [], []
    for x, o in zip((a, b), outs):
        want.append(x.run())
        x.check(want[-1], p_eps(BF, "mma"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(out=o, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i])
            outs[i].zero_()


def test_python_refusals():
    c = Cross([30, 8], [200, 60], 8, 2, 128, 16, BF, seed=14)
    d = c.dev
    for bad in (dict(q=d["q"].float()), dict(block_tables=d["block_tables"][0]), dict(cu_q_lens=d["cu_q_lens"][:2]),
                dict(kv_lens=d["seq_lens"].long()), dict(out=torch.empty(1, device="cuda")), dict(q=d["q"].cpu()),
                dict(v_cache=d["v_cache"].float()), dict(kv_lens=d["seq_lens"][None])):
        with pytest.raises((ValueError, TypeError)):
            c.run(**bad)
    with pytest.raises(pa.PagedAttentionError):
        c.run(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PagedAttentionError):
        c.run(scale=float("nan"))
