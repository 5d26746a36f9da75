"""Inputs and 64-bit references for the 8-bit cache with block scales."""
import math

import torch

from _chunks import attention, make_tables, slots_of, tolerance, used_rows

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def code_values():
    """Values of the 256 e4m3 codes, from the format's definition."""
    c = torch.arange(256)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    x = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    x = torch.where((c & 127) == 127, math.nan, x)
    return torch.where(c > 127, -x, x)


def nearest_e4m3(y):
    """y (fp64) rounded to the nearest e4m3 value, ties to even, infinities and more to +-448, NaN stays."""
    mag = y.abs()
    octave = torch.floor(torch.log2(mag.clamp(min=2.0 ** -12, max=448.0))).clamp(min=-6)
    unit = torch.exp2(octave - 3)
    r = (torch.round(mag / unit) * unit).clamp(max=448.0)
    return torch.where(torch.isnan(y), y, torch.copysign(r, y))


def least_exponent(top):
    """The smallest e in [-126, 120] with top <= 448 * 2^e."""
    e = -126
    while e < 120 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def write_rule(x, values, scales, tables, lens, cu, block, pool):
    """What pa_write_blocks_fp8 makes of rows x [T, Hk, D]: (values of the codes
    [pool, B, Hk, D] in fp64, bytes [pool, Hk]), from those before."""
    values, scales = values.clone(), scales.clone()
    x = x.double()
    for i, L in enumerate(lens):
        n = cu[i + 1] - cu[i]
        for blk in range((L - n) // block, -(-L // block)):
            lo, hi = max(L - n, blk * block), min(L, (blk + 1) * block)
            if lo >= hi:
                continue
            p, off = int(tables[i][blk]), lo - blk * block
            rows = x[cu[i] + lo - (L - n):cu[i] + hi - (L - n)]
            for h in range(x.shape[1]):
                y = rows[:, h]
                fin = y[torch.isfinite(y)].abs()
                e, byte = least_exponent(float(fin.max()) if fin.numel() else 0.0), None
                if off:
                    was = int(scales[p, h])
                    old = min(was, 247) - 127
                    e = max(e, old)
                    byte = was if was > 247 else None
                    if e > old:
                        values[p, :off, h] = nearest_e4m3(values[p, :off, h] * 2.0 ** (old - e))
                scales[p, h] = e + 127 if byte is None else byte
                values[p, off:off + hi - lo, h] = nearest_e4m3(y / 2.0 ** e)
    return values, scales


class Block8:
    """A batch over an 8-bit cache with block scales: n_i new tokens of seq_lens[i]
    positions.  Slots of no sequence hold NaN codes, unused blocks the NaN byte."""

    def __init__(self, q_lens, seq_lens, H, Hk, D, block, seed, spread=4, lead=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.seq_lens, self.block, self.scale = q_lens, seq_lens, block, 1.0 / math.sqrt(D)
        self.tables, pool = make_tables(seq_lens, block, g)
        used = used_rows(self.tables, seq_lens, block, pool).view(pool, block)
        self.vals, codes, scales = [], [], []
        for _ in range(2):
            c = torch.randint(0, 256, (pool, block, Hk, D), generator=g, dtype=torch.int32).to(torch.uint8)
            c = torch.where((c & 127) == 127, c - 8, c)  # no NaN among the used ones
            s = torch.randint(120 - spread, 121, (pool, Hk), generator=g, dtype=torch.int32).to(torch.uint8)
            c[~used] = 0x7f
            s[~used.any(1)] = 255
            codes.append(c)
            scales.append(s)
            self.vals.append(self.decoded(c, s).view(pool * block, Hk, D))
        self.codes, self.scales = codes, scales
        self.lead, cu = lead, [lead]
        for n in q_lens:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.q = torch.randn(cu[-1] + tail, H, D, generator=g).to(BF)
        i32 = torch.int32
        self.dev = dict(q=self.q.cuda(), k_cache=codes[0].cuda().view(E4M3), v_cache=codes[1].cuda().view(E4M3),
                        k_scale=scales[0].cuda(), v_scale=scales[1].cuda(), block_tables=self.tables.cuda(),
                        seq_lens=torch.tensor(seq_lens, dtype=i32).cuda(), cu_q_lens=torch.tensor(cu, dtype=i32).cuda(),
                        scale=self.scale)

    @staticmethod
    def decoded(codes, scales):
        s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
        return code_values()[codes.long()] * s[:, None, :, None]

    def decode_args(self):
        return {k: v for k, v in self.dev.items() if k != "cu_q_lens"}

    def check(self, out, p_eps, tail=0.0):
        """tail: the absolute part of a probability's rounding, of the largest |v| per key."""
        for i, (n, L) in enumerate(zip(self.q_lens, self.seq_lens)):
            if n == 0:
                continue
            r = slots_of(self.tables[i], L, self.block)
            k, v = self.vals[0][r].cuda(), self.vals[1][r].cuda()
            ref, amount, dots, top = attention(self.q[self.cu[i]:self.cu[i + 1]].cuda(), k, v, L - n, self.scale)
            big = float(v.abs().max()) if L else 0.0
            tol = tolerance(BF, ref, amount, dots, top, L, ref.shape[-1], p_eps) + tail * L * big
            got = out[self.cu[i]:self.cu[i + 1]].double()
            assert torch.isfinite(got).all(), "sequence %d has values that are not finite" % i
            worst = float(((got - ref).abs() / tol).max())
            assert worst <= 1.0, "sequence %d: %.2f of the bound" % (i, worst)
