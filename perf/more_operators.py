"""Measured cases of the tables built on the GPU, the 8-bit cache with block
scales and cross attention.

Five operators around a paged cache, each in its plain form (elementary torch
operations in 32 bits, rounded once at the end) and as the library's call:

  tables    a step's bookkeeping: finished requests give their blocks back,
            the others get blocks for their new tokens; block tables, lengths,
            row offsets and slots of the batch (pa_release_tables,
            pa_extend_tables);
  write8b   new tokens' K and V quantised to e4m3 with one power-of-two scale
            per block and KV head (pa_write_blocks_fp8);
  decode8b  single-query attention over that cache (pa_decode_fp8);
  chunk8b   attention of a chunk of new tokens over it, causal within the
            chunk (pa_prefill_fp8);
  cross     attention of decoder tokens over the paged states of an encoder,
            every token over all of them (pa_cross).

A case's lengths follow from the case alone (its "mix"); tables, free lists
and values follow from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BIAS = 127
E_MIN, E_MAX = -126, 120


# ------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = {"op": op, "h": 32, "hk": 8, "d": 128, "b": 16, "dtype": "bf16", "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a handful of short requests, one of them finished: all latency
        _case("tables-tiny", "tables", n=4, rows=8, done=1, width=8, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=27, b=4),
        # a large batch in steady state: decodes and prompts, finished requests
        _case("tables-serve", "tables", n=1024, rows=1536, done=64, width=2048, q_lo=1, q_hi=512, ctx_lo=0, ctx_hi=32000),
        # the cache write of one decode step: most tokens join a partly filled block
        _case("write8b-step", "write8b", n=64, q_lo=1, q_hi=1, ctx_lo=15, ctx_hi=8192),
        # the cache write of a batch of prompts, some behind a few earlier tokens
        _case("write8b-prompts", "write8b", n=48, q_lo=700, q_hi=4500, ctx_lo=0, ctx_hi=100),
        # a few short requests
        _case("decode8b-few", "decode8b", n=4, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=700),
        # mixed lengths, the ordinary decode batch
        _case("decode8b-mixed", "decode8b", n=256, q_lo=1, q_hi=1, ctx_lo=15, ctx_hi=8191),
        # long contexts, 64 query heads
        _case("decode8b-long", "decode8b", n=16, q_lo=1, q_hi=1, ctx_lo=32767, ctx_hi=32767, h=64, b=32),
        # drafted tokens checked by the target model: few rows, long contexts
        _case("chunk8b-draft", "chunk8b", n=64, q_lo=3, q_hi=8, ctx_lo=500, ctx_hi=8192),
        # a chunked scheduler's step: ragged chunks over ragged contexts
        _case("chunk8b-mixed", "chunk8b", n=16, q_lo=17, q_hi=700, ctx_lo=0, ctx_hi=6000),
        # a small fp32 model's decoder over short sources
        _case("cross-tiny-f32", "cross", n=4, q_lo=1, q_hi=9, ctx_lo=4, ctx_hi=31, h=4, hk=4, d=64, b=4, dtype="f32"),
        # beams and drafts of many requests: few tokens each over ragged sources, a KV head per query head
        _case("cross-step", "cross", n=128, q_lo=1, q_hi=8, ctx_lo=100, ctx_hi=1500, h=16, hk=16, d=64),
        # forced target prefixes over long sources
        _case("cross-targets", "cross", n=32, q_lo=64, q_hi=448, ctx_lo=1000, ctx_hi=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


HEADS = [(4, 4), (8, 1), (12, 4), (16, 16), (32, 8), (64, 8)]
MOST_SCORES = 9.0e8    # padded query rows x keys of one drawn chunk or cross call
MOST_TOKENS = 500000   # context tokens x KV heads / 8 of one drawn decode batch


def draw(rng):
    op = rng.choice(["tables", "write8b", "decode8b", "decode8b", "chunk8b", "chunk8b", "cross", "cross"])
    h, hk = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    mix = rng.randrange(1 << 20)
    if op == "tables":
        n, b = _log_int(rng, 1, 1024), rng.choice([4, 16, 16, 32])
        width = _log_int(rng, 4, 2048)
        q_hi = min(_log_int(rng, 1, 512), width * b // 2)
        ctx_hi = width * b - q_hi
        return _case("", op, n=n, rows=n + rng.randint(1, n + 1), done=rng.randint(0, 1 + n // 8), width=width, b=b,
                     q_lo=rng.randint(0, q_hi), q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, mix=mix)
    if op == "write8b":
        while True:
            q_hi = _log_int(rng, 1, 8000)
            c = _case("", op, n=_log_int(rng, 1, 256), q_lo=rng.randint(1, q_hi), q_hi=q_hi, ctx_lo=0,
                      ctx_hi=_log_int(rng, 1, 2000), hk=hk, d=d, b=rng.choice([8, 16, 16, 32, 64]),
                      dtype=rng.choice(["bf16", "bf16", "f32"]), mix=mix)
            if c["n"] * q_hi * hk <= 800000 and c["n"] * c["ctx_hi"] <= 200000:
                return c
    if op == "decode8b":
        if h // hk > 8:
            h = 8 * hk
        while True:
            hi = _log_int(rng, 1, 32768)
            c = _case("", op, n=_log_int(rng, 1, 256), q_lo=1, q_hi=1, ctx_lo=rng.randint(0, hi - 1), ctx_hi=hi - 1, h=h,
                      hk=hk, d=d, b=rng.choice([8, 16, 16, 32, 64]), mix=mix)
            if c["n"] * hi * hk / 8 <= MOST_TOKENS:
                return c
    while True:
        f32 = op == "cross" and rng.random() < 0.25
        q_hi = _log_int(rng, 1, 256 if f32 else 2048)
        ctx_hi = _log_int(rng, 1, 2048 if f32 else 8192)
        c = _case("", op, n=_log_int(rng, 1, 64), q_lo=rng.randint(1, q_hi), q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi),
                  ctx_hi=ctx_hi, h=h, hk=hk, d=d, b=rng.choice([4, 8, 16, 32] if f32 else [8, 16, 16, 32, 64]),
                  dtype="f32" if f32 else "bf16", mix=mix)
        q, ctx = _lens(c)
        keys = [x if op == "cross" else a + x for a, x in zip(q, ctx)]
        if len(q) * h * max(q) * max(max(keys), 1) <= (1.0e8 if f32 else MOST_SCORES) and sum(keys) * hk <= 2400000:
            return c


def _lens(case):
    """(new tokens, earlier or encoder tokens) of each sequence."""
    r = random.Random(case["mix"] * 7 + 1)
    q = [_log_int(r, max(case["q_lo"], 1), case["q_hi"]) if case["q_lo"] > 0 else r.randint(0, case["q_hi"])
         for _ in range(case["n"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    return q, ctx


def _row_lens(case):
    """(lengths of all rows, rows of the batch, rows that are done) of a tables case."""
    r = random.Random(case["mix"] * 7 + 2)
    lens = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["rows"])]
    order = list(range(case["rows"]))
    r.shuffle(order)
    done = min(case["done"], case["rows"] - case["n"])
    rows = order[:case["n"]]
    for i, x in zip(rows, _lens(case)[1]):
        lens[i] = x
    return lens, rows, order[case["n"]:case["n"] + done]


def _max_tokens(case):
    """Rows of the batch's slot map: the tokens, padded to a multiple of 64 as a captured step has them."""
    return -(-max(sum(_lens(case)[0]), 1) // 64) * 64


# ------------------------------------------------------------------ inputs
def _tables(lens, b, gen):
    """Block tables [n, widest] over a shuffled pool a tenth larger than needed, and the pool's blocks."""
    need = [-(-x // b) for x in lens]
    total = sum(need)
    pool = total + total // 10 + 1
    perm = torch.randperm(pool, generator=gen, device=DEV, dtype=torch.int32)
    width = max(1, max(need))
    n = torch.tensor(need, device=DEV)
    first = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=DEV)
    idx = torch.where(col[None] < n[:, None], first[:, None] + col[None], 0)
    return torch.where(col[None] < n[:, None], perm[idx], -1).contiguous(), pool


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rows(shape, gen):
    """Rows whose size varies from token to token, as a model's keys and values do."""
    size = torch.exp2(torch.randn(shape[:2], generator=gen, device=DEV)).unsqueeze(-1)
    return torch.randn(shape, generator=gen, device=DEV) * size


def _pool8(pool, b, hk, d, gen):
    """Codes and block scales of a whole 8-bit pool."""
    x = _rows((pool * b, hk, d), gen).view(pool, b, hk, d)
    e = _exponent(x.abs().amax((1, 3)))
    q = (x * torch.exp2(-e.float())[:, None, :, None]).to(torch.float8_e4m3fn)
    return q, (e + BIAS).to(torch.uint8)


def _prepare_tables(case, s, gen):
    lens, rows, done = _row_lens(case)
    new, b, width = _lens(case)[0], case["b"], case["width"]
    need = sum(-(-x // b) for x in lens)
    grow = sum(-(-(lens[r] + a) // b) - -(-lens[r] // b) for r, a in zip(rows, new))
    pool = need + grow + grow // 8 + 8
    perm = torch.randperm(pool, generator=gen, device=DEV, dtype=torch.int32)
    held = torch.tensor([-(-x // b) for x in lens], device=DEV)[:, None]
    idx = torch.cumsum(held, 0) - held + torch.arange(width, device=DEV)[None]
    s["tables"] = torch.where(torch.arange(width, device=DEV)[None] < held, perm[idx.clamp(max=pool - 1)], -1).contiguous()
    s["free_list"] = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    s["free_list"][:pool - need] = perm[need:]
    s["free_count"] = _i32([pool - need])
    s["lens"], s["rows"], s["done"], s["new"] = _i32(lens), _i32(rows), _i32(done), _i32(new)
    s["b"], s["max_tokens"] = b, _max_tokens(case)
    # where a step puts what it makes; the state before it stays, so that a step can be tried again
    s["lens_1"], s["lens_2"] = torch.empty_like(s["lens"]), torch.empty_like(s["lens"])
    s["count_1"], s["count_2"] = torch.empty_like(s["free_count"]), torch.empty_like(s["free_count"])
    n = len(rows)
    s["out"] = (torch.empty(n, width, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV),
                torch.empty(n + 1, dtype=torch.int32, device=DEV),
                torch.empty(s["max_tokens"], dtype=torch.int32, device=DEV))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + case["mix"])
    h, hk, d, b, dt = case["h"], case["hk"], case["d"], case["b"], _dtype(case)
    s = {"op": case["op"], "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "tables":
        return _prepare_tables(case, s, gen)
    new, ctx = _lens(case)
    cross = case["op"] == "cross"
    lens = ctx if cross else [a + x for a, x in zip(new, ctx)]
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    s["tables"], pool = _tables(lens, b, gen)
    s["lens"], s["cu"] = _i32(lens), _i32(cu)
    s["longest"], s["most_new"] = max(max(lens), 1), max(new)  # the scheduler knows them
    if case["op"] == "write8b":
        s["k"], s["v"] = _rows((cu[-1], hk, d), gen).to(dt), _rows((cu[-1], hk, d), gen).to(dt)
        s["kc"], s["ks"] = _pool8(pool, b, hk, d, gen)
        s["vc"], s["vs"] = _pool8(pool, b, hk, d, gen)
        return s
    if cross:
        s["kc"] = torch.randn(pool, b, hk, d, generator=gen, device=DEV).to(dt)
        s["vc"] = torch.randn(pool, b, hk, d, generator=gen, device=DEV).to(dt)
    else:
        s["kc"], s["ks"] = _pool8(pool, b, hk, d, gen)
        s["vc"], s["vs"] = _pool8(pool, b, hk, d, gen)
    s["q"] = torch.randn(cu[-1], h, d, generator=gen, device=DEV).to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------- plain forms
def _exponent(top):
    """The smallest e in [E_MIN, E_MAX] with top <= 448 * 2^e."""
    m, p = torch.frexp(top)
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(E_MIN, E_MAX)  # 448 = 0.875 * 2^9
    return torch.where(m == 0, E_MIN, e)


def _plain_tables(s):
    tables, b = s["tables"], s["b"]
    col = torch.arange(tables.shape[1], device=DEV)
    # finished requests' blocks go on the stack, request by request
    done, free = s["done"].long(), s["free_list"]
    held = (s["lens"][done] + b - 1) // b
    to = s["free_count"] + (torch.cumsum(held, 0) - held)[:, None] + col[None]
    room = torch.cat([free, free.new_zeros(1)])
    room[torch.where(col[None] < held[:, None], to, free.shape[0])] = tables[done]
    free.copy_(room[:-1])
    s["count_1"].copy_(s["free_count"] + held.sum())
    s["lens_1"].copy_(s["lens"]).index_fill_(0, done, 0)
    # the others' new tokens
    rows, new = s["rows"].long(), s["new"]
    old = s["lens_1"][rows]
    lens = old + new
    nb0, nb1 = (old + b - 1) // b, (lens + b - 1) // b
    first = torch.cumsum(nb1 - nb0, 0) - (nb1 - nb0)
    at = s["count_1"] - 1 - (first[:, None] + col[None] - nb0[:, None])
    fresh = (col[None] >= nb0[:, None]) & (col[None] < nb1[:, None])
    mine = torch.where(fresh, free[at.clamp(0, free.shape[0] - 1).long()], tables[rows])
    tables[rows] = mine
    s["count_2"].copy_(s["count_1"] - (nb1 - nb0).sum())
    s["lens_2"].copy_(s["lens_1"]).index_copy_(0, rows, lens)
    batch, seq_lens, cu, slots = s["out"]
    batch.copy_(torch.where(col[None] < nb1[:, None], mine, -1))
    seq_lens.copy_(lens)
    cu[0] = 0
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(slots.shape[0], device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), t.int(), right=True).clamp(max=rows.shape[0] - 1)
    pos = old[i] + t - cu[i]
    there = t < cu[-1]
    pos = torch.where(there, pos, 0)
    slots.copy_(torch.where(there, mine[i, pos // b] * b + pos % b, -1))
    return s["out"] + (tables, s["lens_2"], free, s["count_2"])


def _tokens(s, t):
    """(sequence, position) of each of the t new tokens."""
    at = torch.arange(t, device=DEV, dtype=torch.int32)
    i = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    return i, s["lens"][i] - s["cu"][i + 1] + at


def _plain_write8b(s):
    t, hk, d = s["k"].shape
    pool, b = s["kc"].shape[:2]
    i, pos = _tokens(s, t)
    phys = s["tables"][i, pos // b].long()
    # sequences whose new tokens begin inside a block: that block, and how many earlier ones it holds
    n = s["cu"][1:] - s["cu"][:-1]
    start = s["lens"] - n
    cut = torch.nonzero((n > 0) & (start % b > 0))[:, 0]
    head, part = s["tables"][cut, start[cut] // b].long(), start[cut] % b
    j, off = torch.nonzero(torch.arange(b, device=DEV)[None] < part[:, None], as_tuple=True)
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()
        e = _exponent(x.new_zeros(pool, hk).index_reduce_(0, phys, x.abs().amax(-1), "amax"))
        before = scales[head].int() - BIAS
        e[head] = torch.maximum(e[head], before)
        scales[phys] = (e[phys] + BIAS).to(torch.uint8)
        rows = codes.view(torch.uint8).view(-1, hk, d)
        old = head[j] * b + off
        shift = (before - e[head])[j].float()
        rows[old] = (rows[old].view(torch.float8_e4m3fn).float() * torch.exp2(shift)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        rows[phys * b + pos % b] = (x * torch.exp2(-e[phys].float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _context(s):
    """K and V of every sequence in 32 bits, padded: [n, hk, longest, d]; zeros past a sequence's end."""
    b = s["kc"].shape[1]
    at = torch.arange(s["longest"], device=DEV)
    there = at[None] < s["lens"][:, None]
    blocks = torch.where(there, s["tables"][:, at // b], 0).long()
    off = (at % b)[None].expand_as(blocks)
    k, v = s["kc"], s["vc"]
    if "ks" in s:
        k = k.view(torch.uint8)[blocks, off].view(torch.float8_e4m3fn).float()
        v = v.view(torch.uint8)[blocks, off].view(torch.float8_e4m3fn).float()
        k *= torch.exp2(s["ks"][blocks].float() - BIAS)[..., None]
        v *= torch.exp2(s["vs"][blocks].float() - BIAS)[..., None]
    else:
        k, v = k[blocks, off].float(), v[blocks, off].float()
    v *= there[..., None, None]
    return k.transpose(1, 2), v.transpose(1, 2)


def _plain_attention(s):
    q = s["q"]
    t, h, d = q.shape
    hk, n, most = s["kc"].shape[2], s["lens"].shape[0], s["most_new"]
    k, v = _context(s)
    i, pos = _tokens(s, t)
    r = torch.arange(t, device=DEV) - s["cu"][i]
    rows = q.new_zeros(n, most, h, d, dtype=torch.float32)
    rows[i, r] = q.float()
    rows = rows.view(n, most, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    x = torch.matmul(rows, k.transpose(-1, -2)).mul_(s["scale"]).view(n, h, most, -1)
    if s["op"] == "cross":
        last = (s["lens"] - 1)[:, None].expand(n, most)
    else:
        last = s["lens"][:, None] - (s["cu"][1:] - s["cu"][:-1])[:, None] + torch.arange(most, device=DEV)[None]
    x.masked_fill_(torch.arange(s["longest"], device=DEV) > last[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, hk, -1, s["longest"]), v).view(n, h, most, d)
    o /= torch.where(total == 0, 1.0, total)  # without a key: zeros
    return s["out"].copy_(o.transpose(1, 2)[i, r])


# --------------------------------------------------------------------- run
def _own(s):
    import paged_kv_cache_150_gb300 as pa

    if s["op"] == "tables":
        if "ws" not in s:  # the scratch that a program keeps for its steps of this size
            need = pa.pa_tables_workspace_bytes(max(s["rows"].shape[0], s["done"].shape[0]), s["tables"].shape[0])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        pa.pa_release_tables(s["tables"], s["lens"], s["free_list"], s["free_count"], s["done"], s["b"],
                             lens_out=s["lens_1"], free_count_out=s["count_1"], workspace=s["ws"])
        pa.pa_extend_tables(s["tables"], s["lens_1"], s["free_list"], s["count_1"], s["new"], s["b"], s["max_tokens"],
                            rows=s["rows"], lens_out=s["lens_2"], free_count_out=s["count_2"], out=s["out"],
                            workspace=s["ws"])
        return s["out"] + (s["tables"], s["lens_2"], s["free_list"], s["count_2"])
    if s["op"] == "write8b":
        pa.pa_write_blocks_fp8(s["k"], s["v"], s["tables"], s["lens"], s["cu"], s["kc"], s["vc"], s["ks"], s["vs"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    t, h, _ = s["q"].shape
    n = s["lens"].shape[0]
    if s["op"] == "decode8b":
        if "ws" not in s:
            need = pa.pa_decode_fp8_workspace_bytes(s["kc"], n, h, k_scale=s["ks"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return pa.pa_decode_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["scale"],
                                out=s["out"], workspace=s["ws"])
    if s["op"] == "chunk8b":
        if "ws" not in s:
            need = pa.pa_prefill_fp8_workspace_bytes(s["kc"], t, n, h)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return pa.pa_prefill_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["cu"], s["scale"],
                                 out=s["out"], workspace=s["ws"])
    if "ws" not in s:
        s["ws"] = torch.empty(pa.pa_cross_workspace_bytes(s["kc"], t, n, h), dtype=torch.uint8, device=DEV)
    return pa.pa_cross(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], s["scale"], out=s["out"],
                       workspace=s["ws"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "tables":
        return _plain_tables(state)
    if state["op"] == "write8b":
        return _plain_write8b(state)
    return _plain_attention(state)


# -------------------------------------------------------------------- work
def work(case):
    h, hk, d, b = case["h"], case["hk"], case["d"], case["b"]
    eb = 4 if case["dtype"] == "f32" else 2
    new, ctx = _lens(case)
    if case["op"] == "tables":
        lens, rows, done = _row_lens(case)
        used = sum(-(-(lens[r] + a) // b) for r, a in zip(rows, new))
        grow = sum(-(-(lens[r] + a) // b) - -(-lens[r] // b) for r, a in zip(rows, new))
        freed = sum(-(-lens[r] // b) for r in done)
        words = 3 * len(lens) + 6 * len(rows) + 2 * grow + 2 * freed + used + len(rows) * case["width"] + _max_tokens(case)
        return {"bytes": 4 * words, "flops": 2 * (len(rows) * case["width"] + _max_tokens(case))}
    tokens = sum(new)
    if case["op"] == "write8b":
        blocks = sum((x + a - 1) // b - x // b + 1 for a, x in zip(new, ctx))
        return {"bytes": 2 * tokens * hk * d * (eb + 1) + 2 * blocks * hk + 4 * blocks + 8 * len(new),
                "flops": 2 * tokens * hk * d * 3}
    cross = case["op"] == "cross"
    keys = sum(ctx) + (0 if cross else tokens)
    blocks = sum(-(-(x + (0 if cross else a)) // b) for a, x in zip(new, ctx))
    pairs = sum(a * x if cross else a * x + a * (a + 1) // 2 for a, x in zip(new, ctx))
    cache = 2 * keys * hk * d * eb if cross else 2 * (keys * hk * d + blocks * hk)
    return {"bytes": 2 * tokens * h * d * eb + cache + 4 * blocks + 8 * len(new), "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------- exact
def _e4m3_nearest(x):
    """The e4m3 value nearest to each |x| <= 448 (ties to an even last place), in 64 bits."""
    octave = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(-6, 8)
    octave = octave + (x.abs() >= torch.exp2(octave + 1)).double() - (x.abs() < torch.exp2(octave)).double()
    step = torch.exp2(octave.clamp(min=-6) - 3)
    return torch.round(x / step) * step  # torch.round: half to even


def _decoded(codes):
    """The values that e4m3 codes stand for, looked up, in 64 bits."""
    c = torch.arange(256, device=codes.device)
    exp, man = ((c >> 3) & 15).double(), (c & 7).double()
    val = torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp - 7), man / 8 * 2.0 ** -6)
    val = torch.where((c & 127) == 127, math.nan, val) * torch.where(c > 127, -1.0, 1.0)
    return val[codes.view(torch.uint8).long()]


def _least_exponent(top):
    """The smallest e in [E_MIN, E_MAX] with top <= 448 * 2^e, by search."""
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def _exact_tables(case, s):
    """The step request by request, on the host."""
    b, width = case["b"], case["width"]
    tables = s["tables"].cpu().tolist()
    stack = s["free_list"].cpu().tolist()
    top = s["free_count"].item()
    lens, rows, done = _row_lens(case)
    for r in done:
        for j in range(-(-lens[r] // b)):
            stack[top] = tables[r][j]
            top += 1
        lens[r] = 0
    batch, slots, cu = [], [], [0]
    for r, a in zip(rows, _lens(case)[0]):
        for pos in range(lens[r], lens[r] + a):
            if pos % b == 0:
                top -= 1
                tables[r][pos // b] = stack[top]
            slots.append(tables[r][pos // b] * b + pos % b)
        lens[r] += a
        cu.append(cu[-1] + a)
        nb = -(-lens[r] // b)
        batch.append(tables[r][:nb] + [-1] * (width - nb))
    slots += [-1] * (_max_tokens(case) - len(slots))
    return (_i32(batch), _i32([lens[r] for r in rows]), _i32(cu), _i32(slots), _i32(tables), _i32(lens), _i32(stack),
            _i32([top]))


def _exact_write8b(case, s):
    """Block by block: (values of the codes, scale bytes) of K and V."""
    b = case["b"]
    new, ctx = _lens(case)
    if sum(new) + 16 * len(new) > 30000 * b:
        return None
    tables, cu = s["tables"].cpu().tolist(), s["cu"].cpu().tolist()
    got = []
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        val, byte, x = _decoded(codes), scales.cpu(), x.double()
        work_list = []
        for i, (a, c) in enumerate(zip(new, ctx)):
            for blk in range(c // b, (c + a - 1) // b + 1):
                lo, hi = max(c, blk * b), min(c + a, (blk + 1) * b)
                work_list.append((tables[i][blk], cu[i] + lo - c, hi - lo, lo - blk * b))
        tops = torch.stack([x[t:t + n].abs().amax((0, 2)) for _, t, n, _ in work_list]).cpu().tolist()
        for (blk, t, n, off), top in zip(work_list, tops):
            e = [_least_exponent(y) for y in top]
            if off:
                was = [int(y) - BIAS for y in byte[blk]]
                e = [max(p, q) for p, q in zip(e, was)]
                shift = torch.tensor([float(p - q) for p, q in zip(was, e)], dtype=torch.float64, device=DEV)
                val[blk, :off] = _e4m3_nearest(val[blk, :off] * torch.exp2(shift)[None, :, None])
            byte[blk] = torch.tensor([y + BIAS for y in e], dtype=torch.uint8)
            unit = torch.exp2(torch.tensor(e, dtype=torch.float64, device=DEV))
            val[blk, off:off + n] = _e4m3_nearest(x[t:t + n] / unit[None, :, None])
        got.append((val, byte.to(DEV)))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(case, s)
    if case["op"] == "write8b":
        return _exact_write8b(case, s)
    q, h, hk, b = s["q"], case["h"], case["hk"], case["b"]
    g = h // hk
    new, ctx = _lens(case)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for i, (a, c) in enumerate(zip(new, ctx)):
        keys = c if case["op"] == "cross" else c + a
        blocks = s["tables"][i, :-(-keys // b)].long()

        def rows(cache, scales):
            if scales is None:
                return cache[blocks].double().flatten(0, 1)[:keys].transpose(0, 1)
            x = _decoded(cache.view(torch.uint8)[blocks]) * torch.exp2(scales[blocks].double() - BIAS)[:, None, :, None]
            return x.flatten(0, 1)[:keys].transpose(0, 1)

        k, v = rows(s["kc"], s.get("ks")), rows(s["vc"], s.get("vs"))
        for r in range(0, a if keys else 0, 256):
            n = min(256, a - r)
            x = torch.einsum("rkgd,kld->kgrl", q[at + r:at + r + n].double().view(n, hk, g, -1), k) * s["scale"]
            if case["op"] != "cross":
                x = torch.where(torch.arange(keys, device=DEV)[None] > c + r + torch.arange(n, device=DEV)[:, None], -math.inf, x)
            p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
            out[at + r:at + r + n] = torch.einsum("kgrl,kld->rkgd", p, v).reshape(n, h, -1)
        at += a
    return out
