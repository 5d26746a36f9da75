"""Tables built on the GPU: rows named twice, and calls that only the C entry makes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_150_gb300 as pa
from test_gpu_tables import BOUNDS, State, error, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,R", [(2, 6), (40, 6000), (1024, 1500), (2500, 3000), (2600, 5000)])
def test_a_row_named_twice_belongs_to_the_first(n, R):
    """The refused call's lengths and tables do not depend on which store comes last."""
    rng = np.random.default_rng(n)
    s = State(R, 4, 4 * R, 4, seed=n)
    s.lens.copy_(i32(rng.integers(1, 15, R)))
    s.tables.copy_(i32(rng.integers(0, 4 * R, (R, 4))))
    rows = rng.integers(0, min(R, max(n // 3, 1)), n)  # each row about three times
    first = np.full(R, n)
    np.minimum.at(first, rows, np.arange(n))
    mine = first[rows] == np.arange(n)
    lens, tables = s.lens.cpu().numpy(), s.tables.cpu().numpy()
    want = np.where(mine, lens[rows], 0)
    blocks = -(-want // 4)
    want_t = np.where(np.arange(4)[None] < blocks[:, None], tables[rows], -1)
    before = s.snapshot()
    for _ in range(5):
        out = s.extend(rows, [1] * n, n)
        assert error() == BOUNDS
        assert (out[1].cpu().numpy() == want).all() and (out[0].cpu().numpy() == want_t).all()
        for x, y in zip(before, s.args()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("n,W,most", [(5, 30, 9), (700, 300, 500), (2100, 40, 30), (3, 5000, 70000)])
@pytest.mark.parametrize("named", [False, True])
def test_a_call_that_wants_no_batch_tables(n, W, most, named):
    """batch_tables NULL (the C entry): state, lengths, offsets and slots as with
    them; small batches in one kernel, larger ones in two."""
    rng = np.random.default_rng(n)
    block, R = 16, n + 4
    rows = rng.permutation(R)[:n] if named else np.arange(n)
    new = np.minimum(rng.integers(0, most + 1, n), W * block // 2)
    max_tokens = int(new.sum()) + 7
    states = []
    for _ in range(2):
        s = State(R, W, int(R * (W // 2 + 2)), block, seed=n)
        first = [int(x) for x in np.random.default_rng(1).integers(0, W * block // 2, R)]
        s.step(None, first)
        states.append(s)
    a, b = states
    want = a.extend(rows if named else None, new, max_tokens)
    lib, ws = pa._lib.load(), torch.empty(pa.pa_tables_workspace_bytes(n, R), dtype=torch.uint8, device="cuda")
    ints = [t.data_ptr() for t in (b.tables, b.lens)] + [None] + [t.data_ptr() for t in (b.free_list, b.free_count)] + [None]
    state = pa._lib.Tables(*ints, R, W, b.free_list.shape[0], block)
    got = [torch.full_like(x, -9) for x in want[1:]]
    r, x = i32(rows), i32(new)
    st = lib.pa_extend_tables(state, r.data_ptr() if named else None, x.data_ptr(), n, None, 0, *[y.data_ptr() for y in got],
                              max_tokens, ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and error() == 0
    for u, v in zip(want[1:], got):
        assert torch.equal(u, v)
    for u, v in zip(a.args(), b.args()):
        assert torch.equal(u, v)
