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
