"""Tables built on the GPU: against the host block manager, call by call, and the
calls that cannot be met."""
import numpy as np
import pytest
import torch

import paged_kv_cache_150_gb300 as pa

pytestmark = pytest.mark.gpu
BOUNDS, NO_BLOCKS = pa._lib.PA_ERR_DEVICE_BOUNDS, pa._lib.PA_ERR_NO_BLOCKS


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def error():
    return pa.pa_get_device_error(raise_on_error=False)


class State:
    """Device state of R rows of W blocks and the host manager that it is compared with."""

    def __init__(self, R, W, pool, block, seed):
        order = np.random.default_rng(seed).permutation(pool).astype(np.int32)
        self.R, self.W, self.block = R, W, block
        self.tables = torch.full((R, W), -7, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.free_list, self.free_count = i32(order), i32([pool])
        self.bm = pa.BlockManager(pool, block, order)
        self.seq = {}

    def args(self):
        return self.tables, self.lens, self.free_list, self.free_count

    def extend(self, rows, new, max_tokens, **kw):
        return pa.pa_extend_tables(*self.args(), i32(new), self.block, max_tokens, rows=None if rows is None else i32(rows), **kw)

    def step(self, rows, new, extra=0, **kw):
        """Both sides; asserts that they agree."""
        got = self.extend(rows, new, int(sum(new)) + extra, **kw)
        assert error() == 0
        names = range(len(new)) if rows is None else rows
        slots = []
        for r, n in zip(names, new):
            if r not in self.seq:
                self.seq[r] = self.bm.new_seq(0)
            slots.append(self.bm.append_tokens(self.seq[r], int(n))[0])
        want_t, want_l = self.bm.export([self.seq[r] for r in names], self.W) if len(new) else (np.zeros((0, self.W)), [])
        width = got[0].shape[1]
        assert (got[0].cpu().numpy() == want_t[:, :width]).all() and (want_t[:, width:] == -1).all()
        assert (got[1].cpu().numpy() == want_l).all()
        assert (got[2].cpu().numpy() == np.concatenate([[0], np.cumsum(new)])).all()
        want = np.concatenate(slots + [np.full(extra, -1)]) if len(new) else np.full(extra, -1)
        assert (got[3].cpu().numpy() == want).all()
        self.check()
        return got

    def release(self, rows, **kw):
        pa.pa_release_tables(*self.args(), i32(rows), self.block, **kw)
        assert error() == 0
        for r in rows:
            self.bm.free_seq(self.seq.pop(r))
        self.check()

    def check(self):
        assert int(self.free_count) == self.bm.stats()[0]
        lens = self.lens.cpu().numpy()
        tables = self.tables.cpu().numpy()
        for r in range(self.R):
            n = self.bm.seq_len(self.seq[r]) if r in self.seq else 0
            assert lens[r] == n
            if n:
                t = self.bm.block_table(self.seq[r])
                assert (tables[r, :len(t)] == t).all()

    def snapshot(self):
        return [x.clone() for x in self.args()]


@pytest.mark.parametrize("block", [1, 4, 16, 48])
def test_steps_of_a_serving_loop(block):
    rng = np.random.default_rng(block)
    s = State(12, 40, 12 * 40, block, seed=block)
    for step in range(25):
        rows = rng.permutation(12)[:rng.integers(0, 13)]
        room = [s.W * block - int(s.lens[r]) for r in rows]
        new = [int(min(rng.choice([0, 1, 1, 1, 7, 60]), x)) for x in room]
        s.step(list(rows), new, extra=int(rng.integers(0, 5)))
        live = list(s.seq)
        if step % 3 == 2 and live:
            s.release([int(r) for r in rng.permutation(live)[:rng.integers(1, len(live) + 1)]])


def test_rows_left_out_and_a_narrow_batch():
    s = State(5, 64, 300, 4, seed=1)
    s.step(None, [9, 0, 17, 4, 30], batch_width=9)
    s.step(None, [1, 1, 1])  # the first rows only
    s.step([4, 2], [3, 40])


def test_batches_of_more_than_one_block_of_threads():
    n = 2600
    s = State(n, 3, 2 * n, 16, seed=2)
    rng = np.random.default_rng(2)
    rows = [int(r) for r in rng.permutation(n)]
    s.step(rows, [int(x) for x in rng.integers(0, 17, n)], extra=100)
    s.step(rows[:1500], [int(x) for x in rng.integers(0, 10, 1500)])
    s.release(rows[100:2300])


def test_long_prompts_and_wide_tables():
    s = State(4, 5000, 12000, 16, seed=3)
    s.step([2, 0], [70001, 33], extra=17)
    s.step([1, 2, 0], [50000, 1, 15])
    s.release([2, 1])
    s.step([3], [79999])


def test_the_state_before_a_step_stays_where_buffers_of_its_own_are_given():
    s = State(6, 20, 60, 4, seed=4)
    s.step(None, [9, 2, 30, 4, 0, 7])
    before = s.snapshot()
    lens2, count2 = torch.full_like(s.lens, -5), torch.full_like(s.free_count, -5)
    outs = [s.extend([3, 1], [5, 6], 16, lens_out=lens2, free_count_out=count2) for _ in range(2)]  # made twice
    assert error() == 0
    assert torch.equal(s.lens, before[1]) and torch.equal(s.free_list, before[2]) and torch.equal(s.free_count, before[3])
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    assert lens2.tolist() == [9, 8, 30, 9, 0, 7]
    got = s.step([3, 1], [5, 6], extra=5)  # the step itself, in place
    for x, y in zip(got, outs[0]):
        assert torch.equal(x, y)
    assert torch.equal(lens2, s.lens) and torch.equal(count2, s.free_count)
    before = s.snapshot()
    pa.pa_release_tables(*s.args(), i32([2, 0]), 4, lens_out=lens2, free_count_out=count2)
    assert torch.equal(s.lens, before[1]) and torch.equal(s.free_count, before[3])
    s.release([2, 0])
    assert torch.equal(lens2, s.lens) and torch.equal(count2, s.free_count)


@pytest.mark.parametrize("rows,new,extra,status,kw", [
    ([0, 1], [200, 9], 0, NO_BLOCKS, {}),                    # more blocks than are free
    ([0, 0], [1, 1], 0, BOUNDS, {}),                         # a row twice
    ([0, 6], [1, 1], 0, BOUNDS, {}), ([-1, 2], [1, 1], 0, BOUNDS, {}), ([0, 2 ** 31 - 1], [1, 1], 0, BOUNDS, {}),
    ([0, 1], [-1, 4], 0, BOUNDS, {}),                        # a negative number of tokens
    ([0, 1], [4, 2 ** 31 - 1], 10, BOUNDS, {}),              # past the row, and past 32 bits
    ([2, 1], [4 * 60 - 30 + 1, 0], 0, BOUNDS, {}),           # one past the row
    ([0, 1], [5, 6], -1, BOUNDS, {}),                        # one more token than the slot map holds
    ([2, 1], [0, 1], 0, BOUNDS, dict(batch_width=7)),        # a table wider than the batch's
])
def test_a_call_that_cannot_be_met_changes_nothing(rows, new, extra, status, kw):
    s = State(6, 60, 60, 4, seed=5)
    s.step(None, [9, 2, 30, 4, 0, 7])
    before, lens = s.snapshot(), s.lens.tolist()
    size = int(min(max(sum(new), 1), 400)) + extra
    out = s.extend(rows, new, size, **kw)
    assert error() == status
    for x, y in zip(before, s.args()):
        assert torch.equal(x, y)
    seen = [lens[r] if 0 <= r < 6 else 0 for r in rows]
    if rows == [0, 0]:  # one of the two is the row's
        assert sorted(out[1].tolist()) == [0, lens[0]]
    else:
        assert out[1].tolist() == seen
    assert out[2].tolist() == [0, 0, 0] and bool((out[3] == -1).all())
    table = out[0].cpu()
    for i, r in enumerate(rows):
        n = -(-out[1].tolist()[i] // 4)
        keep = min(n, table.shape[1])
        assert torch.equal(table[i, :keep], before[0][max(min(r, 5), 0)].cpu()[:keep]) and bool((table[i, keep:] == -1).all())
    s.step([0, 1], [3, 3])  # and the next call works


def test_bad_state():
    s = State(4, 10, 30, 4, seed=6)
    s.step(None, [9, 2, 13, 4])
    for lens in ([-1, 2, 13, 4], [9, 41, 13, 4]):
        out = pa.pa_extend_tables(s.tables, i32(lens), s.free_list, s.free_count, i32([1, 1]), 4, 2)
        assert error() == BOUNDS and out[2].tolist() == [0, 0, 0]
    for count in (-1, 31, 2 ** 31 - 1):
        c = i32([count])
        pa.pa_extend_tables(s.tables, s.lens, s.free_list, c, i32([1, 1]), 4, 2)
        assert error() == BOUNDS and int(c) == count
        pa.pa_release_tables(s.tables, s.lens, s.free_list, c, i32([1]), 4)
        assert error() == BOUNDS and int(c) == count
    s.check()
    # an id outside the pool in a table, or on the stack: no slot
    bad = s.tables.clone()
    bad[1, 0] = 30
    out = pa.pa_extend_tables(bad, s.lens.clone(), s.free_list, s.free_count.clone(), i32([1]), 4, 1, rows=i32([1]))
    assert error() == BOUNDS and out[3].tolist() == [-1]
    stack = s.free_list.clone()
    stack[int(s.free_count) - 1] = -3
    out = pa.pa_extend_tables(bad, s.lens.clone(), stack, s.free_count.clone(), i32([4]), 4, 4, rows=i32([3]))
    assert error() == BOUNDS and out[3].tolist() == [-1] * 4


@pytest.mark.parametrize("rows", [[0, 0], [1, 4], [-2, 1]])
def test_a_release_that_cannot_be_met_changes_nothing(rows):
    s = State(4, 10, 30, 4, seed=7)
    s.step(None, [9, 2, 13, 4])
    before = s.snapshot()
    pa.pa_release_tables(*s.args(), i32(rows), 4)
    assert error() == BOUNDS
    for x, y in zip(before, s.args()):
        assert torch.equal(x, y)
    s.release([0, 1, 2, 3])
    over = i32([28])  # more blocks than the pool has
    s.step(None, [9, 2, 13, 4])
    pa.pa_release_tables(s.tables, s.lens, s.free_list, over, i32([0]), 4)
    assert error() == BOUNDS and int(over) == 28


def test_empty_calls():
    s = State(3, 8, 20, 4, seed=8)
    s.step([], [], extra=5)
    s.step(None, [3, 0, 9])
    lens2, count2 = torch.zeros_like(s.lens), torch.zeros_like(s.free_count)
    pa.pa_release_tables(*s.args(), i32([]), 4, lens_out=lens2, free_count_out=count2)
    assert torch.equal(lens2, s.lens) and torch.equal(count2, s.free_count)
    s.step([1], [0])
    s.release([1])  # a row without blocks


def test_captured_steps_that_share_a_workspace():
    """A graph of one decode step, replayed: every replay is a further step; with a
    release in another graph in between."""
    s = State(5, 30, 100, 4, seed=9)
    s.step(None, [9, 2, 30, 4, 1])
    ws = torch.empty(pa.pa_tables_workspace_bytes(5, 5), dtype=torch.uint8, device="cuda")
    rows, new, gone = i32([4, 0, 2]), i32([1, 1, 1]), i32([3])
    out = tuple(torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((3, 30), 3, 4, 8))
    steps, drop = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(steps):
        pa.pa_extend_tables(*s.args(), new, 4, 8, rows=rows, out=out, workspace=ws)
    with torch.cuda.graph(drop):
        pa.pa_release_tables(*s.args(), gone, 4, workspace=ws)
    for i in range(7):
        steps.replay()
        if i == 3:
            drop.replay()
        torch.cuda.synchronize()
        slots = [int(s.bm.append_tokens(s.seq[r], 1)[0][0]) for r in (4, 0, 2)]
        if i == 3:
            s.bm.free_seq(s.seq.pop(3))
        assert out[3].tolist() == slots + [-1] * 5 and out[2].tolist() == [0, 1, 2, 3]
        s.check()
    assert error() == 0


def test_python_refusals():
    s = State(4, 10, 30, 4, seed=10)
    t, l, f, c = s.args()
    one = i32([1])
    for bad in (lambda: pa.pa_extend_tables(t[0], l, f, c, one, 4, 1), lambda: pa.pa_extend_tables(t, l[:2], f, c, one, 4, 1),
                lambda: pa.pa_extend_tables(t, l, f, c, i32([1] * 5), 4, 5), lambda: pa.pa_extend_tables(t, l, f, i32([1, 2]), one, 4, 1),
                lambda: pa.pa_extend_tables(t, l, f, c, one, 4, 1, rows=i32([0, 1])),
                lambda: pa.pa_extend_tables(t, l, f, c, one, 4, 1, out=(one, one, one, one)),
                lambda: pa.pa_extend_tables(t.long(), l, f, c, one, 4, 1), lambda: pa.pa_extend_tables(t, l, f, c, one.cpu(), 4, 1),
                lambda: pa.pa_extend_tables(t.t(), l, f, c, one, 4, 1), lambda: pa.pa_release_tables(t, l, f, c, i32([[0]]), 4),
                lambda: pa.pa_release_tables(t, l, f, c, i32([0] * 5), 4)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for bad in (lambda: pa.pa_extend_tables(t, l, f, c, one, 4, 1, workspace=small), lambda: pa.pa_extend_tables(t, l, f, c, one, 0, 1),
                lambda: pa.pa_extend_tables(t, l, f, c, one, 4, 1, batch_width=0), lambda: pa.pa_release_tables(t, l, f, c, one, -1)):
        with pytest.raises((pa.PagedAttentionError, ValueError)):
            bad()
