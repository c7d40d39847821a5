"""pa_build_step against the step's definition and the host block allocator.

Everything is whole numbers: outputs are equal, entry for entry, guards
around the buffers included.
"""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build

from step_reference import build_step, ceil_div

pytestmark = pytest.mark.gpu

GUARD = 64


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()
    assert binding.pa_get_device_error() == 0
    return torch.device("cuda:0")


class Guarded:
    """An int32 device buffer with a guard on both sides."""

    def __init__(self, dev, shape, values=None):
        import torch
        n = int(np.prod(shape))
        self.all = torch.full((n + 2 * GUARD,), -77, dtype=torch.int32, device=dev)
        self.t = self.all[GUARD:GUARD + n].view(shape)
        if values is not None:
            self.t.copy_(torch.from_numpy(np.ascontiguousarray(values, np.int32)))

    def get(self):
        a = self.all.cpu().numpy()
        assert (a[:GUARD] == -77).all() and (a[len(a) - GUARD:] == -77).all(), "written past the buffer"
        return self.t.cpu().numpy()


class StepCase:
    def __init__(self, dev, tables, lens, query, free_list, num_free, capacity, block_size, in_place=False, positions=True):
        g = lambda shape, v=None: Guarded(dev, shape, v)  # noqa: E731
        s = len(lens)
        self.args = (tables, np.asarray(lens), np.asarray(query), free_list, num_free, capacity, block_size)
        self.tables, self.lens, self.query = g(tables.shape, tables), g((s,), lens), g((s,), query)
        self.free, self.n = g(free_list.shape, free_list), g((1,), [num_free])
        self.lens_out = self.lens if in_place else g((s,))
        self.n_out = self.n if in_place else g((1,))
        self.cu, self.slots, self.admitted = g((s + 1,)), g((capacity,)), g((1,))
        self.positions = g((capacity,)) if positions else None

    def run(self, stream=None):
        binding.pa_build_step(self.tables.t, self.lens.t, self.query.t, self.free.t, self.n.t, self.lens_out.t, self.n_out.t,
                              self.cu.t, None if self.positions is None else self.positions.t, self.slots.t, self.admitted.t,
                              self.args[-1], stream)

    def check(self, want=None, error=0):
        import torch
        torch.cuda.synchronize()
        want = want or build_step(*self.args)
        assert binding.pa_get_device_error() == error
        assert self.admitted.get()[0] == want["admitted"]
        assert self.n_out.get()[0] == want["num_free"]
        for name, buf in (("cu", self.cu), ("lens", self.lens_out), ("tables", self.tables), ("free_list", self.free),
                          ("slots", self.slots)):
            assert np.array_equal(buf.get(), want[name]), name
        if self.positions is not None:
            assert np.array_equal(self.positions.get(), want["positions"])


def random_case(dev, seed, seqs, block, chunk, spare=1.0, capacity=None, retire=0.15, idle=0.2, longest=200, **kw):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, seqs)
    lens[rng.random(seqs) < 0.2] //= block
    lens = np.where(rng.random(seqs) < 0.2, lens // block * block, lens)  # full last blocks
    query = rng.integers(1, chunk + 1, seqs)
    query[rng.random(seqs) < idle] = 0
    query[rng.random(seqs) < retire] = -1 - rng.integers(0, 3)
    width = ceil_div(longest + chunk, block) + int(rng.integers(0, 3))
    held = -(-lens // block)
    need = int((-(-(lens + np.maximum(query, 0)) // block) - held).sum())
    num_free = int(spare * need)
    nb = int(held.sum()) + max(num_free, need) + 5
    perm = rng.permutation(nb)
    tables = np.full((seqs, width), -1, np.int32)
    at = 0
    for s in range(seqs):
        tables[s, :held[s]] = perm[at:at + held[s]]
        at += held[s]
    free_list = np.full(nb, -9, np.int32)
    free_list[:num_free] = perm[at:at + num_free]
    total = int(np.maximum(query, 0).sum())
    return StepCase(dev, tables, lens, query, free_list, num_free, total + 7 if capacity is None else capacity(total), block, **kw)


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("seqs,block,chunk", [(1, 16, 1), (1, 16, 700), (3, 32, 40), (31, 16, 1), (33, 48, 5), (256, 16, 1),
                                              (1023, 16, 9), (1025, 64, 33), (4096, 16, 20)])
def test_maps_equal_the_definition(dev, seqs, block, chunk, in_place):
    c = random_case(dev, 10 * seqs + block + chunk, seqs, block, chunk, in_place=in_place)
    c.run()
    c.check()


@pytest.mark.parametrize("seed", range(4))
def test_rows_are_served_in_order_until_blocks_run_out(dev, seed):
    c = random_case(dev, 50 + seed, 300, 16, 40, spare=0.3 + 0.2 * seed, retire=0.02)
    c.run()
    c.check()


@pytest.mark.parametrize("capacity", [lambda n: 0, lambda n: 1, lambda n: n // 2, lambda n: n - 1, lambda n: n, lambda n: n + 1000])
def test_rows_are_served_in_order_until_tokens_run_out(dev, capacity):
    c = random_case(dev, 77, 90, 32, 25, capacity=capacity)
    c.run()
    c.check()


def test_without_positions(dev):
    c = random_case(dev, 78, 40, 16, 25, positions=False)
    c.run()
    c.check()


def test_everything_idle_and_everything_finished(dev):
    for kw in (dict(idle=1.1, retire=0.0), dict(idle=0.0, retire=1.1), dict(idle=0.0, retire=0.0)):
        c = random_case(dev, 79, 130, 16, 12, **kw)
        c.run()
        c.check()


def test_an_empty_batch(dev):
    c = StepCase(dev, np.zeros((0, 4), np.int32), [], [], np.arange(8, dtype=np.int32), 5, 10, 16)
    c.run()
    c.check()


def test_no_free_blocks_at_all(dev):
    """Tokens that fit a row's last block need none; the first row that needs one stops the rest."""
    tables = np.array([[2, -1], [0, -1], [1, -1]], np.int32)
    c = StepCase(dev, tables, [10, 16, 3], [6, 1, 2], np.zeros(3, np.int32), 0, 16, 16)
    c.run()
    c.check()
    assert c.admitted.get()[0] == 1


def test_a_finished_rows_blocks_serve_the_same_step(dev):
    tables = np.array([[4, 2, 0, -1], [1, 3, -1, -1]], np.int32)
    c = StepCase(dev, tables, [33, 32], [-1, 17], np.zeros(5, np.int32), 0, 20, 16)
    c.run()
    c.check()  # pops 4 then 2: the finished row's first logical block was pushed last
    assert c.tables.get()[1].tolist() == [1, 3, 4, 2]


def test_inconsistent_rows_are_flagged_and_left(dev):
    """A negative length, a length past the table, and a row that would grow past it: no tokens, no blocks, length kept;
    the other rows are served."""
    rng = np.random.default_rng(3)
    tables = np.full((6, 4), -1, np.int32)
    tables[0, :2], tables[5, :1] = [7, 8], [9]
    lens = np.array([20, -3, 65, 60, 2000000000, 16])
    query = np.array([5, 4, 1, 5, -1, 3])
    free = np.full(16, -1, np.int32)
    free[:7] = rng.permutation(7)
    c = StepCase(dev, tables, lens, query, free, 7, 40, 16)
    c.run()
    quiet = np.where(np.arange(6) % 5 == 0, query, 0)
    want = build_step(tables, np.where(quiet, lens, 0), quiet, free, 7, 40, 16)
    want["lens"] = np.where(quiet, want["lens"], lens).astype(np.int32)
    c.check(want, error=binding.PA_DEVERR_SEQ_LEN)


def test_huge_requests_do_not_wrap(dev):
    """Counts that add up to 2^32 tokens (and to 2^28 blocks): the first huge row is refused, and so is all behind it."""
    import torch
    s, width, cap = 10, 1 << 25, 1500
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    tables = torch.full((s, width), -1, dtype=torch.int32, device=dev)
    free, out = torch.arange(100, dtype=torch.int32, device=dev), [i32([-7] * n) for n in (s, 1, s + 1, cap, 1)]
    lens_out, n_out, cu, slots, admitted = out
    binding.pa_build_step(tables, i32([0] * s), i32([5] + [1 << 29] * 8 + [1]), free, i32([100]), lens_out, n_out, cu, None,
                          slots, admitted, 16)
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    assert int(admitted) == 1 and int(n_out) == 99
    assert cu.tolist() == [0] + [5] * s and lens_out.tolist() == [5] + [0] * (s - 1)
    assert slots[:6].tolist() == [99 * 16 + i for i in range(5)] + [-1] and int(slots[5:].max()) == -1
    assert int(tables[0, 0]) == 99 and int((tables != -1).sum()) == 1


def test_bad_block_ids_never_become_slots(dev):
    """Ids outside the pool on the free list and in a table: flagged, stored as they are, slots -1."""
    tables = np.array([[99, -1, -1], [1, -1, -1]], np.int32)
    free = np.array([2, -5, 3, 0], np.int32)
    c = StepCase(dev, tables, [5, 16], [20, 17], free, 3, 40, 16)
    c.run()
    want = build_step(tables, [5, 16], np.array([20, 17]), free, 3, 40, 16)
    bad = (want["slots"] < 0) | (want["slots"] >= 4 * 16)
    want["slots"][bad] = -1
    c.check(want, error=binding.PA_DEVERR_BLOCK_ID)


@pytest.mark.parametrize("count", [-1, 5, 2000000000])
def test_a_free_count_outside_the_pool_is_held_to_it(dev, count):
    tables = np.full((2, 3), -1, np.int32)
    free = np.array([2, 1, 3, 0], np.int32)
    c = StepCase(dev, tables, [0, 0], [16, 16], free, count, 40, 16)
    c.run()
    c.check(build_step(tables, [0, 0], np.array([16, 16]), free, max(0, min(count, 4)), 40, 16),
            error=binding.PA_DEVERR_BLOCK_ID)


def test_more_blocks_returned_than_the_pool_has(dev):
    """Two finished rows that claim the same blocks: the count stays within the pool, nothing is written past the list."""
    import torch
    tables = np.array([[0, 1, 2], [0, 1, 2]], np.int32)
    c = StepCase(dev, tables, [48, 48], [-1, -1], np.array([3, -1, -1, -1], np.int32), 1, 4, 16)
    c.run()
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
    assert c.n_out.get()[0] == 4 and c.free.get().tolist() == [3, 2, 1, 0]


def test_many_steps_equal_the_host_allocator(dev):
    """120 steps of a serving loop, in place: rows come, grow by prompts and single tokens, finish. The host allocator
    does the same operations; tables, slots, lengths and free counts agree at every step."""
    import torch
    rng = np.random.default_rng(8)
    rows, nb, B, width, cap = 24, 160, 16, 24, 256
    order = rng.permutation(nb).astype(np.int32)
    alloc = binding.BlockAllocator(nb, B, order)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
    tables, lens, free, n = t(np.full((rows, width), -1)), t(np.zeros(rows)), t(order[::-1].copy()), t([nb])
    cu, pos, slots, adm = t(np.zeros(rows + 1)), t(np.zeros(cap)), t(np.zeros(cap)), t([0])
    seqs = [None] * rows
    stopped = 0
    for step in range(120):
        query = np.zeros(rows, np.int32)
        for r in range(rows):
            L = 0 if seqs[r] is None else alloc.seq_len(seqs[r])
            u = rng.random()
            if L and (u < 0.06 or L > width * B - 60):
                query[r] = -1
            elif L == 0:
                query[r] = int(rng.integers(1, 60)) if u < 0.4 else 0
            elif u > 0.15:
                query[r] = 1
        binding.pa_build_step(tables, lens, t(query), free, n, lens, n, cu, pos, slots, adm, B)
        for r in np.nonzero(query < 0)[0]:
            alloc.free_seq(seqs[r])
            seqs[r] = None
        want, cut = [], rows
        for r in range(rows):
            if query[r] <= 0 or cut < rows:
                continue
            L = 0 if seqs[r] is None else alloc.seq_len(seqs[r])
            need = ceil_div(L + int(query[r]), B) - ceil_div(L, B)
            if need > alloc.num_free() or len(want) + query[r] > cap:
                cut = r
                stopped += 1
                continue
            if seqs[r] is None:
                seqs[r] = alloc.add_seq(0)
            want += [alloc.append_token(seqs[r])[0] for _ in range(query[r])]
        assert int(adm[0]) == cut
        assert int(n[0]) == alloc.num_free()
        got = slots.cpu().numpy()
        assert got[:len(want)].tolist() == want and (got[len(want):] == -1).all()
        for r in range(rows):
            L = 0 if seqs[r] is None else alloc.seq_len(seqs[r])
            assert int(lens[r]) == L
            if L:
                assert tables[r, :ceil_div(L, B)].tolist() == alloc.table(seqs[r])
    assert stopped > 0  # the pool did run short
    assert binding.pa_get_device_error() == 0


def test_replayed_from_a_graph_and_on_another_stream(dev):
    """In place in a captured graph: each replay is the next step. The same on a side stream."""
    import torch
    c = random_case(dev, 90, 50, 16, 3, spare=40.0, in_place=True, retire=0.0, longest=20)
    tables = np.concatenate([c.args[0], np.full((50, 40), -1, np.int32)], 1)
    c = StepCase(dev, tables, *c.args[1:], in_place=True)
    c.run()
    c.check()
    state = build_step(*c.args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        c.run()
    side = torch.cuda.Stream()
    for k in range(8):
        if k % 2:
            side.wait_stream(torch.cuda.current_stream())
            c.run(side)
            torch.cuda.current_stream().wait_stream(side)
        else:
            g.replay()
        state = build_step(state["tables"], state["lens"], c.args[2], state["free_list"], state["num_free"], c.args[5], 16)
        c.check(state)
