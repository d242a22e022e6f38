"""Block tables and slot maps on the GPU against a plain model of a stack of blocks; equal in every entry (needs a GB300)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


class Model:
    """Requests one after the other, blocks one after the other."""

    def __init__(self, n, width, block_size, num_blocks, rng):
        self.B, self.width = block_size, width
        self.table = np.full((n, width), -1, np.int32)
        self.lens, self.held = np.zeros(n, np.int32), np.zeros(n, np.int32)
        self.free = rng.permutation(num_blocks).astype(np.int32)
        self.top = num_blocks

    def extend(self, new, rows):
        slots, pos = np.full(rows, -1, np.int64), np.zeros(rows, np.int32)
        start = np.zeros(len(new) + 1, np.int32)
        need = [max(0, -(-(int(L) + int(a)) // self.B) - int(h)) for L, a, h in zip(self.lens, new, self.held)]
        bad = any(a < 0 or L + a > self.width * self.B for L, a in zip(self.lens, new)) or int(np.sum(new)) > rows
        if bad or sum(need) > self.top:
            return slots, pos, start
        r = 0
        for s, a in enumerate(new):
            for _ in range(need[s]):
                self.top -= 1
                self.table[s, self.held[s]] = self.free[self.top]
                self.held[s] += 1
            for i in range(self.lens[s], self.lens[s] + a):
                slots[r], pos[r] = int(self.table[s, i // self.B]) * self.B + i % self.B, i
                r += 1
            self.lens[s] += a
            start[s + 1] = r
        return slots, pos, start

    def trim(self, keep):
        if any(k < 0 or k > L for k, L in zip(keep, self.lens)):
            return
        gone = []
        for s, k in enumerate(keep):
            first = -(-int(k) // self.B)
            gone += list(self.table[s, first:self.held[s]])
            self.table[s, first:self.held[s]] = -1
            self.lens[s], self.held[s] = k, first
        for b in gone[::-1]:
            self.free[self.top] = b
            self.top += 1


class Device:
    def __init__(self, m, rows):
        import torch
        self.m = m
        t = lambda x: torch.from_numpy(np.array(x)).cuda()  # noqa: E731
        self.table, self.lens, self.held, self.free = t(m.table), t(m.lens), t(m.held), t(m.free)
        self.top = t(np.array([m.top], np.int32))
        self.slots = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
        self.pos = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
        self.start = torch.full((len(m.lens) + 1,), 77, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def extend(self, pa, new):
        import torch
        pa.pa_tables_extend(self.table, self.lens, self.held, self.free, self.top,
                            torch.from_numpy(np.asarray(new, np.int32)).cuda(), self.slots, self.pos, self.start, self.m.B,
                            err_flag=self.err)

    def trim(self, pa, keep):
        import torch
        pa.pa_tables_trim(self.table, self.lens, self.held, self.free, self.top,
                          torch.from_numpy(np.asarray(keep, np.int32)).cuda(), self.m.B, err_flag=self.err)

    def check(self, out=None):
        m = self.m
        for got, want in ((self.table, m.table), (self.lens, m.lens), (self.held, m.held), (self.free, m.free),
                          (self.top, [m.top])):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want))
        if out is not None:
            for got, want in zip((self.slots, self.pos, self.start), out):
                assert np.array_equal(got.cpu().numpy(), want)

    def error(self):
        e = int(self.err.item())
        self.err.zero_()
        return e


@pytest.mark.parametrize("n,block_size,rows,most", [(1, 16, 40, 40), (7, 24, 300, 60), (64, 16, 700, 12), (600, 8, 3000, 9),
                                                    (1025, 32, 40000, 70), (513, 16, 90000, 300)])
def test_random_steps(pa, n, block_size, rows, most):
    """Prompts, single tokens, rejected and finished requests, calls that ask for too much."""
    rng = np.random.default_rng(n)
    width = -(-3 * most // block_size) + 1
    m = Model(n, width, block_size, max(4, n * width // 3), rng)
    d = Device(m, rows)
    d.start[0] = 5
    refused = set()
    for step in range(12):
        kind = step % 4
        if kind == 0:
            new = rng.integers(0, most + 1, n)
        elif kind == 1:
            new = np.ones(n, np.int64)
        elif kind == 2:
            new = rng.integers(0, 6, n) * (rng.random(n) < 0.5)
        else:
            new = rng.integers(0, 2, n)
            new[rng.integers(n)] = rng.integers(0, rows // 2 + 1)
        before = (m.lens.copy(), m.top)
        out = m.extend(new, rows)
        changed = not (np.array_equal(before[0], m.lens) and before[1] == m.top) or not np.any(new)
        d.extend(pa, new)
        d.check(out)
        e = d.error()
        assert (e == 0) == changed and e in (0, 6, 7)
        refused.add(e)
        keep = np.maximum(0, m.lens - rng.integers(0, 5, n))
        keep[rng.random(n) < 0.2] = 0
        if step % 5 == 4:
            keep[rng.integers(n)] += most * 4  # more than there is
            m.trim(keep)
            d.trim(pa, keep)
            assert d.error() == 6
        else:
            m.trim(keep)
            d.trim(pa, keep)
            assert d.error() == 0
        d.check()


def test_all_blocks_and_one_more(pa):
    """The last free block is given, the one after it is not there; blocks held in advance are used first."""
    rng = np.random.default_rng(0)
    m = Model(3, 8, 16, 5, rng)
    d = Device(m, 64)
    for new, error in (([32, 0, 16], 0), ([0, 32, 0], 0), ([1, 0, 0], 7), ([0, 0, 0], 0), ([-1, 0, 0], 6), ([0, 0, 200], 6)):
        out = m.extend(new, 64)
        d.extend(pa, new)
        d.check(out)
        assert d.error() == error
    assert m.top == 0
    # blocks kept beyond the length (held_blocks says so) take the next tokens
    m.lens[0] = 3
    d.lens[0] = 3
    out = m.extend([20, 0, 0], 64)
    d.extend(pa, [20, 0, 0])
    d.check(out)
    assert d.error() == 0 and m.top == 0
    m.trim([0, 0, 0])
    d.trim(pa, [0, 0, 0])
    d.check()
    assert m.top == 5


def test_state_that_does_not_fit(pa):
    """Lengths past the blocks held, a stack larger than the pool: refused, nothing changed, only padding rows."""
    rng = np.random.default_rng(1)
    for spoil in ("lens", "held", "top", "negative"):
        m = Model(4, 6, 16, 20, rng)
        d = Device(m, 10)
        d.extend(pa, m.lens + 2)
        m.extend(m.lens + 2, 10)
        d.check()
        if spoil == "lens":
            d.lens[2] = 99
        elif spoil == "held":
            d.held[1] = 7
        elif spoil == "top":
            d.top[0] = 21
        else:
            d.lens[0] = -1
        before = [x.clone() for x in (d.table, d.lens, d.held, d.free, d.top)]
        for call in (lambda: d.extend(pa, [1, 0, 0, 0]), lambda: d.trim(pa, [0, 0, 0, 0])):
            call()
            assert d.error() == 6
            import torch
            assert all(torch.equal(a, b) for a, b in zip(before, (d.table, d.lens, d.held, d.free, d.top)))
        assert bool((d.slots == -1).all()) and bool((d.start == 0).all())


def test_block_outside_the_pool(pa):
    import torch
    m = Model(2, 4, 16, 8, np.random.default_rng(2))
    d = Device(m, 40)
    d.free[7] = 12345
    d.extend(pa, [3, 17])
    assert d.error() == 1
    assert d.slots[:3].tolist() == [-1] * 3 and bool((d.slots[3:20] >= 0).all())
    torch.cuda.synchronize()


def test_no_requests_no_rows_and_the_most(pa):
    import torch
    m = Model(16384, 2, 16, 40000, np.random.default_rng(3))
    d = Device(m, 16384 + 50)
    out = m.extend(np.ones(16384, np.int64), 16384 + 50)
    d.extend(pa, np.ones(16384))
    d.check(out)
    keep = np.arange(16384) % 2
    m.trim(keep)
    d.trim(pa, keep)
    d.check()
    with pytest.raises(pa.PaError):
        d = Device(Model(16385, 1, 16, 8, np.random.default_rng(0)), 1)
        d.extend(pa, np.zeros(16385))
    d = Device(Model(3, 4, 16, 8, np.random.default_rng(0)), 0)
    d.extend(pa, [0, 0, 0])
    assert d.error() == 0 and d.start.tolist() == [0, 0, 0, 0]
    d.extend(pa, [0, 1, 0])
    assert d.error() == 6
    d = Device(Model(0, 4, 16, 8, np.random.default_rng(0)), 5)
    d.extend(pa, [])
    assert d.slots.tolist() == [-1] * 5 and d.start.tolist() == [0]
    d.trim(pa, [])
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [200, 20000])
def test_captured(pa, rows):
    """Extend and trim in a graph, replayed: the state moves on as by calls."""
    import torch
    rng = np.random.default_rng(4)
    m = Model(40, 40, 16, 40 * 40, rng)
    d = Device(m, rows)
    new, keep = np.full(40, 5), np.zeros(40, np.int32)
    dn, dk = torch.from_numpy(new.astype(np.int32)).cuda(), torch.from_numpy(keep).cuda()
    d.extend(pa, new)
    m.extend(new, rows)
    d.check()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        torch.sub(d.lens, 2, out=dk)
        pa.pa_tables_trim(d.table, d.lens, d.held, d.free, d.top, dk, 16, err_flag=d.err)
        pa.pa_tables_extend(d.table, d.lens, d.held, d.free, d.top, dn, d.slots, d.pos, d.start, 16, err_flag=d.err)
    for _ in range(30):
        graph.replay()
        m.trim(m.lens - 2)
        out = m.extend(new, rows)
    torch.cuda.synchronize()
    d.check(out)
    assert d.error() == 0
