"""paged_kv_fork and paged_kv_release against a row-by-row walk on the host."""
import numpy as np
import pytest
import torch

import paged_kv_cache_233_gb300 as pk

pytestmark = pytest.mark.gpu
SEQ_INDEX, CONTEXT_LEN, BLOCK_ID, POSITION = 16, 4, 2, 8
ALL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


class Cache:
    """Rows, holders and the stack on the host, and what the calls mean."""

    def __init__(self, lens, block, width, spare, seed=0):
        rng = np.random.default_rng(seed)
        self.block, self.lens = block, [int(n) for n in lens]
        need = [-(-n // block) for n in self.lens]
        ids = rng.permutation(sum(need) + spare)
        self.tables = np.full((len(lens), width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.blocks = len(ids)
        self.shared = np.zeros(len(ids), np.int32)
        self.stack = list(ids[at:])
        self.room = len(ids)

    def device(self):
        t = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
        free = np.full(self.room, -5, np.int32)
        free[:len(self.stack)] = self.stack
        return dict(lens=t(self.lens), tables=t(self.tables), shared=t(self.shared), free=t(free), count=t([len(self.stack)]))

    def fork(self, parents):
        before, pairs, asked, room = list(self.lens), [[0, 0] for _ in parents], 0, len(self.stack)
        for s, p in enumerate(parents):
            if p < 0 or p >= len(parents) or parents[p] != -1 or not 0 <= before[p] <= self.tables.shape[1] * self.block:
                continue
            whole, rest = divmod(before[p], self.block)
            if rest:
                asked += 1
                if asked > room:
                    continue
            for j in range(whole):
                self.tables[s, j] = self.tables[p, j]
                self.shared[self.tables[p, j]] += 1
            if rest:
                self.tables[s, whole] = self.stack.pop()
                pairs[s] = [int(self.tables[p, whole]), int(self.tables[s, whole])]
            self.lens[s] = before[p]
        return pairs

    def release(self, keep):
        freed = set()
        for s, k in enumerate(keep):
            n = min(k, self.lens[s])
            if k < 0 or not 0 <= self.lens[s] <= self.tables.shape[1] * self.block:
                continue
            for j in range(-(-n // self.block), -(-self.lens[s] // self.block)):
                b = int(self.tables[s, j])
                if self.shared[b] == 0:
                    freed.add(b)
                else:
                    self.shared[b] -= 1
            self.lens[s] = n
        self.stack += sorted(freed)
        self.stack = self.stack[:self.room]

    def check(self, d, lens, count, pairs=None, want_pairs=None):
        assert np.array_equal(d["tables"].cpu().numpy(), self.tables)
        assert np.array_equal(d["shared"].cpu().numpy(), self.shared)
        assert lens.tolist() == self.lens and int(count) == len(self.stack)
        assert d["free"].cpu().tolist()[:len(self.stack)] == [int(b) for b in self.stack]
        assert pairs is None or pairs.tolist() == want_pairs


def fork(c, parents, in_place=False):
    d = c.device()
    pairs = torch.full((len(parents), 2), -9, dtype=torch.int32).cuda()
    lens, count = (d["lens"], d["count"]) if in_place else (torch.full_like(d["lens"], -9), torch.full_like(d["count"], -9))
    pk.paged_kv_fork(torch.tensor(parents, dtype=torch.int32).cuda(), d["lens"], d["tables"], d["shared"], d["free"], d["count"],
                     pairs, c.block, lens, count)
    return d, lens, count, pairs


def release(c, keep, in_place=False):
    d = c.device()
    lens, count = (d["lens"], d["count"]) if in_place else (torch.full_like(d["lens"], -9), torch.full_like(d["count"], -9))
    pk.paged_kv_release(torch.tensor(keep, dtype=torch.int32).cuda(), d["lens"], d["tables"], d["shared"], d["free"], d["count"],
                        c.block, lens, count)
    return d, lens, count


def random_case(S, block, longest, seed, spare=1.0):
    """Rows at random places: half of them parents, some of the others children."""
    rng = np.random.default_rng(seed)
    held = rng.random(S) < 0.5
    held[0] = True
    lens = np.where(held, rng.integers(0, longest + 1, S), 0)
    children = np.where(~held & (rng.random(S) < 0.8), rng.choice(np.flatnonzero(held), S), -1)
    need = int(((lens[children.clip(0)] % block > 0) & (children >= 0)).sum())
    return Cache(lens, block, longest // block + 2, int(spare * need) + 1, seed), [int(x) for x in children], rng


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,block,longest,spare", [
    (1, 16, 40, 1), (2, 8, 0, 1), (7, 16, 100, 1), (33, 8, 500, 0.4), (300, 32, 900, 1), (300, 16, 40, 0.0), (1025, 16, 700, 0.6),
    (4096, 8, 60, 0.7), (50, 12, 700, 1), (3, 1, 300, 1)])
def test_fork_then_release(S, block, longest, spare, in_place):
    c, parents, rng = random_case(S, block, longest, S + block, spare)
    d, lens, count, pairs = fork(c, parents, in_place)
    want = c.fork(parents)
    c.check(d, lens, count, pairs, want)
    fate = rng.integers(0, 4, S)
    keep = [0 if f == 0 else max(0, n - int(rng.integers(0, 2 * block))) if f == 1 else n if f == 2 else ALL
            for f, n in zip(fate, c.lens)]
    d, lens, count = release(c, keep, in_place)
    c.release(keep)
    c.check(d, lens, count)
    # everything: each block is on the stack once
    d, lens, count = release(c, [0] * S, in_place)
    c.release([0] * S)
    c.check(d, lens, count)
    assert sorted(c.stack) == list(range(c.blocks)) and not c.shared.any()
    assert pk.device_errors() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,length", [(3, 100000), (40, 20000)])
def test_release_of_many_blocks(rows, length, in_place):
    """Enough blocks that several blocks of threads push them; some held twice, some not given back."""
    c = Cache([length + 7 * s for s in range(rows)] + [0] * rows, 8, (length + 7 * rows) // 8 + 1, 3 * rows + 5, rows)
    parents = [-1] * rows + [s if s % 2 else -1 for s in range(rows)]
    c.fork(parents)
    keep = [0 if s % 3 else length // 2 for s in range(rows)] + [0 if s % 4 == 1 else ALL for s in range(rows)]
    d, lens, count = release(c, keep, in_place)
    c.release(keep)
    c.check(d, lens, count)
    assert pk.device_errors() == 0


def test_many_children_of_one_parent():
    c = Cache([1000] + [0] * 700, 16, 70, 800, 3)
    parents = [-1] + [0] * 700
    d, lens, count, pairs = fork(c, parents)
    want = c.fork(parents)
    c.check(d, lens, count, pairs, want)
    assert int(c.shared.max()) == 700
    d, lens, count = release(c, [0] * 701)
    c.release([0] * 701)
    c.check(d, lens, count)
    assert not c.shared.any() and pk.device_errors() == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_reports_bad_parents(in_place):
    c = Cache([40, 17, 0, 0, 0, 0, 0, 5], 8, 6, 20, 1)
    parents = [-1, -1, 0, 2, 8, -2, 1, 7]        # a child of a child, past the rows, a bad mark, itself
    d, lens, count, pairs = fork(c, parents, in_place)
    want = c.fork(parents)
    c.check(d, lens, count, pairs, want)
    assert pk.device_errors() == SEQ_INDEX
    c = Cache([40, 0, 0], 8, 6, 20, 1)
    c.lens[0] = 49
    d, lens, count, pairs = fork(c, [-1, 0, 0], in_place)
    want = c.fork([-1, 0, 0])
    c.check(d, lens, count, pairs, want)
    assert pk.device_errors() == CONTEXT_LEN


def test_fork_with_bad_blocks():
    c = Cache([20, 0], 8, 6, 3, 1)
    c.tables[0, 1] = 1 << 20
    d, lens, count, pairs = fork(c, [-1, 0])
    assert pk.device_errors() == BLOCK_ID
    assert d["tables"][1, :2].tolist() == c.tables[0, :2].tolist() and int(d["shared"].sum()) == 1
    c = Cache([20, 0], 8, 6, 3, 1)
    c.stack[-1] = -4
    d, lens, count, pairs = fork(c, [-1, 0])
    assert pk.device_errors() == BLOCK_ID
    assert pairs.tolist() == [[0, 0], [0, 0]] and int(d["tables"][1, 2]) == -4


@pytest.mark.parametrize("in_place", [False, True])
def test_release_reports_bad_rows_and_blocks(in_place):
    c = Cache([40, 17, 9, 30], 8, 6, 5, 2)
    c.lens[1] = -3
    keep = [8, 0, -1, 3]
    d, lens, count = release(c, keep, in_place)
    c.release(keep)
    c.check(d, lens, count)
    assert pk.device_errors() == CONTEXT_LEN
    # a block out of range, and one that two rows hold without a count: once on the stack
    c = Cache([40, 40], 8, 6, 5, 2)
    c.tables[0, 1], c.tables[1, 0] = 99, c.tables[0, 0]
    d, lens, count = release(c, [0, 0], in_place)
    assert pk.device_errors() == BLOCK_ID
    got = d["free"].cpu().tolist()[5:int(count)]
    assert got == sorted({int(x) for x in c.tables[:, :5].flatten() if x < c.blocks})
    assert not bool(d["shared"].any())


@pytest.mark.parametrize("in_place", [False, True])
def test_stack_bounds(in_place):
    """A stack that is too small loses blocks; a bad count is clamped."""
    c = Cache([64, 64], 8, 8, 2, 4)
    c.room = 7
    d, lens, count = release(c, [0, 0], in_place)
    c.release([0, 0])
    c.check(d, lens, count)
    assert pk.device_errors() == POSITION
    c = Cache([64, 5, 0], 8, 8, 4, 4)
    for n, clamped in ((-3, 0), (1000, c.room)):
        d = c.device()
        d["count"].fill_(n)
        lens, out = (d["lens"], d["count"]) if in_place else (torch.zeros_like(d["lens"]), torch.zeros_like(d["count"]))
        pk.paged_kv_release(torch.tensor([ALL, ALL, ALL], dtype=torch.int32).cuda(), d["lens"], d["tables"], d["shared"], d["free"],
                            d["count"], 8, lens, out)
        assert int(out) == clamped and pk.device_errors() == POSITION


def test_no_sequences():
    c = Cache([], 8, 4, 3)
    d, lens, count, pairs = fork(c, [])
    assert int(count) == 3
    d, lens, count = release(c, [])
    assert int(count) == 3
    release(c, [], in_place=True)
    assert pk.device_errors() == 0
