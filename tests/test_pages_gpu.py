"""gdn_pages_* against a pool in plain Python: every integer and every byte equal."""
import random

import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, I32 = "cuda", torch.int32
BOUNDS = gdn.GDN_ERR_DEVICE_BOUNDS


class Model:
    """The pool by the documentation; `caches` are lists of pages."""

    def __init__(self, n_pages, page, n_seqs, width, caches=()):
        self.page, self.width = page, width
        self.refs, self.len = [0] * n_pages, [0] * n_seqs
        self.table = [[-1] * width for _ in range(n_seqs)]
        self.caches = [c.clone() for c in caches]

    def free_pages(self, need):
        got = [p for p, r in enumerate(self.refs) if r <= 0][:need]
        return got if len(got) == need else None

    def up(self, n):
        return -(-n // self.page)

    def sound(self, seqs):
        return len(set(seqs)) == len(seqs) and all(0 <= s < len(self.len) for s in seqs)

    def extend(self, seqs, count, steps):
        """The slots, or None where nothing is done."""
        if not self.sound(seqs) or any(not 0 <= c <= steps or self.len[s] + c > self.width * self.page
                                       for s, c in zip(seqs, count)):
            return None
        fresh = self.free_pages(sum(self.up(self.len[s] + c) - self.up(self.len[s]) for s, c in zip(seqs, count)))
        if fresh is None:
            return None
        slots = []
        for s, c in zip(seqs, count):
            slots.append([-1] * steps)
            for j in range(c):
                col, at = divmod(self.len[s], self.page)
                if at == 0:
                    self.table[s][col] = fresh.pop(0)
                    self.refs[self.table[s][col]] = 1
                slots[-1][j] = self.table[s][col] * self.page + at
                self.len[s] += 1
        return slots

    def copy(self, a, b):
        for c in self.caches:
            c[b] = c[a]

    def trim(self, seqs, to):
        if not self.sound(seqs) or any(not 0 <= n <= self.len[s] for s, n in zip(seqs, to)):
            return False
        own = [n < self.len[s] and n % self.page and self.refs[self.table[s][n // self.page]] > 1
               for s, n in zip(seqs, to)]
        fresh = self.free_pages(sum(map(bool, own)))
        if fresh is None:
            return False
        for s, n, cut in zip(seqs, to, own):
            for col in range(self.up(n), self.up(self.len[s])):
                self.refs[self.table[s][col]] -= 1
                self.table[s][col] = -1
            if cut:
                old, new = self.table[s][n // self.page], fresh.pop(0)
                self.copy(old, new)
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s][n // self.page] = new
            self.len[s] = n
        return True

    def fork(self, src, dst):
        if not self.sound(dst) or any(not 0 <= s < len(self.len) for s in src) or any(self.len[d] for d in dst):
            return False
        fresh = self.free_pages(sum(self.len[s] % self.page > 0 for s in src))
        if fresh is None:
            return False
        for n, s, d in [(self.len[s], s, d) for s, d in zip(src, dst)]:
            for col in range(n // self.page):
                self.table[d][col] = self.table[s][col]
                self.refs[self.table[s][col]] += 1
            if n % self.page:
                col, new = n // self.page, fresh.pop(0)
                self.copy(self.table[s][col], new)
                self.table[d][col] = new
                self.refs[new] = 1
            self.len[d] = n
        return True

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        holes = [p for p in range(len(live)) if self.refs[p] <= 0]
        move = dict(zip([p for p in live if p >= len(live)], holes))
        for a, b in move.items():
            self.copy(a, b)
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, row in enumerate(self.table):
            for col in range(self.up(self.len[s])):
                row[col] = move.get(row[col], row[col])
        return len(live)


class Both:
    """A pool on the GPU and the model beside it."""

    def __init__(self, n_pages, page, n_seqs, width, sizes=(64, 4096 + 32, 16), seed=0):
        g = torch.Generator().manual_seed(seed)
        host = [torch.randint(0, 256, (n_pages, b), generator=g, dtype=torch.uint8) for b in sizes]
        self.m = Model(n_pages, page, n_seqs, width, host)
        self.refs = torch.zeros(n_pages, dtype=I32, device=DEV)
        self.table = torch.full((n_seqs, width), -1, dtype=I32, device=DEV)
        self.len = torch.zeros(n_seqs, dtype=I32, device=DEV)
        self.dev = [h.to(DEV) for h in host]
        self.pool = gdn.make_page_pool(self.refs, self.table, self.len, page)
        self.caches = gdn.make_page_caches(self.dev)
        self.ws = torch.full((gdn.gdn_pages_workspace_bytes(self.pool),), 255, dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(1, dtype=I32, device=DEV)

    def i32(self, x):
        return torch.tensor(x, dtype=I32, device=DEV)

    def same(self, done=True):
        assert gdn.gdn_read_device_status(self.status) == (0 if done else BOUNDS)
        self.status.zero_()
        assert self.refs.tolist() == self.m.refs
        assert self.len.tolist() == self.m.len
        for s, row in enumerate(self.table.tolist()):
            n = self.m.up(self.m.len[s])
            assert row[:n] == self.m.table[s][:n], s
        for c, d in zip(self.m.caches, self.dev):
            assert torch.equal(c, d.cpu())

    def extend(self, seqs, count, steps=None):
        steps = steps or max(count + [1])
        slot = torch.full((len(seqs), steps), 77, dtype=I32, device=DEV)
        gdn.gdn_pages_extend(self.pool, slot, self.ws, seq=self.i32(seqs), count=self.i32(count),
                             device_status=self.status)
        want = self.m.extend(seqs, count, steps)
        self.same(want is not None)
        assert slot.tolist() == (want or [[-1] * steps] * len(seqs))
        return want

    def trim(self, seqs, to):
        gdn.gdn_pages_trim(self.pool, self.caches, self.i32(to), self.ws, seq=self.i32(seqs), device_status=self.status)
        done = self.m.trim(seqs, to)
        self.same(done)
        return done

    def fork(self, src, dst):
        gdn.gdn_pages_fork(self.pool, self.caches, self.i32(src), self.i32(dst), self.ws, device_status=self.status)
        done = self.m.fork(src, dst)
        self.same(done)
        return done

    def free(self, seqs):
        gdn.gdn_pages_free(self.pool, self.i32(seqs), self.ws, device_status=self.status)
        done = self.m.trim(seqs, [0] * len(seqs)) if self.m.sound(seqs) else False
        self.same(done)

    def compact(self):
        live = torch.zeros(1, dtype=I32, device=DEV)
        gdn.gdn_pages_compact(self.pool, self.caches, self.ws, n_live=live, device_status=self.status)
        assert live.item() == self.m.compact()
        self.same()


@pytest.mark.parametrize("n_pages,page,n_seqs,width", [(37, 16, 9, 6), (400, 1, 20, 40), (130, 64, 33, 5), (5, 256, 3, 4)])
@pytest.mark.parametrize("seed", range(3))
def test_a_long_run_of_everything(n_pages, page, n_seqs, width, seed):
    rng = random.Random(seed)
    b = Both(n_pages, page, n_seqs, width, seed=seed)
    for _ in range(60):
        some = rng.sample(range(n_seqs), rng.randint(1, n_seqs))
        kind = rng.choice(["extend", "extend", "extend", "trim", "fork", "free", "compact"])
        if kind == "extend":
            b.extend(some, [rng.randint(0, min(3 * page, max(0, width * page - b.m.len[s]))) for s in some])
        elif kind == "trim":
            b.trim(some, [rng.randint(0, b.m.len[s]) for s in some])
        elif kind == "fork":
            empty = [s for s in range(n_seqs) if b.m.len[s] == 0][:4]
            if empty:
                b.fork([rng.randrange(n_seqs) for _ in empty], empty)
        elif kind == "free":
            b.free(some[:3])
        else:
            b.compact()


def test_all_sequences_by_steps_without_lists():
    b = Both(50, 16, 7, 8)
    for steps in (1, 5, 40):
        slot = torch.zeros(7, steps, dtype=I32, device=DEV)
        gdn.gdn_pages_extend(b.pool, slot, b.ws, device_status=b.status)
        assert slot.tolist() == b.m.extend(list(range(7)), [steps] * 7, steps)
        b.same()
    keep = [46, 0, 1, 16, 17, 32, 33]
    gdn.gdn_pages_trim(b.pool, None, b.i32(keep), b.ws, device_status=b.status)
    b.m.trim(list(range(7)), keep)
    b.same()


def test_refused_calls_change_nothing():
    b = Both(12, 16, 6, 4)
    b.extend([0, 1, 2], [20, 64, 5])
    b.fork([0], [3])
    b.extend([0, 0], [1, 1])                   # named twice
    b.extend([0, 6], [1, 1])                   # no such sequence
    b.extend([0, -1], [1, 1])
    b.extend([0, 4], [1, -1], steps=2)         # counts that may not be
    b.extend([0, 4], [3, 1], steps=2)
    b.extend([0, 1], [1, 1])                   # past the table's width
    b.extend([4, 5], [64, 17])                 # more pages than are free
    assert not b.trim([0, 2], [21, 0]) and not b.trim([0, 2], [-1, 0]) and not b.trim([2, 2], [1, 1])
    assert not b.fork([0], [1])                # not empty
    assert not b.fork([0, 0], [4, 4]) and not b.fork([9], [4]) and not b.fork([0], [17])
    b.free([0, 0])
    b.free([11])
    assert b.extend([4], [48]) and not b.fork([0, 0], [5, 5])
    b.extend([5], [16])                        # the last free page
    assert not b.trim([0], [3]) or b.m.refs    # (shared page: a copy would need a free one)


def test_trimming_into_a_shared_page_makes_a_copy():
    b = Both(20, 16, 6, 4)
    b.extend([0], [50])
    b.fork([0, 0, 0], [1, 2, 3])
    b.trim([1, 2], [20, 16])                   # inside the second page, and at its start
    b.trim([0, 3], [30, 30])                   # the last two holders at once
    b.extend([0, 1, 2, 3], [7, 7, 7, 7])
    assert not b.m.refs[b.m.table[1][1]] > 1


def test_chains_of_forks_in_one_call_go_by_the_start():
    b = Both(20, 16, 6, 4)
    b.extend([0], [37])
    assert b.fork([0, 1, 4], [1, 2, 4])        # 1 holds nothing yet: 2 stays empty; 4 onto itself
    assert b.m.len[2] == 0 and b.m.len[4] == 0 and b.m.len[1] == 37


@pytest.mark.parametrize("n_pages", [1, 2, 3, 31, 4097, 65536, 70001, 300000])
def test_pools_of_all_sizes(n_pages):
    g = torch.Generator().manual_seed(n_pages)
    b = Both(n_pages, 16, 40, 3000, sizes=(16,))
    used = torch.rand(n_pages, generator=g) < (0.5 if n_pages < 60000 else 0.99)
    taken = used.nonzero()[:, 0]
    taken = taken[torch.randperm(len(taken), generator=g)][:40 * 2000].tolist()
    for s in range(40):
        mine = taken[s::40]
        for col, p in enumerate(mine):
            b.m.table[s][col], b.m.refs[p] = p, 1
        b.m.len[s] = 16 * len(mine)
    for p in used.nonzero()[:, 0].tolist():    # pages that tables outside this pool hold
        b.m.refs[p] = max(1, b.m.refs[p])
    b.refs.copy_(torch.tensor(b.m.refs, dtype=I32))
    b.len.copy_(torch.tensor(b.m.len, dtype=I32))
    b.table.copy_(torch.tensor(b.m.table, dtype=I32))
    b.extend(list(range(0, 40, 3)), [16 * (1 + s) for s in range(0, 40, 3)])
    b.extend(list(range(40)), [1] * 40)
    b.compact()
    b.compact()
    b.free(list(range(0, 40, 2)))
    b.compact()


def test_long_lists():
    n = 8192
    b = Both(20000, 16, n, 2, sizes=(16,))
    rng = random.Random(1)
    b.extend(rng.sample(range(n), n), [rng.randint(0, 20) for _ in range(n)])
    b.trim(rng.sample(range(n), n), [0] * n)
    b.extend(rng.sample(range(n), 5000), [rng.randint(0, 30) for _ in range(5000)])
    b.compact()


def test_a_prompt_in_one_call():
    b = Both(700, 64, 2, 600, sizes=(16,))
    b.extend([1], [33333])
    b.extend([0], [70])


def test_copies_between_sets_and_bad_indices():
    g = torch.Generator().manual_seed(0)
    sizes = [(16,), (3, 20, 18 * 64), (8192 + 48,)]
    make = lambda n: [torch.randint(0, 256, (n, *s), generator=g, dtype=torch.uint8, device="cpu") for s in sizes]   # noqa: E731
    src, dst = make(9), make(5)
    ds, dd = [x.to(DEV) for x in src], [x.to(DEV) for x in dst]
    i32 = lambda x: torch.tensor(x, dtype=I32, device=DEV)   # noqa: E731
    a, b = gdn.make_page_caches(ds), gdn.make_page_caches(dd)
    status = torch.zeros(1, dtype=I32, device=DEV)
    gdn.gdn_pages_copy(a, b, i32([8, 3, 3]), i32([0, 4, 2]), device_status=status)
    assert gdn.gdn_read_device_status(status) == 0
    for x, y in zip(src, dst):
        y[[0, 4, 2]] = x[[8, 3, 3]]
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dd, dst))
    gdn.gdn_pages_copy(a, b, i32([9, -1, 1, 2, 5]), i32([1, 1, 5, -1, 3]), device_status=status)
    assert gdn.gdn_read_device_status(status) == BOUNDS
    for x, y in zip(src, dst):
        y[3] = x[5]
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dd, dst))
    gdn.gdn_pages_copy(a, b, n=2)              # pages 0 and 1
    gdn.gdn_pages_copy(a, a, i32([0, 1]), i32([7, 8]))
    for x, y in zip(src, dst):
        y[:2] = x[:2]
        x[7:] = x[:2]
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dd + ds, dst + src))


def test_bf16_caches_and_the_most_of_them():
    n = 128
    g = torch.Generator(device=DEV).manual_seed(0)
    caches = [torch.randn(6, 16, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(n)]
    want = [c.clone() for c in caches]
    gdn.gdn_pages_copy(gdn.make_page_caches(caches), gdn.make_page_caches(caches),
                       torch.tensor([5, 0], dtype=I32, device=DEV), torch.tensor([2, 3], dtype=I32, device=DEV))
    for c, w in zip(caches, want):
        w[2], w[3] = w[5].clone(), w[0].clone()
        assert torch.equal(c, w)


def test_bad_entries_in_a_table_are_named_and_passed_over():
    b = Both(10, 16, 3, 4)
    b.extend([0, 1], [40, 20])
    before = b.refs.clone()
    b.table[0, 1] = 10
    b.table[0, 0] = -5
    gdn.gdn_pages_free(b.pool, b.i32([0]), b.ws, device_status=b.status)
    assert gdn.gdn_read_device_status(b.status) == BOUNDS
    before[b.m.table[0][2]] -= 1
    assert torch.equal(b.refs, before) and b.len.tolist() == [0, 20, 0]


def test_captured_steps_follow_the_pool():
    b = Both(64, 16, 8, 6, sizes=(64,))
    slot = torch.zeros(8, 3, dtype=I32, device=DEV)
    run = lambda: gdn.gdn_pages_extend(b.pool, slot, b.ws, device_status=b.status)   # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    b.m.extend(list(range(8)), [3] * 8, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(12):
        graph.replay()
        assert slot.tolist() == b.m.extend(list(range(8)), [3] * 8, 3)
        b.same()


def test_calls_one_after_another_without_a_wait():
    # each call reads what the one before it wrote, launches overlapping
    b = Both(512, 16, 64, 8, sizes=(4096 + 16, 16))
    slot = torch.zeros(16, 21, dtype=I32, device=DEV)
    first, rest = list(range(16)), list(range(16, 64))
    src, dst, all16 = b.i32([s % 16 for s in rest]), b.i32(rest), b.i32(first)
    for _ in range(20):
        gdn.gdn_pages_extend(b.pool, slot, b.ws, device_status=b.status)
        gdn.gdn_pages_fork(b.pool, b.caches, src, dst, b.ws, device_status=b.status)
        gdn.gdn_pages_trim(b.pool, b.caches, b.i32([9] * 16), b.ws, device_status=b.status)
        gdn.gdn_pages_compact(b.pool, b.caches, b.ws, device_status=b.status)
        gdn.gdn_pages_free(b.pool, dst, b.ws, device_status=b.status)
        gdn.gdn_pages_free(b.pool, all16, b.ws, device_status=b.status)
        b.m.extend(first, [21] * 16, 21)
        b.m.fork([s % 16 for s in rest], rest)
        b.m.trim(first, [9] * 16)
        b.m.compact()
        b.m.trim(rest, [0] * 48)
        b.m.trim(first, [0] * 16)
    b.same()
