"""The page pool's calls against the same bookkeeping on the host."""
import random

import pytest
import torch

import more_operators_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


class Both:
    """A pool on the device and on the host, changed by the same calls."""

    def __init__(self, rp, rows, most, pages, page, caches=3, wide=32, stride=None, seed=0, token_bytes=True):
        self.rp, self.page = rp, page
        self.host = ref.Pool([[-1] * most for _ in range(rows)], [0] * rows, [0] * pages, page)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.kv, self.ref = torch.full((rows, most), -1, **i32), torch.zeros(rows, **i32), torch.zeros(pages, **i32)
        g = torch.Generator().manual_seed(seed)
        self.stride = stride or page * wide
        self.room = torch.randint(0, 255, (caches, pages, self.stride), generator=g, dtype=torch.uint8)
        self.dev = self.room.cuda()
        self.ptrs = torch.tensor([c.data_ptr() for c in self.dev], dtype=torch.int64, device="cuda")
        self.caches = dict(page_size=page, page_bytes=page * wide, page_stride=self.stride)
        self.token_bytes = wide if token_bytes else 0
        self.wide = wide

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def extend(self, rows, add):
        st = self.i32([9] * len(rows))
        self.rp.rssm_page_extend(self.table, self.kv, self.ref, self.i32(rows), self.i32(add), st, page_size=self.page)
        assert st.tolist() == self.host.extend(rows, add)
        self.same()
        return st.tolist()

    def fork(self, src, dst, lengths=None):
        st = self.i32([9] * len(src))
        self.rp.rssm_page_fork(self.ptrs, self.table, self.kv, self.ref, self.i32(src), self.i32(dst), st, token_bytes=self.token_bytes,
                               lengths=None if lengths is None else self.i32(lengths), **self.caches)
        assert st.tolist() == self.host.fork(src, dst, lengths or [None] * len(src))
        self.same()
        return st.tolist()

    def release(self, rows, lengths=None):
        self.rp.rssm_page_release(self.table, self.kv, self.ref, self.i32(rows), page_size=self.page,
                                  lengths=None if lengths is None else self.i32(lengths))
        self.host.release(rows, lengths)
        self.same()

    def compact(self):
        live = self.i32([-7])
        self.rp.rssm_page_compact(self.ptrs, self.table, self.kv, self.ref, live, **self.caches)
        assert live.tolist() == [self.host.compact()]
        self.same()
        return live.item()

    def same(self):
        assert self.table.tolist() == self.host.table and self.kv.tolist() == self.host.kv and self.ref.tolist() == self.host.ref
        for c in self.room:
            body = c[:, :self.page * self.wide].unflatten(1, (self.page, self.wide))
            for s, d, n in self.host.copies:
                n = n if n is None or self.token_bytes else self.page
                body[d, :n] = body[s, :n].clone()
        self.host.copies = []
        assert torch.equal(self.dev.cpu(), self.room)


def test_grow_fork_release_pack(rp):
    b = Both(rp, rows=8, most=6, pages=20, page=16)
    assert b.extend([0, 3, 5], [33, 1, 0]) == [0, 0, 0]
    b.fork([0, 0, 3], [1, 2, 4], [32, 20, 5])
    b.extend([1, 2, 0], [1, 40, 16])
    b.release([0])
    assert b.compact() == sum(n > 0 for n in b.host.ref)
    b.release([2, 1], [17, 0])
    b.compact()
    b.compact()                           # nothing left to move
    b.release([1, 2, 3, 4, 5])
    assert b.compact() == 0 and b.kv.tolist() == [0] * 8 and (b.table == -1).all()


@pytest.mark.parametrize("page,wide,stride,tokens", [(1, 16, None, True), (16, 64, 16 * 64 + 48, True), (24, 128, None, False),
                                                     (7, 16 * 300, None, True), (256, 144, None, True)])
def test_page_layouts(rp, page, wide, stride, tokens):
    """Pages below and above a task's bytes, with room between them, copied in part or whole."""
    b = Both(rp, rows=6, most=4, pages=15, page=page, wide=wide, stride=stride, token_bytes=tokens, seed=page)
    b.extend([0, 1], [3 * page, page + 1])
    b.fork([0, 1, 1, 0], [2, 3, 4, 5], [2 * page + page // 2, page + 1, max(1, page - 1), 1])
    b.release([0, 1])
    b.compact()


def test_too_few_pages(rp):
    """Items get all of their pages or none, in order; those that need none go on."""
    b = Both(rp, rows=8, most=8, pages=10, page=16)
    assert b.extend([0, 1, 2, 3], [64, 64, 64, 16]) == [0, 0, 1, 1]
    assert b.extend([4, 5], [0, 32]) == [0, 0]
    assert b.extend([0], [1]) == [1]
    b.release([0], [50])
    assert b.extend([0], [14]) == [0]
    assert b.fork([0, 0], [6, 7], [16, 17]) == [0, 1]
    b.release([1])
    assert b.fork([0, 4, 0], [7, 2, 3], [17, 0, 33]) == [0, 0, 0]


def test_refusals_on_the_device(rp):
    b = Both(rp, rows=6, most=4, pages=20, page=16)
    assert b.extend([0, 0, 6, -1, 1, 2, 3], [20, 5, 1, 1, -1, 65, 64]) == [0, 2, 2, 2, 2, 2, 0]
    assert b.extend([0], [2 ** 31 - 1]) == [2]
    assert b.fork([0, 0, 9, 0, 0, 4], [1, 1, 2, 3, 0, 2], [20, 3, 1, 1, 1, 5]) == [0, 2, 2, 2, 2, 2]
    assert b.fork([0, 0], [2, 7], [-1, 1]) == [2, 2]
    b.release([17, -3, 0, 0, 3, 3], [0, 0, -1, 400, 5, 40])


def test_a_row_named_twice_is_released_once(rp):
    b = Both(rp, rows=4, most=40, pages=60, page=4)
    b.extend([0, 1], [150, 33])
    b.fork([0], [2])
    b.release([0, 0, 0, 1, 1], [100, 100, 100, 0, 0])
    b.release([0] * 300, None)


def test_a_shared_last_page_is_not_written(rp):
    """A row cut back into a page that another row holds cannot grow before it is forked."""
    b = Both(rp, rows=4, most=4, pages=12, page=16)
    b.extend([0], [40])
    b.fork([0], [1], [32])
    b.release([0], [20])
    assert b.extend([0], [4]) == [3]
    assert b.extend([0], [0]) == [0]
    b.fork([0], [2])
    assert b.extend([2], [4]) == [0]
    b.release([1])
    assert b.extend([0], [4]) == [0]


def test_pages_counted_by_the_caller(rp):
    """A count that no row explains keeps its page, and moves with it."""
    b = Both(rp, rows=2, most=4, pages=12, page=16)
    b.ref[9] = b.host.ref[9] = 2
    b.extend([0], [50])
    b.release([0], [16])
    assert b.compact() == 2 and b.ref[1].item() == 2


@pytest.mark.parametrize("pages", [1, 15, 16, 17, 1023, 16384, 16400, 70001])
def test_pool_sizes(rp, pages):
    """Free pages are found past the borders of a round of the search, lowest first."""
    b = Both(rp, rows=4, most=pages + 1, pages=pages, page=2, caches=0)
    n = max(0, 2 * (pages - 3))
    assert b.extend([0], [n]) == [0]
    assert b.extend([1, 2], [2, 3]) == [0 if pages - n // 2 >= 1 else 1, 0 if pages - n // 2 >= 3 else 1]
    b.release([0], [n // 3])
    b.compact()
    b.extend([3], [5])


def test_many_items(rp):
    """More items than one round, rows in any order."""
    rng = random.Random(3)
    b = Both(rp, rows=3000, most=3, pages=4000, page=8, caches=1, wide=16)
    rows = list(range(2500))
    rng.shuffle(rows)
    b.extend(rows + rows[:40], [rng.randint(0, 20) for _ in range(2540)])
    b.fork([rng.randint(0, 2600) for _ in range(600)], [2500 + rng.randint(0, 499) for _ in range(600)],
           [rng.randint(0, 24) for _ in range(600)])
    b.release([rng.randint(0, 2999) for _ in range(1500)], [rng.randint(0, 12) for _ in range(1500)])
    b.compact()
    b.extend(rows, [rng.randint(0, 9) for _ in rows])


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_any_order_of_calls(rp, seed):
    rng = random.Random(seed)
    rows, most, page = rng.randint(3, 9), rng.randint(2, 9), rng.choice([1, 5, 16])
    b = Both(rp, rows, most, pages=rng.randint(6, 40), page=page, caches=2, wide=16, seed=seed)
    for _ in range(25):
        n = rng.randint(1, 6)
        some = [rng.randint(-1, rows) for _ in range(n)]
        kind = rng.randint(0, 3)
        if kind == 0:
            b.extend(some, [rng.randint(-1, 2 * page) for _ in range(n)])
        elif kind == 1:
            b.fork([rng.randint(0, rows - 1) for _ in range(n)], some, [rng.randint(0, most * page) for _ in range(n)])
        elif kind == 2:
            b.release(some, [rng.randint(-1, most * page) // 2 for _ in range(n)])
        else:
            b.compact()


def test_copy(rp):
    b = Both(rp, rows=1, most=1, pages=30, page=16, wide=1040)
    src, dst = [3, 3, 29, 7, 40, 2], [5, 6, 0, 7, 1, -1]
    rp.rssm_page_copy(b.ptrs, b.i32(src), b.i32(dst), num_pages=30, page_bytes=16 * 1040)
    for s, d in ((3, 5), (3, 6), (29, 0)):
        b.room[:, d] = b.room[:, s]
    assert torch.equal(b.dev.cpu(), b.room)


def test_rows_a_multiple_of_1024_apart(rp):
    """Repeated rows are told from different ones, whichever table finds them."""
    b = Both(rp, rows=4100, most=2, pages=600, page=4, caches=1, wide=16)
    rows = [5, 1029, 5, 2053, 1029, 4096, 0, 1024, 2048, 0, 2053, 7]
    assert b.extend(rows, [3] * 12) == [0, 0, 2, 0, 2, 0, 0, 0, 0, 2, 2, 0]
    assert b.fork([5] * 5, [6, 1030, 6, 4102, 2054], [3, 2, 1, 1, 3]) == [0, 0, 2, 2, 0]
    b.extend(rows * 20, [1] * 240)
    b.extend(rows * 30, [1] * 360)


@pytest.mark.parametrize("items", [1, 64, 65, 255, 256, 257, 1025])
@pytest.mark.parametrize("pages", [300, 5000, 40000])
def test_items_and_pools(rp, items, pages):
    """The forms for few and many items, for pools of one round and several."""
    b = Both(rp, rows=2 * items + 1, most=40, pages=pages, page=2, caches=1, wide=16)
    rng = random.Random(items)
    b.extend(list(range(items)), [rng.randint(0, 70) for _ in range(items)])
    b.fork([rng.randint(0, items) for _ in range(items)], [items + i for i in range(items)], [rng.randint(0, 60) for _ in range(items)])
    b.release(list(range(0, items, 2)))
    b.extend(list(range(items)), [rng.randint(0, 9) for _ in range(items)])


def test_strided_table(rp):
    """Rows of a wider table; what lies beside them stays."""
    wide = torch.full((4, 10), 77, dtype=torch.int32, device="cuda")
    table = wide[:, 2:6]
    table.fill_(-1)
    b = Both(rp, rows=4, most=4, pages=12, page=16)
    b.table = table
    b.extend([2, 0], [20, 50])
    b.fork([0], [1], [30])
    b.release([0], [10])
    b.compact()
    assert (wide[:, :2] == 77).all() and (wide[:, 6:] == 77).all()


def test_captured_and_replayed(rp):
    """One graph of a cycle, replayed: every call sees the tables as they are then, with one workspace for all."""
    a, b = (Both(rp, rows=6, most=6, pages=24, page=16, seed=5) for _ in range(2))
    for p in (a, b):
        p.extend([0, 1], [40, 60])
    ws = torch.full((rp.rssm_pages_workspace(num_items=2, num_rows=6, num_pages=24),), 255, dtype=torch.uint8, device="cuda")
    src, dst, add, live = b.i32([0, 1]), b.i32([2, 3]), b.i32([7, 20]), b.i32([0])
    st = b.i32([0, 0])

    def cycle(p, ws=None):
        rp.rssm_page_fork(p.ptrs, p.table, p.kv, p.ref, src, dst, st, token_bytes=32, workspace=ws, **p.caches)
        rp.rssm_page_extend(p.table, p.kv, p.ref, dst, add, st, page_size=16, workspace=ws)
        rp.rssm_page_release(p.table, p.kv, p.ref, src, page_size=16)
        rp.rssm_page_compact(p.ptrs, p.table, p.kv, p.ref, live, workspace=ws, **p.caches)
        rp.rssm_page_fork(p.ptrs, p.table, p.kv, p.ref, dst, src, st, token_bytes=32, workspace=ws, **p.caches)
        rp.rssm_page_release(p.table, p.kv, p.ref, dst, page_size=16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cycle(b, ws)
    for _ in range(4):
        cycle(a)
        g.replay()
        torch.cuda.synchronize()
        for x, y in ((a.table, b.table), (a.kv, b.kv), (a.ref, b.ref), (a.dev, b.dev)):
            assert torch.equal(x, y)


def test_attention_of_a_fork(rp):
    """A fork answers as its source did, and goes its own way afterwards."""
    page, Hkv, D = 16, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")       # noqa: E731
    kc, vc = rn(12, page, Hkv, D), rn(12, page, Hkv, D)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    table, kv, ref_ = torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), i32(0, 0, 0), torch.zeros(12, dtype=torch.int32, device="cuda")
    st = i32(0)
    rp.rssm_page_extend(table, kv, ref_, i32(0), i32(40), st, page_size=page)
    rp.rssm_paged_append(kc, vc, rn(40, Hkv, D), rn(40, Hkv, D), table[:1], i32(0, 40), kv[:1])
    ptrs = rp.pointer_table([kc, vc], "cuda")
    row = page * Hkv * D * 4
    rp.rssm_page_fork(ptrs, table, kv, ref_, i32(0), i32(1), st, page_size=page, page_bytes=row, token_bytes=Hkv * D * 4)

    def attend(r, q, k=None, v=None):
        if k is not None:
            rp.rssm_page_extend(table, kv, ref_, i32(r), i32(1), st, page_size=page)
            rp.rssm_paged_append(kc, vc, k, v, table[r:r + 1], i32(0, 1), kv[r:r + 1])
        out = torch.empty_like(q)
        rp.rssm_paged_attention(q, kc, vc, table[r:r + 1], i32(0, 1), kv[r:r + 1], out, max_seq_len=1, max_kv_len=64)
        return out
    q = rn(1, 4, D)
    first = attend(0, q)
    assert torch.equal(first, attend(1, q))
    k, v = rn(1, Hkv, D), rn(1, Hkv, D)
    other = attend(1, q, k, v)
    assert torch.equal(attend(0, q), first) and not torch.equal(other, first)
    assert torch.equal(attend(0, q, k, v), other)
