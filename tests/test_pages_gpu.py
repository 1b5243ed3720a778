"""The page management on the GPU (attn_pages_append, _trim, _fork, _compact,
_copy) against the sequential model: table, lengths, counts, status and every
byte of the pages must be equal."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_44_b200 as A
import oracle

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Both:
    """One cache on the GPU and in the model; every call is made on both and compared."""

    def __init__(self, B, cols, n, Hk=2, page=16, d=64, dt=BF, seed=0):
        self.rng = np.random.default_rng(seed)
        self.dt = dt
        self.cache = A.paged_cache(B, cols, n, Hk, page, d, dt)
        for x in (self.cache.k, self.cache.v):
            x.copy_(self.values(x.shape))
        self.book = oracle.PageBook(*(self.bits(x) for x in (self.cache.k, self.cache.v)),
                                    *(x.cpu().numpy() for x in (self.cache.table, self.cache.lens,
                                                               self.cache.refs)))
        A.get_status()

    def values(self, shape):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(self.dt)

    def bits(self, x):
        return x.cpu().view(torch.int16).numpy()

    def same(self, status=0):
        c, b = self.cache, self.book
        torch.cuda.synchronize()
        assert A.get_status() == status
        assert (c.lens.cpu().numpy() == b.lens).all()
        assert (c.table.cpu().numpy() == b.table).all()
        assert (c.refs.cpu().numpy() == b.refs).all()
        assert (self.bits(c.k) == b.k).all() and (self.bits(c.v) == b.v).all()

    def append(self, n_new, counts=None):
        c = self.cache
        shape = (c.lens.shape[0], c.k.shape[1], n_new, c.k.shape[3])
        kn, vn = self.values(shape), self.values(shape)
        A.pages_append(c, kn.cuda(), vn.cuda(), None if counts is None else i32(counts))
        self.same(self.book.append(self.bits(kn), self.bits(vn), counts))

    def trim(self, lens=None, rows=None):
        A.pages_trim(self.cache, None if lens is None else i32(lens), None if rows is None else i32(rows))
        self.same(self.book.trim(lens, rows))

    def fork(self, parents, children):
        A.pages_fork(self.cache, i32(parents), i32(children))
        self.same(self.book.fork(parents, children))

    def compact(self):
        n = A.pages_compact(self.cache)
        assert self.book.compact() == int(n)
        self.same()


@pytest.mark.parametrize("page,d,dt,Hk", [(16, 64, BF, 2), (32, 128, FP, 1), (64, 16, BF, 3),
                                          (128, 32, FP, 2), (256, 128, BF, 1)])
def test_append_across_pages(page, d, dt, Hk):
    x = Both(5, 4, 30, Hk, page, d, dt)
    x.append(1)
    x.append(page - 1, [page - 1, page - 2, 0, 1, page - 1])
    x.append(2 * page + 1, [2 * page + 1, page, 1, 0, 2 * page])
    x.append(3, [0, 1, 2, 3, 0])


def test_append_many_sequences():
    """More sequences than the deciding CTA has threads, more rows than one tile."""
    x = Both(2500, 3, 5000, 1, 16, 16)
    x.append(2)
    x.append(33, list(x.rng.integers(0, 34, 2500)))


def test_append_finds_scattered_free_pages():
    """Free pages past the first step of the search (16384 counts)."""
    x = Both(40, 1000, 40000, 1, 16, 16)
    x.append(16 * 900, [16 * 900] * 20 + [0] * 20)       # 18000 pages
    x.trim(rows=[3])                                       # a hole of 900 pages
    x.append(16 * 500, [0] * 20 + [16 * 500] * 4 + [7] * 16)


def test_append_copies_a_shared_last_page():
    x = Both(6, 4, 16)
    x.append(21, [21, 0, 0, 16, 0, 0])
    x.fork([0, 0, 3], [1, 2, 4])
    x.append(1, [1, 0, 1, 1, 1, 0])        # rows 0 and 2 copy, 3 and 4 start a page
    x.append(1, [1, 1, 1, 0, 0, 0])        # row 1 holds its page alone by now
    x.fork([1], [5])
    x.trim([18], [5])
    x.append(2, [0, 2, 0, 0, 0, 2])        # both copy, the page nobody holds is free again


def test_append_without_enough_pages():
    x = Both(4, 4, 5)
    x.append(20, [20, 3, 20, 20])          # two, one, two: the last is not served
    x.append(13, [1, 13, 0, 1])            # rows 0 and 1 fit their pages, row 3 needs one
    x.trim(rows=[0])
    x.append(17, [17, 17, 17, 17])
    assert x.book.lens.tolist()[0] == 17


def test_append_refuses_what_cannot_be_right():
    x = Both(4, 2, 9)
    x.append(5, [6, 5, -1, 5])             # counts out of range
    x.append(30, [0, 30, 0, 28])           # 5 + 30 > 32 positions
    x.cache.table[1, 0] = 99               # a page that does not exist
    x.book.table[1, 0] = 99
    x.append(1)
    x.cache.lens[3] = -7
    x.book.lens[3] = -7
    x.append(1, [1, 0, 1, 1])


def test_trim_releases_pages():
    x = Both(5, 4, 20)
    x.append(60, [60, 17, 0, 32, 5])
    x.fork([0], [2])
    x.trim([33, 99, 16, 32, 0])            # shared pages keep a reference
    x.trim([5, 20, 1], [0, 0, 3])          # a row listed twice ends at the smaller length
    x.trim([-1, 1, 1], [0, 9, -2])         # nothing here can be right
    x.trim()
    assert (x.book.refs == 0).all()


def test_fork_rules():
    x = Both(8, 3, 20)
    x.append(40, [40, 16, 0, 0, 0, 0, 0, 0])
    x.fork([0, 1, 0], [2, 3, 4])
    x.fork([0, 1, 5], [5, 5, 6])           # child 5 twice; 5 is a parent and a child
    x.fork([0, 9, 1, 7], [1, 6, -1, 7])    # not empty; no such rows; itself
    x.fork([7], [6])                       # an empty parent


@pytest.mark.parametrize("page,d,Hk,n", [(16, 64, 2, 50), (16, 64, 3, 700), (32, 32, 3, 90), (64, 128, 8, 13), (256, 128, 4, 11), (16, 16, 1, 9000)])
def test_compact(page, d, Hk, n):
    x = Both(9, max(2, n // 6), n, Hk, page, d)
    top = page * max(1, n // 12)
    x.append(top, list(x.rng.integers(0, top + 1, 9)))
    x.trim(rows=[0, 2, 5])
    x.fork([1], [2])
    x.compact()
    x.compact()                            # nothing moves
    x.append(3, [3] * 9)


def test_compact_of_an_empty_and_of_a_full_cache():
    x = Both(2, 4, 6)
    x.compact()
    x.append(48, [48, 48])
    x.compact()


def test_compact_into_a_second_table_leaves_the_first_readable():
    x = Both(4, 4, 30)
    x.append(60, [60, 50, 40, 30])
    x.trim(rows=[0, 2])
    c = x.cache
    k0, table0, refs0 = c.k.clone(), c.table.clone(), c.refs.clone()
    table, refs = torch.empty_like(c.table), torch.full_like(c.refs, 77)
    n = A.pages_compact(c, table_out=table, refs_out=refs)
    torch.cuda.synchronize()
    assert A.get_status() == 0 and torch.equal(c.table, table0) and torch.equal(c.refs, refs0)
    x.book.compact()
    assert int(n) == (x.book.refs > 0).sum()
    assert (table.cpu().numpy() == x.book.table).all() and (refs.cpu().numpy() == x.book.refs).all()
    held = table0[table0 >= 0].long()
    assert torch.equal(c.k[held], k0[held])                       # the old places
    assert torch.equal(c.k[table[table0 >= 0].long()], k0[held])  # the new ones


@pytest.mark.parametrize("Hk,page,d", [(3, 32, 128), (1, 16, 16), (3, 16, 32), (1, 64, 64), (2, 32, 128)])
def test_copy_pages(Hk, page, d):
    x = Both(1, 1, 12, Hk, page, d)
    c = x.cache
    k, v = c.k.clone(), c.v.clone()
    A.pages_copy(c, i32([1, 5, -1, 7, 3]), i32([2, 6, 0, 7, 11]))
    torch.cuda.synchronize()
    assert A.get_status() == 0
    to, of = [2, 6, 11], [1, 5, 3]
    k[to], v[to] = k[of], v[of]
    assert torch.equal(c.k, k) and torch.equal(c.v, v)
    A.pages_copy(c, i32([12, 1, 2]), i32([0, 12, -1]))            # outside the cache
    torch.cuda.synchronize()
    assert A.get_status() == A.ATTN_ERR_INVALID_ARG
    assert torch.equal(c.k, k) and torch.equal(c.v, v)


@pytest.mark.parametrize("seed", range(12))
def test_random_runs(seed):
    rng = np.random.default_rng(100 + seed)
    page = int(rng.choice([16, 32, 64]))
    B = int(rng.integers(2, 12))
    x = Both(B, 5, int(rng.integers(8, 40)), int(rng.integers(1, 4)), page, int(rng.choice([16, 64])),
             [BF, FP][seed % 2], seed)
    for _ in range(12):
        what = rng.integers(5)
        if what <= 1:
            n = int(rng.integers(1, 2 * page))
            x.append(n, list(rng.integers(0, n + 1, B)))
        elif what == 2:
            m = int(rng.integers(1, B + 1))
            x.trim(list(rng.integers(0, 4 * page, m)), list(rng.integers(0, B, m)))
        elif what == 3:
            m = int(rng.integers(1, 4))
            x.fork(list(rng.integers(0, B, m)), list(rng.integers(0, B, m)))
        else:
            x.compact()


def test_replayed_from_a_graph_and_on_another_stream():
    """A step of fork, append and trim, captured once: each replay does it again."""
    x = Both(4, 4, 16)
    x.append(21, [21, 0, 30, 0])
    c = x.cache
    kn, vn = (x.values((4, 2, 1, 64)) for _ in range(2))
    kd, vd = kn.cuda(), vn.cuda()
    counts, rows, parents, children = i32([0, 1, 0, 1]), i32([1, 3]), i32([0, 2]), i32([1, 3])
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def step():
        A.pages_trim(c, None, rows)
        A.pages_fork(c, parents, children)
        A.pages_append(c, kd, vd, counts, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    for _ in range(5):
        x.book.trim(None, [1, 3])
        x.book.fork([0, 2], [1, 3])
        x.book.append(x.bits(kn), x.bits(vn), [0, 1, 0, 1])
    x.same()


@pytest.mark.parametrize("over", [1, 17, 2 ** 31 - 1])
@pytest.mark.parametrize("rows", [[1], [1, 1], [0, 1, 1, 2]])
def test_trim_leaves_a_row_whose_length_cannot_be_right(rows, over):
    """A length past the table (or below 0) stays, with the row's pages and their counts,
    however often the row is listed; the other rows are trimmed."""
    x = Both(4, 3, 20)
    x.append(48, [48, 48, 20, 5])
    for bad in (min(48 + over, 2 ** 31 - 1), -over):
        x.cache.lens[1] = bad
        x.book.lens[1] = bad
        x.trim([17 - i for i in range(len(rows))], rows)
        assert x.book.lens[1] == bad
    x.cache.lens[1] = 48
    x.book.lens[1] = 48
    x.trim()
    assert (x.book.refs == 0).all()


@pytest.mark.parametrize("count", [0, -3])
def test_append_does_not_write_to_a_page_that_counts_as_free(count):
    """A partly filled last page whose count says free could be handed to another sequence
    in the same call; its own sequence gets nothing, the others do."""
    x = Both(4, 3, 8)
    x.append(20, [20, 5, 16, 0])
    page = int(x.book.table[1, 0])
    x.cache.refs[page] = count
    x.book.refs[page] = count
    x.append(6, [6, 6, 0, 0])
    assert x.book.lens.tolist() == [26, 5, 16, 0]
