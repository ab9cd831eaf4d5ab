"""kv_plan on the GPU against the book kept in plain Python: every number of every step is equal."""
import random

import pytest
import torch

import serve_reference as sref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_matrix_vector_amd as nm
    nm.lib()
    return nm


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Book:
    """A KVPages and the same in plain Python."""

    def __init__(self, nm, B, width, n_pages, page, seed=0):
        self.nm, self.page = nm, page
        self.pages = nm.KVPages(B, width, n_pages, page)
        order = list(range(n_pages))
        random.Random(seed).shuffle(order)
        self.pages.free.copy_(i32(order))
        self.table, self.lens, self.free, self.n_free = [[0] * width for _ in range(B)], [0] * B, order, n_pages

    def put(self, lens=None, n_free=None, table=None):
        if lens is not None:
            self.lens = list(lens)
            self.pages.lens.copy_(i32(lens))
        if n_free is not None:
            self.n_free = n_free
            self.pages.n_free.fill_(n_free)
        if table is not None:
            self.table = [list(r) for r in table]
            self.pages.table.copy_(i32(table))

    def step(self, adds, rows, **kw):
        got = self.nm.kv_plan(self.pages, i32(adds), rows, **kw)
        self.n_free, *want = sref.plan(self.table, self.lens, self.free, self.n_free, self.page, adds, rows)
        for name, g, w in zip(("starts", "slots", "positions", "granted"), got, want):
            assert g.tolist() == w, name
        self.same()
        return got

    def same(self):
        p = self.pages
        assert p.lens.tolist() == self.lens and p.n_free.item() == self.n_free
        assert p.free.tolist() == self.free and p.table.tolist() == self.table


@pytest.mark.parametrize("page", (16, 32, 64, 128, 256))
@pytest.mark.parametrize("B", (1, 2, 33, 64, 200))
def test_random_steps(nm, B, page):
    """Sequences that start, grow, shrink and end, with too few pages, rows or places in the table now and then."""
    r = random.Random(B * page)
    width = r.randint(1, 9)
    book = Book(nm, B, width, max(2, B * width // 2), page, seed=B)
    for _ in range(12):
        adds = []
        for b in range(B):
            kind = r.random()
            adds.append(0 if kind < 0.2 else r.randint(1, 3) if kind < 0.4 else r.randint(1, width * page) if kind < 0.7
                        else -r.randint(1, 40) if kind < 0.85 else -r.randint(1, 2 * width * page))
        book.step(adds, r.choice((0, 1, B, B * page, B * width * page)))


@pytest.mark.parametrize("B", (1, 1023, 1024, 1025, 2500, 5000))
def test_many_sequences(nm, B):
    """Several sequences a thread; rows in one launch and in two."""
    r = random.Random(B)
    book = Book(nm, B, 4, 2 * B + 1, 16, seed=B)
    for rows in (B * 64, 9000, 3, B * 64):
        book.step([r.choice((0, 1, 5, 17, 40, -3, -64)) for _ in range(B)], rows)


@pytest.mark.parametrize("rows", (8191, 8192, 8193, 30000))
def test_many_rows(nm, rows):
    """Long prompts among sequences that ask for nothing, on both sides of the second launch."""
    book = Book(nm, 300, 600, 2000, 16)
    adds = [0] * 300
    adds[0], adds[7], adds[299] = 100, rows - 101, 1
    book.step(adds, rows)
    adds[7] = -(rows - 200)
    book.step([-a if a < 0 else 0 for a in adds], rows)
    book.step(adds, rows)


def test_undo(nm):
    """Dropping what was just granted leaves the stack and the lengths as they were."""
    book = Book(nm, 50, 8, 300, 16)
    r = random.Random(1)
    book.step([r.randint(0, 60) for _ in range(50)], 5000)
    before = (list(book.free), book.n_free, list(book.lens))
    adds = [r.randint(0, 50) for _ in range(50)]
    granted = book.step(adds, 5000)[3]
    book.step([-g for g in granted.tolist()], 0)
    assert (book.n_free, book.lens) == before[1:] and book.free[:book.n_free] == before[0][:book.n_free]


def test_padding_and_odd_books(nm):
    """Padding rows, a count of free pages outside its range, lengths that the table cannot hold, negative pages."""
    book = Book(nm, 4, 2, 10, 16)
    book.put(lens=[-1, -7, 0, -2 ** 31])
    book.step([5, -5, 3, 2 ** 31 - 1], 100)
    book.put(n_free=-3)
    book.step([0, 0, 20, 0], 100)
    book.put(n_free=2 ** 31 - 1)
    book.step([0, 0, 20, 0], 100)
    book.put(lens=[1000, 33, 3, 0], n_free=4, table=[[1, 2], [3, 4], [-5, 6], [7, 8]])
    book.step([-990, -1, 4, 2 ** 31 - 1], 100)
    book.put(lens=[0, 2 ** 31 - 1, 3, 16], n_free=9)
    book.step([-2 ** 31, -2 ** 31, -2 ** 31, 16], 100)


def test_order(nm):
    """The first that finds no room closes the door behind it, whatever the later ones ask for."""
    book = Book(nm, 5, 4, 6, 16)
    book.step([40, 0, 64, 1, 1], 1000)                  # 3 pages, then 4 of the 3 left
    assert book.lens == [40, 0, 0, 0, 0]
    book.step([1, 65, 8, 1, 1], 10)                     # too long for its row, then two that fill the rows
    assert book.lens == [41, 0, 8, 1, 0]


def test_pages_of_one_step(nm):
    """Pages that end in a step serve its new sequences, the first one first."""
    book = Book(nm, 2, 4, 4, 16)
    book.step([64, 0], 64)
    pages = list(book.table[0])
    book.step([-40, 48], 64)                            # pages 2, 3 come back; three are asked for
    assert book.lens == [24, 0]
    book.step([-1, 32], 64)
    assert book.table[1][:2] == pages[2:]


def test_out_stream_and_graph(nm):
    book = Book(nm, 3, 64, 100, 16)
    out = (torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(20, dtype=torch.int64, device="cuda"),
           torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"))
    got = book.step([5, 0, 9], 20, out=out)
    assert all(a is b for a, b in zip(got, out))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    nm.kv_plan(book.pages, i32([0, 0, 0]), 20, stream=s)
    s.synchronize()
    adds = i32([1, 2, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nm.kv_plan(book.pages, adds, 20, out=out)
    for i in range(5):
        step = [i, 3, -1]
        adds.copy_(i32(step))
        g.replay()
        torch.cuda.synchronize()
        book.n_free, *want = sref.plan(book.table, book.lens, book.free, book.n_free, 16, step, 20)
        assert [t.tolist() for t in out] == want
        book.same()


def test_refusals(nm):
    pages = nm.KVPages(2, 4, 8, 16)
    with pytest.raises(TypeError):
        nm.kv_plan(object(), i32([1, 1]), 4)
    with pytest.raises(ValueError):
        nm.kv_plan(pages, i32([1, 1, 1]), 4)
    with pytest.raises(TypeError):
        nm.kv_plan(pages, torch.tensor([1, 1], device="cuda"), 4)
    with pytest.raises(ValueError):
        nm.kv_plan(pages, i32([1, 1]), -1)
    with pytest.raises(ValueError):
        nm.kv_plan(pages, i32([1, 1]), 4, out=(i32([0, 0, 0]),))
    with pytest.raises(nm.NmError):                     # adds among the outputs
        adds = i32([1, 1])
        nm.kv_plan(pages, adds, 0, out=(i32([0, 0, 0]), torch.empty(0, dtype=torch.int64, device="cuda"), i32([]), adds))
