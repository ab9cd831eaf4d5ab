"""Pages given back by books of more than 1024 sequences, where a thread of the deciding block has several sequences: most
of all threads' pages are then dealt out again to all threads, which read the other sequences' rows, lengths and requests
while the step is decided.  Every number of every step is equal to the book kept in plain Python."""
import random

import pytest

from test_gpu_pages import Book, nm  # noqa: F401

pytestmark = pytest.mark.gpu

PAGE, WIDTH = 16, 24
THREADS, FEW = 1024, 8                  # of the deciding block; pages that a thread gives back by itself


def most_of_a_thread(book, adds):
    """The most pages that the sequences of one thread give back in this step."""
    B = len(adds)
    each = 4 if B <= 4 * THREADS else -(-B // THREADS)
    freed = [-(-n // PAGE) - -(-max(n + min(a, 0), 0) // PAGE) if n > 0 else 0 for n, a in zip(book.lens, adds)]
    return max(sum(freed[t:t + each]) for t in range(0, B, each))


def grown(nm, B, r, pages=None):  # noqa: F811
    """A book whose sequences hold 0 to 20 pages (some are padding)."""
    book = Book(nm, B, WIDTH, pages or B * WIDTH // 2 + 7, PAGE, seed=B)
    book.put(lens=[-1 if r.random() < 0.02 else 0 for _ in range(B)])
    book.step([r.choice((0, 1, 160, r.randint(1, 320))) for _ in range(B)], B * 320)
    return book


@pytest.mark.parametrize("B", (1025, 2500, 4096, 4097, 5000))
def test_many_end_while_others_grow(nm, B):  # noqa: F811
    r = random.Random(B)
    book = grown(nm, B, r)
    for rows in (B * 200, 3000, B * 200):
        adds = [r.choice((-n, -n, -r.randint(0, n), 5, 17, 150, 0)) if n > 0 else r.choice((-3, 0, 40, 200)) for n in book.lens]
        assert most_of_a_thread(book, adds) > FEW
        book.step(adds, rows)
    adds = [-2 ** 31] * B
    assert most_of_a_thread(book, adds) > FEW
    book.step(adds, 4)
    assert sorted(book.free) == list(range(len(book.free)))


@pytest.mark.parametrize("B", (1025, 4096, 5000))
@pytest.mark.parametrize("at", ("first", "middle", "last"))
def test_one_thread_gives_back_much(nm, B, at):  # noqa: F811
    """Its neighbours' sequences give nothing back, hold nothing or are padding; in the same step others grow."""
    r = random.Random(B)
    book = grown(nm, B, r)
    b = {"first": 0, "middle": B // 2, "last": B - 1}[at]
    book.put(lens=[320 if i == b else n for i, n in enumerate(book.lens)],
             table=[list(range(WIDTH)) if i == b else row for i, row in enumerate(book.table)])
    for back in (-150, -170):                           # from 20 pages, of which the second leaves none
        adds = [0] * B
        adds[b] = back
        for i in range(0, B, 97):
            if i != b:
                adds[i] = 33
        assert most_of_a_thread(book, adds) > FEW
        book.step(adds, 4000)
    assert book.lens[b] == 0


@pytest.mark.parametrize("B", (2500, 5000))
def test_a_full_stack(nm, B):  # noqa: F811
    """Counts of free pages near their end: what does not fit on the stack is dropped, and the rest serves the step."""
    r = random.Random(B)
    book = grown(nm, B, r)
    pages = len(book.free)
    for n_free in (pages - 1000, pages - 1, pages, pages + 5, -1):
        held = list(book.lens)
        book.put(n_free=n_free)
        adds = [-n if i % 3 == 0 and n > 0 else 20 if i % 7 == 0 else 0 for i, n in enumerate(held)]
        assert most_of_a_thread(book, adds) > FEW
        book.step(adds, 100000)
        book.put(lens=held)
