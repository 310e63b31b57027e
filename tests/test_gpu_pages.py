"""Pages of the caches against their statement in plain Python: whole numbers, equal everywhere."""
import numpy as np
import pytest

import serve_testlib as T
from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


def ints(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Both:
    """A handle and table, and their statement."""

    def __init__(self, P, n_pages, page, table, lens, refs, batch=None):
        import torch
        self.torch, self.P = torch, P
        self.want = T.Pages(n_pages, page, table, lens, refs)
        self.pages = P.PacePages(n_pages, page, batch or len(table))
        self.pages.refs.copy_(ints(torch, refs))
        self.table, self.lens = ints(torch, table), ints(torch, lens)

    def same(self, moves=False):
        got = [self.table.cpu().numpy(), self.lens.cpu().numpy(), self.pages.refs.cpu().numpy()]
        for x, y, what in zip(got, (self.want.table, self.want.lens, self.want.refs), ("table", "lens", "refs")):
            assert np.array_equal(x, y), f"{what}\n{x}\n{y}"
        if moves:
            n = int(self.pages.n_moves)
            assert list(zip(self.pages.src[:n].tolist(), self.pages.dst[:n].tolist())) == self.want.moves

    def select(self, src=None):
        self.pages.select(self.table, self.lens, None if src is None else ints(self.torch, src))
        self.want.select(src)
        self.same()

    def take(self, n_new):
        fits = self.torch.full((len(self.want.table),), -7, dtype=self.torch.int32, device="cuda")
        self.pages.take(self.table, self.lens, ints(self.torch, n_new), fits)
        want, bad = self.want.take(n_new)
        assert np.array_equal(fits.cpu().numpy(), want)
        self.same(moves=True)
        assert self.pages.status(clear=True) == (self.P.PACE_PAGES_BAD_CELL if any(bad) else 0)
        return want

    def compact(self):
        self.pages.compact(self.table)
        self.want.compact()
        self.same(moves=True)

    def grow(self, by):
        """The caller's part: the rows that got their pages have their tokens."""
        by = np.asarray(by)
        self.want.lens = self.want.lens + by
        self.lens += ints(self.torch, by)


def filled(P, rng, B, cols, page, n_pages, lens):
    table = np.full((B, cols), -1)
    refs = np.zeros(n_pages, int)
    order = iter(rng.permutation(n_pages))
    for b in range(B):
        for c in range(-(-lens[b] // page)):
            table[b, c] = next(order)
            refs[table[b, c]] = 1
    return Both(P, n_pages, page, table, lens, refs)


@pytest.mark.parametrize("B,cols,page,n_pages", [(1, 1, 32, 1), (3, 5, 32, 40), (7, 9, 64, 300), (40, 20, 32, 900), (130, 17, 128, 20000),
                                                 (1000, 9, 32, 12000), (5, 300, 64, 1700)])
def test_a_serving_life(P, B, cols, page, n_pages):
    """Rows grow, are shared, reordered, shortened and freed at random, and the pool is compacted; every step as stated."""
    rng = np.random.default_rng(B * 10 + cols)
    lens = rng.integers(0, cols * page // 2 + 1, B)
    lens[rng.random(B) < 0.2] = 0
    while (-(-lens // page)).sum() > n_pages:
        lens //= 2
    x = filled(P, rng, B, cols, page, n_pages, lens)
    for step in range(12):
        what = step % 6
        if what in (0, 3):
            src = rng.integers(-1, B, B) if what == 0 else np.where(rng.random(B) < 0.3, -1, np.arange(B))
            x.select(src)
        elif what in (1, 4):
            room = cols * page - x.want.lens
            by = np.minimum(rng.integers(0, 2 * page, B) if what == 1 else rng.integers(0, 4, B), room)
            got = x.take(by)
            x.grow(by * got)
        elif what == 2:
            back = np.minimum(rng.integers(0, page, B), x.want.lens)
            x.grow(-back)
            x.select()
        else:
            x.compact()
    assert x.pages.status() == 0


def test_samples_of_one_prompt(P):
    """All holders of a last page write: the first keeps it, the others copy."""
    x = filled(P, np.random.default_rng(0), 6, 4, 32, 16, [40, 0, 0, 64, 0, 0])
    x.select([0, 0, 0, 3, 3, 3])
    x.take([1] * 6)
    assert len(x.want.moves) == 2                # (rows 3..5 end with a whole page)
    x.grow([1] * 6)
    x.select([0, 0, 2, 2, 4, -1])
    x.take([0, 5, 1, 30, 1, 0])


def test_a_full_pool_serves_rows_in_order(P):
    x = filled(P, np.random.default_rng(0), 5, 8, 32, 12, [64, 33, 32, 0, 32])
    assert x.take([32 * 3, 0, 32 * 5, 40, 0]).tolist() == [1, 1, 0, 0, 1]
    assert x.take([0, 32, 0, 0, 1]).tolist() == [1, 1, 1, 1, 1]
    x.select([-1] * 5)
    assert not x.want.refs.any()


@pytest.mark.parametrize("lens,n_pages,fits", [([37, 41], 2, [0, 1]), ([41, 37], 2, [1, 0]), ([37, 41, 37, 63], 3, [1, 0, 0, 1]),
                                               ([40, 40, 40], 2, [1, 0, 0]), ([37, 41, 39], 4, [1, 1, 1])])
def test_the_longest_holder_keeps_a_page(P, lens, n_pages, fits):
    """Rows that share their first two pages and end at different tokens of the second. However far the pool goes, no row's tokens lie where
    another one may write."""
    table = [[0, 1, -1]] * len(lens)
    x = Both(P, n_pages, 32, table, lens, [len(lens), len(lens)] + [0] * (n_pages - 2))
    got = x.take([1] * len(lens))
    assert got.tolist() == fits
    for b, n in enumerate(lens):
        for o, m in enumerate(lens):
            if o != b and got[b] and x.want.table[b][1] == x.want.table[o][1]:
                assert n >= m, (b, o)


def test_taken_pages_stay_until_the_row_is_shortened(P):
    x = filled(P, np.random.default_rng(1), 2, 6, 32, 20, [30, 10])
    x.take([100, 0])
    x.take([100, 5])
    assert not x.want.moves
    x.grow([3, 0])
    x.select()


def test_bad_cells_rows_and_counts(P):
    x = filled(P, np.random.default_rng(1), 4, 3, 32, 20, [40, 40, 40, 40])
    got = x.take([100, 1, 1, -5])                # no room in the table
    assert got.tolist() == [0, 1, 1, 1]
    x.want.table[1, 1] = -1                      # the last page is missing
    x.table[1, 1] = -1
    x.want.table[2, 1] = 20                      # outside the pool
    x.table[2, 1] = 20
    assert x.take([1, 1, 1, 1]).tolist() == [1, 0, 0, 1]
    x.select([0, 1, 2, 9])
    assert x.pages.status(clear=True) == P.PACE_PAGES_BAD_CELL | P.PACE_PAGES_BAD_ROW
    x.select([0, -2, 2, 3])
    assert x.pages.status(clear=True) == P.PACE_PAGES_BAD_ROW


@pytest.mark.parametrize("bits,d,Hkv,page", [(4, 64, 1, 32), (8, 128, 8, 64), (4, 256, 3, 128)])
def test_copied_pages(P, bits, d, Hkv, page):
    import torch
    n = 70
    kv = P.PaceKV(P.make_kv_config(Hkv, Hkv, d, n, 1, bits=bits, page_tokens=page))
    view = kv.pages()
    assert view.shape == (n, P.pace_kv_tile_bytes(kv.cfg) * Hkv * page // 32)
    view.copy_(torch.randint(0, 256, view.shape, dtype=torch.uint8, device="cuda"))
    want = view.clone()
    src, dst = list(range(0, 60, 2)), list(range(1, 60, 2))
    P.pace_kv_copy_pages(kv.handle, ints(torch, src), ints(torch, dst), ints(torch, [20]))
    want[dst[:20]] = want[src[:20]]
    assert torch.equal(view, want)
    P.pace_kv_copy_pages(kv.handle, ints(torch, src), ints(torch, dst))
    want[dst] = want[src]
    assert torch.equal(view, want) and kv.status() == 0
    for count in (-3, 1000):
        P.pace_kv_copy_pages(kv.handle, ints(torch, [60, 70, -1, 61]), ints(torch, [69, 1, 2, 70]), ints(torch, [count]))
        if count > 0:
            want[69] = want[60]
            assert kv.status(clear=True) == P.PACE_KV_BAD_PAGE
        assert torch.equal(view, want) and kv.status() == 0


def test_pool_past_32_bits(P):
    import torch
    kv = P.PaceKV(P.make_kv_config(16, 16, 256, 600, 1, bits=8, page_tokens=1024))      # 8.5 MB a page, 5 GB
    view = kv.pages()
    view[3].copy_(torch.randint(0, 256, view[3].shape, dtype=torch.uint8, device="cuda"))
    P.pace_kv_copy_pages(kv.handle, ints(torch, [3]), ints(torch, [599]))
    assert torch.equal(view[599], view[3]) and not view[598].any()


def test_on_another_stream_and_in_a_graph(P):
    import torch
    rng = np.random.default_rng(5)
    x = filled(P, rng, 8, 6, 32, 60, rng.integers(1, 100, 8))
    start = [t.clone() for t in (x.table, x.lens, x.pages.refs)]
    src, n_new, fits = ints(torch, [0, 0, 2, 2, 4, 4, 6, -1]), ints(torch, [3] * 8), torch.zeros(8, dtype=torch.int32, device="cuda")

    def step():
        x.pages.select(x.table, x.lens, src)
        x.pages.take(x.table, x.lens, n_new, fits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    x.want.select(src.cpu().numpy())
    want, _ = x.want.take([3] * 8)
    x.same(moves=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t, s in zip((x.table, x.lens, x.pages.refs), start):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        x.same(moves=True)


def test_refusals(P):
    import torch
    pages = P.PacePages(10, 32, 2)
    table, lens = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(P.PaceError, match="max_batch"):
        pages.select(torch.full((3, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"))
    for call in (lambda: pages.select(table.long(), lens), lambda: pages.select(table[:, ::2], lens), lambda: pages.select(table, lens[:1]),
                 lambda: pages.take(table, lens, lens, lens[:1]), lambda: pages.take(table, None, lens, lens), lambda: pages.compact(lens),
                 lambda: pages.select(table, lens, src=lens.cpu())):
        with pytest.raises(ValueError):
            call()
    empty = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    pages.n_moves.fill_(5)
    pages.take(empty, lens[:0], lens[:0], lens[:0])
    assert int(pages.n_moves) == 0
    pages.select(empty, lens[:0])
    pages.compact(empty)
    assert pages.status() == 0
