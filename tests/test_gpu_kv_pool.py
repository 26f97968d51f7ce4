"""The page pool on the GPU: tables, counts, lengths, codes and scales equal to the plain reference (tests/poolref.py)."""
import numpy as np
import pytest

import poolref
import quantized_weight_mat_gb300 as pq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


def ints(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Gpu:
    """The pool on the GPU beside its reference."""

    def __init__(self, ref):
        import torch
        self.ref = ref
        self.refs, self.table, self.len = ints(ref.refs), ints(ref.table), ints(ref.len)
        up = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.codes = [[up(c) for c in layer] for layer in ref.codes]
        self.scales = [[up(c) for c in layer] for layer in ref.scales]
        self.pool = pq.pq_kv_pool(self.refs, self.table, self.len, ref.n_pages, ref.page, ref.n_seq, ref.table_ld)
        self.layers = pq.pq_kv_layers([
            pq.pq_kv_cache(*codes, *scales, self.table, self.len, ref.n_pages, n_kv, ref.page, d, ref.n_seq, ref.table_ld)
            for codes, scales, (n_kv, d) in zip(self.codes, self.scales, ref.layers)]) if ref.layers else None
        n = pq.pq_kv_pool_ws_bytes(self.pool)
        assert n > 0
        self.ws, self.n_ws = torch.full((n + 64,), 0x55, dtype=torch.uint8, device="cuda"), n
        self.status = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        self.moved = torch.full((ref.n_pages + 1,), -9, dtype=torch.int32, device="cuda")

    def fork(self, frm, to, tokens=None):
        self.ref.fork(frm, to, tokens)
        pq.pq_kv_fork(self.pool, len(to), ints(frm), ints(to), ints(tokens), self.ws, self.n_ws)
        self.check()

    def free(self, seq=None, begin=None, end=None, n=None):
        self.ref.free(seq, begin, end, n)
        n = n if n is not None else len(seq) if seq is not None else self.ref.n_seq
        pq.pq_kv_free(self.pool, n, ints(seq), ints(begin), ints(end))
        self.check()

    def reserve(self, new):
        want = self.ref.reserve(new)
        pq.pq_kv_reserve(self.pool, self.layers, ints(new), self.status, self.ws, self.n_ws)
        assert self.status.tolist() == [*want, -7, -7]
        self.check()
        return want

    def compact(self, told=True):
        moved, used = self.ref.compact()
        pq.pq_kv_compact(self.pool, self.layers, self.moved if told else None, self.status[2:], self.ws, self.n_ws)
        assert self.status.tolist()[2:] == [used, -7]
        self.status.fill_(-7)
        if told:
            assert np.array_equal(self.moved.cpu().numpy(), np.append(moved, -9))
        self.check()

    def check(self):
        r = self.ref
        assert np.array_equal(self.table.cpu().numpy(), r.table)
        assert np.array_equal(self.refs.cpu().numpy(), r.refs)
        assert np.array_equal(self.len.cpu().numpy(), r.len)
        for got, want in zip(self.codes + self.scales, r.codes + r.scales):
            for a, b in zip(got, want):
                assert np.array_equal(a.cpu().numpy(), b)
        assert bool((self.ws[self.n_ws:] == 0x55).all())


def make(n_seq, table_ld, n_pages, page, lens=None, layers=((2, 32), (1, 64)), room=0, seed=1):
    r = poolref.Pool(n_seq, table_ld, n_pages, page, list(layers), seed)
    if lens is not None:
        r.fill(lens, seed, room)
    return Gpu(r)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_beam_search(page):
    # parents with several children, children that swap places, dead beams
    n = 6
    lens = [3 * page + 5, 0, 0, 0, 0, 0]
    g = make(n, 8, 60, page, lens)
    g.fork([0] * 6, list(range(6)))
    rng = np.random.default_rng(page)
    for step in range(12):
        assert g.reserve([1] * n) == (0, 0)
        g.ref.check()
        # the tokens are there now, and what was appended differs from beam to beam
        for s in range(n):
            p, slot = g.ref.table[s, g.ref.len[s] // page], g.ref.len[s] % page
            for codes, up in zip(g.ref.codes, g.codes):
                for a, b in zip(codes, up):
                    a[p, :, slot] = s + step
                    b[p, :, slot] = s + step
        g.ref.len += 1
        g.len += 1
        g.fork(rng.integers(0, n, n), list(range(n)))
        g.ref.check()


@pytest.mark.parametrize("layers", [[(8, 128)], [(1, 16)], [(3, 80), (1, 256), (4, 64)], [(1, 16)] * 70, []])
def test_layers_of_any_shape(layers):
    g = make(5, 6, 40, 32, [70, 0, 64, 33, 0], layers)
    g.fork([0, 3, 3], [1, 4, 2])
    if not layers:
        g.reserve([40, 40, 40, 40, 40])
    else:
        assert g.reserve([1, 2, 40, 33, 5]) == (0, 0)
    g.ref.check()
    g.free([0, 2])
    g.compact()
    g.ref.check()


def test_a_prompt_shared_by_its_first_tokens():
    g = make(6, 8, 60, 16, [100, 0, 0, 0, 0, 50])
    # a whole number of pages, part of one, nothing, more than there is, below 0
    g.fork([0, 0, 0, 0, 5], [1, 2, 3, 4, 5], [64, 37, 0, 1000, 17])
    g.ref.check()
    assert g.ref.len.tolist() == [100, 64, 37, 0, 100, 17]
    assert g.reserve([1, 1, 1, 1, 1, 1]) == (0, 0)
    g.fork([0], [1], [-5])
    g.ref.check()


def test_pairs_that_do_not_count():
    g = make(5, 6, 40, 16, [40, 20, 0, 0, 0])
    top = 2 ** 31 - 1
    g.fork([-1, 0, 1, 5, 0], [2, 2, 2, 3, top])      # the first pair names no sequence, so the second has 2
    g.ref.check()
    assert g.ref.len.tolist() == [40, 20, 40, 0, 0]
    g.fork([], [])


def test_swap_and_cut_in_place():
    g = make(4, 6, 40, 16, [90, 20, 33, 0], room=10)
    g.fork([1, 0, 2, 3], [0, 1, 2, 2], [1000, 1000, 17, 5])
    assert g.ref.len.tolist() == [20, 90, 17, 0]
    g.ref.check()


def test_who_keeps_a_shared_page():
    g = make(6, 6, 40, 16, [20, 0, 0, 0, 0, 0])
    g.fork([0, 0, 0], [2, 3, 5])
    page = int(g.ref.table[0, 1])
    g.reserve([0, 0, 1, 1, 0, 0])                     # two of four write: both copy
    assert int(g.ref.refs[page]) == 2
    g.reserve([1, 0, 0, 0, 0, 1])                     # both that are left write: the lowest keeps it
    assert int(g.ref.table[0, 1]) == page and int(g.ref.refs[page]) == 1
    g.ref.check()
    g.reserve([1, 0, 1, 1, 0, 1])                     # nothing is lacking any more
    g.ref.check()


def test_shared_room_behind_the_tokens():
    # a sequence taken back into pages that others hold too: blocks behind its tokens are replaced, nothing is copied there
    g = make(3, 8, 40, 16, [100, 0, 0])
    g.fork([0, 0], [1, 2])
    for t, r in ((g.len, g.ref.len),):
        t[1] = 20
        r[1] = 20
    assert g.reserve([0, 60, 0]) == (0, 0)
    g.ref.check()


@pytest.mark.parametrize("new", [[200, 0, 0, 0], [100, 0, 30, 0], [0, 1000, 0, 0], [0, 2 ** 31 - 1, 0, 2 ** 31 - 1], [100, 1000, 100, 50]])
def test_not_enough_pages_or_too_short_rows(new):
    g = make(4, 12, 14, 16, [40, 20, 17, 0])
    g.fork([0], [3])
    want = g.reserve(new)
    assert want != (0, 0)
    g.ref.check()
    assert g.reserve([1, 1, 1, 1]) == (0, 0)          # a smaller wish is met after that


def test_the_last_free_page():
    g = make(2, 4, 4, 16, [32, 16])
    assert g.reserve([16, 0]) == (0, 0) and g.reserve([16, 1]) == (1, 0)
    assert g.reserve([16, 0]) == (0, 0)


def test_free_in_every_way():
    g = make(8, 10, 90, 16, [100, 90, 80, 70, 60, 50, 0, 160], room=16)
    g.free([1])                                       # a whole sequence, its room too
    g.free([0, 9, -1, 0], [37, 0, 0, 5])              # back to 37 tokens; numbers out of range; twice the same
    assert g.ref.len[0] == 37
    g.free([2, 3], None, [40, 64])                    # what a window has left: whole pages before the end
    g.free([4], [20], [50])                           # a hole
    g.free([5, 6], [10, 0], [10, 0])                  # empty ranges
    assert g.ref.len.tolist() == [37, 0, 80, 70, 60, 50, 0, 160]
    g.free([5, 7], [17, 33], [50, 1000])              # up to the end
    g.free([0], [500])                                # room only
    g.free([4], [-20], [-3])
    g.ref.check()
    g.free(n=3)
    g.free()
    assert not g.ref.refs.any()
    g.free([], n=0)


def test_entries_that_name_no_page():
    r = poolref.Pool(4, 6, 30, 16, [(2, 32)], 1)
    r.fill([90, 60, 33, 0], 1)
    r.refs[r.table[0, 2]] = r.refs[r.table[1, 1]] = 0
    r.table[0, 2], r.table[1, 1], r.table[2, 5], r.table[3, 0] = -5, 30, 2 ** 31 - 1, -2 ** 31
    r.len[3] = -4
    g = Gpu(r)
    g.fork([0, 3], [3, 2])
    g.ref.check()
    assert g.reserve([3, 10, 20, 1]) == (0, 0)
    g.ref.check()
    g.compact()
    g.free([0, 1])
    g.compact(told=False)


def test_pages_held_beside_the_tables():
    # the caller's own hold: shared as far as writers go, kept by a compaction
    g = make(3, 6, 30, 16, [40, 0, 20])
    page = int(g.ref.table[0, 2])
    g.ref.refs[page] += 1
    g.refs[page] += 1
    g.reserve([1, 0, 0])
    assert int(g.ref.table[0, 2]) != page and int(g.ref.refs[page]) == 1
    g.free([0])
    g.compact()


@pytest.mark.parametrize("n_pages", [1, 2, 3, 5, 4095, 16384, 16385, 32769, 70001, 131075])
def test_pools_of_any_size(n_pages):
    # scanned in one piece and in several, with the ends inside a thread's four
    rng = np.random.default_rng(n_pages)
    n_seq, width = 9, max(1, n_pages // 6)
    lens = [int(x) for x in rng.integers(1, 16 * max(1, n_pages // 12) + 1, 8)] + [0]
    if n_pages < 9:
        lens = [1 if s < n_pages - 1 else 0 for s in range(9)]
    g = make(n_seq, width, n_pages, 16, lens, [(1, 16)])
    g.compact()
    g.ref.check()
    if n_pages > 9:
        g.free([1, 4])
        new = [0, int(g.ref.len[2]) // 2 + 1, 0, 0, 16 * (n_pages // 12), 0, 0, 0, 5]
        g.reserve(new)
        g.fork([0, 4], [8, 1])
        g.reserve([1] * 9)
        g.ref.check()
        g.compact()
    if n_pages == 1:
        assert g.reserve([1] + [0] * 8) == (0, 0)


@pytest.mark.parametrize("n_pages", [16384, 40000])
def test_requests_of_many_blocks(n_pages):
    # more blocks than a CTA's threads hold at a time, shared pages among the first and the last of them
    width = 11000
    g = make(3, width, n_pages, 16, [16 * 9000 + 5, 0, 7], [(1, 16)])
    g.fork([0, 2], [1, 2])
    for t, r in ((g.len, g.ref.len),):              # taken back into pages that both hold
        t[0] = 3
        r[0] = 3
    short, narrow = g.reserve([16 * 9000, 16, 0])
    assert narrow == 0 and (short > 0) == (n_pages == 16384)
    g.free([1])
    assert g.reserve([16 * 9000, 16, 0]) == (0, 0)
    g.reserve([16 * 20, 16 * 500, 16 * 1000])
    g.ref.check()
    g.compact()


@pytest.mark.parametrize("n_seq", [1, 255, 256, 1000, 9001])
def test_many_sequences(n_seq):
    rng = np.random.default_rng(n_seq)
    lens = [int(x) for x in rng.integers(0, 60, n_seq)]
    g = make(n_seq, 6, 8 * n_seq + 9, 16, lens, [(1, 16)])
    g.fork(rng.integers(-1, n_seq + 1, n_seq), rng.integers(-1, n_seq + 1, n_seq), rng.integers(-3, 70, n_seq))
    g.ref.check()
    g.reserve(rng.integers(-2, 20, n_seq))
    g.ref.check()
    g.free(rng.integers(-1, n_seq + 1, n_seq), rng.integers(-5, 50, n_seq), rng.integers(-5, 80, n_seq))
    g.ref.check()
    g.compact()
    g.ref.check()


def test_steps_in_a_graph():
    import torch
    g = make(4, 12, 48, 16, [30, 0, 0, 0], [(2, 64)] * 3)
    frm, to, new = ints([0, 0, 0, 0]), ints([0, 1, 2, 3]), ints([1, 1, 1, 1])

    def step():
        pq.pq_kv_fork(g.pool, 4, frm, to, None, g.ws, g.n_ws)
        pq.pq_kv_reserve(g.pool, g.layers, new, g.status, g.ws, g.n_ws)
        g.len.add_(1)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(1)
    for _ in range(40):
        f = rng.integers(0, 4, 4)
        frm.copy_(ints(f))
        graph.replay()
        g.ref.fork(f, [0, 1, 2, 3])
        assert g.ref.reserve([1] * 4) == (0, 0)
        g.ref.len += 1
        g.check()
    g.ref.check()


def test_give_back_and_compact_in_a_graph():
    import torch
    g = make(6, 12, 80, 16, [100, 150, 60, 0, 90, 10], [(2, 64)] * 2, room=20)
    g.fork([0], [3], [33])
    seq, begin, end = ints([1, 3, 5]), ints([0, 0, 0]), ints([0, 0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq.pq_kv_free(g.pool, 3, seq, begin, end)
        pq.pq_kv_compact(g.pool, g.layers, g.moved, g.status[2:], g.ws, g.n_ws)
    for b, e in (([20, 0, 3], [150, 16, 3]), ([0, 17, 0], [16, 40, 10]), ([0, 0, 0], [1000, 1000, 1000])):
        begin.copy_(ints(b))
        end.copy_(ints(e))
        graph.replay()
        g.ref.free([1, 3, 5], b, e)
        moved, used = g.ref.compact()
        assert int(g.status[2]) == used and np.array_equal(g.moved.cpu().numpy(), np.append(moved, -9))
        g.check()
    g.ref.check()


def test_lists_of_views_and_layers_apart():
    # lists that are slices of others, layers that lie in no order
    import torch
    r = poolref.Pool(5, 6, 40, 16, [(2, 32), (1, 64), (2, 32)], 3)
    r.fill([50, 20, 0, 0, 33], 3)
    g = Gpu(r)
    order = [2, 0, 1]
    layers = pq.pq_kv_layers([g.layers[i] for i in order])
    both = ints([7, 0, 4, 2, 3, 9])
    g.ref.fork([0, 4], [2, 3])
    pq.pq_kv_fork(g.pool, 2, both[1:], both[3:], None, g.ws, g.n_ws)
    new = ints([5, 1, 0, 0, 1, 1, 5])
    assert g.ref.reserve([1, 0, 0, 1, 1]) == (0, 0)
    pq.pq_kv_reserve(g.pool, layers, new[1:], g.status, g.ws, g.n_ws)
    torch.cuda.synchronize()
    g.check()


def test_offsets_past_32_bits():
    import torch
    n_kv, page, d = 8, 64, 128
    n_pages = 2 ** 32 // (n_kv * page * d) + 64
    k = torch.zeros(n_pages, n_kv, page, d, dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = torch.zeros(n_pages, n_kv, device="cuda"), torch.zeros(n_pages, n_kv, device="cuda")
    top = n_pages - 3
    for x in (k, v):
        x[top] = torch.randint(-127, 128, (n_kv, page, d), dtype=torch.int8, device="cuda")
    ks[top], vs[top] = 1.5, 2.5
    was = [x[top].clone() for x in (k, v, ks, vs)]
    # all pages but the last two are in use, the one before them by two sequences
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[top], refs[top + 1:] = 2, 0
    table = torch.tensor([[top, -1], [top, -1]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    pool = pq.pq_kv_pool(refs, table, ln, n_pages, page, 2, 2)
    layers = pq.pq_kv_layers([pq.pq_kv_cache(k, v, ks, vs, table, ln, n_pages, n_kv, page, d, 2, 2)])
    ws = torch.empty(pq.pq_kv_pool_ws_bytes(pool), dtype=torch.uint8, device="cuda")
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    pq.pq_kv_reserve(pool, layers, ints([0, 1]), status, ws, ws.numel())
    assert status.tolist() == [0, 0, 0] and table.tolist() == [[top, -1], [top + 1, -1]]
    for x, y in zip((k, v), was):
        assert torch.equal(x[top + 1, :, :40], y[:, :40]) and not x[top + 1, :, 40:].any()
    assert torch.equal(ks[top + 1], was[2]) and torch.equal(vs[top + 1], was[3])
    # the others are given back, and both move to the bottom
    refs[:top] = 0
    pq.pq_kv_compact(pool, layers, None, status[2:], ws, ws.numel())
    assert status.tolist() == [0, 0, 2] and table.tolist() == [[0, -1], [1, -1]]
    assert all(torch.equal(x[0], y) for x, y in zip((k, v, ks, vs), was))
    assert refs[:2].tolist() == [1, 1] and not refs[2:].any()


def test_two_pools_on_two_streams():
    import torch
    gs = [make(5, 8, 60, 32, [100, 0, 0, 200, 0], seed=s) for s in (1, 2)]
    lists = [ints([0, 3]), ints([1, 4]), ints([5, 5, 0, 9, 9])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(20):
        for g, st in zip(gs, streams):
            pq.pq_kv_fork(g.pool, 2, lists[0], lists[1], None, g.ws, g.n_ws, stream=st)
            pq.pq_kv_reserve(g.pool, g.layers, lists[2], g.status, g.ws, g.n_ws, stream=st)
            pq.pq_kv_compact(g.pool, g.layers, None, g.status[2:], g.ws, g.n_ws, stream=st)
    torch.cuda.synchronize()
    for g in gs:
        for _ in range(20):
            g.ref.fork([0, 3], [1, 4])
            assert g.ref.reserve([5, 5, 0, 9, 9]) == (0, 0)
            g.ref.compact()
        g.check()
