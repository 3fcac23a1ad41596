"""mla_page_fork, mla_page_free and mla_page_compact against a model in plain integers; every result is equal
to the bit.  The refusals run on the CPU.
"""
import pytest
import torch

ROW = {0: (torch.bfloat16, 576), 1: (torch.float8_e4m3fn, 576), 2: (torch.int8, 576), 3: (torch.int8, 576), 4: (torch.uint8, 336)}
INT8_PAGE = 3


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
BASE = 1 << 32
FORK = dict(kv=BASE, pages=100, page=16, dtype=4, ps=None, pt=1 << 20, maxp=8, lens=1 << 21, slots=6, refs=1 << 22,
            parents=1 << 10, children=1 << 11, new=1 << 12, n=3)
FREE = dict(pt=1 << 20, maxp=8, lens=1 << 21, slots=6, page=16, refs=1 << 22, pages=100, list=1 << 10, keep=1 << 11, n=3,
            freed=1 << 23, count=1 << 12)
COMPACT = dict(kv=BASE, pages=100, page=16, dtype=4, ps=None, pt=1 << 20, maxp=8, lens=1 << 21, slots=6, refs=1 << 22,
               live=1 << 12, ws=1 << 24, ws_bytes=4096)


def _raw(fn, base, **kw):
    a = dict(base, **kw)
    return fn(*[a[k] for k in base], None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(slots=0), dict(maxp=0), dict(pages=0), dict(pages=(1 << 30) + 1), dict(dtype=5), dict(dtype=-1), dict(ps=1 << 9),
    dict(dtype=3), dict(kv=None), dict(pt=None), dict(lens=None), dict(refs=None), dict(parents=None), dict(children=None),
    dict(new=None), dict(kv=BASE + 8), dict(pt=2), dict(lens=6), dict(refs=2), dict(parents=2), dict(children=2), dict(new=2),
    dict(pt=BASE + 1024), dict(refs=(1 << 20) + 4), dict(lens=(1 << 20) + 188), dict(parents=(1 << 21) + 20), dict(new=(1 << 22) + 396),
    dict(children=(1 << 20) - 8), dict(dtype=3, ps=BASE + 64)])
def test_fork_refuses_invalid_arguments(mla, bad):
    assert _raw(mla.lib.mla_page_fork, FORK, **bad) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(slots=0), dict(maxp=0), dict(pages=0), dict(pages=(1 << 30) + 1), dict(pt=None), dict(lens=None), dict(refs=None),
    dict(list=None), dict(keep=None), dict(freed=None), dict(count=None), dict(pt=2), dict(lens=2), dict(refs=2), dict(list=2),
    dict(keep=2), dict(freed=2), dict(count=2), dict(freed=(1 << 22) + 396), dict(count=(1 << 22) + 4), dict(lens=(1 << 20) + 188),
    dict(list=(1 << 21) + 20), dict(keep=(1 << 23) - 8), dict(n=0, refs=None), dict(n=0, freed=1 << 22)])
def test_free_refuses_invalid_arguments(mla, bad):
    assert _raw(mla.lib.mla_page_free, FREE, **bad) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(slots=0), dict(maxp=0), dict(pages=0), dict(pages=(1 << 30) + 1), dict(dtype=5), dict(dtype=-1), dict(ps=1 << 9), dict(dtype=3),
    dict(kv=None), dict(pt=None), dict(lens=None), dict(refs=None), dict(live=None), dict(ws=None), dict(kv=BASE + 8), dict(pt=2),
    dict(lens=2), dict(refs=2), dict(live=2), dict(ws=(1 << 24) + 16), dict(live=(1 << 24) + 256), dict(lens=(1 << 20) + 188),
    dict(refs=BASE + 4), dict(ws=(1 << 22) + 256)])
def test_compact_refuses_invalid_arguments(mla, bad):
    assert _raw(mla.lib.mla_page_compact, COMPACT, **bad) == mla.MLA_ERR_INVALID_ARG


def test_other_refusals(mla):
    assert _raw(mla.lib.mla_page_fork, FORK, page=48) == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla.lib.mla_page_fork, FORK, n=65536, parents=1 << 26, children=1 << 27, new=1 << 28) == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla.lib.mla_page_fork, FORK, n=0, kv=None, parents=None, refs=None) == mla.MLA_OK
    assert _raw(mla.lib.mla_page_free, FREE, page=12) == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla.lib.mla_page_free, FREE, n=65536, list=1 << 26, keep=1 << 27) == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla.lib.mla_page_compact, COMPACT, page=512) == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla.lib.mla_page_compact, COMPACT, ws_bytes=256) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    need = mla.page_compact_workspace_for(1000, "cpu").numel()
    assert _raw(mla.lib.mla_page_compact, COMPACT, pages=1000, ws_bytes=need - 1, kv=BASE, ws=1 << 25) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    assert mla.lib.mla_page_compact_workspace(0, None) == mla.MLA_ERR_INVALID_ARG
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for call in (lambda: mla.page_fork(torch.zeros(4, 16, 336, dtype=torch.uint8), i(2, 2), i(2), i(4), i(1), i(1), i(1), mla.MLA_KV_FP4),
                 lambda: mla.page_free(i(2, 2), i(2), i(4), i(1), i(1), 16),
                 lambda: mla.page_compact(torch.zeros(4, 16, 336, dtype=torch.uint8), i(2, 2), i(2), i(4), mla.MLA_KV_FP4)):
        with pytest.raises(mla.MlaError) as e:  # not on a CUDA device
            call()
        assert e.value.code == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ a cache and its model
class Cache:
    """Requests of given lengths on random pages of a pool of random bytes; `prefix` tokens' full pages are shared."""

    def __init__(self, seed, lens, page, kind=4, prefix=0, spare=7, width=None, slots=None):
        g = torch.Generator().manual_seed(seed)
        self.page, self.kind = page, kind
        shared = prefix // page
        own = [max(0, -(-L // page) - shared) for L in lens]
        n = shared + sum(own) + spare
        order = torch.randperm(n, generator=g).tolist()
        width = max([-(-L // page) for L in lens] + [1]) + 2 if width is None else width
        slots = len(lens) + 3 if slots is None else slots
        self.table = torch.randint(-5, 2 ** 30, (slots, width), generator=g, dtype=torch.int32)  # unused entries mean nothing
        self.lens = torch.zeros(slots, dtype=torch.int32)
        self.refs = torch.zeros(n, dtype=torch.int32)
        common, at = order[:shared], shared
        for s, (L, k) in enumerate(zip(lens, own)):
            row = common[:-(-L // page)] if L <= shared * page else common + order[at:at + k]
            at += k
            self.lens[s] = L
            self.table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
            for x in row:
                self.refs[x] += 1
        self.unused = order[at:]
        dtype, cols = ROW[kind]
        es = torch.empty(0, dtype=dtype).element_size()
        self.pool = torch.randint(0, 256, (n, page, cols * es), generator=g, dtype=torch.uint8)
        self.scales = torch.rand(n, generator=g) if kind == INT8_PAGE else None

    def cuda(self):
        d = object.__new__(Cache)
        d.page, d.kind = self.page, self.kind
        d.pool = self.pool.cuda().view(ROW[self.kind][0])
        d.table, d.lens, d.refs = self.table.cuda(), self.lens.cuda(), self.refs.cuda()
        d.scales = None if self.scales is None else self.scales.cuda()
        return d

    def same(self, d):
        assert torch.equal(d.table.cpu(), self.table)
        assert torch.equal(d.lens.cpu(), self.lens)
        assert torch.equal(d.refs.cpu(), self.refs)
        assert torch.equal(d.pool.view(torch.uint8).cpu(), self.pool)
        assert self.scales is None or torch.equal(d.scales.cpu(), self.scales)

    # the model: as the header says, one listed slot after the other
    def fork(self, parents, children, new):
        P, bad = self.page, False
        for i, (a, c, x) in enumerate(zip(parents, children, new)):
            ok = 0 <= a < len(self.lens) and 0 <= c < len(self.lens) and c not in parents and c not in children[:i]
            L = int(self.lens[a]) if ok else 0
            ok = ok and 0 <= L <= self.table.shape[1] * P
            full, rest = (L // P, L % P) if ok else (0, 0)
            if rest:
                last = int(self.table[a, full])
                ok = 0 <= x < len(self.refs) and x not in new[:i] and int(self.refs[x]) == 0 and 0 <= last < len(self.refs)
            if not ok:
                bad = True
                continue
            for j in range(full):
                y = int(self.table[a, j])
                self.table[c, j] = y
                if 0 <= y < len(self.refs):
                    self.refs[y] += 1
                else:
                    bad = True
            self.lens[c] = L
            if rest:
                self.table[c, full], self.refs[x] = x, 1
                self.pool[x, :rest] = self.pool[last, :rest]
                if self.scales is not None:
                    self.scales[x] = self.scales[last]
        return bad

    def free(self, slots, keep):
        P, bad, gone = self.page, False, []
        for i, (s, k) in enumerate(zip(slots, keep)):
            if not (0 <= s < len(self.lens) and s not in slots[:i] and 0 <= k <= int(self.lens[s]) <= self.table.shape[1] * P):
                bad = True
                continue
            for j in range(-(-k // P), -(-int(self.lens[s]) // P)):
                x = int(self.table[s, j])
                if 0 <= x < len(self.refs) and self.refs[x] > 0:
                    self.refs[x] -= 1
                    if self.refs[x] == 0:
                        gone.append(x)
                else:
                    bad = True
            self.lens[s] = k
        return sorted(gone), bad

    def compact(self):
        n = len(self.refs)
        live = int((self.refs > 0).sum())
        holes = [x for x in range(live) if self.refs[x] <= 0]
        movers = [x for x in range(live, n) if self.refs[x] > 0]
        to, bad = dict(zip(movers, holes)), False
        for a, b in to.items():
            self.pool[b] = self.pool[a]
            self.refs[b], self.refs[a] = self.refs[a].clone(), 0
            if self.scales is not None:
                self.scales[b] = self.scales[a]
        for s in range(len(self.lens)):
            L, w = int(self.lens[s]), self.table.shape[1]
            bad |= L > w * self.page
            for j in range(min(w, max(0, -(-L // self.page)))):
                x = int(self.table[s, j])
                if not 0 <= x < n or (x >= live and x not in to):
                    bad = True
                elif x >= live:
                    self.table[s, j] = to[x]
        return live, bad


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def do_fork(mla, d, parents, children, new, **kw):
    mla.page_fork(d.pool, d.table, d.lens, d.refs, dev(parents), dev(children), dev(new), d.kind, d.scales, **kw)


def do_free(mla, d, slots, keep, freed=None, **kw):
    freed = torch.full_like(d.refs, -77) if freed is None else freed
    freed, n = mla.page_free(d.table, d.lens, d.refs, dev(slots), dev(keep), d.page, freed, torch.full((1,), -1, dtype=torch.int32, device="cuda"), **kw)
    return freed.cpu(), int(n)


def check_free(mla, c, d, slots, keep):
    gone, bad = c.free(slots, keep)
    freed, n = do_free(mla, d, slots, keep)
    assert n == len(gone) and freed[:n].tolist() == gone and (freed[n:] == -77).all()
    c.same(d)
    assert mla.get_status() == (mla.MLA_ERR_DEVICE_ARG if bad else mla.MLA_OK)


# ------------------------------------------------------------------------------ fork
@pytest.mark.gpu
@pytest.mark.parametrize("kind,page", [(0, 64), (1, 16), (2, 32), (3, 64), (4, 8), (4, 64), (4, 256), (0, 8), (1, 256)])
def test_fork(mla, kind, page):
    lens = [0, 1, page - 1, page, page + 1, 5 * page, 7 * page + page // 2 + 1, 2 * page - 1]
    c = Cache(page + kind, lens, page, kind, prefix=2 * page, spare=20, slots=20)
    parents, children = [6, 0, 6, 1, 3, 5, 4, 7, 2, 6], [8, 9, 10, 11, 12, 13, 14, 15, 17, 16]
    new = [x if lens[a] % page else -1 for a, x in zip(parents, c.unused)]
    d = c.cuda()
    assert not c.fork(parents, children, new)
    do_fork(mla, d, parents, children, new)
    c.same(d)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_fork_many_children_of_long_parents(mla):
    c = Cache(5, [16 * 3001 + 5, 16 * 1024, 37], 16, 4, spare=60, slots=63)
    children = list(range(3, 63))
    parents = [i % 3 for i in children]
    new = [x if a != 1 else -1 for a, x in zip(parents, c.unused)]
    d = c.cuda()
    assert not c.fork(parents, children, new)
    do_fork(mla, d, parents, children, new)
    c.same(d)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["parent", "child", "same child", "child a parent", "page", "page used", "page twice", "length", "negative",
                                  "last page", "full page"])
def test_fork_bad_input_leaves_that_child(mla, what):
    c = Cache(9, [37, 64, 20], 16, 3, spare=9, slots=9)
    p, ch, new = [0, 0, 2, 1], [3, 4, 5, 6], [*c.unused[:3], -1]
    if what == "parent":
        p[0], p[2] = 9, -1
    elif what == "child":
        ch[0], ch[2] = -1, 9
    elif what == "same child":
        ch[2] = 3
    elif what == "child a parent":
        ch[1] = 2
    elif what == "page":
        new[0], new[2] = -1, len(c.refs)
    elif what == "page used":
        new[1] = int(c.table[1, 0])
    elif what == "page twice":
        new[2] = new[0]
    elif what == "length":
        c.lens[0] = c.table.shape[1] * 16 + 1
    elif what == "negative":
        c.lens[2] = -1
    elif what == "last page":
        c.table[0, 2] = len(c.refs)
    elif what == "full page":
        c.table[1, 1] = -1
    d = c.cuda()
    assert c.fork(p, ch, new)
    do_fork(mla, d, p, ch, new)
    c.same(d)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG


# ------------------------------------------------------------------------------ free
@pytest.mark.gpu
@pytest.mark.parametrize("page", [8, 16, 64, 256])
def test_free(mla, page):
    lens = [0, 1, page, page + 1, 9 * page, 40 * page + 3, 3 * page - 1, 4 * page, 6 * page]
    c = Cache(page, lens, page, prefix=3 * page)
    slots, keep = [5, 0, 1, 8, 3, 4, 7], [17 * page + 1, 0, 0, 0, page + 1, 3 * page, 4 * page - 1]
    check_free(mla, c, c.cuda(), slots, keep)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 31, 257, 8193, 100003])
def test_free_lists_pages_of_pools_of_any_size(mla, pages):
    """Every page of the pool is dropped, then none."""
    c = Cache(pages, [8 * pages], 8, spare=0, slots=1)
    d = c.cuda()
    check_free(mla, c, d, [0], [0])
    check_free(mla, c, d, [], [])
    check_free(mla, c, d, [0], [0])


@pytest.mark.gpu
def test_free_shared_pages_come_free_with_their_last_reference(mla):
    """300 slots on the same 40 pages, given back in two calls."""
    c = Cache(1, [640 + 3] * 300, 16, prefix=640, slots=300)
    d = c.cuda()
    check_free(mla, c, d, list(range(0, 300, 2)), [5] * 150)
    check_free(mla, c, d, list(range(299, -1, -1)), [3 if s % 2 == 0 else 0 for s in range(299, -1, -1)])
    check_free(mla, c, d, list(range(0, 300, 2)), [0] * 150)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["slot", "twice", "keep", "negative keep", "length", "page", "no count"])
def test_free_bad_input_leaves_that_slot(mla, what):
    c = Cache(3, [100, 50, 200, 33], 16)
    slots, keep = [0, 1, 2, 3], [20, 0, 160, 1]
    if what == "slot":
        slots[1], slots[3] = -1, len(c.lens)
    elif what == "twice":
        slots[3] = 0
    elif what == "keep":
        keep[2] = 201
    elif what == "negative keep":
        keep[2] = -1
    elif what == "length":
        c.lens[2] = c.table.shape[1] * 16 + 1
    elif what == "page":
        c.table[0, 3], c.table[1, 0] = len(c.refs), -1
    elif what == "no count":
        c.table[0, 3] = c.table[1, 0]  # one count for two entries
        c.table[2, 12] = c.unused[0]
    d = c.cuda()
    check_free(mla, c, d, slots, keep)


# ------------------------------------------------------------------------------ compact
@pytest.mark.gpu
@pytest.mark.parametrize("kind,page", [(0, 64), (1, 32), (2, 16), (3, 64), (4, 8), (4, 64), (4, 256)])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.97, 1.0])
def test_compact(mla, kind, page, share):
    """Requests on random pages of a pool, `share` of which stay."""
    lens = [(7 * i * page) // 3 + i for i in range(12)]
    c = Cache(kind * 7 + page, lens, page, kind, prefix=4 * page, spare=30)
    ended = [s for s in range(12) if s >= 12 * share]
    c.free(ended, [0] * len(ended))
    d = c.cuda()
    live, bad = c.compact()
    ws = mla.page_compact_workspace_for(len(c.refs), "cuda").fill_(255)
    got = mla.page_compact(d.pool, d.table, d.lens, d.refs, kind, workspace=ws, page_scales=d.scales)
    assert int(got) == live and not bad
    c.same(d)
    assert int(mla.page_compact(d.pool, d.table, d.lens, d.refs, kind, page_scales=d.scales)) == live  # nothing left to move
    c.same(d)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 2, 255, 4099, 70001])
def test_compact_pools_of_any_size(mla, pages):
    c = Cache(pages, [8 * (pages - pages // 3)], 8, spare=pages // 3)
    d = c.cuda()
    live, bad = c.compact()
    assert int(mla.page_compact(d.pool, d.table, d.lens, d.refs, 4)) == live and not bad
    c.same(d)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "no count", "length"])
def test_compact_bad_input(mla, what):
    c = Cache(2, [100, 50, 200, 33], 16, spare=40)
    if what == "page":
        c.table[0, 3], c.table[1, 0] = len(c.refs), -1
    elif what == "no count":
        c.table[2, 1] = max(c.unused)
        c.refs[max(c.unused)] = 0
    elif what == "length":
        c.lens[2] = c.table.shape[1] * 16 + 1
        c.table[2] = c.table[2, 0]
    d = c.cuda()
    live, bad = c.compact()
    assert bad
    assert int(mla.page_compact(d.pool, d.table, d.lens, d.refs, 4)) == live
    c.same(d)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG


# ------------------------------------------------------------------------------ streams, graphs, long pools
@pytest.mark.gpu
def test_captured_and_on_another_stream(mla):
    """Fork, free and compact in one graph, replayed on fresh inputs; and plainly on a stream that is not current."""
    make = lambda seed: Cache(seed, [100, 333, 64, 7], 16, spare=12, slots=8)
    c = make(1)
    d = c.cuda()
    parents, children, new = dev([1, 0, 3]), dev([4, 5, 6]), dev([0, 0, 0])
    slots, keep = dev([1, 5, 0]), dev([160, 2, 0])
    freed, n = torch.zeros_like(d.refs), dev([0])
    live, ws = dev([0]), mla.page_compact_workspace_for(len(c.refs), "cuda")

    def go(stream=None):
        mla.page_fork(d.pool, d.table, d.lens, d.refs, parents, children, new, 4, stream=stream)
        mla.page_free(d.table, d.lens, d.refs, slots, keep, 16, freed, n, stream=stream)
        mla.page_compact(d.pool, d.table, d.lens, d.refs, 4, live, ws, stream=stream)

    def load(c):
        for to, v in ((d.pool, c.pool), (d.table, c.table), (d.lens, c.lens), (d.refs, c.refs), (new, torch.tensor(c.unused[:3]))):
            to.copy_(v)

    def check(c):
        assert not c.fork([1, 0, 3], [4, 5, 6], c.unused[:3])
        gone, bad = c.free([1, 5, 0], [160, 2, 0])
        assert not bad and freed[:int(n)].tolist() == gone
        assert c.compact() == (int(live), False)
        c.same(d)

    side = torch.cuda.Stream()
    load(c)
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    check(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for seed in (2, 3):
        c = make(seed)
        load(c)
        graph.replay()
        check(c)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_pools_beyond_32_bits(mla):
    """The last pages of a pool of 5.3 GB (4-bit rows) fork and move."""
    page, n = 256, 62000
    pool = torch.zeros(n, page, 336, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    rows = torch.randint(0, 256, (2, page, 336), generator=g, dtype=torch.uint8).cuda()
    pool[n - 3], pool[n - 2] = rows[0], rows[1]
    table, lens, refs = dev([[n - 3, n - 2], [5, 5]]), dev([page + 100, 0]), torch.zeros(n, dtype=torch.int32, device="cuda")
    refs[n - 3:n - 1] = 1
    mla.page_fork(pool, table, lens, refs, dev([0]), dev([1]), dev([n - 1]), 4)
    assert torch.equal(pool[n - 1, :100], rows[1, :100]) and not pool[n - 1, 100:].any()
    assert table.tolist() == [[n - 3, n - 2], [n - 3, n - 1]] and refs[n - 3:].tolist() == [2, 1, 1]
    assert int(mla.page_compact(pool, table, lens, refs, 4)) == 3
    assert table.tolist() == [[0, 1], [0, 2]] and refs[:3].tolist() == [2, 1, 1] and not refs[3:].any()
    assert torch.equal(pool[0], rows[0]) and torch.equal(pool[1], rows[1]) and torch.equal(pool[2, :100], rows[1, :100])
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_millions_of_pages(mla):
    """More pages than the scan keeps marks of: half of 2.3 million are given back, the others (5.9 GB with the holes) move."""
    page, n = 8, 2_300_003
    g = torch.Generator(device="cuda").manual_seed(6)
    order = torch.randperm(n, generator=g, device="cuda").int()
    kept = n // 2
    table = order.view(1, n).clone()
    lens, refs = dev([n * page]), torch.ones(n, dtype=torch.int32, device="cuda")
    freed, count = mla.page_free(table, lens, refs, dev([0]), dev([kept * page - 3]), page)
    gone = order[kept:].sort().values
    assert int(count) == n - kept and torch.equal(freed[:n - kept], gone) and not freed[n - kept:].any()
    assert int(lens) == kept * page - 3 and int(refs.sum()) == kept and not refs[gone.long()].any()
    pool = torch.empty(n, page, 336, dtype=torch.uint8, device="cuda")
    name = torch.arange(n, dtype=torch.int32, device="cuda")
    for r in (0, page - 1):  # each page's first and last bytes say which it is
        pool[:, r, (0 if r == 0 else 332):][:, :4] = name.view(torch.uint8).view(n, 4)
    assert int(mla.page_compact(pool, table, lens, refs, 4)) == kept
    now = table[0, :kept].long()
    assert torch.equal(now.sort().values, torch.arange(kept, device="cuda"))
    assert (refs[:kept] == 1).all() and not refs[kept:].any() and torch.equal(table[0, kept:], order[kept:])
    for r in (0, page - 1):
        there = pool[:, r, (0 if r == 0 else 332):][:, :4].contiguous().view(torch.int32).flatten()
        assert torch.equal(there[now], order[:kept])
    stay = order[:kept] < kept
    assert torch.equal(now[stay], order[:kept][stay].long())  # what lies below stays
    moved = now[~stay][order[:kept][~stay].argsort()]  # ascending pages take ascending holes
    assert torch.equal(moved, moved.sort().values)
    assert mla.get_status() == mla.MLA_OK
