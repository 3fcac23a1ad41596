"""A 4-bit cache kept on the device, as a server runs it: append prompts, fork them, append trees of drafts, attend,
take the rejected drafts and a finished request back, gather, evict, compact, and go on there.

The test keeps each request's rows for itself (the bytes that were in the pool right after they were appended), so a row
written, shared, copied or moved to the wrong place shows: attention is compared with 64-bit arithmetic over these
rows, as in test_fp4_decode.py, and gathered rows with their values rounded once.
"""
import pytest
import torch

import fp4_rows
from test_fp4_decode import KV_SCALE, SCALE, chain, check, random_tree, reference
from test_kv_append import table as angle_table

pytestmark = pytest.mark.gpu
T, H, SLOTS, WIDTH = 4, 16, 8, 64
D = "cuda"


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=D)


class Server:
    def __init__(self, mla, page, pages):
        self.mla, self.page = mla, page
        self.pool = torch.zeros(pages, page, 336, dtype=torch.uint8, device=D)
        self.table, self.lens = ints([[-1] * WIDTH] * SLOTS), ints([0] * SLOTS)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=D)
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(page)).tolist()
        self.rows = [torch.zeros(0, 336, dtype=torch.uint8) for _ in range(SLOTS)]
        self.cs = angle_table(4096).to(D)

    def take(self):
        p = self.free.pop()
        self.refs[p] = 1
        return p

    def append(self, g, counts, q=None):
        """counts: {slot: new tokens}."""
        where, pos = [], []
        for s, n in counts.items():
            L = len(self.rows[s])
            for j in range(L, L + n):
                if j % self.page == 0:
                    self.table[s, j // self.page] = self.take()
                where.append((s, j))
                pos.append(j)
        s, j = torch.tensor(where, device=D).T
        slots = self.table[s, j // self.page].long() * self.page + j % self.page
        kv = (torch.randn(len(where), 576, generator=g) * 2).bfloat16().to(D)
        w = (1 + 0.1 * torch.randn(512, generator=g)).bfloat16().to(D)
        out = self.mla.kv_append(q, kv, ints(pos), slots, self.cs, self.pool, w, kv_dtype=self.mla.MLA_KV_FP4, kv_scale=KV_SCALE)
        got = self.pool.view(-1, 336)[slots].cpu()
        at = 0
        for s, n in counts.items():
            self.rows[s] = torch.cat([self.rows[s], got[at:at + n]])
            self.lens[s] = len(self.rows[s])
            at += n
        return out

    def fork(self, parents, children):
        new = [self.free.pop() if len(self.rows[p]) % self.page else -1 for p in parents]
        self.mla.page_fork(self.pool, self.table, self.lens, self.refs, ints(parents), ints(children), ints(new), self.mla.MLA_KV_FP4)
        for p, c in zip(parents, children):
            self.rows[c] = self.rows[p]

    def shrink(self, keep):
        """keep: {slot: length}."""
        freed, n = self.mla.page_free(self.table, self.lens, self.refs, ints(list(keep)), ints(list(keep.values())), self.page)
        back = freed[:int(n)].tolist()
        assert not set(back) & set(self.free)
        self.free += back
        for s, k in keep.items():
            self.rows[s] = self.rows[s][:k]

    def compact(self):
        live = int(self.mla.page_compact(self.pool, self.table, self.lens, self.refs, self.mla.MLA_KV_FP4))
        assert live == len(self.refs) - len(self.free)
        self.free = list(range(len(self.refs) - 1, live - 1, -1))

    def live(self):
        return [s for s in range(SLOTS) if len(self.rows[s])]

    def attend(self, g, words=None):
        """The last T tokens of every live request over its cache; checked."""
        s = self.live()
        lens = [len(self.rows[i]) for i in s]
        q = torch.randn(len(s), T, H, 576, generator=g).bfloat16()
        table, sl = self.table[s].contiguous(), self.lens[s].contiguous()
        assert sl.tolist() == lens
        make = self.mla.decode_plan if words is None else self.mla.decode_tree_plan
        plan = make(lens, T, H, self.page, WIDTH, len(self.refs), self.mla.MLA_KV_FP4)
        if words is None:
            out, lse = self.mla.decode(plan, q.to(D), self.pool, table, sl, SCALE, KV_SCALE)
        else:
            out, lse = self.mla.decode_tree(plan, q.to(D), self.pool, table, sl, words.to(D), SCALE, KV_SCALE)
        flat = torch.cat([self.rows[i] for i in s])[:, None]
        where, at = torch.zeros(len(s), max(lens), dtype=torch.int32), 0
        for i, n in enumerate(lens):
            where[i, :n] = torch.arange(at, at + n)
            at += n
        check(out, lse, reference(q, flat, where, lens, chain(len(s), T) if words is None else words))

    def gather(self):
        s = self.live()
        lens = [len(self.rows[i]) for i in s]
        cu = [sum(lens[:i]) for i in range(len(s) + 1)]
        out = torch.zeros(cu[-1], 576, dtype=torch.bfloat16, device=D)
        self.mla.kv_gather(self.pool, self.table[s].contiguous(), ints(cu), out, kv_dtype=self.mla.MLA_KV_FP4, kv_scale=KV_SCALE)
        want = (fp4_rows.values(torch.cat([self.rows[i] for i in s])).float() * torch.tensor(KV_SCALE)).bfloat16()
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("page", [8, 64])
def test_append_fork_attend_free_gather_evict_compact(mla, page):
    g = torch.Generator().manual_seed(11)
    s = Server(mla, page, 4000 // page)
    s.append(g, {0: 6 * page + 3, 1: 2 * page, 2: 5})
    s.fork([0, 0, 1], [3, 4, 5])
    s.gather()
    for step in range(3):
        s.append(g, {i: T for i in s.live()})
        words = random_tree(g, len(s.live()), T)
        s.attend(g, words if step != 1 else None)
        # each request keeps some of its drafts; in the middle one sample ends and another one is forked from the first
        s.shrink({i: len(s.rows[i]) - (i + step) % (T + 1) for i in s.live()})
        if step == 1:
            s.shrink({4: 0, 1: 0})
            s.gather()
            s.fork([3, 3], [4, 6])
            s.compact()
        s.gather()
    # the longest request is cut to a third by the weights of its keys, in new pages
    n, keep = len(s.rows[0]), len(s.rows[0]) // 3
    mass = torch.rand(1, n, generator=g).to(D)
    fresh = [s.take() for _ in range(-(-keep // page))]
    kept, new_lens, _ = mla.kv_evict(s.pool, s.table[:1].contiguous(), s.lens[:1].contiguous(), ints([keep]), mass, ints([fresh]), 2, 2, n, keep,
                                     kv_dtype=mla.MLA_KV_FP4)
    ids = kept[0, :int(new_lens)].long().cpu()
    assert len(ids) == keep
    rows = s.rows[0][ids]
    s.shrink({0: 0})
    s.table[0, :len(fresh)] = ints(fresh)
    s.lens[0], s.rows[0] = keep, rows
    s.compact()
    s.gather()
    s.append(g, {i: T for i in s.live()})
    s.attend(g, random_tree(g, len(s.live()), T))
    s.gather()
    s.shrink({i: 0 for i in s.live()})
    assert sorted(s.free) == list(range(len(s.refs))) and not s.refs.any() and mla.get_status() == mla.MLA_OK


def test_a_step_in_one_graph(mla):
    """Fork, append on the child, attention of both, the child taken back and a compaction, captured together and replayed
    with other inputs: the same bytes as the calls made one by one."""
    page, L = 16, 5 * 16 + 14
    g = torch.Generator().manual_seed(2)
    s = Server(mla, page, 64)
    s.append(g, {0: L})
    tail = [s.take(), s.take()]  # the rest of the child's drafts: its partial page is a copy, the next page here
    kv = torch.zeros(T, 576, dtype=torch.bfloat16, device=D)
    q = torch.zeros(2, T, H, 576, dtype=torch.bfloat16, device=D)
    parents, children, new = ints([0]), ints([1]), ints([s.free.pop()])
    zero, one = ints([1]), ints([0])
    pos, slots = ints(range(L, L + T)), torch.zeros(T, dtype=torch.int64, device=D)
    plan = mla.decode_plan([L, L + T], T, H, page, WIDTH, 64, mla.MLA_KV_FP4)
    ws, cws = mla.workspace_for(plan, D), mla.page_compact_workspace_for(64, D)
    out, lse = torch.zeros(2, T, H, 512, dtype=torch.bfloat16, device=D), torch.zeros(2, T, H, device=D)
    freed, count, live = torch.zeros(64, dtype=torch.int32, device=D), ints([0]), ints([0])
    j = torch.arange(L, L + T, device=D)

    def step():
        mla.page_fork(s.pool, s.table, s.lens, s.refs, parents, children, new, mla.MLA_KV_FP4)
        s.table[1, L // page + 1].fill_(tail[0])
        slots.copy_(s.table[1].index_select(0, j // page).long() * page + j % page)
        mla.kv_append(None, kv, pos, slots, s.cs, s.pool, kv_dtype=mla.MLA_KV_FP4, kv_scale=KV_SCALE)
        s.lens[1:2].add_(T)
        mla.decode(plan, q, s.pool, s.table[:2], s.lens[:2], SCALE, KV_SCALE, out=out, lse=lse, workspace=ws)
        mla.page_free(s.table, s.lens, s.refs, zero, one, page, freed, count)
        mla.page_compact(s.pool, s.table, s.lens, s.refs, mla.MLA_KV_FP4, live, cws)

    state = [s.pool, s.table, s.lens, s.refs, freed]
    start = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in range(3):
        h = torch.Generator().manual_seed(seed)
        kv.copy_(torch.randn(kv.shape, generator=h).bfloat16())
        q.copy_(torch.randn(q.shape, generator=h).bfloat16())
        results = []
        for go in (graph.replay, step):
            for t, v in zip(state, start):
                t.copy_(v)
            go()
            torch.cuda.synchronize()
            results.append([t.clone() for t in state] + [out.clone(), lse.clone(), count.clone(), live.clone()])
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert int(count) == 2 and int(live) == L // page + 2 and torch.isfinite(lse).all()
    assert mla.get_status() == mla.MLA_OK


def test_calls_on_two_streams_at_once(mla):
    """Attention over one pool on two streams, each with its workspace, while a third forks, frees and compacts another cache:
    the same bytes as one after the other."""
    from test_fp4_decode import make
    from test_pages import Cache
    calls = []
    for seed, (lens, T_, H_) in enumerate((([5000, 777, 64], 1, 16), ([3000, 2500], 3, 16))):
        q, pool, table = make(lens, T_, H_, 16, seed)
        plan = mla.decode_plan(lens, T_, H_, 16, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
        args = (plan, q.to(D), pool.to(D), table.to(D), ints(lens), SCALE, KV_SCALE)
        calls.append((args, mla.workspace_for(plan, D), mla.decode(*args)))
    c = Cache(7, [100, 333, 64, 7], 16, spare=12, slots=8)
    start = [t.cuda() for t in (c.pool, c.table, c.lens, c.refs)]
    now = [t.clone() for t in start]
    new, freed, n = ints(c.unused[:2]), torch.zeros_like(now[3]), ints([0])
    pages_ws, live = mla.page_compact_workspace_for(len(c.refs), D), ints([0])
    p, ch, sl, keep = ints([1, 3]), ints([4, 5]), ints([1, 5]), ints([160, 2])
    want = None
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(30):
        got = []
        for s, (args, ws, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(mla.decode(*args, workspace=ws))
        with torch.cuda.stream(streams[2]):
            for t, v in zip(now, start):
                t.copy_(v)
            mla.page_fork(now[0], now[1], now[2], now[3], p, ch, new, mla.MLA_KV_FP4)
            mla.page_free(now[1], now[2], now[3], sl, keep, 16, freed, n)
            mla.page_compact(now[0], now[1], now[2], now[3], mla.MLA_KV_FP4, live, pages_ws)
        torch.cuda.synchronize()
        for (out, lse), (_, _, ref) in zip(got, calls):
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        if want is None:
            assert not c.fork([1, 3], [4, 5], c.unused[:2])
            want, bad = c.free([1, 5], [160, 2])
            assert not bad and c.compact() == (int(live), False)
        assert freed[:int(n)].tolist() == want
        for t, v in zip(now, (c.pool, c.table, c.lens, c.refs)):
            assert torch.equal(t.cpu(), v)
    assert mla.get_status() == mla.MLA_OK
