"""The cache's operators in one loop, as a server runs them: append the prefix, then per step
append a tree of drafts, attend over it, weigh the keys; evict into new pages; go on there.

Each step is compared with 64-bit arithmetic over rows that the test keeps for itself (the
bytes that were in the pool right after they were appended), so a row written, read, kept or
moved to the wrong place shows.  Tolerances as in test_decode_tree.py and test_key_mass.py.
"""
import math

import pytest
import torch

import test_decode_tree as tree
import test_key_mass as weight
from test_kv_append import EPS, check_bf16, check_codes, reference as append_reference, table as angle_table
from test_kv_evict import chosen

pytestmark = pytest.mark.gpu

T, H, PAGE = 5, 16, 16
D = "cuda"


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


class Cache:
    """A pool with a page list per request, and the rows that should be in it."""

    def __init__(self, mla, kind, B, pages):
        self.mla, self.kind, self.B = mla, kind, B
        self.dtype = {"bf16": torch.bfloat16, "e4m3": torch.uint8, "int8": torch.int8}[kind]
        self.scale = {"bf16": 1.0, "e4m3": 6.0 / 448, "int8": 5.0 / 127}[kind]
        self.pool = torch.zeros(pages, PAGE, 576, dtype=self.dtype, device=D)
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
        self.pages = [[] for _ in range(B)]
        self.rows = [torch.zeros(0, 576, dtype=self.dtype) for _ in range(B)]
        self.cs = angle_table(4096)

    def lens(self):
        return [r.shape[0] for r in self.rows]

    def table(self, pages=None):
        pages = self.pages if pages is None else pages
        t = torch.zeros(self.B, max(len(p) for p in pages), dtype=torch.int32)
        for b, p in enumerate(pages):
            t[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        return t

    def append(self, g, counts, positions, q=None):
        """Append counts[b] new tokens to every request (one padded token at the end)."""
        slots = []
        for b, n in enumerate(counts):
            for j in range(len(self.rows[b]), len(self.rows[b]) + n):
                if j // PAGE == len(self.pages[b]):
                    self.pages[b].append(self.free.pop())
                slots.append(self.pages[b][j // PAGE] * PAGE + j % PAGE)
        n = sum(counts)
        kv = torch.randn(n + 1, 576, generator=g).bfloat16() * 2
        w = (1 + 0.1 * torch.randn(512, generator=g)).bfloat16()
        pos = torch.tensor(positions + [0], dtype=torch.int32)
        slot = torch.tensor(slots + [-1])
        kd = tree.KINDS[self.kind]
        qd = None if q is None else torch.cat([q, q[:1]]).to(D)
        out = self.mla.kv_append(qd, kv.to(D), pos.to(D), slot.to(D), self.cs.to(D), self.pool, w.to(D), eps=EPS, kv_dtype=kd,
                                 kv_scale=self.scale)
        got = self.pool.cpu().view(-1, 576)[slot[:n]]
        qr, kr = append_reference(q, kv[:n], pos[:n], self.cs, None, w, True)
        if self.kind == "bf16":
            check_bf16(got, kr)
        else:
            check_codes(got, kr, self.scale, self.kind)
        at = 0
        for b, c in enumerate(counts):
            self.rows[b] = torch.cat([self.rows[b], got[at:at + c]])
            at += c
        if q is not None:
            check_bf16(out[:n].cpu(), qr)
            return out[:n]

    def values(self):
        """The kept rows as one page per row, in 64 bits, with a table that names them."""
        f = {"bf16": lambda r: r.double(), "e4m3": lambda r: r.view(torch.float8_e4m3fn).double(), "int8": lambda r: r.double()}
        flat = torch.cat(self.rows)
        t = torch.zeros(self.B, max(self.lens()), dtype=torch.int32)
        at = 0
        for b, n in enumerate(self.lens()):
            t[b, :n] = torch.arange(at, at + n)
            at += n
        return f[self.kind](flat)[:, None, :] * self.scale, t


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_append_attend_weigh_evict_and_go_on(mla, kind):
    g = torch.Generator().manual_seed(7)
    B = 3
    c = Cache(mla, kind, B, 400)
    prefix = [400, 37, 900]
    c.append(g, prefix, [j for n in prefix for j in range(n)])
    mass = torch.zeros(B, 2048, device=D)
    seen = torch.zeros(B, 2048)  # what mass should hold
    here = list(prefix)          # next position of every request
    for step in range(3):
        words = tree.random_tree(g, B, T)
        depth = [[bin(int(words[b, t]) & ((1 << T) - 1)).count("1") - 1 for t in range(T)] for b in range(B)]
        q = torch.randn(B * T, H, 576, generator=g).bfloat16()
        rotated = c.append(g, [T] * B, [here[b] + depth[b][t] for b in range(B) for t in range(T)], q)
        lens = c.lens()
        kd = tree.KINDS[kind]
        tab = c.table()
        plan = mla.decode_tree_plan(lens, T, H, PAGE, tab.shape[1], c.pool.shape[0], kd)
        sl = torch.tensor(lens, dtype=torch.int32, device=D)
        qd = rotated.view(B, T, H, 576)
        out, lse = mla.decode_tree(plan, qd, c.pool, tab.to(D), sl, words.to(D), tree.SCALE, c.scale)
        val, vt = c.values()
        tree.check(out, lse, tree.reference(qd.cpu(), val, vt, lens, words), kind)
        mla.key_mass(plan, qd, c.pool, tab.to(D), sl, lse, mass, tree.SCALE, c.scale, tree_mask=words.to(D), decay=0.5)
        seen, tol = weight.reference(qd.cpu(), val, vt, lens, words, lse.cpu(), seen, 0.5, kind)
        assert ((mass.cpu().double() - seen).abs() <= tol).all()
        seen = mass.cpu()
        here = [h + 2 for h in here]
        if step == 1:
            # shrink every request; the middle one keeps everything
            keeps = [150, 1000, 333]
            kept_n = [min(k, n) for k, n in zip(keeps, lens)]
            new = [[c.free.pop() for _ in range(-(-n // PAGE))] for n in kept_n]
            mass2 = torch.zeros_like(mass)
            kept, new_lens, _ = mla.kv_evict(c.pool, tab.to(D), sl, torch.tensor(keeps, dtype=torch.int32, device=D), mass,
                                             c.table(new).to(D), 4, 20, max(lens), max(kept_n), kv_dtype=kd, mass_out=mass2)
            for b in range(B):
                ids = torch.tensor(chosen(seen[b], lens[b], keeps[b], 4, 20))
                assert kept[b, :len(ids)].tolist() == ids.tolist() and int(new_lens[b]) == len(ids)
                c.rows[b] = c.rows[b][ids]
                seen[b] = torch.cat([seen[b, ids], torch.zeros(2048 - len(ids))])
            c.free += [p for pages in c.pages for p in pages]  # the old pages are free again
            c.pages, mass = new, mass2
            assert torch.equal(mass.cpu(), seen)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_whole_step_in_one_graph(mla, kind):
    """Append, attention, weights and eviction captured together, replayed with other inputs: the
    same bytes as the calls made one by one, on a stream of their own."""
    g = torch.Generator().manual_seed(3)
    B, L = 2, 700
    kd = tree.KINDS[kind]
    c = Cache(mla, kind, B, 200)
    c.append(g, [L] * B, list(range(L)) * B)
    for b in range(B):
        while len(c.pages[b]) * PAGE < L + T:
            c.pages[b].append(c.free.pop())
    tab = c.table().to(D)
    new = [[c.free.pop() for _ in range(13)] for _ in range(B)]
    dst = c.table(new).to(D)
    lens = [L + T] * B
    plan = mla.decode_tree_plan(lens, T, H, PAGE, tab.shape[1], c.pool.shape[0], kd)
    ws = mla.workspace_for(plan, D)
    sl = torch.tensor(lens, dtype=torch.int32, device=D)
    keeps = torch.tensor([200, 190], dtype=torch.int32, device=D)
    slots = torch.tensor([c.pages[b][j // PAGE] * PAGE + j % PAGE for b in range(B) for j in range(L, L + T)], device=D)
    q, kv = (torch.randn(B * T, n, generator=g).bfloat16().to(D) for n in (H * 576, 576))
    pos = torch.arange(L, L + B * T, dtype=torch.int32, device=D)
    cs = c.cs.to(D)
    words = tree.random_tree(g, B, T).to(D)
    mass = torch.zeros(B, 1024, device=D)
    outs = [torch.zeros(B * T, H, 576, dtype=torch.bfloat16, device=D), torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device=D),
            torch.zeros(B, T, H, device=D), torch.zeros(B, 200, dtype=torch.int32, device=D), torch.zeros(B, dtype=torch.int32, device=D),
            torch.zeros(B, 200, device=D)]

    def step():
        mla.kv_append(q.view(B * T, H, 576), kv, pos, slots, cs, c.pool, kv_dtype=kd, kv_scale=c.scale, q_out=outs[0])
        qd = outs[0].view(B, T, H, 576)
        mla.decode_tree(plan, qd, c.pool, tab, sl, words, tree.SCALE, c.scale, out=outs[1], lse=outs[2], workspace=ws)
        mla.key_mass(plan, qd, c.pool, tab, sl, outs[2], mass, tree.SCALE, c.scale, tree_mask=words, decay=0.75)
        mla.kv_evict(c.pool, tab, sl, keeps, mass, dst, 4, 16, L + T, 200, kv_dtype=kd, kept=outs[3], new_lens=outs[4], mass_out=outs[5])

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
        q.copy_(torch.randn(q.shape, generator=h).bfloat16())
        kv.copy_(torch.randn(kv.shape, generator=h).bfloat16())
        words.copy_(tree.random_tree(h, B, T))
        pool, m = c.pool.clone(), mass.clone()
        graph.replay()
        torch.cuda.synchronize()
        first = [o.clone() for o in outs] + [mass.clone(), c.pool.clone()]
        c.pool.copy_(pool)
        mass.copy_(m)
        for o in outs:
            o.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(first, outs + [mass, c.pool]):
            assert torch.equal(a, b)
    assert mla.get_status() == mla.MLA_OK


def test_a_given_stream_owns_what_a_call_allocates(mla):
    """Calls on a given stream while the current one is busy with memory it has just given back:
    nothing of the results waits for the current stream or is overwritten by it."""
    g = torch.Generator().manual_seed(5)
    B, L = 2, 300
    c = Cache(mla, "bf16", B, 100)
    c.append(g, [L] * B, list(range(L)) * B)
    tab, sl = c.table().to(D), torch.tensor([L] * B, dtype=torch.int32, device=D)
    plan = mla.decode_tree_plan([L] * B, T, H, PAGE, tab.shape[1], c.pool.shape[0], 0)
    q = torch.randn(B, T, H, 576, generator=g).bfloat16().to(D)
    words = tree.random_tree(g, B, T).to(D)
    pos, cs = torch.arange(B * T, dtype=torch.int32, device=D), c.cs.to(D)
    keeps, mass = torch.tensor([90, 50], dtype=torch.int32, device=D), torch.rand(B, L, generator=g).to(D)
    dst = torch.tensor([[c.free.pop() for _ in range(6)] for _ in range(B)], dtype=torch.int32, device=D)

    def calls(stream):
        yield lambda: mla.decode_tree(plan, q, c.pool, tab, sl, words, tree.SCALE, stream=stream)
        yield lambda: (mla.kv_append(q.view(B * T, H, 576), None, pos, None, cs, None, stream=stream),)
        yield lambda: mla.kv_evict(c.pool, tab, sl, keeps, mass, dst, 4, 16, L, 90, stream=stream)

    want = [[o.clone() for o in call()] for call in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for call, outs in zip(calls(side), want):
        busy = [torch.empty_like(o) for o in outs]
        torch.cuda._sleep(20_000_000)  # (some 10 ms)
        for o in busy:
            o.fill_(7)
        del o, busy
        got = call()
        side.synchronize()
        got = [o.clone() for o in got]
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(mla, kind):
    """Append, weights and eviction at the end of a pool of over 2^32 bytes."""
    pages, B, L = (9_000_000_000 if kind == "bf16" else 4_700_000_000) // (PAGE * 576 * (2 if kind == "bf16" else 1)), 1, 100
    g = torch.Generator().manual_seed(2)
    c = Cache(mla, kind, B, 8)
    c.pool = torch.zeros(pages, PAGE, 576, dtype=c.dtype, device=D)
    kd = tree.KINDS[kind]
    own = list(range(pages - 7, pages))
    kv = torch.randn(L, 576, generator=g).bfloat16()
    pos = torch.arange(L, dtype=torch.int32)
    slots = torch.tensor([own[j // PAGE] * PAGE + j % PAGE for j in range(L)])
    mla.kv_append(None, kv.to(D), pos.to(D), slots.to(D), c.cs.to(D), c.pool, kv_dtype=kd, kv_scale=c.scale)
    rows = c.pool.view(-1, 576)[slots.to(D)].cpu()
    want = append_reference(None, kv, pos, c.cs, None, None, True)[1]
    if kind == "bf16":
        check_bf16(rows, want)
    else:
        check_codes(rows, want, c.scale, kind)
    c.rows = [rows]
    q = torch.randn(B, 1, H, 576, generator=g).bfloat16()
    tab = torch.tensor([own], dtype=torch.int32, device=D)
    sl = torch.tensor([L], dtype=torch.int32, device=D)
    plan = mla.decode_plan([L], 1, H, PAGE, 7, pages, kd)
    val, vt = c.values()
    lse = weight.true_lse(q, val, vt, [L], None)
    mass = torch.zeros(1, L, device=D)
    mla.key_mass(plan, q.to(D), c.pool, tab, sl, lse.to(D), mass, tree.SCALE, c.scale, decay=0.0)
    new, tol = weight.reference(q, val, vt, [L], None, lse, torch.zeros(1, L), 0.0, kind)
    assert ((mass.cpu().double() - new).abs() <= tol).all()
    dst = torch.arange(pages - 12, pages - 7, dtype=torch.int32, device=D)[None]
    kept, _, _ = mla.kv_evict(c.pool, tab, sl, torch.tensor([70], dtype=torch.int32, device=D), mass, dst, 2, 5, L, 70, kv_dtype=kd)
    ids = chosen(mass[0].cpu(), L, 70, 2, 5)
    assert kept[0].tolist() == ids
    assert torch.equal(c.pool[pages - 12:pages - 7].view(-1, 576)[:70].cpu(), rows[torch.tensor(ids)])
    assert mla.get_status() == mla.MLA_OK
