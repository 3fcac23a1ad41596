"""mla_kv_evict: the heaviest keys of every request, copied in order into new pages.

The refusals run on the CPU; the GPU cases compare indices, masses, lengths and rows with a
plain selection on the host.  Everything is a choice or a copy, so everything is exact.
"""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
OK = dict(pool=1 << 30, num_pages=64, page=64, dtype=0, table=1 << 8, max_pages=4, lens=1 << 9, keep=1 << 10, mass=1 << 16,
          mass_stride=256, dst=1 << 11, max_dst=4, batch=2, sink=0, recent=0, max_seq=256, max_keep=128, kept=1 << 20,
          kept_stride=128, new_lens=1 << 12, mass_out=1 << 18, out_stride=128)


def _raw(mla, **kw):
    a = dict(OK, **kw)
    return mla.lib.mla_kv_evict(*[a[k] for k in OK], None)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(num_pages=0), dict(max_pages=0), dict(max_dst=0), dict(sink=-1), dict(recent=-1), dict(max_seq=-1),
    dict(max_keep=-1), dict(dtype=9), dict(pool=None), dict(table=None), dict(lens=None), dict(keep=None), dict(mass=None),
    dict(dst=None), dict(kept=None), dict(new_lens=None), dict(mass_out=None), dict(pool=8), dict(mass=2), dict(kept=2),
    dict(mass_stride=255), dict(kept_stride=127), dict(out_stride=100), dict(mass_out=1 << 16), dict(mass_out=(1 << 16) + 2044),
    dict(new_lens=1 << 9), dict(new_lens=(1 << 10) + 4)])
def test_invalid_arguments_are_refused(mla, bad):
    assert _raw(mla, **bad) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(page=4), dict(page=96), dict(page=512), dict(dtype=3), dict(batch=65536),
                                 dict(max_seq=(1 << 24) + 1, mass_stride=1 << 25)])
def test_unsupported_shapes_are_refused(mla, bad):
    assert _raw(mla, **bad) == mla.MLA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(mla):
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)
    with pytest.raises(mla.MlaError) as e:
        mla.kv_evict(z(2, 8, 576, dtype=torch.bfloat16), i(1, 1), i(1), i(1), z(1, 8), i(1, 1), 0, 0, 8, 8)
    assert e.value.code == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ reference
def chosen(mass, L, keep, sink, recent):
    """Kept indices by definition: a stable sort of the middle keys, heaviest first."""
    K = min(keep, L)
    s = min(sink, K)
    r = min(recent, K - s)
    w = [(-math.inf, 1) if math.isnan(x) else (x, 0) for x in mass[s:L - r].tolist()]
    order = sorted(range(len(w)), key=lambda i: (w[i][1], -w[i][0], i))  # NaN last
    return list(range(s)) + sorted(s + i for i in order[:K - s - r]) + list(range(L - r, L))


def run(mla, lens, keeps, mass, page, kind, sink, recent, seed=0, share=False, max_keep=None, stride=None):
    """One call on a random pool; every output against the definition."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [max(1, -(-n // page)) for n in lens]
    dst = [max(1, -(-min(k, n) // page)) for n, k in zip(lens, keeps)]
    pages = sum(need) + sum(dst) + 1
    perm = torch.randperm(pages, generator=g).int()
    table = torch.zeros(B, max(need) + 1, dtype=torch.int32)
    dtab = torch.zeros(B, max(dst), dtype=torch.int32)
    at = 0
    for t, counts in ((table, need), (dtab, dst)):
        for b, n in enumerate(counts):
            t[b, :n] = perm[at:at + n]
            at += n
    if share:  # a prefix that every request reads through the same pages
        table[:, :min(need)] = table[0, :min(need)]
    dt, dtype = {"bf16": (mla.MLA_KV_BF16, torch.bfloat16), "e4m3": (mla.MLA_KV_E4M3, torch.uint8),
                 "int8": (mla.MLA_KV_INT8, torch.int8)}[kind]
    pool = torch.randint(0, 120, (pages, page, 576), generator=g).to(dtype)
    max_seq = max(max(lens), 1)
    max_keep = max(max(min(k, n) for n, k in zip(lens, keeps)), 1) if max_keep is None else max_keep
    d = "cuda"
    pd = pool.to(d)
    kept = torch.full((B, max_keep + 3), -7, dtype=torch.int32, device=d)
    mass_out = torch.full((B, max_keep + 5), -7.0, device=d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    _, new_lens, _ = mla.kv_evict(pd, table.to(d), i32(lens), i32(keeps), mass.to(d), dtab.to(d), sink, recent, max_seq, max_keep,
                                  dt, kept=kept, mass_out=mass_out)
    assert mla.get_status() == mla.MLA_OK
    want = pool.view(-1, 576).clone()
    for b in range(B):
        ids = chosen(mass[b], lens[b], keeps[b], sink, recent)
        K = len(ids)
        assert int(new_lens[b]) == K
        assert kept[b, :K].tolist() == ids and (kept[b, K:] == -7).all()
        i = torch.arange(K)
        ids = torch.tensor(ids, dtype=torch.long)
        got, ref = mass_out[b, :K].cpu(), mass[b, ids]
        assert torch.equal(got.view(torch.int32), ref.view(torch.int32)) and (mass_out[b, K:] == -7).all()
        want[dtab[b].long()[i // page] * page + i % page] = pool.view(-1, 576)[table[b].long()[ids // page] * page + ids % page]
    assert torch.equal(pd.cpu().view(-1, 576), want)
    return kept


def masses(B, n, seed, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    m = torch.randn(B, n, generator=g).mul(2.0).exp()
    if kind == "ties":
        m = torch.randint(0, 4, (B, n), generator=g).float()
    elif kind == "equal":
        m = torch.full((B, n), 0.25)
    elif kind == "special":
        m = torch.randn(B, n, generator=g)
        pick = torch.randint(0, 9, (B, n), generator=g)
        for v, x in ((0, math.nan), (1, math.inf), (2, -math.inf), (3, 0.0), (4, -0.0), (5, 1e-45), (6, -1e-45)):
            m[pick == v] = x
    return m


CASES = [  # lens, keeps, page, kind, sink, recent, masses
    ([1], [1], 64, "bf16", 0, 0, "heavy"),
    ([1], [0], 64, "bf16", 4, 4, "heavy"),
    ([0, 5], [3, 2], 8, "e4m3", 1, 1, "heavy"),
    ([40, 7, 63], [40, 100, 62], 16, "int8", 2, 3, "ties"),
    ([300, 129, 65], [1, 2, 3], 32, "bf16", 1, 5, "special"),
    ([1000, 777], [500, 13], 64, "bf16", 4, 9, "ties"),
    ([1025, 1024, 1023], [600, 1, 1000], 128, "e4m3", 0, 64, "equal"),
    ([2049, 4000], [2048, 1999], 256, "int8", 600, 700, "special"),
    ([9000, 30000, 17], [4000, 29999, 17], 64, "bf16", 4, 128, "heavy"),
    ([11264, 9999], [5000, 9000], 64, "e4m3", 4, 30, "ties"),      # the longest that one CTA selects
    ([11265, 300], [5000, 299], 64, "e4m3", 4, 30, "special"),
    ([70001], [33333], 64, "e4m3", 0, 0, "ties"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keeps,page,kind,sink,recent,m", CASES)
def test_against_the_definition(mla, lens, keeps, page, kind, sink, recent, m):
    run(mla, lens, keeps, masses(len(lens), max(max(lens), 1) + 2, sum(lens), m), page, kind, sink, recent, seed=sum(keeps))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keeps,max_keep", [([5, 70], [0, 0], 0), ([0, 0], [3, 0], 0), ([0], [9], 4)])
def test_nothing_kept(mla, lens, keeps, max_keep):
    """Bounds of zero: empty outputs, and masses that nobody reads."""
    d = "cuda"
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    pool = torch.randint(0, 99, (8, 64, 576)).bfloat16().to(d)
    was = pool.clone()
    B = len(lens)
    table, dst = torch.zeros(B, 2, dtype=torch.int32, device=d), torch.full((B, 1), 7, dtype=torch.int32, device=d)
    kept, new_lens, mass_out = mla.kv_evict(pool, table, i32(lens), i32(keeps), torch.rand(B, max(lens), device=d), dst, 2, 2,
                                            max(lens), max_keep, new_lens=i32([-3] * B))
    assert mla.get_status() == mla.MLA_OK
    assert new_lens.tolist() == [0] * B and kept.shape == mass_out.shape == (B, max_keep) and torch.equal(pool, was)


@pytest.mark.gpu
def test_a_long_request_among_many_short_ones(mla):
    lens = [150000] + [64 + 3 * i for i in range(40)]
    run(mla, lens, [70000] + [50] * 40, masses(41, 150000, 5), 64, "e4m3", 4, 32)


@pytest.mark.gpu
def test_shared_source_pages_stay_whole(mla):
    run(mla, [200, 256, 190], [70, 80, 90], masses(3, 256, 8), 64, "bf16", 4, 16, share=True)


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported_and_skipped(mla):
    d = "cuda"
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    pool = torch.randint(0, 99, (8, 8, 576)).bfloat16().to(d)
    was = pool.clone()
    mass = torch.rand(4, 16, device=d)
    table, dst = i32([[0, 1], [2, 3], [0, 1], [0, 1]]), i32([[4], [5], [6], [7]])
    # beyond max_seq_len, a negative keep, more kept than the destination row holds, fine
    for lens, keeps, good in (([17, 4, 16, 3], [4, -1, 9, 2], 3), ([-1, 16, 16, 8], [4, 9, 12, 8], 3)):
        kept, new_lens, _ = mla.kv_evict(pool, table, i32(lens), i32(keeps), mass, dst, 1, 1, 16, 12, new_lens=i32([-3] * 4))
        assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
        assert new_lens.tolist() == [-3, -3, -3, keeps[good]] and (kept[:3] == 0).all()
        assert torch.equal(pool[:7], was[:7])
        pool.copy_(was)
    # a page outside the pool: its rows are not copied, the others are
    for t, dt in ((i32([[0, 8]]), i32([[4]])), (i32([[0, -1]]), i32([[4]]))):
        mla.kv_evict(pool, t, i32([16]), i32([8]), torch.arange(16., device=d)[None].neg().abs(), dt, 4, 4, 16, 8)
        assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
        assert torch.equal(pool[4, :4], was[0, :4]) and torch.equal(pool[4, 4:], was[4, 4:])
        pool.copy_(was)
    mla.kv_evict(pool, i32([[0, 1]]), i32([16]), i32([8]), mass[:1], i32([[9]]), 4, 4, 16, 8)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG and torch.equal(pool, was)


@pytest.mark.gpu
@pytest.mark.parametrize("L,keep,m", [(393_216 + 5, 100_001, "ties"), (700_003, 699_000, "special")])
def test_requests_longer_than_shared_memory_holds(mla, L, keep, m):
    """More masses than a cluster keeps in shared memory; logical pages that share a few real ones."""
    P, real, d = 64, 50, "cuda"
    g = torch.Generator().manual_seed(L)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    n_dst = -(-keep // P)
    pool = torch.randint(0, 120, (real + n_dst, P, 576), generator=g, dtype=torch.uint8).to(d)
    table = torch.randint(0, real, (1, -(-L // P)), generator=g).int()
    mass = masses(1, L, 3, m)
    kept, new_lens, mass_out = mla.kv_evict(pool, table.to(d), i32([L]), i32([keep]), mass.to(d),
                                            torch.arange(real, real + n_dst, dtype=torch.int32, device=d)[None], 4, 100, L, keep,
                                            mla.MLA_KV_E4M3)
    assert mla.get_status() == mla.MLA_OK
    ids = torch.tensor(chosen(mass[0], L, keep, 4, 100))
    assert int(new_lens) == keep and torch.equal(kept[0].cpu().long(), ids)
    assert torch.equal(mass_out[0].cpu().view(torch.int32), mass[0, ids].view(torch.int32))
    ids = ids.to(d)
    src = pool[table.to(d)[0].long()[ids // P], ids % P]
    assert torch.equal(pool[real:].view(-1, 576)[:keep], src)


@pytest.mark.gpu
def test_captured_with_new_lengths_and_masses(mla):
    """A captured call follows the device's lengths and masses at replay."""
    d = "cuda"
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    pool = torch.randint(0, 99, (64, 16, 576)).bfloat16().to(d)
    table, dst = torch.arange(40, dtype=torch.int32, device=d).view(2, 20), torch.arange(40, 60, dtype=torch.int32, device=d).view(2, 10)
    lens, keeps, mass = i32([10, 20]), i32([5, 5]), torch.rand(2, 320, device=d)
    side = torch.cuda.Stream()
    kept, new_lens, mass_out = i32([[0] * 160] * 2), i32([0, 0]), torch.zeros(2, 160, device=d)
    call = lambda: mla.kv_evict(pool, table, lens, keeps, mass, dst, 2, 3, 320, 160, kept=kept, new_lens=new_lens, mass_out=mass_out)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for new, keep in (([320, 17], [160, 30]), ([100, 310], [99, 150])):
        lens.copy_(i32(new))
        keeps.copy_(i32(keep))
        mass.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            ids = chosen(mass[b].cpu(), new[b], keep[b], 2, 3)
            assert kept[b, :len(ids)].tolist() == ids and int(new_lens[b]) == len(ids)
            i = torch.arange(len(ids), device=d)
            ids = torch.tensor(ids, device=d)
            assert torch.equal(pool[dst[b].long()[i // 16], i % 16], pool[table[b].long()[ids // 16], ids % 16])
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_mass_and_mass_out_as_column_ranges_of_one_buffer(mla):
    """Rows that lie side by side do not overlap; one column in common does."""
    d = "cuda"
    B, L, keep, P = 3, 200, 90, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
    both = torch.rand(B, 320, device=d)
    was = both.clone()
    mass = both[:, 10:210].cpu()
    pool = torch.randint(0, 99, (20, P, 576)).bfloat16().to(d)
    table, dst = torch.arange(12, dtype=torch.int32, device=d).view(B, 4), torch.arange(12, 18, dtype=torch.int32, device=d).view(B, 2)
    kept, new_lens = torch.zeros(B, keep, dtype=torch.int32, device=d), i32([0] * B)
    lens, keeps = i32([L, 150, 97]), i32([keep, 60, 89])
    stream = torch.cuda.current_stream().cuda_stream

    def call(at, out_stride=320, max_keep=keep):
        return mla.lib.mla_kv_evict(pool.data_ptr(), 20, P, 0, table.data_ptr(), 4, lens.data_ptr(), keeps.data_ptr(),
                                    both.data_ptr() + 40, 320, dst.data_ptr(), 2, B, 2, 3, L, max_keep, kept.data_ptr(), keep,
                                    new_lens.data_ptr(), both.data_ptr() + 4 * at, out_stride, stream)

    for at, stride in ((209, 320), (10 - keep + 1 + 320, 320), (0, 320), (60, 320), (210, 319)):
        assert call(at, stride) == mla.MLA_ERR_INVALID_ARG
    assert torch.equal(both, was)
    assert call(210) == mla.MLA_OK and mla.get_status() == mla.MLA_OK
    for b, (n, k) in enumerate(((L, keep), (150, 60), (97, 89))):
        ids = chosen(mass[b], n, k, 2, 3)
        assert kept[b, :k].tolist() == ids
        assert torch.equal(both[b, 210:210 + k].cpu(), mass[b, ids])
        assert torch.equal(both[b, 210 + k:], was[b, 210 + k:]) and torch.equal(both[b, :210], was[b, :210])


def test_every_overlap_of_mass_and_mass_out_is_refused(mla):
    """All offsets (elements) at which some row of one touches a row of the other, strides equal or not."""
    base = 1 << 16
    for B, stride, n, keep in ((1, 256, 100, 60), (2, 128, 100, 60), (3, 161, 100, 60), (3, 160, 160, 160)):
        rows = {b * stride + i for b in range(B) for i in range(n)}
        for out_stride in (stride, stride + 3):
            for off in range(-keep - (B - 1) * out_stride - 2, B * stride + 2):
                out = {off + b * out_stride + i for b in range(B) for i in (0, keep - 1)}
                out |= {off + b * out_stride + i for b in range(B) for i in range(0, keep, 7)}
                if rows & out:
                    assert _raw(mla, batch=B, mass=base, mass_stride=stride, max_seq=n, max_keep=keep, kept_stride=keep,
                                kept=1 << 24, mass_out=base + 4 * off, out_stride=out_stride) == mla.MLA_ERR_INVALID_ARG
