"""mla_kv_append and mla_kv_evict on a 4-bit pool, and mla_kv_gather on every pool.

The refusals run on the CPU.  The 4-bit rows are compared to the bit with the formula in 32 bits (the mean
of squares in 64, rounded once; no product fused with a sum), since a code may hang on the last bit; the
queries within one bf16 rounding.  Gathered values are codes times a scale in 32 bits, rounded once: equal too.
"""
import math

import pytest
import torch

import fp4_rows
from test_kv_append import check_bf16, normed, rot, table

EPS = 1e-6
KV_SCALE = 6.0 / 448.0


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
GATHER = dict(kv=1 << 20, pages=10, page=64, dtype=4, scale=1.0, ps=None, pt=1 << 8, maxp=4, cu=1 << 10, B=2, total=100,
              out=1 << 28, stride=576)


def _gather(mla, **kw):
    a = dict(GATHER, **kw)
    return mla.lib.mla_kv_gather(*[a[k] for k in GATHER], None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(total=-1), dict(pages=0), dict(maxp=0), dict(dtype=5), dict(dtype=-1), dict(ps=1 << 9), dict(dtype=3),
    dict(kv=None), dict(pt=None), dict(cu=None), dict(out=None), dict(kv=8), dict(pt=2), dict(cu=6), dict(out=8),
    dict(stride=568), dict(stride=580), dict(stride=0), dict(scale=0.0), dict(scale=math.nan),
    dict(out=(1 << 20) + 1024), dict(out=(1 << 20) - 16), dict(pt=(1 << 28) + 64), dict(cu=(1 << 28) + 99 * 1152 + 1148)])
def test_gather_refuses_invalid_arguments(mla, bad):
    assert _gather(mla, **bad) == mla.MLA_ERR_INVALID_ARG


def test_gather_other_refusals(mla):
    assert _gather(mla, page=48) == mla.MLA_ERR_UNSUPPORTED
    assert _gather(mla, total=0, kv=None, out=None) == mla.MLA_OK
    z = torch.zeros
    for pool, out in ((z(4, 16, 576, dtype=torch.uint8), z(3, 576).bfloat16()), (z(4, 16, 336, dtype=torch.uint8), z(3, 576))):
        with pytest.raises(mla.MlaError) as e:
            mla.kv_gather(pool, z(1, 4).int(), z(2).int(), out, kv_dtype=mla.MLA_KV_FP4)
        assert e.value.code == mla.MLA_ERR_INVALID_ARG


def test_append_takes_a_pool_of_its_own_rows(mla):
    """A 4-bit pool's extent is 336 bytes a row: keys behind it are not inside it."""
    from test_kv_append import OK
    a = dict(OK, dtype=4, scale=0.0)
    assert mla.lib.mla_kv_append(*[a[k] for k in OK], None) == mla.MLA_ERR_INVALID_ARG
    a = dict(OK, dtype=4, kv=(1 << 30) + 64 * 336 - 16)
    assert mla.lib.mla_kv_append(*[a[k] for k in OK], None) == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ append
def rows32(kv, kv_w, pos, cos_sin, interleaved, scale):
    """The rows in units of kv_scale, as the formula says it in 32 bits."""
    x = kv.float()
    latent, r = x[:, :512], x[:, 512:]
    if kv_w is not None:
        mean = (latent.double() ** 2).mean(-1, keepdim=True).float()
        inv = torch.tensor(1.0) / torch.sqrt(mean + torch.tensor(EPS))
        latent = latent * inv * kv_w.float()
    cs = cos_sin[pos.long()]
    c, s = cs[:, :32], cs[:, 32:]
    a, b = (r[:, 0::2], r[:, 1::2]) if interleaved else (r[:, :32], r[:, 32:])
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack([u, v], -1).flatten(1) if interleaved else torch.cat([u, v], 1)
    return torch.cat([latent, r], 1) * (torch.tensor(1.0) / torch.tensor(scale))


def append(mla, n, heads, page, interleaved, norm, pad, seed, tweak=None, scale=KV_SCALE, stride=576):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(n, heads, 64, generator=g).bfloat16()
    buf = (torch.randn(n, stride, generator=g) * 2).bfloat16()
    kv = buf[:, :576]
    if tweak:
        tweak(kv)
    w = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16() if norm else None
    pos = torch.randint(0, 300, (n,), generator=g).int()
    cs = table(300)
    pages = -(-n // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:n]
    if pad:
        slots[n - pad:] = -1
    pool = torch.randint(0, 256, (pages, page, 336), generator=g).to(torch.uint8)
    d = "cuda"
    dev = pool.to(d)
    out = mla.kv_append(q.to(d), buf.to(d)[:, :576], pos.to(d), slots.to(d), cs.to(d), dev, kv_weight=None if w is None else w.to(d), eps=EPS,
                        interleaved=interleaved, kv_dtype=mla.MLA_KV_FP4, kv_scale=scale)
    assert mla.get_status() == mla.MLA_OK
    ref = pool.clone().view(-1, 336)
    real = slots >= 0
    ref[slots[real]] = fp4_rows.encode(rows32(kv, w, pos, cs, interleaved, scale))[real]
    check_bf16(out.cpu(), rot(q.double(), cs.double()[pos.long()][:, None], interleaved))
    return dev.cpu().view(-1, 336), ref


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,page,interleaved,norm,pad", [
    (1, 1, 64, True, True, 0), (2, 16, 8, False, True, 0), (5, 3, 16, True, False, 2), (33, 16, 64, False, True, 3),
    (257, 8, 128, True, True, 15), (900, 16, 64, True, True, 0), (1300, 16, 32, False, False, 7)])
def test_append_to_the_bit(mla, n, heads, page, interleaved, norm, pad):
    got, ref = append(mla, n, heads, page, interleaved, norm, pad, seed=n)
    assert torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
def test_append_values_at_the_borders(mla, norm):
    """Zeros and minus zeros, ties of every code and of the exponent, values that saturate or vanish, and what is not finite."""
    def tweak(kv):
        kv[0] = 0
        kv[1, ::3] = -0.0
        if norm:
            return
        for e in range(12):  # (scale 1: the values are the codes' own)
            kv[2 + e, :512] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.125]).repeat(32) * 2.0 ** (e - 5)
        kv[14, :512] = torch.tensor([7.0, 0.5, -1.0, 3.0] * 4).repeat(32)     # rounds within the exponent
        kv[15, :512] = torch.tensor([7.03125, 0.5, -1.0, 3.0] * 4).repeat(32)  # just past it
        kv[16, :512] = 1e30
        kv[17, :512] = -1e-30
        kv[18, :512:5] = math.inf
        kv[19, 1:512:7] = -math.inf
        kv[20, 2:512:9] = math.nan
        kv[21, 512:] = 1e9
    got, ref = append(mla, 40, 2, 16, True, norm, 0, seed=5, tweak=tweak, scale=KV_SCALE if norm else 1.0)
    assert torch.equal(got[:, :272], ref[:, :272])
    # (a rotated NaN may carry either sign)
    a, b = got[:, 272:].contiguous().view(torch.float8_e4m3fn).float(), ref[:, 272:].contiguous().view(torch.float8_e4m3fn).float()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.gpu
def test_append_strided_keys_and_bad_places(mla):
    got, ref = append(mla, 21, 4, 16, False, True, 0, seed=8, stride=640)
    assert torch.equal(got, ref)
    d = "cuda"
    kv = torch.randn(4, 576, device=d).bfloat16()
    pool = torch.full((2, 16, 336), 9, dtype=torch.uint8, device=d)
    pos = torch.tensor([0, 1000, 2, -1], dtype=torch.int32, device=d)
    slots = torch.tensor([32, 1, 5, 6], device=d)
    mla.kv_append(None, kv, pos, slots, table(300).to(d), pool, kv_dtype=mla.MLA_KV_FP4, kv_scale=KV_SCALE)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    flat = pool.view(-1, 336)
    assert (flat[5] != 9).any() and (flat[[i for i in range(32) if i != 5]] == 9).all()


# ------------------------------------------------------------------------------ gather
KINDS = {"bf16": 0, "e4m3": 1, "int8": 2, "int8page": 3, "fp4": 4}


def any_pool(kind, pages, page, g):
    """A pool, its scales, and its values in 32 bits."""
    x = torch.randn(pages, page, 576, generator=g)
    if kind == "bf16":
        p = x.bfloat16()
        return p, 1.0, None, p.float()
    if kind == "e4m3":
        p = (x / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
        return p.view(torch.uint8), KV_SCALE, None, p.float() * torch.tensor(KV_SCALE)
    if kind == "fp4":
        p = fp4_rows.encode((x / KV_SCALE).view(-1, 576)).view(pages, page, 336)
        return p, KV_SCALE, None, fp4_rows.values(p).float() * torch.tensor(KV_SCALE)
    p = (x * 25).round().clamp(-127, 127).to(torch.int8)
    if kind == "int8":
        return p, 0.04, None, p.float() * torch.tensor(0.04)
    s = torch.rand(pages, generator=g) * 0.05
    return p, 0.05, s, p.float() * s[:, None, None]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("page,lens", [(64, [1]), (16, [5, 0, 0, 130, 1, 64, 17]), (8, [100] * 70), (256, [0, 300, 513]), (32, [0, 0])])
def test_gather(mla, kind, page, lens):
    g = torch.Generator().manual_seed(page + len(lens))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g).int()
    tab = torch.full((len(lens), max(need) + 1), -3, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tab[b, :n] = perm[at:at + n]
        at += n
    pool, scale, ps, val = any_pool(kind, pages, page, g)
    cu = torch.tensor([0] + lens).cumsum(0).int()
    total = int(cu[-1])
    d = "cuda"
    buf = torch.full((total + 3, 640), 7.0, device=d).bfloat16()
    out = buf[:, :576]
    mla.kv_gather(pool.to(d), tab.to(d), cu.to(d), out, kv_dtype=KINDS[kind], kv_scale=scale, page_scales=None if ps is None else ps.to(d))
    assert mla.get_status() == mla.MLA_OK
    ref = torch.full((total + 3, 576), 7.0)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        ref[cu[b]:cu[b + 1]] = val[tab[b].long()[j // page], j % page]
    assert torch.equal(out.cpu(), ref.bfloat16()) and (buf[:, 576:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_gather_reports_bad_pages_and_lengths(mla, kind):
    g = torch.Generator().manual_seed(3)
    pool, scale, _, val = any_pool(kind, 6, 16, g)
    tab = torch.tensor([[0, 99, 2], [3, 4, -1]], dtype=torch.int32)
    d = "cuda"

    def run(cu, rows):
        out = torch.full((rows, 576), 7.0, device=d).bfloat16()
        mla.kv_gather(pool.to(d), tab.to(d), torch.tensor(cu, dtype=torch.int32, device=d), out, kv_dtype=KINDS[kind], kv_scale=scale)
        assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
        return out.cpu().float()
    out = run([0, 40, 72], 80)
    v = val.bfloat16().float()
    assert torch.equal(out[:16], v[0]) and (out[16:32] == 0).all() and torch.equal(out[32:40], v[2, :8])
    assert torch.equal(out[40:72], torch.cat([v[3], v[4]])) and (out[72:] == 7).all()
    out = run([0, 10, 70], 70)  # the second request is longer than its table row: 48 of its 60 rows
    assert torch.equal(out[10:42], torch.cat([v[3], v[4]])) and (out[42:58] == 0).all() and (out[58:] == 7).all()
    out = run([0, 10, 70], 30)  # beyond total_rows
    assert torch.equal(out[:10], v[0, :10]) and torch.equal(out[10:30], torch.cat([v[3], v[4]])[:20])
    out = run([-5, 10, 20], 20)
    assert torch.equal(out[:10], v[0, 5:15]) and torch.equal(out[10:], v[3, :10])


# ------------------------------------------------------------------------------ eviction
@pytest.mark.gpu
def test_evict_copies_4_bit_rows(mla):
    g = torch.Generator().manual_seed(1)
    lens, keeps, page = [100, 33, 700], [40, 50, 333], 16
    need = [-(-n // page) for n in lens]
    dst = [-(-min(k, n) // page) for k, n in zip(keeps, lens)]
    pages = sum(need) + sum(dst)
    perm = torch.randperm(pages, generator=g).int()
    tab, dtab = torch.zeros(3, max(need), dtype=torch.int32), torch.zeros(3, max(dst), dtype=torch.int32)
    at = 0
    for t, ns in ((tab, need), (dtab, dst)):
        for b, n in enumerate(ns):
            t[b, :n] = perm[at:at + n]
            at += n
    pool = torch.randint(0, 256, (pages, page, 336), generator=g).to(torch.uint8)
    mass = torch.rand(3, max(lens), generator=g)
    d = "cuda"
    dev = pool.to(d)
    kept, new, _ = mla.kv_evict(dev, tab.to(d), torch.tensor(lens, dtype=torch.int32, device=d), torch.tensor(keeps, dtype=torch.int32, device=d),
                                mass.to(d), dtab.to(d), 4, 8, max(lens), max(keeps), mla.MLA_KV_FP4)
    assert mla.get_status() == mla.MLA_OK
    ref = pool.clone()
    for b in range(3):
        k = min(keeps[b], lens[b])
        ids = kept[b, :k].cpu().long()
        assert int(new[b]) == k and (ids[1:] > ids[:-1]).all()
        i = torch.arange(k)
        ref[dtab[b].long()[i // page], i % page] = pool[tab[b].long()[ids // page], ids % page]
    assert torch.equal(dev.cpu(), ref)
