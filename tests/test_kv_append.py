"""mla_kv_append: latent norm, rotation of queries and keys, paged write.

The refusals run on the CPU.  The GPU cases compare every value against the formulas in 64
bits on the CPU.  Tolerances: one rounding to the output type (bf16: half a step, 2^-8 of
the value; e4m3: 2^-4 of the value, or half its smallest step 2^-10 below the normal range;
int8: half a code) plus the fp32 arithmetic before it.  That is at most 24 roundings of 2^-24
on any path (the sum of 576 squares is a tree of depth below 16, each rounding counted once, then
square root, division, two products and the rotation's two products and sum), relative to the
operands' size, which a rotation can cancel: 2^-19 of the largest value of the row.
"""
import ctypes
import math

import pytest
import torch

EPS = 1e-6
FP32 = 2.0 ** -19
E4M3_SCALE = 6.0 / 448.0


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
OK = dict(q_in=1 << 20, qit=192, qih=192, q_out=1 << 28, qot=192, qoh=192, heads=1, q_dim=192, q_weight=None,
          kv=1 << 12, kvt=576, kv_weight=None, eps=1e-6, cs=1 << 8, max_pos=10, pos=4, slots=8, n=2, inter=1,
          pool=1 << 30, num_slots=64, dtype=0, scale=1.0)


def _raw(mla, **kw):
    a = dict(OK, **kw)
    return mla.lib.mla_kv_append(*[a[k] for k in OK], None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(max_pos=0), dict(eps=-1.0), dict(eps=math.nan), dict(dtype=7), dict(heads=0), dict(qit=-8),
    dict(cs=None), dict(pos=None), dict(pos=6), dict(cs=24), dict(q_out=None), dict(q_in=(1 << 20) + 8),
    dict(q_out=(1 << 28) + 2), dict(q_weight=8), dict(qit=100), dict(qoh=4), dict(qot=184), dict(qot=0),
    dict(heads=2, qot=192, qoh=192), dict(q_out=(1 << 20) + 64), dict(q_out=1 << 20, qot=384),
    dict(pool=None), dict(slots=None), dict(num_slots=0), dict(slots=12), dict(pool=8), dict(kv=(1 << 12) + 2),
    dict(kvt=570), dict(kvt=-576), dict(kv_weight=4), dict(dtype=1, scale=0.0), dict(dtype=1, scale=math.nan),
    dict(dtype=2, scale=-1.0), dict(q_in=None, kv=None)])
def test_invalid_arguments_are_refused(mla, bad):
    assert _raw(mla, **bad) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(q_dim=584), dict(q_dim=56), dict(q_dim=100), dict(heads=1025, qot=192 * 1025),
                                 dict(dtype=3), dict(n=(1 << 20) + 1)])
def test_unsupported_shapes_are_refused(mla, bad):
    assert _raw(mla, **bad) == mla.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kv", [(1 << 30) - 1152, (1 << 30) + 64 * 1152 - 16, (1 << 30) + 16, (1 << 30) - 2 * 1152 + 16])
def test_keys_inside_the_pool_are_refused(mla, kv):
    assert _raw(mla, kv=kv) == mla.MLA_ERR_INVALID_ARG


def test_no_tokens_is_no_work(mla):
    assert _raw(mla, n=0) == mla.MLA_OK
    assert _raw(mla, n=0, q_in=None, kv=None, pool=None) == mla.MLA_OK


def test_binding_refuses_host_tensors(mla):
    z = torch.zeros
    with pytest.raises(mla.MlaError) as e:
        mla.kv_append(z(1, 1, 64, dtype=torch.bfloat16), None, z(1, dtype=torch.int32), None, z(4, 64), None)
    assert e.value.code == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ reference
def rot(x, cs, interleaved):
    c, s = cs[..., :32], cs[..., 32:]
    y = x.clone()
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def normed(x, w):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()


def reference(q, kv, pos, cos_sin, q_w, kv_w, interleaved):
    cs = cos_sin.double()[pos.long()]
    qr = kr = None
    if q is not None:
        v = normed(q.double(), q_w)
        qr = torch.cat([v[..., :-64], rot(v[..., -64:], cs[:, None], interleaved)], -1)
    if kv is not None:
        x = kv.double()
        kr = torch.cat([normed(x[:, :512], kv_w), rot(x[:, 512:], cs, interleaved)], -1)
    return qr, kr


def check_bf16(got, ref):
    got = got.double()
    size = ref.abs().amax(-1, keepdim=True)
    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + FP32 * size).all()


def check_codes(code, ref, scale, kind):
    x = ref / scale
    size = x.abs().amax(-1, keepdim=True)
    if kind == "int8":
        x = x.clamp(-127, 127)
        assert ((code.double() - x).abs() <= 0.5 + FP32 * size).all()
    else:
        x = x.clamp(-448, 448)
        got = code.view(torch.float8_e4m3fn).double()
        assert ((got - x).abs() <= torch.clamp(2.0 ** -4 * x.abs(), min=2.0 ** -10) + FP32 * size).all()


def table(n):
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def inputs(n, heads, dim, seed, big=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    q = (r(n, heads, dim) * big).bfloat16()
    kv = (r(n, 576) * big).bfloat16()
    return q, kv, (1 + 0.2 * r(dim)).bfloat16(), (1 + 0.2 * r(512)).bfloat16(), g


CASES = [  # n, heads, q_dim, page, kind, interleaved, q norm, kv norm, padded tokens
    (1, 16, 64, 64, "bf16", True, False, True, 0),
    (1, 1, 192, 8, "bf16", False, True, False, 0),
    (5, 3, 72, 16, "bf16", True, True, True, 2),
    (7, 16, 192, 32, "e4m3", False, True, True, 1),
    (33, 16, 64, 64, "int8", True, False, True, 4),
    (65, 128, 64, 256, "e4m3", True, False, True, 0),
    (130, 5, 576, 128, "bf16", False, True, True, 7),
    (257, 2, 320, 64, "int8", False, False, False, 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,dim,page,kind,inter,qn,kn,pad", CASES)
def test_against_the_formulas(mla, n, heads, dim, page, kind, inter, qn, kn, pad):
    q, kv, qw, kw, g = inputs(n, heads, dim, seed=n * 7 + dim)
    qw, kw = qw if qn else None, kw if kn else None
    cs = table(500)
    pos = torch.randint(0, 500, (n,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 499, 0
    pages = n // page + 2
    dt, dtype, scale = {"bf16": (mla.MLA_KV_BF16, torch.bfloat16, 1.0), "e4m3": (mla.MLA_KV_E4M3, torch.uint8, E4M3_SCALE),
                        "int8": (mla.MLA_KV_INT8, torch.int8, 0.031)}[kind]
    pool = torch.randint(0, 100, (pages, page, 576), generator=g).to(dtype)
    before = pool.clone()
    slots = torch.randperm(pages * page, generator=g)[:n]
    if pad:
        slots[torch.randperm(n, generator=g)[:pad]] = -1
    d = "cuda"
    dev = lambda t: None if t is None else t.to(d)
    pool_d = pool.to(d)
    out = mla.kv_append(q.to(d), kv.to(d), pos.to(d), slots.to(d), cs.to(d), pool_d, dev(kw), dev(qw), EPS, inter, dt, scale)
    assert mla.get_status() == mla.MLA_OK
    qr, kr = reference(q, kv, pos, cs, qw, kw, inter)
    check_bf16(out.cpu(), qr)
    flat, was = pool_d.cpu().view(-1, 576), before.view(-1, 576)
    live = slots >= 0
    if kind == "bf16":
        check_bf16(flat[slots[live]], kr[live])
    else:
        check_codes(flat[slots[live]], kr[live], scale, kind)
    rest = torch.ones(flat.shape[0], dtype=torch.bool)
    rest[slots[live]] = False
    assert torch.equal(flat[rest], was[rest])


@pytest.mark.gpu
def test_saturation_and_special_values(mla):
    """Codes saturate; a NaN becomes the e4m3 NaN code and int8 0; a zero row stays zero."""
    cs = table(4)
    kv = torch.zeros(3, 576, dtype=torch.bfloat16)
    kv[0, :4] = torch.tensor([1e4, -1e4, float("inf"), -float("inf")])
    kv[1, 7] = float("nan")
    pos = torch.zeros(3, dtype=torch.int32)
    slots = torch.arange(3)
    for kind, dtype, dt in (("e4m3", torch.uint8, mla.MLA_KV_E4M3), ("int8", torch.int8, mla.MLA_KV_INT8)):
        pool = torch.zeros(1, 8, 576, dtype=dtype, device="cuda")
        mla.kv_append(None, kv.cuda(), pos.cuda(), slots.cuda(), cs.cuda(), pool, kv_dtype=dt, kv_scale=0.5)
        assert mla.get_status() == mla.MLA_OK
        rows = pool[0].cpu()
        if kind == "int8":
            assert rows[0, :4].tolist() == [127, -127, 127, -127] and rows[1, 7] == 0
        else:
            v = rows.view(torch.float8_e4m3fn).float()
            assert v[0, :4].tolist() == [448.0, -448.0, 448.0, -448.0] and torch.isnan(v[1, 7])
        assert (rows[2] == 0).all()


@pytest.mark.gpu
def test_strided_views_in_place_and_broadcast(mla):
    q, kv, qw, kw, g = inputs(9, 4, 192, seed=3)
    cs, pos = table(64), torch.arange(9, dtype=torch.int32) * 7
    d = "cuda"
    csd, posd = cs.to(d), pos.to(d)
    # the last 64 columns of [N, H, 192] into the last 64 of [N, H, 576]
    wide = torch.randn(9, 4, 576, generator=g).bfloat16().to(d)
    keep = wide[..., :512].clone()
    mla.kv_append(q.to(d)[..., 128:], None, posd, None, csd, None, q_out=wide[..., 512:])
    check_bf16(wide[..., 512:].cpu(), reference(q[..., 128:], None, pos, cs, None, None, True)[0])
    assert torch.equal(wide[..., :512], keep)
    # head-major storage, in place
    hm = q.transpose(0, 1).contiguous().to(d)
    mla.kv_append(hm.transpose(0, 1), None, posd, None, csd, None, q_weight=qw.to(d), interleaved=False, q_out=hm.transpose(0, 1))
    check_bf16(hm.transpose(0, 1).cpu(), reference(q, None, pos, cs, qw, None, False)[0])
    # one head's row for all heads, a padded latent row stride
    lat = torch.zeros(9, 640, dtype=torch.bfloat16)
    lat[:, :576] = kv
    pool = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device=d)
    out = mla.kv_append(q[:, :1].to(d).expand(9, 4, 192), lat.to(d)[:, :576], posd, torch.arange(9).to(d), csd, pool, kw.to(d))
    qr, kr = reference(q[:, :1].expand(9, 4, 192), kv, pos, cs, None, kw, True)
    check_bf16(out.cpu(), qr)
    check_bf16(pool.view(-1, 576)[:9].cpu(), kr)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_bad_positions_and_slots_are_reported_and_skipped(mla):
    q, kv, _, kw, g = inputs(4, 2, 64, seed=5)
    cs = table(16)
    d = "cuda"
    pos = torch.tensor([3, 16, -1, 15], dtype=torch.int32)
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device=d)
    pool = torch.full((1, 8, 576), 5.0, dtype=torch.bfloat16, device=d)
    mla.kv_append(q.to(d), kv.to(d), pos.to(d), torch.arange(4).to(d), cs.to(d), pool, kw.to(d), q_out=out)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    qr, kr = reference(q[[0, 3]], kv[[0, 3]], pos[[0, 3]], cs, None, kw, True)
    check_bf16(out[[0, 3]].cpu(), qr)
    check_bf16(pool[0, [0, 3]].cpu(), kr)
    assert (out[[1, 2]] == 5).all() and (pool[0, [1, 2, 4, 5, 6, 7]] == 5).all()
    pool.fill_(5.0)
    mla.kv_append(None, kv.to(d), pos.clamp(0, 15).to(d), torch.tensor([0, 8, 2, 1 << 40]).to(d), cs.to(d), pool, kw.to(d))
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    assert (pool[0, [1, 3, 4, 5, 6, 7]] == 5).all()
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_captured_and_on_another_stream(mla):
    q, kv, qw, kw, g = inputs(20, 16, 192, seed=11)
    cs, pos = table(128), torch.arange(20, dtype=torch.int32)
    d = "cuda"
    args = [q.to(d), kv.to(d), pos.to(d), torch.arange(20).to(d), cs.to(d)]
    pool = torch.zeros(1, 32, 576, dtype=torch.bfloat16, device=d)
    out = torch.empty(20, 16, 192, dtype=torch.bfloat16, device=d)
    kwd, qwd = kw.to(d), qw.to(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    mla.kv_append(*args, pool, kwd, qwd, q_out=out, stream=side)
    side.synchronize()
    first, rows = out.clone(), pool.clone()
    out.zero_()
    pool.zero_()
    with torch.cuda.graph(graph, stream=side):
        mla.kv_append(*args, pool, kwd, qwd, q_out=out)
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(pool, rows)
    assert mla.get_status() == mla.MLA_OK


MANY = [  # tokens x heads above 12288: two steps of four heads a warp, 16 lanes a key
    # n, heads, q_dim, kind, interleaved, q norm, kv norm, padded tokens
    (129, 128, 64, "bf16", True, False, True, 9),        # 16512 rows, rotated columns alone
    (1025, 13, 64, "e4m3", False, True, True, 100),      # 13325: a step that is partly past the heads
    (769, 16, 192, "bf16", False, False, True, 0),       # 12304
    (800, 16, 192, "int8", True, True, False, 33),
    (2050, 7, 168, "e4m3", True, True, True, 1),         # 14350: chunks that do not fill the lanes
    (999, 13, 576, "bf16", True, True, True, 17),        # wide rows: two turns of one step
    (1300, 10, 320, "e4m3", False, False, True, 0),
    (1541, 8, 264, "int8", False, True, True, 5),        # 12328
    (12289, 1, 192, "bf16", True, True, True, 3),        # one head: three of a step's four rows are idle
]


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,dim,kind,inter,qn,kn,pad", MANY)
def test_many_rows_against_the_formulas(mla, n, heads, dim, kind, inter, qn, kn, pad):
    test_against_the_formulas(mla, n, heads, dim, 64, kind, inter, qn, kn, pad)


@pytest.mark.gpu
@pytest.mark.parametrize("n,dim", [(96, 192), (97, 192), (96, 576), (97, 576), (96, 64), (97, 64)])
def test_both_sides_of_the_many_rows_border(mla, n, dim):
    """12288 rows still run as few, 12416 as many."""
    for inter in (True, False):
        test_against_the_formulas(mla, n, 128, dim, 64, "bf16", inter, dim > 64, True, 2)


@pytest.mark.parametrize("bad", [
    dict(q_out=(1 << 30) + 1152), dict(q_out=(1 << 30) - 384), dict(q_out=(1 << 30) + 64 * 1152 - 16),
    dict(q_in=(1 << 30) + 64), dict(q_in=(1 << 30) - 16), dict(q_in=1 << 30, q_out=1 << 30)])
def test_queries_inside_the_pool_are_refused(mla, bad):
    assert _raw(mla, **bad) == mla.MLA_ERR_INVALID_ARG
