"""mla_key_mass: the attention weight of each cached key, accumulated.

The refusals run on the CPU; the GPU cases compare every entry with the definition in 64 bits.
Tolerance per key, with w its exact weight of this call: a score off by d scales a row's share by
exp(d), and d is at most 2^-17 of A = scale max sum_i |q_i k_i| (36 accumulation steps of at most
2^-23 each), on an e4m3 pool also the query split's scale 2^-17 max|q| sum_i |k_i|; the exponent's
argument is rounded at its size, 2^-22 (|s| + |lse|); the exponential and the sum of R terms add
2^-22 + R 2^-24; the update of the old mass 2^-23 of it.
"""
import ctypes
import math

import pytest
import torch

from test_decode_tree import KINDS, SCALE, make, random_tree, rows_of


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
def _raw(mla, plan, **kw):
    a = dict(q=1 << 20, kv=1 << 21, ps=None, pt=1 << 22, sl=1 << 23, mask=None, lse=1 << 25, T=plan.q_len, H=plan.num_heads,
             scale=0.07, kvs=1.0, decay=1.0, mass=1 << 24, stride=20000, ws=1 << 26, wsb=1 << 40)
    a.update(kw)
    return mla.lib.mla_key_mass(ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(kv=None), dict(pt=None), dict(sl=None), dict(lse=None), dict(mass=None), dict(ps=1 << 9), dict(T=5),
    dict(H=15), dict(scale=0.0), dict(scale=math.nan), dict(kvs=0.0), dict(decay=-0.5), dict(decay=math.nan), dict(stride=8999),
    dict(q=8), dict(kv=8), dict(lse=2), dict(mass=2), dict(mask=4)])
def test_invalid_arguments_are_refused(mla, bad):
    plan = mla.decode_plan([9000, 300], 4, 16, 64, 200, 400, 0, 152)
    assert _raw(mla, plan, **bad) == mla.MLA_ERR_INVALID_ARG


def test_wide_plans_need_a_workspace(mla):
    plan = mla.decode_plan([9000, 300], 20, 16, 64, 200, 400, 0, 152)
    need = ctypes.c_size_t(7)
    assert mla.lib.mla_key_mass_workspace(ctypes.byref(plan), ctypes.byref(need)) == mla.MLA_OK
    if need.value:
        assert _raw(mla, plan, ws=None) == mla.MLA_ERR_INVALID_ARG
        assert _raw(mla, plan, ws=(1 << 26) + 8) == mla.MLA_ERR_INVALID_ARG
        assert _raw(mla, plan, wsb=need.value - 1) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    assert mla.lib.mla_key_mass_workspace(None, ctypes.byref(need)) == mla.MLA_ERR_INVALID_ARG


def test_trees_of_more_than_64_drafts_are_refused(mla):
    plan = mla.decode_plan([9000, 300], 65, 1, 64, 200, 400, 0, 152)
    assert _raw(mla, plan, mask=1 << 12) == mla.MLA_ERR_UNSUPPORTED


def test_page_scales_belong_to_their_format_alone(mla):
    plan = mla.decode_plan([9000, 300], 4, 16, 64, 200, 400, 3, 152)
    assert _raw(mla, plan) == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ reference
def reference(q, val, table, lens, words, lse, mass, decay, kind):
    """New masses and their tolerance, in 64 bits."""
    B, T, H, _ = q.shape
    new, tol = mass.double().clone(), torch.zeros_like(mass, dtype=torch.float64)
    for b, L in enumerate(lens):
        k = rows_of(val, table, b, L)
        qb = q[b].double().reshape(T * H, 576)
        x = (qb @ k.T * SCALE).view(T, H, L)
        d = 2.0 ** -17 * (qb.abs() @ k.abs().T).view(T, H, L) * SCALE
        if kind == "e4m3":
            d = d + SCALE * 2.0 ** -17 * q[b].double().abs().amax(-1)[..., None] * k.abs().sum(1)
        l = lse[b].double()[..., None]
        d = d + 2.0 ** -22 * (x.abs() + l.abs()) + 2.0 ** -22 + T * H * 2.0 ** -24
        seen = torch.ones(T, L, dtype=torch.bool)
        for t in range(T):
            for u in range(T):
                seen[t, L - T + u] = u <= t if words is None else bool((int(words[b, t]) >> u) & 1)
        live = seen[:, None, :] & torch.isfinite(l)
        w = torch.where(live, torch.exp(x - torch.where(torch.isfinite(l), l, 0.0)), 0.0)
        old = decay * mass[b, :L].double() if decay else torch.zeros(L, dtype=torch.float64)
        new[b, :L] = old + w.sum((0, 1))
        tol[b, :L] = torch.where(live, w * 1.01 * d, 0.0).sum((0, 1)) + 2.0 ** -23 * (old.abs() + new[b, :L].abs())
    return new, tol


def true_lse(q, val, table, lens, words):
    B, T, H, _ = q.shape
    out = torch.zeros(B, T, H)
    for b, L in enumerate(lens):
        x = (q[b].double().reshape(T * H, 576) @ rows_of(val, table, b, L).T * SCALE).view(T, H, L)
        for t in range(T):
            for u in range(T):
                if not (u <= t if words is None else (int(words[b, t]) >> u) & 1):
                    x[t, :, L - T + u] = -math.inf
        out[b] = torch.logsumexp(x, -1).float()
    return out


def run(mla, lens, T, H, page, kind, words, decay=1.0, seed=0, sms=0, pad=5):
    q, pool, table, scales, kv_scale, val = make(lens, T, H, page, kind, seed)
    lse = true_lse(q, val, table, lens, words)
    g = torch.Generator().manual_seed(seed + 1)
    mass = torch.rand(len(lens), max(lens) + pad, generator=g)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, page, table.shape[1], pool.shape[0], KINDS[kind], sms)
    md = mass.to(d)
    if decay == 0:
        md[:, ::2] = math.nan  # not read
        for b, L in enumerate(lens):
            md[b, L:] = mass[b, L:].to(d)
    mla.key_mass(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), lse.to(d), md, SCALE,
                 kv_scale, tree_mask=None if words is None else words.to(d),
                 page_scales=None if scales is None else scales.to(d), decay=decay)
    assert mla.get_status() == mla.MLA_OK
    got = md.cpu()
    new, tol = reference(q, val, table, lens, words, lse, mass, decay, kind)
    bad = (got.double() - new).abs() > tol
    assert not bad.any() and not torch.isnan(got).any(), ((got.double() - new).abs() / tol.clamp(min=1e-300)).max()
    for b, L in enumerate(lens):
        assert torch.equal(got[b, L:], mass[b, L:])
    return got


CASES = [  # lens, T, H, page, kind, tree, decay, SMs planned for
    ([1], 1, 1, 64, "bf16", False, 1.0, 0),
    ([1, 127, 128, 129], 1, 16, 64, "bf16", False, 0.5, 0),
    ([5, 64, 65, 400], 5, 3, 16, "bf16", True, 1.0, 1),
    ([700, 2, 257], 2, 16, 8, "bf16", False, 0.0, 0),
    ([1000, 333], 4, 16, 128, "bf16", True, 0.97, 0),           # 64 rows
    ([500, 90], 5, 16, 64, "bf16", True, 1.0, 0),               # 80 rows
    ([640, 1999], 8, 16, 256, "bf16", False, 0.9, 0),           # 128 rows
    ([300, 129], 9, 16, 32, "bf16", True, 1.0, 0),              # 144 rows
    ([200, 900], 64, 16, 64, "bf16", True, 0.25, 0),            # 1024 rows
    ([400, 300], 200, 2, 64, "bf16", False, 1.0, 0),            # more drafts than a tree may have
    ([1, 33, 130], 1, 16, 64, "e4m3", False, 0.0, 0),
    ([600, 77], 5, 16, 64, "e4m3", True, 0.97, 0),
    ([2000, 64], 2, 8, 16, "e4m3", False, 1.0, 0),
    ([300, 1300], 33, 16, 128, "e4m3", True, 0.5, 0),           # 528 rows
    ([90, 777], 3, 5, 8, "e4m3", True, 1.0, 0),
    ([400, 129] + [64 + 7 * i for i in range(60)], 2, 8, 64, "e4m3", False, 0.5, 0),  # more requests than a warp's lanes
    ([64 + 3 * i for i in range(200)], 1, 16, 64, "bf16", False, 1.0, 0),             # more requests than SMs
    ([65, 700], 5, 16, 64, "int8", True, 1.0, 0),
    ([1200, 90], 9, 16, 8, "int8", False, 0.3, 0),
    ([65, 700], 5, 16, 64, "int8page", False, 0.9, 0),
    ([129, 600], 12, 20, 32, "int8page", True, 0.0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,H,page,kind,tree,decay,sms", CASES)
def test_against_the_definition(mla, lens, T, H, page, kind, tree, decay, sms):
    words = random_tree(torch.Generator().manual_seed(T), len(lens), T) if tree else None
    got = run(mla, lens, T, H, page, kind, words, decay, seed=sum(lens), sms=sms)
    if decay == 0:  # every row's weights add up to 1
        total = sum(got[b, :L].double().sum() for b, L in enumerate(lens))
        assert abs(total - len(lens) * T * H) < 1e-3 * len(lens) * T * H


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_rows_without_a_finite_lse_add_nothing(mla, kind):
    def tweak(q, lse):
        lse[0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, math.nan])
        lse[1, 2] = -math.inf
        if kind == "bf16":
            q[0, 0, 0] = math.nan

    q, pool, table, scales, kv_scale, val = make([300, 64], 3, 16, 64, kind, 4)
    lse = true_lse(q, val, table, [300, 64], None)
    tweak(q, lse)
    mass = torch.rand(2, 300)
    d = "cuda"
    plan = mla.decode_plan([300, 64], 3, 16, 64, table.shape[1], pool.shape[0], KINDS[kind])
    got = mla.key_mass(plan, q.to(d), pool.to(d), table.to(d), torch.tensor([300, 64], dtype=torch.int32, device=d), lse.to(d),
                       mass.to(d), SCALE, kv_scale).cpu()
    assert mla.get_status() == mla.MLA_OK
    q = torch.nan_to_num(q)
    new, tol = reference(q, val, table, [300, 64], None, lse, mass, 1.0, kind)
    assert ((got.double() - new).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_not_finite_keys_stay_their_own(mla, kind):
    """NaN rows behind the end and in a draft that rows do not see leave every other key alone."""
    lens, T, H = [100, 70], 4, 16
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 4)
    words = random_tree(torch.Generator().manual_seed(3), 2, T) & ~2
    words[:, 1] |= 1  # nobody sees draft 1, not even itself
    lse = true_lse(q, val, table, lens, words)
    for b, L in enumerate(lens):
        for j in [L - T + 1] + list(range(L, 128)):
            pool[table[b, j // 64], j % 64] = math.nan if kind == "bf16" else 0x7F
    mass = torch.rand(2, 128)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    got = mla.key_mass(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), lse.to(d),
                       mass.to(d), SCALE, kv_scale, tree_mask=words.to(d)).cpu()
    new, tol = reference(q, val, table, lens, words, lse, mass, 1.0, kind)
    assert ((got.double() - new).abs() <= tol).all()
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_bad_lengths_and_pages_are_reported(mla, kind):
    lens, T, H = [200, 300, 260], 4, 16
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 3)
    lse = true_lse(q, val, table, lens, None)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    mass = torch.rand(3, 300)
    md = mass.to(d)
    call = lambda tb, ls: mla.key_mass(plan, q.to(d), pool.to(d), tb.to(d), torch.tensor(ls, dtype=torch.int32, device=d), lse.to(d),
                                       md, SCALE, kv_scale)
    call(table, [3, 301, 260])
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    new, tol = reference(q, val, table, lens, None, lse, mass, 1.0, kind)
    got = md.cpu()
    assert torch.equal(got[:2], mass[:2]) and ((got[2].double() - new[2]).abs() <= tol[2]).all()
    md.copy_(mass)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = pool.shape[0], -5
    call(bad, lens)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    got = md.cpu()
    ok = torch.ones(3, 300, dtype=torch.bool)
    ok[0, 64:128], ok[1, 128:192] = False, False
    assert ((got.double() - new).abs() <= tol)[ok].all()
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T", [("bf16", 2), ("bf16", 20), ("e4m3", 5), ("int8", 3), ("int8", 20)])
def test_captured_calls_follow_the_device_inputs(mla, kind, T):
    lens, H = [900, 2000], 16
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 6)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    ws = mla.key_mass_workspace_for(plan, d)
    lse = true_lse(q, val, table, lens, None)
    sl, ld, md = torch.tensor(lens, dtype=torch.int32, device=d), lse.to(d), torch.zeros(2, 2000, device=d)
    qd, pd, td = q.to(d), pool.to(d), table.to(d)
    call = lambda: mla.key_mass(plan, qd, pd, td, sl, ld, md, SCALE, kv_scale, decay=0.5, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for new_lens in ([900, 2000], [T, 1111]):
        mass = torch.rand(2, 2000)
        md.copy_(mass)
        sl.copy_(torch.tensor(new_lens, dtype=torch.int32))
        l = true_lse(q, val, table, new_lens, None)
        ld.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        new, tol = reference(q, val, table, new_lens, None, l, mass, 0.5, kind)
        assert ((md.cpu().double() - new).abs() <= tol).all()
    first = md.clone()
    md.copy_(mass)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(md, first)  # the same sums, in the same order
    assert mla.get_status() == mla.MLA_OK


# ------------------------------------------------------------------------------ page scales
@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 20])  # 20 drafts of 16 heads: row groups, summed by a second kernel
@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("factor", [math.nan, math.inf, -math.inf, -1e-3, 300.0])
def test_page_scales_out_of_range_are_reported_and_add_nothing(mla, T, decay, factor):
    """As mla_decode_int8_paged: a scale that is not finite or outside [0, 255 kv_scale] on a page that
    is read.  Its keys get no weight; a page that no request reads may hold anything."""
    lens, H, kind = [300, 200], 16, "int8page"
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 5)
    lse = true_lse(q, val, table, lens, None)
    mass = torch.rand(2, 300)
    new, tol = reference(q, val, table, lens, None, lse, mass, decay, kind)
    unread = (set(range(pool.shape[0])) - set(table[0, :5].tolist()) - set(table[1, :4].tolist())).pop()
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    call = lambda m: mla.key_mass(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), lse.to(d),
                                  m, SCALE, kv_scale, page_scales=scales.to(d), decay=decay).cpu().double()
    scales[unread] = factor
    got = call(mass.to(d))
    assert mla.get_status() == mla.MLA_OK
    assert ((got - new).abs() <= tol).all()
    # the second page of the first request, the last (partial) one of the other
    scales[table[0, 1]] = scales[table[1, 3]] = factor * kv_scale
    for b, j in ((0, slice(64, 128)), (1, slice(192, 200))):
        new[b, j] = decay * mass[b, j].double()
        tol[b, j] = 2.0 ** -23 * new[b, j]
    got = call(mass.to(d))
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    assert ((got - new).abs() <= tol).all()
    assert mla.get_status() == mla.MLA_OK


# ------------------------------------------------------------------------------ workspace
@pytest.mark.parametrize("T,groups", [(1, 1), (8, 1), (20, 3), (64, 8)])
@pytest.mark.parametrize("kv", [0, 1, 2, 3])
def test_workspace_holds_the_row_groups_sums(mla, kv, T, groups):
    """One fp32 sum per row group, request and key; at most 128 rows are one group and need none."""
    plan = mla.decode_plan([9000, 300], T, 16, 64, 200, 400, kv, 152)
    need = ctypes.c_size_t(7)
    assert mla.lib.mla_key_mass_workspace(ctypes.byref(plan), ctypes.byref(need)) == mla.MLA_OK
    assert need.value == (0 if groups == 1 else groups * 2 * 9000 * 4)
    ps = 1 << 9 if kv == 3 else None
    if need.value:
        assert _raw(mla, plan, ps=ps, ws=None) == mla.MLA_ERR_INVALID_ARG
        assert _raw(mla, plan, ps=ps, ws=(1 << 26) + 8) == mla.MLA_ERR_INVALID_ARG
        assert _raw(mla, plan, ps=ps, wsb=need.value - 1) == mla.MLA_ERR_WORKSPACE_TOO_SMALL


def test_the_workspace_begins_at_129_rows(mla):
    need = ctypes.c_size_t(7)
    for T, bytes_ in ((128, 0), (129, 2 * 2 * 9000 * 4)):
        plan = mla.decode_plan([9000, 300], T, 1, 64, 200, 400, 0, 152)
        assert mla.lib.mla_key_mass_workspace(ctypes.byref(plan), ctypes.byref(need)) == mla.MLA_OK
        assert need.value == bytes_
