"""mla_decode_tree: attention of a tree of drafted tokens over the paged latent cache.

The refusals run on the CPU.  The GPU cases compare every output with the definition in 64
bits.  Tolerances, per output element, with w_j the exact weights and W = sum_j w_j |v_j|:
  * the output's own rounding, 2^-8 |out|;
  * the weights' rounding before the second product, 2^-8 W (bf16; the split 8-bit pair of an
    e4m3 pool 2^-8 too, and 2^-20 of the largest weight for each of the n keys below its normal
    range, i.e. n 2^-20 max|v| / sum_j exp(s_j - max s); f16 on int8 pools is closer);
  * the scores: 36 accumulation steps of the first product, each off by at most 2^-23 of
    A = scale max_j sum_i |q_i k_ji| (2^-17 A in all), and on an e4m3 pool the query split's
    2^-17 max|q| per element, E = scale 2^-17 max|q| max_j sum_i |k_ji|.  A score off by d
    moves lse by d and the output by 2 d W;
  * lse: also 2^-20 (1 + |lse|) for the exponentials and logarithms.
"""
import ctypes
import math

import pytest
import torch

SCALE = 1.0 / math.sqrt(192.0)
KINDS = {"bf16": 0, "e4m3": 1, "int8": 2, "int8page": 3}


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ refusals
def _plan(mla, lens=(9000, 300), T=4, H=16, kv=0, sms=152):
    return mla.decode_tree_plan(list(lens), T, H, 64, 200, 400, kv, sms)


def _raw(mla, plan, **kw):
    a = dict(q=1 << 20, kv=1 << 21, ps=None, pt=1 << 22, sl=1 << 23, mask=1 << 12, T=plan.q_len, H=plan.num_heads,
             scale=0.07, kvs=1.0, out=1 << 24, lse=1 << 25, ws=1 << 26, wsb=plan.workspace_bytes)
    a.update(kw)
    return mla.lib.mla_decode_tree(ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("kv,width", [(0, 4), (1, 2), (2, 2), (3, 2)])
@pytest.mark.parametrize("T", [1, 2, 4, 20])
def test_tree_plan_sizes_its_partials(mla, kv, width, T):
    """fp32 rows over a bf16 pool, 16-bit rows over 8-bit ones; narrow trees split as mla_decode."""
    tree, chain = _plan(mla, T=T, kv=kv), mla.decode_plan([9000, 300], T, 16, 64, 200, 400, kv, 152)
    assert tree.max_splits > 1 and tree.rows == 16 * T
    parts = 2 * tree.max_splits * 16 * T
    assert tree.workspace_bytes == 256 + parts * 512 * width + parts * 4
    if kv or T <= 4:
        assert (tree.max_splits, tree.chunk_tokens) == (chain.max_splits, chain.chunk_tokens)


@pytest.mark.parametrize("bad,code", [
    (dict(mask=None), 1), (dict(mask=12), 1), (dict(q=None), 1), (dict(kv=None), 1), (dict(pt=None), 1), (dict(sl=None), 1),
    (dict(out=None), 1), (dict(lse=None), 1), (dict(T=5), 1), (dict(H=15), 1), (dict(scale=0.0), 1), (dict(kvs=-1.0), 1),
    (dict(ps=1 << 9), 1), (dict(ws=None), 1), (dict(ws=(1 << 26) + 64), 1), (dict(q=(1 << 20) + 8), 1)])
def test_invalid_arguments_are_refused(mla, bad, code):
    assert _raw(mla, _plan(mla), **bad) == code


def test_workspace_of_a_chain_plan_is_too_small(mla):
    chain = mla.decode_plan([9000, 300], 4, 16, 64, 200, 400, 0, 152)
    assert _raw(mla, chain) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    tree = _plan(mla)
    assert _raw(mla, tree, wsb=tree.workspace_bytes - 1) == mla.MLA_ERR_WORKSPACE_TOO_SMALL


def test_page_scales_belong_to_their_format_alone(mla):
    assert _raw(mla, _plan(mla, kv=3)) == mla.MLA_ERR_INVALID_ARG


def test_more_than_64_drafts_are_refused(mla):
    with pytest.raises(mla.MlaError) as e:
        _plan(mla, T=65)
    assert e.value.code == mla.MLA_ERR_UNSUPPORTED
    assert _raw(mla, mla.decode_plan([9000, 300], 65, 1, 64, 200, 400, 0, 152), wsb=1 << 40) == mla.MLA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(mla):
    plan = _plan(mla, lens=[64], sms=1)
    z = torch.zeros
    with pytest.raises(mla.MlaError) as e:
        mla.decode_tree(plan, z(1), z(400, 64, 576, dtype=torch.bfloat16), z(1), z(1), z(1), SCALE)
    assert e.value.code == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ reference
def random_tree(g, B, T):
    """Ancestor masks (self included) of random trees, as int64 words."""
    words = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            w = 1 << t
            if t:
                w |= int(words[b, int(torch.randint(0, t, (1,), generator=g))]) & ((1 << 64) - 1)
            words[b, t] = w - (1 << 64) if w >> 63 else w
    return words


def make(lens, T, H, page, kind, seed, peaked=False, extra=3):
    """q, pool, page table, page scales, kv_scale and each request's rows in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=g).int()
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    x = torch.randn(pages, page, 576, generator=g)
    q = (torch.randn(B, T, H, 576, generator=g) * (8.0 if peaked else 1.0)).bfloat16()
    kv_scale, scales = 1.0, None
    if kind == "bf16":
        pool = x.bfloat16()
        val = pool.double()
    elif kind == "e4m3":
        kv_scale = 6.0 / 448
        pool = (x / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        val = pool.view(torch.float8_e4m3fn).double() * kv_scale
    else:
        kv_scale = 5.0 / 127
        per = torch.full((pages,), kv_scale)
        if kind == "int8page":
            scales = per = kv_scale * torch.rand(pages, generator=g).float()
        pool = (x / kv_scale).round().clamp(-127, 127).to(torch.int8)
        val = pool.double() * per.double()[:, None, None]
    return q, pool, table, scales, kv_scale, val


def rows_of(val, table, b, L):
    page = val.shape[1]
    j = torch.arange(L)
    return val[table[b].long()[j // page], j % page]


def reference(q, val, table, lens, words):
    """out, lse and the tolerances' parts, in 64 bits."""
    B, T, H, _ = q.shape
    out = torch.zeros(B, T, H, 512, dtype=torch.float64)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64)
    W, A, E = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    small = torch.zeros_like(lse)
    for b, L in enumerate(lens):
        k = rows_of(val, table, b, L)
        x = q[b].double().reshape(T * H, 576) @ k.T * SCALE
        a = (q[b].double().abs().reshape(T * H, 576) @ k.abs().T).amax(1) * SCALE
        A[b] = a.view(T, H)
        E[b] = SCALE * 2.0 ** -17 * q[b].double().abs().amax(-1) * k.abs().sum(1).max()
        seen = torch.ones(T, L, dtype=torch.bool)
        for t in range(T):
            for u in range(T):
                seen[t, L - T + u] = bool((int(words[b, t]) >> u) & 1)
        x = x.view(T, H, L).masked_fill(~seen[:, None, :], -math.inf)
        lse[b] = torch.logsumexp(x, -1)
        some = lse[b] > -math.inf
        w = torch.where(some[..., None], torch.exp(x - torch.where(some, lse[b], 0.0)[..., None]), 0.0)
        out[b] = w @ k[:, :512]
        W[b] = w @ k[:, :512].abs()
        # n 2^-20 max|v| / sum exp(s - max): the largest weight is 1 / that sum
        small[b] = L * 2.0 ** -20 * k.abs().max() * w.amax(-1)
    return out, lse, W, A, E, small


def check(got, glse, ref, kind):
    out, lse, W, A, E, small = ref
    got, glse = got.double().cpu(), glse.double().cpu()
    none = lse == -math.inf
    assert (glse[none] == -math.inf).all() and (got[none] == 0).all()
    d = 2.0 ** -17 * A + (E if kind == "e4m3" else 0)
    tol_l = d + 2.0 ** -20 * (1 + lse.abs())
    assert ((glse - lse).abs() <= tol_l)[~none].all(), ((glse - lse).abs() / tol_l)[~none].max()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * d[..., None] + 2.0 ** -18) * W
    if kind != "bf16":
        tol = tol + small[..., None]
    bad = (got - out).abs() > tol
    assert not bad[~none].any(), ((got - out).abs() / tol)[~none].max()


def run(mla, lens, T, H, page, kind, words, seed=0, sms=0, peaked=False, tweak=None, stream=None):
    q, pool, table, scales, kv_scale, val = make(lens, T, H, page, kind, seed, peaked)
    if tweak:
        tweak(q, pool, table, val)
    plan = mla.decode_tree_plan(lens, T, H, page, table.shape[1], pool.shape[0], KINDS[kind], sms)
    d = "cuda"
    out, lse = mla.decode_tree(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d),
                               words.to(d), SCALE, kv_scale, page_scales=None if scales is None else scales.to(d))
    assert mla.get_status() == mla.MLA_OK
    return out, lse, reference(q, val, table, lens, words), plan


CASES = [  # lens, T, H, page, kind, SMs planned for (1: never split)
    ([1], 1, 16, 64, "bf16", 1),
    ([5, 64, 65], 5, 3, 64, "bf16", 1),
    ([64, 127, 128, 129, 200], 2, 16, 64, "bf16", 1),          # 32 rows
    ([130, 70, 64], 64, 1, 64, "bf16", 1),
    ([300, 1000], 7, 7, 16, "bf16", 0),
    ([63, 640, 2000], 4, 16, 8, "bf16", 0),                    # 64 rows
    ([1500, 90], 3, 16, 128, "bf16", 0),                       # 48 rows
    ([64, 65, 2500], 11, 3, 64, "bf16", 0),                    # 33 rows
    ([700, 130, 5], 5, 8, 8, "bf16", 1),                       # 40 rows
    ([47, 111, 3000], 47, 1, 32, "bf16", 0),
    ([300, 2000], 4, 16, 64, "bf16", 0),                       # 64 rows
    ([900, 5, 129], 5, 13, 16, "bf16", 0),                     # 65 rows
    ([128, 1000], 8, 16, 64, "bf16", 1),                       # 128 rows
    ([1000, 70], 43, 3, 64, "bf16", 0),                        # 129 rows
    ([777, 2100], 16, 16, 64, "bf16", 0),                      # 256 rows
    ([1025, 70, 129], 33, 8, 256, "bf16", 0),
    ([200, 1111], 64, 16, 64, "bf16", 0),                      # 1024 rows
    ([40, 3000], 12, 40, 32, "bf16", 0),
    ([1, 33, 65], 1, 16, 64, "e4m3", 1),
    ([64, 128, 1000], 12, 16, 64, "e4m3", 0),
    ([70, 2111], 2, 8, 16, "e4m3", 0),
    ([300, 129], 64, 5, 128, "e4m3", 0),
    ([900, 66], 31, 16, 32, "e4m3", 0),
    ([100, 333], 9, 4, 8, "e4m3", 0),
    ([65, 700], 5, 16, 64, "int8", 0),
    ([64, 130], 64, 2, 16, "int8", 1),
    ([1200, 90], 9, 16, 128, "int8", 0),
    ([65, 700], 5, 16, 64, "int8page", 0),
    ([129, 1400], 20, 7, 32, "int8page", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,H,page,kind,sms", CASES)
def test_random_trees(mla, lens, T, H, page, kind, sms):
    words = random_tree(torch.Generator().manual_seed(T * H), len(lens), T)
    out, lse, ref, plan = run(mla, lens, T, H, page, kind, words, seed=sum(lens), sms=sms)
    check(out, lse, ref, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8", "int8page"])
@pytest.mark.parametrize("T,H", [(4, 8), (8, 16), (64, 4)])
def test_empty_rows_and_arbitrary_masks(mla, kind, T, H):
    """Rows that see nothing, only a prefix, only others, or everything; bits past T are ignored."""
    g = torch.Generator().manual_seed(T)
    lens = [T, T + 1, 64 + T // 2, 500]
    words = torch.randint(-(1 << 62), 1 << 62, (4, T), generator=g)
    words[:, 0] = 0
    words[0, T // 2] = 0
    words[:, T - 1] = -1
    out, lse, ref, _ = run(mla, lens, T, H, 64, kind, words, seed=9)
    if T < 64:
        assert (ref[1][0, 0] == -math.inf).all()
    check(out, lse, ref, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("H", [2, 16, 40])
def test_splits_agree_and_peaked_scores(mla, kind, H):
    """Any split count, among them last splits that hold drafts alone."""
    T = 6
    lens = [64 * 9 + 3, 64 * 5 + 6, 6, 4000]
    words = random_tree(torch.Generator().manual_seed(4), 4, T)
    for sms in (1, 20, 300):
        out, lse, ref, plan = run(mla, lens, T, H, 64, kind, words, seed=1, sms=sms, peaked=True)
        check(out, lse, ref, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,H", [(3, 8), (3, 16), (4, 16), (6, 16), (20, 16)])
def test_not_finite_drafts_reach_only_those_that_see_them(mla, kind, T, H):
    """NaN and infinite rows in drafts; NaN in every row behind the request's end."""
    lens = [64 + 2 + T, 500]
    g = torch.Generator().manual_seed(2)
    words = random_tree(g, 2, T)
    words[:, 2:] &= ~2  # only draft 1 sees draft 1
    words[:, 0] &= ~2

    def spoil(q, pool, table, val):
        page = pool.shape[1]
        for b, L in enumerate(lens):
            for j in [L - T + 1] + list(range(L, table.shape[1] * page)):
                if j >= -(-L // page) * page:
                    break
                row = pool[table[b, j // page], j % page]
                if kind == "bf16":
                    row[::3] = math.nan
                    row[1::3] = math.inf
                    row[2::3] = -math.inf
                else:
                    row[:] = 0x7F
                    row[::2] = 0xFF
                val[table[b, j // page], j % page] = 0.0

    out, lse, ref, _ = run(mla, lens, T, H, 64, kind, words, seed=5, tweak=spoil)
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all()
    keep = [t for t in range(T) if t != 1]
    ref = tuple(x[:, keep] for x in ref)
    check(out[:, keep], lse[:, keep], ref, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8", "int8page"])
def test_a_chain_is_the_ordinary_decode(mla, kind):
    """The mask of a chain gives what mla_decode gives, to the two calls' roundings."""
    T, H, lens = 5, 16, [300, 2000, 66]
    words = torch.tensor([[(2 << t) - 1 for t in range(T)]] * 3)
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 3)
    d = "cuda"
    sl = torch.tensor(lens, dtype=torch.int32, device=d)
    args = (q.to(d), pool.to(d))
    chain = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    if scales is None:
        o1, l1 = mla.decode(chain, *args, table.to(d), sl, SCALE, kv_scale)
    else:
        o1, l1 = mla.decode_int8_paged(chain, *args, scales.to(d), table.to(d), sl, SCALE, kv_scale)
    tree = mla.decode_tree_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    o2, l2 = mla.decode_tree(tree, *args, table.to(d), sl, words.to(d), SCALE, kv_scale,
                             page_scales=None if scales is None else scales.to(d))
    assert mla.get_status() == mla.MLA_OK
    ref = reference(q, val, table, lens, words)
    check(o2, l2, ref, kind)
    assert ((l1 - l2).abs() <= 1e-4).all()
    assert ((o1.float() - o2.float()).abs().cpu() <= 2.0 ** -6 * ref[2].float() + 1e-6).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_lengths_and_pages_are_reported(mla, kind):
    T, H, lens = 4, 16, [200, 300, 260]
    words = random_tree(torch.Generator().manual_seed(1), 3, T)
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 3)
    d = "cuda"
    plan = mla.decode_tree_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind], 1)
    out = torch.full((3, T, H, 512), 7.0, dtype=torch.bfloat16, device=d)
    lse = torch.full((3, T, H), 7.0, device=d)
    call = lambda tb, ls: mla.decode_tree(plan, q.to(d), pool.to(d), tb.to(d), torch.tensor(ls, dtype=torch.int32, device=d),
                                          words.to(d), SCALE, kv_scale, out=out, lse=lse)
    call(table, [3, 301, 260])  # too short, beyond the plan, fine
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    assert (out[:2] == 7).all() and (lse[:2] == 7).all()
    check(out[2:], lse[2:], tuple(x[2:] for x in reference(q, val, table, lens, words)), kind)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = pool.shape[0], -5
    call(bad, lens)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    check(out[2:], lse[2:], tuple(x[2:] for x in reference(q, val, table, lens, words)), kind)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,H", [("bf16", 2, 16), ("bf16", 3, 16), ("bf16", 4, 16), ("bf16", 8, 16), ("bf16", 32, 16),
                                       ("e4m3", 8, 16), ("int8", 4, 16)])
def test_captured_calls_follow_the_device_inputs(mla, kind, T, H):
    """Two captured calls on one workspace, replayed with new masks, lengths and queries."""
    lens = [1000, 3000]
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 8)
    d = "cuda"
    plan = mla.decode_tree_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    ws = mla.workspace_for(plan, d)
    assert ws is not None
    qd, pd, td = q.to(d), pool.to(d), table.to(d)
    sl = torch.tensor(lens, dtype=torch.int32, device=d)
    w1, w2 = (random_tree(torch.Generator().manual_seed(s), 2, T).to(d) for s in (1, 2))
    side = torch.cuda.Stream()
    call = lambda w: mla.decode_tree(plan, qd, pd, td, sl, w, SCALE, kv_scale, workspace=ws)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(w1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r1, r2 = call(w1), call(w2)
    for seed, new in ((5, [1000, 3000]), (6, [64 + T, 2999])):
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(q.shape, generator=g).bfloat16()
        words = [random_tree(g, 2, T) for _ in range(2)]
        qd.copy_(q)
        w1.copy_(words[0])
        w2.copy_(words[1])
        sl.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for r, w in zip((r1, r2), words):
            check(*r, reference(q, val, table, new, w), kind)
    assert mla.get_status() == mla.MLA_OK


@pytest.mark.gpu
def test_offsets_past_32_bits(mla):
    """A bf16 pool of over 2^32 bytes and elements, with the request's pages at its end."""
    T, H, page, pages = 4, 16, 64, 120_000  # 4.4e9 elements, 8.8e9 bytes
    lens = [1000]
    words = random_tree(torch.Generator().manual_seed(3), 1, T)
    q, small, table, _, _, val = make(lens, T, H, page, "bf16", 4, extra=0)
    d = "cuda"
    pool = torch.zeros(pages, page, 576, dtype=torch.bfloat16, device=d)
    pool[pages - small.shape[0]:] = small.to(d)
    plan = mla.decode_tree_plan(lens, T, H, page, table.shape[1], pages)
    out, lse = mla.decode_tree(plan, q.to(d), pool, (table + pages - small.shape[0]).to(d),
                               torch.tensor(lens, dtype=torch.int32, device=d), words.to(d), SCALE)
    assert mla.get_status() == mla.MLA_OK
    check(out, lse, reference(q, val, table, lens, words), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,H", [("bf16", 3, 16), ("bf16", 6, 16), ("bf16", 20, 16), ("e4m3", 6, 16)])
@pytest.mark.parametrize("page", [8, 16, 32, 128])
def test_not_finite_rows_and_bad_pages_at_other_page_sizes(mla, kind, T, H, page):
    """NaN drafts and NaN behind the requests' ends, and page ids outside the pool for one of them."""
    lens = [64 + 2 + T, 500, 259]
    g = torch.Generator().manual_seed(page)
    words = random_tree(g, 3, T)
    words[:, 2:] &= ~2  # only draft 1 sees draft 1
    words[:, 0] &= ~2

    def spoil(q, pool, table, val):
        for b, L in enumerate(lens):
            for j in [L - T + 1] + list(range(L, -(-L // page) * page)):
                pool[table[b, j // page], j % page] = math.nan if kind == "bf16" else 0x7F
                val[table[b, j // page], j % page] = 0.0

    out, lse, ref, plan = run(mla, lens, T, H, page, kind, words, seed=5, tweak=spoil)
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all()
    keep = [t for t in range(T) if t != 1]
    ref = tuple(x[:, keep] for x in ref)
    check(out[:, keep], lse[:, keep], ref, kind)
    q, pool, table, scales, kv_scale, val = make(lens, T, H, page, kind, 5)
    spoil(q, pool, table, val)
    table[0, 0], table[1, 2] = pool.shape[0] + 3, -1
    d = "cuda"
    out, lse = mla.decode_tree(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d),
                               words.to(d), SCALE, kv_scale)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    check(out[2:, keep], lse[2:, keep], tuple(x[2:] for x in ref), kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,H", [("bf16", 2, 16), ("bf16", 3, 16), ("bf16", 4, 16), ("bf16", 8, 16), ("e4m3", 8, 16),
                                       ("int8", 4, 16)])
def test_an_ordinary_plan_with_a_trees_workspace(mla, kind, T, H):
    lens = [4000, 300, 77]
    words = random_tree(torch.Generator().manual_seed(6), 3, T)
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 6)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind])
    rows = 3 * plan.max_splits * T * H
    assert plan.max_splits > 1
    ws = torch.empty(256 + rows * (512 * (4 if kind == "bf16" else 2) + 4), dtype=torch.uint8, device=d)
    args = (q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), words.to(d), SCALE, kv_scale)
    out, lse = mla.decode_tree(plan, *args, workspace=ws)
    assert mla.get_status() == mla.MLA_OK
    check(out, lse, reference(q, val, table, lens, words), kind)
    with pytest.raises(mla.MlaError) as e:
        mla.decode_tree(plan, *args, workspace=ws[:-256])
    assert e.value.code == mla.MLA_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(3, 8), (3, 16), (4, 16), (6, 16), (20, 16), (64, 2)])  # 24, 48, 64, 96, 320, 128 rows
@pytest.mark.parametrize("page,sms", [(64, 1), (64, 0), (8, 0), (128, 0)])
def test_one_infinity_in_a_draft_reaches_those_that_see_it(mla, T, H, page, sms):
    """An infinite value whose score is -infinity has weight 0, and 0 x infinity is NaN in its column, in
    the rows that see it and no other; in the rotated columns it is no value, and the key alone is lost."""
    lens = [576 + T, 500, 130 + T, 64 + T]
    words = random_tree(torch.Generator().manual_seed(T), 4, T)
    words[:, 2:] &= ~2  # draft 1 is seen by itself and, where there is one, by the last draft alone
    words[:, 0] &= ~2
    words[:, T - 1] |= 2
    # request: column and value of draft 1; the last request's infinity lies in its prefix, which all see
    where = [(5, math.inf, None), (300, -math.inf, None), (540, math.inf, None), (511, math.inf, 10)]

    def spoil(q, pool, table, val):
        q[..., ::2, :] = q[..., ::2, :].abs()       # even heads: the score has the infinity's sign
        q[..., 1::2, :] = -q[..., 1::2, :].abs()
        q[q == 0] = 0.01
        for b, (c, v, j) in enumerate(where):
            j = lens[b] - T + 1 if j is None else j
            pool[table[b, j // page], j % page, c] = v
            val[table[b, j // page], j % page, c] = 0.0

    q, pool, table, scales, kv_scale, val = make(lens, T, H, page, "bf16", 3)
    spoil(q, pool, table, val)
    plan = mla.decode_tree_plan(lens, T, H, page, table.shape[1], pool.shape[0], 0, sms)
    d = "cuda"
    out, lse = mla.decode_tree(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), words.to(d),
                               SCALE)
    assert mla.get_status() == mla.MLA_OK
    out, lse = out.cpu(), lse.cpu()
    # rows whose score is -infinity give the key no weight: the reference without it
    ref = list(reference(q, val, table, lens, words & ~2))
    for b, (c, v, j) in enumerate(where):
        sees = ((words[b] >> 1) & 1).bool() if j is None else torch.ones(T, dtype=torch.bool)
        up = torch.arange(H) % 2 == (0 if v > 0 else 1)
        lost = sees[:, None] & up[None]             # a score of +infinity
        some = sees[:, None] & ~up[None]            # a score of -infinity
        assert torch.isnan(out[b][lost]).all() and not torch.isfinite(lse[b][lost]).any()
        if j is not None:  # without the prefix key: its weight is exp(-infinity)
            rows = rows_of(val, table, b, lens[b])
            x = (q[b].double().reshape(T * H, 576) @ rows.T * SCALE).view(T, H, -1)
            x[..., j] = -math.inf
            for t in range(T):
                for u in range(T):
                    if not (int(words[b, t]) >> u) & 1:
                        x[t, :, lens[b] - T + u] = -math.inf
            ref[1][b] = torch.logsumexp(x, -1)
            w = torch.exp(x - ref[1][b][..., None])
            ref[0][b] = w @ rows[:, :512]
            ref[2][b] = w @ rows[:, :512].abs()
        if c < 512:
            assert torch.isnan(out[b, :, :, c][some]).all()
            out[b, :, :, c] = torch.where(some, ref[0][b, :, :, c].to(out.dtype), out[b, :, :, c])
        keep = ~lost
        check(out[b][keep], lse[b][keep], tuple(r[b][keep] for r in ref), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,H", [("bf16", 2, 16), ("bf16", 3, 16), ("bf16", 5, 16), ("bf16", 8, 16), ("bf16", 12, 16),
                                       ("e4m3", 8, 16), ("int8", 5, 16)])
def test_an_ordinary_decode_on_a_trees_plan(mla, kind, T, H):
    """mla_decode accepts the plan of a tree, whose chunks and launch order a pair's cost chose."""
    lens = [9000, 300, 77 + T] + [500 + 64 * i for i in range(20)]
    words = torch.tensor([[(2 << t) - 1 for t in range(T)]] * len(lens))
    q, pool, table, scales, kv_scale, val = make(lens, T, H, 64, kind, 7)
    d = "cuda"
    for sms in (0, 8):
        plan = mla.decode_tree_plan(lens, T, H, 64, table.shape[1], pool.shape[0], KINDS[kind], sms)
        out, lse = mla.decode(plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d), SCALE, kv_scale)
        assert mla.get_status() == mla.MLA_OK
        ref = reference(q, val, table, lens, words)
        # (bf16 partials of a split request: one more rounding, 2^-8 of the weighted values)
        assert ((lse.cpu().double() - ref[1]).abs() <= 2.0 ** -17 * ref[3] + ref[4] + 2.0 ** -20 * (1 + ref[1].abs())).all()
        tol = 2.0 ** -8 * ref[0].abs() + (2.0 ** -7 + 2 * (2.0 ** -17 * ref[3] + ref[4])[..., None] + 2.0 ** -17) * ref[2] + ref[5][..., None]
        assert ((out.cpu().double() - ref[0]).abs() <= tol).all()
