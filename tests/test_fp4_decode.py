"""mla_decode and mla_decode_tree over a 4-bit pool.

The refusals run on the CPU.  The GPU cases compare every output with the definition in 64 bits on the
values that the pool's codes stand for.  Tolerances, with w_j the exact weights and W = sum_j w_j |v_j|:
  * the output's own rounding, 2^-8 |out|, and 2^-11 W for a split's f16 partial;
  * a weight is carried as hi + lo / 28, both e4m3: hi is off by at most 2^-4, lo by at most 2^-5 of that
    residual's binade top, together 2^-9 of the weight, and by 2^-11 from the f16 value that is split; with as
    much for what the normalisation adds, 2^-8 + 2^-10 of W; below e4m3's normal
    range the error is at most 2^-20 of the largest weight for each of the n keys, n 2^-20 max|v| w_max;
  * the scores: the keys are exact; 36 accumulation steps of the first product, each off by at most 2^-23
    of A = scale max_j sum_i |q_i k_ji| (2^-17 A in all), and the query split's 2^-17 max|q| per element,
    E = scale 2^-17 max|q| max_j sum_i |k_ji|.  A score off by d moves lse by d and the output by 2 d W;
  * lse: 2^-20 (1 + |lse|) for exponentials and logarithms, and (n / 128 + 16) 2^-24 for the sums.
"""
import ctypes
import math

import pytest
import torch

import fp4_rows

SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 6.0 / 448.0


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


# ------------------------------------------------------------------------------ the plain rows, and refusals
def test_rows_round_trip():
    """Every code under every exponent: values, and back to the same bytes (zero's exponent apart)."""
    n = 12
    mag = torch.arange(8).repeat(64).expand(n, 512).clone()
    neg = (torch.arange(512) // 8 % 2 == 1).expand(n, 512).clone()
    exp = torch.arange(n).int()[:, None].expand(n, 32).clone()
    rope = torch.arange(64).to(torch.uint8).expand(n, 64).clone()
    rows = fp4_rows.pack(mag.int(), neg, exp, rope)
    v = fp4_rows.values(rows)
    assert v[5, :8].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] and v[5, 13].item() == -3.0
    assert v[11, 7].item() == fp4_rows.TOP and v[0, 1].item() == 2.0 ** -6
    assert torch.equal(fp4_rows.encode(v), rows)


def _plan(mla, lens=(9000, 300), T=4, H=16, tree=False, sms=152):
    make = mla.decode_tree_plan if tree else mla.decode_plan
    return make(list(lens), T, H, 64, 200, 400, mla.MLA_KV_FP4, sms)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (1, 17), (2, 16), (4, 16), (20, 16)])
def test_plan_sizes_its_partials(mla, tree, T, H):
    plan = _plan(mla, T=T, H=H, tree=tree)
    rows = T * H
    assert plan.max_splits > 1 and plan.chunk_tokens % 128 == 0
    assert plan.head_groups == -(-rows // (16 if rows <= 16 else 32))
    parts = 2 * plan.max_splits * rows
    assert plan.workspace_bytes == 256 + parts * 512 * 2 + parts * 4


def _raw(mla, plan, **kw):
    a = dict(q=1 << 20, kv=1 << 21, pt=1 << 22, sl=1 << 23, T=plan.q_len, H=plan.num_heads,
             scale=0.07, kvs=1.0, out=1 << 24, lse=1 << 25, ws=1 << 26, wsb=plan.workspace_bytes)
    a.update(kw)
    return mla.lib.mla_decode(ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(out=None), 1), (dict(lse=None), 1),
    (dict(T=5), 1), (dict(H=15), 1), (dict(scale=0.0), 1), (dict(kvs=0.0), 1), (dict(ws=None), 1),
    (dict(q=(1 << 20) + 8), 1), (dict(kv=(1 << 21) + 4), 1), (dict(out=(1 << 24) + 8), 1), (dict(wsb=1000), 3)])
def test_invalid_arguments_are_refused(mla, bad, code):
    assert _raw(mla, _plan(mla), **bad) == code


def test_calls_that_do_not_take_the_format(mla):
    plan = _plan(mla)
    dummy = ctypes.c_void_p(1 << 20)
    assert mla.lib.mla_decode_int8_paged(ctypes.byref(plan), *[dummy] * 5, 4, 16, 0.07, 1.0, *[dummy] * 3, 1 << 30, None) == 1
    assert mla.lib.mla_key_mass(ctypes.byref(plan), dummy, dummy, None, dummy, dummy, None, dummy, 4, 16, 0.07, 1.0, 1.0, dummy,
                                1 << 20, None, 0, None) == 2


@pytest.mark.parametrize("shape,dtype", [((400, 64, 576), torch.uint8), ((400, 64, 336), torch.int8), ((400, 64, 288), torch.uint8)])
def test_binding_refuses_other_pools(mla, shape, dtype):
    plan = _plan(mla, tree=True)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(mla.MlaError) as e:
        mla.decode_tree(plan, torch.zeros(2, 4, 16, 576).bfloat16(), torch.zeros(shape, dtype=dtype), i, i, i, SCALE)
    assert e.value.code == mla.MLA_ERR_INVALID_ARG


def test_binding_refuses_pools_of_another_size(mla):
    """A pool of 8-bit rows under a 4-bit plan, one of 4-bit rows under another, and one of too few pages."""
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 16, 576).bfloat16()
    fp4, e4m3 = (torch.zeros(400, 64, n, dtype=torch.uint8) for n in (336, 576))
    plan = _plan(mla)
    other = mla.decode_plan([9000, 300], 4, 16, 64, 200, 400, mla.MLA_KV_E4M3, 152)
    for call in (mla.decode, mla.decode_partial, mla.decode_noalloc):
        for p, pool in ((plan, e4m3), (plan, fp4[:399]), (other, fp4), (other, e4m3[:399])):
            with pytest.raises(mla.MlaError) as e:
                call(p, q, pool, i, i, SCALE)
            assert e.value.code == mla.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ reference
def chain(B, T):
    """Drafts in order, as a tree's words."""
    w = [(2 << t) - 1 for t in range(T)]
    return torch.tensor([v - (1 << 64) if v >> 63 else v for v in w], dtype=torch.int64).expand(B, T).clone()


def random_tree(g, B, T):
    words = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            w = 1 << t
            if t:
                w |= int(words[b, int(torch.randint(0, t, (1,), generator=g))]) & ((1 << 64) - 1)
            words[b, t] = w - (1 << 64) if w >> 63 else w
    return words


def make(lens, T, H, page, seed, peaked=False, extra=3):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=g).int()
    table = torch.full((B, max(need)), -7, dtype=torch.int32)  # (entries past a request's end mean nothing)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    x = torch.randn(pages * page, 576, generator=g) / KV_SCALE
    # groups of very different sizes, among them some below the smallest exponent's range
    x[:, :512] *= (2.0 ** torch.randint(-10, 2, (pages * page, 32), generator=g).clamp(min=-8)).repeat_interleave(16, 1)
    pool = fp4_rows.encode(x).view(pages, page, 336)
    q = (torch.randn(B, T, H, 576, generator=g) * (8.0 if peaked else 1.0)).bfloat16()
    return q, pool, table


def reference(q, pool, table, lens, words):
    """out, lse and the tolerances' parts, in 64 bits."""
    B, T, H, _ = q.shape
    page = pool.shape[1]
    val = fp4_rows.values(pool) * KV_SCALE
    out = torch.zeros(B, T, H, 512, dtype=torch.float64)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64)
    W, A, E, n_sum = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse), torch.zeros_like(lse)
    small = torch.zeros_like(lse)
    for b, L in enumerate(lens):
        j = torch.arange(L)
        k = val[table[b].long()[j // page], j % page]
        x = q[b].double().reshape(T * H, 576) @ k.T * SCALE
        A[b] = ((q[b].double().abs().reshape(T * H, 576) @ k.abs().T).amax(1) * SCALE).view(T, H)
        E[b] = SCALE * 2.0 ** -17 * q[b].double().abs().amax(-1) * k.abs().sum(1).max()
        n_sum[b] = (L / 128 + 16) * 2.0 ** -24
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
        small[b] = L * 2.0 ** -20 * k.abs().max() * w.amax(-1)
    return out, lse, W, 2.0 ** -17 * A + E, small, n_sum


def check(got, glse, ref):
    out, lse, W, d, small, n_sum = ref
    got, glse = got.double().cpu(), glse.double().cpu()
    none = lse == -math.inf
    assert (glse[none] == -math.inf).all() and (got[none] == 0).all()
    tol_l = d + 2.0 ** -20 * (1 + lse.abs()) + n_sum
    assert ((glse - lse).abs() <= tol_l)[~none].all(), ((glse - lse).abs() / tol_l)[~none].max()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11 + 2 * d[..., None]) * W + small[..., None]
    bad = (got - out).abs() > tol
    assert not bad[~none].any(), ((got - out).abs() / tol)[~none].max()


def call(mla, plan, q, pool, table, lens, words, **kw):
    d = "cuda"
    a = (plan, q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d))
    got = mla.decode(*a, SCALE, KV_SCALE, **kw) if words is None else mla.decode_tree(*a, words.to(d), SCALE, KV_SCALE, **kw)
    return got


def run(mla, lens, T, H, page, words, seed=0, sms=0, peaked=False, tweak=None):
    q, pool, table = make(lens, T, H, page, seed, peaked)
    if tweak:
        tweak(q, pool, table)
    make_plan = mla.decode_plan if words is None else mla.decode_tree_plan
    plan = make_plan(lens, T, H, page, table.shape[1], pool.shape[0], mla.MLA_KV_FP4, sms)
    out, lse = call(mla, plan, q, pool, table, lens, words)
    assert mla.get_status() == mla.MLA_OK
    return out, lse, reference(q, pool, table, lens, chain(len(lens), T) if words is None else words), plan


CASES = [  # lens, T, H, page, SMs planned for (1: never split)
    ([1], 1, 1, 64, 1),
    ([1, 2, 127, 128, 129], 1, 16, 64, 1),
    ([31, 32, 33, 64, 65, 255, 256, 257], 1, 8, 8, 1),
    ([700], 1, 16, 64, 0),
    ([1000, 3000], 1, 16, 16, 0),
    ([5000, 129, 1], 1, 3, 128, 0),
    ([40, 1500], 1, 17, 32, 0),                # 17 rows: the 32-row kernel, half idle
    ([64, 130, 2000], 2, 16, 64, 0),           # 32 rows
    ([3, 384, 640], 3, 11, 256, 1),            # 33 rows: a second group of one
    ([130, 900, 2500], 4, 16, 64, 0),          # 64 rows
    ([77, 1290], 7, 16, 8, 0),
    ([200, 1111], 1, 128, 64, 0),
    ([300], 64, 5, 16, 0),
    ([1000], 200, 2, 64, 0),                   # a chunk of 200 new tokens, absorbed
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,H,page,sms", CASES)
def test_drafts_in_order(mla, lens, T, H, page, sms):
    q, pool, table = make(lens, T, H, page, sum(lens))
    plan = mla.decode_plan(lens, T, H, page, table.shape[1], pool.shape[0], mla.MLA_KV_FP4, sms)
    out, lse = call(mla, plan, q, pool, table, lens, None)
    assert mla.get_status() == mla.MLA_OK
    if T <= 64:
        check(out, lse, reference(q, pool, table, lens, chain(len(lens), T)))
    else:  # each draft as a request of its own length
        for t in (0, 1, T // 2, T - 1):
            ref = reference(q[:, t:t + 1], pool, table, [n - T + t + 1 for n in lens], chain(len(lens), 1))
            check(out[:, t:t + 1], lse[:, t:t + 1], ref)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [31, 33, 70, 512, 513])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 20)])
def test_batches(mla, B, T, H):
    """Many requests, two of them long: whole splits first up to 512 requests, beyond that in the orders of other pools."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(T, 140, (B,), generator=g).tolist()
    lens[B // 3], lens[B - 1] = 6000, 3333
    out, lse, ref, plan = run(mla, lens, T, H, 16, None, seed=B)
    assert plan.max_splits > 1 and (plan.split_major == 2) == (B <= 512)
    assert plan.num_splits == (sum(-(-n // plan.chunk_tokens) for n in lens) if B <= 512 else 0)
    check(out, lse, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 16), (2, 16), (3, 16)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,L", [(7, 2000), (40, 4500)])
def test_more_and_fewer_splits_than_planned(mla, T, H, tree, B, L):
    """Planned for one long request among short ones, run with all of them long: of 40 requests the grid has a CTA for each planned
    split, and CTAs take several.  And run with fewer splits than planned."""
    q, pool, table = make([L] * B, T, H, 16, 77)
    make_plan = mla.decode_tree_plan if tree else mla.decode_plan
    plan = make_plan([L] + [100] * (B - 1), T, H, 16, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
    assert plan.max_splits > 1 and plan.num_splits == plan.max_splits + B - 1
    words = chain(B, T) if tree else None
    for lens in ([L] * B, [L - 97 * i for i in range(B)], [50] * (B - 1) + [129]):
        out, lse = call(mla, plan, q, pool, table, lens, words)
        assert mla.get_status() == mla.MLA_OK
        check(out, lse, reference(q, pool, table, lens, chain(B, T)))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,H,page,sms", [c for c in CASES if c[1] <= 64])
def test_random_trees(mla, lens, T, H, page, sms):
    lens = [max(n, T) for n in lens]
    words = random_tree(torch.Generator().manual_seed(T * H), len(lens), T)
    out, lse, ref, _ = run(mla, lens, T, H, page, words, seed=sum(lens), sms=sms)
    check(out, lse, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(4, 4), (4, 8), (8, 16), (64, 4)])
def test_empty_rows_and_arbitrary_masks(mla, T, H):
    """Rows that see nothing, only a prefix, only others, or everything; bits past T are ignored."""
    g = torch.Generator().manual_seed(T)
    lens = [T, T + 1, 64 + T // 2, 128 + T // 2, 500]
    words = torch.randint(-(1 << 62), 1 << 62, (len(lens), T), generator=g)
    words[:, 0] = 0
    words[0, T // 2] = 0
    words[:, T - 1] = -1
    out, lse, ref, _ = run(mla, lens, T, H, 64, words, seed=9)
    assert (ref[1][0, 0] == -math.inf).all()
    check(out, lse, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 16), (2, 16), (6, 8), (6, 40)])
@pytest.mark.parametrize("tree", [False, True])
def test_splits_agree_and_peaked_scores(mla, T, H, tree):
    """Any split count, among them last splits that hold drafts alone; scores that move the running maximum often."""
    lens = [128 * 9 + T - 1, 2048 + 1, 640]
    words = random_tree(torch.Generator().manual_seed(1), len(lens), T) if tree else None
    for sms in (1, 4, 20, 152):
        out, lse, ref, plan = run(mla, lens, T, H, 32, words, seed=3, sms=sms, peaked=True)
        check(out, lse, ref)


@pytest.mark.gpu
def test_rising_scores(mla):
    """Each tile's scores exceed the last one's: every tile rescales what came before it."""
    lens, T, H = [128 * 20], 2, 16

    def rise(q, pool, table):
        x = torch.randn(lens[0], 576, generator=torch.Generator().manual_seed(1)) / KV_SCALE / 4
        x[:, 512:] = (torch.arange(lens[0]) / 60.0)[:, None] * q[0, 0, 0, 512:].float().sign()
        rows = fp4_rows.encode(x)
        pool.view(-1, 336)[(table[0].long()[:, None] * 64 + torch.arange(64)).view(-1)] = rows
    for sms in (1, 152):
        out, lse, ref, _ = run(mla, lens, T, H, 64, None, seed=5, sms=sms, tweak=rise)
        check(out, lse, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("share", [0.5, 0.99, 0.0])
@pytest.mark.parametrize("first", [0, 19999])
def test_a_heavy_key_and_an_even_tail(mla, H, share, first):
    """20000 keys of one score each and one key that takes `share` of the weight, first or last: the tail's weights are far
    below the largest, where few of their bits are carried."""
    n = 20001
    g = torch.Generator().manual_seed(3)
    x = torch.randn(n, 576, generator=g) / KV_SCALE
    x[:, :16] = 0
    x[:, 512:] = 0
    if share:
        x[first, :16] = 256.0
    pages = -(-n // 64)
    pool = fp4_rows.encode(torch.cat([x, torch.zeros(pages * 64 - n, 576)])).view(pages, 64, 336)
    q = torch.zeros(1, 1, H, 576)
    q[..., :16] = math.log(20000.0 * share / (1 - share)) / (SCALE * KV_SCALE * 256.0 * 16) if share else 0.0
    q = q.bfloat16()
    table = torch.arange(pages, dtype=torch.int32)[None]
    plan = mla.decode_plan([n], 1, H, 64, pages, pages, mla.MLA_KV_FP4)
    out, lse = call(mla, plan, q, pool, table, [n], None)
    ref = reference(q, pool, table, [n], chain(1, 1))
    check(out, lse, ref)
    # random signs of the values: far inside the bound, which adds every key's error up
    assert ((out.double().cpu() - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + 2.0 ** -7 * ref[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,page", [(1, 16, 64), (2, 16, 8), (6, 40, 32)])
def test_repeated_calls_agree_to_the_bit(mla, T, H, page):
    """Many row groups over the same pages (whose copies come back early from L2), 300 times."""
    lens = [128 * 9 + T - 1, 2049, 640]
    q, pool, table = make(lens, T, H, page, 3, True)
    d = "cuda"
    a = (q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d))
    for sms in (1, 20, 152):
        plan = mla.decode_plan(lens, T, H, page, table.shape[1], pool.shape[0], mla.MLA_KV_FP4, sms)
        first = mla.decode(plan, *a, SCALE, KV_SCALE)
        differ = torch.zeros((), dtype=torch.int64, device=d)
        for _ in range(100):
            out, lse = mla.decode(plan, *a, SCALE, KV_SCALE)
            differ += (out != first[0]).sum() + (lse != first[1]).sum()
        assert int(differ) == 0
        check(*first, reference(q, pool, table, lens, chain(3, T)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(3, 4), (3, 16), (6, 16)])
def test_not_finite_keys_reach_only_those_that_see_them(mla, T, H):
    """A draft whose rotated columns are NaN codes: NaN for the rows that see it, nothing for the others."""
    lens = [300, 64 + T]
    words = chain(2, T)

    def spoil(q, pool, table):
        for b, n in enumerate(lens):
            j = n - 1  # the last draft: seen by the last row alone
            pool[table[b, j // 16], j % 16, 272:] = 0x7F
    q, pool, table = make(lens, T, H, 16, 5)
    ref = reference(q, pool, table, lens, words)
    spoil(q, pool, table)
    for w in (None, words):
        plan = (mla.decode_plan if w is None else mla.decode_tree_plan)(lens, T, H, 16, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
        out, lse = call(mla, plan, q, pool, table, lens, w)
        assert mla.get_status() == mla.MLA_OK
        assert out[:, -1].isnan().all() and lse[:, -1].isnan().all()
        check(out[:, :-1], lse[:, :-1], tuple(x[:, :-1] for x in ref))


@pytest.mark.gpu
def test_queries_that_are_not_finite(mla):
    """Infinite or NaN queries make their own rows NaN; zero queries weigh every key alike."""
    lens, T, H = [400], 2, 16
    q, pool, table = make(lens, T, H, 64, 6)
    q[0, 0, 3, 7], q[0, 1, 5, 570], q[0, 1, 9] = math.inf, math.nan, 0.0
    clean = q.clone()
    clean[0, 0, 3, 7] = clean[0, 1, 5, 570] = 0.0
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
    out, lse = call(mla, plan, q, pool, table, lens, None)
    ref = reference(clean, pool, table, lens, chain(1, T))
    bad = torch.zeros(1, T, H, dtype=torch.bool)
    bad[0, 0, 3] = bad[0, 1, 5] = True
    assert out.cpu()[bad].isnan().all() and lse.cpu()[bad].isnan().all()
    check(out.cpu()[~bad], lse.cpu()[~bad], tuple(x[~bad] for x in ref))


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported(mla):
    lens, T, H = [500, 300, 260], 2, 16
    q, pool, table = make(lens, T, H, 16, 7)
    plan = mla.decode_plan(lens, T, H, 16, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
    d = "cuda"
    out, lse = torch.full((3, T, H, 512), 7.0, device=d).bfloat16(), torch.full((3, T, H), 7.0, device=d)
    ln = torch.tensor([501, 1, 260], dtype=torch.int32, device=d)
    mla.decode(plan, q.to(d), pool.to(d), table.to(d), ln, SCALE, KV_SCALE, out=out, lse=lse)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    assert (out[:2] == 7).all() and (lse[:2] == 7).all()
    ref = reference(q, pool, table, lens, chain(3, T))
    check(out[2:], lse[2:], tuple(x[2:] for x in ref))
    # a page outside the pool reads as zeros
    wild, zero = table.clone(), pool.clone()
    wild[1, 3], wild[2, 16], wild[0, 0] = pool.shape[0], -1, 1 << 30
    zero[table[1, 3]] = zero[table[2, 16]] = zero[table[0, 0]] = 0
    out, lse = call(mla, plan, q, pool, wild, lens, None)
    assert mla.get_status() == mla.MLA_ERR_DEVICE_ARG
    check(out, lse, reference(q, zero, table, lens, chain(3, T)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 16), (4, 16)])
def test_captured_calls_follow_the_device_inputs(mla, T, H):
    """A captured call replayed on other pages, queries and lengths; another stream; a partial and a combine apart."""
    lens = [700, 1300]
    q, pool, table = make(lens, T, H, 64, 8)
    d = "cuda"
    plan = mla.decode_plan(lens, T, H, 64, table.shape[1], pool.shape[0], mla.MLA_KV_FP4)
    a = [q.to(d), pool.to(d), table.to(d), torch.tensor(lens, dtype=torch.int32, device=d)]
    ws = mla.workspace_for(plan, d)
    out, lse = mla.decode(plan, *a, SCALE, KV_SCALE, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.decode(plan, *a, SCALE, KV_SCALE, out=out, lse=lse, workspace=ws)
    q2, pool2, _ = make(lens, T, H, 64, 9)
    less = [600, 1299]
    a[0].copy_(q2.to(d)), a[1].copy_(pool2.to(d)), a[3].copy_(torch.tensor(less, dtype=torch.int32))
    graph.replay()
    assert mla.get_status() == mla.MLA_OK
    ref = reference(q2, pool2, table, less, chain(2, T))
    check(out, lse, ref)
    first = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    mla.decode_partial(plan, *a, SCALE, KV_SCALE, out=out, lse=lse, workspace=ws, stream=s)
    mla.decode_combine(plan, a[3], out, lse, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    out2, lse2 = mla.decode_noalloc(plan, *a, SCALE, KV_SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out2, first) and torch.equal(lse2, lse)


@pytest.mark.gpu
def test_offsets_past_32_bits(mla):
    """Pages that lie behind 2^32 bytes of pool."""
    page, pages = 64, 220000  # 4.7e9 bytes
    lens, T, H = [300, 200], 2, 16
    q, small, table = make(lens, T, H, page, 11)
    pool = torch.zeros(pages, page, 336, dtype=torch.uint8, device="cuda")
    far = table + (pages - small.shape[0])
    pool[pages - small.shape[0]:] = small.cuda()
    plan = mla.decode_plan(lens, T, H, page, table.shape[1], pages, mla.MLA_KV_FP4)
    out, lse = mla.decode(plan, q.cuda(), pool, far.int().cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), SCALE, KV_SCALE)
    assert mla.get_status() == mla.MLA_OK
    check(out, lse, reference(q, small, table, lens, chain(2, T)))
