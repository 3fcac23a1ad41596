"""The weights of a decode over a 4-bit pool when a few keys stand far above the others.

A heavy key's values are zero here (an attention sink), so the output is what the others add up to, and all of their
values have one sign, so that what is lost of them shows.  Outputs are compared with 64-bit arithmetic on the values
that the codes stand for.  Tolerances, of non-negative terms w_j v_j:
  * a weight is carried as hi + lo / 28, both e4m3, of its f16 value: hi is off by at most 2^-4, lo by at most 2^-5 of that
    residual's binade top, together 2^-9 of the weight; 2^-11 for the f16; as much as these once more for what a sum of
    them may differ from the rounded terms' (the sum that divides them is of the unrounded weights);
  * below lo's normal range it is off by at most half of lo's last step, 2^-10 / 28 < 2^-14.8, in units in which a tile's
    largest weight is at least 2^-5, so 2^-9.8 of that, once the reference has followed it down: by 2^8 after two tiles below
    2^-5 and one that goes by.  Beside a heavy key, which is 448 in these units, and in the three tiles behind it, that is
    2^-23.6 of its weight, 2^-8 of that in the next three, and so on.  Of several at one height the least weight is 40, and
    references that have come up again wait for more tiles: 2^-20.1 up to the next heavy key.
    And it is never off by more than itself: what is carried is between 0 and twice the weight;
  * the output's rounding 2^-8, a split's f16 partial 2^-11 and 2^-25 of the codes' unit;
  * scores: A = scale sum_i |q_i k_i|, the largest of any key: 36 accumulation steps 2^-17 A, the query's split at most
    2^-18 max|q| for each element that is not zero; a score off by d moves the output by 2 d, lse by d;
  * lse: 2^-20 (1 + |lse|), the sums' (n / 128 + 16) 2^-24, and 2^-22 for each reference that moves.
"""
import math

import pytest
import torch

import fp4_rows

SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 6.0 / 448.0
HEAVY = 256.0  # columns 0-15 of a heavy key, in units of KV_SCALE


@pytest.fixture(scope="module")
def mla():
    from mla_attention_paged_gb300 import build
    build.build()
    from mla_attention_paged_gb300 import mla as m
    return m


def inputs(n, H, gaps, sigma, seed, T=1, without=()):
    """n keys, those of `gaps` that many (log2) above scores that are even or of deviation sigma (nats).  Rows
    `without` do not see the heavy keys' height."""
    g = torch.Generator().manual_seed(seed)
    some = min(n, 4096)
    x = torch.zeros(some, 576)
    x[:, 16:512] = (torch.rand(some, 496, generator=g) + 0.5) / KV_SCALE
    x[:, 512] = torch.randn(some, generator=g) / KV_SCALE
    rows = fp4_rows.encode(x)
    k = fp4_rows.values(rows).repeat(-(-n // some), 1)[:n].clone()
    rows = rows.repeat(-(-n // some), 1)[:n].clone()
    y = torch.zeros(len(gaps), 576)
    top = max(gaps.values(), default=0.0)
    for i, gap in enumerate(gaps.values()):
        y[i, :16] = HEAVY * gap / top
    if gaps:
        rows[list(gaps)] = fp4_rows.encode(y)
        k[list(gaps)] = fp4_rows.values(fp4_rows.encode(y))
    pages = -(-n // 64)
    pool = torch.cat([rows, torch.zeros(pages * 64 - n, 336, dtype=torch.uint8)]).view(pages, 64, 336)
    q = torch.zeros(1, T, H, 576)
    q[..., :16] = top * math.log(2.0) / (SCALE * KV_SCALE * HEAVY * 16)
    q.view(T * H, 576)[list(without), :16] = 0
    q[..., 512] = sigma / SCALE
    q *= torch.linspace(1.0, 0.95, H)[:, None]
    return q.bfloat16(), pool, torch.arange(pages, dtype=torch.int32)[None], k * KV_SCALE


def floors(w, v, heavy):
    """What weights w [H, n] may lose below their range, times v."""
    H, n = w.shape
    tiles = -(-n // 128)
    per = torch.zeros(H, tiles * 128, dtype=torch.float64, device=w.device)
    per[:, :n] = w
    floor = per.view(H, tiles, 128).amax(-1) * 2.0 ** -9.8
    for j in heavy:
        for t in range(j // 128, min(tiles, j // 128 + 19)):
            down = max(0, t - j // 128 - 1) // 3 * 8
            floor[:, t] = torch.maximum(floor[:, t], per[:, j] * 2.0 ** (-23.6 - down if len(heavy) == 1 else -20.1))
    for j in heavy:
        others = (w[:, j // 128 * 128:(j // 128 + 1) * 128] * 1.0)
        others[:, j % 128] = 0
        top = per[:, j] * 2.0 ** (-23.6 if len(heavy) == 1 else -20.1)
        floor[:, j // 128] = torch.maximum(top, others.amax(-1) * 2.0 ** -9.8)
    floor = floor.repeat_interleave(128, 1)[:, :n]
    return torch.minimum(floor, w) @ v


def run(mla, n, H, gaps, sigma, sms=1, tree=False, seed=3, T=1, without=()):
    q, pool, table, k = inputs(n, H, gaps, sigma, seed, T, without)
    pages = pool.shape[0]
    plan = (mla.decode_tree_plan if tree else mla.decode_plan)([n], T, H, 64, pages, pages, mla.MLA_KV_FP4, sms)
    assert sms != 1 or plan.max_splits == 1
    d = "cuda"
    a = (plan, q.to(d), pool.to(d), table.to(d), torch.tensor([n], dtype=torch.int32, device=d))
    if tree:
        out, lse = mla.decode_tree(*a, torch.tensor([[(2 << t) - 1 for t in range(T)]], device=d), SCALE, KV_SCALE)
    else:
        out, lse = mla.decode(*a, SCALE, KV_SCALE)
    assert mla.get_status() == mla.MLA_OK
    # 64 bits
    k = k.to(d)
    qd = q[0].double().view(T * H, 576).to(d)
    x = qd @ k.T * SCALE
    x = x.masked_fill(torch.arange(n, device=d) > n - T + torch.arange(T * H, device=d)[:, None] // H, -math.inf)
    ref_lse = torch.logsumexp(x, -1)
    w = torch.exp(x - ref_lse[:, None])
    v = k[:, :512]
    ref = w @ v
    floor = floors(w, v, list(gaps))
    dx = 2.0 ** -17 * SCALE * (qd.abs() @ k.abs().T).amax(-1) + SCALE * 2.0 ** -18 * qd.abs().amax(-1) * k[:, :16].abs().sum(1).max()
    tol = (2.0 ** -8 + 2 * (2.0 ** -9 + 2.0 ** -11) + 2.0 ** -11 + 2 * dx[:, None]) * ref + floor + 2.0 ** -25 * KV_SCALE
    moves = 2 * len(gaps) + 64
    tol_l = dx + 2.0 ** -20 * (1 + ref_lse.abs()) + (n / 128 + 16) * 2.0 ** -24 + moves * 2.0 ** -22
    got, got_l = out[0].double().view(T * H, 512), lse[0].double().view(T * H)
    tail = slice(16, 512)
    worst = ((got - ref).abs() / tol)[:, tail].max()
    print(f"tail's share {1 - float(w[0, list(gaps)].sum()):.3g}: off by {float(((got - ref).abs() / ref)[:, tail].max()):.4f} of itself, "
          f"{float(worst):.2f} of the tolerance ({float((tol / ref)[:, tail].max()):.4f}), splits {plan.max_splits}")
    assert worst <= 1
    assert ((got - ref).abs()[:, :16] <= (2.0 ** -7 + 2 * dx[:, None]) * ref[:, :16] + tol[:, 16:].amax(1, True)).all()
    assert ((got_l - ref_lse).abs() <= tol_l).all(), ((got_l - ref_lse).abs() / tol_l).max()


def gap(n, share):
    return math.log2(n * share / (1 - share))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("sigma", [0.0, 1.0])
@pytest.mark.parametrize("n,share", [(300, 0.99), (4096, 0.5), (4096, 0.99), (20001, 0.9), (20001, 0.99), (20001, 0.9999), (131071, 0.5), (131071, 0.9), (131071, 0.999)])
@pytest.mark.parametrize("where", ["first", "inside", "last"])
def test_a_sink_leaves_the_others_their_share(mla, H, sigma, n, share, where):
    at = {"first": 0, "inside": n // 3, "last": n - 1}[where]
    run(mla, n, H, {at: gap(n, share)}, sigma)


@pytest.mark.gpu
@pytest.mark.parametrize("H,tree", [(16, True), (32, True), (40, False)])
@pytest.mark.parametrize("sms", [1, 3, 152])
def test_a_sink_in_any_split(mla, H, tree, sms):
    for at in (0, 7000, 20000):
        run(mla, 20001, H, {at: gap(20001, 0.99)}, 0.5, sms, tree)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("step", [1, 2, 3, 7])
def test_references_that_go_up_and_down_again(mla, H, step):
    """A heavy key in every step-th tile: the reference goes up there and down in the next tile, if that has none."""
    n = 128 * 60 + 5
    total = gap(n, 0.9) - math.log2(60 / step)
    run(mla, n, H, {128 * t + 17 * t % 128: total - 0.02 * t for t in range(0, 60, step)}, 0.3)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(2, 8), (2, 16), (5, 16), (6, 7)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n", [200, 1300, 128 * 31 + 1])
def test_rows_of_drafts_with_and_without_a_sink(mla, T, H, tree, n):
    """Some rows' references go down while others' stay; the last tiles hold drafts that rows do not see."""
    without = [r for r in range(T * H) if r % 3 == 1]
    for at in (0, n // 2, n - T):
        for sms in (1, 152):
            run(mla, n, H, {at: gap(n, 0.99)}, 0.5, sms, tree, T=T, without=without)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [200])
def test_a_chunk_of_drafts_behind_a_sink(mla, T):
    """Rows that see nothing of many of the last tiles."""
    run(mla, 900, 2, {3: gap(900, 0.99)}, 0.5, T=T)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("height", [30.0, 38.0, 41.0, 60.0, 100.0, 160.0])
def test_heights_beyond_what_sums_of_32_bits_hold(mla, H, height):
    """The others' share falls below what a sum of 32 bits holds, and below the depth to which references follow: whatever is
    left of them is finite, never negative and no more than their largest value times a bound of their share."""
    n = 3000
    q, pool, table, k = inputs(n, H, {100: height}, 0.5, 5)
    plan = mla.decode_plan([n], 1, H, 64, pool.shape[0], pool.shape[0], mla.MLA_KV_FP4, 1)
    d = "cuda"
    out, lse = mla.decode(plan, q.to(d), pool.to(d), table.to(d), torch.tensor([n], dtype=torch.int32, device=d), SCALE, KV_SCALE)
    assert mla.get_status() == mla.MLA_OK
    x = q[0, 0].double() @ k.T * SCALE
    ref_lse = torch.logsumexp(x, -1)
    w = torch.exp(x - ref_lse[:, None])
    ref = (w @ k[:, :512])[:, 16:]
    got = out[0, 0].double().cpu()[:, 16:]
    dx = 2.0 ** -16 * x.abs().amax(-1)
    assert got.isfinite().all() and (got >= 0).all()
    assert ((lse[0, 0].double().cpu() - ref_lse).abs() <= dx + 2.0 ** -20 * (1 + ref_lse.abs()) + 64 * 2.0 ** -22).all()
    # (and the depth: lo's last step at 2^40 below, n 2^-60)
    floor = floors(w, k[:, :512], [100])[:, 16:] + n * 2.0 ** -60 * k.max()
    assert ((got - ref).abs() <= (2.0 ** -6 + 2 * dx[:, None]) * ref + floor).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 16), (2, 16), (6, 16)])
def test_moving_references_agree_to_the_bit(mla, T, H):
    """The same call 100 times, references going up and down in every few tiles of some rows."""
    n = 128 * 30
    heavy = {128 * t + 5: gap(n, 0.9) for t in (0, 2, 3, 8, 13, 21)}
    q, pool, table, _ = inputs(n, H, heavy, 0.7, 9, T, [r for r in range(T * H) if r % 5 == 1])
    d = "cuda"
    a = (q.to(d), pool.to(d), table.to(d), torch.tensor([n], dtype=torch.int32, device=d), SCALE, KV_SCALE)
    for sms in (1, 4):
        plan = mla.decode_plan([n], T, H, 64, pool.shape[0], pool.shape[0], mla.MLA_KV_FP4, sms)
        first = mla.decode(plan, *a)
        differ = torch.zeros((), dtype=torch.int64, device=d)
        for _ in range(100):
            out, lse = mla.decode(plan, *a)
            differ += (out != first[0]).sum() + (lse != first[1]).sum()
        assert mla.get_status() == mla.MLA_OK and int(differ) == 0 and first[0].isfinite().all()
