"""Cases of the serving operators around the paged latent cache, with their plain forms.

Four operators of one decode step of a speculative MLA server:

  tree    attention of a tree of drafted tokens over the paged latent cache
  mass    the attention weight that each cached key received, accumulated over steps
  append  latent norm, position rotation of queries and keys, (quantised) write into the pages
  evict   the heaviest keys of every request, packed into new pages

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true,
through the public entry points of ``mla_attention_paged_gb300.mla``.
"""
import math

import torch

own = False

LATENT = 576   # 512 latent columns + 64 rotated ones
VALUE = 512    # the value is the first 512 latent columns
ROPE = 64
SCALE = 1.0 / math.sqrt(192.0)
E4M3_SCALE = 6.0 / 448.0
DECAY = 0.97
EPS = 1e-6
POSITIONS = 65536


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short context, a small draft tree: the latency of a verification step
        dict(name="tree one request", op="tree", batch=1, drafts=8, heads=16, short=1000, long=1000, page=64, kv="bf16"),
        # a handful of ragged requests on an 8-bit cache, trees of a dozen nodes
        dict(name="tree e4m3 ragged", op="tree", batch=4, drafts=12, heads=16, short=3001, long=12289, page=64, kv="e4m3"),
        # a full batch of long contexts with three drafts each: bound by reading the cache
        dict(name="tree long contexts", op="tree", batch=16, drafts=3, heads=16, short=8192, long=131072, page=64, kv="bf16"),
        # wide trees over long contexts: bound by the matrix products
        dict(name="tree wide", op="tree", batch=8, drafts=32, heads=16, short=20001, long=65536, page=64, kv="bf16"),
        # the weight of each key after a single-token step of one short request
        dict(name="mass one token", op="mass", batch=1, drafts=1, heads=16, short=1025, long=1025, page=64, kv="bf16", tree=False),
        # the same after a step with draft trees on an 8-bit cache
        dict(name="mass e4m3 tree", op="mass", batch=8, drafts=5, heads=16, short=2000, long=16001, page=64, kv="e4m3", tree=True),
        # a full batch of long contexts, two tokens a step
        dict(name="mass long contexts", op="mass", batch=16, drafts=2, heads=16, short=8192, long=131072, page=64, kv="bf16", tree=False),
        # a decode step of four requests: the rotated columns go into the absorbed queries
        dict(name="append decode", op="append", tokens=4, pad=0, heads=16, q_dim=64, q_norm=False, interleaved=True, page=64, kv="bf16"),
        # a padded draft batch into an 8-bit cache
        dict(name="append e4m3 drafts", op="append", tokens=257, pad=15, heads=16, q_dim=64, q_norm=False, interleaved=True, page=64, kv="e4m3"),
        # a prefill chunk with normed queries
        dict(name="append prefill", op="append", tokens=8191, pad=3, heads=16, q_dim=192, q_norm=True, interleaved=False, page=64, kv="bf16"),
        # one request shrunk to half its keys
        dict(name="evict one request", op="evict", batch=1, short=1999, long=1999, percent=50, sink=4, recent=64, page=64, kv="bf16"),
        # a batch of long contexts on an 8-bit cache, a fifth kept
        dict(name="evict long contexts", op="evict", batch=16, short=8192, long=131072, percent=20, sink=4, recent=512, page=64, kv="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "mass", "append", "evict"))
    top = {k: max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")}
    while True:
        c = _draw(rng, op)
        # no more than the largest listed cases of its kind, in bytes and in products
        if all(work(c)[k] <= top[k] for k in top):
            return c


def _draw(rng, op):
    kv = rng.choice(("bf16", "e4m3"))
    page = rng.choice((16, 32, 64, 64, 128))
    if op in ("tree", "mass"):
        drafts, long = _log(rng, 1, 64), _log(rng, 100, 131072)
        c = dict(op=op, batch=_log(rng, 1, 16), drafts=drafts, heads=rng.choice((4, 8, 16, 16, 32)),
                 short=max(drafts, _log(rng, max(long // 8, 50), long)), long=long, page=page, kv=kv)
        return dict(c, tree=rng.random() < 0.5) if op == "mass" else c
    if op == "append":
        tokens = _log(rng, 1, 8000)
        q_dim = rng.choice((64, 192))
        return dict(op=op, tokens=tokens, pad=rng.randint(0, tokens // 8), heads=rng.choice((8, 16, 16)), q_dim=q_dim,
                    q_norm=q_dim == 192 and rng.random() < 0.5, interleaved=rng.random() < 0.5, page=page, kv=kv)
    long = _log(rng, 200, 131072)
    return dict(op=op, batch=_log(rng, 1, 16), short=_log(rng, max(long // 8, 100), long), long=long, percent=rng.randint(3, 60),
                sink=rng.randint(0, 8), recent=_log(rng, 1, 60), page=page, kv=kv)


def _lens(c):
    """The requests' lengths: from the longest down to the shortest, evenly."""
    b = c["batch"]
    return [c["long"] - (c["long"] - c["short"]) * i // max(1, b - 1) for i in range(b)]


def _keeps(c):
    return [max(1, n * c["percent"] // 100) for n in _lens(c)]


def _row_bytes(c):
    return LATENT * (2 if c["kv"] == "bf16" else 1)


def work(c):
    if c["op"] in ("tree", "mass"):
        keys, rows = sum(_lens(c)), c["drafts"] * c["heads"]
        read = keys * _row_bytes(c) + c["batch"] * (rows * (LATENT * 2) + c["drafts"] * 8) + 4 * keys // c["page"]
        if c["op"] == "tree":
            return {"bytes": read + c["batch"] * rows * (VALUE * 2 + 4), "flops": 2 * (LATENT + VALUE) * rows * keys}
        return {"bytes": read + c["batch"] * rows * 4 + keys * 8, "flops": 2 * LATENT * rows * keys}
    if c["op"] == "append":
        n = c["tokens"]
        per = c["heads"] * c["q_dim"] * 4 + LATENT * 2 + _row_bytes(c) + ROPE * 4 + 12
        return {"bytes": n * per, "flops": n * (c["heads"] * c["q_dim"] + LATENT) * 4}
    keys, kept = sum(_lens(c)), sum(_keeps(c))
    return {"bytes": keys * 4 + kept * (2 * _row_bytes(c) + 8), "flops": keys}


# ------------------------------------------------------------------------------- inputs
def _paged(g, lens, page, spare=0):
    """A page table over one shared pool in random order, and the pool's page count."""
    need = [(n + page - 1) // page for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + spare, perm[at:]


def _pool(g, pages, page, kv):
    """Latent rows after their norm: about N(0, 1)."""
    pool = torch.empty(pages, page, LATENT, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (page * LATENT))
    for s in range(0, pages, step):
        x = torch.randn(min(step, pages - s), page, LATENT, generator=g, device="cuda")
        pool[s:s + step] = x.to(torch.bfloat16) if kv == "bf16" else (x / E4M3_SCALE).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def _tree_masks(g, batch, drafts):
    """Ancestor masks of random trees: bit u of [b, t] says that draft t sees draft u."""
    mask = torch.zeros(batch, drafts, dtype=torch.int64, device="cuda")
    for t in range(drafts):
        up = torch.zeros(batch, dtype=torch.int64, device="cuda")
        if t:
            parent = torch.randint(0, t, (batch,), generator=g, device="cuda")
            up = mask.gather(1, parent[:, None])[:, 0]
        mask[:, t] = up | (1 << t)
    return mask


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c, "kv_scale": 1.0 if c["kv"] == "bf16" else E4M3_SCALE}
    if c["op"] in ("tree", "mass"):
        lens, B, T, H = _lens(c), c["batch"], c["drafts"], c["heads"]
        s["table"], pages, _ = _paged(g, lens, c["page"])
        s["pool"] = _pool(g, pages, c["page"], c["kv"])
        s["q"] = torch.randn(B, T, H, LATENT, generator=g, device="cuda").to(torch.bfloat16)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["mask"] = _tree_masks(g, B, T) if c["op"] == "tree" or c["tree"] else None
        s["longest"] = max(lens)
        if c["op"] == "mass":
            # the log-sum-exp that the step's attention left: scores of N(0, 1) latents are normal
            s["lse"] = torch.log(s["lens"].float())[:, None, None] + 0.5 * (SCALE * s["q"].float().norm(dim=-1)) ** 2
            # what earlier steps of the same size have left behind
            level = T * H / (s["lens"].float()[:, None] * (1.0 - DECAY))
            s["mass"] = torch.rand(B, max(lens), generator=g, device="cuda") * 2.0 * level
        else:
            s["out"] = torch.empty(B, T, H, VALUE, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device="cuda")
        if own:  # a server plans a batch once per set of lengths and keeps its workspace
            from mla_attention_paged_gb300 import mla
            kind = mla.MLA_KV_BF16 if c["kv"] == "bf16" else mla.MLA_KV_E4M3
            args = (lens, T, H, c["page"], s["table"].shape[1], pages, kind)
            if c["op"] == "tree":
                s["plan"] = mla.decode_tree_plan(*args)
                s["ws"] = mla.workspace_for(s["plan"], "cuda")
            else:
                s["plan"] = mla.decode_plan(*args)
                s["ws"] = mla.key_mass_workspace_for(s["plan"], "cuda")
    elif c["op"] == "append":
        n, H = c["tokens"], c["heads"]
        s["q_src"] = torch.randn(n, H, 192, generator=g, device="cuda").to(torch.bfloat16)
        wide = c["q_dim"] == ROPE
        # absorbed queries hold 512 columns from a projection already; the rotated 64 come here
        s["q_dst"] = torch.randn(n, H, LATENT if wide else 192, generator=g, device="cuda").to(torch.bfloat16)
        s["q_in"] = s["q_src"][..., 128:] if wide else s["q_src"]
        s["q_out"] = s["q_dst"][..., VALUE:] if wide else s["q_dst"]
        s["kv"] = (torch.randn(n, LATENT, generator=g, device="cuda") * 2.0).to(torch.bfloat16)
        s["kv_weight"] = (1.0 + 0.1 * torch.randn(VALUE, generator=g, device="cuda")).to(torch.bfloat16)
        s["q_weight"] = (1.0 + 0.1 * torch.randn(192, generator=g, device="cuda")).to(torch.bfloat16) if c["q_norm"] else None
        s["pos"] = torch.randint(0, POSITIONS, (n,), generator=g, device="cuda", dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        pages = (n + c["page"] - 1) // c["page"] + 2
        s["pool"] = _pool(g, pages, c["page"], c["kv"])
        # the pool's last row belongs to no token; padded tokens have no slot
        s["slots"] = torch.randperm(pages * c["page"] - 1, generator=g, device="cuda")[:n].clone()
        s["slots"][n - c["pad"]:] = -1
    else:
        lens, keeps = _lens(c), _keeps(c)
        dst = [(n + c["page"] - 1) // c["page"] for n in keeps]
        s["table"], pages, free = _paged(g, lens, c["page"], sum(dst))
        s["dst_table"] = torch.zeros(len(lens), max(dst), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(dst):
            s["dst_table"][b, :n] = free[at:at + n]
            at += n
        s["pool"] = _pool(g, pages, c["page"], c["kv"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["keeps"] = torch.tensor(keeps, dtype=torch.int32, device="cuda")
        s["longest"], s["most"] = max(lens), max(keeps)
        # accumulated weights are heavy-tailed; some keys never got any
        m = torch.randn(len(lens), max(lens), generator=g, device="cuda").mul_(2.0).exp_()
        s["mass"] = torch.where(torch.rand(m.shape, generator=g, device="cuda") < 0.05, torch.zeros_like(m), m)
        s["kept"] = torch.zeros(len(lens), max(keeps), dtype=torch.int32, device="cuda")
        s["mass_out"] = torch.zeros(len(lens), max(keeps), device="cuda")
        s["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _rows_of(s):
    """Every request's latent rows in 32 bits, [B, longest, 576], with the slots they lie in."""
    page = s["case"]["page"]
    j = torch.arange(s["longest"], device="cuda")
    slot = s["table"].long()[:, j // page] * page + j % page
    flat = s["pool"].view(-1, LATENT)[slot]
    if s["case"]["kv"] == "bf16":
        return flat.float()
    return flat.view(torch.float8_e4m3fn).float() * E4M3_SCALE


def _seen(s):
    """[B, T, longest]: the keys that each draft sees."""
    T = s["case"]["drafts"]
    j = torch.arange(s["longest"], device="cuda")[None, None, :]
    first = (s["lens"].long() - T)[:, None, None]
    u = j - first
    if s["mask"] is None:
        t = torch.arange(T, device="cuda")[None, :, None]
        return u <= t
    bit = (s["mask"][:, :, None] >> u.clamp(0, 63)) & 1
    return (u < 0) | ((u < T) & (bit == 1))


def _scores(s, rows):
    """[B, T, H, longest] scaled scores, -inf where a draft does not see the key."""
    B, T, H, _ = s["q"].shape
    x = (s["q"].float().view(B, T * H, LATENT) @ rows.transpose(1, 2)).view(B, T, H, -1) * SCALE
    return x.masked_fill(~_seen(s)[:, :, None, :], -math.inf)


def _plain_tree(s):
    rows = _rows_of(s)
    x = _scores(s, rows)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    B, T, H, n = p.shape
    o = (p.view(B, T * H, n) @ rows[..., :VALUE]).view(B, T, H, VALUE) / total
    s["out"].copy_(o)
    s["lse"].copy_((top + torch.log(total))[..., 0])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_mass(s):
    x = _scores(s, _rows_of(s))
    got = torch.exp(x - s["lse"][..., None]).sum((1, 2))
    inside = torch.arange(s["longest"], device="cuda")[None, :] < s["lens"][:, None]
    s["mass"].copy_(torch.where(inside, s["mass"] * DECAY + got, s["mass"]))
    return {"mass": s["mass"]}


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_append(s):
    c = s["case"]
    both = s["cos_sin"][s["pos"].long()]
    cos, sin = both[:, :ROPE // 2], both[:, ROPE // 2:]
    q = s["q_in"].float()
    if s["q_weight"] is not None:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_weight"].float()
    q = torch.cat([q[..., :-ROPE], _rotate(q[..., -ROPE:], cos[:, None], sin[:, None], c["interleaved"])], -1)
    s["q_out"].copy_(q)
    x = s["kv"].float()
    latent = x[:, :VALUE]
    latent = latent / torch.sqrt((latent * latent).mean(-1, keepdim=True) + EPS) * s["kv_weight"].float()
    row = torch.cat([latent, _rotate(x[:, VALUE:], cos, sin, c["interleaved"])], -1)
    if c["kv"] == "bf16":
        row = row.to(torch.bfloat16)
    else:
        row = (row / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    flat = s["pool"].view(-1, LATENT)
    last = flat[-1].clone()  # padded tokens go to the row of no token, which is put back
    flat.index_copy_(0, torch.where(s["slots"] < 0, flat.shape[0] - 1, s["slots"]), row)
    flat[-1] = last
    return {"q": s["q_dst"], "pool": _values(s)}


def _plain_evict(s):
    c = s["case"]
    page, n, most = c["page"], s["longest"], s["most"]
    j = torch.arange(n, device="cuda")[None, :]
    lens, keep = s["lens"].long()[:, None], torch.minimum(s["keeps"], s["lens"]).long()[:, None]
    sink = keep.clamp(max=c["sink"])
    recent = torch.minimum(torch.full_like(keep, c["recent"]), keep - sink)
    weight = torch.where((j < sink) | (j >= lens - recent), math.inf, s["mass"])
    weight = torch.where(j < lens, weight, -math.inf)
    order = torch.sort(weight, dim=1, descending=True, stable=True).indices  # equal ones: the lowest index first
    chosen = torch.zeros(weight.shape, dtype=torch.bool, device="cuda")
    chosen.scatter_(1, order, j.expand_as(order) < keep)
    # kept keys in their order, then the others
    at = torch.sort(torch.where(chosen, j, j + n), dim=1).values[:, :most]
    i = torch.arange(most, device="cuda")[None, :]
    here = i < keep
    at = torch.where(here, at, 0)
    s["kept"].copy_(torch.where(here, at.int(), s["kept"]))
    s["mass_out"].copy_(torch.where(here, s["mass"].gather(1, at), s["mass_out"]))
    s["new_lens"].copy_(keep[:, 0])
    flat = s["pool"].view(-1, LATENT)
    src = s["table"].long().gather(1, at // page) * page + at % page
    dst = s["dst_table"].long().gather(1, (i // page).expand_as(at)) * page + i % page
    # places past a request's last kept key repeat its first one
    first_src, first_dst = src[:, :1].expand_as(src), dst[:, :1].expand_as(dst)
    flat.index_copy_(0, torch.where(here, dst, first_dst).flatten(), flat[torch.where(here, src, first_src).flatten()])
    return {"kept": s["kept"], "lens": s["new_lens"], "mass": s["mass_out"], "pool": _values(s)}


def _values(s):
    """The pool as the values it stands for (8-bit codes without their scale)."""
    return s["pool"] if s["case"]["kv"] == "bf16" else s["pool"].view(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        return {"tree": _plain_tree, "mass": _plain_mass, "append": _plain_append, "evict": _plain_evict}[c["op"]](s)
    from mla_attention_paged_gb300 import mla
    if c["op"] == "tree":
        mla.decode_tree(s["plan"], s["q"], s["pool"], s["table"], s["lens"], s["mask"], SCALE, s["kv_scale"],
                        out=s["out"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        mla.key_mass(s["plan"], s["q"], s["pool"], s["table"], s["lens"], s["lse"], s["mass"], SCALE, s["kv_scale"],
                     tree_mask=s["mask"], decay=DECAY, workspace=s["ws"])
        return {"mass": s["mass"]}
    kind = mla.MLA_KV_BF16 if c["kv"] == "bf16" else mla.MLA_KV_E4M3
    if c["op"] == "append":
        mla.kv_append(s["q_in"], s["kv"], s["pos"], s["slots"], s["cos_sin"], s["pool"], kv_weight=s["kv_weight"],
                      q_weight=s["q_weight"], eps=EPS, interleaved=c["interleaved"], kv_dtype=kind,
                      kv_scale=s["kv_scale"], q_out=s["q_out"])
        return {"q": s["q_dst"], "pool": _values(s)}
    mla.kv_evict(s["pool"], s["table"], s["lens"], s["keeps"], s["mass"], s["dst_table"], sink=c["sink"],
                 recent=c["recent"], max_seq_len=s["longest"], max_keep=s["most"], kv_dtype=kind,
                 kept=s["kept"], new_lens=s["new_lens"], mass_out=s["mass_out"])
    return {"kept": s["kept"], "lens": s["new_lens"], "mass": s["mass_out"], "pool": _values(s)}


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 9e12:  # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    c = s["case"]
    page = c["page"]
    flat = s["pool"].view(-1, LATENT)

    def values(rows):
        return rows.double() if c["kv"] == "bf16" else rows.view(torch.float8_e4m3fn).double()

    if c["op"] in ("tree", "mass"):
        T, H = c["drafts"], c["heads"]
        out = torch.zeros(c["batch"], T, H, VALUE, dtype=torch.float64, device="cuda")
        lse = torch.zeros(c["batch"], T, H, dtype=torch.float64, device="cuda")
        mass = s["mass"].double() if c["op"] == "mass" else None
        for b, n in enumerate(_lens(c)):
            pages = s["table"][b, :(n + page - 1) // page].long()
            keys = values(s["pool"][pages].reshape(-1, LATENT)[:n]) * s["kv_scale"]
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for t in range(T):
                if s["mask"] is None:
                    ids = torch.arange(n - T + t + 1, device="cuda")
                else:
                    m = int(s["mask"][b, t]) & ((1 << 64) - 1)
                    ids = torch.tensor(list(range(n - T)) + [n - T + u for u in range(T) if m >> u & 1], device="cuda")
                seen = keys[ids]
                x = s["q"][b, t].double() @ seen.T * SCALE
                if c["op"] == "mass":
                    got.index_add_(0, ids, torch.exp(x - s["lse"][b, t].double()[:, None]).sum(0))
                else:
                    lse[b, t] = torch.logsumexp(x, 1)
                    out[b, t] = torch.exp(x - lse[b, t][:, None]) @ seen[:, :VALUE]
            if c["op"] == "mass":
                mass[b, :n] = mass[b, :n] * DECAY + got
        return {"mass": mass} if c["op"] == "mass" else {"out": out, "lse": lse}
    pool = values(flat)
    if c["op"] == "append":
        half = ROPE // 2
        pair = torch.arange(half, device="cuda")
        even, odd = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + half)

        def turned(x):
            z = torch.complex(x[..., even], x[..., odd])
            f = s["cos_sin"].double()[s["pos"].long()]
            w = torch.complex(f[:, :half], f[:, half:])
            z = z * (w[:, None] if x.dim() == 3 else w)
            y = torch.empty_like(x)
            y[..., even], y[..., odd] = z.real, z.imag
            return y

        def normed(x, weight):
            return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()

        q, dst = s["q_in"].double(), s["q_dst"].double()
        if s["q_weight"] is not None:
            q = normed(q, s["q_weight"])
        dst[..., -c["q_dim"]:-ROPE] = q[..., :-ROPE]
        dst[..., -ROPE:] = turned(q[..., -ROPE:])
        rows = torch.cat([normed(s["kv"][:, :VALUE].double(), s["kv_weight"]), turned(s["kv"][:, VALUE:].double())], 1)
        if c["kv"] == "e4m3":
            rows = (rows / s["kv_scale"]).clamp(-448, 448)
        real = s["slots"] >= 0
        pool[s["slots"][real]] = rows[real]
        return {"q": dst, "pool": pool}
    mass = s["mass_out"].double()
    for b, (n, k) in enumerate(zip(_lens(c), _keeps(c))):
        k = min(n, k)
        first = min(c["sink"], k)
        tail = min(c["recent"], k - first)
        middle = s["mass"][b, first:n - tail].double().cpu().numpy()
        heavy = sorted((-middle).argsort(kind="stable")[:k - first - tail].tolist())
        ids = torch.tensor(list(range(first)) + [first + i for i in heavy] + list(range(n - tail, n)), device="cuda")
        i = torch.arange(k, device="cuda")
        mass[b, :k] = s["mass"][b, ids].double()
        pool[s["dst_table"][b].long()[i // page] * page + i % page] = values(flat[s["table"][b].long()[ids // page] * page + ids % page])
    return {"kept": None, "lens": None, "mass": mass, "pool": pool}
