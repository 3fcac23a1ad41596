"""Cases of the 4-bit latent cache and of the page operators, with their plain forms.

Five operators of an MLA server whose latent cache lies in pages:

  decode   attention over a cache held in 4 bits: drafts in order, or a tree of them
  chunk    a prefill chunk: its keys quantised into the 4-bit pages, then all rows of the requests
           gathered out of the pages for the up-projection
  fork     requests continue as several: full pages shared, a partial last page copied
  free     requests shrink or end: pages that nothing refers to any more, in ascending order
  compact  the live pages move to the front of the pool, tables and counts follow

A row of the 4-bit pool is 336 bytes, all values in units of kv_scale:

  0..255    512 latent columns, eight in a 32-bit word: byte k holds the magnitudes of columns 2k and 2k+1
            in bits 0-2 and 4-6, the sign of column k in bit 7 and that of column 4+k in bit 3; magnitudes
            0, 1/2, 1, 3/2, 2, 3, 4, 6 times 2^(e-5)
  256..271  e of each 16 columns, 0..11, the lower nibble first
  272..335  64 rotated columns, e4m3

``run`` computes them with elementary torch operations, or, where ``own`` is true, through the public
entry points of ``mla_attention_paged_gb300.mla``.
"""
import math

import torch

own = False

LATENT = 576   # 512 latent columns + 64 rotated ones
VALUE = 512    # the value is the first 512 latent columns
ROPE = 64
FP4_ROW = 336
SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 6.0 / 448.0
EPS = 1e-6
POSITIONS = 65536
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short context, one token: the latency of a step
        dict(name="decode one request", op="decode", batch=1, drafts=1, heads=16, short=1000, long=1000, page=64, tree=False),
        # a handful of ragged requests with four drafts each
        dict(name="decode ragged drafts", op="decode", batch=4, drafts=4, heads=16, short=3001, long=12289, page=64, tree=False),
        # a full batch of long contexts, two tokens a step: bound by reading the cache
        dict(name="decode long contexts", op="decode", batch=16, drafts=2, heads=16, short=8192, long=131072, page=64, tree=False),
        # draft trees over long contexts
        dict(name="decode tree", op="decode", batch=8, drafts=8, heads=16, short=20001, long=65536, page=64, tree=True),
        # the first chunk of a short prompt behind a cached system prompt
        dict(name="chunk short", op="chunk", batch=1, new=37, prefix=700, pad=3, heads=16, page=64, interleaved=True),
        # four long prompts in chunks of two thousand
        dict(name="chunk long", op="chunk", batch=4, new=2047, prefix=14001, pad=0, heads=16, page=64, interleaved=False),
        # one prompt sampled four times
        dict(name="fork samples", op="fork", parents=1, children=4, short=2000, long=2000, page=64, kv="bf16"),
        # a step of a beam search that reorders 64 states
        dict(name="fork beams", op="fork", parents=64, children=64, short=8193, long=32768, page=64, kv="e4m3"),
        # a batch gives back the pages of its rejected drafts
        dict(name="free drafts", op="free", requests=16, freed=16, short=8192, long=131072, page=16, drop=64),
        # half of the requests end
        dict(name="free finished", op="free", requests=512, freed=256, short=1000, long=16000, page=16, drop=0),
        # a small pool after a burst
        dict(name="compact small", op="compact", requests=8, short=300, long=2000, spare=40, page=32, kv="e4m3"),
        # a large pool, half of it free
        dict(name="compact large", op="compact", requests=64, short=4000, long=20000, spare=100, page=64, kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "decode", "chunk", "fork", "free", "compact"))
    top = {k: max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")}
    while True:
        c = _draw(rng, op)
        # no more than the largest listed cases of its kind, in bytes and in products
        if all(work(c)[k] <= top[k] for k in top):
            return c


def _draw(rng, op):
    page = rng.choice((16, 32, 64, 64, 128))
    kv = rng.choice(("bf16", "e4m3"))
    if op == "decode":
        drafts, long = _log(rng, 1, 16), _log(rng, 100, 131072)
        return dict(op=op, batch=_log(rng, 1, 16), drafts=drafts, heads=rng.choice((4, 8, 16, 16, 32)),
                    short=max(drafts, _log(rng, max(long // 8, 50), long)), long=long, page=page, tree=rng.random() < 0.4)
    if op == "chunk":
        new = _log(rng, 1, 2000)
        return dict(op=op, batch=_log(rng, 1, 8), new=new, prefix=_log(rng, 1, 15000), pad=rng.randint(0, new // 8),
                    heads=rng.choice((8, 16, 16)), page=page, interleaved=rng.random() < 0.5)
    if op == "fork":
        long = _log(rng, 50, 32768)
        return dict(op=op, parents=_log(rng, 1, 64), children=_log(rng, 1, 64), short=_log(rng, max(long // 8, 20), long),
                    long=long, page=page, kv=kv)
    if op == "free":
        requests, long = _log(rng, 1, 512), _log(rng, 50, 16000)
        return dict(op=op, requests=requests, freed=_log(rng, 1, requests), short=_log(rng, max(long // 8, 20), long),
                    long=long, page=page, drop=rng.choice((0, rng.randint(1, 64))))
    long = _log(rng, 100, 20000)
    return dict(op=op, requests=_log(rng, 2, 64), short=_log(rng, max(long // 8, 50), long), long=long,
                spare=rng.randint(5, 100), page=page, kv=kv)


def _spread(n, short, long):
    """The requests' lengths: from the longest down to the shortest, evenly."""
    return [long - (long - short) * i // max(1, n - 1) for i in range(n)]


def _pages(n, page):
    return (n + page - 1) // page


def _row_bytes(c):
    return LATENT * (2 if c["kv"] == "bf16" else 1)


def _family(c):
    """Requests that share a prefix (free, compact): eight at a time, a quarter of the shortest one's whole pages."""
    return 8, c["short"] // 4 // c["page"]


def _kept(c, lens):
    """What the listed slots keep (free): all but their drafts, or nothing."""
    return [max(0, n - 1 - 7 * i % c["drop"]) if c["drop"] else 0 for i, n in enumerate(lens[:c["freed"]])]


def _total_pages(c):
    """Pages that the requests hold (free, compact), a shared one once."""
    lens = _spread(c["requests"], c["short"], c["long"])
    size, shared = _family(c)
    return sum(_pages(n, c["page"]) for n in lens) - shared * (len(lens) - _pages(len(lens), size))


def work(c):
    if c["op"] == "decode":
        keys, rows = sum(_spread(c["batch"], c["short"], c["long"])), c["drafts"] * c["heads"]
        per = rows * (LATENT * 2 + VALUE * 2 + 4) + (c["drafts"] * 8 if c["tree"] else 0)
        return {"bytes": keys * FP4_ROW + c["batch"] * per + 4 * keys // c["page"], "flops": 2 * (LATENT + VALUE) * rows * keys}
    if c["op"] == "chunk":
        n, rows = c["batch"] * c["new"], c["batch"] * (c["prefix"] + c["new"])
        per = c["heads"] * ROPE * 4 + LATENT * 2 + FP4_ROW + ROPE * 4 + 12
        return {"bytes": n * per + rows * (FP4_ROW + LATENT * 2), "flops": n * (c["heads"] * ROPE + LATENT) * 4 + rows * LATENT}
    page = c["page"]
    if c["op"] == "fork":
        lens = _spread(c["parents"], c["short"], c["long"])
        mean, rest = sum(lens) / len(lens) / page, sum(n % page for n in lens) / len(lens)
        return {"bytes": int(c["children"] * (16 * mean + 2 * rest * _row_bytes(c))), "flops": int(c["children"] * mean)}
    if c["op"] == "free":
        lens = _spread(c["requests"], c["short"], c["long"])
        dropped = sum(_pages(n, page) - _pages(k, page) for n, k in zip(lens, _kept(c, lens)))
        # (the plain answer is in ascending order: one look at each page's count)
        return {"bytes": 16 * dropped + 4 * int(1.3 * _total_pages(c)), "flops": dropped}
    live, share = _total_pages(c), 100 / (100 + c["spare"])
    entries = sum(_pages(n, page) for n in _spread(c["requests"], c["short"], c["long"]))
    moved = live * (1 - share)
    return {"bytes": int(2 * moved * page * _row_bytes(c) + 8 * entries + 4 * live / share), "flops": entries}


# ------------------------------------------------------------------------------- the 4-bit rows
def _encode(y):
    """Rows [n, 576] in units of kv_scale, 32 bits, as [n, 336] bytes."""
    n = y.shape[0]
    g = y[:, :VALUE].reshape(n, 32, 16)
    # the smallest power of two whose top step still rounds the group's largest value to at most half a step
    borders = 7.0 * 2.0 ** torch.arange(-5, 6, device=y.device, dtype=torch.float32)
    e = (g.abs().amax(-1, keepdim=True) > borders).sum(-1)
    t = g.abs() * torch.exp2((5 - e).float())[..., None]
    # to nearest, ties to the even magnitude code
    mag = ((t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0)).view(n, 64, 4, 2)
    sign = torch.signbit(g).to(torch.uint8).view(n, 64, 2, 4)
    codes = mag[..., 0] | (mag[..., 1] << 4) | (sign[:, :, 0] << 7) | (sign[:, :, 1] << 3)
    e = e.to(torch.uint8).view(n, 16, 2)
    rope = y[:, VALUE:].clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes.view(n, 256), e[..., 0] | (e[..., 1] << 4), rope], 1)


def _decode(rows):
    """Rows [..., 336] of bytes as values [..., 576] in 32 bits, kv_scale included."""
    lead = rows.shape[:-1]
    b = rows[..., :256].reshape(*lead, 64, 4)
    mag = torch.tensor(MAGNITUDES, device=rows.device)[torch.stack([b & 7, (b >> 4) & 7], -1).view(*lead, 64, 8).int()]
    sign = torch.cat([b >> 7, (b >> 3) & 1], -1)
    e = rows[..., 256:272]
    power = torch.exp2(torch.stack([e & 15, e >> 4], -1).view(*lead, 32).float() - 5.0) * KV_SCALE
    latent = torch.where(sign == 1, -mag, mag).view(*lead, 32, 16) * power[..., None]
    return torch.cat([latent.view(*lead, VALUE), rows[..., 272:].view(torch.float8_e4m3fn).float() * KV_SCALE], -1)


# ------------------------------------------------------------------------------- inputs
def _paged(g, lens, page, spare=0):
    """A page table over one shared pool in random order, and the pool's page count and free pages."""
    need = [_pages(n, page) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + spare, perm[at:]


def _pool(g, pages, page, kv):
    """Latent rows after their norm: about N(0, 1)."""
    width = FP4_ROW if kv == "fp4" else LATENT
    pool = torch.empty(pages, page, width, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (page * LATENT))
    for s in range(0, pages, step):
        x = torch.randn(min(step, pages - s), page, LATENT, generator=g, device="cuda")
        if kv == "fp4":
            pool[s:s + step] = _encode((x / KV_SCALE).view(-1, LATENT)).view(-1, page, width)
        else:
            pool[s:s + step] = x.to(torch.bfloat16) if kv == "bf16" else (x / KV_SCALE).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _shared_tables(g, c, spare_pages):
    """Tables of requests that share prefixes in families, and how often each page is referred to."""
    page, lens = c["page"], _spread(c["requests"], c["short"], c["long"])
    size, shared = _family(c)
    pages = _total_pages(c) + spare_pages
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), _pages(c["long"], page), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        first = 0
        if b % size:
            first = shared
            table[b, :first] = table[b - b % size, :first]
        n = _pages(n, page)
        table[b, first:n] = perm[at:at + n - first]
        at += n - first
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    inside = torch.arange(table.shape[1], device="cuda")[None, :] < _ints([_pages(n, page) for n in lens])[:, None]
    refs.scatter_add_(0, table.flatten().long(), inside.flatten().int())
    return lens, pages, table, refs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    page = c["page"]
    if c["op"] == "decode":
        lens, B, T, H = _spread(c["batch"], c["short"], c["long"]), c["batch"], c["drafts"], c["heads"]
        s["table"], pages, _ = _paged(g, lens, page)
        s["pool"] = _pool(g, pages, page, "fp4")
        s["q"] = torch.randn(B, T, H, LATENT, generator=g, device="cuda").to(torch.bfloat16)
        s["lens"], s["longest"] = _ints(lens), max(lens)
        s["mask"] = _tree_masks(g, B, T) if c["tree"] else None
        s["out"] = torch.empty(B, T, H, VALUE, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device="cuda")
        if own:  # a server plans a batch once per set of lengths and keeps its workspace
            from mla_attention_paged_gb300 import mla
            make = mla.decode_tree_plan if c["tree"] else mla.decode_plan
            s["plan"] = make(lens, T, H, page, s["table"].shape[1], pages, mla.MLA_KV_FP4)
            s["ws"] = mla.workspace_for(s["plan"], "cuda")
    elif c["op"] == "chunk":
        B, new, H = c["batch"], c["new"], c["heads"]
        n, rows = B * new, c["prefix"] + new
        s["table"], pages, _ = _paged(g, [rows] * B, page, 1)
        s["pool"] = _pool(g, pages, page, "fp4")
        # absorbed queries hold 512 columns from a projection already; the rotated 64 come here
        s["q_src"] = torch.randn(n, H, 192, generator=g, device="cuda").to(torch.bfloat16)
        s["q_dst"] = torch.randn(n, H, LATENT, generator=g, device="cuda").to(torch.bfloat16)
        s["q_in"], s["q_out"] = s["q_src"][..., 128:], s["q_dst"][..., VALUE:]
        s["kv"] = (torch.randn(n, LATENT, generator=g, device="cuda") * 2.0).to(torch.bfloat16)
        s["kv_weight"] = (1.0 + 0.1 * torch.randn(VALUE, generator=g, device="cuda")).to(torch.bfloat16)
        j = torch.arange(c["prefix"], rows, device="cuda")
        s["pos"] = j.int().repeat(B)
        s["slots"] = (s["table"][:, j // page].long() * page + j % page).view(-1)
        s["slots"][n - c["pad"]:] = -1  # padded tokens have no slot
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["cu"], s["rows"] = _ints([rows * b for b in range(B + 1)]), rows
        s["out"] = torch.empty(B * rows, LATENT, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "fork":
        lens, n = _spread(c["parents"], c["short"], c["long"]), c["children"]
        parent = torch.randint(0, len(lens), (n,), generator=g, device="cuda")
        held, pages, free = _paged(g, lens, page, n)
        s["table"] = torch.zeros(len(lens) + n, held.shape[1], dtype=torch.int32, device="cuda")
        s["table"][:len(lens)] = held
        s["pool"] = _pool(g, pages, page, c["kv"])
        s["lens"] = _ints(lens + [0] * n)
        inside = torch.arange(held.shape[1], device="cuda")[None, :] * page < s["lens"][:len(lens), None]
        s["refs0"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["refs0"].scatter_add_(0, held.flatten().long(), inside.flatten().int())
        s["refs"] = s["refs0"].clone()
        s["parents"] = parent.int()
        s["children"] = _ints(range(len(lens), len(lens) + n))
        # a parent that fills its last page needs no new one
        s["new"] = torch.where(s["lens"][parent] % page == 0, -1, free.int())
    elif c["op"] == "free":
        lens, pages, s["table"], refs = _shared_tables(g, c, int(0.3 * _total_pages(c)))
        # what a pass changes lies in one buffer, which the next one restores: counts, lengths
        s["before"] = torch.cat([refs, _ints(lens)])
        s["now"] = s["before"].clone()
        s["refs"], s["lens"] = s["now"][:pages], s["now"][pages:]
        order = torch.randperm(len(lens), generator=g, device="cuda")[:c["freed"]]
        s["slots"] = order.int()
        kept = _kept(c, [lens[i] for i in order.tolist()])
        s["keep"] = _ints(kept)
        s["freed"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        live = _total_pages(c)
        lens, pages, table, refs = _shared_tables(g, c, max(1, live * c["spare"] // 100))
        # counts and tables, which a pass changes
        s["before"] = torch.cat([refs, table.flatten()])
        s["now"] = s["before"].clone()
        s["refs"], s["table"] = s["now"][:pages], s["now"][pages:].view(table.shape)
        s["lens"] = _ints(lens)
        s["pool"] = _pool(g, pages, page, c["kv"])
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if own:
            from mla_attention_paged_gb300 import mla
            s["ws"] = mla.page_compact_workspace_for(pages, "cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_decode(s):
    B, T, H, _ = s["q"].shape
    page, n = s["case"]["page"], s["longest"]
    j = torch.arange(n, device="cuda")
    rows = _decode(s["pool"].view(-1, FP4_ROW)[s["table"].long()[:, j // page] * page + j % page])
    u = j[None, None, :] - (s["lens"].long() - T)[:, None, None]
    if s["mask"] is None:
        seen = u <= torch.arange(T, device="cuda")[None, :, None]
    else:
        seen = (u < 0) | ((u < T) & (((s["mask"][:, :, None] >> u.clamp(0, 63)) & 1) == 1))
    x = (s["q"].float().view(B, T * H, LATENT) @ rows.transpose(1, 2)).view(B, T, H, n) * SCALE
    x = x.masked_fill(~seen[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    s["out"].copy_((p.view(B, T * H, n) @ rows[..., :VALUE]).view(B, T, H, VALUE) / total)
    s["lse"].copy_((top + torch.log(total))[..., 0])
    return {"out": s["out"], "lse": s["lse"]}


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_chunk(s):
    c = s["case"]
    both = s["cos_sin"][s["pos"].long()]
    cos, sin = both[:, :ROPE // 2], both[:, ROPE // 2:]
    s["q_out"].copy_(_rotate(s["q_in"].float(), cos[:, None], sin[:, None], c["interleaved"]))
    x = s["kv"].float()
    latent = x[:, :VALUE]
    # (the mean in 64 bits: a code of four bits may hang on the last bit of the norm)
    mean = latent.double().square().mean(-1, keepdim=True).float()
    latent = latent * (1.0 / torch.sqrt(mean + EPS)) * s["kv_weight"].float()
    row = _encode(torch.cat([latent, _rotate(x[:, VALUE:], cos, sin, c["interleaved"])], -1) / KV_SCALE)
    flat = s["pool"].view(-1, FP4_ROW)
    real = (s["slots"] >= 0).nonzero()[:, 0]
    flat[s["slots"][real]] = row[real]
    j = torch.arange(s["rows"], device="cuda")
    s["out"].copy_(_decode(flat[(s["table"].long()[:, j // c["page"]] * c["page"] + j % c["page"]).view(-1)]))
    return {"q": s["q_dst"], "rows": s["out"]}


def _plain_fork(s):
    page = s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    lens, rows = s["lens"][parents], s["table"][parents]
    full, rest = lens // page, lens % page
    j = torch.arange(rows.shape[1], device="cuda")[None, :]
    s["refs"].scatter_add_(0, rows.flatten().long(), (j < full[:, None]).flatten().int())
    mine = torch.where(j < full[:, None], rows, s["table"][children])
    last = (j == full[:, None]) & (rest[:, None] > 0)
    s["table"][children] = torch.where(last, s["new"][:, None], mine)
    s["lens"][children] = lens
    part = rest.nonzero()[:, 0]
    s["refs"][s["new"][part].long()] = 1
    r = torch.arange(page, device="cuda")[None, :]
    inside = r < rest[part, None]
    src = (rows[part, full[part].long()].long()[:, None] * page + r)[inside]
    dst = (s["new"][part].long()[:, None] * page + r)[inside]
    flat = s["pool"].view(-1, LATENT)
    flat[dst] = flat[src]


def _plain_free(s):
    page = s["case"]["page"]
    at, keep = s["slots"].long(), s["keep"]
    rows = s["table"][at]
    j = torch.arange(rows.shape[1], device="cuda")[None, :]
    gone = (j >= ((keep + page - 1) // page)[:, None]) & (j < ((s["lens"][at] + page - 1) // page)[:, None])
    drop = torch.zeros_like(s["refs"]).scatter_add_(0, rows.flatten().long(), gone.flatten().int())
    s["refs"].sub_(drop)
    out = ((s["refs"] == 0) & (drop > 0)).nonzero()[:, 0].int()
    s["freed"][:out.numel()] = out
    s["count"].fill_(out.numel())
    s["lens"][at] = keep


def _plain_compact(s):
    page = s["case"]["page"]
    live = s["refs"] > 0
    n = int(live.sum())
    holes, from_ = (~live[:n]).nonzero()[:, 0], live[n:].nonzero()[:, 0] + n
    to = torch.arange(live.numel(), dtype=torch.int32, device="cuda")
    to[from_] = holes.int()
    s["pool"][holes] = s["pool"][from_]
    s["refs"][holes] = s["refs"][from_]
    s["refs"][from_] = 0
    j = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    inside = j < ((s["lens"] + page - 1) // page)[:, None]
    s["table"].copy_(torch.where(inside, to[s["table"].long()], s["table"]))
    s["count"].fill_(n)


def _values(s):
    return s["pool"] if s["case"]["kv"] == "bf16" else s["pool"].view(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from mla_attention_paged_gb300 import mla
    if op == "decode":
        if own:
            if s["mask"] is None:
                mla.decode(s["plan"], s["q"], s["pool"], s["table"], s["lens"], SCALE, KV_SCALE, out=s["out"], lse=s["lse"], workspace=s["ws"])
            else:
                mla.decode_tree(s["plan"], s["q"], s["pool"], s["table"], s["lens"], s["mask"], SCALE, KV_SCALE, out=s["out"], lse=s["lse"], workspace=s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        return _plain_decode(s)
    if op == "chunk":
        if own:
            mla.kv_append(s["q_in"], s["kv"], s["pos"], s["slots"], s["cos_sin"], s["pool"], kv_weight=s["kv_weight"], eps=EPS,
                          interleaved=s["case"]["interleaved"], kv_dtype=mla.MLA_KV_FP4, kv_scale=KV_SCALE, q_out=s["q_out"])
            mla.kv_gather(s["pool"], s["table"], s["cu"], s["out"], kv_dtype=mla.MLA_KV_FP4, kv_scale=KV_SCALE)
            return {"q": s["q_dst"], "rows": s["out"]}
        return _plain_chunk(s)
    if op == "fork":
        s["refs"].copy_(s["refs0"])  # (so that the new pages are free again)
        if own:
            kind = mla.MLA_KV_BF16 if s["case"]["kv"] == "bf16" else mla.MLA_KV_E4M3
            mla.page_fork(s["pool"], s["table"], s["lens"], s["refs"], s["parents"], s["children"], s["new"], kv_dtype=kind)
        else:
            _plain_fork(s)
        return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "pool": _values(s)}
    if op == "free":
        s["now"].copy_(s["before"])
        if own:
            mla.page_free(s["table"], s["lens"], s["refs"], s["slots"], s["keep"], s["case"]["page"], freed=s["freed"], num_freed=s["count"])
        else:
            _plain_free(s)
        return {"freed": s["freed"], "count": s["count"], "refs": s["refs"], "lens": s["lens"]}
    s["now"].copy_(s["before"])
    if own:
        kind = mla.MLA_KV_BF16 if s["case"]["kv"] == "bf16" else mla.MLA_KV_E4M3
        mla.page_compact(s["pool"], s["table"], s["lens"], s["refs"], kv_dtype=kind, num_live=s["count"], workspace=s["ws"])
    else:
        _plain_compact(s)
    return {"table": s["table"], "refs": s["refs"], "live": s["count"], "pool": _values(s)}


# ------------------------------------------------------------------------------- 64 bits
def _rows64(rows):
    """[n, 336] bytes as values in 64 bits, kv_scale included."""
    word = rows[:, :256].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    i = torch.arange(8, device=rows.device)
    m = (word[:, :, None] >> (4 * i)) & 7
    # magnitude code m = 2 x + y: y / 2 where x is 0, else (1 + y / 2) 2^(x - 1)
    x, y = m // 2, (m % 2).double() / 2
    size = torch.where(x == 0, y, (1 + y) * torch.pow(2.0, (x - 1).double()))
    negative = (word[:, :, None] >> torch.where(i < 4, 8 * i + 7, 8 * i - 29)) & 1
    e = rows[:, 256:272].contiguous().view(torch.int64)
    e = torch.stack([(e[:, i // 16] >> (4 * (i % 16))) & 15 for i in range(32)], 1)
    v = (size * (1 - 2 * negative)).reshape(-1, 32, 16) * torch.pow(2.0, (e - 5).double())[:, :, None]
    return torch.cat([v.reshape(-1, VALUE), rows[:, 272:].contiguous().view(torch.float8_e4m3fn).double()], 1) * KV_SCALE


def _quantised64(y):
    """Latents [n, 512] in units of kv_scale, 64 bits, as the values that the 4-bit codes would stand for."""
    g = y.reshape(-1, 32, 16)
    top = g.abs().amax(-1, keepdim=True).clamp(min=1e-30)
    power = torch.pow(2.0, torch.ceil(torch.log2(top / 7.0)).clamp(-5, 6))
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=y.device)
    t = (g.abs() / power).clamp(max=6.0)
    near = grid[(t[..., None] - grid).abs().argmin(-1)]
    return (torch.copysign(near, g) * power).reshape(-1, VALUE)


def _exact_decode(s, c):
    B, T, H, page = c["batch"], c["drafts"], c["heads"], c["page"]
    out = torch.zeros(B, T, H, VALUE, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_spread(B, c["short"], c["long"])):
        pages = s["table"][b, :_pages(n, page)].long()
        keys = _rows64(s["pool"][pages].reshape(-1, FP4_ROW)[:n])
        for t in range(T):
            if s["mask"] is None:
                ids = torch.arange(n - T + t + 1, device="cuda")
            else:
                m = int(s["mask"][b, t]) & ((1 << 64) - 1)
                ids = torch.tensor(list(range(n - T)) + [n - T + u for u in range(T) if m >> u & 1], device="cuda")
            x = s["q"][b, t].double() @ keys[ids].T * SCALE
            lse[b, t] = torch.logsumexp(x, 1)
            out[b, t] = torch.exp(x - lse[b, t][:, None]) @ keys[ids, :VALUE]
    return {"out": out, "lse": lse}


def _exact_chunk(s, c):
    half, page = ROPE // 2, c["page"]
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

    q = s["q_dst"].double()
    q[..., VALUE:] = turned(s["q_in"].double())
    x = s["kv"][:, :VALUE].double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["kv_weight"].double()
    rope = (turned(s["kv"][:, VALUE:].double()) / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).double()
    new = torch.cat([_quantised64(x / KV_SCALE), rope], 1) * KV_SCALE
    rows = []
    for b in range(c["batch"]):
        pages = s["table"][b].long()
        r = _rows64(s["pool"][pages].reshape(-1, FP4_ROW)[:s["rows"]])
        for_b = slice(b * c["new"], (b + 1) * c["new"])
        r[c["prefix"]:] = torch.where(s["slots"][for_b, None] >= 0, new[for_b], r[c["prefix"]:])
        rows.append(r)
    return {"q": q, "rows": torch.cat(rows)}


def exact(case, seed):
    if work(case)["flops"] > 9e12:  # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "decode":
        return _exact_decode(s, c)
    if c["op"] == "chunk":
        return _exact_chunk(s, c)
    if c["op"] == "free":
        return None  # whole numbers alone
    pool, page = _values(s).to(torch.float32).clone(), c["page"]
    if c["op"] == "fork":
        for i, p in enumerate(s["parents"].tolist()):
            n = int(s["lens"][p])
            if n % page:
                pool[int(s["new"][i]), :n % page] = pool[int(s["table"][p, n // page]), :n % page]
        return {"table": None, "lens": None, "refs": None, "pool": pool.double()}
    refs = s["refs"].cpu().numpy()
    n = int((refs > 0).sum())
    holes = [i for i in range(n) if refs[i] == 0]
    moved = [i for i in range(n, len(refs)) if refs[i] > 0]
    if moved:
        pool[torch.tensor(holes, device="cuda")] = pool[torch.tensor(moved, device="cuda")]
    return {"table": None, "refs": None, "live": None, "pool": pool.double()}
