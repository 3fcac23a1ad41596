"""The 336-byte rows of a 4-bit pool in plain torch: encoding and 64-bit values (include/mla.h, MLA_KV_FP4)."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
TOP = 6.0 * 2.0 ** 6  # the largest latent value in units of kv_scale


def pack(mag, neg, exp, rope):
    """Magnitude codes and signs [n, 512], exponents [n, 32], e4m3 bytes [n, 64] -> [n, 336] bytes."""
    n = mag.shape[0]
    out = torch.zeros(n, 336, dtype=torch.uint8)
    for i in range(8):
        at = slice(i // 2, 256, 4)
        out[:, at] |= (mag[:, i::8] << (4 * (i % 2))).to(torch.uint8)
        s = slice(i % 4, 256, 4)
        out[:, s] |= (neg[:, i::8].to(torch.uint8) << (7 if i < 4 else 3))
    out[:, 256:272] = (exp[:, 0::2] | (exp[:, 1::2] << 4)).to(torch.uint8)
    out[:, 272:] = rope
    return out


def encode(y):
    """Rows [n, 576] in units of kv_scale: nearest codes (ties to even) under the smallest exponent that
    rounds the group's largest value by at most half a step."""
    y = y.double()
    n = y.shape[0]
    g = y[:, :512].reshape(n, 32, 16)
    g = torch.where(g.isnan(), 0.0, g)
    top = g.abs().amax(-1)
    exp = torch.full_like(top, 11, dtype=torch.int32)
    for e in range(10, -1, -1):
        exp[top <= 7 * 2.0 ** (e - 5)] = e
    t = (g.abs() * 2.0 ** (5 - exp.double())[..., None]).clamp(max=6.0)
    d = (t[..., None] - GRID).abs()
    near = d.argmin(-1)
    tie = (d.gather(-1, near[..., None]) == d.gather(-1, (near + 1).clamp(max=7)[..., None]))[..., 0] & (near < 7)
    mag = torch.where(tie & (near % 2 == 1), near + 1, near)
    rope = y[:, 512:].float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return pack(mag.reshape(n, 512).int(), torch.signbit(g).reshape(n, 512), exp, rope)


def values(rows):
    """[..., 336] bytes -> [..., 576] in 64 bits, in units of kv_scale."""
    lead = rows.shape[:-1]
    b = rows.reshape(-1, 336).int()
    out = torch.zeros(b.shape[0], 576, dtype=torch.float64)
    for i in range(8):
        mag = (b[:, i // 2:256:4] >> (4 * (i % 2))) & 7
        neg = (b[:, i % 4:256:4] >> (7 if i < 4 else 3)) & 1
        out[:, i:512:8] = GRID[mag.long()] * (1 - 2 * neg)
    e = torch.stack([b[:, 256:272] & 15, b[:, 256:272] >> 4], -1).reshape(-1, 32)
    out[:, :512] *= 2.0 ** (e.double() - 5).repeat_interleave(16, 1)
    out[:, 512:] = rows.reshape(-1, 336)[:, 272:].contiguous().view(torch.float8_e4m3fn).double()
    return out.reshape(*lead, 576)
