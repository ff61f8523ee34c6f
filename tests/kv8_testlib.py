"""Plain float64 restatements of the 8-bit cache and of the norms with rotation,
written from their definitions (torch on the CPU, one sequence at a time), and
builders of small caches.  Test infrastructure only."""
from __future__ import annotations

import math

import torch

from gated_block_sparse_token_b200 import sas

D, BLK = 128, 64
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
AMIN = 2.0 ** -100
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


# ---------------------------------------------------------------- norms with rotation
def rotate(x, pos, base, back=False):
    """Rotate-half pairs (i, i + 64) of x [..., 128] by +-pos * base^(-2i/128), float64."""
    i = torch.arange(64, dtype=torch.float64)
    th = pos.double()[..., None] * base ** (-2.0 * i / D)
    c, s = th.cos(), th.sin() * (-1 if back else 1)
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def norm_rope(x, gamma, pos, base, eps):
    """x [B][H][T][128], pos [B][T]; returns y and the bound sum of |z| pairs used by the tolerances."""
    x, gamma = x.double(), gamma.double()
    z = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma
    size = z[..., :64].abs() + z[..., 64:].abs()
    return rotate(z, pos[:, None], base), torch.cat([size, size], -1)


def norm_rope_grad(x, gamma, pos, base, eps, dy):
    """(dx, its bound, dgamma, its bound); rows with a negative position contribute nothing."""
    x, gamma = x.double(), gamma.double()
    live = (pos >= 0)[:, None, :, None].double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    dy = dy.double() * live
    z = rotate(dy, pos.clamp_min(0)[:, None], base, back=True)
    size = dy[..., :64].abs() + dy[..., 64:].abs()
    size = torch.cat([size, size], -1)
    xh = x * r
    u = z * gamma
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    ub = size * gamma.abs()
    dxb = r * (ub + xh.abs() * (ub * xh.abs()).mean(-1, keepdim=True))
    return dx, dxb, (z * xh).sum((0, 1, 2)), (size * xh.abs()).sum((0, 1, 2))


# ---------------------------------------------------------------- the cache
def quantise(x, code):
    """Codes (float64 values) and scale of one block x [64][128]: scale = a / qmax, code = rn(x qmax / a)."""
    x = x.double()
    if not torch.isfinite(x).all():
        return torch.zeros_like(x), math.nan
    a = max(float(x.abs().max()), AMIN)
    y = x * QMAX[code] / a
    # the quotient of two bf16 values is either exactly half-way or at least 2^-16 of its value away from it: snap
    # float64's last bits so that the ties are seen as ties
    if code == INT8:
        y = torch.where((2 * y - (2 * y).round()).abs() < 1e-9, (2 * y).round() / 2, y)
        return y.round(), a / QMAX[code]
    e = torch.floor(torch.log2(torch.clamp(y.abs() * (1 + 1e-12), min=2.0 ** -6)))
    step = 2.0 ** (e - 3)
    t = y / step
    t = torch.where((2 * t - (2 * t).round()).abs() < 1e-9, (2 * t).round() / 2, t)
    return t.round() * step, a / QMAX[code]


def make_cache(B, hkv, blocks, code, paged, lens, device, seed=0, spare=0, fill=True):
    """A KvCache8 with random codes, scales and tails (tail rows past the length are NaN)."""
    g = torch.Generator().manual_seed(seed)
    n = B * blocks + spare

    def codes():
        x = torch.randn((n, hkv, BLK, D), generator=g) * 0.25
        c = (x * 300).clamp(-448, 448).to(E4M3) if code == E4M3 else (x * 100).round().clamp(-127, 127).to(INT8)
        return c if fill else torch.zeros_like(c.view(torch.uint8)).view(code)

    def shape(c):
        if paged:
            return c.to(device)
        return c.view(torch.uint8)[:B * blocks].view(B, blocks, hkv, BLK, D).transpose(1, 2).reshape(
            B, hkv, blocks * BLK, D).view(code).contiguous().to(device)

    def scales():
        s = torch.rand((n, hkv), generator=g) * 0.02 + 0.005
        s = s if paged else s[:B * blocks].view(B, blocks, hkv).transpose(1, 2).contiguous()
        return s.to(device)

    def tail():
        x = torch.randn((B, hkv, BLK, D), generator=g).bfloat16()
        for i, L in enumerate(lens):
            x[i, :, (L - 1) % BLK + 1:] = math.nan
        return x.to(device)

    table = torch.randperm(n, generator=g)[:B * blocks].to(torch.int32).view(B, blocks).to(device) if paged else None
    return sas.KvCache8(shape(codes()), shape(codes()), scales(), scales(), tail(), tail(),
                        torch.tensor(lens, dtype=torch.int32, device=device), table)


def block(kv, name, s, h, b):
    """Codes as float64 [64][128] and the scale of block b."""
    c, sc = getattr(kv, name), getattr(kv, name + "_scale")
    if kv.block_table is not None:
        p = int(kv.block_table[s, b])
        return c[p, h].cpu().double(), float(sc[p, h])
    return c[s, h, b * BLK:(b + 1) * BLK].cpu().double(), float(sc[s, h, b])


def tokens(kv, name, s, h, blocks, L):
    """Stored values (float64) of the listed blocks' tokens below L: code * scale, the current block from the tail."""
    cur = (L - 1) // BLK
    out = []
    for b in blocks:
        if b == cur:
            out.append(getattr(kv, name + "_tail")[s, h, :L - b * BLK].cpu().double())
        else:
            c, sc = block(kv, name, s, h, b)
            out.append(c * sc)
    return torch.cat(out)


def attend(kv, q, s, h, G, blocks, L, scale):
    """(out, sum of p |v|) of the G heads of KV head h, float64."""
    k, v = tokens(kv, "k", s, h, blocks, L), tokens(kv, "v", s, h, blocks, L)
    p = torch.softmax(q[s, h * G:(h + 1) * G].cpu().double() @ k.T * scale, -1)
    return p @ v, p @ v.abs()
