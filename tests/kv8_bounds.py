"""How exact the 8-bit decode attention has to be, by the arithmetic it
documents, and inputs on which a coarser arithmetic shows.  Test infrastructure
only (torch on the CPU, float64).

out = sum_j p_j v_j / sum_j p_j for one KV head's queries; an error of d_j in
logit j moves out by at most sum_j p_j d_j (|v_j| + |out|) / sum_j p_j.
* the query of the stored keys: int8 its multiple of 2^-21 E, E the power of two
  below the head's largest value: exact down to 2^-14 E, within 2^-22 E below;
  e4m3 f16 of q / E: at least as exact.
* products: int8 sums are exact, their three digits' sum is rounded twice: 2^-24 of
  the logit and of 2^-6 E sum |k|.  e4m3, and the bf16 tail: exact products, summed
  in fp32 (cut or rounded: 2^-23 of sum |q k| an addition).
* the logit's factors (scale, log2 e, unit, block scale) and its difference to the
  maximum: 2^-21 (|logit| + largest |logit|).
* p: exp2 2^-22, again for up to three changes of the maximum and merges; P's terms
  2^-22: 2^-20 of size = sum p |v| / sum p.  Sums of n keys: 2^-23 for each of the up
  to 16 of one matrix product, 2^-24 for each of a warp's n / 128 products.
* the output: half a step of bf16, three roundings in fp32."""
from __future__ import annotations

import torch

import kv8_testlib as K


def largest_power(q):
    return torch.exp2(torch.floor(torch.log2(q.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -126))))


def tolerance(q, k, v, tail, scale, code, out, times=None):
    """(out, tolerance) [G][128] of q [G][128] over keys k and values v [n][128], the last `tail` of them from the
    tail, key j counted times[j] times (default 1); all float64."""
    n = k.shape[0]
    stored = (torch.arange(n) < n - tail).double()
    times = torch.ones(n, dtype=torch.float64) if times is None else times
    E = largest_power(q)
    logit = q @ k.T * scale
    dq = torch.where(q.abs() >= E * 2.0 ** -14, 0.0, torch.minimum(q.abs(), E * 2.0 ** -22))
    products = ((q != 0).double() @ (k != 0).double().T - 1).clamp_min(0)
    summed = 2.0 ** -23 * products * (q.abs() @ k.abs().T) * scale
    digits = 2.0 ** -24 * (logit.abs() + 2.0 ** -6 * E * k.abs().sum(-1) * scale)
    d = dq @ k.abs().T * scale * stored + 2.0 ** -21 * (logit.abs() + logit.abs().amax(-1, keepdim=True))
    d = d + (torch.where(stored > 0, digits, summed) if code == K.INT8 else summed)
    p = torch.softmax(logit + times.log(), -1)
    want, size = p @ v, p @ v.abs()
    n = float(times.sum())
    term = 2.0 ** -20 + 2.0 ** -23 * min(n, 16) + 2.0 ** -24 * (n / 128)
    half = 2.0 ** -8 if out == "bf16" else 3 * 2.0 ** -24
    moved = (p * d) @ v.abs() + (p * d).sum(-1, keepdim=True) * want.abs()
    return want, moved + term * size + half * want.abs()


def roundings(q, k, v, tail, scale, code, digits=3, terms=2, tail_terms=3):
    """The attention in float64 with only its documented roundings of q and P (or coarser ones)."""
    E = largest_power(q)
    if code == K.INT8:      # two digits: up to 127/128 of 2^15
        top = 2.0 ** 21 if digits == 3 else 2.0 ** 14 * 127 / 128
        qr = torch.round(q / E * top) / top * E
    else:
        qr = (q / E).half().double() * E
    n = k.shape[0]
    logit = torch.cat([qr @ k[:n - tail].T, q @ k[n - tail:].T], -1) * scale
    p = torch.exp(logit - logit.amax(-1, keepdim=True))

    def split(x, count, dtype):
        s = torch.zeros_like(x)
        for _ in range(count):
            s = s + (x - s).to(dtype).double()
        return s
    w = torch.cat([split(p[:, :n - tail] * 2048, terms, torch.float16) / 2048,
                   split(p[:, n - tail:], tail_terms, torch.bfloat16)], -1)
    return w @ v / p.sum(-1, keepdim=True)


# ---------------------------------------------------------------- inputs: (cache, queries [B][8][128], scale), one KV head
def _set(codes, value):
    codes.copy_(value.to(torch.float32).to(codes.dtype))


def outlier(code, peak, device, seed=31):
    """N(0, 1) queries with one dominant channel, keys of rms 3 that are small there: what learned gains of queries
    and keys make."""
    lens = [64 * 32 + 1, 64 * 9 + 1]
    kv = K.make_cache(2, 1, 33, code, False, lens, "cpu", seed=seed)
    kv.k_scale.fill_(3.0 / (75.0 if code == K.E4M3 else 25.0))      # rms of the codes
    sign = torch.where(torch.arange(33 * 64) % 3 == 0, -1.0, 1.0)
    kv.k.view(torch.uint8)[..., 5] = sign.to(code).view(torch.uint8)
    kv.k_tail.mul_(3.0)
    kv.k_tail[..., 5] *= 0.02
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(seed + 1))
    q[..., 5] = peak
    return moved(kv, device), q.bfloat16(), 128 ** -0.5


def one_channel(code, stored, device, seed=41):
    """Queries and keys of a single channel: every logit is one exact product, so that what is left is the rounding
    of P.  Each sequence has one key of logit 0 and value 0 (the tail's first), and keys of one logit in -0.7 .. 0: 64
    stored ones, or one more of the tail."""
    B = 48
    lens = [65 if stored else 2] * B
    kv = K.make_cache(B, 1, 2, code, False, lens, "cpu", seed=seed)
    g = torch.Generator().manual_seed(seed)
    size = 0.2 + 0.25 * torch.rand(B, generator=g)
    kv.k.view(torch.uint8).zero_()
    kv.k_tail.zero_()
    kv.v_tail[:, :, 0] = 0
    if stored:
        kv.k.view(torch.uint8)[..., 5] = torch.full(kv.k.shape[:-1], -1.0).to(code).view(torch.uint8)
        kv.k_scale.copy_(size[:, None, None].expand_as(kv.k_scale))
        kv.v.view(torch.uint8)[:] = (torch.rand(kv.v.shape, generator=g) * 60 + 60).to(code).view(torch.uint8)
    else:
        kv.k_tail[:, 0, 1, 5] = -size.bfloat16()
        kv.v_tail[:, :, 1] = (torch.rand((B, 1, 128), generator=g) + 1).bfloat16()
    q = torch.zeros(B, 8, 128)
    q[..., 5] = 0.5 + torch.rand((B, 8), generator=g)
    return moved(kv, device), q.bfloat16(), 1.0


def moved(kv, device):
    from gated_block_sparse_token_b200 import sas
    return sas.KvCache8(*(getattr(kv, n).to(device) for n in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail", "seq_lens")))


def heads(kv, q):
    """(sequence, q, k, v, tail) of every sequence, float64 on the CPU."""
    for s, L in enumerate(kv.seq_lens.tolist()):
        blocks = range((L - 1) // 64 + 1)
        yield (s, q[s].double().cpu(), K.tokens(kv, "k", s, 0, blocks, L), K.tokens(kv, "v", s, 0, blocks, L),
               (L - 1) % 64 + 1)
