"""The operators around the 8-bit KV cache, as they are measured.

A decode or prefill layer with an 8-bit cache goes through: the norms of its
queries and keys with the position rotation (``sas.qk_norm_rope``, and its
gradient), the cache write, which quantises each completed 64-token block
under one scale per KV head (``sas.kv8_append``), the read-back
(``sas.kv8_read``), the gate keys pooled from the stored blocks
(``sas.pool_keys_kv8``), and the block-sparse decode attention over the codes
(``sas.sparse_decode_kv8``).

``run`` computes them in plain torch (32 bits, angles in 64) or, with ``own``,
by the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
D = 128                      # head_dim
BLK = 64                     # tokens of a block
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE_T = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
AMIN = 2.0 ** -100           # smallest magnitude a block's scale stands for
EPS = 1e-6
BASE = 1e6                   # position base of the attention rotation
GATE_BASE = 1e4              # position base of the gate keys
WS_BYTES = 4 << 20           # workspace, as a serving program keeps one per stream


# ---------------------------------------------------------------- cases
def listed():
    return [
        # queries and keys of one decode step, batch 8, far positions: latency
        dict(name="norm_rope_decode_b8", kind="norm", hq=32, hkv=8, batch=8, tokens=1, first=32000, pad=False, dtype="bf16"),
        # a prefill of two 32k chunks that continue long sequences
        dict(name="norm_rope_prefill_2x32k", kind="norm", hq=32, hkv=8, batch=2, tokens=32768, first=98304, pad=False,
             dtype="bf16"),
        # gradient of a ragged, padded training batch (odd length, group of 5)
        dict(name="norm_rope_grad_8x1021", kind="norm_grad", hq=40, hkv=8, batch=8, tokens=1021, first=0, pad=True,
             dtype="bf16"),
        # one decoded token a sequence, a quarter of them complete a block
        dict(name="write_decode_b32", kind="write", hkv=8, batch=32, new=1, old=16000, code="e4m3", read=64),
        # packed prefill chunks of different lengths, written and read back for the chunk's attention
        dict(name="write_chunk_b6_int8", kind="write", hkv=8, batch=6, new=8190, old=4096, code="int8", read=8190),
        # a stored prefix read back in bf16
        dict(name="read_prefix_4x32k", kind="read", hkv=8, batch=4, length=32768, code="e4m3", paged=True),
        # gate keys of the blocks a decode step completed
        dict(name="pool_decode_b16", kind="pool", hkv=8, batch=16, length=8192, blocks=1, code="e4m3", paged=True),
        # gate keys of a whole prompt batch
        dict(name="pool_prompt_4x32k", kind="pool", hkv=8, batch=4, length=32768, blocks=512, code="int8", paged=False),
        # one short conversation under the smallest budget: latency
        dict(name="attend_b1_4k", kind="attend", hq=32, hkv=8, batch=1, lo=4000, hi=4000, budget=1024, code="e4m3",
             paged=False, out="bf16"),
        # the benchmark's decode layer on an 8-bit cache
        dict(name="attend_b8_32k", kind="attend", hq=32, hkv=8, batch=8, lo=32768, hi=32768, budget=2048, code="e4m3",
             paged=False, out="bf16"),
        # ragged serving batch, paged, group of 5, largest budget, fp32 output
        dict(name="attend_ragged_b32_int8", kind="attend", hq=40, hkv=8, batch=32, lo=8192, hi=65536, budget=4096,
             code="int8", paged=True, out="f32"),
        # every block of two long contexts (a layer that keeps dense attention)
        dict(name="attend_all_b2_128k", kind="attend", hq=32, hkv=8, batch=2, lo=120001, hi=131072, budget=0, code="e4m3",
             paged=True, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "write", "read", "pool", "attend", "attend"])
    code = rng.choice(["e4m3", "int8"])
    paged = rng.random() < 0.5
    hkv = rng.choice([1, 2, 4, 8])
    if kind in ("norm", "norm_grad"):
        group = rng.choice([1, 2, 4, 5, 8])
        most = 150_000_000 // (hkv * (group + 1) * D)          # elements: below the largest listed case
        if kind == "norm_grad":
            most //= 4
        rows = _log_int(rng, 1, min(most, 65536))
        batch = rng.randint(1, max(1, min(rows, 8)))
        return dict(kind=kind, hq=hkv * group, hkv=hkv, batch=batch, tokens=max(1, rows // batch),
                    first=_log_int(rng, 1, 200000), pad=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if kind == "write":
        new = _log_int(rng, 1, 8192)
        return dict(kind=kind, hkv=hkv, batch=rng.randint(1, 32 if new < 256 else 6), new=new,
                    old=64 * _log_int(rng, 1, 256), code=code, read=max(64, new))
    if kind == "read":
        return dict(kind=kind, hkv=hkv, batch=rng.randint(1, 4), length=_log_int(rng, 1, 32768), code=code, paged=paged)
    if kind == "pool":
        length = _log_int(rng, 64, 32768)
        return dict(kind=kind, hkv=hkv, batch=rng.randint(1, 4), length=length, blocks=rng.randint(1, length // 64),
                    code=code, paged=paged)
    budget = rng.choice([0, 256, 1024, 2048, 4096, 6400])
    hi = _log_int(rng, 1, 65536)
    batch = rng.randint(1, 16 if budget else 2)
    return dict(kind=kind, hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv, batch=batch, lo=max(1, hi // 3), hi=hi,
                budget=budget, code=code, paged=paged, out=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _encode(x, code):
    """Codes and scale of blocks x [..., 64, 128] in 32 bits: one scale a block.  The products by 448 or 127 are exact
    (bf16 values), so the quotient is the rounded exact one."""
    a = x.abs().amax(dim=(-1, -2), keepdim=True).clamp_min(AMIN)
    y = (x * QMAX[code]) / a
    c = y.to(torch.float8_e4m3fn) if code == "e4m3" else y.round().to(torch.int8)
    return c, (a / QMAX[code])[..., 0, 0]


def _cache(case, lens, g, most=0):
    """An 8-bit cache that holds lens[s] tokens a sequence (with room for `most`), keys and values N(0, 1) with a mean of each block's own."""
    B, hkv = case["batch"], case["hkv"]
    nblk = -(-max(lens + [most]) // BLK)
    s = {"lens": lens, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "nblk": nblk}
    paged = case.get("paged", True)
    for name in ("k", "v"):
        codes = torch.empty((B * nblk + 1, hkv, BLK, D) if paged else (B, hkv, nblk * BLK, D), dtype=CODE_T[case["code"]],
                            device=DEV)
        flat = codes.view(-1, hkv, BLK, D) if paged else codes.view(-1, 1, BLK, D)
        scale = torch.empty(flat.shape[:2], device=DEV)
        for at in range(0, flat.shape[0], 4096):
            n = min(4096, flat.shape[0] - at)
            x = torch.randn((n,) + flat.shape[1:], generator=g, device=DEV)
            x += 0.5 * torch.randn((n, flat.shape[1], 1, D), generator=g, device=DEV)
            c, sc = _encode(x.bfloat16().float(), case["code"])
            flat[at:at + n].view(torch.uint8).copy_(c.view(torch.uint8))
            scale[at:at + n] = sc
        s[name] = codes
        s[name + "_scale"] = scale if paged else scale.view(B, hkv, nblk)
        s[name + "_tail"] = torch.randn((B, hkv, BLK, D), generator=g, device=DEV).bfloat16()
    s["table"] = torch.randperm(B * nblk, generator=g, device=DEV).to(torch.int32).view(B, nblk) if paged else None
    return s


def _lengths(case, g):
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=g, device=DEV)
    lens[0] = case["hi"]
    return lens.tolist()


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": case, "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)}
    if kind in ("norm", "norm_grad"):
        B, T, hq, hkv, dt = case["batch"], case["tokens"], case["hq"], case["hkv"], _dtype(case["dtype"])
        # the projections' packed output: a token's query, key and value heads side by side
        qkv = torch.randn((B, T, hq + 2 * hkv, D), generator=g, device=DEV, dtype=torch.float32).to(dt)
        s["q"], s["k"] = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hkv].transpose(1, 2)
        s["gamma_q"] = 1 + 0.25 * torch.randn(D, generator=g, device=DEV)
        s["gamma_k"] = 1 + 0.25 * torch.randn(D, generator=g, device=DEV)
        pos = case["first"] + torch.arange(T, device=DEV)[None] + torch.randint(0, 64, (B, 1), generator=g, device=DEV)
        if case["pad"]:  # a padded batch: rows behind a sequence's end have position -1
            n = torch.randint(max(1, T // 2), T + 1, (B, 1), generator=g, device=DEV)
            pos = torch.where(torch.arange(T, device=DEV)[None] < n, pos, -1)
        s["pos"] = pos.to(torch.int32)
        s["q_out"] = torch.zeros((B, hq, T, D), dtype=dt, device=DEV)
        s["k_out"] = torch.zeros((B, hkv, T, D), dtype=dt, device=DEV)
        if kind == "norm_grad":
            s["d_q"] = torch.randn((B, hq, T, D), generator=g, device=DEV).to(dt)
            s["d_k"] = torch.randn((B, hkv, T, D), generator=g, device=DEV).to(dt)
            s["d_gamma"] = torch.zeros((2, D), device=DEV)
        return s
    if kind == "write":
        B, hkv = case["batch"], case["hkv"]
        r = torch.rand(B, generator=g, device=DEV).tolist()
        if case["new"] <= 32:  # decode: old lengths anywhere in a block that the new tokens do not leave
            old = [case["old"] + int(x * (BLK - case["new"])) for x in r]
            old = [case["old"] + BLK - case["new"] if i % 4 == 0 else o for i, o in enumerate(old)]
            new = [case["new"]] * B
        else:                  # prefill chunks, block-aligned starts
            old = [BLK * int(x * case["old"] / BLK) for x in r]
            new = [max(1, case["new"] - int(case["new"] * 0.9 * x)) if i else case["new"] for i, x in enumerate(r)]
        lens = [o + n for o, n in zip(old, new)]
        s.update(_cache(case, lens, g, most=case["old"] + BLK + case["new"]))
        starts = [sum(new[:i]) for i in range(B)]
        s["old"], s["new"], s["starts"] = old, new, starts
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["new_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        # packed tokens, keys and values side by side
        kv = torch.randn((sum(new), 2 * hkv, D), generator=g, device=DEV).bfloat16()
        s["k_new"], s["v_new"] = kv[:, :hkv].transpose(0, 1)[None], kv[:, hkv:].transpose(0, 1)[None]
        begin = [o if case["new"] > 32 else max(0, n - case["read"]) for o, n in zip(old, lens)]
        s["begin"] = torch.tensor(begin, dtype=torch.int32, device=DEV)
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros((B, hkv, case["read"], D), dtype=torch.bfloat16, device=DEV)
        # the blocks that the write touches, for the plain form
        nb = (case["new"] + BLK - 1) // BLK + 1
        o, n = torch.tensor(old, device=DEV)[:, None], torch.tensor(lens, device=DEV)[:, None]
        s["o"], s["n"] = o, n
        s["blk"] = o // BLK + torch.arange(nb, device=DEV)[None]
        return s
    if kind == "read":
        lens = [max(1, case["length"] - 37 * i) for i in range(case["batch"])]
        s.update(_cache(case, lens, g))
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros((case["batch"], case["hkv"], max(lens), D), dtype=torch.bfloat16, device=DEV)
        return s
    if kind == "pool":
        B, hkv = case["batch"], case["hkv"]
        s.update(_cache(case, [case["length"]] * B, g))
        s["first"] = case["length"] // BLK - case["blocks"]
        s["blk_begin"] = torch.full((B,), s["first"], dtype=torch.int32, device=DEV)
        s["w_k"] = (torch.randn((hkv, 3 * D, D), generator=g, device=DEV) / math.sqrt(3 * D)).bfloat16()
        s["gamma_k"] = 1 + 0.25 * torch.randn(D, generator=g, device=DEV)
        s["gate_keys"] = torch.zeros((B, hkv, s["nblk"], D), device=DEV)
        return s
    # attend
    B, hq, hkv = case["batch"], case["hq"], case["hkv"]
    lens = _lengths(case, g)
    s.update(_cache(case, lens, g))
    s["q"] = torch.randn((B, hq, D), generator=g, device=DEV).bfloat16()
    s["out"] = torch.zeros((B, hq, D), dtype=_dtype(case["out"]), device=DEV)
    c = (s["seq_lens"].long() - 1) // BLK
    if case["budget"]:
        keep = case["budget"] // BLK
        blocks = torch.arange(s["nblk"], device=DEV)
        score = torch.rand((B, hkv, s["nblk"]), generator=g, device=DEV)
        score = torch.where(blocks < c[:, None, None], score, -1.0).masked_fill(blocks == c[:, None, None], 2.0)
        top = score.topk(min(keep, s["nblk"]), dim=-1)
        idx = torch.where(top.values >= 0, top.indices, 1 << 30).sort(dim=-1).values
        s["sel_idx"] = torch.zeros((B, hkv, keep), dtype=torch.int32, device=DEV)
        s["sel_idx"][..., :idx.shape[-1]] = torch.where(idx < (1 << 30), idx, 0).to(torch.int32)
        s["sel_count"] = (c + 1).clamp_max(keep).to(torch.int32)[:, None].expand(B, hkv).contiguous()
    else:
        s["sel_idx"] = s["sel_count"] = None
    return s


# ---------------------------------------------------------------- plain forms
def _angles(pos, base):
    freq = torch.tensor(float(base), dtype=torch.float64, device=DEV) ** (-torch.arange(0, D, 2, device=DEV).double() / D)
    a = pos.double()[..., None] * freq
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin):
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_norm(s):
    cos, sin = (t[:, None] for t in _angles(s["pos"].clamp_min(0), BASE))
    live = (s["pos"] >= 0)[:, None, :, None]
    outs = []
    for x, gamma in ((s["q"], s["gamma_q"]), (s["k"], s["gamma_k"])):
        x32 = x.float()
        y = _rotate(x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * gamma, cos, sin)
        outs.append(torch.where(live, y, 0.0).to(x.dtype))
    return outs


def _plain_norm_grad(s):
    cos, sin = (t[:, None] for t in _angles(s["pos"].clamp_min(0), BASE))
    live = (s["pos"] >= 0)[:, None, :, None]
    outs, gains = [], []
    for x, gamma, dy in ((s["q"], s["gamma_q"], s["d_q"]), (s["k"], s["gamma_k"], s["d_k"])):
        x32 = x.float()
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
        z = torch.where(live, _rotate(dy.float(), cos, -sin), 0.0)
        gains.append((z * x32 * r).sum(dim=(0, 1, 2), dtype=torch.float64).float())
        u = z * gamma
        outs.append((r * u - x32 * r ** 3 * (u * x32).mean(-1, keepdim=True)).to(x.dtype))
    return outs + [torch.stack(gains)]


def _stored(s, name, b, blk):
    """Codes as 32-bit values and scales of blocks blk [n...] of sequences b (same shape): [n..., Hkv, 64, 128], [n..., Hkv]."""
    if s["table"] is not None:
        page = s["table"][b, blk].long()
        return s[name].view(torch.uint8)[page].view(s[name].dtype).float(), s[name + "_scale"][page]
    c = s[name].view(s[name].shape[0], s[name].shape[1], -1, BLK, D).transpose(1, 2).view(torch.uint8)
    return c[b, blk].view(s[name].dtype).float(), s[name + "_scale"].transpose(1, 2)[b, blk]


def _plain_read(s, name, begin, tokens):
    """Tokens begin[s] .. begin[s] + tokens - 1 of every sequence as [B][Hkv][tokens][128], 0 past the length."""
    B = begin.shape[0]
    n = s["seq_lens"].long()[:, None]
    first = begin.long()[:, None] // BLK
    nb = (tokens + BLK - 1) // BLK + 1
    blk = first + torch.arange(nb, device=DEV)[None]
    b = torch.arange(B, device=DEV)[:, None].expand_as(blk)
    codes, scale = _stored(s, name, b, blk.clamp_max(s["nblk"] - 1))
    x = codes * scale[..., None, None]
    x = torch.where((blk == (n - 1) // BLK)[..., None, None, None], s[name + "_tail"].float()[:, None], x)
    x = x.transpose(1, 2).reshape(B, x.shape[2], nb * BLK, D)
    at = (begin.long()[:, None] - first * BLK) + torch.arange(tokens, device=DEV)[None]
    x = x[torch.arange(B, device=DEV)[:, None], :, at].transpose(1, 2)
    live = begin.long()[:, None] + torch.arange(tokens, device=DEV)[None] < n
    return torch.where(live[:, None, :, None], x, 0.0).to(torch.bfloat16)


def _plain_write(s):
    code, B = s["case"]["code"], s["case"]["batch"]
    o, n, blk = s["o"], s["n"], s["blk"]
    pos = blk[..., None] * BLK + torch.arange(BLK, device=DEV)            # [B, nb, 64]
    row = s["new_starts"].long()[:, None, None] + pos - o[..., None]
    fresh = (pos >= o[..., None]) & (pos < n[..., None])
    done = (blk + 1) * BLK <= n
    b = torch.arange(B, device=DEV)[:, None]
    # blocks the write does not complete go to the spare last page
    page = torch.where(done, s["table"][b, blk.clamp_max(s["nblk"] - 1)].long(), s["k"].shape[0] - 1)
    for name in ("k", "v"):
        new = s[name + "_new"][0]                                         # [Hkv, N, 128]
        tail = s[name + "_tail"]
        x = new[:, row.clamp(0, new.shape[1] - 1)].permute(1, 2, 0, 3, 4)     # [B, nb, Hkv, 64, 128]
        head = torch.where((pos < o[..., None])[:, :, None, :, None], tail[:, None], 0.0)
        x = torch.where(fresh[:, :, None, :, None], x, head)
        c, scale = _encode(x.float(), code)
        s[name].view(torch.uint8)[page] = c.view(torch.uint8)
        s[name + "_scale"][page] = scale
        cur = ((n - 1) // BLK - blk[:, :1])[:, 0].clamp_min(0)
        at = torch.arange(B, device=DEV)
        tail.copy_(torch.where(fresh[at, cur][:, None, :, None], x[at, cur], tail))
    return _written(s, [_plain_read(s, name, s["begin"], s["case"]["read"]) for name in ("k", "v")])


def _written(s, back):
    return back + [s["k_tail"], s["v_tail"], s["k_scale"][:-1], s["v_scale"][:-1]]


def _plain_pool(s):
    B, n = s["case"]["batch"], s["case"]["blocks"]
    blk = s["first"] + torch.arange(n, device=DEV)[None].expand(B, n)
    b = torch.arange(B, device=DEV)[:, None].expand_as(blk)
    codes, scale = _stored(s, "k", b, blk)
    x = codes * scale[..., None, None]
    p = torch.cat([x.amax(-2), x.amin(-2), x.mean(-2)], -1)               # [B, n, Hkv, 384]
    u = torch.einsum("bnhp,hpd->bhnd", p, s["w_k"].float())
    u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * s["gamma_k"]
    cos, sin = (t[:, None] for t in _angles(blk, GATE_BASE))
    s["gate_keys"][:, :, s["first"]:s["first"] + n] = _rotate(u, cos, sin)
    return s["gate_keys"]


def _plain_attend(s):
    case = s["case"]
    B, hq, hkv = case["batch"], case["hq"], case["hkv"]
    n = s["seq_lens"].long()
    c = (n - 1) // BLK
    if s["sel_idx"] is None:
        blk = torch.arange(s["nblk"], device=DEV).expand(B, hkv, -1)
        used = blk <= c[:, None, None]
    else:
        blk = s["sel_idx"].long()
        used = torch.arange(blk.shape[-1], device=DEV) < s["sel_count"][..., None]
    at = torch.where(used, blk, 0)
    b = torch.arange(B, device=DEV)[:, None, None].expand_as(at)
    h = torch.arange(hkv, device=DEV)[None, :, None].expand_as(at)
    xs = []
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8)
        if s["table"] is not None:
            page = s["table"][b, at].long()
            x, scale = codes[page, h], s[name + "_scale"][page, h]
        else:
            x, scale = codes.view(B, hkv, -1, BLK, D)[b, h, at], s[name + "_scale"][b, h, at]
        x = x.view(s[name].dtype).float() * scale[..., None, None]        # [B, Hkv, n, 64, 128]
        x = torch.where((at == c[:, None, None])[..., None, None], s[name + "_tail"].float()[:, :, None], x)
        xs.append(x.reshape(B, hkv, -1, D))
    live = (at[..., None] * BLK + torch.arange(BLK, device=DEV) < n[:, None, None, None]) & used[..., None]
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    logits = (q @ xs[0].transpose(-1, -2)) / math.sqrt(D)
    logits = logits.masked_fill(~live.reshape(B, hkv, 1, -1), -math.inf)
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    v = torch.where(live.reshape(B, hkv, -1, 1), xs[1], 0.0)
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.reshape(B, hq, D).to(s["out"].dtype)


# ---------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program keeps beside its tensors: the configuration and the cache's description."""
    if "cfg" not in s:
        from gated_block_sparse_token_b200 import sas
        case = s["case"]
        s["sas"] = sas
        s["cfg"] = sas.Config(case.get("hq", case["hkv"]), case["hkv"], token_budget=case.get("budget") or 2048,
                              kv_dtype=case.get("dtype", "bf16"), out_dtype=case.get("out", "bf16"), norm_eps=EPS,
                              rope_base=GATE_BASE)
        if "k_scale" in s:
            s["kv"] = sas.KvCache8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"], s["seq_lens"],
                                   s["table"])
    return s["sas"], s["cfg"], s.get("kv")


def _own(s):
    sas, cfg, kv = _handles(s)
    case = s["case"]
    kind = case["kind"]
    if kind == "norm":
        sas.qk_norm_rope(cfg, s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["q_out"], s["k_out"], BASE, positions=s["pos"])
        return [s["q_out"], s["k_out"]]
    if kind == "norm_grad":
        s["d_gamma"].zero_()
        sas.qk_norm_rope_backward(cfg, s["d_q"], s["d_k"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["q_out"],
                                  s["k_out"], s["d_gamma"][0], s["d_gamma"][1], BASE, s["ws"], positions=s["pos"])
        return [s["q_out"], s["k_out"], s["d_gamma"]]
    if kind == "write":
        sas.kv8_append(cfg, kv, s["k_new"], s["v_new"], s["ws"], new_starts=s["new_starts"], new_lens=s["new_lens"],
                       max_new=case["new"])
        sas.kv8_read(cfg, kv, s["k_out"], s["v_out"], s["ws"], begin=s["begin"])
        return _written(s, [s["k_out"], s["v_out"]])
    if kind == "read":
        sas.kv8_read(cfg, kv, s["k_out"], s["v_out"], s["ws"])
        return [s["k_out"], s["v_out"]]
    if kind == "pool":
        sas.pool_keys_kv8(cfg, kv, s["w_k"], s["gamma_k"], s["gate_keys"], s["ws"], blk_begin=s["blk_begin"],
                          num_blocks=case["blocks"])
        return s["gate_keys"]
    sas.sparse_decode_kv8(cfg, s["q"], kv, s["sel_idx"], s["sel_count"], s["out"], s["ws"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    kind = s["case"]["kind"]
    if kind == "norm":
        return _plain_norm(s)
    if kind == "norm_grad":
        return _plain_norm_grad(s)
    if kind == "write":
        return _plain_write(s)
    if kind == "read":
        begin = torch.zeros_like(s["seq_lens"])
        return [_plain_read(s, name, begin, s["k_out"].shape[2]) for name in ("k", "v")]
    if kind == "pool":
        return _plain_pool(s)
    return _plain_attend(s)


# ---------------------------------------------------------------- what a pass has to read, write and compute
def work(case):
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        n = case["batch"] * case["tokens"] * (case["hq"] + case["hkv"]) * D
        size = 2 if case["dtype"] == "bf16" else 4
        if case["pad"]:
            n *= 0.75                                          # mean share of live rows
        return {"bytes": n * size * (2 if kind == "norm" else 3), "flops": n * (8 if kind == "norm" else 16)}
    if kind == "write":
        row = case["hkv"] * D * 2                              # elements of a token's keys and values
        new = case["batch"] * case["new"] * (1.0 if case["new"] <= 32 else 0.55)
        read = case["batch"] * case["read"] if case["new"] <= 32 else new
        return {"bytes": row * (new * 3 + read * 2), "flops": row * new * 6}
    if kind == "read":
        n = case["batch"] * case["hkv"] * case["length"] * D * 2
        return {"bytes": n * 3, "flops": n}
    if kind == "pool":
        n = case["batch"] * case["hkv"] * case["blocks"]
        return {"bytes": n * (BLK * D + 4 + D * 4) + case["hkv"] * 3 * D * D * 2, "flops": n * (3 * BLK * D + 2 * 3 * D * D)}
    B, hkv, hq = case["batch"], case["hkv"], case["hq"]
    mean = (case["lo"] + case["hi"]) / 2
    tokens = min(mean, case["budget"]) if case["budget"] else mean
    last = min(BLK, tokens)
    per_pair = (tokens - last) * D * 2 + (tokens - last) / BLK * 8 + last * D * 4 * 0.5
    size = 2 if case["out"] == "bf16" else 4
    return {"bytes": B * hkv * per_pair + B * hq * D * (2 + size), "flops": 4 * B * hq * tokens * D}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rope(x, pos, base, back=False):
    """Each pair (i, i + 64) as a complex number times e^(+-j pos base^(-i/64))."""
    i = torch.arange(D // 2, dtype=torch.float64, device=DEV)
    th = pos.to(torch.float64).unsqueeze(-1) * torch.exp(-(i / (D // 2)) * math.log(base))
    z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous())
    z = z * torch.polar(torch.ones_like(th), -th if back else th)
    return torch.cat((z.real, z.imag), dim=-1)


def _exact_code(x, code):
    """The values that blocks x [..., 64, 128] are stored as, and their scales."""
    a = torch.clamp(x.abs().flatten(-2).max(-1).values, min=AMIN)
    y = x * (QMAX[code] / a)[..., None, None]
    y = torch.where((y * 2 - (y * 2).round()).abs() < 1e-9, (y * 2).round() / 2, y) if code == "int8" else y
    if code == "int8":
        y = y.round()
    else:  # four significant bits, exponents from -6; ties to even
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6) * (1 + 1e-13))) - 3)
        t = y / step
        t = torch.where((t * 2 - (t * 2).round()).abs() < 1e-9, (t * 2).round() / 2, t)
        y = t.round() * step
    scale = a / QMAX[code]
    return y * scale[..., None, None], scale


def _exact_block(s, name, i, j):
    """Stored values of block j of sequence i: [Hkv, 64, 128] in 64 bits."""
    if s["table"] is not None:
        page = int(s["table"][i, j])
        return s[name][page].double() * s[name + "_scale"][page].double()[:, None, None]
    return s[name][i, :, j * BLK:(j + 1) * BLK].double() * s[name + "_scale"][i, :, j].double()[:, None, None]


def _exact_blocks(s, name, i, blocks):
    """The same for a list of blocks: [n, Hkv, 64, 128]."""
    if s["table"] is not None:
        page = s["table"][i].long()[blocks]
        return s[name].view(torch.uint8)[page].view(s[name].dtype).double() * s[name + "_scale"].double()[page][..., None, None]
    c = s[name][i].view(torch.uint8).view(s[name].shape[1], -1, BLK, D)[:, blocks].view(s[name].dtype).double()
    return (c * s[name + "_scale"][i].double()[:, blocks][..., None, None]).transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        live = (s["pos"] >= 0)[:, None, :, None].double()
        pos = s["pos"].clamp_min(0)[:, None]
        outs, gains = [], []
        for x, gamma, dy in ((s["q"], s["gamma_q"], s.get("d_q")), (s["k"], s["gamma_k"], s.get("d_k"))):
            x, gamma = x.double(), gamma.double()
            rms = (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
            if kind == "norm":
                outs.append(_exact_rope(x / rms * gamma, pos, BASE) * live)
                continue
            z = _exact_rope(dy.double(), pos, BASE, back=True) * live
            xh = x / rms
            gains.append((z * xh).sum((0, 1, 2)))
            u = z * gamma
            outs.append((u - xh * ((u * xh).sum(-1, keepdim=True) / D)) / rms)
        return outs + ([torch.stack(gains)] if gains else [])
    if kind == "write":
        outs = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        tails, scales = [], []
        for which, name in enumerate(("k", "v")):
            tail, scale = s[name + "_tail"].double(), s[name + "_scale"].double()[:-1]
            for i, (o, n, at) in enumerate(zip(s["old"], s["new"], s["starts"])):
                first = o // BLK
                x = torch.cat([tail[i, :, :o % BLK], s[name + "_new"][0, :, at:at + n].double()], 1)   # from block `first`
                full = x.shape[1] // BLK
                back = x.clone()
                if full:
                    vals, sc = _exact_code(x[:, :full * BLK].reshape(-1, full, BLK, D), case["code"])
                    back[:, :full * BLK] = vals.reshape(-1, full * BLK, D)
                    scale[s["table"][i, first:first + full].long()] = sc.transpose(0, 1)
                last = (o + n - 1) // BLK                       # the current block is read from its tail
                back[:, (last - first) * BLK:] = x[:, (last - first) * BLK:]
                rows = o + n - last * BLK
                begin = int(s["begin"][i])
                tail[i, :, max(0, o - last * BLK):rows] = x[:, (last - first) * BLK:][:, max(0, o - last * BLK):]
                if begin < first * BLK:                         # blocks that were there before
                    prev = [_exact_block(s, name, i, j) for j in range(begin // BLK, first)]
                    back = torch.cat(prev + [back], 1)
                    first = begin // BLK
                back = back[:, begin - first * BLK:][:, :case["read"]]
                outs[which][i, :, :back.shape[1]] = back
            tails.append(tail)
            scales.append(scale)
        return outs + tails + scales
    if kind == "read":
        outs = []
        for name in ("k", "v"):
            out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV)
            for i, n in enumerate(s["lens"]):
                last = (n - 1) // BLK
                if last:
                    x = _exact_blocks(s, name, i, torch.arange(last, device=DEV))
                    out[i, :, :last * BLK] = x.transpose(0, 1).reshape(-1, last * BLK, D)
                out[i, :, last * BLK:n] = s[name + "_tail"][i, :, :n - last * BLK].double()
            outs.append(out)
        return outs
    if kind == "pool":
        out = torch.zeros(s["gate_keys"].shape, dtype=torch.float64, device=DEV)
        blocks = torch.arange(s["first"], s["first"] + case["blocks"], device=DEV)
        for i in range(case["batch"]):
            x = _exact_blocks(s, "k", i, blocks)
            p = torch.cat([x.max(2).values, x.min(2).values, x.sum(2) / BLK], -1).transpose(0, 1)   # [Hkv, n, 384]
            u = torch.bmm(p, s["w_k"].double())
            u = u / (u.square().sum(-1, keepdim=True) / D + EPS).sqrt() * s["gamma_k"].double()
            out[i, :, blocks] = _exact_rope(u, blocks, GATE_BASE)
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    group = case["hq"] // case["hkv"]
    for i, n in enumerate(s["lens"]):
        last = (n - 1) // BLK
        for h in range(case["hkv"]):
            if s["sel_idx"] is None:
                blocks = torch.arange(last + 1, device=DEV)
            else:
                blocks = s["sel_idx"][i, h, :int(s["sel_count"][i, h])].long()
            kv = []
            for name in ("k", "v"):
                if s["table"] is not None:
                    page = s["table"][i].long()[blocks[:-1]]
                    x = s[name].view(torch.uint8)[page, h].view(s[name].dtype).double()
                    x = x * s[name + "_scale"][page, h].double()[:, None, None]
                else:
                    x = s[name][i, h].view(torch.uint8).view(-1, BLK, D)[blocks[:-1]].view(s[name].dtype).double()
                    x = x * s[name + "_scale"][i, h, blocks[:-1]].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, D), s[name + "_tail"][i, h, :n - last * BLK].double()]))
            p = torch.softmax(s["q"][i, h * group:(h + 1) * group].double() @ kv[0].T / math.sqrt(D), -1)
            out[i, h * group:(h + 1) * group] = p @ kv[1]
    return out
