"""The 8-bit cache's write, read-back and attention at the ends of their ranges
and in the loops that only many blocks reach.

Attention over few distinct pages that many blocks share: the float64 side then
weighs every page by how often it is listed."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_bounds as N
import kv8_testlib as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [K.E4M3, K.INT8]
INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1


def status(ws):
    torch.cuda.synchronize()
    return sas.get_device_status(ws)


def test_append_lengths_at_the_ends_of_int32():
    """A length that no count can be taken from is reported like every other bad one, and writes nothing."""
    lens = [INT_MIN, INT_MIN + 3, -1, INT_MAX, 70]
    cfg = sas.Config(1, 1)
    kv = K.make_cache(5, 1, 4, K.INT8, False, [70] * 5, DEV, seed=2)
    x = torch.randn((5, 1, 70, 128), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    before = [t.clone() for t in (kv.k.view(torch.uint8), kv.v.view(torch.uint8), kv.k_scale, kv.k_tail.view(torch.int16),
                                  kv.v_tail.view(torch.int16))]
    new = torch.tensor([1, 70, 70, 70, 70], dtype=torch.int32, device=DEV)
    for n in (None, new):
        ws = sas.make_workspace(cfg, DEV)
        kv.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        sas.kv8_append(cfg, kv, x, x, ws, new_lens=n)
        assert status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
        for t, b in zip((kv.k.view(torch.uint8), kv.v.view(torch.uint8), kv.k_scale, kv.k_tail.view(torch.int16),
                         kv.v_tail.view(torch.int16)), before):
            assert torch.equal(t[:4], b[:4])
        assert torch.equal(kv.k_tail[4, 0, :6].cpu(), x[4, 0, 64:].cpu())


# ---------------------------------------------------------------- loops of the write and the read-back
def expected(kv, name, s, L, dt):
    """What [Hkv][L][128] reads back as, on the GPU: one fp32 product and one rounding to dt."""
    cur = (L - 1) // 64
    c, sc = getattr(kv, name), getattr(kv, name + "_scale")
    if kv.block_table is not None:
        at = kv.block_table[s, :cur].long()
        x = c.view(torch.uint8)[at].view(c.dtype).float() * sc[at][..., None, None]
        x = x.transpose(0, 1).reshape(c.shape[1], cur * 64, 128)
    else:
        x = c[s, :, :cur * 64].float().reshape(c.shape[1], cur, 64, 128) * sc[s, :, :cur, None, None]
        x = x.reshape(c.shape[1], cur * 64, 128)
    return torch.cat([x.to(dt), getattr(kv, name + "_tail")[s, :, :L - cur * 64].to(dt)], 1)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("paged", [False, True])
def test_write_and_read_back_that_walk_over_blocks(code, paged):
    """600 pairs: a CTA writes and reads up to four blocks one after another.  The write agrees bit for bit with the
    same tokens in steps of at most 64, which give a CTA one block; the read-back with code * scale."""
    B, hkv, blocks = 100, 6, 10
    g = torch.Generator().manual_seed(1)
    new = torch.randint(1, 64 * 9, (B,), generator=g).tolist()
    old = torch.randint(0, 64, (B,), generator=g).tolist()
    new[0], new[1], old[0] = 64 * 9, 64 * 9 - 1, 63
    n = max(new) + 64
    kvn = (torch.randn((B, n, 2 * hkv, 128), generator=g) * torch.rand((B, n, 1, 1), generator=g).add(0.1)).bfloat16().to(DEV)
    k, v = kvn[:, :, :hkv].transpose(1, 2), kvn[:, :, hkv:].transpose(1, 2)
    cfg = sas.Config(hkv, hkv)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    caches = []
    for steps in ([old, new], None):
        kv = K.make_cache(B, hkv, blocks, code, paged, [1] * B, DEV, seed=5, fill=False)
        for t in (kv.k_scale, kv.v_scale, kv.k_tail, kv.v_tail, kv.seq_lens):
            t.zero_()
        ws = sas.make_workspace(cfg, DEV)
        if steps is None:
            total = torch.tensor(old) + torch.tensor(new)
            steps = [(total - 64 * i).clamp(0, 64).tolist() for i in range(blocks)]
        at = torch.zeros(B, dtype=torch.int32)
        for step in steps:
            # the rows of this step to the front: token i of a sequence is row i
            rows = at[:, None] + torch.arange(max(step))
            pick = lambda x: x.gather(2, rows[:, None, :, None].clamp_max(n - 1).to(DEV).expand(B, hkv, -1, 128))  # noqa: E731
            at = at + torch.tensor(step, dtype=torch.int32)
            kv.seq_lens.copy_(at)
            sas.kv8_append(cfg, kv, pick(k), pick(v), ws, new_lens=i32(step))
        assert status(ws) == sas.SAS_OK
        caches.append(kv)
    a, b = caches
    for name in ("k", "v"):
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8))
        assert torch.equal(getattr(a, name + "_scale"), getattr(b, name + "_scale"))
    lens = a.seq_lens.tolist()
    for s, L in enumerate(lens):
        r = (L - 1) % 64 + 1
        assert torch.equal(a.k_tail[s, :, :r], b.k_tail[s, :, :r]) and torch.equal(a.v_tail[s, :, :r], b.v_tail[s, :, :r])
    for s in (0, 1, 50):                                             # the definition
        for b in range(lens[s] // 64):
            c, sc = K.block(a, "v", s, 5, b)
            want, w = K.quantise(v[s, 5, 64 * b:64 * b + 64].cpu(), code)
            assert torch.equal(c, want) and sc == float(torch.tensor(w, dtype=torch.float64).float())
    for out in ("bf16", "f32"):
        cfg = sas.Config(hkv, hkv, out_dtype=out)
        dt = sas.out_dtype(cfg)
        begin = [0, 65, 63] + [min(3 * i, lens[i] - 1) for i in range(3, B)]
        count = 64 * blocks - 20
        ko, vo = (torch.full((B, hkv, count, 128), 9.0, dtype=dt, device=DEV) for _ in range(2))
        ws = sas.make_workspace(cfg, DEV)
        sas.kv8_read(cfg, a, ko, vo, ws, begin=i32(begin))
        assert status(ws) == sas.SAS_OK
        for name, got in (("k", ko), ("v", vo)):
            for s, L in enumerate(lens):
                want = expected(a, name, s, L, dt)[:, begin[s]:begin[s] + count]
                assert torch.equal(got[s, :, :want.shape[1]], want), (name, s)
                assert bool((got[s, :, want.shape[1]:] == 9.0).all())
    if paged:                                                        # a page out of range within a walk
        page = int(a.block_table[0, 5])
        a.block_table[0, 5] = 1 << 30
        sas.kv8_read(cfg, a, ko, None, ws)
        assert status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
        a.block_table[0, 5] = page
        want = expected(a, "k", 0, lens[0], dt)[:, :count]
        want[:, 320:384] = 0
        assert torch.equal(ko[0, :, :want.shape[1]], want)


# ---------------------------------------------------------------- loops of the attention
def few_pages(lens, blocks, code, seed, pages=24):
    """One KV head whose sequences' tables list the same few pages over and over."""
    c = K.make_cache(1, 1, pages, code, True, [1], DEV, seed=seed)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    table = torch.randint(0, pages, (B, blocks), generator=g).to(torch.int32).to(DEV)
    tails = [torch.randn((B, 1, 64, 128), generator=g).bfloat16().to(DEV) for _ in range(2)]
    return sas.KvCache8(c.k, c.v, c.k_scale, c.v_scale, *tails, torch.tensor(lens, dtype=torch.int32, device=DEV), table)


def check_few_pages(kv, cfg, q, o, lists, lens, code, but=()):
    pages = kv.k.shape[0]
    ks, vs = ((getattr(kv, n).float().cpu().double() * getattr(kv, n + "_scale").cpu().double()[..., None, None]).reshape(-1, 128)
              for n in ("k", "v"))
    table, o = kv.block_table.cpu(), o.cpu().double()
    for s, L in enumerate(lens):
        if s in but:
            continue
        cur = (L - 1) // 64
        r = L - 64 * cur
        used = table[s, :cur] if lists is None else table[s, torch.tensor(lists[s][:-1], dtype=torch.long)]
        times = torch.bincount(used.long(), minlength=pages).double().repeat_interleave(64)
        keep = times > 0
        k = torch.cat([ks[keep], kv.k_tail[s, 0, :r].cpu().double()])
        v = torch.cat([vs[keep], kv.v_tail[s, 0, :r].cpu().double()])
        times = torch.cat([times[keep], torch.ones(r, dtype=torch.float64)])
        want, tol = N.tolerance(q[s].cpu().double(), k, v, r, cfg.attn_scale, code, cfg.out_dtype, times)
        err = (o[s] - want).abs()
        assert bool((err <= tol).all()), (s, float((err / tol).max()))


def run(kv, cfg, lists, ws, seed=3):
    B, G = kv.batch, cfg.num_q_heads
    q = torch.randn((B, G, 128), generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
    o = torch.full((B, G, 128), float("nan"), dtype=sas.out_dtype(cfg), device=DEV)
    sel = cnt = None
    if lists is not None:
        sel = torch.full((B, 1, cfg.max_sel), -7, dtype=torch.int32)
        for s, blocks in enumerate(lists):
            sel[s, 0, :len(blocks)] = torch.tensor(blocks, dtype=torch.int32)
        sel = sel.to(DEV)
        cnt = torch.tensor([[len(b)] for b in lists], dtype=torch.int32, device=DEV)
    sas.sparse_decode_kv8(cfg, q, kv, sel, cnt, o, ws)
    return q, o


def long_lists(lens, keep, seed):
    g = torch.Generator().manual_seed(seed)
    return [sorted(torch.randperm((L - 1) // 64, generator=g)[:keep - 1].tolist()) + [(L - 1) // 64] for L in lens]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,keep", [(80, 256), (160, 256), (160, 70), (300, 256)])    # clusters of 2, 1, 1 and 2
def test_attend_lists_of_many_blocks(code, out, B, keep):
    """More than 32 stored blocks a group of warps: their numbers are read and checked in portions."""
    g = torch.Generator().manual_seed(B + keep)
    lens = torch.randint(64 * 200, 64 * 400, (B,), generator=g).tolist()
    lens[0], lens[1], lens[2] = 64 * 400, 64 * 129, 64 * 66 + 1
    kv = few_pages(lens, 400, code, B)
    cfg = sas.Config(3, 1, token_budget=64 * keep, out_dtype=out)
    ws = sas.make_workspace(cfg, DEV)
    lists = long_lists(lens, keep, 8)
    q, o = run(kv, cfg, lists, ws)
    assert status(ws) == sas.SAS_OK
    check_few_pages(kv, cfg, q, o, lists, lens, code)


@pytest.mark.parametrize("B", [80, 160])
def test_attend_bad_entries_far_down_the_list(B):
    """Entries past the first portion out of order, past the current block or on a page out of range: zeros for their
    sequence, the status bit, and the others right."""
    lens = [64 * 399 + 5] * B
    kv = few_pages(lens, 400, K.INT8, 9)
    cfg = sas.Config(2, 1, token_budget=64 * 256)
    ws = sas.make_workspace(cfg, DEV)
    lists = long_lists(lens, 256, 8)
    lists[3][200], lists[3][201] = lists[3][201], lists[3][200]
    lists[4][254] = 5000
    lists[5][230] = -1
    kv.block_table[6, lists[6][250]] = 24
    kv.block_table[7, lists[7][129]] = -3
    lists[8][253] = lists[8][254]
    q, o = run(kv, cfg, lists, ws)
    assert status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
    bad = {3, 4, 5, 6, 7, 8}
    for s in bad:
        assert float(o[s].float().abs().max()) == 0, s
    check_few_pages(kv, cfg, q, o, lists, lens, K.INT8, but=bad)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,blocks,chunks", [(1, 1300, False), (160, 300, False), (148, 300, True), (148, 600, True)])
def test_attend_every_block_in_portions(code, out, B, blocks, chunks):
    """The same without lists, by clusters and in chunks of more than 64 blocks."""
    g = torch.Generator().manual_seed(B + blocks)
    lens = torch.randint(64 * (blocks - 40), 64 * blocks, (B,), generator=g).tolist()
    lens[0] = 64 * blocks
    kv = few_pages(lens, blocks, code, B)
    cfg = sas.Config(3, 1, out_dtype=out)
    n = sas.sparse_decode_kv8_workspace_bytes(cfg, B) if chunks else 256
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    q, o = run(kv, cfg, None, ws)
    assert status(ws) == sas.SAS_OK
    check_few_pages(kv, cfg, q, o, None, lens, code)


def test_single_entries_with_odd_strides():
    """One sequence, one head, one token, with whatever strides: norms, write and read-back."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(1, 1, 1, 128, generator=g).bfloat16().to(DEV)
    odd = x.as_strided((1, 1, 1, 128), (3, 5, 7, 1))
    gain = torch.ones(128, device=DEV)
    cfg = sas.Config(1, 1)
    a, b = torch.zeros_like(x), torch.zeros_like(x)
    sas.qk_norm_rope(cfg, x, x, gain, gain, a, b, 1e4)
    c, d = torch.zeros_like(x), torch.zeros_like(x)
    sas.qk_norm_rope(cfg, odd, odd, gain, gain, c.as_strided((1, 1, 1, 128), (1, 1, 1, 1)),
                     d.as_strided((1, 1, 1, 128), (9, 9, 9, 1)), 1e4)
    kv = K.make_cache(1, 1, 2, K.INT8, False, [1], DEV)
    ws = sas.make_workspace(cfg, DEV)
    sas.kv8_append(cfg, kv, odd, odd, ws)
    back = torch.zeros_like(x)
    sas.kv8_read(cfg, kv, back.as_strided((1, 1, 1, 128), (1, 3, 5, 1)), None, ws)
    assert status(ws) == sas.SAS_OK
    assert torch.equal(a, c) and torch.equal(b, d) and torch.equal(back, x)


@pytest.mark.parametrize("B", [1024, 1025])
def test_attend_every_block_of_more_sequences_than_are_cut(B):
    """The most sequences that are cut into chunks, and one more, which go by clusters."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 300, (B,), generator=g).tolist()
    lens[0], lens[1], lens[B - 1], lens[B - 2] = 64 * 70, 1, 64 * 69 + 1, 64 * 40
    kv = few_pages(lens, 70, K.E4M3, 3)
    cfg = sas.Config(2, 1)
    ws = torch.zeros(sas.sparse_decode_kv8_workspace_bytes(cfg, B), dtype=torch.uint8, device=DEV)
    q, o = run(kv, cfg, None, ws)
    assert status(ws) == sas.SAS_OK
    check_few_pages(kv, cfg, q, o, None, lens, K.E4M3)
