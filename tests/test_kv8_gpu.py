"""The 8-bit KV cache against float64 restatements of its definitions.

Exact (bit for bit): codes, scales, tails and read-back values -- every one of
them is a single rounding of a quantity the definition fixes.  Attention: one
rounding of the output (2^-8 of it in bf16); probabilities as f16 (2^-11) when
the output is bf16, else two terms (2^-16 from the tail's two bf16 terms is the
larger one); logits of at most ~60 in fp32 to 2^-19 relative, which moves p by
less than 2^-13 (bf16 output) -- all of it times sum p |v|.  For the fp32 output
the logits of these inputs stay below 8, so the product error 128 * 2^-24 of
sum |q k| moves p by less than 2^-16."""
import math

import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_testlib as K
import sas_testlib as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [K.E4M3, K.INT8]


def ws_for(cfg):
    return sas.make_workspace(cfg, DEV)


def ok(ws):
    torch.cuda.synchronize()
    return sas.get_device_status(ws) == sas.SAS_OK


# ---------------------------------------------------------------- write and read back
def expected(kv, s, h, b):
    """What block b of (s, h) reads back as."""
    c, sc = K.block(kv, "k", s, h, b)
    return c * sc


def check_history(kv, hist_k, hist_v, lens, code):
    """Codes, scales and tails after appends whose tokens were hist [s] = [Hkv][L][128] (bf16, CPU)."""
    for name, hist in (("k", hist_k), ("v", hist_v)):
        for s, L in enumerate(lens):
            if L == 0:
                continue
            for h in range(hist[s].shape[0]):
                for b in range(L // 64):
                    c, sc = K.block(kv, name, s, h, b)
                    want, ws = K.quantise(hist[s][h, 64 * b:64 * b + 64], code)
                    assert torch.equal(c, want), (name, s, h, b)
                    assert sc == float(torch.tensor(ws, dtype=torch.float64).float()), (name, s, h, b)
                cur = (L - 1) // 64
                tail = getattr(kv, name + "_tail")[s, h, :L - 64 * cur].cpu()
                assert torch.equal(tail, hist[s][h, 64 * cur:L]), (name, s, h)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("chunks", [[[1], [63], [1], [64], [2]], [[200, 1, 0], [56, 64, 1], [0, 70, 128], [1, 1, 63]],
                                    [[130], [1], [1], [60], [129]]])
def test_append_any_split(code, paged, chunks):
    """Ragged appends in any split give the same cache: the blocks of the whole history quantised once."""
    B, hkv, blocks = len(chunks[0]), 2, 8
    cfg = sas.Config(4, hkv)
    kv = K.make_cache(B, hkv, blocks, code, paged, [1] * B, DEV, seed=5, spare=3)
    kv.seq_lens.zero_()
    ws = ws_for(cfg)
    g = torch.Generator().manual_seed(6)
    hist_k = [torch.zeros(hkv, 0, 128, dtype=torch.bfloat16) for _ in range(B)]
    hist_v = [x.clone() for x in hist_k]
    lens = [0] * B
    for step, new in enumerate(chunks):
        n = sum(new)
        kvn = (torch.randn((n, 2, hkv, 128), generator=g) * (1 + 10 * step)).bfloat16()
        starts = [sum(new[:i]) for i in range(B)]
        for i in range(B):
            lens[i] += new[i]
            hist_k[i] = torch.cat([hist_k[i], kvn[starts[i]:starts[i] + new[i], 0].transpose(0, 1)], 1)
            hist_v[i] = torch.cat([hist_v[i], kvn[starts[i]:starts[i] + new[i], 1].transpose(0, 1)], 1)
        d = kvn.to(DEV)
        kv.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        before = kv.k_tail.clone()
        sas.kv8_append(cfg, kv, d[:, 0].transpose(0, 1)[None], d[:, 1].transpose(0, 1)[None], ws,
                       new_starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                       new_lens=torch.tensor(new, dtype=torch.int32, device=DEV), max_new=max(new))
        # a sequence without a token has length 0 and nothing new: it is left alone
        assert ok(ws)
        check_history(kv, hist_k, hist_v, lens, code)
        for i, L in enumerate(lens):                                # tail rows past the length stay
            r = (L - 1) % 64 + 1 if L else 0
            kept = before[i, :, r:], kv.k_tail[i, :, r:]
            if L and (L - new[i]) // 64 == (L - 1) // 64:           # same block: nothing above was written
                assert torch.equal(kept[0].view(torch.int16), kept[1].view(torch.int16))


def test_shared_prefix_and_cutting_back():
    """A sequence that starts on another's completed pages, and one cut back within its current block, go on as if
    they had been written alone."""
    cfg = sas.Config(2, 1)
    kv = K.make_cache(2, 1, 5, K.E4M3, True, [1, 1], DEV, seed=8, spare=1)
    ws = ws_for(cfg)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 1, 200, 128, generator=g).bfloat16()
    y = torch.randn(1, 1, 80, 128, generator=g).bfloat16()
    one = lambda n: torch.tensor(n, dtype=torch.int32, device=DEV)  # noqa: E731

    def append(rows, lens, new, starts):
        kv.seq_lens.copy_(one(lens))
        r = rows.to(DEV)
        sas.kv8_append(cfg, kv, r, r, ws, new_starts=one(starts), new_lens=one(new), max_new=max(new))
    append(x, [200, 0], [200, 0], [0, 0])
    append(x[:, :, :7], [195 + 7, 0], [7, 0], [0, 0])                # cut back to 195, seven more
    kv.block_table[1, :2] = kv.block_table[0, :2]                    # the first two pages of sequence 0
    append(y, [202, 128 + 80], [0, 80], [0, 0])
    assert ok(ws)
    a = torch.cat([x[0, 0, :195], x[0, 0, :7]])
    b = torch.cat([x[0, 0, :128], y[0, 0]])
    check_history(kv, [a[None], b[None]], [a[None], b[None]], [202, 208], K.E4M3)
    q, o = run_attend(kv, cfg, 2, None, ws)
    assert ok(ws)
    check_attend(kv, cfg, 2, None, q, o, [202, 208])


def test_append_padded_batch_strided_rows():
    """[B][Hkv][T][128] inputs (views of a packed projection), max_new for all."""
    B, hkv, T_ = 2, 3, 77
    cfg = sas.Config(6, hkv)
    kv = K.make_cache(B, hkv, 4, K.INT8, False, [77, 77], DEV, seed=8)
    ws = ws_for(cfg)
    x = torch.randn((B, T_, 4 * hkv, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    d = x.to(DEV)
    sas.kv8_append(cfg, kv, d[:, :, hkv:2 * hkv].transpose(1, 2), d[:, :, 2 * hkv:3 * hkv].transpose(1, 2), ws)
    assert ok(ws)
    check_history(kv, [x[i, :, hkv:2 * hkv].transpose(0, 1) for i in range(B)],
                  [x[i, :, 2 * hkv:3 * hkv].transpose(0, 1) for i in range(B)], [77, 77], K.INT8)


@pytest.mark.parametrize("code", CODES)
def test_quantiser_values(code):
    """Ties, the range's ends, tiny and huge blocks, zeros, and blocks with NaN or infinity."""
    hkv, nb = 1, 8
    cfg = sas.Config(1, 1)
    x = torch.zeros(1, hkv, nb * 64, 128)
    b = x.view(nb, 64, 128)
    b[0] = torch.linspace(-1, 1, 64 * 128).view(64, 128)            # amax 1: half-way codes occur (int8: x = amax / 2)
    b[0, 0, :4] = torch.tensor([0.5, -0.5, 1.0, -1.0])
    k = torch.arange(64 * 128) % 254                                # multiples of amax / 254: every int8 tie
    b[1] = ((k - 127).float() * 2.0 ** -3).view(64, 128)
    b[1, 0, 0] = 254 * 2.0 ** -3 / 2 * 2
    b[2] = 3.0e38                                                   # near bf16's largest
    b[2, 0, 0] = 1e30
    b[3] = 2.0 ** -110                                              # below the smallest magnitude a scale stands for
    b[3, 5, 5] = 2.0 ** -101
    b[4] = 0.0
    b[5] = torch.randn(64, 128, generator=torch.Generator().manual_seed(2)) * 1e-30
    b[6, 3, 3] = math.nan
    b[7, 9, 9] = -math.inf
    x = x.bfloat16()
    kv = K.make_cache(1, hkv, nb, code, False, [nb * 64], DEV)
    ws = ws_for(cfg)
    sas.kv8_append(cfg, kv, x.to(DEV), x.to(DEV), ws)
    assert ok(ws)
    for i in range(nb):
        c, sc = K.block(kv, "k", 0, 0, i)
        want, w = K.quantise(x[0, 0, 64 * i:64 * i + 64], code)
        assert torch.equal(c, want), i
        if i < 6:
            assert sc == float(torch.tensor(w, dtype=torch.float64).float()), i
        else:
            assert math.isnan(sc)
    out = torch.zeros(1, 1, nb * 64, 128, dtype=torch.bfloat16, device=DEV)
    sas.kv8_read(cfg, kv, out, None, ws)
    assert bool(out[0, 0, 6 * 64:7 * 64].isnan().all()) and bool(out[0, 0, :6 * 64].isfinite().all())
    assert torch.equal(out[0, 0, 7 * 64:].cpu(), x[0, 0, 7 * 64:])   # the last block is current: read from the tail


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_read_back(code, paged, out):
    lens = [1, 64, 65, 300]
    B, hkv = len(lens), 2
    cfg = sas.Config(2, hkv, out_dtype=out)
    kv = K.make_cache(B, hkv, 6, code, paged, lens, DEV, seed=3)
    ws = ws_for(cfg)
    dt = sas.out_dtype(cfg)
    for begin, n in (([0, 0, 0, 0], 320), ([0, 63, 1, 250], 70), ([0, 0, 64, 299], 1)):
        ko = torch.full((B, n, hkv, 128), 9.0, dtype=dt, device=DEV).transpose(1, 2)
        vo = torch.full((B, hkv, n, 128), 9.0, dtype=dt, device=DEV)
        sas.kv8_read(cfg, kv, ko, vo, ws, begin=torch.tensor(begin, dtype=torch.int32, device=DEV))
        assert ok(ws)
        for name, got in (("k", ko), ("v", vo)):
            for s, L in enumerate(lens):
                for h in range(hkv):
                    # the product in float64 is exact (24 + 8 bits): one rounding to fp32, one to the output's type
                    all_ = K.tokens(kv, name, s, h, range((L - 1) // 64 + 1), L).float().to(dt)
                    want = all_[begin[s]:begin[s] + n]
                    assert torch.equal(got[s, h, :want.shape[0]].cpu(), want), (name, s, h)
                    assert bool((got[s, h, want.shape[0]:] == 9.0).all())


def test_empty_slots():
    """Length 0: append with nothing new, read-back and pooling leave the slot alone and report nothing; the
    attention, like the bf16 one, reports it and zeroes its output."""
    cfg = sas.Config(2, 1)
    kv = K.make_cache(3, 1, 4, K.INT8, True, [130, 1, 64], DEV, seed=4)
    kv.seq_lens[1] = 0
    ws = ws_for(cfg)
    x = torch.zeros(3, 1, 1, 128, dtype=torch.bfloat16, device=DEV)
    before = [t.clone() for t in (kv.k, kv.k_tail.view(torch.int16), kv.k_scale)]
    sas.kv8_append(cfg, kv, x, x, ws, new_lens=torch.zeros(3, dtype=torch.int32, device=DEV))
    out = torch.full((3, 1, 130, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    sas.kv8_read(cfg, kv, out, None, ws)
    gk = torch.full((3, 1, 4, 128), 5.0, device=DEV)
    sas.pool_keys_kv8(cfg, kv, torch.zeros(1, 384, 128, dtype=torch.bfloat16, device=DEV), torch.ones(128, device=DEV),
                      gk, ws)
    assert ok(ws) and bool((out[1] == 5).all()) and bool((gk[1] == 5).all())
    assert torch.equal(kv.k, before[0]) and torch.equal(kv.k_tail.view(torch.int16), before[1])
    assert torch.equal(kv.k_scale, before[2])
    q, o = run_attend(kv, cfg, 2, None, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_ERR_DEVICE_BOUNDS and float(o[1].float().abs().max()) == 0
    for s, L in ((0, 130), (2, 64)):
        want, size = K.attend(kv, q, s, 0, 2, list(range((L - 1) // 64 + 1)), L, cfg.attn_scale)
        assert bool(((o[s].cpu().double() - want).abs() <= 2.0 ** -10 * size + 2.0 ** -8 * want.abs()).all())


# ---------------------------------------------------------------- gate keys
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("gk16", [0, 1])
@pytest.mark.parametrize("hkv", [1, 12])           # one CTA a block, and 128 blocks a CTA
def test_pool_keys(code, paged, gk16, hkv):
    from oracle import sas_oracle as O
    lens = [64, 63, 700, 64 * 140 + 5]
    B, blocks = len(lens), 142
    cfg = sas.Config(hkv, hkv, gate_keys_bf16=gk16)
    kv = K.make_cache(B, hkv, blocks, code, paged, lens, DEV, seed=11)
    ws = ws_for(cfg)
    g = torch.Generator().manual_seed(4)
    w_k = (torch.randn((hkv, 384, 128), generator=g) / 384 ** 0.5).bfloat16().to(DEV)
    gamma = (1 + 0.25 * torch.randn(128, generator=g)).to(DEV)
    gk = torch.full((B, hkv, blocks, 128), 3.0, dtype=sas.gate_key_dtype(cfg), device=DEV)
    raw = torch.full((B, hkv, blocks, 384), 3.0, device=DEV)
    sas.pool_keys_kv8(cfg, kv, w_k, gamma, gk, ws, pooled_raw=raw)
    assert ok(ws)
    for s, L in enumerate(lens):
        n = L // 64
        assert bool((gk[s, :, n:] == 3).all()) and bool((raw[s, :, n:] == 3).all())
        for h in sorted({0, hkv - 1}):
            if n == 0:
                continue
            want_raw, vals = [], []
            for b in range(n):
                c, sc = K.block(kv, "k", s, h, b)
                p = torch.cat([c.max(0).values, c.min(0).values, c.mean(0)])
                want_raw.append((p * sc).float())                   # code units are exact: one fp32 rounding
                vals.append(c * sc)
            assert torch.equal(raw[s, h, :n].cpu(), torch.stack(want_raw))
            want = O.gate_keys_for_sequence(torch.cat(vals).numpy(), n, w_k[h].double().cpu().numpy(),
                                            gamma.double().cpu().numpy())
            rtol = T.BF16_ULP if gk16 else T.SCORE_RTOL
            T.assert_close_rel(gk[s, h, :n].double().cpu().numpy(), want, f"gate keys {s} {h}", rtol=rtol)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("step", [1, 7, 20])
def test_pool_keys_incremental_agrees_with_all_at_once(code, step):
    """Few blocks and many take different kernels, whose fp32 sums run in different orders: 384 products each, so
    the two agree to the bar of the gate keys; the same call twice is bit-identical."""
    n = 60
    lens = [64 * n, 64 * 37 + 3]
    kv = K.make_cache(2, 8, n, code, True, lens, DEV, seed=12)
    cfg = sas.Config(8, 8)
    ws = ws_for(cfg)
    w_k = (torch.randn((8, 384, 128), generator=torch.Generator().manual_seed(4)) / 20).bfloat16().to(DEV)
    gamma = torch.ones(128, device=DEV)
    a, a2, b = (torch.zeros(2, 8, n, 128, device=DEV) for _ in range(3))
    ra, rb = (torch.zeros(2, 8, n, 384, device=DEV) for _ in range(2))
    sas.pool_keys_kv8(cfg, kv, w_k, gamma, a, ws, pooled_raw=ra)
    sas.pool_keys_kv8(cfg, kv, w_k, gamma, a2, ws)
    for i in range(0, n, step):
        sas.pool_keys_kv8(cfg, kv, w_k, gamma, b, ws, num_blocks=step, pooled_raw=rb,
                          blk_begin=torch.tensor([i, n - step - i], dtype=torch.int32, device=DEV))
    assert ok(ws) and torch.equal(a, a2)
    assert torch.equal(ra[0], rb[0]) and torch.equal(a == 0, b == 0)
    T.assert_close_rel(b.cpu().numpy(), a.cpu().numpy(), "incremental")


# ---------------------------------------------------------------- attention
def run_attend(kv, cfg, G, lists, ws, seed=20, q=None):
    B, hkv = kv.batch, cfg.num_kv_heads
    if q is None:
        q = torch.randn((B, hkv * G, 128), generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
    out = torch.full((B, hkv * G, 128), float("nan"), dtype=sas.out_dtype(cfg), device=DEV)
    sel = cnt = None
    if lists is not None:
        sel = torch.full((B, hkv, cfg.max_sel), -7, dtype=torch.int32, device=DEV)
        cnt = torch.zeros((B, hkv), dtype=torch.int32, device=DEV)
        for s in range(B):
            for h in range(hkv):
                sel[s, h, :len(lists[s][h])] = torch.tensor(lists[s][h], dtype=torch.int32)
                cnt[s, h] = len(lists[s][h])
    sas.sparse_decode_kv8(cfg, q, kv, sel, cnt, out, ws)
    return q, out


def check_attend(kv, cfg, G, lists, q, out, lens):
    f32 = cfg.out_dtype == "f32"
    for s, L in enumerate(lens):
        for h in range(cfg.num_kv_heads):
            blocks = lists[s][h] if lists is not None else list(range((L - 1) // 64 + 1))
            want, size = K.attend(kv, q, s, h, G, blocks, L, cfg.attn_scale)
            err = (out[s, h * G:(h + 1) * G].cpu().double() - want).abs()
            tol = (2.0 ** -15 if f32 else 2.0 ** -11 + 2.0 ** -13) * size + (2.0 ** -23 if f32 else 2.0 ** -8) * want.abs()
            assert bool((err <= tol).all()), (s, h, float((err / tol.clamp_min(1e-30)).max()))


def random_lists(lens, hkv, keep, seed):
    g = torch.Generator().manual_seed(seed)
    out = []
    for L in lens:
        c = (L - 1) // 64
        out.append([sorted(torch.randperm(c, generator=g)[:keep - 1].tolist()) + [c] for _ in range(hkv)])
    return out


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8])
def test_attend_groups(code, out, G):
    lens = [1, 17, 64, 65, 1000, 2047]
    cfg = sas.Config(2 * G, 2, token_budget=512, out_dtype=out)
    kv = K.make_cache(len(lens), 2, 32, code, G % 2 == 0, lens, DEV, seed=G, spare=2)
    ws = ws_for(cfg)
    lists = random_lists(lens, 2, 8, 7)
    q, o = run_attend(kv, cfg, G, lists, ws)
    assert ok(ws)
    check_attend(kv, cfg, G, lists, q, o, lens)


@pytest.mark.parametrize("B", [3, 40, 100, 200, 300])   # clusters of 8, 4, 2, 1 and 2
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_attend_cluster_sizes(B, out):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 64 * 40, (B,), generator=g).tolist()
    lens[0], lens[1] = 64 * 40, 1
    code = K.INT8 if B % 3 else K.E4M3
    cfg = sas.Config(5, 1, token_budget=64 * 24, out_dtype=out)
    kv = K.make_cache(B, 1, 40, code, True, lens, DEV, seed=B)
    ws = ws_for(cfg)
    lists = random_lists(lens, 1, 24, 8)
    q, o = run_attend(kv, cfg, 5, lists, ws)
    assert ok(ws)
    q2, o2 = run_attend(kv, cfg, 5, lists, ws)
    assert torch.equal(o, o2)
    keep = [0, 1] + torch.randperm(B, generator=g)[:20].tolist()
    for s in keep:
        want, size = K.attend(kv, q, s, 0, 5, lists[s][0], lens[s], cfg.attn_scale)
        tol = (2.0 ** -15 if out == "f32" else 2.0 ** -11 + 2.0 ** -13) * size
        tol = tol + (2.0 ** -23 if out == "f32" else 2.0 ** -8) * want.abs()
        assert bool(((o[s].cpu().double() - want).abs() <= tol).all()), s


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("budget", [64, 128, 192, 1024, 4096, 16384])
def test_attend_budgets(code, budget):
    lens = [64 * 300 + 31, 40, 64 * 70]
    cfg = sas.Config(4, 1, token_budget=budget)
    kv = K.make_cache(3, 1, 301, code, True, lens, DEV, seed=2)
    ws = ws_for(cfg)
    lists = random_lists(lens, 1, budget // 64, 8)
    q, o = run_attend(kv, cfg, 4, lists, ws)
    assert ok(ws)
    check_attend(kv, cfg, 4, lists, q, o, lens)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("lens", [[1], [64], [129, 1], [5000, 3, 2500], [30001]])
def test_attend_every_block(code, paged, lens):
    cfg = sas.Config(6, 2, out_dtype="f32" if len(lens) == 2 else "bf16")
    kv = K.make_cache(len(lens), 2, (max(lens) + 63) // 64, code, paged, lens, DEV, seed=3)
    ws = ws_for(cfg)
    q, o = run_attend(kv, cfg, 3, None, ws)
    assert ok(ws)
    check_attend(kv, cfg, 3, None, q, o, lens)


def chunk_ws(cfg, B):
    return torch.full((sas.sparse_decode_kv8_workspace_bytes(cfg, B),), 0, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[30001], [20000, 1, 64, 9000, 65], [4097, 4096, 4095], [70000, 33]])
def test_attend_every_block_in_chunks(code, out, lens):
    """With the larger workspace: few and ragged sequences cut into chunks; left-over contents of the workspace do
    not matter, and two calls agree bit for bit."""
    cfg = sas.Config(6, 2, out_dtype=out)
    kv = K.make_cache(len(lens), 2, (max(lens) + 63) // 64, code, len(lens) != 3, lens, DEV, seed=3)
    ws = chunk_ws(cfg, len(lens))
    ws[256:] = 255
    q, o = run_attend(kv, cfg, 3, None, ws)
    assert ok(ws)
    check_attend(kv, cfg, 3, None, q, o, lens)
    o2 = run_attend(kv, cfg, 3, None, ws)[1]
    assert torch.equal(o, o2)


def test_attend_chunks_many_short_sequences_and_bad_ones():
    """More sequences than a warp, most of them short, some with lengths or pages out of range."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 200, (300,), generator=g).tolist()
    lens[7], lens[299] = 5000, 4800
    cfg = sas.Config(2, 1)
    kv = K.make_cache(300, 1, 80, K.E4M3, True, lens, DEV, seed=4, spare=1)
    ws = chunk_ws(cfg, 300)
    kv.seq_lens[11] = 0
    kv.seq_lens[12] = 80 * 64 + 1
    kv.block_table[299, 3] = -1
    q, o = run_attend(kv, cfg, 2, None, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
    bad = {11, 12, 299}
    for s in bad:
        assert float(o[s].float().abs().max()) == 0
    for s in [0, 7, 10, 13, 150, 255, 256, 298]:
        want, size = K.attend(kv, q, s, 0, 2, list(range((lens[s] - 1) // 64 + 1)), lens[s], cfg.attn_scale)
        assert bool(((o[s].cpu().double() - want).abs() <= 2.0 ** -10 * size + 2.0 ** -8 * want.abs()).all()), s


@pytest.mark.parametrize("scale", [2.0 ** -120, 1e-20, 1.0, 1e15])
def test_attend_query_range(scale):
    """The query is brought into f16's range by a power of two per head: only attn_scale * q counts."""
    lens = [700]
    cfg = sas.Config(4, 1, token_budget=512, attn_scale=float(torch.tensor(0.05 / scale).clamp(max=1e30)))
    kv = K.make_cache(1, 1, 11, K.E4M3, False, lens, DEV, seed=9)
    ws = ws_for(cfg)
    q = (torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(1)) * scale).bfloat16().to(DEV)
    q[0, 2] = 0                                                      # a zero query: the mean of the values
    lists = random_lists(lens, 1, 8, 8)
    q, o = run_attend(kv, cfg, 4, lists, ws, q=q)
    assert ok(ws)
    check_attend(kv, cfg, 4, lists, q, o, lens)


@pytest.mark.parametrize("code", CODES)
def test_attend_largest_queries(code):
    """Queries in bf16's last binade (2^127 and above), keys as much smaller."""
    lens = [700]
    cfg = sas.Config(4, 1, token_budget=512, attn_scale=2.0 ** -34)
    kv = K.make_cache(1, 1, 11, code, False, lens, DEV, seed=9)
    kv.k_scale.mul_(2.0 ** -97)
    kv.k_tail.mul_(2.0 ** -97)
    g = torch.Generator().manual_seed(1)
    q = (1 + 0.98 * torch.rand((1, 4, 128), generator=g)) * 2.0 ** 127 * (torch.randint(0, 2, (1, 4, 128), generator=g) * 2 - 1)
    ws = ws_for(cfg)
    lists = random_lists(lens, 1, 8, 8)
    q, o = run_attend(kv, cfg, 4, lists, ws, q=q.bfloat16().to(DEV))
    assert ok(ws)
    check_attend(kv, cfg, 4, lists, q, o, lens)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out,drop", [("bf16", 23.4), ("f32", 20.4)])
def test_attend_one_key_takes_the_weight(code, out, drop):
    """One key `drop` powers of two above all others, its value zero: the output is the others' share alone."""
    lens = [64 * 40]
    cfg = sas.Config(2, 1, token_budget=4096, attn_scale=1.0, out_dtype=out)
    kv = K.make_cache(1, 1, 40, code, False, lens, DEV, seed=9)
    kv.k.view(torch.uint8).zero_()
    kv.k[0, 0, 0] = torch.ones(128, device=DEV).to(code)
    kv.k_scale.fill_(drop * math.log(2) / 128)
    kv.k_tail.zero_()
    # values in the 16 rows of each block that meet the large key's maximum first
    v = (torch.rand((1, 1, 40, 64, 128), generator=torch.Generator().manual_seed(3)) * 100 + 20).to(code)
    v.view(torch.uint8)[:, :, :, 16:] = 0
    v.view(torch.uint8)[:, :, 0, 0] = 0
    kv.v.copy_(v.view(1, 1, 2560, 128).to(DEV))
    kv.v_tail[:, :, 16:] = 0
    q = torch.ones(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    ws = ws_for(cfg)
    lists = [[list(range(40))]]
    q, o = run_attend(kv, cfg, 2, lists, ws, q=q)
    assert ok(ws)
    check_attend(kv, cfg, 2, lists, q, o, lens)


def test_attend_rising_logits():
    """Logits that grow block by block by far more than the lazy maximum's step."""
    lens = [64 * 40]
    cfg = sas.Config(2, 1, token_budget=4096, attn_scale=1.0)
    kv = K.make_cache(1, 1, 40, K.INT8, False, lens, DEV, seed=9)
    kv.k.fill_(1)
    kv.k_scale.copy_(torch.arange(40, device=DEV).float().view(1, 1, 40) * 0.1)
    kv.k_tail.fill_(-1.0)
    q = torch.ones(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    q[0, 1] = -1.0
    ws = ws_for(cfg)
    lists = [[list(range(40))]]
    q, o = run_attend(kv, cfg, 2, lists, ws, q=q)
    assert ok(ws)
    check_attend(kv, cfg, 2, lists, q, o, lens)


def test_attend_reports_bad_lists_and_pages():
    """Bad lists, lengths and pages: zeros for their (sequence, head) only, and the status bit."""
    lens = [1000, 1000, 1000, 1000, 1000, 1000]
    B = len(lens)
    cfg = sas.Config(4, 2, token_budget=512)
    kv = K.make_cache(B, 2, 16, K.E4M3, True, lens, DEV, seed=1, spare=1)
    ws = ws_for(cfg)
    lists = random_lists(lens, 2, 8, 9)
    lists[0][0] = [3, 3, 15]                 # not ascending
    lists[1][1] = [3, 4]                     # does not end with the current block
    lists[2][0] = [3, 20, 15]                # beyond the current block
    kv.block_table[3, lists[3][0][2]] = 1 << 28
    kv.seq_lens[4] = 16 * 64 + 1             # beyond the cache
    q, o = run_attend(kv, cfg, 2, lists, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
    bad = {(0, 0), (1, 1), (2, 0), (3, 0), (4, 0), (4, 1)}
    if lists[3][0][2] in lists[3][1]:
        bad.add((3, 1))
    for s in range(B):
        for h in range(2):
            got = o[s, 2 * h:2 * h + 2]
            if (s, h) in bad:
                assert float(got.float().abs().max()) == 0, (s, h)
            else:
                want, size = K.attend(kv, q, s, h, 2, lists[s][h], lens[s], cfg.attn_scale)
                assert bool(((got.cpu().double() - want).abs() <= 2.0 ** -10 * size + 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("code", CODES)
def test_poisoned_and_masked_values(code):
    """A listed block with scale NaN makes its (sequence, head) NaN and no other; NaN in stale tail rows, in blocks
    that are not listed and in other sequences' pages does not."""
    lens = [900, 900]
    cfg = sas.Config(4, 2, token_budget=256)
    kv = K.make_cache(2, 2, 15, code, True, lens, DEV, seed=1)
    lists = [[[1, 5, 9, 14], [0, 2, 3, 14]], [[1, 5, 9, 14], [0, 2, 3, 14]]]
    kv.k_scale[kv.block_table[0, 5].long(), 0] = float("nan")        # listed by (0, 0) alone
    kv.v_scale[kv.block_table[1, 4].long()] = float("nan")           # listed by none
    ws = ws_for(cfg)
    q, o = run_attend(kv, cfg, 2, lists, ws)
    assert ok(ws)
    assert bool(o[0, :2].isnan().all())
    for s, h in ((0, 1), (1, 0), (1, 1)):
        want, size = K.attend(kv, q, s, h, 2, lists[s][h], 900, cfg.attn_scale)
        got = o[s, 2 * h:2 * h + 2].cpu().double()
        assert bool(((got - want).abs() <= (2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -8 * want.abs()).all()), (s, h)


def test_append_reports_bad_sequences():
    """Lengths, counts and pages out of range skip their sequence and leave the rest right."""
    B, hkv, n = 6, 1, 70
    cfg = sas.Config(1, hkv)
    kv = K.make_cache(B, hkv, 4, K.INT8, True, [70] * B, DEV, seed=2, spare=1)
    ws = ws_for(cfg)
    kv.seq_lens.copy_(torch.tensor([70, 50, 257, 70, 70, 70], dtype=torch.int32))   # 1: fewer than n; 2: too long
    kv.block_table[3, 0] = -1
    starts = torch.tensor([0, 0, 0, 0, 60, 0], dtype=torch.int32, device=DEV)       # 4: rows past the end
    lens = torch.tensor([70, 70, 70, 70, 70, 71], dtype=torch.int32, device=DEV)    # 5: more than max_new
    x = torch.randn((1, hkv, n, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    before = [t.clone() for t in (kv.k.view(torch.uint8), kv.k_tail.view(torch.int16), kv.k_scale)]
    sas.kv8_append(cfg, kv, x.to(DEV), x.to(DEV), ws, new_starts=starts, new_lens=lens, max_new=70)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
    check_history(kv, [x[0]], [x[0]], [70], K.INT8)
    p = int(kv.block_table[0, 0])
    keep = torch.arange(kv.k.shape[0], device=DEV) != p
    assert torch.equal(kv.k.view(torch.uint8)[keep], before[0][keep])
    assert torch.equal(kv.k_scale[keep], before[2][keep])
    assert torch.equal(kv.k_tail.view(torch.int16)[1:], before[1][1:])


def test_read_reports_bad_pages():
    cfg = sas.Config(1, 1)
    kv = K.make_cache(2, 1, 4, K.INT8, True, [200, 200], DEV, seed=2)
    kv.block_table[0, 1] = 99
    ws = ws_for(cfg)
    out = torch.full((2, 1, 200, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    sas.kv8_read(cfg, kv, out, None, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
    assert float(out[0, 0, 64:128].float().abs().max()) == 0
    kv.block_table[0, 1] = 0
    for s, rows in ((0, list(range(0, 64)) + list(range(128, 200))), (1, list(range(200)))):
        want = K.tokens(kv, "k", s, 0, range(4), 200).float().bfloat16()
        assert torch.equal(out[s, 0, rows].cpu(), want[rows])
