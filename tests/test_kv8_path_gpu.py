"""The 8-bit cache's operators together, as a serving loop uses them: norms and
rotation, append, gate keys, scores, selection and attention, step by step;
eager against synchronised, captured and replayed, on a side stream, with a
shared workspace; and a cache whose codes lie beyond 4 GiB."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas
from oracle import sas_oracle as O

import kv8_testlib as K
import sas_testlib as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
BASE = 1e6


class Layer:
    """One layer's decode state: weights, an 8-bit paged cache, gate keys, outputs."""

    def __init__(self, B, hq, hkv, cap, code, budget, seed, paged=True):
        g = torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.g = B, hq, hkv, g
        self.cfg = sas.Config(hq, hkv, token_budget=budget)
        self.kv = K.make_cache(B, hkv, cap // 64, code, paged, [1] * B, DEV, seed=seed, spare=2, fill=False)
        self.kv.k_scale.zero_(), self.kv.v_scale.zero_(), self.kv.seq_lens.zero_()
        self.ws = sas.make_workspace(self.cfg, DEV)
        self.mg = cap // 64
        self.gate_keys = torch.zeros(B, hkv, self.mg, 128, device=DEV)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.w_q = (r(hq, 128, 128) / 128 ** 0.5).bfloat16().to(DEV)
        self.w_k = (r(hkv, 384, 128) / 384 ** 0.5).bfloat16().to(DEV)
        self.gam = [(1 + 0.25 * r(128)).to(DEV) for _ in range(4)]      # attention q, k; gate q, k
        self.scores = torch.zeros(B, hkv, self.mg, device=DEV)
        self.sel = torch.zeros(B, hkv, budget // 64, dtype=torch.int32, device=DEV)
        self.cnt = torch.zeros(B, hkv, dtype=torch.int32, device=DEV)
        self.out = torch.zeros(B, hq, 128, dtype=torch.bfloat16, device=DEV)
        self.pos = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
        self.blk = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.qkv = torch.zeros(B, 1, hq + 2 * hkv, 128, dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros(B, hq, 1, 128, dtype=torch.bfloat16, device=DEV)

    def tokens(self, n):
        return torch.randn(self.B, n, self.hq + 2 * self.hkv, 128, generator=self.g).bfloat16().to(DEV)

    def prefill(self, lens):
        """The first lens[s] tokens of every sequence (padded batch)."""
        n = max(lens)
        x = self.tokens(n)
        q, k, v = self.views(x)
        pos = torch.arange(n, device=DEV)[None].expand(self.B, n)
        at = torch.tensor(lens, dtype=torch.int32, device=DEV)
        pos = torch.where(pos < at[:, None], pos, -1).to(torch.int32).contiguous()
        sas.qk_norm_rope(self.cfg, None, k, None, self.gam[1], None, k, BASE, positions=pos)
        self.kv.seq_lens.copy_(at)
        sas.kv8_append(self.cfg, self.kv, k, v, self.ws, new_lens=at)
        sas.pool_keys_kv8(self.cfg, self.kv, self.w_k, self.gam[3], self.gate_keys, self.ws)

    def views(self, x):
        return (x[:, :, :self.hq].transpose(1, 2), x[:, :, self.hq:self.hq + self.hkv].transpose(1, 2),
                x[:, :, self.hq + self.hkv:].transpose(1, 2))

    def step(self, sync=False, stream=None):
        """One decode step on self.qkv: every sequence grows by a token."""
        c, kv, ws = self.cfg, self.kv, self.ws
        wait = torch.cuda.synchronize if sync else (lambda: None)
        q, k, v = self.views(self.qkv)
        self.pos.copy_(kv.seq_lens[:, None])
        self.blk.copy_(kv.seq_lens // 64)                              # the block the new token falls in
        kv.seq_lens.add_(1)
        wait()
        sas.qk_norm_rope(c, q, k, self.gam[0], self.gam[1], self.q, k, BASE, positions=self.pos, stream=stream)
        wait()
        sas.kv8_append(c, kv, k, v, ws, stream=stream)
        wait()
        sas.pool_keys_kv8(c, kv, self.w_k, self.gam[3], self.gate_keys, ws, blk_begin=self.blk, num_blocks=1, stream=stream)
        wait()
        q1 = self.q.view(self.B, self.hq, 128)
        sas.gate_scores(c, q1, kv.seq_lens, self.w_q, self.gam[2], self.gate_keys, self.scores, ws, stream=stream)
        wait()
        sas.topk_blocks(c, self.scores, kv.seq_lens, self.sel, self.cnt, ws, stream=stream)
        wait()
        sas.sparse_decode_kv8(c, q1, kv, self.sel, self.cnt, self.out, ws, stream=stream)
        wait()

    def state(self):
        kv = self.kv
        return [t.clone() for t in (self.out, self.sel, self.cnt, self.scores, self.gate_keys, kv.k.view(torch.uint8),
                                    kv.v.view(torch.uint8), kv.k_scale, kv.v_scale, kv.k_tail.view(torch.int16),
                                    kv.v_tail.view(torch.int16), kv.seq_lens, self.q)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("code", [K.E4M3, K.INT8])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_loop_against_the_oracle(code, paged):
    """70 steps from ragged prompts; every tenth one, and those around a block's end, against the oracle on the
    cache's stored values."""
    lens = [1000, 63, 512]
    hq, hkv, G = 8, 2, 4
    L = Layer(3, hq, hkv, 1280, code, 512, 1, paged)
    L.prefill(lens)
    wq, wk = L.w_q.double().cpu().numpy(), L.w_k.double().cpu().numpy()
    gq, gk = L.gam[2].double().cpu().numpy(), L.gam[3].double().cpu().numpy()
    import numpy as np
    for i in range(70):
        L.qkv.copy_(L.tokens(1))
        raw = L.qkv.clone()
        L.step()
        lens = [n + 1 for n in lens]
        if not (i % 10 == 0 or any(n % 64 in (0, 1) for n in lens)):
            continue
        torch.cuda.synchronize()
        assert sas.get_device_status(L.ws) == sas.SAS_OK
        q = L.q.view(3, hq, 128)
        for s, n in enumerate(lens):
            want, size = K.norm_rope(raw[s:s + 1, :, :hq].transpose(1, 2).cpu(), L.gam[0].cpu(),
                                     torch.tensor([[n - 1]]), BASE, 1e-6)
            assert bool(((q[s].cpu().double() - want[0, :, 0]).abs() <= 2.0 ** -8 * want[0, :, 0].abs()
                         + 2.0 ** -19 * size[0, :, 0]).all())
            c = (n - 1) // 64
            for h in range(hkv):
                ks = K.tokens(L.kv, "k", s, h, range(c), n) if c else torch.zeros(0, 128).double()
                keys = O.gate_keys_for_sequence(ks.numpy(), c, wk[h], gk)
                if c:
                    T.assert_close_rel(L.gate_keys[s, h, :c].cpu().numpy(), keys, f"keys {i} {s} {h}")
                stored = L.gate_keys[s, h, :c].double().cpu().numpy()
                qg = q[s, h * G:(h + 1) * G].double().cpu().numpy()
                r = O.decode_one_group(qg, np.zeros((n, 128)), np.zeros((n, 128)), n, stored,
                                       wq[h * G:(h + 1) * G], np.tile(gq, (G, 1)), 512)
                m = int(L.cnt[s, h])
                got = L.sel[s, h, :m].tolist()
                T.assert_selection(got, r["sel"], r["S"], 512 // 64 - 1, f"step {i} {s} {h}")
                want, size = K.attend(L.kv, q, s, h, G, got, n, L.cfg.attn_scale)
                err = (L.out[s, h * G:(h + 1) * G].cpu().double() - want).abs()
                assert bool((err <= (2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -8 * want.abs()).all()), (i, s, h)


def test_back_to_back_captured_and_synchronised_steps_agree():
    """The same 130 steps: one at a time, back to back (overlapping launches), replayed from a graph, and on a side
    stream -- bit for bit."""
    xs = [torch.randn(2, 1, 12, 128, generator=torch.Generator().manual_seed(50 + i)).bfloat16().to(DEV) for i in range(130)]

    def run(how):
        L = Layer(2, 8, 2, 1024, K.E4M3, 256, 3)
        L.prefill([500, 70])
        if how == "graph":
            L.qkv.copy_(xs[0])
            L.step()                                                   # set-up before the capture
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            before = [t.clone() for t in (L.kv.seq_lens, L.qkv)]
            with torch.cuda.graph(g):
                L.step()
            L.kv.seq_lens.copy_(before[0])
            for x in xs[1:]:
                L.qkv.copy_(x)
                g.replay()
        elif how == "stream":
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                for x in xs:
                    L.qkv.copy_(x)
                    L.step(stream=st)
            torch.cuda.current_stream().wait_stream(st)
        else:
            for x in xs:
                L.qkv.copy_(x)
                L.step(sync=how == "sync")
        torch.cuda.synchronize()
        assert sas.get_device_status(L.ws) == sas.SAS_OK
        return L.state()

    want = run("sync")
    for how in ("eager", "graph", "stream"):
        assert same(want, run(how)), how


def test_two_graphs_share_a_workspace():
    """Two layers' captured steps and dense attention in chunks, replayed in turn with one workspace."""
    A, Bl = (Layer(2, 4, 1, 8192, c, 256, s) for c, s in ((K.E4M3, 5), (K.INT8, 6)))
    ws = torch.zeros(sas.sparse_decode_kv8_workspace_bytes(A.cfg, 2), dtype=torch.uint8, device=DEV)
    runs = []
    for L in (A, Bl):
        L.ws = ws
        L.prefill([8000, 5000])
        L.qkv.copy_(L.tokens(1))
        L.step()
        L.dense = torch.zeros_like(L.out)
        sas.sparse_decode_kv8(L.cfg, L.q.view(2, 4, 128), L.kv, None, None, L.dense, ws)
        torch.cuda.synchronize()
        want = L.dense.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sas.sparse_decode_kv8(L.cfg, L.q.view(2, 4, 128), L.kv, None, None, L.dense, ws)
            sas.sparse_decode_kv8(L.cfg, L.q.view(2, 4, 128), L.kv, L.sel, L.cnt, L.out, ws)
        runs.append((g, L, want, L.out.clone()))
    for _ in range(3):
        for g, L, want, out in runs:
            L.dense.zero_(), L.out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, L, want, out in runs:
            assert torch.equal(L.dense, want) and torch.equal(L.out, out)


def test_gradient_captured_and_replayed():
    """The norms' gradient in a graph, beside an eager call with the same workspace."""
    q, k = (torch.randn(2, h, 300, 128, generator=torch.Generator().manual_seed(h)).bfloat16().to(DEV) for h in (4, 2))
    gq = gk = torch.ones(128, device=DEV)
    cfg = sas.Config(4, 2)
    ws = torch.zeros(sas.qk_norm_rope_workspace_bytes(), dtype=torch.uint8, device=DEV)
    dq, dk, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros(2, 128, device=DEV)

    def call():
        dg.zero_()
        sas.qk_norm_rope_backward(cfg, q, k, q, k, gq, gk, dq, dk, dg[0], dg[1], BASE, ws)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dq, dk, dg)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in (dq, dk, dg):
            t.fill_(3.0)
        g.replay()
        call()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (dq, dk, dg)))


@pytest.mark.slow
def test_codes_and_rows_beyond_4_gib():
    """Pages past the 32-bit byte offset, and packed rows past the 32-bit element offset."""
    pages = (1 << 32) // (64 * 128) + 64
    codes = [torch.zeros(pages, 1, 64, 128, dtype=torch.uint8, device=DEV).view(torch.int8) for _ in range(2)]
    scale = [torch.zeros(pages, 1, device=DEV) for _ in range(2)]
    tail = [torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    n = 64 * 5 + 9
    table = torch.tensor([[pages - 1, 3, pages - 7, pages - 2, (1 << 31) // 8192 + 1, 0]], dtype=torch.int32, device=DEV)
    kv = sas.KvCache8(*codes, *scale, *tail, torch.tensor([n], dtype=torch.int32, device=DEV), table)
    cfg = sas.Config(2, 1, token_budget=256)
    ws = sas.make_workspace(cfg, DEV)
    # the new tokens at the end of a buffer of more than 2^31 elements
    stride = (1 << 31) // 300 // 128 * 128 + 128
    big = torch.empty(stride * (n - 1) + 128, dtype=torch.bfloat16, device=DEV)
    rows = big.as_strided((1, 1, n, 128), (0, 128, stride, 1))
    x = torch.randn(n, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    rows.copy_(x.to(DEV)[None, None])
    sas.qk_norm_rope(cfg, None, rows, None, torch.ones(128, device=DEV), None, rows, BASE)
    y = rows[0, 0].cpu()
    want, size = K.norm_rope(x[None, None], torch.ones(128), torch.arange(n)[None], BASE, 1e-6)
    assert bool(((y.double() - want[0, 0]).abs() <= 2.0 ** -8 * want[0, 0].abs() + 2.0 ** -19 * size[0, 0]).all())
    sas.kv8_append(cfg, kv, rows, rows, ws)
    out = torch.zeros(1, 1, n, 128, dtype=torch.bfloat16, device=DEV)
    sas.kv8_read(cfg, kv, out, None, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_OK
    for b in range(5):
        c, sc = K.block(kv, "v", 0, 0, b)
        wc, wsc = K.quantise(y[64 * b:64 * b + 64], K.INT8)
        assert torch.equal(c, wc) and sc == float(torch.tensor(wsc, dtype=torch.float64).float())
        assert torch.equal(out[0, 0, 64 * b:64 * b + 64].cpu(), (c * sc).float().bfloat16())
    q = torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    o = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    sel = torch.tensor([[[0, 2, 4, 5]]], dtype=torch.int32, device=DEV)
    sas.sparse_decode_kv8(cfg, q, kv, sel, torch.full((1, 1), 4, dtype=torch.int32, device=DEV), o, ws)
    want, size = K.attend(kv, q, 0, 0, 2, [0, 2, 4, 5], n, cfg.attn_scale)
    assert bool(((o[0].cpu().double() - want).abs() <= 2.0 ** -10 * size + 2.0 ** -8 * want.abs()).all())
    raw = torch.zeros(1, 1, 6, 384, device=DEV)
    gk = torch.zeros(1, 1, 6, 128, device=DEV)
    wk = torch.ones(1, 384, 128, dtype=torch.bfloat16, device=DEV)
    sas.pool_keys_kv8(cfg, kv, wk, torch.ones(128, device=DEV), gk, ws, pooled_raw=raw)
    c, sc = K.block(kv, "k", 0, 0, 4)
    assert torch.equal(raw[0, 0, 4, :128].cpu(), (c.max(0).values * sc).float())
