"""How exact the 8-bit decode attention is, on inputs where a coarser arithmetic
shows."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_bounds as N
import kv8_testlib as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [K.E4M3, K.INT8]


def attend(kv, hq, q, out, ws, lists=None, **cfg):
    """sparse_decode_kv8 over every block, or the first len(lists[s]) entries of a list per sequence (one KV head)."""
    cfg = sas.Config(hq, 1, out_dtype=out, **cfg)
    o = torch.full((kv.batch, hq, 128), float("nan"), dtype=sas.out_dtype(cfg), device=DEV)
    sel = cnt = None
    if lists is not None:
        sel = torch.full((kv.batch, 1, cfg.max_sel), -7, dtype=torch.int32, device=DEV)
        for s, blocks in enumerate(lists):
            sel[s, 0, :len(blocks)] = torch.tensor(blocks, dtype=torch.int32)
        cnt = torch.tensor([[len(b)] for b in lists], dtype=torch.int32, device=DEV)
    sas.sparse_decode_kv8(cfg, q.to(DEV), kv, sel, cnt, o, ws)
    torch.cuda.synchronize()
    assert sas.get_device_status(ws) == sas.SAS_OK
    return o


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("listed", [False, True])
def test_bf16_output_is_the_fp32_one_rounded(code, chunks, listed):
    """One arithmetic for both outputs: the bf16 output is the fp32 output rounded once, bit for bit."""
    lens = [64 * 90 + 17, 5, 64 * 70, 2049]
    kv = K.make_cache(4, 1, 91, code, True, lens, DEV, seed=17)
    cfg = sas.Config(8, 1)
    n = sas.sparse_decode_kv8_workspace_bytes(cfg, 4) if chunks else 256
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    lists = [[b for b in range(0, (L - 1) // 64, 3)][:31] + [(L - 1) // 64] for L in lens] if listed else None
    a = attend(kv, 8, q, "f32", ws, lists)
    b = attend(kv, 8, q, "bf16", ws, lists)
    assert torch.equal(a.bfloat16(), b)


def check(inputs, code, out):
    kv, q, scale = inputs
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    o = attend(kv, 8, q, out, ws, attn_scale=scale).cpu().double()
    for s, qh, k, v, tail in N.heads(kv, q):
        want, tol = N.tolerance(qh, k, v, tail, scale, code, out)
        err = (o[s] - want).abs()
        assert bool((err <= tol).all()), (s, float((err / tol).max()))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("peak", [64.0, 300.0])
def test_dominant_query_channel(code, out, peak):
    """The other channels keep their bf16 values."""
    check(N.outlier(code, peak, DEV), code, out)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("stored", [False, True])
def test_terms_of_p(code, stored):
    """Exact logits: what the terms of P leave is all there is."""
    check(N.one_channel(code, stored, DEV), code, "f32")


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("low", [0, -60, -117, 117])
def test_queries_and_keys_at_opposite_ends(code, low):
    """Queries 2^low, keys as much larger or smaller: their products, and so the bounds, are those of low = 0."""
    lens = [640 + 7]
    kv = K.make_cache(1, 1, 11, code, False, lens, "cpu", seed=9)
    kv.k_scale.mul_(2.0 ** -low)
    kv.k_tail.mul_(2.0 ** -low)
    q = (torch.randn((1, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16().float() * 2.0 ** low).bfloat16()
    check((N.moved(kv, DEV), q, 0.08), code, "f32")
