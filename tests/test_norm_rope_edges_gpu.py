"""sas_qk_norm_rope and its gradient where rows contribute nothing (norm_eps 0
with rows that are padded or lie behind the last token; outputs of padded rows),
and the gradient's walk over more tokens than its grid holds.

Tolerances: those of the same sums in the other norm tests -- one rounding of
the output's type, 2^-18 of the terms' magnitudes in dx, 2^-17 of the sum of
magnitudes in the gains' gradient."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_testlib as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sides(B, T, hq, hkv, dtype, seed):
    """(x, gamma, dy) of the queries and of the keys."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return [(r(B, h, T, 128).to(dtype).to(DEV), (1 + 0.25 * r(128)).to(DEV), r(B, h, T, 128).to(dtype).to(DEV))
            for h in (hq, hkv)]


def gradient(two, pos, base, eps, dt):
    """dx, dgamma of both sides (dx filled with 7, the gains' gradient with 1 before)."""
    (q, gq, dyq), (k, gk, dyk) = two
    cfg = sas.Config(q.shape[1], k.shape[1], kv_dtype=dt, norm_eps=eps)
    ws = torch.full((sas.qk_norm_rope_workspace_bytes(),), 255, dtype=torch.uint8, device=DEV)
    dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    dg = torch.ones(2, 128, device=DEV)
    sas.qk_norm_rope_backward(cfg, dyq, dyk, q, k, gq, gk, dq, dk, dg[0], dg[1], base, ws,
                              positions=None if pos is None else pos.to(DEV))
    torch.cuda.synchronize()
    return (dq, dg[0]), (dk, dg[1])


def check_gradient(two, got, pos, base, eps):
    live = (pos >= 0)[:, None, :, None]
    for (x, gamma, dy), (dx, dg) in zip(two, got):
        half = torch.finfo(x.dtype).eps / 2
        want, size, wg, gsize = K.norm_rope_grad(x.cpu(), gamma.cpu(), pos, base, eps, dy.cpu())
        dx = dx.cpu().double()
        assert bool((torch.where(live, (dx - want).abs() - half * want.abs() - 2.0 ** -18 * size, -1.0) <= 0).all())
        assert bool((torch.where(live, 7.0, dx) == 7.0).all())      # padded rows untouched
        assert bool(((dg.cpu().double() - 1 - wg).abs() <= 2.0 ** -17 * (gsize + 1)).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,hq,hkv,pad", [(1, 1, 1, 1, False), (1, 33, 4, 2, False), (2, 32, 4, 2, True), (3, 45, 8, 8, True),
                                            (2, 700, 16, 4, True)])
def test_gradient_without_eps(dt, B, T, hq, hkv, pad):
    """norm_eps 0: rows that are padded and lanes behind the last token, whose mean square is 0, leave no trace."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    two = sides(B, T, hq, hkv, dtype, 11)
    pos = torch.arange(B * T, dtype=torch.int32).view(B, T)
    if pad:
        pos[:, T - T // 3:] = -1
        pos[0, 0] = -5
    check_gradient(two, gradient(two, pos, 1e4, 0.0, dt), pos, 1e4, 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,hq,hkv", [(1, 40_003, 4, 2), (3, 6_700, 2, 1)])
def test_gradient_walks_over_tokens(dt, B, T, hq, hkv):
    """More than 592 x 32 tokens: a CTA takes several groups of them, whose padding differs from one to the next."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    two = sides(B, T, hq, hkv, dtype, 13)
    pos = torch.arange(B * T, dtype=torch.int32).view(B, T)
    g = torch.Generator().manual_seed(5)
    pos[torch.rand((B, T), generator=g) < 0.2] = -1
    pos[:, T // 2:T // 2 + 3000] = -1                              # whole groups without a live row
    got = gradient(two, pos, 1e6, 1e-6, dt)
    check_gradient(two, got, pos, 1e6, 1e-6)
    for a, b in zip(got, gradient(two, pos, 1e6, 1e-6, dt)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,hq,hkv", [(5, 1, 8, 2), (2, 77, 1, 1), (3, 500, 32, 8)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_padded_rows_keep_their_output(dt, B, T, hq, hkv, eps):
    """Forward: a row with a negative position leaves its output as it was, into another tensor and in place, whatever
    its input holds."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    (q, gq, _), (k, gk, _) = sides(B, T, hq, hkv, dtype, 17)
    g = torch.Generator().manual_seed(6)
    pos = torch.arange(B * T, dtype=torch.int32).view(B, T)
    pad = torch.rand((B, T), generator=g) < 0.4
    pad[0, 0] = True
    pos[pad] = -1 - pos[pad]
    live = ~pad[:, None, :, None]
    for x in (q, k):
        x.masked_fill_(~live.to(DEV), float("nan"))
        x[0, :, 0] = 0
    cfg = sas.Config(hq, hkv, kv_dtype=dt, norm_eps=eps)
    qo, ko = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    sas.qk_norm_rope(cfg, q, k, gq, gk, qo, ko, 1e5, positions=pos.to(DEV))
    half = torch.finfo(dtype).eps / 2
    for x, gamma, y in ((q, gq, qo), (k, gk, ko)):
        want, size = K.norm_rope(x.cpu().nan_to_num(1.0), gamma.cpu(), pos.clamp_min(0), 1e5, eps)
        y = y.cpu().double()
        err = torch.where(live, (y - want).abs() - half * want.abs() - 2.0 ** -19 * size, -1.0)
        assert bool((err <= 0).all()) and bool((torch.where(live, 5.0, y) == 5.0).all())
    q0, k0 = q.clone(), k.clone()
    sas.qk_norm_rope(cfg, q, k, gq, gk, q, k, 1e5, positions=pos.to(DEV))
    torch.cuda.synchronize()
    for x, x0, y in ((q, q0, qo), (k, k0, ko)):
        bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
        assert torch.equal(x.view(bits), torch.where(live.to(DEV), y, x0).view(bits))
