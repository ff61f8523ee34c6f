"""sas_qk_norm_rope and its gradient where rows contribute nothing: norm_eps 0
with rows that are padded or lie behind the last token.

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
