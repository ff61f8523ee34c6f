"""sas_qk_norm_rope and its gradient against float64 on the same inputs.

Tolerances: one rounding to bf16 is at most 2^-8 of the value.  The fp32 part:
the reduced angle (2^-23 half turns, times pi), cos and sin (2 ulp), the
reciprocal root (2 ulp), the 128-term sum and five products stay below 2^-19 of
|z_i| + |z_(i+64)| (forward) and 2^-18 of the terms' magnitudes (gradient); the
gain gradient adds fp32 sums of a few hundred terms per lane, below 2^-17 of
the sum of magnitudes."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_testlib as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _inputs(B, T, hq, hkv, dt, layout, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, hq + 2 * hkv, 128), generator=g).to(dt).to(DEV)
    q, k = x[:, :, :hq].transpose(1, 2), x[:, :, hq:hq + hkv].transpose(1, 2)  # views of a packed projection
    if layout == "bhtd":
        q, k = q.contiguous(), k.contiguous()
    gq, gk = (1 + 0.25 * torch.randn(128, generator=g)).to(DEV), (1 + 0.25 * torch.randn(128, generator=g)).to(DEV)
    return q, k, gq, gk, g


CASES = [  # B, T, hq, hkv, dtype, layout, base, first position
    (1, 1, 4, 1, "bf16", "packed", 1e6, 0), (3, 1, 32, 8, "bf16", "packed", 1e6, 131071), (2, 37, 5, 1, "bf16", "bhtd", 1e4, 5),
    (1, 65, 8, 8, "f32", "packed", 1e6, 2_000_000_000), (2, 200, 16, 2, "f32", "bhtd", 1e4, 100_000),
    (1, 1500, 40, 8, "bf16", "packed", 1e6, 0),
]


@pytest.mark.parametrize("B,T,hq,hkv,dt,layout,base,first", CASES)
def test_forward(B, T, hq, hkv, dt, layout, base, first):
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    q, k, gq, gk, g = _inputs(B, T, hq, hkv, dtype, layout, 1)
    pos = (first + torch.arange(B * T).view(B, T)).to(torch.int32)
    cfg = sas.Config(hq, hkv, kv_dtype=dt, norm_eps=EPS)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    sas.qk_norm_rope(cfg, q, k, gq, gk, qo, ko, base, positions=pos.to(DEV))
    torch.cuda.synchronize()
    half = torch.finfo(dtype).eps / 2
    for x, gamma, out in ((q, gq, qo), (k, gk, ko)):
        want, size = K.norm_rope(x.cpu(), gamma.cpu(), pos, base, EPS)
        err = (out.cpu().double() - want).abs()
        assert bool((err <= half * want.abs() + 2.0 ** -19 * size).all()), float(err.max())


@pytest.mark.parametrize("B,T,hq,hkv,dt,layout,base,first", CASES)
def test_gradient(B, T, hq, hkv, dt, layout, base, first):
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    q, k, gq, gk, g = _inputs(B, T, hq, hkv, dtype, layout, 2)
    pos = (first + torch.arange(B * T).view(B, T)).to(torch.int32)
    if T > 1:
        pos[:, T - T // 3:] = -1                                   # padded rows
    cfg = sas.Config(hq, hkv, kv_dtype=dt, norm_eps=EPS)
    dyq = torch.randn(q.shape, generator=g).to(dtype).to(DEV)
    dyk = torch.randn(k.shape, generator=g).to(dtype).to(DEV)
    ws = torch.zeros(sas.qk_norm_rope_workspace_bytes(), dtype=torch.uint8, device=DEV)
    runs = []
    for _ in range(2):
        dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        dgq, dgk = torch.ones(128, device=DEV), torch.full((128,), 2.0, device=DEV)
        sas.qk_norm_rope_backward(cfg, dyq, dyk, q, k, gq, gk, dq, dk, dgq, dgk, base, ws, positions=pos.to(DEV))
        torch.cuda.synchronize()
        runs.append((dq, dk, dgq, dgk))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    half = torch.finfo(dtype).eps / 2
    live = (pos >= 0)[:, None, :, None]
    for x, gamma, dy, dx, dg, start in ((q, gq, dyq, dq, dgq, 1.0), (k, gk, dyk, dk, dgk, 2.0)):
        want, size, wg, gsize = K.norm_rope_grad(x.cpu(), gamma.cpu(), pos, base, EPS, dy.cpu())
        got = dx.cpu().double()
        assert bool((torch.where(live, (got - want).abs() - half * want.abs() - 2.0 ** -18 * size, -1.0) <= 0).all())
        assert bool((torch.where(live, 7.0, got) == 7.0).all())     # padded rows untouched
        assert bool(((dg.cpu().double() - start - wg).abs() <= 2.0 ** -17 * (gsize + start)).all())


def test_gradient_against_differences():
    """Central differences of the fp32 kernel's own forward."""
    B, T, hq, hkv = 1, 3, 2, 1
    q, k, gq, gk, g = _inputs(B, T, hq, hkv, torch.float32, "bhtd", 3)
    cfg = sas.Config(hq, hkv, kv_dtype="f32", norm_eps=EPS)
    wq, wk = torch.randn(q.shape, generator=g).to(DEV), torch.randn(k.shape, generator=g).to(DEV)

    def loss(q, k, gq, gk):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        sas.qk_norm_rope(cfg, q, k, gq, gk, qo, ko, 1e4)
        return float((qo.double() * wq).sum() + (ko.double() * wk).sum())

    ws = torch.zeros(sas.qk_norm_rope_workspace_bytes(), dtype=torch.uint8, device=DEV)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dgq, dgk = torch.zeros(128, device=DEV), torch.zeros(128, device=DEV)
    sas.qk_norm_rope_backward(cfg, wq, wk, q, k, gq, gk, dq, dk, dgq, dgk, 1e4, ws)
    args, grads = [q, k, gq, gk], [dq, dk, dgq, dgk]
    h = 2.0 ** -6
    for n, (x, d) in enumerate(zip(args, grads)):
        for i in (0, 5, 64, 100, x.numel() - 1):
            out = []
            for s in (h, -h):
                y = [a.clone() for a in args]
                y[n].view(-1)[i] += s
                out.append(loss(*y))
            num = (out[0] - out[1]) / (2 * h)
            # third-derivative term h^2/6 f''' (|f'''| of a normalised row below ~30) and the fp32 noise of the two
            # losses (about 400 terms of size ~1, each 2^-21) over 2h
            assert abs(num - float(d.reshape(-1)[i])) <= 30 * h * h / 6 + 400 * 2.0 ** -21 / (2 * h), (n, i)


def test_in_place_one_side_and_default_positions():
    q, k, gq, gk, _ = _inputs(2, 9, 4, 2, torch.bfloat16, "packed", 4)
    cfg = sas.Config(4, 2)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    pos = torch.arange(9, dtype=torch.int32, device=DEV).expand(2, 9).contiguous()
    sas.qk_norm_rope(cfg, q, k, gq, gk, want_q, want_k, 1e6, positions=pos)
    only = torch.empty_like(k)
    sas.qk_norm_rope(cfg, None, k, None, gk, None, only, 1e6)
    sas.qk_norm_rope(cfg, q, k, gq, gk, q, k, 1e6)                  # the packed projection itself
    torch.cuda.synchronize()
    assert torch.equal(only, want_k) and torch.equal(q, want_q) and torch.equal(k, want_k)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_in_place_and_one_side(dt):
    """dx over dy and over x; keys alone; broadcast (stride 0) upstream gradients."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    q, k, gq, gk, g = _inputs(2, 50, 4, 2, dtype, "packed", 6)
    cfg = sas.Config(4, 2, kv_dtype=dt)
    dyq, dyk = torch.randn(q.shape, generator=g).to(dtype).to(DEV), torch.randn(k.shape, generator=g).to(dtype).to(DEV)
    ws = torch.zeros(sas.qk_norm_rope_workspace_bytes(), dtype=torch.uint8, device=DEV)

    def run(dyq, dyk, q, k, dq, dk):
        dg = torch.zeros(2, 128, device=DEV)
        sas.qk_norm_rope_backward(cfg, dyq, dyk, q, k, gq if q is not None else None, gk, dq, dk,
                                  dg[0] if q is not None else None, dg[1], 1e6, ws)
        return dg
    wq, wk = torch.empty_like(q), torch.empty_like(k)
    want = run(dyq, dyk, q, k, wq, wk)
    only = torch.empty_like(k)
    dg = run(None, dyk, None, k, None, only)
    assert torch.equal(only, wk) and torch.equal(dg[1], want[1]) and float(dg[0].abs().max()) == 0
    a, b = dyq.clone(), k.clone()
    dg = run(a, dyk, q, b, a, b)
    assert torch.equal(a, wq) and torch.equal(b, wk) and torch.equal(dg, want)
    one = torch.randn(1, 1, 1, 128, generator=g).to(dtype).to(DEV)
    x, y = torch.empty_like(q), torch.empty_like(k)
    dg = run(one.expand(q.shape), one.expand(k.shape), q, k, x, y)
    x2, y2 = torch.empty_like(q), torch.empty_like(k)
    dg2 = run(one.expand(q.shape).contiguous(), one.expand(k.shape).contiguous(), q, k, x2, y2)
    assert torch.equal(x, x2) and torch.equal(y, y2) and torch.equal(dg, dg2)


def test_one_gain_for_queries_and_keys():
    """One gain and one gradient buffer for both sides: the buffer gets the sum of the two."""
    B, T, hq, hkv = 2, 700, 16, 4
    q, k, gain, _, g = _inputs(B, T, hq, hkv, torch.bfloat16, "packed", 7)
    cfg = sas.Config(hq, hkv, norm_eps=EPS)
    dyq, dyk = torch.randn(q.shape, generator=g).bfloat16().to(DEV), torch.randn(k.shape, generator=g).bfloat16().to(DEV)
    ws = torch.zeros(sas.qk_norm_rope_workspace_bytes(), dtype=torch.uint8, device=DEV)
    pos = torch.arange(T, dtype=torch.int32).expand(B, T)
    sides = [K.norm_rope_grad(x.cpu(), gain.cpu(), pos, 1e4, EPS, dy.cpu()) for x, dy in ((q, dyq), (k, dyk))]
    want, size = sides[0][2] + sides[1][2], sides[0][3] + sides[1][3]
    for _ in range(3):
        dg = torch.ones(128, device=DEV)
        sas.qk_norm_rope_backward(cfg, dyq, dyk, q, k, gain, gain, torch.empty_like(q), torch.empty_like(k), dg, dg,
                                  1e4, ws)
        assert bool(((dg.cpu().double() - 1 - want).abs() <= 2.0 ** -17 * (size + 1)).all())


def test_zero_rows_and_empty_batch():
    """A zero row stays zero (eps carries the norm); an empty batch does nothing."""
    cfg = sas.Config(2, 1)
    gq = torch.ones(128, device=DEV)
    q = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, 1, 3, 128, dtype=torch.bfloat16, device=DEV)
    sas.qk_norm_rope(cfg, q, k, gq, gq, q, k, 1e6)
    assert float(q.abs().max()) == 0 and float(k.abs().max()) == 0
    sas.qk_norm_rope(cfg, q[:0], k[:0], gq, gq, q[:0], k[:0], 1e6)
    sas.qk_norm_rope(cfg, q[:, :, :0], k[:, :, :0], gq, gq, q[:, :, :0], k[:, :, :0], 1e6)
    torch.cuda.synchronize()
