"""The norm and 8-bit cache entry points without a GPU: struct layouts against
the header, host validation before any CUDA call (dummy pointers, never
dereferenced), the binding's refusals, and pins of the float64 restatements that
the GPU tests compare with."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from gated_block_sparse_token_b200 import build as B
from gated_block_sparse_token_b200 import sas

import kv8_testlib as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sas.h")
FAKE = 0x100000
OK, INVALID, UNSUPPORTED, WORKSPACE = sas.SAS_OK, sas.SAS_ERR_INVALID_ARG, sas.SAS_ERR_UNSUPPORTED, sas.SAS_ERR_WORKSPACE

nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host validation runs on CPU-only hosts")


@pytest.fixture(scope="module")
def L():
    B.build()
    return sas.lib()


def test_struct_layouts():
    fields = {"sas_rows": (sas._Rows, ["data", "seq_stride", "token_stride", "head_stride", "tokens"]),
              "sas_kv8": (sas._Kv8, ["k", "v", "k_scale", "v_scale", "k_tail", "v_tail", "block_table", "seq_lens",
                                     "batch", "capacity", "num_pages", "max_blocks_per_seq", "code"])}
    body = "".join(f'printf("{t} %zu\\n", sizeof({t}));' + "".join(
        f'printf("{t}.{f} %zu\\n", offsetof({t}, {f}));' for f in fs) for t, (_, fs) in fields.items())
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write('#include <stdio.h>\n#include <stddef.h>\n#include "sas.h"\nint main(void){' + body + "return 0;}")
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), c, "-o", exe], check=True)
        got = dict(l.split() for l in subprocess.run([exe], capture_output=True, text=True).stdout.splitlines())
    for t, (cls, fs) in fields.items():
        assert int(got[t]) == ctypes.sizeof(cls)
        for f in fs:
            assert getattr(cls, f).offset == int(got[f"{t}.{f}"]), (t, f)


def cfg(**kw):
    base = dict(num_q_heads=32, num_kv_heads=8)
    base.update(kw)
    return ctypes.byref(sas.Config(**base).c())


def rows(**kw):
    r = sas._Rows(FAKE, 8 * 64 * 128, 128, 64 * 128, 64)
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.byref(r)


def kv8(**kw):
    v = sas._Kv8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 2, 4096, 0, 0, 0)
    for k, x in kw.items():
        setattr(v, k, x)
    return ctypes.byref(v)


BAD_KV8 = [(dict(code=2), INVALID), (dict(code=-1), INVALID), (dict(batch=-1), INVALID), (dict(k=None), INVALID),
           (dict(v=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_tail=None), INVALID), (dict(k=FAKE + 8), INVALID),
           (dict(v_tail=FAKE + 2), INVALID), (dict(k_scale=FAKE + 2), INVALID), (dict(seq_lens=None), INVALID),
           (dict(capacity=100), INVALID), (dict(capacity=0), INVALID), (dict(block_table=FAKE), INVALID),
           (dict(block_table=FAKE, num_pages=4), INVALID), (dict(block_table=FAKE + 1, num_pages=4, max_blocks_per_seq=4), INVALID),
           (dict(batch=9000), UNSUPPORTED), (dict(batch=8000, capacity=1 << 30), UNSUPPORTED)]


@nogpu
@pytest.mark.parametrize("kw,status", BAD_KV8)
def test_every_cache_call_checks_the_cache(L, kw, status):
    assert L.sas_kv8_append(cfg(), kv8(**kw), rows(), rows(), None, None, 1, FAKE, 256, None) == status
    assert L.sas_kv8_read(cfg(), kv8(**kw), None, 64, rows(), rows(), FAKE, 256, None) == status
    assert L.sas_pool_keys_kv8(cfg(), kv8(**kw), None, 1, FAKE, FAKE, FAKE, 64, None, FAKE, 256, None) == status
    assert L.sas_sparse_decode_kv8(cfg(), FAKE, kv8(**kw), FAKE, FAKE, FAKE, FAKE, 256, None) == status


@nogpu
def test_append_validation(L):
    def call(c=None, kv=None, k=None, v=None, starts=None, lens=None, n=1, ws=FAKE, wsb=256):
        return L.sas_kv8_append(c or cfg(), kv or kv8(), k or rows(), v or rows(), starts, lens, n, ws, wsb, None)
    assert call(c=cfg(kv_dtype="f32")) == UNSUPPORTED
    assert call(n=-1) == INVALID and call(n=0) == OK and call(kv=kv8(batch=0)) == OK
    assert call(ws=None) == WORKSPACE and call(wsb=8) == WORKSPACE and call(ws=FAKE + 4) == WORKSPACE
    assert call(starts=FAKE + 2) == INVALID and call(lens=FAKE + 1) == INVALID
    for bad in (dict(data=None), dict(data=FAKE + 8), dict(token_stride=129), dict(head_stride=-8), dict(seq_stride=4)):
        assert call(k=rows(**bad)) == INVALID and call(v=rows(**bad)) == INVALID
    assert L.sas_kv8_append(cfg(), kv8(), None, rows(), None, None, 1, FAKE, 256, None) == INVALID


@nogpu
def test_read_validation(L):
    def call(c=None, begin=None, n=64, k=None, v=None):
        return L.sas_kv8_read(c or cfg(), kv8(), begin, n, k, v, FAKE, 256, None)
    assert call() == OK and call(n=0, k=rows()) == OK                     # nothing wanted
    assert call(n=-1, k=rows()) == INVALID and call(n=65, k=rows()) == INVALID   # more tokens than rows
    assert call(begin=FAKE + 2, k=rows()) == INVALID
    # outputs whose rows coincide
    for bad in (dict(token_stride=0), dict(head_stride=64), dict(seq_stride=0), dict(data=FAKE + 4)):
        assert call(v=rows(**bad)) == INVALID
    assert call(c=cfg(out_dtype="f32"), k=rows(token_stride=130)) == INVALID


@nogpu
def test_pool_and_attend_validation(L):
    def pool(c=None, begin=None, n=1, wk=FAKE, gk=FAKE, mg=64, raw=None, gam=FAKE):
        return L.sas_pool_keys_kv8(c or cfg(), kv8(), begin, n, wk, gam, gk, mg, raw, FAKE, 256, None)
    assert pool(n=-1) == INVALID and pool(n=0) == OK and pool(mg=0) == INVALID and pool(mg=1 << 20) == INVALID
    assert pool(wk=None) == INVALID and pool(gk=FAKE + 4) == INVALID and pool(raw=FAKE + 1) == INVALID
    assert pool(gam=None) == INVALID and pool(begin=FAKE + 1) == INVALID

    def att(c=None, q=FAKE, idx=FAKE, cnt=FAKE, out=FAKE, wsb=256):
        return L.sas_sparse_decode_kv8(c or cfg(), q, kv8(), idx, cnt, out, FAKE, wsb, None)
    assert att(q=None) == INVALID and att(q=FAKE + 8) == INVALID and att(out=None) == INVALID
    assert att(idx=None) == INVALID and att(cnt=None) == INVALID and att(idx=FAKE + 2) == INVALID
    assert att(c=cfg(kv_dtype="f32")) == UNSUPPORTED and att(c=cfg(gate_mode=1)) == UNSUPPORTED
    assert att(c=cfg(head_dim=64)) == UNSUPPORTED and att(c=cfg(num_q_heads=72)) == UNSUPPORTED and att(wsb=8) == WORKSPACE


@nogpu
def test_norm_validation(L):
    def fwd(c=None, q=1, k=1, gq=FAKE, gk=FAKE, pos=None, b=2, t=64, base=1e6, qo=1, ko=1):
        r = lambda x: rows(seq_stride=32 * 64 * 128) if x == 1 else x  # noqa: E731
        return L.sas_qk_norm_rope(c or cfg(), r(q), r(k), gq, gk, pos, b, t, base, r(qo), r(ko), None)
    assert fwd(b=0) == OK and fwd(t=0) == OK and fwd(q=None, k=None, qo=None, ko=None) == OK
    assert fwd(base=0.0) == INVALID and fwd(base=float("inf")) == INVALID and fwd(b=-1) == INVALID and fwd(t=-1) == INVALID
    assert fwd(gq=None) == INVALID and fwd(qo=None) == INVALID and fwd(q=None) == INVALID and fwd(gk=FAKE + 2) == INVALID
    assert fwd(pos=FAKE + 1) == INVALID and fwd(t=65) == INVALID
    assert fwd(b=1 << 20, t=1 << 10) == UNSUPPORTED
    assert fwd(qo=rows(token_stride=0)) == INVALID and fwd(q=rows(data=FAKE + 8)) == INVALID
    assert fwd(c=cfg(kv_dtype="f32"), q=rows(token_stride=130)) == INVALID
    need = int(L.sas_qk_norm_rope_workspace_bytes())

    def back(ws=FAKE, wsb=need, dq=1, dg=FAKE, t=64, q=1):
        r = lambda x: rows(seq_stride=32 * 64 * 128) if x == 1 else x  # noqa: E731
        return L.sas_qk_norm_rope_backward(cfg(), r(dq), r(1), r(q), r(1), FAKE, FAKE, None, 2, t, 1e6, r(1), r(1), dg,
                                           FAKE, ws, wsb, None)
    assert back(ws=None) == WORKSPACE and back(wsb=need - 1) == WORKSPACE and back(ws=FAKE + 8) == WORKSPACE
    assert back(dq=None) == INVALID and back(dg=None) == INVALID and back(q=None) == INVALID and back(t=0) == OK


def test_workspace_sizes(L):
    c = sas.Config(32, 8)
    sizes = [sas.sparse_decode_kv8_workspace_bytes(c, b) for b in (0, 1, 4, 9, 10, 64, 8000, 1 << 28)]
    assert sizes == sorted(sizes) and sizes[0] == 256
    assert sas.workspace_bytes(c) == 256                                   # every other call needs the status word alone


def _cache(**kw):
    t = dict(k=torch.zeros(6, 2, 64, 128, dtype=torch.int8), v=torch.zeros(6, 2, 64, 128, dtype=torch.int8),
             k_scale=torch.zeros(6, 2), v_scale=torch.zeros(6, 2), k_tail=torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16),
             v_tail=torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16), seq_lens=torch.ones(3, dtype=torch.int32),
             block_table=torch.zeros(3, 2, dtype=torch.int32))
    t.update(kw)
    return sas.KvCache8(**t)


def test_cache_object_refuses_mismatched_tensors():
    good = _cache()
    assert good.batch == 3 and good.kv_heads == 2 and good.c(sas.Config(2, 2)).code == sas.KV8_INT8
    z = torch.zeros
    for kw in (dict(k=z(6, 2, 64, 128)), dict(v=z(6, 2, 64, 128, dtype=torch.float8_e4m3fn)),
               dict(k=z(6, 2, 32, 128, dtype=torch.int8)), dict(k=z(6, 2, 64, 256, dtype=torch.int8)[..., :128]),
               dict(k_scale=z(6, 3)), dict(v_scale=z(6, 2, dtype=torch.bfloat16)), dict(k_tail=z(2, 2, 64, 128, dtype=torch.bfloat16)),
               dict(v_tail=z(3, 2, 64, 128)), dict(seq_lens=z(3, dtype=torch.int64)), dict(block_table=z(3, 2, dtype=torch.int64)),
               dict(block_table=z(2, 2, dtype=torch.int32)), dict(block_table=None)):
        with pytest.raises(ValueError):
            _cache(**kw)
    with pytest.raises(ValueError):
        good.c(sas.Config(4, 4))
    with pytest.raises(Exception):
        good.k = good.v                                                    # the description was taken from the tensors


def test_binding_refuses_before_the_library(monkeypatch):
    def no_library():
        raise AssertionError("the library was called")
    monkeypatch.setattr(sas, "lib", no_library)
    c, kv, ws = sas.Config(4, 2), _cache(), torch.zeros(256, dtype=torch.uint8)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    q, k, g = z(1, 4, 5, 128), z(1, 2, 5, 128), torch.ones(128)
    bad = [lambda: sas.qk_norm_rope(c, None, None, g, g, None, None, 1e6),
           lambda: sas.qk_norm_rope(c, q, k, g, g, q, z(1, 2, 4, 128), 1e6),
           lambda: sas.qk_norm_rope(c, q, k, g, g, z(1, 4, 5, 256)[..., ::2], k, 1e6),
           lambda: sas.qk_norm_rope(c, q, k, g.double(), g, q, k, 1e6),
           lambda: sas.qk_norm_rope(c, q, None, g, g, q, k, 1e6),
           lambda: sas.qk_norm_rope(c, q, k, g, g, q, k, 1e6, positions=torch.zeros(5)),
           lambda: sas.qk_norm_rope(c, q.float(), k, g, g, q, k, 1e6),
           lambda: sas.qk_norm_rope_backward(c, q, None, q, k, g, g, q, k, g, g, 1e6, ws),
           lambda: sas.qk_norm_rope_backward(c, q, k, q, k, g, g, q, k, g.bfloat16(), g, 1e6, ws),
           lambda: sas.kv8_append(c, kv, z(2, 2, 1, 128), z(2, 2, 1, 128), ws),
           lambda: sas.kv8_append(c, kv, z(3, 2, 1, 128), z(3, 2, 2, 128), ws),
           lambda: sas.kv8_append(c, kv, z(3, 2, 1, 128), z(3, 2, 1, 128), ws, new_starts=torch.zeros(3, dtype=torch.int32)),
           lambda: sas.kv8_append(c, kv, z(3, 2, 1, 128), z(3, 2, 1, 128), ws, new_lens=torch.zeros(3)),
           lambda: sas.kv8_read(c, kv, None, None, ws), lambda: sas.kv8_read(c, kv, z(3, 2, 5, 128), z(3, 2, 6, 128), ws),
           lambda: sas.kv8_read(c, kv, z(3, 2, 5, 128, d=torch.float32), None, ws),
           lambda: sas.pool_keys_kv8(c, kv, z(2, 384, 128), g, torch.zeros(3, 2, 4, 64), ws),
           lambda: sas.sparse_decode_kv8(c, z(3, 4, 128), kv, torch.zeros(3, 2, 32, dtype=torch.int32), None, z(3, 4, 128), ws),
           lambda: sas.sparse_decode_kv8(c, z(3, 4, 128), kv, None, None, z(3, 4, 128, d=torch.float32), ws),
           lambda: sas.sparse_decode_kv8(c, z(3, 4, 128), kv, torch.zeros(3, 2, 31, dtype=torch.int32),
                                         torch.zeros(3, 2, dtype=torch.int32), z(3, 4, 128), ws)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")


# ---------------------------------------------------------------- pins of the restatements
def test_restated_norm_gradient_matches_differences():
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(1, 2, 3, 128, generator=g).double(), torch.randn(1, 2, 3, 128, generator=g).double()
    gamma = (1 + 0.2 * torch.randn(128, generator=g)).double()
    pos = torch.tensor([[5, -1, 70000]])
    live = (pos >= 0)[:, None, :, None]
    loss = lambda x, gamma: float((K.norm_rope(x, gamma, pos.clamp_min(0), 1e4, 1e-6)[0] * w * live).sum())  # noqa: E731
    dx, _, dg, _ = K.norm_rope_grad(x, gamma, pos, 1e4, 1e-6, w)
    h = 1e-6
    for i in (0, 63, 64, 130, 300, 700, 767):
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        # rounding of two sums of ~500 terms over 2h, and the h^2 term
        assert abs((loss(a, gamma) - loss(b, gamma)) / (2 * h) - float((dx * live).view(-1)[i])) < 1e-6
    for i in (0, 64, 127):
        a, b = gamma.clone(), gamma.clone()
        a[i] += h
        b[i] -= h
        assert abs((loss(x, a) - loss(x, b)) / (2 * h) - float(dg[i])) < 1e-6


def test_restated_rotation_is_the_closed_form():
    x = torch.zeros(1, 128, dtype=torch.float64)
    x[0, 0] = 1.0                                               # pair (0, 64): one turn per 2 pi positions
    y = K.rotate(x, torch.tensor([3]), 1e4)
    assert abs(float(y[0, 0]) - -0.9899924966004454) < 1e-15 and abs(float(y[0, 64]) - 0.1411200080598672) < 1e-15
    assert torch.allclose(K.rotate(y, torch.tensor([3]), 1e4, back=True), x, atol=1e-15)


@pytest.mark.parametrize("code", [K.E4M3, K.INT8])
def test_restated_quantiser(code):
    """Against torch's own 32-bit casts, and ties by hand."""
    g = torch.Generator().manual_seed(1)
    for scale in (1e-20, 1.0, 3e5):
        x = (torch.randn(64, 128, generator=g) * scale).bfloat16()
        c, s = K.quantise(x, code)
        a = float(x.abs().max())
        y = x.float() * K.QMAX[code] / torch.tensor(a)
        want = y.to(torch.float8_e4m3fn).double() if code == K.E4M3 else y.round().double()
        assert torch.equal(c, want) and s == a / K.QMAX[code]
    x = torch.zeros(64, 128, dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 1.0, 0.5                                 # 63.5 -> 64 (even); 224 is a code
    assert float(K.quantise(x, code)[0][0, 1]) == (64.0 if code == K.INT8 else 224.0)
