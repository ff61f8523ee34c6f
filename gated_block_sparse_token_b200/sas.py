"""Thin ctypes binding of libsas (include/sas.h): argument marshalling only.

Every function here forwards torch tensors' device pointers and sizes to the
C ABI of the same name and raises ``SasError`` on a non-OK status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback.  The
library must have been built (``python -m gated_block_sparse_token_b200.build``).
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass, field
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SAS_LIBRARY selects another build of the same ABI (e.g. the phase-trace build).
LIB_PATH = os.environ.get("SAS_LIBRARY", os.path.join(_HERE, "libsas.so"))
ABI_VERSION = 10            # the include/sas.h this binding marshals for

SAS_OK = 0
SAS_ERR_INVALID_ARG = 1
SAS_ERR_UNSUPPORTED = 2
SAS_ERR_WORKSPACE = 3
SAS_ERR_CUDA = 4
SAS_ERR_DEVICE_BOUNDS = 5
SAS_ERR_TIMEOUT = 6

KV8_E4M3 = 0               # 8-bit cache codes
KV8_INT8 = 1
_CODES = {torch.float8_e4m3fn: KV8_E4M3, torch.int8: KV8_INT8}

GATE_SELECT_ONLY = 0       # selected blocks weighted 1
GATE_LOGSIGMOID_BIAS = 1   # + log(sigmoid(gate score)) on a selected historical block's logits

DTYPE_BF16 = 0
DTYPE_F32 = 1
_DT = {"bf16": DTYPE_BF16, "f32": DTYPE_F32}
_TORCH_DT = {DTYPE_BF16: torch.bfloat16, DTYPE_F32: torch.float32}


class SasError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class _Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("gate_hidden", ctypes.c_int32), ("token_budget", ctypes.c_int32),
                ("rope_base", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("attn_scale", ctypes.c_float), ("gate_scale", ctypes.c_float),
                ("kv_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("gate_mode", ctypes.c_int32), ("gate_keys_bf16", ctypes.c_int32),
                ("static_weights", ctypes.c_int32)]


class _Kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("token_budgets", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("tokens", ctypes.c_int64)]


class _Kv8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("code", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsas.so from the package directory (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gated_block_sparse_token_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfgp, kvp = ctypes.POINTER(_Config), ctypes.POINTER(_Kv)
        kv8p, rwp = ctypes.POINTER(_Kv8), ctypes.POINTER(_Rows)
        sigs = {
            "sas_abi_version": (i32, []),
            "sas_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "sas_workspace_bytes": (sz, [cfgp, i32, i32]),
            "sas_reset_device_status": (ctypes.c_int, [vp, vp]),
            "sas_get_device_status": (ctypes.c_int, [vp, vp, ctypes.POINTER(ctypes.c_int)]),
            "sas_pool_keys": (ctypes.c_int, [cfgp, kvp, vp, i32, vp, vp, vp, i32, vp, vp, sz, vp]),
            "sas_gate_scores": (ctypes.c_int, [cfgp, vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
            "sas_topk_blocks": (ctypes.c_int, [cfgp, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp]),
            "sas_sparse_decode": (ctypes.c_int, [cfgp, vp, kvp, vp, vp, vp, vp, sz, vp]),
            "sas_decode_step": (ctypes.c_int, [cfgp, vp, kvp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "sas_decode_step_static": (ctypes.c_int, [cfgp, vp, kvp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]),
            "sas_decode_step_host": (ctypes.c_int, [cfgp, vp, vp, kvp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                                    sz, vp]),
            "sas_gate_backward": (ctypes.c_int, [cfgp, vp, kvp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "sas_prefill_block_sparse": (ctypes.c_int, [cfgp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "sas_qk_norm_rope": (ctypes.c_int, [cfgp, rwp, rwp, vp, vp, vp, i32, i32, ctypes.c_float, rwp, rwp, vp]),
            "sas_qk_norm_rope_workspace_bytes": (sz, []),
            "sas_qk_norm_rope_backward": (ctypes.c_int, [cfgp, rwp, rwp, rwp, rwp, vp, vp, vp, i32, i32, ctypes.c_float,
                                                         rwp, rwp, vp, vp, vp, sz, vp]),
            "sas_kv8_append": (ctypes.c_int, [cfgp, kv8p, rwp, rwp, vp, vp, i32, vp, sz, vp]),
            "sas_kv8_read": (ctypes.c_int, [cfgp, kv8p, vp, i32, rwp, rwp, vp, sz, vp]),
            "sas_pool_keys_kv8": (ctypes.c_int, [cfgp, kv8p, vp, i32, vp, vp, vp, i32, vp, vp, sz, vp]),
            "sas_sparse_decode_kv8_workspace_bytes": (sz, [cfgp, i32]),
            "sas_sparse_decode_kv8": (ctypes.c_int, [cfgp, vp, kv8p, vp, vp, vp, vp, sz, vp]),
            "sas_prefill_gate_backward": (ctypes.c_int, [cfgp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp,
                                                         vp, vp, vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        if L.sas_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI {L.sas_abi_version()}, this binding wants {ABI_VERSION}: "
                               "rebuild it")
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().sas_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != SAS_OK:
        raise SasError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# the handle alone, without the Stream object that current_stream() makes (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device()) or None
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


@dataclass
class Config:
    """Mirror of sas_config.  Defaults are the released setting (budget 2,048)."""
    num_q_heads: int
    num_kv_heads: int
    token_budget: int = 2048
    kv_dtype: str = "bf16"
    out_dtype: str = "bf16"
    rope_base: float = 10000.0
    norm_eps: float = 1e-6
    attn_scale: float = 1.0 / math.sqrt(128.0)
    gate_scale: float = 1.0 / math.sqrt(128.0)
    head_dim: int = 128
    block_size: int = 64
    gate_hidden: int = 128
    gate_mode: int = 0        # GATE_SELECT_ONLY or GATE_LOGSIGMOID_BIAS
    gate_keys_bf16: int = 0   # 1: the gate-key cache is bf16 (else fp32)
    # 1: w_q, gamma_q, w_k and gamma_k are never written while decode kernels
    # may run, so the kernels read them before the kernels ahead of them on
    # the stream have finished; 0: every input after those have finished
    static_weights: int = 0

    def c(self) -> _Config:
        return _Config(self.num_q_heads, self.num_kv_heads, self.head_dim, self.block_size,
                       self.gate_hidden, self.token_budget, self.rope_base, self.norm_eps,
                       self.attn_scale, self.gate_scale, _DT[self.kv_dtype], _DT[self.out_dtype],
                       self.gate_mode, self.gate_keys_bf16, self.static_weights)

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads

    @property
    def max_sel(self) -> int:
        return self.token_budget // 64


_CONFIGS: dict = {}


def _config(cfg: Config) -> _Config:
    """cfg.c(), kept per content (a serving loop passes the same few)."""
    key = tuple(cfg.__dict__.values())
    c = _CONFIGS.get(key)
    if c is None:
        if len(_CONFIGS) >= 64:
            _CONFIGS.clear()
        c = _CONFIGS[key] = cfg.c()
    return c


@dataclass
class KvCache:
    """Mirror of sas_kv holding the tensors alive.  block_table None: contiguous
    [B][Hkv][capacity][128]; else paged [num_pages][Hkv][64][128]."""
    k: torch.Tensor
    v: torch.Tensor
    seq_lens: torch.Tensor
    block_table: Optional[torch.Tensor] = None
    token_budgets: Optional[torch.Tensor] = None   # int32 [B]; None: the config's budget
    _c: Optional[_Kv] = field(default=None, repr=False)

    @property
    def batch(self) -> int:
        return int(self.seq_lens.shape[0])

    def c(self) -> _Kv:
        if self.block_table is None:
            return _Kv(_ptr(self.k), _ptr(self.v), None, _ptr(self.seq_lens), self.batch,
                       int(self.k.shape[2]), 0, 0, _ptr(self.token_budgets))
        return _Kv(_ptr(self.k), _ptr(self.v), _ptr(self.block_table), _ptr(self.seq_lens),
                   self.batch, 0, int(self.k.shape[0]), int(self.block_table.shape[1]),
                   _ptr(self.token_budgets))


@dataclass(frozen=True)
class KvCache8:
    """sas_kv8 holding the tensors alive.  The codes' dtype
    (torch.float8_e4m3fn or torch.int8) selects the code.  block_table None:
    codes [B][Hkv][capacity][128], scales [B][Hkv][capacity/64]; else paged
    codes [num_pages][Hkv][64][128], scales [num_pages][Hkv].  Tails are bf16
    [B][Hkv][64][128] and hold each sequence's current block.  Shapes, dtypes
    and layouts are checked, and the C description taken, when the object is
    made: change the tensors' contents freely, but not their storage."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_tail: torch.Tensor
    v_tail: torch.Tensor
    seq_lens: torch.Tensor
    block_table: Optional[torch.Tensor] = None

    def __post_init__(self):
        k, v, bt, lens = self.k, self.v, self.block_table, self.seq_lens
        code = _CODES.get(k.dtype)
        if code is None or v.dtype != k.dtype:
            raise ValueError(f"codes are {k.dtype} / {v.dtype}: both torch.float8_e4m3fn or both torch.int8 are wanted")
        ks = k.shape
        if len(ks) != 4 or ks != v.shape or ks[3] != 128:
            raise ValueError(f"codes are {tuple(ks)} / {tuple(v.shape)}")
        if lens.dim() != 1:
            raise ValueError(f"seq_lens is {tuple(lens.shape)}")
        _i32("seq_lens", lens)
        B, hkv = lens.shape[0], ks[1]
        if bt is None:
            if ks[0] != B or ks[2] % 64:
                raise ValueError(f"contiguous codes are {tuple(ks)} for batch {B}")
            want, cap, pages, width = (B, hkv, ks[2] // 64), ks[2], 0, 0
        else:
            if ks[2] != 64 or bt.dim() != 2 or bt.shape[0] != B:
                raise ValueError(f"paged codes are {tuple(ks)} with a block table {tuple(bt.shape)} for batch {B}")
            _i32("block_table", bt)
            want, cap, pages, width = (ks[0], hkv), 0, ks[0], bt.shape[1]
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("codes must be contiguous")
        _plain("k_scale", self.k_scale, want, torch.float32)
        _plain("v_scale", self.v_scale, want, torch.float32)
        _plain("k_tail", self.k_tail, (B, hkv, 64, 128), torch.bfloat16)
        _plain("v_tail", self.v_tail, (B, hkv, 64, 128), torch.bfloat16)
        dev = k.get_device()
        _on(dev, v, self.k_scale, self.v_scale, self.k_tail, self.v_tail, lens, bt)
        c = _Kv8(k.data_ptr(), v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.k_tail.data_ptr(),
                 self.v_tail.data_ptr(), _ptr(bt), lens.data_ptr(), B, cap, pages, width, code)
        for name, value in (("batch", B), ("kv_heads", hkv), ("device", dev), ("_c", c)):
            object.__setattr__(self, name, value)

    def c(self, cfg: Config) -> _Kv8:
        if cfg.num_kv_heads != self.kv_heads:
            raise ValueError(f"the cache has {self.kv_heads} KV heads, the config {cfg.num_kv_heads}")
        return self._c


def _plain(name: str, t, shape, dtype) -> None:
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}{'' if t.is_contiguous() else ' (strided)'}: "
                         f"contiguous {tuple(shape)} {dtype} is wanted")


def _i32(name: str, t, n: Optional[int] = None) -> None:
    if t.dtype is not torch.int32 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}: contiguous int32"
                         + ("" if n is None else f" with {n} values") + " is wanted")


def _rows(name: str, t, shape, dtype) -> _Rows:
    """sas_rows of a tensor of shape [B][H][T][128] with any strides (last one 1)."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}: [B][H][T][128] = {tuple(shape)} {dtype} is wanted")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name}: the 128 elements of a row must be contiguous")
    return _Rows(t.data_ptr(), st[0], st[2], st[1], shape[2])


def _on(dev: int, *tensors) -> None:
    """Every tensor on CUDA device `dev`."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, cuda:{dev} is wanted")


def _current(dev: int) -> None:
    """The library launches on the current device."""
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on device {dev}, the current device is cuda:{torch.cuda.current_device()}")


def abi_version() -> int:
    return int(lib().sas_abi_version())


def workspace_bytes(cfg: Config, batch: int = 0, max_seq_len: int = 0) -> int:
    c = cfg.c()
    return int(lib().sas_workspace_bytes(ctypes.byref(c), batch, max_seq_len))


def make_workspace(cfg: Config, device, batch: int = 0, max_seq_len: int = 0) -> torch.Tensor:
    """Caller-side workspace allocation (torch), zeroed."""
    return torch.zeros(workspace_bytes(cfg, batch, max_seq_len), dtype=torch.uint8, device=device)


def reset_device_status(ws: torch.Tensor, stream=None) -> None:
    _check(lib().sas_reset_device_status(_ptr(ws), _stream(stream)), "sas_reset_device_status")


def get_device_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int(-1)
    _check(lib().sas_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(out)),
           "sas_get_device_status")
    return int(out.value)


def pool_keys(cfg: Config, kv: KvCache, w_k, gamma_k, gate_keys, ws, blk_begin=None,
              num_blocks: Optional[int] = None, pooled_raw=None, stream=None) -> None:
    """sas_pool_keys.  num_blocks defaults to gate_keys.shape[2] (all rows)."""
    _check_gk(cfg, gate_keys)
    mg = int(gate_keys.shape[2])
    nb = mg if num_blocks is None else int(num_blocks)
    c, k = cfg.c(), kv.c()
    _check(lib().sas_pool_keys(ctypes.byref(c), ctypes.byref(k), _ptr(blk_begin), nb, _ptr(w_k),
                               _ptr(gamma_k), _ptr(gate_keys), mg, _ptr(pooled_raw), _ptr(ws),
                               ws.numel(), _stream(stream)), "sas_pool_keys")


def gate_scores(cfg: Config, q, seq_lens, w_q, gamma_q, gate_keys, group_scores, ws,
                head_scores=None, stream=None) -> None:
    _check_gk(cfg, gate_keys)
    c = cfg.c()
    _check(lib().sas_gate_scores(ctypes.byref(c), _ptr(q), _ptr(seq_lens), int(seq_lens.shape[0]),
                                 _ptr(w_q), _ptr(gamma_q), _ptr(gate_keys), int(gate_keys.shape[2]),
                                 _ptr(head_scores), _ptr(group_scores), _ptr(ws), ws.numel(),
                                 _stream(stream)), "sas_gate_scores")


def topk_blocks(cfg: Config, group_scores, seq_lens, sel_idx, sel_count, ws, stream=None,
                token_budgets=None) -> None:
    c = cfg.c()
    _check(lib().sas_topk_blocks(ctypes.byref(c), _ptr(group_scores), _ptr(seq_lens), _ptr(token_budgets),
                                 int(seq_lens.shape[0]), int(group_scores.shape[2]), _ptr(sel_idx),
                                 _ptr(sel_count), _ptr(ws), ws.numel(), _stream(stream)),
           "sas_topk_blocks")


def sparse_decode(cfg: Config, q, kv: KvCache, sel_idx, sel_count, out, ws, stream=None) -> None:
    c, k = cfg.c(), kv.c()
    _check(lib().sas_sparse_decode(ctypes.byref(c), _ptr(q), ctypes.byref(k), _ptr(sel_idx),
                                   _ptr(sel_count), _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(stream)), "sas_sparse_decode")


def decode_step(cfg: Config, q, kv: KvCache, w_q, gamma_q, gate_keys, out, ws, sel_idx=None,
                sel_count=None, group_scores=None, w_k=None, gamma_k=None, stream=None) -> None:
    """sas_decode_step.  With w_k / gamma_k the step also pools the block the
    decoded token completes into gate_keys (see include/sas.h)."""
    _check_gk(cfg, gate_keys)
    c, k = cfg.c(), kv.c()
    _check(lib().sas_decode_step(ctypes.byref(c), _ptr(q), ctypes.byref(k), _ptr(w_q),
                                 _ptr(gamma_q), _ptr(w_k), _ptr(gamma_k), _ptr(gate_keys),
                                 int(gate_keys.shape[2]), _ptr(out), _ptr(sel_idx), _ptr(sel_count),
                                 _ptr(group_scores), _ptr(ws), ws.numel(), _stream(stream)),
           "sas_decode_step")


def decode_step_host(cfg: Config, q_host, q_dev, kv: KvCache, w_q, gamma_q, gate_keys, out_dev, out_host, ws,
                     sel_idx=None, sel_count=None, group_scores=None, w_k=None, gamma_k=None,
                     stream=None) -> None:
    """sas_decode_step_host: the step with q and out in host memory (pinned
    CPU tensors keep the copies asynchronous); q_dev / out_dev are device
    staging buffers of the same shapes.  out_host holds the output once the
    stream has passed the call.  The library sizes both transfers from the
    config, so each host tensor must be a contiguous CPU tensor of its
    staging buffer's shape and dtype (checked here)."""
    _check_gk(cfg, gate_keys)
    for name, h, d in (("q_host", q_host, q_dev), ("out_host", out_host, out_dev)):
        if h.device.type != "cpu" or not h.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
        if h.shape != d.shape or h.dtype != d.dtype:
            raise ValueError(f"{name} is {tuple(h.shape)} {h.dtype}, its device buffer {tuple(d.shape)} {d.dtype}")
    c, k = cfg.c(), kv.c()
    _check(lib().sas_decode_step_host(ctypes.byref(c), _ptr(q_host), _ptr(q_dev), ctypes.byref(k), _ptr(w_q),
                                      _ptr(gamma_q), _ptr(w_k), _ptr(gamma_k), _ptr(gate_keys),
                                      int(gate_keys.shape[2]), _ptr(out_dev), _ptr(out_host), _ptr(sel_idx),
                                      _ptr(sel_count), _ptr(group_scores), _ptr(ws), ws.numel(),
                                      _stream(stream)), "sas_decode_step_host")


def decode_step_static(cfg: Config, q, kv: KvCache, w_q, gamma_q, gate_keys, out, sel_idx=None,
                       sel_count=None, group_scores=None, w_k=None, gamma_k=None, status_out=None,
                       stream=None) -> None:
    """sas_decode_step_static: the same step with no workspace argument, for
    callers that cannot allocate; status_out (optional device uint32/int32
    tensor) receives the call's status bits."""
    _check_gk(cfg, gate_keys)
    c, k = cfg.c(), kv.c()
    _check(lib().sas_decode_step_static(ctypes.byref(c), _ptr(q), ctypes.byref(k), _ptr(w_q),
                                        _ptr(gamma_q), _ptr(w_k), _ptr(gamma_k), _ptr(gate_keys),
                                        int(gate_keys.shape[2]), _ptr(out), _ptr(sel_idx),
                                        _ptr(sel_count), _ptr(group_scores), _ptr(status_out),
                                        _stream(stream)), "sas_decode_step_static")


def gate_backward(cfg: Config, q, kv: KvCache, w_q, gamma_q, w_k, gamma_k, sel_idx, sel_count, d_out,
                  dw_q, dw_k, dgamma_q, dgamma_k, ws, stream=None) -> None:
    """sas_gate_backward: adds dL/dW_q, dL/dW_k, dL/dgamma_q, dL/dgamma_k (fp32)
    of the gated decode step, block lists held fixed, for d_out = dL/dout."""
    c, k = cfg.c(), kv.c()
    _check(lib().sas_gate_backward(ctypes.byref(c), _ptr(q), ctypes.byref(k), _ptr(w_q), _ptr(gamma_q),
                                   _ptr(w_k), _ptr(gamma_k), _ptr(sel_idx), _ptr(sel_count), _ptr(d_out),
                                   _ptr(dw_q), _ptr(dw_k), _ptr(dgamma_q), _ptr(dgamma_k), _ptr(ws),
                                   ws.numel(), _stream(stream)), "sas_gate_backward")


def prefill_block_sparse(cfg: Config, q, k, v, w_q, gamma_q, w_k, gamma_k, gate_keys, out, ws,
                         sel_idx=None, sel_count=None, stream=None, token_budgets=None) -> None:
    """sas_prefill_block_sparse: q [B][Hq][T][128], k / v [B][Hkv][T][128] (bf16),
    out like q; writes gate_keys [B][Hkv][MG][128]; ws from
    make_workspace(cfg, device, batch=B, max_seq_len=T); token_budgets: None or
    int32 [B] on the device (each a multiple of 64, at most cfg.token_budget)."""
    _check_gk(cfg, gate_keys)
    c = cfg.c()
    B, T = int(q.shape[0]), int(q.shape[2])
    _check(lib().sas_prefill_block_sparse(ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), B, T,
                                          _ptr(token_budgets), _ptr(w_q),
                                          _ptr(gamma_q), _ptr(w_k), _ptr(gamma_k), _ptr(gate_keys),
                                          int(gate_keys.shape[2]), _ptr(out), _ptr(sel_idx),
                                          _ptr(sel_count), _ptr(ws), ws.numel(), _stream(stream)),
           "sas_prefill_block_sparse")


def prefill_gate_backward(cfg: Config, q, k, v, w_q, gamma_q, w_k, gamma_k, gate_keys, sel_idx, sel_count,
                          d_out, dw_q, dw_k, dgamma_q, dgamma_k, ws, stream=None) -> None:
    """sas_prefill_gate_backward: adds dL/dW_q, dL/dW_k, dL/dgamma_q, dL/dgamma_k
    (fp32) of the gated prefill, its block lists held fixed, for d_out =
    dL/dout [B][Hq][T][128] fp32; ws from make_workspace(cfg, device, batch=B,
    max_seq_len=T)."""
    _check_gk(cfg, gate_keys)
    c = cfg.c()
    B, T = int(q.shape[0]), int(q.shape[2])
    _check(lib().sas_prefill_gate_backward(ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), B, T, _ptr(w_q),
                                           _ptr(gamma_q), _ptr(w_k), _ptr(gamma_k), _ptr(gate_keys),
                                           int(gate_keys.shape[2]), _ptr(sel_idx), _ptr(sel_count), _ptr(d_out),
                                           _ptr(dw_q), _ptr(dw_k), _ptr(dgamma_q), _ptr(dgamma_k), _ptr(ws),
                                           ws.numel(), _stream(stream)), "sas_prefill_gate_backward")


def qk_norm_rope(cfg: Config, q, k, gamma_q, gamma_k, q_out, k_out, rope_base: float, positions=None,
                 stream=None) -> None:
    """sas_qk_norm_rope: per-head RMSNorm and position rotation of q
    [B][Hq][T][128] and k [B][Hkv][T][128] (cfg.kv_dtype, any strides with
    contiguous rows) into q_out / k_out (may be q / k); q or k may be None.
    positions: int32 [B][T] (negative: the row is skipped) or None (0 .. T-1)."""
    dt = kv_dtype(cfg)
    B, T = _batch_tokens(q, k)
    qr, qo = _norm_side("q", q, gamma_q, q_out, cfg.num_q_heads, dt, B, T)
    kr, ko = _norm_side("k", k, gamma_k, k_out, cfg.num_kv_heads, dt, B, T)
    if positions is not None:
        _i32("positions", positions, B * T)
    dev = (q if q is not None else k).get_device()
    _current(dev)
    _on(dev, q, k, gamma_q, gamma_k, q_out, k_out, positions)
    c = _config(cfg)
    _check(lib().sas_qk_norm_rope(ctypes.byref(c), _ref(qr), _ref(kr), _ptr(gamma_q), _ptr(gamma_k), _ptr(positions),
                                  B, T, rope_base, _ref(qo), _ref(ko), _stream(stream)), "sas_qk_norm_rope")


def qk_norm_rope_workspace_bytes() -> int:
    return int(lib().sas_qk_norm_rope_workspace_bytes())


def qk_norm_rope_backward(cfg: Config, dq_out, dk_out, q, k, gamma_q, gamma_k, dq, dk, dgamma_q, dgamma_k,
                          rope_base: float, ws, positions=None, stream=None) -> None:
    """sas_qk_norm_rope_backward: writes dq / dk (may be dq_out / dk_out or
    q / k) and adds to dgamma_q / dgamma_k (fp32 [128]); ws holds at least
    qk_norm_rope_workspace_bytes() bytes."""
    dt = kv_dtype(cfg)
    B, T = _batch_tokens(q, k)
    args = []
    for n, x, g, o, d, dg, h in (("q", q, gamma_q, dq, dq_out, dgamma_q, cfg.num_q_heads),
                                 ("k", k, gamma_k, dk, dk_out, dgamma_k, cfg.num_kv_heads)):
        r, o_r = _norm_side(n, x, g, o, h, dt, B, T)
        if (x is None) != (d is None) or (x is None) != (dg is None):
            raise ValueError(f"d{n}_out and dgamma_{n} go with {n}: all of them or none")
        if x is not None:
            _plain(f"dgamma_{n}", dg, (128,), torch.float32)
        args.append((r, o_r, None if d is None else _rows(f"d{n}_out", d, (B, h, T, 128), dt)))
    if positions is not None:
        _i32("positions", positions, B * T)
    dev = ws.get_device()
    _current(dev)
    _on(dev, q, k, gamma_q, gamma_k, dq, dk, dq_out, dk_out, dgamma_q, dgamma_k, positions)
    c = _config(cfg)
    (qr, qo, qd), (kr, ko, kd) = args
    _check(lib().sas_qk_norm_rope_backward(ctypes.byref(c), _ref(qd), _ref(kd), _ref(qr), _ref(kr), _ptr(gamma_q),
                                           _ptr(gamma_k), _ptr(positions), B, T, rope_base, _ref(qo), _ref(ko),
                                           _ptr(dgamma_q), _ptr(dgamma_k), _ptr(ws), ws.nbytes, _stream(stream)),
           "sas_qk_norm_rope_backward")


def _batch_tokens(q, k):
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    sh = x.shape
    if len(sh) != 4:
        raise ValueError(f"[B][H][T][128] is wanted, got {tuple(sh)}")
    return sh[0], sh[2]


def _norm_side(name, x, gamma, out, heads, dtype, batch, tokens):
    if x is None:
        if out is not None:
            raise ValueError(f"an output for {name} without {name}")
        return None, None
    if gamma is None or out is None:
        raise ValueError(f"{name} needs its gain and its output")
    shape = (batch, heads, tokens, 128)
    _plain("its gain", gamma, (128,), torch.float32)
    return _rows(name, x, shape, dtype), _rows("its output", out, shape, dtype)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def kv8_append(cfg: Config, kv: KvCache8, k_new, v_new, ws, new_starts=None, new_lens=None,
               max_new: Optional[int] = None, stream=None) -> None:
    """sas_kv8_append: k_new / v_new bf16 [B][Hkv][T][128] (any strides), or
    packed [1][Hkv][N][128] with new_starts int32 [B]; new_lens int32 [B] or
    None (max_new tokens for every sequence); max_new defaults to T.
    kv.seq_lens counts the new tokens in."""
    B = kv.batch
    packed = new_starts is not None
    if k_new.dim() != 4:
        raise ValueError(f"k_new is {tuple(k_new.shape)}: [B][H][T][128] is wanted")
    shape = (1 if packed else B, cfg.num_kv_heads, k_new.shape[2], 128)
    kr = _rows("k_new", k_new, shape, torch.bfloat16)
    vr = _rows("v_new", v_new, shape, torch.bfloat16)
    if packed:
        kr.seq_stride = vr.seq_stride = 0
        _i32("new_starts", new_starts, B)
    if new_lens is not None:
        _i32("new_lens", new_lens, B)
    _current(kv.device)
    _on(kv.device, k_new, v_new, new_starts, new_lens, ws)
    c, c8 = _config(cfg), kv.c(cfg)
    _check(lib().sas_kv8_append(ctypes.byref(c), ctypes.byref(c8), ctypes.byref(kr), ctypes.byref(vr),
                                _ptr(new_starts), _ptr(new_lens), kr.tokens if max_new is None else max_new, _ptr(ws),
                                ws.nbytes, _stream(stream)), "sas_kv8_append")


def kv8_read(cfg: Config, kv: KvCache8, k_out, v_out, ws, begin=None, stream=None) -> None:
    """sas_kv8_read: tokens begin[s] .. of every sequence into k_out / v_out
    [B][Hkv][T][128] (cfg.out_dtype, any strides; either may be None)."""
    x = k_out if k_out is not None else v_out
    if x is None or x.dim() != 4:
        raise ValueError("k_out or v_out [B][H][T][128] is wanted")
    shape, dt = (kv.batch, cfg.num_kv_heads, x.shape[2], 128), out_dtype(cfg)
    kr = None if k_out is None else _rows("k_out", k_out, shape, dt)
    vr = None if v_out is None else _rows("v_out", v_out, shape, dt)
    if begin is not None:
        _i32("begin", begin, kv.batch)
    _current(kv.device)
    _on(kv.device, k_out, v_out, begin, ws)
    c, c8 = _config(cfg), kv.c(cfg)
    _check(lib().sas_kv8_read(ctypes.byref(c), ctypes.byref(c8), _ptr(begin), shape[2], _ref(kr), _ref(vr),
                              _ptr(ws), ws.nbytes, _stream(stream)), "sas_kv8_read")


def pool_keys_kv8(cfg: Config, kv: KvCache8, w_k, gamma_k, gate_keys, ws, blk_begin=None,
                  num_blocks: Optional[int] = None, pooled_raw=None, stream=None) -> None:
    """sas_pool_keys_kv8: pool_keys over an 8-bit cache."""
    _check_gk(cfg, gate_keys)
    B, hkv, mg = kv.batch, cfg.num_kv_heads, int(gate_keys.shape[2])
    _plain("gate_keys", gate_keys, (B, hkv, mg, 128), gate_key_dtype(cfg))
    _plain("w_k", w_k, (hkv, 384, 128), torch.bfloat16)
    _plain("gamma_k", gamma_k, (128,), torch.float32)
    if pooled_raw is not None:
        _plain("pooled_raw", pooled_raw, (B, hkv, mg, 384), torch.float32)
    if blk_begin is not None:
        _i32("blk_begin", blk_begin, B)
    _current(kv.device)
    _on(kv.device, w_k, gamma_k, gate_keys, pooled_raw, blk_begin, ws)
    c, c8 = _config(cfg), kv.c(cfg)
    _check(lib().sas_pool_keys_kv8(ctypes.byref(c), ctypes.byref(c8), _ptr(blk_begin),
                                   mg if num_blocks is None else int(num_blocks), _ptr(w_k), _ptr(gamma_k),
                                   _ptr(gate_keys), mg, _ptr(pooled_raw), _ptr(ws), ws.nbytes, _stream(stream)),
           "sas_pool_keys_kv8")


def sparse_decode_kv8_workspace_bytes(cfg: Config, batch: int) -> int:
    return int(lib().sas_sparse_decode_kv8_workspace_bytes(ctypes.byref(_config(cfg)), batch))


def sparse_decode_kv8(cfg: Config, q, kv: KvCache8, sel_idx, sel_count, out, ws, stream=None) -> None:
    """sas_sparse_decode_kv8: q bf16 [B][Hq][128], out cfg.out_dtype likewise;
    sel_idx / sel_count as topk_blocks writes them, or both None: every block
    (then with sparse_decode_kv8_workspace_bytes(cfg, B) bytes of ws, few or
    ragged long sequences use the whole GPU, and calls that may overlap need a
    workspace each)."""
    B, hkv = kv.batch, cfg.num_kv_heads
    _plain("q", q, (B, cfg.num_q_heads, 128), torch.bfloat16)
    _plain("out", out, (B, cfg.num_q_heads, 128), out_dtype(cfg))
    if (sel_idx is None) != (sel_count is None):
        raise ValueError("sel_idx and sel_count: both or neither")
    if sel_idx is not None:
        _i32("sel_idx", sel_idx, B * hkv * cfg.max_sel)
        _i32("sel_count", sel_count, B * hkv)
    _current(kv.device)
    _on(kv.device, q, out, sel_idx, sel_count, ws)
    c, c8 = _config(cfg), kv.c(cfg)
    _check(lib().sas_sparse_decode_kv8(ctypes.byref(c), _ptr(q), ctypes.byref(c8), _ptr(sel_idx), _ptr(sel_count),
                                       _ptr(out), _ptr(ws), ws.nbytes, _stream(stream)), "sas_sparse_decode_kv8")


def out_dtype(cfg: Config) -> torch.dtype:
    return _TORCH_DT[_DT[cfg.out_dtype]]


def gate_key_dtype(cfg: Config) -> torch.dtype:
    """Element type of the gate-key cache under cfg (bf16 or fp32)."""
    return torch.bfloat16 if cfg.gate_keys_bf16 else torch.float32


def _check_gk(cfg: Config, gate_keys) -> None:
    if gate_keys is not None and gate_keys.dtype != gate_key_dtype(cfg):
        raise ValueError(f"gate_keys is {gate_keys.dtype}, the config wants {gate_key_dtype(cfg)}")


def kv_dtype(cfg: Config) -> torch.dtype:
    return _TORCH_DT[_DT[cfg.kv_dtype]]
