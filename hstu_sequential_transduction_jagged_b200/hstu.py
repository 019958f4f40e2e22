"""ctypes binding of libhstu (include/hstu.h): argument marshalling only.

Every step of the HSTU layer runs in the CUDA library; this module turns torch
tensors into pointers, sizes and structs, allocates outputs/workspaces with
torch (device memory plumbing only) and raises HSTUError on a non-zero status.
There is no CPU fallback: if libhstu.so is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from collections import namedtuple
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhstu.so")

ACT = {"identity": 0, "relu": 1, "silu": 2, "softmax": 3}
DTYPE = {"bf16": 0, "fp32": 1, "fp16": 2}
TORCH_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp16": torch.float16}
# dtype of the per-layer key/value cache of a layer configured with `dtype`
CACHE_DTYPE = {"bf16": torch.float16, "fp32": torch.float32}
STATUS = {0: "HSTU_OK", 1: "HSTU_ERR_INVALID_ARGUMENT", 2: "HSTU_ERR_UNSUPPORTED",
          3: "HSTU_ERR_CUDA", 4: "HSTU_ERR_WORKSPACE_TOO_SMALL", 5: "HSTU_ERR_DEVICE_TIMEOUT",
          6: "HSTU_ERR_DEVICE_CHECK"}


class HSTUError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


class JaggedT(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("max_len", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("timestamps", ctypes.c_void_p), ("segments", ctypes.c_void_p),
                ("max_static", ctypes.c_int32)]


FLAG_FUSED_F2 = 1


class LayerCfgT(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("dqk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("num_pos_buckets", ctypes.c_int32), ("num_time_buckets", ctypes.c_int32),
                ("phi1", ctypes.c_int32), ("phi2", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class KernelTimeT(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double)]


class CacheT(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("kv", ctypes.c_void_p),
                ("timestamps", ctypes.c_void_p), ("ref_count", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


class LayerWeightsT(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w1", "b1", "w2", "b2", "rab_pos", "rab_time", "ln_gamma", "ln_beta")]


_PAGED_ATTN_ARGS = ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                     ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                     ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 4)

EXPORTS = {
    "hstu_version": (ctypes.c_char_p, []),
    "hstu_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "hstu_layer_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int64]),
    "hstu_forward_workspace_bytes": (ctypes.c_size_t,
                                     [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64]),
    "hstu_mfalcon_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int64]),
    "hstu_attn_fwd": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_size_t, ctypes.c_void_p]),
    "hstu_attn_fwd_f32": (ctypes.c_int, [ctypes.c_void_p] * 9),
    "hstu_attn_bwd": (ctypes.c_int, [ctypes.c_void_p] * 14),
    "hstu_layer_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int64]),
    "hstu_layer_bwd": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_void_p, ctypes.c_size_t,
                                                              ctypes.c_void_p]),
    "mfalcon_attn_fwd": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int64, ctypes.c_int32]
                         + [ctypes.c_void_p] * 8),
    "hstu_layer_fwd": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_size_t, ctypes.c_void_p]),
    "hstu_layer_fwd_static": (ctypes.c_int, [ctypes.c_void_p] * 9),
    "hstu_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 6
                     + [ctypes.c_size_t, ctypes.c_void_p]),
    "mfalcon_score": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]),
    "hstu_stochastic_length": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                              ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64]
                               + [ctypes.c_void_p] * 7),
    "hstu_cache_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "hstu_cache_reserve": (ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_size_t, ctypes.c_void_p]),
    "hstu_cache_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "hstu_cache_gather": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 3),
    "hstu_cache_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 3),
    "hstu_cache_release": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]),
    "hstu_cache_compact": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_size_t, ctypes.c_void_p]),
    "hstu_paged_attn_fwd": (ctypes.c_int, _PAGED_ATTN_ARGS),
    "hstu_paged_attn_fwd_f32": (ctypes.c_int, _PAGED_ATTN_ARGS),
    "hstu_extend_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_void_p,
                                                      ctypes.c_int32, ctypes.c_int64]),
    "hstu_extend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 4
                    + [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 3
                    + [ctypes.c_size_t, ctypes.c_void_p]),
    "hstu_get_device_status": (ctypes.c_int, [ctypes.c_void_p]),
    "hstu_profiler_start": (ctypes.c_int, []),
    "hstu_profiler_stop": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "hstu_time_bucket_thresholds": (ctypes.c_int, [ctypes.c_int32, ctypes.c_void_p]),
    "hstu_debug_rab_index": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "hstu_debug_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_void_p]),
}

_lib = None


def lib():
    """Load libhstu.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m hstu_sequential_transduction_jagged_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise HSTUError(status, where)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


@dataclass
class LayerConfig:
    d_model: int
    num_heads: int
    num_pos_buckets: int
    num_time_buckets: int
    dqk: int = 64
    dv: int = 64
    phi1: str = "relu"
    phi2: str = "silu"
    ln_eps: float = 1e-5
    dtype: str = "bf16"
    fused_f2: bool = False  # True sets HSTU_FLAG_FUSED_F2

    def c(self) -> LayerCfgT:
        return LayerCfgT(self.d_model, self.num_heads, self.dqk, self.dv, self.num_pos_buckets,
                         self.num_time_buckets, ACT[self.phi1], ACT[self.phi2], self.ln_eps,
                         DTYPE[self.dtype], FLAG_FUSED_F2 if self.fused_f2 else 0)

    @property
    def torch_dtype(self):
        return TORCH_DTYPE[self.dtype]

    @property
    def cache_dtype(self):
        """dtype of the K/V cache hstu_layer_fwd / hstu_forward write."""
        return CACHE_DTYPE[self.dtype]

    @property
    def n1(self) -> int:
        return 2 * self.num_heads * (self.dqk + self.dv)


@dataclass
class Jagged:
    offsets: torch.Tensor      # int64 [B+1] on the device
    timestamps: torch.Tensor   # int64 [T] on the device
    max_len: int
    total_tokens: int
    segments: Optional[torch.Tensor] = None  # int32 [B, 2] (n_us, n_r): generalised masks
    max_static: int = 0                      # >= every n_us

    @property
    def batch(self) -> int:
        return self.offsets.numel() - 1

    def c(self) -> JaggedT:
        return JaggedT(self.batch, self.total_tokens, self.max_len, self.offsets.data_ptr(),
                       self.timestamps.data_ptr() if self.timestamps.numel() else None,
                       None if self.segments is None else self.segments.data_ptr(),
                       self.max_static)


@dataclass
class LayerWeights:
    w1: torch.Tensor
    b1: torch.Tensor
    w2: torch.Tensor
    b2: torch.Tensor
    rab_pos: torch.Tensor
    rab_time: torch.Tensor
    ln_gamma: Optional[torch.Tensor] = None
    ln_beta: Optional[torch.Tensor] = None

    def c(self) -> LayerWeightsT:
        def ptr(t):
            return None if t is None else t.data_ptr()
        return LayerWeightsT(ptr(self.w1), ptr(self.b1), ptr(self.w2), ptr(self.b2),
                             ptr(self.rab_pos), ptr(self.rab_time), ptr(self.ln_gamma),
                             ptr(self.ln_beta))


def version() -> str:
    return lib().hstu_version().decode()


def layer_workspace_bytes(cfg: LayerConfig, total_tokens: int) -> int:
    c = cfg.c()
    return lib().hstu_layer_workspace_bytes(ctypes.byref(c), total_tokens)


def forward_workspace_bytes(cfg: LayerConfig, num_layers: int, total_tokens: int) -> int:
    c = cfg.c()
    return lib().hstu_forward_workspace_bytes(ctypes.byref(c), num_layers, total_tokens)


def mfalcon_workspace_bytes(cfg: LayerConfig, num_cand: int) -> int:
    c = cfg.c()
    return lib().hstu_mfalcon_workspace_bytes(ctypes.byref(c), num_cand)


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A new tensor for a call on `stream` (None: the current one).  It comes from that
    stream's memory: a block of another stream's may still be in use by work pending
    there, and may be handed out again, once dropped, before the call has run.  A
    result that the current stream goes on to use is kept for that stream too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if current != stream:
        t.record_stream(current)
    return t


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor], stream=None):
    if workspace is not None:
        return workspace
    return _empty(max(nbytes, 1), torch.uint8, device, stream)


def attn_fwd(cfg: LayerConfig, jag: Jagged, q, k, v, rab_pos, rab_time, av_out=None,
             stream=None) -> torch.Tensor:
    """Eq. 2 over a jagged batch: AV[T, H*dv] in cfg dtype."""
    if av_out is None:
        av_out = torch.empty((jag.total_tokens, cfg.num_heads * cfg.dv), dtype=cfg.torch_dtype,
                             device=q.device)
    c, j = cfg.c(), jag.c()
    _check(lib().hstu_attn_fwd(ctypes.byref(c), ctypes.byref(j), _p(q), _p(k), _p(v),
                               _p(rab_pos), _p(rab_time), _p(av_out), None, 0,
                               _stream(stream)), "hstu_attn_fwd")
    return av_out


def attn_fwd_f32(cfg: LayerConfig, jag: Jagged, q, k, v, rab_pos, rab_time, av_out=None,
                 stream=None) -> torch.Tensor:
    """Eq. 2 over a jagged batch with the result in fp32: AV[T, H*dv] float32."""
    if av_out is None:
        av_out = torch.empty((jag.total_tokens, cfg.num_heads * cfg.dv), dtype=torch.float32,
                             device=q.device)
    c, j = cfg.c(), jag.c()
    _check(lib().hstu_attn_fwd_f32(ctypes.byref(c), ctypes.byref(j), _p(q), _p(k), _p(v),
                                   _p(rab_pos), _p(rab_time), _p(av_out), _stream(stream)),
           "hstu_attn_fwd_f32")
    return av_out


def attn_bwd(cfg: LayerConfig, jag: Jagged, q, k, v, d_o, rab_pos, rab_time, stream=None):
    """Backward of the causal attention: returns dq, dk, dv ([T, H*64] fp32) and
    drab_pos [H, P], drab_time [H, Tb] (fp32) for dO = d_o.  dq and the table
    gradients are sums of reductions in no fixed order: their last bits vary
    from run to run."""
    dev = rab_pos.device
    T, hv = jag.total_tokens, cfg.num_heads * cfg.dv
    dq, dk, dv = (torch.empty((max(T, 1), hv), dtype=torch.float32, device=dev) for _ in range(3))
    drp = torch.empty((cfg.num_heads, cfg.num_pos_buckets), dtype=torch.float32, device=dev)
    drt = torch.empty((cfg.num_heads, cfg.num_time_buckets), dtype=torch.float32, device=dev)
    c, j = cfg.c(), jag.c()
    _check(lib().hstu_attn_bwd(ctypes.byref(c), ctypes.byref(j), _p(q), _p(k), _p(v), _p(d_o),
                               _p(rab_pos), _p(rab_time), _p(dq), _p(dk), _p(dv), _p(drp),
                               _p(drt), _stream(stream)), "hstu_attn_bwd")
    return dq[:T], dk[:T], dv[:T], drp, drt


class LayerGradsT(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("dw1", "db1", "dw2", "db2", "drab_pos", "drab_time", "dgamma", "dbeta")]


def layer_bwd_workspace_bytes(cfg: LayerConfig, total_tokens: int) -> int:
    c = cfg.c()
    return int(lib().hstu_layer_bwd_workspace_bytes(ctypes.byref(c), total_tokens))


def layer_bwd(cfg: LayerConfig, w: "LayerWeights", jag: Jagged, x_in, dy, x_res=None,
              workspace=None, stream=None) -> dict:
    """Backward of one bf16 layer for dY = dy ([T, d] fp32): returns a dict with
    dx [T, d] and the parameter gradients (fp32): dw1, db1, dw2, db2, drab_pos,
    drab_time and, when the layer has them, dgamma / dbeta."""
    dev = dy.device
    T, d, hv, n1 = jag.total_tokens, cfg.d_model, cfg.num_heads * cfg.dv, cfg.n1
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dx": torch.empty((max(T, 1), d), **f32), "dw1": torch.empty((n1, d), **f32),
           "db1": torch.empty(n1, **f32), "dw2": torch.empty((d, hv), **f32),
           "db2": torch.empty(d, **f32),
           "drab_pos": torch.empty((cfg.num_heads, cfg.num_pos_buckets), **f32),
           "drab_time": torch.empty((cfg.num_heads, cfg.num_time_buckets), **f32),
           "dgamma": torch.empty(hv, **f32) if w.ln_gamma is not None else None,
           "dbeta": torch.empty(hv, **f32) if w.ln_beta is not None else None}
    g = LayerGradsT(*[None if out[n] is None else out[n].data_ptr() for n in
                      ("dw1", "db1", "dw2", "db2", "drab_pos", "drab_time", "dgamma", "dbeta")])
    ws = _workspace(layer_bwd_workspace_bytes(cfg, T), dev, workspace, stream)
    c, j, wc = cfg.c(), jag.c(), w.c()
    _check(lib().hstu_layer_bwd(ctypes.byref(c), ctypes.byref(wc), ctypes.byref(j), _p(x_in),
                                _p(x_res), _p(dy), _p(out["dx"]), ctypes.byref(g), _p(ws),
                                ws.numel(), _stream(stream)), "hstu_layer_bwd")
    out["dx"] = out["dx"][:T]
    return out


def mfalcon_attn_fwd(cfg: LayerConfig, history: Jagged, k_hist, v_hist, cand_offsets,
                     max_cand: int, q, k, v, request_ts, rab_pos, rab_time, av_out=None,
                     stream=None) -> torch.Tensor:
    """Candidate-mode attention alone (history keys/values plus self): AV [M, H*dv] fp32."""
    M = q.shape[0]
    if av_out is None:
        av_out = torch.empty((M, cfg.num_heads * cfg.dv), dtype=torch.float32, device=q.device)
    c, j = cfg.c(), history.c()
    _check(lib().mfalcon_attn_fwd(ctypes.byref(c), ctypes.byref(j), _p(k_hist), _p(v_hist),
                                  _p(cand_offsets), M, max_cand, _p(q), _p(k), _p(v),
                                  _p(request_ts), _p(rab_pos), _p(rab_time), _p(av_out),
                                  _stream(stream)), "mfalcon_attn_fwd")
    return av_out


def layer_fwd(cfg: LayerConfig, w: LayerWeights, jag: Jagged, x_in, x_res=None, y_out=None,
              y_out_lp=None, kv_cache_out=None, workspace=None, stream=None) -> torch.Tensor:
    """One HSTU layer; returns the fp32 residual-stream output Y [T, d].  For bf16
    layers x_in may be None when x_res (fp32) is given: f1 then reads x_res
    rounded to fp16."""
    dev = (x_in if x_in is not None else x_res).device
    if y_out is None:
        y_out = torch.empty((jag.total_tokens, cfg.d_model), dtype=torch.float32, device=dev)
    nbytes = layer_workspace_bytes(cfg, jag.total_tokens)
    ws = _workspace(nbytes, dev, workspace, stream)
    c, j, wc = cfg.c(), jag.c(), w.c()
    _check(lib().hstu_layer_fwd(ctypes.byref(c), ctypes.byref(wc), ctypes.byref(j), _p(x_in),
                                _p(x_res), _p(y_out), _p(y_out_lp), _p(kv_cache_out), _p(ws),
                                ws.numel(), _stream(stream)), "hstu_layer_fwd")
    return y_out


STATIC_SCRATCH_BYTES = 64 << 20


def layer_fwd_static(cfg: LayerConfig, w: LayerWeights, jag: Jagged, x_in, x_res=None,
                     y_out=None, y_out_lp=None, kv_cache_out=None, stream=None) -> torch.Tensor:
    """hstu_layer_fwd without a caller workspace: the library's fixed scratch array
    (STATIC_SCRATCH_BYTES per GPU) is used, so the C call itself allocates nothing."""
    if y_out is None:
        y_out = torch.empty((jag.total_tokens, cfg.d_model), dtype=torch.float32,
                            device=(x_in if x_in is not None else x_res).device)
    c, j, wc = cfg.c(), jag.c(), w.c()
    _check(lib().hstu_layer_fwd_static(ctypes.byref(c), ctypes.byref(wc), ctypes.byref(j),
                                       _p(x_in), _p(x_res), _p(y_out), _p(y_out_lp),
                                       _p(kv_cache_out), _stream(stream)),
           "hstu_layer_fwd_static")
    return y_out


def forward(cfg: LayerConfig, weights: Sequence[LayerWeights], jag: Jagged, x_in, y_out=None,
            kv_cache_out=None, workspace=None, stream=None) -> torch.Tensor:
    """A stack of HSTU layers; returns Y [T, d] fp32."""
    dev = x_in.device
    L = len(weights)
    if y_out is None:
        y_out = torch.empty((jag.total_tokens, cfg.d_model), dtype=torch.float32, device=dev)
    ws = _workspace(forward_workspace_bytes(cfg, L, jag.total_tokens), dev, workspace, stream)
    arr = (LayerWeightsT * L)(*[w.c() for w in weights])
    c, j = cfg.c(), jag.c()
    _check(lib().hstu_forward(ctypes.byref(c), L, arr, ctypes.byref(j), _p(x_in), _p(y_out),
                              _p(kv_cache_out), _p(ws), ws.numel(), _stream(stream)),
           "hstu_forward")
    return y_out


def mfalcon_score(cfg: LayerConfig, weights: Sequence[LayerWeights], history: Jagged, kv_cache,
                  cand_offsets, cand_emb, request_ts, microbatch: int, max_cand: int,
                  scores=None, cand_y_out=None, workspace=None, stream=None) -> torch.Tensor:
    """M-FALCON candidate scores [num_cand] fp32.  With `cand_y_out` ([num_cand, d]
    float32) each candidate's final residual-stream row is written there too."""
    dev = cand_emb.device
    M = cand_emb.shape[0]
    L = len(weights)
    if scores is None:
        scores = torch.empty(M, dtype=torch.float32, device=dev)
    ws = _workspace(mfalcon_workspace_bytes(cfg, M), dev, workspace, stream)
    arr = (LayerWeightsT * L)(*[w.c() for w in weights])
    c, j = cfg.c(), history.c()
    _check(lib().mfalcon_score(ctypes.byref(c), L, arr, ctypes.byref(j), _p(kv_cache),
                               _p(cand_offsets), M, max_cand, _p(cand_emb), _p(request_ts),
                               microbatch, _p(scores), _p(cand_y_out), _p(ws), ws.numel(),
                               _stream(stream)),
           "mfalcon_score")
    return scores


def stochastic_length(jag: Jagged, alpha: float, seed: int, step: int, x=None, stream=None):
    """Stochastic Length subsampling on the GPU.  Returns a dict with the output
    offsets [B+1], lengths [B], max_len [1], kept_index [T_full] (first T_out
    valid), timestamps [T_full] and, when x is given, the gathered rows
    [T_full, ...] (first T_out valid).  T_out = offsets[B] stays on the device."""
    dev = jag.offsets.device
    B, T = jag.batch, jag.total_tokens
    out = {"offsets": torch.empty(B + 1, dtype=torch.int64, device=dev),
           "lengths": torch.empty(max(B, 1), dtype=torch.int32, device=dev),
           "max_len": torch.zeros(1, dtype=torch.int32, device=dev),
           "kept_index": torch.empty(max(T, 1), dtype=torch.int64, device=dev),
           "timestamps": torch.empty(max(T, 1), dtype=torch.int64, device=dev)}
    row_bytes = 0
    if x is not None:
        out["x"] = torch.empty((max(T, 1),) + tuple(x.shape[1:]), dtype=x.dtype, device=dev)
        row_bytes = x[0].numel() * x.element_size() if T else 16
    j = jag.c()
    _check(lib().hstu_stochastic_length(ctypes.byref(j), _p(x), row_bytes, alpha, seed, step,
                                        _p(out["offsets"]), _p(out["lengths"]),
                                        _p(out["max_len"]), _p(out["kept_index"]),
                                        _p(out["timestamps"]), _p(out.get("x")),
                                        _stream(stream)), "hstu_stochastic_length")
    return out


_CACHE_DTYPE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


class PagedCache(namedtuple("PagedCache", "kv timestamps ref_count block_table lengths desc")):
    """A paged history cache: the caller's five device tensors (see hstu_cache_t).
      kv           [L, num_pages, 2, H, page_size, 64], the cache type
      timestamps   int64 [num_pages, page_size]
      ref_count    int32 [num_pages]
      block_table  int32 [num_seqs, max_blocks], -1 = no page
      lengths      int32 [num_seqs]
    The handle checks their layout and keeps their addresses: make another one for
    other tensors."""
    __slots__ = ()

    def __new__(cls, kv, timestamps, ref_count, block_table, lengths):
        # the calls hand bare pointers on, so the layout is checked here
        ks, bs, i32 = kv.shape, block_table.shape, torch.int32
        dtype = _CACHE_DTYPE.get(kv.dtype)
        if not (dtype is not None and len(ks) == 6 and ks[2] == 2 and ks[5] == 64
                and timestamps.shape == (ks[1], ks[4]) and timestamps.dtype is torch.int64
                and ref_count.shape == (ks[1],) and len(bs) == 2 and lengths.shape == (bs[0],)
                and ref_count.dtype is i32 and block_table.dtype is i32 and lengths.dtype is i32
                and kv.is_contiguous() and timestamps.is_contiguous()
                and block_table.is_contiguous() and ref_count.is_contiguous()
                and lengths.is_contiguous() and timestamps.get_device() == kv.get_device()
                == ref_count.get_device() == block_table.get_device() == lengths.get_device()):
            raise ValueError("PagedCache: kv [L, pages, 2, H, page, 64] (fp16, bf16 or fp32), "
                             "timestamps int64 [pages, page], ref_count int32 [pages], "
                             "block_table int32 [seqs, blocks] and lengths int32 [seqs], contiguous, "
                             "on one device")
        return super().__new__(cls, kv, timestamps, ref_count, block_table, lengths, CacheT(
            ks[0], ks[3], dtype, ks[4], ks[1], bs[0], bs[1], kv.data_ptr(), timestamps.data_ptr(),
            ref_count.data_ptr(), block_table.data_ptr(), lengths.data_ptr()))

    @staticmethod
    def empty(num_layers: int, num_heads: int, num_pages: int, num_seqs: int, max_blocks: int,
              page_size: int = 64, dtype: str = "fp16", device="cuda") -> "PagedCache":
        """A new cache with every page free.  The pages are not initialised: no
        call reads a slot that was not written."""
        i32 = dict(dtype=torch.int32, device=device)
        return PagedCache(
            torch.empty((num_layers, num_pages, 2, num_heads, page_size, 64),
                        dtype=TORCH_DTYPE[dtype], device=device),
            torch.empty((num_pages, page_size), dtype=torch.int64, device=device),
            torch.zeros(num_pages, **i32), torch.full((num_seqs, max_blocks), -1, **i32),
            torch.zeros(num_seqs, **i32))

    def _replace(self, **kw):
        """A handle with other tensors in some places (a tuple's own would keep the old
        addresses)."""
        parts = [kw.pop(name, old) for name, old in zip(self._fields[:5], self)]
        if kw:
            raise ValueError(f"PagedCache: no tensor named {sorted(kw)}")
        return PagedCache(*parts)

    def c(self) -> CacheT:
        return self.desc


def _ids(ids, n: int, what: str):
    """Pointer of `n` int32 sequence numbers (None: 0 .. n - 1)."""
    if ids is None:
        return None
    if ids.dtype is not torch.int32 or ids.numel() != n or not ids.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous int32 sequence numbers are needed")
    return ids.data_ptr()


def _cache_stream(cache: PagedCache, stream, what: str, *tensors) -> int:
    """The raw stream of a call on `cache`, which is launched on the current GPU: the cache
    and the other tensors (None: not given) have to be there."""
    dev = cache.kv.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{what}: the cache is not on the current GPU")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{what}: a tensor is not on the cache's GPU")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"{what}: the stream is not the cache's GPU's")
    return stream.cuda_stream


def _chunk(chunk: Jagged, what: str):
    """The chunk's C description and its timestamps (None: it has no rows, and needs none)."""
    o, i64, total, seg = chunk.offsets, torch.int64, chunk.total_tokens, chunk.segments
    t = chunk.timestamps if total else None
    if not (o.dtype is i64 and o.is_contiguous()
            and (t is None or (t.dtype is i64 and t.numel() >= total and t.is_contiguous()))):
        raise ValueError(f"{what}: the chunk needs contiguous int64 offsets and int64 timestamps "
                         "of total_tokens rows")
    return JaggedT(o.numel() - 1, total, chunk.max_len, o.data_ptr(), None if t is None else t.data_ptr(),
                   None if seg is None else seg.data_ptr(), chunk.max_static), t


def _dense(t: torch.Tensor, shape, dtype, what: str, name: str):
    """A contiguous tensor of a shape and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous, {list(shape)} {dtype}")


def cache_workspace_bytes(cache: PagedCache, batch: int) -> int:
    return lib().hstu_cache_workspace_bytes(ctypes.byref(cache.c()), batch)


def cache_reserve(cache: PagedCache, chunk: Jagged, seq_ids=None, workspace=None, stream=None):
    """Make room for the chunk's new events (chunk.offsets: their row ranges per
    sequence) and lengthen the sequences; shared partial last pages are copied.
    A pool that is too small leaves everything as it was and is reported in
    device_status()."""
    c, (j, times) = cache.c(), _chunk(chunk, "cache_reserve")
    ids = _ids(seq_ids, j.batch, "cache_reserve")
    raw = _cache_stream(cache, stream, "cache_reserve", chunk.offsets, times, seq_ids, workspace)
    if workspace is None:
        nbytes = lib().hstu_cache_workspace_bytes(ctypes.byref(c), j.batch)
        workspace = _workspace(nbytes, cache.kv.device, None, stream)
    _check(lib().hstu_cache_reserve(ctypes.byref(c), ctypes.byref(j), ids, _p(workspace),
                                    workspace.numel(), raw), "hstu_cache_reserve")


def _rows_ld(t: torch.Tensor, what: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError(f"{what}: rows of contiguous elements are needed")
    return st[0] if t.shape[0] > 1 else t.shape[1]


def cache_append(cache: PagedCache, layer: int, chunk: Jagged, k, v, seq_ids=None, stream=None):
    """Write K and V ([T, H*64], any row stride) of the chunk's rows into a layer's pages."""
    dtype, rows = cache.kv.dtype, (chunk.total_tokens, cache.desc.num_heads * 64)
    if k.dtype is not dtype or v.dtype is not dtype or k.shape != rows or v.shape != rows:
        raise ValueError("cache_append: k and v must be [total_tokens, num_heads * 64] in the cache's type")
    c, (j, times) = cache.c(), _chunk(chunk, "cache_append")
    ids = _ids(seq_ids, j.batch, "cache_append")
    raw = _cache_stream(cache, stream, "cache_append", k, v, chunk.offsets, times, seq_ids)
    _check(lib().hstu_cache_append(ctypes.byref(c), layer, ctypes.byref(j), ids, k.data_ptr(),
                                   _rows_ld(k, "k"), v.data_ptr(), _rows_ld(v, "v"), raw),
           "hstu_cache_append")


def cache_gather(cache: PagedCache, offsets, total: int, seq_ids=None, kv_out=None, stream=None):
    """Whole sequences out of their pages: returns (kv [L, total, 2*H*64] in the
    layout of forward()'s kv_cache_out, timestamps [total])."""
    L, _, _, H, _, _ = cache.kv.shape
    n = offsets.numel() - 1
    if offsets.dtype is not torch.int64 or not offsets.is_contiguous():
        raise ValueError("cache_gather: offsets must be contiguous int64")
    if kv_out is not None:
        _dense(kv_out, (L, total, 2 * H * 64), cache.kv.dtype, "cache_gather", "kv_out")
    ids = _ids(seq_ids, n, "cache_gather")
    raw = _cache_stream(cache, stream, "cache_gather", offsets, seq_ids, kv_out)
    if kv_out is None:
        kv_out = _empty((L, total, 2 * H * 64), cache.kv.dtype, cache.kv.device, stream)
    ts = _empty(total, torch.int64, cache.kv.device, stream)
    _check(lib().hstu_cache_gather(ctypes.byref(cache.c()), n, ids, _p(offsets), total, _p(kv_out),
                                   _p(ts), raw), "hstu_cache_gather")
    return kv_out, ts


def cache_fork(cache: PagedCache, src_ids, dst_ids, stream=None):
    """dst_ids[i] (an empty sequence) becomes a copy of src_ids[i] sharing its pages."""
    n = src_ids.numel()
    src, dst = _ids(src_ids, n, "cache_fork"), _ids(dst_ids, n, "cache_fork")
    raw = _cache_stream(cache, stream, "cache_fork", src_ids, dst_ids)
    _check(lib().hstu_cache_fork(ctypes.byref(cache.c()), n, src, dst, raw), "hstu_cache_fork")


def cache_release(cache: PagedCache, seq_ids, window: int = 0, sinks: int = 0, stream=None):
    """Release whole sequences, or with a window the pages that no later event sees
    through it (later extensions take no wider one)."""
    n = seq_ids.numel()
    ids = _ids(seq_ids, n, "cache_release")
    raw = _cache_stream(cache, stream, "cache_release", seq_ids)
    _check(lib().hstu_cache_release(ctypes.byref(cache.c()), n, ids, window, sinks, raw),
           "hstu_cache_release")


def cache_compact(cache: PagedCache, workspace=None, stream=None) -> torch.Tensor:
    """Move the used pages into the lowest ids; returns their number (int32 [1], device)."""
    raw = _cache_stream(cache, stream, "cache_compact", workspace)
    live = _empty(1, torch.int32, cache.kv.device, stream)
    c = cache.c()
    if workspace is None:
        nbytes = lib().hstu_cache_workspace_bytes(ctypes.byref(c), 0)
        workspace = _workspace(nbytes, cache.kv.device, None, stream)
    _check(lib().hstu_cache_compact(ctypes.byref(c), _p(live), _p(workspace), workspace.numel(), raw),
           "hstu_cache_compact")
    return live


def _paged_attn(fn, cfg, cache, layer, chunk, q, rab_pos, rab_time, max_context, window, sinks,
                seq_ids, av_out, out_dtype, stream):
    kv, heads = cache.kv, cfg.num_heads
    rows = (chunk.total_tokens, heads * 64)
    if q.dtype is not kv.dtype or q.shape != rows:
        raise ValueError(f"{fn}: q must be [total_tokens, num_heads * 64] in the cache's type")
    f32 = torch.float32
    _dense(rab_pos, (heads, cfg.num_pos_buckets), f32, fn, "rab_pos")
    _dense(rab_time, (heads, cfg.num_time_buckets), f32, fn, "rab_time")
    if av_out is not None:
        _dense(av_out, rows, out_dtype, fn, "av_out")
    c, (j, times) = cfg.c(), _chunk(chunk, fn)
    ids = None if seq_ids is None else _ids(seq_ids, j.batch, fn)
    raw = _cache_stream(cache, stream, fn, q, rab_pos, rab_time, chunk.offsets, times,
                        seq_ids, av_out)
    if av_out is None:
        if stream is None and out_dtype is q.dtype:  # less host work than a shape and a device
            av_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            av_out = _empty(rows, out_dtype, q.device, stream)
    status = getattr(lib(), fn)(
        ctypes.byref(c), ctypes.byref(cache.desc), layer, ctypes.byref(j), ids, max_context, window,
        sinks, q.data_ptr(), _rows_ld(q, "q"), rab_pos.data_ptr(), rab_time.data_ptr(),
        av_out.data_ptr(), raw)
    _check(status, fn)
    return av_out


def paged_attn_fwd(cfg: LayerConfig, cache: PagedCache, layer: int, chunk: Jagged, q, rab_pos,
                   rab_time, max_context: int, window: int = 0, sinks: int = 0, seq_ids=None,
                   av_out=None, stream=None) -> torch.Tensor:
    """Eq. 2 for the chunk's rows (the last events of their sequences) over the
    cache: AV [T, H*64] in cfg dtype.  window > 0: a row sees the last `window`
    events up to itself and the first `sinks` events of its sequence."""
    return _paged_attn("hstu_paged_attn_fwd", cfg, cache, layer, chunk, q, rab_pos, rab_time,
                       max_context, window, sinks, seq_ids, av_out, cache.kv.dtype, stream)


def paged_attn_fwd_f32(cfg: LayerConfig, cache: PagedCache, layer: int, chunk: Jagged, q, rab_pos,
                       rab_time, max_context: int, window: int = 0, sinks: int = 0, seq_ids=None,
                       av_out=None, stream=None) -> torch.Tensor:
    """paged_attn_fwd with the result in fp32."""
    return _paged_attn("hstu_paged_attn_fwd_f32", cfg, cache, layer, chunk, q, rab_pos, rab_time,
                       max_context, window, sinks, seq_ids, av_out, torch.float32, stream)


def extend_workspace_bytes(cfg: LayerConfig, cache: PagedCache, batch: int, total_tokens: int) -> int:
    return lib().hstu_extend_workspace_bytes(ctypes.byref(cfg.c()), ctypes.byref(cache.c()), batch,
                                             total_tokens)


def extend(cfg: LayerConfig, weights: Sequence[LayerWeights], cache: PagedCache, chunk: Jagged,
           x_in, max_context: int, window: int = 0, sinks: int = 0, seq_ids=None, y_out=None,
           workspace=None, stream=None) -> torch.Tensor:
    """New events through the stack against the cache (reserve, then per layer f1,
    append, paged attention, f2); returns Y [T, d] fp32.  A pool that is too small, a
    sequence that would pass max_context or a missing page that a new row sees leaves the
    cache as it was and is reported in device_status()."""
    dev = x_in.device
    L = len(weights)
    rows = (chunk.total_tokens, cfg.d_model)
    _dense(x_in, rows, cfg.torch_dtype, "extend", "x_in")
    if y_out is not None:
        _dense(y_out, rows, torch.float32, "extend", "y_out")
    c, ca, (j, times) = cfg.c(), cache.c(), _chunk(chunk, "extend")
    ids = _ids(seq_ids, j.batch, "extend")
    raw = _cache_stream(cache, stream, "extend", x_in, chunk.offsets, times, seq_ids,
                        y_out, workspace)
    if y_out is None:
        y_out = _empty(rows, torch.float32, dev, stream)
    if workspace is None:
        nbytes = lib().hstu_extend_workspace_bytes(ctypes.byref(c), ctypes.byref(ca), j.batch,
                                                   j.total_tokens)
        workspace = _workspace(nbytes, dev, None, stream)
    arr = (LayerWeightsT * L)(*[w.c() for w in weights])
    _check(lib().hstu_extend(ctypes.byref(c), L, arr, ctypes.byref(ca), ctypes.byref(j),
                             ids, max_context, window, sinks, _p(x_in), _p(y_out), _p(workspace),
                             workspace.numel(), raw), "hstu_extend")
    return y_out


def device_status(stream=None) -> int:
    """Synchronise, read and clear the library's device status word."""
    return lib().hstu_get_device_status(_stream(stream))


def time_bucket_thresholds(num_time_buckets: int):
    import numpy as np
    out = np.zeros(num_time_buckets, dtype=np.int64)
    _check(lib().hstu_time_bucket_thresholds(num_time_buckets,
                                             out.ctypes.data_as(ctypes.c_void_p)),
           "hstu_time_bucket_thresholds")
    return out


def debug_rab_index(jag: Jagged, num_pos_buckets: int, num_time_buckets: int, stream=None):
    """Per-user n x n blocks of (position bucket, time bucket), -1 above the diagonal."""
    lens = (jag.offsets[1:] - jag.offsets[:-1]).to(torch.int64)
    blk = torch.zeros(jag.batch + 1, dtype=torch.int64, device=jag.offsets.device)
    blk[1:] = torch.cumsum(lens * lens, 0)
    total = int(blk[-1].item())
    pos = torch.full((max(total, 1),), -7, dtype=torch.int32, device=jag.offsets.device)
    tim = torch.full((max(total, 1),), -7, dtype=torch.int32, device=jag.offsets.device)
    j = jag.c()
    _check(lib().hstu_debug_rab_index(ctypes.byref(j), num_pos_buckets, num_time_buckets,
                                      _p(blk), _p(pos), _p(tim), _stream(stream)),
           "hstu_debug_rab_index")
    return blk, pos[:total], tim[:total]


def debug_wait_timeout(timeout_ns: int, stream=None):
    _check(lib().hstu_debug_wait_timeout(timeout_ns, _stream(stream)), "hstu_debug_wait_timeout")


def profiler_start():
    """Start bracketing every library kernel launch with CUDA events."""
    _check(lib().hstu_profiler_start(), "hstu_profiler_start")


def profiler_stop() -> dict:
    """Stop the profiler; returns {kernel name: (launches, total milliseconds)}."""
    arr = (KernelTimeT * 32)()
    n = ctypes.c_int32(0)
    _check(lib().hstu_profiler_stop(arr, 32, ctypes.byref(n)), "hstu_profiler_stop")
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}
