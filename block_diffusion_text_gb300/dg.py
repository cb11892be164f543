"""Python binding of libdg (ctypes).

Argument marshalling only: every step of the path runs in the CUDA kernels of
libdg.  PyTorch supplies device memory and the current stream.  The binding
fails loudly if the library has not been built (there is no CPU fallback).
The functions ``dg_*`` of the C ABI are reachable as ``lib().dg_*``; the
helpers below take torch tensors.
"""
from __future__ import annotations

import ctypes as ct
import math
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdg.so")
_lock = threading.Lock()
_lib = None

DG_OK, DG_ERR_ARG, DG_ERR_SHAPE, DG_ERR_CAPACITY, DG_ERR_WORKSPACE, DG_ERR_CUDA, DG_ERR_TIMEOUT, DG_ERR_VALUE = range(8)

# Every function the C header declares (checked by the tests).
EXPORTS = ("dg_status_string", "dg_workspace_size", "dg_read_status", "dg_tau", "dg_canvas_init",
           "dg_denoise_step", "dg_denoise_canvas", "dg_commit_block", "dg_debug_gemm",
           "dg_attention_noalloc", "dg_attention_noalloc_status", "dg_debug_wait_timeout",
           "dg_canvas_init_masked", "dg_denoise_step_masked", "dg_denoise_canvas_masked", "dg_prefill",
           "dg_quantize_rows_e4m3", "dg_kv8_append", "dg_kv8_read", "dg_kv8_attention_workspace",
           "dg_kv8_attention", "dg_w4_bytes", "dg_w4_quantize", "dg_w4_pack", "dg_w4_read", "dg_w4_matvec", "dg_w4_status",
           "dg_qk_norm_rope", "dg_moe_tokens_workspace", "dg_moe_tokens", "dg_sample")


class DgError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class dg_dims(ct.Structure):
    _fields_ = [("V", ct.c_int32), ("d", ct.c_int32), ("C", ct.c_int32), ("B", ct.c_int32),
                ("Hq", ct.c_int32), ("Hkv", ct.c_int32), ("hd", ct.c_int32), ("F", ct.c_int32),
                ("rope_base", ct.c_float), ("rms_eps", ct.c_float), ("L", ct.c_int32),
                ("n_exp", ct.c_int32), ("top_k", ct.c_int32), ("Fe", ct.c_int32)]


class dg_model(ct.Structure):
    _fields_ = [("dims", dg_dims)] + [(n, ct.c_void_p) for n in ("E", "Wq", "Wk", "Wv", "Wo", "W1", "W2",
                                                                 "E8", "E8_scale", "Wr", "We1", "We2")]


class dg_kv_cache(ct.Structure):
    _fields_ = [("K", ct.c_void_p), ("V", ct.c_void_p), ("cap", ct.c_int32), ("len", ct.c_int32)]


class dg_canvas(ct.Structure):
    _fields_ = [("tokens", ct.c_void_p), ("z", ct.c_void_p), ("alpha", ct.c_void_p),
                ("prev_argmax", ct.c_void_p)]


class dg_step_debug(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("a", "q", "k", "v", "o", "h", "u", "g", "logits", "moe_idx", "moe_gate",
                                           "moe_logits", "moe_x")]


class dg_step_out(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("entropy", "argmax", "accept", "n_acc", "mean_H", "stop")] + [
        ("debug", ct.POINTER(dg_step_debug)), ("events", ct.POINTER(ct.c_void_p))]


class dg_kv8_cache(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("K", "V", "K_exp", "V_exp", "len", "status")] + [
        (n, ct.c_int32) for n in ("B", "Hkv", "cap", "hd")]


class dg_w4(ct.Structure):
    _fields_ = [("codes", ct.c_void_p), ("scales", ct.c_void_p), ("N", ct.c_int32), ("K", ct.c_int32),
                ("group", ct.c_int32)]


class dg_sampling(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("temperature", "top_p", "min_p", "top_k")] + [
        (n, ct.c_float) for n in ("temperature_all", "top_p_all", "min_p_all")] + [("top_k_all", ct.c_int32)]


# Kernel slots of one step (dg_step_out.events), in launch order.
PROF_SLOTS = ("embed", "qkv", "attn", "oproj", "lmhead", "stats", "sampler", "p0", "selfcond",
              "reduce", "ffw1", "ffw2", "moe")


class dg_sched(ct.Structure):
    _fields_ = [("tau0", ct.c_float), ("tau1", ct.c_float), ("N", ct.c_int32), ("b", ct.c_float),
                ("stop_H", ct.c_float)]


class dg_canvas_result(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("steps_taken", "converged", "accepted", "xhat0")]


def load():
    """Load libdg.so; raises if it is missing (build it with __graft_entry__.build())."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libdg is not built ({LIB_PATH} missing); run __graft_entry__.build()")
            L = ct.CDLL(LIB_PATH)
            L.dg_status_string.restype = ct.c_char_p
            L.dg_status_string.argtypes = [ct.c_int32]
            for name in EXPORTS[1:]:
                getattr(L, name).restype = ct.c_int32
            L.dg_workspace_size.argtypes = [ct.POINTER(dg_dims), ct.c_int32, ct.POINTER(ct.c_size_t)]
            L.dg_read_status.argtypes = [ct.c_void_p, ct.POINTER(ct.c_int32), ct.c_void_p]
            L.dg_tau.argtypes = [ct.POINTER(dg_sched), ct.c_int32, ct.POINTER(ct.c_float)]
            L.dg_attention_noalloc_status.argtypes = [ct.POINTER(ct.c_int32), ct.c_void_p]
            L.dg_canvas_init_masked.argtypes = [ct.c_void_p, ct.c_int32, ct.c_int32, ct.c_int32, ct.c_void_p]
            L.dg_denoise_step_masked.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache),
                                                 ct.POINTER(dg_canvas), ct.c_float, ct.c_int32, ct.c_int32,
                                                 ct.c_int32, ct.c_void_p, ct.c_size_t, ct.POINTER(dg_step_out),
                                                 ct.c_void_p]
            L.dg_denoise_canvas_masked.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache),
                                                   ct.POINTER(dg_canvas), ct.POINTER(dg_sched), ct.c_int32,
                                                   ct.c_void_p, ct.c_size_t, ct.POINTER(dg_canvas_result),
                                                   ct.c_void_p]
            L.dg_canvas_init.argtypes = [ct.c_void_p, ct.c_int32, ct.c_int32, ct.c_int32, ct.c_uint64,
                                         ct.c_int32, ct.c_void_p]
            L.dg_denoise_step.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache),
                                          ct.POINTER(dg_canvas), ct.c_float, ct.c_float, ct.c_uint64,
                                          ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_size_t,
                                          ct.POINTER(dg_step_out), ct.c_void_p]
            L.dg_denoise_canvas.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache),
                                            ct.POINTER(dg_canvas), ct.POINTER(dg_sched), ct.c_uint64,
                                            ct.c_int32, ct.c_void_p, ct.c_size_t,
                                            ct.POINTER(dg_canvas_result), ct.c_void_p]
            L.dg_commit_block.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache), ct.c_void_p,
                                          ct.c_void_p, ct.c_size_t, ct.c_void_p]
            L.dg_prefill.argtypes = [ct.POINTER(dg_model), ct.POINTER(dg_kv_cache), ct.c_void_p, ct.c_int32,
                                     ct.c_void_p, ct.c_size_t, ct.c_void_p]
            L.dg_debug_wait_timeout.argtypes = [ct.POINTER(ct.c_int32), ct.c_void_p]
            L.dg_quantize_rows_e4m3.argtypes = [ct.c_void_p, ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_void_p,
                                                ct.c_void_p]
            L.dg_debug_gemm.argtypes = [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int32, ct.c_int32,
                                        ct.c_int32, ct.c_int32, ct.c_void_p]
            L.dg_attention_noalloc.argtypes = [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int32, ct.c_int32,
                                               ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int32, ct.c_int32,
                                               ct.c_int32, ct.c_int32, ct.c_int32, ct.c_void_p]
            L.dg_kv8_append.argtypes = [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int32, ct.c_void_p, ct.c_void_p]
            L.dg_kv8_read.argtypes = [ct.c_void_p, ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_void_p, ct.c_int32,
                                      ct.c_void_p]
            L.dg_kv8_attention_workspace.argtypes = [ct.c_void_p, ct.c_int32, ct.c_int32, ct.POINTER(ct.c_size_t)]
            L.dg_kv8_attention.argtypes = [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                           ct.c_int32, ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_size_t,
                                           ct.c_void_p]
            i32, i64, vp = ct.c_int32, ct.c_int64, ct.c_void_p
            L.dg_w4_bytes.argtypes = [i32, i32, i32, ct.POINTER(ct.c_size_t), ct.POINTER(ct.c_size_t)]
            L.dg_w4_quantize.argtypes = [vp, vp, i64, vp, vp]
            L.dg_w4_pack.argtypes = [vp, vp, vp, vp]
            L.dg_w4_read.argtypes = [vp, vp, i64, vp]
            L.dg_w4_matvec.argtypes = [vp, vp, i64, i32, vp, ct.c_float, vp, i64, vp, i64, i32, vp]
            L.dg_w4_status.argtypes = [ct.POINTER(i32), vp]
            L.dg_qk_norm_rope.argtypes = [vp, i64, i64] + [vp] * 6 + [i32] * 5 + [ct.c_float] * 2 + [vp]
            L.dg_moe_tokens_workspace.argtypes = [vp, i32, ct.POINTER(ct.c_size_t)]
            L.dg_moe_tokens.argtypes = [vp, i32, vp, vp, i32, vp, vp, vp, ct.c_size_t, vp]
            L.dg_sample.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp]
            _lib = L
    return _lib


lib = load


def status_string(code: int) -> str:
    try:
        return load().dg_status_string(code).decode()
    except Exception:  # library missing while formatting an error
        return "status"


def _check(code, what):
    if code != DG_OK:
        raise DgError(code, what)


def _ptr(t):
    return None if t is None else ct.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ct.c_void_p(s.cuda_stream)


def make_dims(d) -> dg_dims:
    return dg_dims(V=d.V, d=d.d, C=d.C, B=d.B, Hq=d.Hq, Hkv=d.Hkv, hd=d.hd, F=d.F,
                   rope_base=d.rope_base, rms_eps=d.rms_eps, L=getattr(d, "L", 1),
                   n_exp=getattr(d, "n_exp", 0), top_k=getattr(d, "top_k", 0), Fe=getattr(d, "Fe", 0))


def workspace_size(dims, cap: int) -> int:
    n = ct.c_size_t()
    _check(load().dg_workspace_size(ct.byref(make_dims(dims)), int(cap), ct.byref(n)), "dg_workspace_size")
    return n.value


class Model:
    """Weights (bf16 device tensors, [out][in]) and the prefix cache of a batch of canvases."""

    def __init__(self, dims, w: dict, cache_len: int | None = None, fp8_head: bool = False):
        """fp8_head: quantize E per row to E4M3 (quantize_rows_e4m3) and take the
        LM head's logits on the FP8 tensor cores; E8 / E8_scale are then kept
        here as the codes and scales."""
        self.dims = dims
        self.w = w
        self.K, self.V = w["Kc"], w["Vc"]
        self.cap = self.K.shape[-2]
        self.len = dims.P if cache_len is None else cache_len
        self.E8 = self.E8_scale = None
        if fp8_head:
            self.E8, self.E8_scale = quantize_rows_e4m3(w["E"])
        self.s = dg_model(make_dims(dims), *[ct.c_void_p(w[k].data_ptr()) for k in
                                             ("E", "Wq", "Wk", "Wv", "Wo", "W1", "W2")],
                          ct.c_void_p(self.E8.data_ptr() if fp8_head else None),
                          ct.c_void_p(self.E8_scale.data_ptr() if fp8_head else None),
                          *[ct.c_void_p(w[k].data_ptr() if k in w else None) for k in ("Wr", "We1", "We2")])
        self.ws_bytes = workspace_size(dims, self.cap)
        # zero-initialised: the first word is the device status word
        self.ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=self.K.device)
        off = (-self.ws.data_ptr()) % 256
        self.ws_ptr = ct.c_void_p(self.ws.data_ptr() + off)

    def cache(self) -> dg_kv_cache:
        key = (self.K.data_ptr(), self.V.data_ptr(), self.cap, self.len)
        if getattr(self, "_cache_key", None) != key:
            self._cache_s = dg_kv_cache(ct.c_void_p(key[0]), ct.c_void_p(key[1]), self.cap, self.len)
            self._cache_key = key
        return self._cache_s

    def workspace_for(self, cap: int):
        """(pointer, bytes) of a workspace for a cache of `cap` rows: the model's own when that is
        large enough, else one allocated once per capacity (a commit into a larger cache)."""
        if cap <= self.cap:
            return self.ws_ptr, self.ws_bytes
        extra = getattr(self, "_ws_extra", {})
        if cap not in extra:
            nb = workspace_size(self.dims, cap)
            t = torch.zeros(nb + 256, dtype=torch.uint8, device=self.K.device)
            extra[cap] = (t, ct.c_void_p(t.data_ptr() + (-t.data_ptr()) % 256), nb)
            self._ws_extra = extra
        return extra[cap][1], extra[cap][2]

    def status(self) -> int:
        """The device status word (first non-zero over the model's workspaces)."""
        for ptr in [self.ws_ptr] + [e[1] for e in getattr(self, "_ws_extra", {}).values()]:
            st = ct.c_int32()
            _check(load().dg_read_status(ptr, ct.byref(st), _stream()), "dg_read_status")
            if st.value:
                return st.value
        return 0


@dataclass
class Canvas:
    tokens: torch.Tensor          # int32 [B, C]
    z: torch.Tensor               # bf16 [B, C, d]
    alpha: torch.Tensor           # fp32 [B, C]
    prev_argmax: torch.Tensor | None = None

    def __post_init__(self):
        if self.prev_argmax is None:
            self.prev_argmax = torch.zeros_like(self.tokens)

    def struct(self) -> dg_canvas:
        key = (self.tokens.data_ptr(), self.z.data_ptr(), self.alpha.data_ptr(), self.prev_argmax.data_ptr())
        if getattr(self, "_key", None) != key:
            self._s = dg_canvas(*[ct.c_void_p(p) for p in key])
            self._key = key
        return self._s


_STEP_OUT_CACHE: dict = {}


def denoise_step(model: Model, canvas: Canvas, tau: float, b: float, seed: int, step: int, block: int = 0,
                 debug: bool = False, stream=None, events=None, out=None, masked=None) -> dict:
    """One denoising step (dg_denoise_step); updates canvas in place, returns outputs.

    events: optional list of 2 * len(PROF_SLOTS) recorded torch.cuda.Event (per-kernel timing).
    out: optional dict of preallocated output tensors (as returned by a previous call).
    masked: optional (mask_id, N): a step of masked confidence decoding (dg_denoise_step_masked)
    instead; b, seed and block are then not used.
    """
    d = model.dims
    dev = canvas.tokens.device
    M = d.B * d.C
    if out is None:
        out = dict(entropy=torch.empty(d.B, d.C, dtype=torch.float32, device=dev),
                   argmax=torch.empty(d.B, d.C, dtype=torch.int32, device=dev),
                   accept=torch.empty(d.B, d.C, dtype=torch.uint8, device=dev),
                   n_acc=torch.empty(d.B, dtype=torch.int32, device=dev),
                   mean_H=torch.empty(d.B, dtype=torch.float32, device=dev),
                   stop=torch.empty(d.B, dtype=torch.int32, device=dev))
    keys = ("entropy", "argmax", "accept", "n_acc", "mean_H", "stop")
    ptrs = tuple(out[k].data_ptr() for k in keys)
    so = _STEP_OUT_CACHE.get(ptrs) if events is None and not debug else None
    if so is None:
        so = dg_step_out(*[ct.c_void_p(p) for p in ptrs])
        if events is None and not debug:
            _STEP_OUT_CACHE.clear()  # one entry: the output set of the latest plain call
            _STEP_OUT_CACHE[ptrs] = so
    if events is not None:
        if len(events) != 2 * len(PROF_SLOTS):
            raise ValueError(f"events: expected {2 * len(PROF_SLOTS)} entries, got {len(events)}")
        arr = (ct.c_void_p * len(events))(*[ct.c_void_p(e.cuda_event if e is not None else 0) for e in events])
        so.events = ct.cast(arr, ct.POINTER(ct.c_void_p))
    dbg = None
    if debug:
        bf = dict(dtype=torch.bfloat16, device=dev)
        dbg_t = dict(a=torch.empty(M, d.d, **bf), q=torch.empty(d.B, d.Hq, d.C, d.hd, **bf),
                     k=torch.empty(d.B, d.Hkv, d.C, d.hd, **bf), v=torch.empty(d.B, d.Hkv, d.C, d.hd, **bf),
                     o=torch.empty(M, d.Hq * d.hd, **bf), h=torch.empty(M, d.d, **bf),
                     u=torch.empty(M, d.d, **bf), g=torch.empty(M, d.F, **bf),
                     logits=torch.empty(M, d.V, dtype=torch.float32, device=dev))
        ne, tk = getattr(d, "n_exp", 0), getattr(d, "top_k", 0)
        if ne > 0:
            dbg_t.update(moe_idx=torch.empty(M, tk, dtype=torch.int32, device=dev),
                         moe_gate=torch.empty(M, tk, dtype=torch.float32, device=dev),
                         moe_logits=torch.empty(M, ne, dtype=torch.float32, device=dev),
                         moe_x=torch.empty(M, d.d, **bf))
        dbg = dg_step_debug(*[_ptr(dbg_t.get(k)) for k in ("a", "q", "k", "v", "o", "h", "u", "g", "logits",
                                                            "moe_idx", "moe_gate", "moe_logits", "moe_x")])
        so.debug = ct.pointer(dbg)
        out["debug"] = dbg_t
    cs = canvas.struct()
    cache = model.cache()
    if masked is not None:
        mask_id, N = masked
        rc = load().dg_denoise_step_masked(ct.byref(model.s), ct.byref(cache), ct.byref(cs), float(tau),
                                           int(mask_id), int(step), int(N), model.ws_ptr, model.ws_bytes,
                                           ct.byref(so), _stream(stream))
        _check(rc, "dg_denoise_step_masked")
        return out
    rc = load().dg_denoise_step(ct.byref(model.s), ct.byref(cache), ct.byref(cs), float(tau), float(b),
                                int(seed), int(step), int(block), model.ws_ptr, model.ws_bytes,
                                ct.byref(so), _stream(stream))
    _check(rc, "dg_denoise_step")
    return out


def tau(step: int, N: int = 48, tau0: float = 0.8, tau1: float = 0.4) -> float:
    """Temperature of step `step` of the annealed schedule, as the library computes it (dg_tau)."""
    t = ct.c_float()
    _check(load().dg_tau(ct.byref(dg_sched(tau0, tau1, N, 0.1, 0.005)), int(step), ct.byref(t)), "dg_tau")
    return t.value


def tau_schedule(N=48, tau0=0.8, tau1=0.4):
    """Temperatures of steps 0..N-1 (dg_tau for each step)."""
    return [tau(s, N, tau0, tau1) for s in range(N)]


def denoise_canvas(model: Model, canvas: Canvas, seed: int, block: int = 0, N: int = 48, tau0: float = 0.8,
                   tau1: float = 0.4, b: float = 0.1, stop_H: float = 0.005, stream=None) -> dict:
    """The annealed loop (dg_denoise_canvas); returns device tensors of the result."""
    d = model.dims
    dev = canvas.tokens.device
    res = dict(steps_taken=torch.empty(d.B, dtype=torch.int32, device=dev),
               converged=torch.empty(d.B, dtype=torch.int32, device=dev),
               accepted=torch.empty(d.B, N, dtype=torch.int32, device=dev),
               xhat0=torch.empty(d.B, d.C, dtype=torch.int32, device=dev))
    rs = dg_canvas_result(*[_ptr(res[k]) for k in ("steps_taken", "converged", "accepted", "xhat0")])
    sched = dg_sched(tau0, tau1, N, b, stop_H)
    cs = canvas.struct()
    cache = model.cache()
    rc = load().dg_denoise_canvas(ct.byref(model.s), ct.byref(cache), ct.byref(cs), ct.byref(sched), int(seed),
                                  int(block), model.ws_ptr, model.ws_bytes, ct.byref(rs), _stream(stream))
    _check(rc, "dg_denoise_canvas")
    return res


def denoise_canvas_masked(model: Model, canvas: Canvas, mask_id: int, N: int = 16, tau: float = 1.0,
                          stream=None) -> dict:
    """Masked confidence decoding loop (dg_denoise_canvas_masked): N steps at temperature tau."""
    d = model.dims
    dev = canvas.tokens.device
    res = dict(steps_taken=torch.empty(d.B, dtype=torch.int32, device=dev),
               converged=torch.empty(d.B, dtype=torch.int32, device=dev),
               accepted=torch.empty(d.B, N, dtype=torch.int32, device=dev),
               xhat0=torch.empty(d.B, d.C, dtype=torch.int32, device=dev))
    rs = dg_canvas_result(*[_ptr(res[k]) for k in ("steps_taken", "converged", "accepted", "xhat0")])
    sched = dg_sched(tau, tau, N, 0.0, 0.0)
    cs = canvas.struct()
    cache = model.cache()
    rc = load().dg_denoise_canvas_masked(ct.byref(model.s), ct.byref(cache), ct.byref(cs), ct.byref(sched),
                                         int(mask_id), model.ws_ptr, model.ws_bytes, ct.byref(rs), _stream(stream))
    _check(rc, "dg_denoise_canvas_masked")
    return res


def canvas_init_masked(B, C, mask_id, device="cuda", stream=None) -> torch.Tensor:
    """A canvas of [MASK] tokens (dg_canvas_init_masked)."""
    t = torch.empty(B, C, dtype=torch.int32, device=device)
    _check(load().dg_canvas_init_masked(_ptr(t), B, C, int(mask_id), _stream(stream)), "dg_canvas_init_masked")
    return t


def commit_block(model: Model, tokens: torch.Tensor, stream=None, cache=None) -> int:
    """Append the re-encoded K/V of tokens [B, C] to the cache (dg_commit_block).

    cache: optional (K, V, len) of another cache with the model's layout ([B, Hkv, cap, hd] bf16);
    by default the model's own cache, whose length is advanced.  Returns the new length."""
    if cache is None:
        cs = model.cache()
    else:
        K, V, n = cache
        cs = dg_kv_cache(ct.c_void_p(K.data_ptr()), ct.c_void_p(V.data_ptr()), K.shape[-2], int(n))
    ws, wsb = model.workspace_for(cs.cap)
    rc = load().dg_commit_block(ct.byref(model.s), ct.byref(cs), _ptr(tokens), ws, wsb, _stream(stream))
    _check(rc, "dg_commit_block")
    if cache is None:
        model.len = cs.len
    return cs.len


def prefill(model: Model, tokens: torch.Tensor, stream=None) -> int:
    """Causal prefill of tokens [B, n] into every layer's cache (dg_prefill); returns the new length."""
    cache = model.cache()
    tok = tokens.contiguous()
    rc = load().dg_prefill(ct.byref(model.s), ct.byref(cache), _ptr(tok), int(tok.shape[-1]), model.ws_ptr,
                           model.ws_bytes, _stream(stream))
    _check(rc, "dg_prefill")
    model.len = cache.len
    return cache.len


def canvas_init(B, C, V, seed, block=0, device="cuda", stream=None) -> torch.Tensor:
    t = torch.empty(B, C, dtype=torch.int32, device=device)
    _check(load().dg_canvas_init(_ptr(t), B, C, V, int(seed), int(block), _stream(stream)), "dg_canvas_init")
    return t


def debug_gemm(A: torch.Tensor, Bm: torch.Tensor, b_mn_major: int = 0, stream=None) -> torch.Tensor:
    """fp32 A B^T on the tensor-core engine; B is [N][K] (b_mn_major 0, 3 on CTA pairs, 5-8 on
    the cluster split-K engine) or [K][N] (1 or 2, or 4 on CTA pairs)."""
    M, K = A.shape
    N = Bm.shape[0] if b_mn_major in (0, 3, 5, 6, 7, 8) else Bm.shape[1]
    D = torch.empty(M, N, dtype=torch.float32, device=A.device)
    _check(load().dg_debug_gemm(_ptr(A), _ptr(Bm), _ptr(D), M, N, K, b_mn_major, _stream(stream)),
           "dg_debug_gemm")
    return D


def debug_wait_timeout(stream=None) -> int:
    """Run the never-satisfied bounded wait (dg_debug_wait_timeout); returns the status word it left."""
    st = ct.c_int32(-1)
    _check(load().dg_debug_wait_timeout(ct.byref(st), _stream(stream)), "dg_debug_wait_timeout")
    return st.value


def attention_noalloc(q, K, V, cache_len, k, v, o=None, stream=None) -> torch.Tensor:
    """Step attention with the library's static scratch (dg_attention_noalloc), for callers
    that cannot allocate device memory; q [B,Hq,C,hd], K/V [B,Hkv,cap,hd], k/v [B,Hkv,C,hd]."""
    B, Hq, C, hd = q.shape
    Hkv, cap = K.shape[1], K.shape[2]
    if o is None:
        o = torch.empty(B * C, Hq * hd, dtype=q.dtype, device=q.device)
    _check(load().dg_attention_noalloc(_ptr(q), _ptr(K), _ptr(V), cap, int(cache_len), _ptr(k), _ptr(v), _ptr(o),
                                       B, C, Hq, Hkv, hd, _stream(stream)), "dg_attention_noalloc")
    return o


def attention_noalloc_status(stream=None) -> int:
    """Status word of the last attention_noalloc call on this device (synchronises the stream)."""
    st = ct.c_int32(-1)
    _check(load().dg_attention_noalloc_status(ct.byref(st), _stream(stream)), "dg_attention_noalloc_status")
    return st.value


def quantize_rows_e4m3(X: torch.Tensor, stream=None):
    """Per-row E4M3 codes (uint8 [R, d]) and scales (fp32 [R]) of a bf16 matrix X [R, d]."""
    assert X.dtype == torch.bfloat16 and X.dim() == 2 and X.is_contiguous()
    R, d = X.shape
    Q = torch.empty((R, d), dtype=torch.uint8, device=X.device)
    sc = torch.empty(R, dtype=torch.float32, device=X.device)
    _check(load().dg_quantize_rows_e4m3(_ptr(X), R, d, _ptr(Q), _ptr(sc), _stream(stream)),
           "dg_quantize_rows_e4m3")
    return Q, sc


KV8_BLOCK = 64  # cached tokens per scale of the 8-bit cache

# Workspaces of kv8_attention, one for each (device, stream): the calls of a stream run one after another, so the caches
# of a stack share it.  The lock is held until a call's launches are enqueued: those of two host threads on one stream
# must not mix, and none may replace a workspace that another has not launched with yet.
_kv8_workspaces = {}
_kv8_lock = threading.Lock()


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class Kv8Cache:
    """An 8-bit prefix cache (dg_kv8_cache): E4M3 codes with a power-of-two scale per 64 rows and head.

    K, V: uint8 [B, Hkv, cap, hd] codes; K_exp, V_exp: uint8 [B, Hkv, ceil(cap / 64)] exponent bytes (scale
    2^(x - 127)); len: int32 [B], the rows each sequence holds; all on one CUDA device, contiguous, and kept by
    this object.  No call advances len: after the appends of all layers do ``cache.len += n`` on the same stream.
    status: int32 [1] device word, shared by the caches of a stack when given."""

    def __init__(self, K, V, K_exp, V_exp, len, status=None):
        _need(K.dim() == 4 and V.shape == K.shape and K.dtype == V.dtype == torch.uint8,
              "K, V: uint8 codes [B, Hkv, cap, hd]")
        B, Hkv, cap, hd = K.shape
        nblk = -(-cap // KV8_BLOCK)
        _need(K_exp.shape == V_exp.shape == (B, Hkv, nblk) and K_exp.dtype == V_exp.dtype == torch.uint8,
              f"K_exp, V_exp: uint8 [{B}, {Hkv}, {nblk}]")
        _need(len.shape == (B,) and len.dtype == torch.int32, f"len: int32 [{B}]")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=K.device)
        _need(status.shape == (1,) and status.dtype == torch.int32, "status: int32 [1]")
        for t in (K, V, K_exp, V_exp, len, status):
            _need(t.is_cuda and t.device == K.device and t.is_contiguous(),
                  "the cache's tensors are contiguous and on one CUDA device")
        self.K, self.V, self.K_exp, self.V_exp, self._len, self.status_word = K, V, K_exp, V_exp, len, status
        self.B, self.Hkv, self.cap, self.hd = B, Hkv, cap, hd
        self.device = K.device
        self.s = dg_kv8_cache(*[t.data_ptr() for t in (K, V, K_exp, V_exp, len, status)], B, Hkv, cap, hd)
        self._ref = ct.byref(self.s)
        self._lib = load()
        self._index = K.device.index
        self._ws_bytes, self._shapes = {}, {}

    @property
    def len(self) -> torch.Tensor:
        """The device lengths that every call reads: int32 [B]."""
        return self._len

    @len.setter
    def len(self, value):
        # the calls hold the tensor's address: an assignment writes into it
        if value is not self._len:
            self._len.copy_(value)

    @classmethod
    def empty(cls, B, Hkv, cap, hd, device="cuda"):
        """A cache of `cap` rows per sequence that holds none yet."""
        u8 = dict(dtype=torch.uint8, device=device)
        nblk = -(-cap // KV8_BLOCK)
        return cls(torch.zeros(B, Hkv, cap, hd, **u8), torch.zeros(B, Hkv, cap, hd, **u8),
                   torch.zeros(B, Hkv, nblk, **u8), torch.zeros(B, Hkv, nblk, **u8),
                   torch.zeros(B, dtype=torch.int32, device=device))

    def status(self, stream=None) -> int:
        """The device status word (synchronises the stream)."""
        st = ct.c_int32()
        _check(load().dg_read_status(_ptr(self.status_word), ct.byref(st), _stream(stream)), "dg_read_status")
        return st.value

    def workspace_bytes(self, C: int, Hq: int) -> int:
        """Bytes of workspace of kv8_attention with C new tokens and Hq query heads."""
        n = self._ws_bytes.get((C, Hq))
        if n is None:
            z = ct.c_size_t()
            _check(self._lib.dg_kv8_attention_workspace(self._ref, C, Hq, ct.byref(z)), "dg_kv8_attention_workspace")
            n = self._ws_bytes[(C, Hq)] = z.value
        return n

    def _attention_shapes(self, q):
        """(C, Hq, shape of k and v, shape of the output, bytes of workspace) of queries shaped like q."""
        if q.dim() != 4 or q.shape[0] != self.B or q.shape[3] != self.hd:
            raise ValueError(f"q: contiguous bf16 [{self.B}, Hq, C, {self.hd}], got {tuple(q.shape)}")
        self._bf16(q, q.shape, "q")
        _, Hq, C, _ = q.shape
        r = self._shapes[q.shape] = (C, Hq, torch.Size((self.B, self.Hkv, C, self.hd)),
                                     torch.Size((self.B * C, Hq * self.hd)), self.workspace_bytes(C, Hq))
        return r

    def _bf16(self, t, shape, what):
        """The address of a contiguous bf16 tensor of that shape on the cache's device."""
        if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{what}: contiguous bf16 {list(shape)} on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _launch_stream(self, stream):
        """The raw stream of a launch: the library launches on the current device, so that must be the cache's."""
        if torch._C._cuda_getDevice() != self._index:
            raise ValueError(f"the cache lies on {self.device}, the current device is another")
        return torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream


def kv8_append(cache: Kv8Cache, k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None,
               stream=None) -> None:
    """Quantise rows k, v (bf16 [B, Hkv, n, hd]) into the cache at rows len.. (dg_kv8_append).

    counts: optional int32 [B], rows of each sequence (the rest is padding).  len is not advanced."""
    n = k.shape[2] if k.dim() == 4 else -1
    shape = (cache.B, cache.Hkv, n, cache.hd)
    kp, vp, cp = cache._bf16(k, shape, "k"), cache._bf16(v, shape, "v"), None
    if counts is not None:
        if counts.shape != (cache.B,) or counts.dtype is not torch.int32 or counts.get_device() != cache._index \
                or not counts.is_contiguous():
            raise ValueError(f"counts: contiguous int32 [{cache.B}] on {cache.device}")
        cp = counts.data_ptr()
    if n == 0:
        return
    rc = cache._lib.dg_kv8_append(cache._ref, kp, vp, n, cp, cache._launch_stream(stream))
    if rc:
        raise DgError(rc, "dg_kv8_append")


def kv8_read(cache: Kv8Cache, row0: int, n: int, out=None, stream=None):
    """Rows row0 .. row0 + n of every sequence as bf16 (dg_kv8_read): (K, V), each [B, Hkv, n, hd].

    out: optional (K, V) of at least n rows, e.g. the caches of a Model; rows at or past a sequence's length are
    left as they are (zeros where this call makes the tensors)."""
    st = cache._launch_stream(stream)
    if out is None:
        with torch.cuda.stream(stream):
            K = torch.zeros(cache.B, cache.Hkv, n, cache.hd, dtype=torch.bfloat16, device=cache.device)
            V = torch.zeros_like(K)
    else:
        K, V = out
        pitch = K.shape[2] if K.dim() == 4 else -1
        shape = (cache.B, cache.Hkv, pitch, cache.hd)
        cache._bf16(K, shape, "out[0]")
        cache._bf16(V, shape, "out[1]")
    if n == 0:
        return K, V
    rc = cache._lib.dg_kv8_read(cache._ref, row0, n, K.data_ptr(), V.data_ptr(), K.shape[2], st)
    if rc:
        raise DgError(rc, "dg_kv8_read")
    return K, V


def kv8_attention(cache: Kv8Cache, q: torch.Tensor, k: torch.Tensor | None = None, v: torch.Tensor | None = None,
                  causal: bool = False, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Attention of C new tokens over the cached rows and their own k, v (dg_kv8_attention); o [B*C, Hq*hd].

    q: bf16 [B, Hq, C, hd]; k, v: bf16 [B, Hkv, C, hd], or None for the cached rows alone.  ws: optional uint8
    workspace of cache.workspace_bytes(C, Hq) bytes, not shared by calls that may overlap; by default the calls of a
    stream share one, which is kept (kv8_release_workspaces), and a captured call takes one from the graph's pool."""
    C, Hq, new, shape, wn = cache._shapes.get(q.shape) or cache._attention_shapes(q)
    qp, kp, vp = cache._bf16(q, q.shape, "q"), None, None
    if k is not None and v is not None:
        kp, vp = cache._bf16(k, new, "k"), cache._bf16(v, new, "v")
    elif k is not v:
        raise ValueError("k and v come together")
    st = cache._launch_stream(stream)
    if out is not None:
        op = cache._bf16(out, shape, "out")
    else:
        if stream is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        else:
            with torch.cuda.stream(stream):  # memory of the launching stream
                out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        op = out.data_ptr()

    wp, flag = None, 1 if causal else 0
    if ws is not None:
        _need(ws.device == cache.device and ws.is_contiguous(), "ws: contiguous, on the cache's device")
        wp, wn = ws.data_ptr(), ws.numel() * ws.element_size()
    elif wn:
        if not _capturing(stream):
            with _kv8_lock:
                t = _kv8_workspaces.get((cache._index, st))
                if t is None or t.numel() < wn:
                    with torch.cuda.stream(stream):  # memory of the launching stream
                        t = torch.empty(wn, dtype=torch.uint8, device=cache.device)
                    _kv8_workspaces[cache._index, st] = t
                wp = t.data_ptr()
                rc = cache._lib.dg_kv8_attention(cache._ref, qp, kp, vp, op, C, Hq, flag, wp, wn, st)
            if rc:
                raise DgError(rc, "dg_kv8_attention")
            return out
        # from the graph's own pool, so that graphs that overlap share none; held until the launches are enqueued, since
        # the pool gives the memory of a tensor to the next one as soon as it is let go
        with torch.cuda.stream(stream):
            ws = torch.empty(wn, dtype=torch.uint8, device=cache.device)
        wp = ws.data_ptr()
    rc = cache._lib.dg_kv8_attention(cache._ref, qp, kp, vp, op, C, Hq, flag, wp, wn, st)
    if rc:
        raise DgError(rc, "dg_kv8_attention")
    return out


def _capturing(stream):
    """Whether the stream (None: the current one) is being captured into a graph."""
    if stream is None:
        return torch._C._cuda_isCurrentStreamCapturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def kv8_release_workspaces(device=None) -> None:
    """Let go of the workspaces that kv8_attention keeps for the streams of `device` (default: of every device).

    Their memory goes back to PyTorch's allocator in the order of each stream; the next call takes a new one.  To be
    called before a stream that PyTorch does not own is destroyed: another may come to have its handle."""
    index = None if device is None else torch.device(device).index
    if device is not None and index is None:
        index = torch.cuda.current_device()
    with _kv8_lock:
        for key in [k for k in _kv8_workspaces if index is None or k[0] == index]:
            del _kv8_workspaces[key]


# ------------------------------------------------- operators of a decoded token
# Their device time is a few microseconds for small calls, so the checks of the usual case are few and made in place.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _on(t, dtype, what, index):
    """Checks a tensor's type and device (a CUDA device's index); returns the tensor."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{what}: {dtype} on cuda:{index}, got {t.dtype} on {t.device}")
    return t


def _index_of(t, what):
    """The index of the tensor's CUDA device."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{what}: a CUDA tensor, got one on {t.device}")
    return i


def _raw_stream(index, stream):
    """The raw stream of a launch: the library launches on the current device, so that must be the tensors'."""
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the tensors lie on cuda:{index}, the current device is another")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """Memory of the launching stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _i32(what, *sizes):
    """Sizes go to the library as 32 bits, and ctypes cuts larger ones: they are refused as it refuses what is too large."""
    for v in sizes:
        if not -1 << 31 <= v < 1 << 31:
            raise DgError(DG_ERR_SHAPE, what)


def _rows_of(t, dtype, width, what, index):
    """(rows, pitch) of a 2-D tensor whose rows of `width` elements are contiguous."""
    _on(t, dtype, what, index)
    if t.dim() != 2 or t.shape[1] != width or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: [rows, {width}] with contiguous rows, got {tuple(t.shape)}, strides {t.stride()}")
    rows = t.shape[0]
    return rows, (t.stride(0) if rows > 1 else max(width, t.stride(0)))


class W4Matrix:
    """A matrix [N, K] of 4-bit weights with a bf16 scale for each row and `group` columns (dg_w4), laid out for
    w4_matvec.  Made by w4_quantize or W4Matrix.from_codes; read() gives the weights back."""

    def __init__(self, N, K, group, device="cuda"):
        self._lib = load()
        _i32("dg_w4_bytes", N, K, group)
        nc, ns = ct.c_size_t(), ct.c_size_t()
        _check(self._lib.dg_w4_bytes(N, K, group, ct.byref(nc), ct.byref(ns)), "dg_w4_bytes")
        self.codes = torch.empty(nc.value, dtype=torch.uint8, device=device)
        self.scales = torch.empty(ns.value // 2, dtype=torch.bfloat16, device=device)
        self.N, self.K, self.group = N, K, group
        self._index = _index_of(self.codes, "device")
        self._device = torch.device("cuda", self._index)
        self._call = self._lib.dg_w4_matvec
        self.s = dg_w4(self.codes.data_ptr(), self.scales.data_ptr(), N, K, group)
        self._ref = ct.byref(self.s)

    @classmethod
    def from_codes(cls, codes, scales, stream=None):
        """Lay out codes (uint8 [N, K], 0 to 15, weight s * (c - 8)) and scales (bf16 [N, K / group]) (dg_w4_pack)."""
        i = _index_of(codes, "codes")
        _on(codes, torch.uint8, "codes", i)
        _on(scales, torch.bfloat16, "scales", i)
        _need(codes.dim() == 2 and scales.dim() == 2 and scales.shape[0] == codes.shape[0] and scales.shape[1] > 0
              and codes.shape[1] % scales.shape[1] == 0, "codes [N, K], scales [N, K / group]")
        _need(codes.is_contiguous() and scales.is_contiguous(), "codes and scales: contiguous")
        st = _raw_stream(i, stream)
        with torch.cuda.stream(stream):
            w = cls(codes.shape[0], codes.shape[1], codes.shape[1] // scales.shape[1], codes.device)
        _check(w._lib.dg_w4_pack(w._ref, codes.data_ptr(), scales.data_ptr(), st), "dg_w4_pack")
        return w

    def read(self, stream=None) -> torch.Tensor:
        """The weights as float32 [N, K], exactly (dg_w4_read)."""
        st = _raw_stream(self._index, stream)
        out = _empty((self.N, self.K), torch.float32, self._device, stream)
        _check(self._lib.dg_w4_read(self._ref, out.data_ptr(), self.K, st), "dg_w4_read")
        return out


def w4_quantize(W: torch.Tensor, group: int = 64, status: torch.Tensor | None = None, stream=None) -> W4Matrix:
    """4-bit weights of a bf16 matrix [N, K] (dg_w4_quantize).

    status: optional int32 [1] device word, set to DG_ERR_VALUE where W holds infinities or NaN; without it the
    call waits for the stream and raises DgError in that case."""
    i = _index_of(W, "W")
    _on(W, torch.bfloat16, "W", i)
    _need(W.dim() == 2, "W: [N, K]")
    _, ld = _rows_of(W, torch.bfloat16, W.shape[1], "W", i)
    st = _raw_stream(i, stream)
    with torch.cuda.stream(stream):
        w = W4Matrix(W.shape[0], W.shape[1], group, W.device)
        word = torch.zeros(1, dtype=torch.int32, device=W.device) if status is None else status
    _need(_on(word, torch.int32, "status", i).shape == (1,), "status: int32 [1]")
    _check(w._lib.dg_w4_quantize(w._ref, W.data_ptr(), ld, word.data_ptr(), st), "dg_w4_quantize")
    if status is None:
        code = ct.c_int32()
        _check(w._lib.dg_read_status(word.data_ptr(), ct.byref(code), st), "dg_read_status")
        _check(code.value, "dg_w4_quantize: the matrix")
    return w


def w4_matvec(w: W4Matrix, x: torch.Tensor, alpha: torch.Tensor | None = None, coef: float = 1.0,
              resid: torch.Tensor | None = None, dtype=torch.bfloat16, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """coef * alpha[m] * (x w^T) + resid for 1 to 32 rows x (bf16 [M, K]) (dg_w4_matvec); bf16 or float32 [M, N].

    alpha: optional float32 [M]; resid: optional bf16 [M, N], which may also be `out`."""
    i, N, ap, rp, ldr = w._index, w.N, None, None, 0
    if x.dtype is _BF16 and x.get_device() == i and x.dim() == 2 and x.is_contiguous() and x.shape[1] == w.K:
        M, ldx = x.shape[0], w.K
    else:
        M, ldx = _rows_of(x, _BF16, w.K, "x", i)
    if alpha is not None:
        if alpha.dtype is not _F32 or alpha.get_device() != i or alpha.shape != (M,) or not alpha.is_contiguous():
            raise ValueError(f"alpha: contiguous float32 [{M}] on cuda:{i}")
        ap = alpha.data_ptr()
    if resid is not None:
        if resid.dtype is _BF16 and resid.get_device() == i and resid.shape == (M, N) and resid.is_contiguous():
            ldr = N
        else:
            rr, ldr = _rows_of(resid, _BF16, N, "resid", i)
            _need(rr == M, f"resid: [{M}, {N}]")
        rp = resid.data_ptr()
    st = _raw_stream(i, stream)
    if out is None:
        out, ldy = _empty((M, N), dtype, w._device, stream), N
    else:
        dtype = out.dtype
        rr, ldy = _rows_of(out, dtype, N, "out", i)
        _need(rr == M, f"out: [{M}, {N}]")
    if dtype is not _F32 and dtype is not _BF16:
        raise ValueError(f"the product is bfloat16 or float32, not {dtype}")
    rc = w._call(w._ref, x.data_ptr(), ldx, M, ap, coef, rp, ldr, out.data_ptr(), ldy, 1 if dtype is _F32 else 0, st)
    if rc:
        raise DgError(rc, "dg_w4_matvec")
    return out


def w4_status(stream=None) -> int:
    """Status word of the 4-bit products on the current device (dg_w4_status; synchronises the stream)."""
    st = ct.c_int32()
    _check(load().dg_w4_status(ct.byref(st), _stream(stream)), "dg_w4_status")
    return st.value


_qk_plans = {}  # shapes, strides and heads of qkv -> (B, C, hd, strides, output shapes)


def _qk_plan(qkv, Hq, Hkv):
    H = Hq + 2 * Hkv
    if qkv.dim() != 3 or Hq < 1 or Hkv < 1 or qkv.shape[2] % H or (qkv.shape[2] > 1 and qkv.stride(2) != 1):
        raise ValueError(f"qkv: bf16 [B, C, {H} hd] with contiguous tokens, got {tuple(qkv.shape)}")
    B, C, W = qkv.shape
    sb, sc, _ = qkv.stride()
    sc = sc if C > 1 else W
    plan = (B, C, W // H, sb if B > 1 else C * max(sc, W), sc, (B, Hq, C, W // H), (B, Hkv, C, W // H))
    if len(_qk_plans) >= 256:
        _qk_plans.clear()
    _qk_plans[(qkv.shape, qkv.stride(), Hq, Hkv)] = plan
    return plan


def _gain(t, hd, what, index):
    if t.dtype is not _BF16 or t.get_device() != index or t.shape != (hd,) or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous bf16 [{hd}] on cuda:{index}")
    return t.data_ptr()


def qk_norm_rope(qkv: torch.Tensor, pos: torch.Tensor, Hq: int, Hkv: int, q_gain: torch.Tensor | None = None,
                 k_gain: torch.Tensor | None = None, rms_eps: float = 1e-6, rope_base: float = 10000.0, out=None,
                 stream=None):
    """RMSNorm and rotation of the q and k heads of packed projections (dg_qk_norm_rope): (q, k, v).

    qkv: bf16 [B, C, (Hq + 2 Hkv) hd]; pos: int32 [B], position of each sequence's first token (e.g. cache.len);
    q_gain, k_gain: optional bf16 [hd].  q [B, Hq, C, hd], k, v [B, Hkv, C, hd], as kv8_append and kv8_attention take
    them; out: optional (q, k, v) to write."""
    plan = _qk_plans.get((qkv.shape, qkv.stride(), Hq, Hkv)) or _qk_plan(qkv, Hq, Hkv)
    B, C, hd, sb, sc, sq, sk = plan
    i = qkv.get_device()
    if i < 0 or qkv.dtype is not _BF16:
        raise ValueError(f"qkv: a bf16 CUDA tensor, got {qkv.dtype} on {qkv.device}")
    if pos.dtype is not _I32 or pos.get_device() != i or pos.shape != (B,) or not pos.is_contiguous():
        raise ValueError(f"pos: contiguous int32 [{B}] on cuda:{i}")
    qg = kg = None
    if q_gain is not None:
        qg = _gain(q_gain, hd, "q_gain", i)
    if k_gain is not None:
        kg = _gain(k_gain, hd, "k_gain", i)
    st = _raw_stream(i, stream)
    if out is None:
        dev = qkv.device
        q, k, v = _empty(sq, _BF16, dev, stream), _empty(sk, _BF16, dev, stream), _empty(sk, _BF16, dev, stream)
    else:
        q, k, v = out
        for t, s, what in ((q, sq, "q"), (k, sk, "k"), (v, sk, "v")):
            if _on(t, _BF16, what, i).shape != s or not t.is_contiguous():
                raise ValueError(f"{what}: contiguous bf16 {list(s)}")
    if B * C == 0:
        return q, k, v
    rc = (_lib or load()).dg_qk_norm_rope(qkv.data_ptr(), sb, sc, pos.data_ptr(), qg, kg, q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), B, C, Hq, Hkv, hd, rope_base, rms_eps, st)
    if rc:
        raise DgError(rc, "dg_qk_norm_rope")
    return q, k, v


# Workspaces of moe_tokens, one for each (device, stream), zeroed when made; the lock as _kv8_lock's.
_moe_workspaces = {}
_moe_lock = threading.Lock()


class MoeFfn:
    """The mixture-of-experts block of one layer for moe_tokens: router Wr [n_exp, d], expert matrices We1
    [n_exp + 1, Fe, d] and We2 [n_exp + 1, d, Fe] (index n_exp: the shared expert), bf16, contiguous."""

    def __init__(self, Wr, We1, We2, top_k, rms_eps=1e-6):
        i = self._index = _index_of(Wr, "Wr")
        _need(Wr.dim() == 2 and We1.dim() == 3, "Wr [n_exp, d], We1 [n_exp + 1, Fe, d], We2 [n_exp + 1, d, Fe]")
        n, d = Wr.shape
        Fe = We1.shape[1]
        for t, shape, what in ((Wr, (n, d), "Wr"), (We1, (n + 1, Fe, d), "We1"), (We2, (n + 1, d, Fe), "We2")):
            _need(_on(t, torch.bfloat16, what, i).shape == shape and t.is_contiguous(), f"{what}: contiguous bf16 {list(shape)}")
        self.Wr, self.We1, self.We2 = Wr, We1, We2
        self.d, self.n_exp, self.top_k, self.Fe, self.rms_eps = d, n, int(top_k), Fe, float(rms_eps)
        _i32("dg_moe_tokens", d, n, self.top_k, Fe)
        self.s = dg_model()
        self.s.dims = dg_dims(d=d, n_exp=n, top_k=self.top_k, Fe=Fe, rms_eps=self.rms_eps, L=1)
        self.s.Wr, self.s.We1, self.s.We2 = Wr.data_ptr(), We1.data_ptr(), We2.data_ptr()
        self._ref = ct.byref(self.s)
        self._lib = load()
        self._device = torch.device("cuda", i)
        self._ws_bytes = {}
        self.workspace_bytes(1)

    @classmethod
    def of(cls, model: Model, layer: int = 0):
        """The block of a layer of a Model with experts."""
        _need(model.dims.n_exp > 0 and 0 <= layer < model.dims.L, "a layer of a model with experts")
        w = [model.w[k] if model.dims.L == 1 else model.w[k][layer] for k in ("Wr", "We1", "We2")]
        return cls(*w, top_k=model.dims.top_k, rms_eps=model.dims.rms_eps)

    def workspace_bytes(self, M: int) -> int:
        """Bytes of workspace of moe_tokens with M tokens."""
        n = self._ws_bytes.get(M)
        if n is None:
            _i32("dg_moe_tokens_workspace", M)
            z = ct.c_size_t()
            _check(self._lib.dg_moe_tokens_workspace(self._ref, M, ct.byref(z)), "dg_moe_tokens_workspace")
            n = self._ws_bytes[M] = z.value
        return n


def moe_tokens(ffn: MoeFfn, h: torch.Tensor, out: torch.Tensor | None = None, routing=None, ws: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The whole mixture-of-experts block, residual included, for 1 to 32 tokens h (bf16 [M, d]) (dg_moe_tokens).

    out: optional bf16 [M, d], which may be h.  routing: optional (int32 [M, top_k], float32 [M, top_k]) to receive
    the experts and their gates.  ws: optional uint8 workspace of ffn.workspace_bytes(M) bytes, zeroed before its
    first use and not shared by calls that may overlap; by default the calls of a stream share one, which is kept
    (moe_tokens_status, moe_release_workspaces), and a captured call takes one from the graph's pool, whose status
    word nothing reads: a graph whose status matters is given a ws."""
    i, d = ffn._index, ffn.d
    M = h.shape[0] if h.dim() == 2 else 0
    if h.dtype is not _BF16 or h.get_device() != i or h.shape != (M, d) or not h.is_contiguous():
        raise ValueError(f"h: contiguous bf16 [M, {d}] on cuda:{i}, got {h.dtype} {tuple(h.shape)} on {h.device}")
    if out is not None and (_on(out, _BF16, "out", i).shape != (M, d) or not out.is_contiguous()):
        raise ValueError(f"out: contiguous bf16 [{M}, {d}], got {tuple(out.shape)}")
    ip = gp = None
    if routing is not None:
        for t, dt in zip(routing, (torch.int32, torch.float32)):
            if _on(t, dt, "routing", i).shape != (M, ffn.top_k) or not t.is_contiguous():
                raise ValueError(f"routing: contiguous int32 and float32 [{M}, {ffn.top_k}]")
        ip, gp = routing[0].data_ptr(), routing[1].data_ptr()
    st = _raw_stream(i, stream)
    wn = ffn._ws_bytes.get(M) or ffn.workspace_bytes(M)
    if out is None:
        out = _empty((M, d), _BF16, ffn._device, stream)
    call, hp, op = ffn._lib.dg_moe_tokens, h.data_ptr(), out.data_ptr()
    if ws is not None:
        _need(ws.get_device() == i and ws.is_contiguous(), "ws: contiguous, on the block's device")
        rc = call(ffn._ref, 0, hp, op, M, ip, gp, ws.data_ptr(), ws.numel() * ws.element_size(), st)
    elif _capturing(stream):
        # from the graph's own pool, zeroed by the graph, held until the launch is enqueued
        with torch.cuda.stream(stream):
            ws = torch.zeros(wn, dtype=torch.uint8, device=i)
        rc = call(ffn._ref, 0, hp, op, M, ip, gp, ws.data_ptr(), wn, st)
    else:
        with _moe_lock:
            t = _moe_workspaces.get((i, st))
            if t is None or t.numel() < wn:
                with torch.cuda.stream(stream):
                    was, t = t, torch.zeros(wn, dtype=torch.uint8, device=i)
                    if was is not None:
                        t[:4].copy_(was[:4])  # the status word goes along
                _moe_workspaces[i, st] = t
            rc = call(ffn._ref, 0, hp, op, M, ip, gp, t.data_ptr(), wn, st)
    if rc:
        raise DgError(rc, "dg_moe_tokens")
    return out


def moe_tokens_status(device=None, stream=None) -> int:
    """The status word of the workspace that moe_tokens keeps for the stream (synchronises it): DG_OK, or what its
    calls have met since moe_release_workspaces.  After DG_ERR_TIMEOUT the workspace is let go of, and the next call
    takes a new one."""
    i = torch.cuda.current_device() if device is None else torch.device(device).index
    key = (i, _raw_stream(i, stream))
    with _moe_lock:
        t = _moe_workspaces.get(key)
    if t is None:
        return DG_OK
    code = ct.c_int32()
    _check(load().dg_read_status(t.data_ptr(), ct.byref(code), key[1]), "dg_read_status")
    if code.value == DG_ERR_TIMEOUT:
        with _moe_lock:
            if _moe_workspaces.get(key) is t:
                del _moe_workspaces[key]
    return code.value


def moe_release_workspaces(device=None) -> None:
    """Let go of the workspaces that moe_tokens keeps, as kv8_release_workspaces does of its own."""
    index = None if device is None else torch.device(device).index
    if device is not None and index is None:
        index = torch.cuda.current_device()
    with _moe_lock:
        for key in [k for k in _moe_workspaces if index is None or k[0] == index]:
            del _moe_workspaces[key]


def _setting(t, dtype, R, what, index):
    if t.dtype is not dtype or t.get_device() != index or t.shape != (R,) or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous {dtype} [{R}] on cuda:{index}, or a number")
    return t.data_ptr()


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, stream=None):
    """A token for each row of logits (float32 or bf16 [R, V]) by the random numbers u (float32 [R], in [0, 1)), with
    temperature, top-k, top-p and min-p (dg_sample): (token int32, logprob float32, kept int32), each [R].

    The settings are numbers, or tensors [R] with one for each row (float32; top_k int32): 0 / 0 / 1 / 0 are greedy and
    no cut.  A row that cannot be drawn from (NaN, +inf, no finite logit, a setting or u outside its range) gets token
    -1.  out: optional (token, logprob, kept) to write."""
    i = logits.get_device()
    dt = logits.dtype
    if i < 0 or (dt is not _F32 and dt is not _BF16) or logits.dim() != 2:
        raise ValueError(f"logits: float32 or bfloat16 [R, V] on a CUDA device, got {dt} {tuple(logits.shape)} on {logits.device}")
    R, V = logits.shape
    if (R | V) >> 31:
        _i32("dg_sample", R, V)
    ld = V if logits.is_contiguous() else _rows_of(logits, dt, V, "logits", i)[1]
    if u.dtype is not _F32 or u.get_device() != i or u.shape != (R,) or not u.is_contiguous():
        raise ValueError(f"u: contiguous float32 [{R}] on cuda:{i}")
    how = dg_sampling()
    if isinstance(temperature, torch.Tensor):
        how.temperature = _setting(temperature, _F32, R, "temperature", i)
    else:
        how.temperature_all = temperature
    if isinstance(top_p, torch.Tensor):
        how.top_p = _setting(top_p, _F32, R, "top_p", i)
    else:
        how.top_p_all = top_p
    if isinstance(min_p, torch.Tensor):
        how.min_p = _setting(min_p, _F32, R, "min_p", i)
    else:
        how.min_p_all = min_p
    if isinstance(top_k, torch.Tensor):
        how.top_k = _setting(top_k, _I32, R, "top_k", i)
    else:
        how.top_k_all = max(-1, min(top_k, V))  # (V and more keep all; 32 bits go to the library)
    st = _raw_stream(i, stream)
    if out is None:
        dev, shape = logits.device, (R,)
        out = (_empty(shape, _I32, dev, stream), _empty(shape, _F32, dev, stream), _empty(shape, _I32, dev, stream))
    else:
        for t, want, what in zip(out, (_I32, _F32, _I32), ("token", "logprob", "kept")):
            if _on(t, want, what, i).shape != (R,) or not t.is_contiguous():
                raise ValueError(f"{what}: contiguous {want} [{R}]")
    if R == 0:
        return out
    rc = (_lib or load()).dg_sample(logits.data_ptr(), 1 if dt is _BF16 else 0, ld, R, V, ct.byref(how), u.data_ptr(),
                                    out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), st)
    if rc:
        raise DgError(rc, "dg_sample")
    return out
