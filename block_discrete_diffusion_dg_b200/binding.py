"""Thin ctypes binding of ``libdg.so`` (the C ABI in include/dg.h).

Argument marshalling only: every step of the computation runs in the library's CUDA kernels.
Functions carry the C names; tensors are passed as torch tensors (device memory) and turned into
raw pointers; a non-zero status raises :class:`DgError`.  There is no fallback: if the shared
library is missing, :func:`lib` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_UNSUPPORTED, DG_ERR_CAPACITY, DG_ERR_CUDA, \
    DG_ERR_NUMERIC, DG_ERR_TIMEOUT, DG_ERR_WORKSPACE = range(8)
DG_F32, DG_BF16, DG_E4M3, DG_NVFP4 = 0, 1, 2, 3
DG_ROPE_HALF, DG_ROPE_INTERLEAVED = 0, 1
DG_ROPE_UNSCALED, DG_ROPE_LINEAR, DG_ROPE_BY_PARTS = 0, 1, 2
STATUS_NAMES = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED", 3: "DG_ERR_CAPACITY",
                4: "DG_ERR_CUDA", 5: "DG_ERR_NUMERIC", 6: "DG_ERR_TIMEOUT", 7: "DG_ERR_WORKSPACE"}


class DgError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}"
                         + (f" ({_lib.dg_last_cuda_error().decode()})" if code == DG_ERR_CUDA and _lib else ""))
        self.code = code


class DgConfig(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("canvas", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("rope_theta", ctypes.c_double), ("rms_eps", ctypes.c_double),
                ("act_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("emb_dtype", ctypes.c_int32), ("n_shared", ctypes.c_int32)]


class DgLayerWeights(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("s_qkv", ctypes.c_void_p),
                ("w_o", ctypes.c_void_p), ("s_o", ctypes.c_void_p),
                ("w_router", ctypes.c_void_p),
                ("w_gate_up", ctypes.c_void_p), ("s_gate_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


class DgModel(ctypes.Structure):
    _fields_ = [("layers", ctypes.POINTER(DgLayerWeights)), ("emb", ctypes.c_void_p),
                ("emb_scale", ctypes.c_void_p), ("emb_scale_global", ctypes.c_float)]


class DgSampler(ctypes.Structure):
    """dg_sampler: temperature schedule (tau_start at step 0 .. tau_end at the last step of the
    budget; <= 0 greedy), the generator's 64-bit seed, and revisable drafts (noise canvas)."""
    _fields_ = [("tau_start", ctypes.c_double), ("tau_end", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("revise", ctypes.c_int32)]


def make_sampler(tau_start=0.0, tau_end=None, seed=0, revise=False) -> DgSampler:
    return DgSampler(float(tau_start), float(tau_start if tau_end is None else tau_end),
                     int(seed) & 0xFFFFFFFFFFFFFFFF, 1 if revise else 0)


class DgRope(ctypes.Structure):
    """dg_rope: rotated part of a head, pair layout and frequency scaling."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("mscale", ctypes.c_double)]


def make_rope(rot_dim, layout=DG_ROPE_HALF, scaling=DG_ROPE_UNSCALED, factor=1.0, orig_len=0.0,
              beta_slow=1.0, beta_fast=32.0, mscale=1.0) -> DgRope:
    return DgRope(int(rot_dim), int(layout), int(scaling), float(factor), float(orig_len),
                  float(beta_slow), float(beta_fast), float(mscale))


class DgPagedKv(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None
_VP, _I32, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_PCFG, _PMODEL, _PLW = ctypes.POINTER(DgConfig), ctypes.POINTER(DgModel), ctypes.POINTER(DgLayerWeights)
_PSMP = ctypes.POINTER(DgSampler)
_PROPE, _PKV = ctypes.POINTER(DgRope), ctypes.POINTER(DgPagedKv)

_SIGS = {
    "dg_workspace_size": (_SZ, [_PCFG, _I32, _I32, _I32]),
    "dg_read_status": (_I32, [_VP, _VP]),
    "dg_clear_status": (_I32, [_VP, _VP]),
    "dg_last_cuda_error": (ctypes.c_char_p, []),
    "dg_launch_count": (ctypes.c_uint64, []),
    "dg_profile_begin": (_I32, [_I32]),
    "dg_profile_mark": (_I32, [_VP]),
    "dg_profile_end": (_I32, [ctypes.POINTER(ctypes.c_float), _I32, ctypes.POINTER(ctypes.c_int)]),
    "dg_profile_name": (ctypes.c_char_p, [_I32]),
    "dg_canvas_attn": (_I32, [_PCFG, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _VP,
                              _VP, _VP, _SZ, _VP, _VP]),
    "dg_moe_route": (_I32, [_PCFG, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dg_moe_ffn": (_I32, [_PCFG, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _PLW, _VP, _VP, _VP, _SZ, _VP,
                          _VP]),
    "dg_logits_entropy": (_I32, [_PCFG, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dg_logits_entropy_static": (_I32, [_PCFG, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "dg_logits_entropy_nvfp4": (_I32, [_PCFG, _I32, _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP,
                                       _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dg_eb_select": (_I32, [_I32, _I32, _VP, _VP, ctypes.c_double, _I32, _VP, _VP, _VP, _VP, _VP,
                            _VP, _I32, _VP, _VP]),
    "dg_kv_append": (_I32, [_PCFG, _PMODEL, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _SZ,
                            _VP, _VP]),
    "dg_canvas_step": (_I32, [_PCFG, _PMODEL, _I32, _VP, _VP, _VP, _VP, _VP, _I32, ctypes.c_double,
                              _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dg_generate": (_I32, [_PCFG, _PMODEL, _I32, _VP, _VP, _VP, _VP, _VP, _I32, ctypes.c_double,
                           _PSMP, _VP, _VP, _VP, _I32, _I32, _VP, _SZ, _VP, _VP]),
    "dg_canvas_step_sampler": (_I32, [_PCFG, _PMODEL, _I32, _VP, _VP, _VP, _VP, _VP, _I32,
                                      ctypes.c_double, _PSMP, _VP, _VP, _VP, _I32, _VP, _VP, _VP,
                                      _VP, _VP, _SZ, _VP, _VP]),
    "dg_debug_wait_probe": (_I32, [ctypes.c_longlong, _I32, _VP, _VP]),
    "dg_noise_canvas": (_I32, [_I32, _I32, _I32, ctypes.c_uint64, _VP, _VP, _VP, _VP, _VP, _VP]),
    "dg_qk_norm_rope": (_I32, [_PCFG, _I32, _I32, _VP, ctypes.c_longlong, _VP, _VP, _VP, _PROPE, _VP,
                               _VP, _VP, _VP, _VP]),
    "dg_paged_append": (_I32, [_PCFG, _I32, _I32, _VP, _VP, _VP, ctypes.c_longlong, _VP, _VP, _PROPE,
                               _PKV, _VP, _VP, _VP]),
    "dg_paged_workspace_size": (_SZ, [_PCFG, _I32, _I32, _I32]),
    "dg_paged_attn": (_I32, [_PCFG, _I32, _I32, _VP, _VP, _VP, _PKV, _I32, _VP, _VP, _SZ, _VP, _VP]),
    "dg_prefix_attn": (_I32, [_PCFG, _I32, _I32, _VP, _VP, _I32, _VP, _PKV, _I32, _VP, _VP, _SZ, _VP,
                              _VP]),
    "dg_ar_step": (_I32, [_PCFG, _PMODEL, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _PSMP, _VP, _VP,
                          _VP, _VP, _VP, _SZ, _VP, _VP]),
}


def lib() -> ctypes.CDLL:
    """Load libdg.so (build it with ``python -m block_discrete_diffusion_dg_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; the CUDA library has not been built")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the library takes device tensors")
    if not t.is_contiguous():
        raise ValueError("the library takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, what: str):
    if rc != DG_OK:
        raise DgError(rc, what)


# ----------------------------------------------------------------------------- structures

def make_config(c) -> DgConfig:
    """dg_config from a workload description (``synth.Cfg`` or any object with the fields)."""
    act = DG_F32 if c.act == "f32" else DG_BF16
    emb = DG_NVFP4 if getattr(c, "emb", "") == "nvfp4" else act
    return DgConfig(c.d_model, c.n_q_heads, c.n_kv_heads, c.head_dim, c.n_experts, c.top_k, c.d_ff,
                    c.vocab, c.canvas, c.n_layers, float(c.rope_theta), float(c.rms_eps), act,
                    {"f32": DG_F32, "bf16": DG_BF16, "e4m3": DG_E4M3}[c.w], emb,
                    int(getattr(c, "n_shared", 0)))


def make_layer(lay: dict) -> DgLayerWeights:
    g = lambda k: _p(lay.get(k)) if lay.get(k) is not None else None  # noqa: E731
    return DgLayerWeights(g("w_qkv"), g("s_qkv"), g("w_o"), g("s_o"), g("w_router"),
                          g("w_gate_up"), g("s_gate_up"), g("w_down"), g("s_down"))


class Model:
    """Host-side dg_model over device weight tensors (keeps the ctypes arrays alive)."""

    def __init__(self, model: dict):
        self.tensors = model
        n = len(model["layers"])
        self.layer_array = (DgLayerWeights * n)(*[make_layer(l) for l in model["layers"]])
        sc = model.get("emb_scale")
        self.struct = DgModel(ctypes.cast(self.layer_array, ctypes.POINTER(DgLayerWeights)),
                              _p(model["emb"]), _p(sc) if sc is not None else None,
                              float(model.get("emb_scale_global", 1.0)))

    def layer(self, l: int) -> DgLayerWeights:
        return self.layer_array[l]


# ----------------------------------------------------------------------------- entry points

def dg_workspace_size(cfg: DgConfig, batch: int, n_tokens: int, cache_cap: int) -> int:
    return lib().dg_workspace_size(ctypes.byref(cfg), batch, n_tokens, cache_cap)


def _on(device):
    """Makes `device` current where it names one: the sizes of workspaces are those of the current device."""
    d = torch.device(device)
    return torch.cuda.device(d) if d.type == "cuda" and d.index is not None else contextlib.nullcontext()


def alloc_workspace(cfg: DgConfig, batch: int, n_tokens: int, cache_cap: int, device="cuda"):
    with _on(device):
        n = dg_workspace_size(cfg, batch, n_tokens, cache_cap)
    if n == 0:
        raise DgError(DG_ERR_INVALID_ARG, "dg_workspace_size")
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def _ws(ws: torch.Tensor):
    base = ws.data_ptr()
    aligned = (base + 255) & ~255
    return aligned, ws.numel() - (aligned - base)


def dg_read_status(dev_status: torch.Tensor, stream=None) -> int:
    return lib().dg_read_status(_p(dev_status), _stream(stream))


def dg_clear_status(dev_status: torch.Tensor, stream=None):
    _check(lib().dg_clear_status(_p(dev_status), _stream(stream)), "dg_clear_status")


def dg_launch_count() -> int:
    return int(lib().dg_launch_count())


def dg_profile_begin(max_records: int):
    _check(lib().dg_profile_begin(max_records), "dg_profile_begin")


def dg_profile_mark(stream=None):
    _check(lib().dg_profile_mark(_stream(stream)), "dg_profile_mark")


def dg_profile_end(max_out: int = 1 << 16):
    """Returns [(kernel name, ms)] for each recorded launch (the time to the next record)."""
    buf = (ctypes.c_float * max_out)()
    n = ctypes.c_int(0)
    _check(lib().dg_profile_end(buf, max_out, ctypes.byref(n)), "dg_profile_end")
    return [(lib().dg_profile_name(i).decode(), float(buf[i])) for i in range(n.value)]


def dg_canvas_attn(cfg, batch, n_tokens, q, k_cache, v_cache, cache_len, cache_cap, k_new, v_new,
                   causal, done, out, ws, dev_status=None, stream=None):
    w, wb = _ws(ws)
    _check(lib().dg_canvas_attn(ctypes.byref(cfg), batch, n_tokens, _p(q), _p(k_cache), _p(v_cache),
                                _p(cache_len), cache_cap, _p(k_new), _p(v_new), int(causal),
                                _p(done), _p(out), w, wb, _p(dev_status), _stream(stream)),
           "dg_canvas_attn")


def dg_moe_route(cfg, n_tokens, y, w_router, token_live, topk_idx, topk_w, expert_off, perm,
                 inv_perm, ws, dev_status=None, stream=None):
    w, wb = _ws(ws)
    _check(lib().dg_moe_route(ctypes.byref(cfg), n_tokens, _p(y), _p(w_router), _p(token_live),
                              _p(topk_idx), _p(topk_w), _p(expert_off), _p(perm), _p(inv_perm),
                              w, wb, _p(dev_status), _stream(stream)), "dg_moe_route")


def dg_moe_ffn(cfg, n_tokens, y, topk_idx, topk_w, expert_off, perm, inv_perm, layer, residual,
               out, ws, dev_status=None, stream=None):
    w, wb = _ws(ws)
    _check(lib().dg_moe_ffn(ctypes.byref(cfg), n_tokens, _p(y), _p(topk_idx), _p(topk_w),
                            _p(expert_off), _p(perm), _p(inv_perm), ctypes.byref(layer),
                            _p(residual), _p(out), w, wb, _p(dev_status), _stream(stream)),
           "dg_moe_ffn")


def dg_logits_entropy(cfg, n_rows, n_rows_dev, h, row_idx, w_lm, entropy, argmax, logits_dbg, ws,
                      dev_status=None, stream=None):
    w, wb = _ws(ws)
    _check(lib().dg_logits_entropy(ctypes.byref(cfg), n_rows, _p(n_rows_dev), _p(h), _p(row_idx),
                                   _p(w_lm), _p(entropy), _p(argmax), _p(logits_dbg), w, wb,
                                   _p(dev_status), _stream(stream)), "dg_logits_entropy")


def dg_logits_entropy_static(cfg, n_rows, n_rows_dev, h, row_idx, w_lm, entropy, argmax,
                             dev_status=None, stream=None):
    """dg_logits_entropy without a scratch argument (its scratch is a fixed array in the library)."""
    _check(lib().dg_logits_entropy_static(ctypes.byref(cfg), n_rows, _p(n_rows_dev), _p(h),
                                          _p(row_idx), _p(w_lm), _p(entropy), _p(argmax),
                                          _p(dev_status), _stream(stream)),
           "dg_logits_entropy_static")


def dg_logits_entropy_nvfp4(cfg, n_rows, n_rows_dev, h, row_idx, w_codes, w_scale, w_scale_global,
                            entropy, argmax, logits_dbg, ws, dev_status=None, stream=None):
    """dg_logits_entropy with the LM head in NVFP4: uint8 codes [d/64][Vp][32], uint8 E4M3
    scales [d/64][Vp][4] and the fp32 tensor scale (cfg.emb_dtype must be DG_NVFP4)."""
    w, wb = _ws(ws)
    _check(lib().dg_logits_entropy_nvfp4(ctypes.byref(cfg), n_rows, _p(n_rows_dev), _p(h),
                                         _p(row_idx), _p(w_codes), _p(w_scale),
                                         float(w_scale_global), _p(entropy), _p(argmax),
                                         _p(logits_dbg), w, wb, _p(dev_status), _stream(stream)),
           "dg_logits_entropy_nvfp4")


def dg_eb_select(batch, canvas, entropy, argmax, gamma, max_steps, tokens, masked, selected,
                 n_masked, done, step, dev_status=None, stream=None, revise=False):
    _check(lib().dg_eb_select(batch, canvas, _p(entropy), _p(argmax), float(gamma), max_steps,
                              _p(tokens), _p(masked), _p(selected), _p(n_masked), _p(done), _p(step),
                              1 if revise else 0, _p(dev_status), _stream(stream)), "dg_eb_select")


def dg_kv_append(cfg, model: Model, batch, tokens, n_tokens, k_cache, v_cache, cache_len, cache_cap,
                 ws, dev_status=None, stream=None, forced_topk=None):
    w, wb = _ws(ws)
    _check(lib().dg_kv_append(ctypes.byref(cfg), ctypes.byref(model.struct), batch, _p(tokens),
                              n_tokens, _p(k_cache), _p(v_cache), _p(cache_len), cache_cap,
                              _p(forced_topk), w, wb, _p(dev_status), _stream(stream)),
           "dg_kv_append")


def dg_canvas_step(cfg, model: Model, batch, tokens, masked, n_masked, done, step, max_steps, gamma,
                   k_cache, v_cache, cache_len, cache_cap, entropy_out, argmax_out, logits_dbg, ws,
                   dev_status=None, stream=None, expert_load=None, forced_topk=None):
    w, wb = _ws(ws)
    _check(lib().dg_canvas_step(ctypes.byref(cfg), ctypes.byref(model.struct), batch, _p(tokens),
                                _p(masked), _p(n_masked), _p(done), _p(step), max_steps,
                                float(gamma), _p(k_cache), _p(v_cache), _p(cache_len), cache_cap,
                                _p(entropy_out), _p(argmax_out), _p(logits_dbg), _p(expert_load),
                                _p(forced_topk), w, wb, _p(dev_status), _stream(stream)),
           "dg_canvas_step")


def dg_generate(cfg, model: Model, batch, tokens, masked, n_masked, done, step, max_steps, gamma,
                k_cache, v_cache, cache_len, cache_cap, append, ws, dev_status=None, stream=None,
                sampler: Optional[DgSampler] = None):
    """The step loop on the device until every canvas is done (one CUDA graph with a
    conditional while node, cached per argument set), then the append if `append`."""
    w, wb = _ws(ws)
    _check(lib().dg_generate(ctypes.byref(cfg), ctypes.byref(model.struct), batch, _p(tokens),
                             _p(masked), _p(n_masked), _p(done), _p(step), max_steps, float(gamma),
                             None if sampler is None else ctypes.byref(sampler),
                             _p(k_cache), _p(v_cache), _p(cache_len), cache_cap, int(append), w, wb,
                             _p(dev_status), _stream(stream)),
           "dg_generate")


def dg_canvas_step_sampler(cfg, model: Model, batch, tokens, masked, n_masked, done, step,
                           max_steps, gamma, sampler: DgSampler, k_cache, v_cache, cache_len,
                           cache_cap, entropy_out, argmax_out, logits_dbg, ws, dev_status=None,
                           stream=None, forced_topk=None):
    """dg_canvas_step with a sampler variant (temperature-annealed draws, revisable drafts)."""
    w, wb = _ws(ws)
    _check(lib().dg_canvas_step_sampler(ctypes.byref(cfg), ctypes.byref(model.struct), batch,
                                        _p(tokens), _p(masked), _p(n_masked), _p(done), _p(step),
                                        max_steps, float(gamma), ctypes.byref(sampler),
                                        _p(k_cache), _p(v_cache), _p(cache_len), cache_cap,
                                        _p(entropy_out), _p(argmax_out), _p(logits_dbg),
                                        _p(forced_topk), w, wb, _p(dev_status), _stream(stream)),
           "dg_canvas_step_sampler")


def dg_noise_canvas(batch, canvas, vocab, seed, tokens, masked, n_masked, done, step, stream=None):
    """Uniform-noise canvases (every position a revisable draft)."""
    _check(lib().dg_noise_canvas(batch, canvas, vocab, int(seed) & 0xFFFFFFFFFFFFFFFF, _p(tokens),
                                 _p(masked), _p(n_masked), _p(done), _p(step), _stream(stream)),
           "dg_noise_canvas")


def dg_ar_step(cfg, model: Model, batch, tokens, n_tokens, k_cache, v_cache, cache_len, cache_cap,
               next_token, entropy, logits_dbg, ws, dev_status=None, stream=None,
               sampler: Optional[DgSampler] = None, forced_topk=None):
    """Autoregressive mode: append the tokens, predict each sequence's next token."""
    w, wb = _ws(ws)
    _check(lib().dg_ar_step(ctypes.byref(cfg), ctypes.byref(model.struct), batch, _p(tokens),
                            n_tokens, _p(k_cache), _p(v_cache), _p(cache_len), cache_cap,
                            None if sampler is None else ctypes.byref(sampler), _p(next_token),
                            _p(entropy), _p(logits_dbg), _p(forced_topk), w, wb, _p(dev_status),
                            _stream(stream)),
           "dg_ar_step")


# ----------------------------------------------------------------------------- paged cache

class PagedKV:
    """Host-side dg_paged_kv over one layer's pages: k_pages, v_pages [n_pages][Hkv][page][hd] and
    the int32 page table [n_seqs][max_pages] (keeps the tensors alive)."""

    def __init__(self, k_pages, v_pages, page_table):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages are alike, [n_pages][Hkv][page][hd]")
        if page_table.dim() != 2 or page_table.dtype != torch.int32:
            raise ValueError("the page table is int32 [n_seqs][max_pages]")
        if not k_pages.device == v_pages.device == page_table.device:
            raise ValueError("pages and page table on different devices")
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.act, self.kv_heads, self.head_dim = k_pages.dtype, k_pages.shape[1], k_pages.shape[3]
        self.seqs, self.dev = page_table.shape[0], k_pages.get_device()
        self.struct = DgPagedKv(_p(k_pages), _p(v_pages), _p(page_table), k_pages.shape[0],
                                k_pages.shape[2], page_table.shape[1])
        self.ref = ctypes.byref(self.struct)


_ACT = {DG_F32: torch.float32, DG_BF16: torch.bfloat16}


# A call for a few rows takes the device less time than the host, so the checks are one expression
# each and say what was wrong only on the way out (with a call per property, and the config's fields
# read by each, dg_qk_norm_rope took 9.7 us of host time; now 8.7).
def _misfit(t, name, want, dev):
    here = t.get_device()
    if here < 0 or not t.is_contiguous():
        raise ValueError(f"{name}: the library takes contiguous device tensors")
    if dev is not None and here != dev:
        raise ValueError(f"{name}: on device {here}, the call's rows are on {dev}")
    raise ValueError(f"{name}: {want} wanted, {t.dtype} {tuple(t.shape)} given")


def _rows(t, name, dtype, shape, dev=None):
    """Pointer of a contiguous tensor of this type on device `dev` (None: on any) that holds exactly
    `shape`."""
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or
            (t.get_device() != dev and (dev is not None or not t.is_cuda))):
        _misfit(t, name, f"{dtype} {shape}", dev)
    return t.data_ptr()


def _index(t, name, n, dev=None):
    if (t.dtype is not torch.int32 or t.ndim != 1 or t.numel() < n or not t.is_contiguous() or
            (t.get_device() != dev and (dev is not None or not t.is_cuda))):
        _misfit(t, name, f"int32 of at least {n}", dev)
    return t.data_ptr()


def _heads(cfg):
    """Activation type, query heads, kv heads and head size of a config."""
    return _ACT[cfg.act_dtype], cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim


def _qkv_rows(cfg, qkv, rows, heads=None):
    """Pointer, row stride and device of projected rows [rows][(Hq + 2 Hkv) hd]; the rows may lie
    apart."""
    act, hq, hkv, hd = heads or _heads(cfg)
    width, dev = (hq + 2 * hkv) * hd, qkv.get_device()
    if qkv.dtype is not act or qkv.shape != (rows, width):
        raise ValueError(f"qkv: {act} {(rows, width)} wanted, {qkv.dtype} {tuple(qkv.shape)} given")
    ld, step = qkv.stride()
    if dev < 0 or step != 1:
        raise ValueError("qkv: device rows of contiguous elements wanted")
    return qkv.data_ptr(), (ld if rows > 1 else width), dev


def _gain(g, name, hd, dev):
    return None if g is None else _rows(g, name, torch.float32, (hd,), dev)


def _pages(kv: PagedKV, heads, n_seqs, dev):
    act, _, hkv, hd = heads
    if kv.act is not act or kv.kv_heads != hkv or kv.head_dim != hd:
        raise ValueError("the pages do not fit the config")
    if kv.seqs < n_seqs:
        raise ValueError("the page table has fewer rows than there are sequences")
    if kv.dev != dev:
        raise ValueError(f"pages on device {kv.dev}, the call's rows are on {dev}")
    return kv.ref


def _status(t, dev):
    return None if t is None else _index(t, "dev_status", 1, dev)


def _scratch(ws, dev):
    if ws.get_device() != dev or not ws.is_contiguous():
        _misfit(ws, "ws", "workspace", dev)
    return _ws(ws)


# The two lookups of a launch without the Python layers above them (4 us of a 14 us call).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(name, dev, stream, *args):
    """The library's `name`(*args, stream) on the tensors' device, which need not be the current
    one; stream None: that device's current stream."""
    fn = getattr(_lib or lib(), name)
    s = _raw_stream(dev) if stream is None else _stream(stream)
    if dev == _current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != DG_OK:
        raise DgError(rc, name)


def dg_qk_norm_rope(cfg, batch, n_tokens, qkv, cache_len, q_gain, k_gain, rope: Optional[DgRope], q,
                    k_new, v_new, dev_status=None, stream=None):
    """Per-head norms, rotation and head split of projected rows (ready for dg_canvas_attn)."""
    heads = act, hq, hkv, hd = _heads(cfg)
    ptr, ld, dev = _qkv_rows(cfg, qkv, batch * n_tokens, heads)
    _launch("dg_qk_norm_rope", dev, stream, ctypes.byref(cfg), batch, n_tokens, ptr, ld,
            _index(cache_len, "cache_len", batch, dev), _gain(q_gain, "q_gain", hd, dev),
            _gain(k_gain, "k_gain", hd, dev), None if rope is None else ctypes.byref(rope),
            _rows(q, "q", act, (batch, n_tokens, hq, hd), dev),
            _rows(k_new, "k_new", act, (batch, hkv, n_tokens, hd), dev),
            _rows(v_new, "v_new", act, (batch, hkv, n_tokens, hd), dev), _status(dev_status, dev))


def dg_paged_append(cfg, n_seqs, n_tokens, seq_off, kv_len, qkv, q_gain, k_gain,
                    rope: Optional[DgRope], kv: PagedKV, q, dev_status=None, stream=None):
    """Per-head norms and rotation of packed rows; q packed, K and V into their pages."""
    heads = act, hq, _, hd = _heads(cfg)
    ptr, ld, dev = _qkv_rows(cfg, qkv, n_tokens, heads)
    _launch("dg_paged_append", dev, stream, ctypes.byref(cfg), n_seqs, n_tokens,
            _index(seq_off, "seq_off", n_seqs + 1, dev), _index(kv_len, "kv_len", n_seqs, dev), ptr,
            ld, _gain(q_gain, "q_gain", hd, dev), _gain(k_gain, "k_gain", hd, dev),
            None if rope is None else ctypes.byref(rope), _pages(kv, heads, n_seqs, dev),
            None if q is None else _rows(q, "q", act, (n_tokens, hq, hd), dev),
            _status(dev_status, dev))


def dg_paged_workspace_size(cfg, n_seqs, n_tokens, shared_len=0) -> int:
    return lib().dg_paged_workspace_size(ctypes.byref(cfg), n_seqs, n_tokens, shared_len)


def alloc_paged_workspace(cfg, n_seqs, n_tokens, shared_len=0, device="cuda"):
    with _on(device):
        n = dg_paged_workspace_size(cfg, n_seqs, n_tokens, shared_len)
    if n == 0:
        raise DgError(DG_ERR_INVALID_ARG, "dg_paged_workspace_size")
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def dg_paged_attn(cfg, n_seqs, n_tokens, seq_off, kv_len, q, kv: PagedKV, causal, out, ws,
                  dev_status=None, stream=None):
    """Attention of packed sequences over their pages (the new K and V already appended)."""
    dev = q.get_device()
    w, wb = _scratch(ws, dev)
    heads = act, hq, _, hd = _heads(cfg)
    _launch("dg_paged_attn", dev, stream, ctypes.byref(cfg), n_seqs, n_tokens,
            _index(seq_off, "seq_off", n_seqs + 1, dev), _index(kv_len, "kv_len", n_seqs, dev),
            _rows(q, "q", act, (n_tokens, hq, hd)), _pages(kv, heads, n_seqs, dev), 1 if causal else 0,
            _rows(out, "out", act, (n_tokens, hq, hd), dev), w, wb, _status(dev_status, dev))


def dg_prefix_attn(cfg, n_seqs, n_tokens, seq_off, kv_len, shared_len, q, kv: PagedKV, causal, out,
                   ws, dev_status=None, stream=None):
    """dg_paged_attn where the first shared_len keys are common to all sequences, read once for up to
    256 / (Hq / Hkv) packed rows: for next tokens and other sequences of few rows."""
    dev = q.get_device()
    w, wb = _scratch(ws, dev)
    heads = act, hq, _, hd = _heads(cfg)
    _launch("dg_prefix_attn", dev, stream, ctypes.byref(cfg), n_seqs, n_tokens,
            _index(seq_off, "seq_off", n_seqs + 1, dev), _index(kv_len, "kv_len", n_seqs, dev),
            shared_len, _rows(q, "q", act, (n_tokens, hq, hd)), _pages(kv, heads, n_seqs, dev),
            1 if causal else 0, _rows(out, "out", act, (n_tokens, hq, hd), dev), w, wb,
            _status(dev_status, dev))


def dg_debug_wait_probe(limit_cycles, arrive, dev_status, stream=None):
    """Run the bounded device wait alone (see dg.h); expiry records DG_ERR_TIMEOUT."""
    _check(lib().dg_debug_wait_probe(int(limit_cycles), 1 if arrive else 0, _p(dev_status),
                                     _stream(stream)), "dg_debug_wait_probe")


def exported_symbols() -> Sequence[str]:
    return list(_SIGS)
