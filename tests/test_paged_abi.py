"""Refusals of the paged-cache calls that need no GPU: bad arguments return an error before any
launch, and the binding refuses tensors that do not fit."""
import ctypes
import math

import pytest
import torch

import synth
from block_discrete_diffusion_dg_b200 import binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_discrete_diffusion_dg_b200 import build
    build.build()


def _cfg(**kw):
    c = B.make_config(synth.reduced("layer"))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


PAGES = dict(k_pages=256, v_pages=256, page_table=256, n_pages=8, page_size=64, max_pages=4)


def _kv(**kw):
    return B.DgPagedKv(**{**PAGES, **kw})


def _call(name, cfg, args):
    return getattr(B.lib(), name)(ctypes.byref(cfg), *args)


BAD_PAGES = [dict(page_size=48), dict(page_size=8), dict(page_size=2048), dict(n_pages=0),
             dict(max_pages=0), dict(k_pages=None), dict(v_pages=264), dict(page_table=None),
             dict(n_pages=1 << 24), dict(max_pages=1 << 26)]


def _attn_args(kv):
    # n_seqs, n_tokens, seq_off, kv_len, q, kv, causal, out, ws, ws_bytes, status, stream
    return [2, 5, 256, 256, 256, ctypes.byref(kv), 1, 256, 256, 1 << 30, None, None]


def _append_args(kv, rope):
    # n_seqs, n_tokens, seq_off, kv_len, qkv, ld, q_gain, k_gain, rope, kv, q, status, stream
    return [2, 5, 256, 256, 256, 4096, None, None, ctypes.byref(rope), ctypes.byref(kv), 256, None,
            None]


def _norm_args(rope):
    # batch, n_tokens, qkv, ld, cache_len, q_gain, k_gain, rope, q, k, v, status, stream
    return [2, 5, 256, 4096, 256, None, None, ctypes.byref(rope), 256, 256, 256, None, None]


def test_attention_refusals():
    n0 = B.dg_launch_count()
    cfg, kv = _cfg(), _kv()
    for i, v in ((0, 0), (1, 0), (1, 1 << 30), (2, None), (3, None), (4, None), (4, 264), (5, None),
                 (7, None), (7, 264), (8, None), (8, 384)):
        a = _attn_args(kv)
        a[i] = v
        assert _call("dg_paged_attn", cfg, a) == B.DG_ERR_INVALID_ARG, (i, v)
    for bad in BAD_PAGES:
        assert _call("dg_paged_attn", cfg, _attn_args(_kv(**bad))) == B.DG_ERR_INVALID_ARG, bad
    a = _attn_args(kv)
    a[9] = 1024
    assert _call("dg_paged_attn", cfg, a) == B.DG_ERR_WORKSPACE
    assert _call("dg_paged_attn", _cfg(head_dim=96), _attn_args(kv)) == B.DG_ERR_INVALID_ARG
    wide = _cfg(n_q_heads=65, n_kv_heads=1)
    assert _call("dg_paged_attn", wide, _attn_args(kv)) == B.DG_ERR_UNSUPPORTED
    assert B.dg_paged_workspace_size(wide, 2, 5) == 0
    # more steps of work than the split's 32-bit costs hold
    a = _attn_args(_kv(max_pages=1 << 20, page_size=1024))
    a[0] = a[1] = 64
    assert _call("dg_paged_attn", cfg, a) == B.DG_ERR_UNSUPPORTED
    # shared prefix: positive, whole pages, within the page table
    for shared in (0, -64, 32, 320):
        a = _attn_args(kv)
        a.insert(4, shared)
        assert _call("dg_prefix_attn", cfg, a) == B.DG_ERR_INVALID_ARG, shared
    assert B.dg_launch_count() == n0


def test_append_and_norm_refusals():
    n0 = B.dg_launch_count()
    cfg, kv, rope = _cfg(), _kv(), B.make_rope(128)
    for i, v in ((0, 0), (1, 0), (2, None), (3, None), (4, None), (4, 264), (5, 4088), (5, 4100),
                 (6, 264), (7, 264), (9, None), (10, 264)):
        a = _append_args(kv, rope)
        a[i] = v
        assert _call("dg_paged_append", cfg, a) == B.DG_ERR_INVALID_ARG, (i, v)
    for bad in BAD_PAGES:
        assert _call("dg_paged_append", cfg, _append_args(_kv(**bad), rope)) == B.DG_ERR_INVALID_ARG
    for i, v in ((0, 0), (1, 0), (2, None), (2, 264), (3, 4088), (3, 4100), (4, None), (5, 264), (6, 264), (8, None),
                 (9, None), (9, 264), (10, None)):
        a = _norm_args(rope)
        a[i] = v
        assert _call("dg_qk_norm_rope", cfg, a) == B.DG_ERR_INVALID_ARG, (i, v)
    bad_ropes = [B.make_rope(136), B.make_rope(-16), B.make_rope(24), B.make_rope(144),
                 B.make_rope(128, layout=2), B.make_rope(128, scaling=3),
                 B.make_rope(128, mscale=math.nan), B.make_rope(128, scaling=B.DG_ROPE_LINEAR, factor=0),
                 B.make_rope(128, scaling=B.DG_ROPE_LINEAR, factor=math.inf),
                 B.make_rope(128, scaling=B.DG_ROPE_BY_PARTS, factor=2, orig_len=0),
                 B.make_rope(128, scaling=B.DG_ROPE_BY_PARTS, factor=2, orig_len=9, beta_slow=32),
                 B.make_rope(128, scaling=B.DG_ROPE_BY_PARTS, factor=2, orig_len=9, beta_slow=-1)]
    for r in bad_ropes:
        assert _call("dg_qk_norm_rope", cfg, _norm_args(r)) == B.DG_ERR_INVALID_ARG
        assert _call("dg_paged_append", cfg, _append_args(kv, r)) == B.DG_ERR_INVALID_ARG
    assert B.dg_launch_count() == n0


def test_workspace_size():
    cfg = _cfg()
    a = B.dg_paged_workspace_size(cfg, 4, 64)
    assert a > 0 and a % 256 == 0
    assert B.dg_paged_workspace_size(cfg, 4, 64, 128) > a
    assert B.dg_paged_workspace_size(cfg, 0, 64) == 0
    assert B.dg_paged_workspace_size(cfg, 4, 0) == 0
    assert B.dg_paged_workspace_size(cfg, 4, 64, -1) == 0
    assert B.dg_paged_workspace_size(_cfg(head_dim=80), 4, 64) == 0
    with pytest.raises(B.DgError):
        B.alloc_paged_workspace(cfg, 4, 0)


def test_binding_refuses_misfits():
    t = torch.zeros
    with pytest.raises(ValueError):                       # shapes differ
        B.PagedKV(t(2, 1, 16, 64), t(2, 1, 32, 64), t(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):                       # 64-bit page table
        B.PagedKV(t(2, 1, 16, 64), t(2, 1, 16, 64), t(1, 4, dtype=torch.int64))
    with pytest.raises(ValueError):                       # host tensors
        B.PagedKV(t(2, 1, 16, 64), t(2, 1, 16, 64), t(1, 4, dtype=torch.int32))
    cfg = _cfg()
    with pytest.raises(ValueError):                       # wrong type of rows
        B._qkv_rows(cfg, t(5, 4096), 5)
    with pytest.raises(ValueError):                       # wrong width
        B._qkv_rows(cfg, t(5, 4000, dtype=torch.bfloat16), 5)
    with pytest.raises(ValueError):
        B._rows(t(4, 4), "q", torch.bfloat16, (4, 4))
    with pytest.raises(ValueError):
        B._index(t(4, dtype=torch.int64), "seq_off", 2)
    with pytest.raises(ValueError):
        B._index(t(2, dtype=torch.int32), "seq_off", 3)


class _Elsewhere:
    """What the binding asks of a tensor, on a device of its own."""

    is_cuda = True

    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape, self.ndim = dev, dtype, shape, len(shape)

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return 256


def test_binding_refuses_tensors_of_several_devices():
    n0, cfg, bf = B.dg_launch_count(), _cfg(), torch.bfloat16
    hq, hkv, hd = cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    kv = object.__new__(B.PagedKV)
    kv.act, kv.kv_heads, kv.head_dim, kv.seqs = bf, hkv, hd, 2
    kv.struct = B.DgPagedKv(**PAGES)
    kv.ref = ctypes.byref(kv.struct)
    i32 = torch.int32
    names = ("off", "lens", "q", "out", "ws", "status", "pages")
    for far in names:
        dev = {n: 1 if n == far else 0 for n in names}
        kv.dev = dev["pages"]
        args = (_Elsewhere(dev["off"], i32, 3), _Elsewhere(dev["lens"], i32, 2))
        rest = (_Elsewhere(dev["q"], bf, 5, hq, hd), kv, 1, _Elsewhere(dev["out"], bf, 5, hq, hd),
                _Elsewhere(dev["ws"], torch.uint8, 1 << 30), _Elsewhere(dev["status"], i32, 1))
        with pytest.raises(ValueError):
            B.dg_paged_attn(cfg, 2, 5, *args, *rest)
        with pytest.raises(ValueError):
            B.dg_prefix_attn(cfg, 2, 5, *args, 64, *rest)
    for name in ("cache_len", "gain", "status"):
        t = {"cache_len": _Elsewhere(1, i32, 4), "gain": _Elsewhere(1, torch.float32, hd),
             "status": _Elsewhere(1, i32, 1)}[name]
        with pytest.raises(ValueError):
            {"cache_len": lambda: B._index(t, "cache_len", 4, 0),
             "gain": lambda: B._gain(t, "q_gain", hd, 0), "status": lambda: B._status(t, 0)}[name]()
    with pytest.raises(ValueError):                       # a status word of another type
        B._status(_Elsewhere(0, torch.int64, 1), 0)
    assert B.dg_launch_count() == n0
