"""Timed cases of the paged-cache operators: per-head norms with the position rotation, the append
to a paged K/V cache, attention of packed sequences over that cache, and attention for a batch that
shares a long prefix.

`run` computes an operator in its plain form (elementary torch operations) or, with `own` set, by
the library's call.  `exact` restates the operators in 64 bits, apart from the plain form.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0

# ------------------------------------------------------------------------------------- cases

_BASE = dict(op="", act="bf16", hq=16, hkv=8, hd=128, page=64, seqs=1, new_lo=1, new_hi=1,
             kv_lo=0, kv_hi=0, causal=True, shared=0, lens=1, pad=0, norm=True, rot=128,
             layout="half", scaling="none", factor=1.0)


def _case(name, **kw):
    c = dict(_BASE)
    c.update(kw)
    c["name"] = name
    return c


def listed():
    return [
        # one half-refined canvas behind a prompt: a projection's rows on their way to the attention
        _case("norm_rope_canvas", op="norm_rope", new_lo=256, new_hi=256, kv_lo=4096, kv_hi=4096),
        # 32 canvases in one call, positions far in a context that the rotation was stretched for
        _case("norm_rope_batch", op="norm_rope", seqs=32, new_lo=256, new_hi=256, kv_lo=1024,
              kv_hi=131072, lens=3, scaling="by_parts", factor=8.0),
        # single precision, few heads, interleaved pairs over half of the head, padded rows
        _case("norm_rope_odd", op="norm_rope", act="f32", hq=6, hkv=2, hd=64, seqs=3, new_lo=333,
              new_hi=333, kv_lo=1, kv_hi=5000, lens=5, pad=24, rot=32, layout="interleaved",
              scaling="linear", factor=4.0),
        # one new token for each sequence of a serving batch
        _case("append_tokens", op="append", page=16, seqs=64, kv_lo=1, kv_hi=8192, lens=7),
        # prompts of different lengths, packed, written to a new cache
        _case("append_prompts", op="append", page=64, seqs=12, new_lo=64, new_hi=8192, lens=11,
              scaling="by_parts", factor=8.0),
        # a single short sequence's next token: latency
        _case("attn_token", op="attn", page=16, kv_lo=777, kv_hi=777),
        # the next token of 64 sequences of very different lengths: the cache is read once
        _case("attn_tokens_ragged", op="attn", page=16, seqs=64, kv_lo=64, kv_hi=16384, lens=13),
        # prompts of different lengths, packed, causal
        _case("attn_prompts", op="attn", page=64, seqs=9, new_lo=100, new_hi=16384, lens=93),
        # one canvas, all of it visible to itself, over a long context
        _case("attn_canvas_long", op="attn", page=128, new_lo=256, new_hi=256, kv_lo=131072,
              kv_hi=131072, causal=False),
        # single precision, an odd head group, a chunk of a prompt behind an odd length
        _case("attn_odd", op="attn", act="f32", hq=7, hkv=1, hd=64, page=16, seqs=3, new_lo=5,
              new_hi=97, kv_lo=17, kv_hi=700, lens=17),
        # 128 continuations of one long prompt, a token each
        _case("prefix_tokens", op="prefix", page=64, seqs=128, kv_lo=1, kv_hi=512, lens=19,
              shared=8192),
        # 16 canvases drawn for one long prompt, each behind what it has written itself
        _case("prefix_canvases", op="prefix", page=64, seqs=16, new_lo=256, new_hi=256, kv_lo=1,
              kv_hi=1024, lens=23, shared=8192, causal=False),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


HEADS = ((16, 8), (16, 4), (8, 1), (12, 4), (14, 2), (8, 8), (32, 8), (5, 1))


def _draw_once(rng):
    op = rng.choice(("norm_rope", "append", "attn", "attn", "prefix"))
    act = "f32" if rng.random() < 0.25 else "bf16"
    hq, hkv = rng.choice(HEADS)
    hd = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128, 256))
    c = _case("", op=op, act=act, hq=hq, hkv=hkv, hd=hd, page=page, lens=rng.randrange(1 << 30))
    del c["name"]
    c["rot"] = hd
    if op in ("norm_rope", "append"):
        c["norm"] = rng.random() < 0.75
        c["rot"] = rng.choice((hd, hd, hd // 2, hd // 4))
        c["layout"] = rng.choice(("half", "interleaved"))
        c["scaling"] = rng.choice(("none", "linear", "by_parts"))
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice((2.0, 4.0, 8.0))
        c["pad"] = rng.choice((0, 0, 8, 72))
    if op == "norm_rope":
        c["seqs"] = _log_int(rng, 1, 64)
        c["new_lo"] = c["new_hi"] = _log_int(rng, 1, 2048)
        c["kv_lo"], c["kv_hi"] = 1, _log_int(rng, 1, 131072)
        return c
    kind = rng.choice(("tokens", "prompts", "canvases"))
    small = act == "f32" and op != "append"   # single precision: the parity-sized workloads
    c["seqs"] = _log_int(rng, 1, 8 if small else (256 if kind == "tokens" else 24))
    if kind == "tokens":
        c["kv_lo"], c["kv_hi"] = 1, _log_int(rng, 1, 2048 if small else 32768)
    elif kind == "prompts":
        c["new_lo"], c["new_hi"] = 1, _log_int(rng, 1, 512 if small else 16384)
        c["kv_lo"], c["kv_hi"] = 0, rng.choice((0, _log_int(rng, 1, 1024 if small else 8192)))
    else:
        c["new_lo"] = c["new_hi"] = rng.choice((16, 64, 256))
        c["kv_lo"], c["kv_hi"] = 1, _log_int(rng, 1, 1024 if small else 65536)
        c["causal"] = False
    if op == "prefix":
        c["shared"] = max(1, _log_int(rng, 256, 2048 if small else 32768) // page) * page
        if kind == "prompts":
            c["new_hi"] = min(c["new_hi"], 2048)
        c["kv_hi"] = min(c["kv_hi"], 4096)
    return c


def draw(rng):
    most = [work(c) for c in listed()]
    top_bytes = max(w["bytes"] for w in most)
    top_flops = max(w["flops"] for w in most)
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return c


def _lengths(case):
    """New tokens and cached keys of each sequence: part of the case, the same for every seed."""
    rng = random.Random(case["lens"])
    n = case["seqs"]
    new = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(n)]
    lo, hi = case["kv_lo"], case["kv_hi"]
    kv = [_log_int(rng, lo, hi) if lo > 0 else rng.randint(lo, hi) for _ in range(n)]
    return new, [case["shared"] + x for x in kv]


def work(case):
    new, kv = _lengths(case)
    tokens = sum(new)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    e = 4 if case["act"] == "f32" else 2
    row = (hq + 2 * hkv) * hd
    index = 4 * (2 * case["seqs"] + 1)
    if case["op"] in ("norm_rope", "append"):
        per = (7 if case["norm"] else 0) * hd + 3 * case["rot"]
        gains = 2 * hd * 4 if case["norm"] else 0
        return {"bytes": 2 * tokens * row * e + gains + index,
                "flops": tokens * (hq + hkv) * per}
    pairs = 0
    for n, k in zip(new, kv):
        pairs += n * k + (n * (n + 1) // 2 if case["causal"] else n * n)
    keys = case["shared"] + sum(n + k - case["shared"] for n, k in zip(new, kv))
    pages = sum(-(-(n + k) // case["page"]) for n, k in zip(new, kv))
    return {"bytes": 2 * tokens * hq * hd * e + 2 * keys * hkv * hd * e + index + 4 * pages,
            "flops": 4 * pairs * hq * hd}


# ------------------------------------------------------------------------------------ inputs

def _orig_len(case):
    return 16384.0


def _mscale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["act"]]
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    new, kv = _lengths(case)
    tokens = sum(new)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    off = [0]
    for n in new:
        off.append(off[-1] + n)
    st = SimpleNamespace(case=case, new=new, kv=kv, off=off, tokens=tokens, dt=dt)
    st.seq_off = torch.tensor(off, dtype=torch.int32, device=dev)
    st.kv_len = torch.tensor(kv, dtype=torch.int32, device=dev)
    if case["op"] in ("norm_rope", "append"):
        width = (hq + 2 * hkv) * hd
        # rows of a projection: heads of different sizes
        buf = randn(tokens, width + case["pad"])
        scale = torch.exp(0.5 * randn(hq + 2 * hkv)).repeat_interleave(hd)
        buf[:, :width] *= scale
        st.qkv = buf.to(dt)[:, :width]
        st.q_gain = 1.0 + 0.2 * randn(hd) if case["norm"] else None
        st.k_gain = 1.0 + 0.2 * randn(hd) if case["norm"] else None
        st.q = torch.empty((tokens, hq, hd), dtype=dt, device=dev)
    if case["op"] == "norm_rope":
        n = new[0]
        st.q = st.q.view(case["seqs"], n, hq, hd)
        st.k = torch.empty((case["seqs"], hkv, n, hd), dtype=dt, device=dev)
        st.v = torch.empty_like(st.k)
    else:
        shared_pages = case["shared"] // page
        own_pages = [-(-(n + k) // page) - shared_pages for n, k in zip(new, kv)]
        n_pages = shared_pages + sum(own_pages) + 3
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu()
        table = torch.zeros((case["seqs"], shared_pages + max(own_pages)), dtype=torch.int32)
        at = shared_pages
        for s, p in enumerate(own_pages):
            table[s, :shared_pages] = order[:shared_pages]
            table[s, shared_pages:shared_pages + p] = order[at:at + p]
            at += p
        st.table = table.to(dev)
        shape = (n_pages, hkv, page, hd)
        if case["op"] == "append":
            st.k_pages = torch.zeros(shape, dtype=dt, device=dev)
            st.v_pages = torch.zeros(shape, dtype=dt, device=dev)
        else:
            # what earlier sequences left stands behind the last key of a page
            st.k_pages = torch.empty(shape, dtype=dt, device=dev)
            st.v_pages = torch.empty(shape, dtype=dt, device=dev)
            for t in (st.k_pages, st.v_pages):
                for a in range(0, n_pages, 512):
                    b = min(n_pages, a + 512)
                    t[a:b] = randn(b - a, hkv, page, hd).to(dt)
            # trained queries meet some keys much better than others
            st.q = (1.5 * randn(tokens, hq, hd)).to(dt)
            st.out = torch.empty_like(st.q)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    from block_discrete_diffusion_dg_b200 import binding as B
    c = st.case
    kind = "f32" if c["act"] == "f32" else "bf16"
    st.cfg = B.make_config(SimpleNamespace(
        d_model=2048, n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["hd"], n_experts=8,
        top_k=2, d_ff=64, vocab=512, canvas=256, n_layers=1, rope_theta=THETA, rms_eps=EPS,
        act=kind, w=kind))
    st.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["op"] in ("norm_rope", "append"):
        layout = {"half": B.DG_ROPE_HALF, "interleaved": B.DG_ROPE_INTERLEAVED}[c["layout"]]
        scaling = {"none": B.DG_ROPE_UNSCALED, "linear": B.DG_ROPE_LINEAR,
                   "by_parts": B.DG_ROPE_BY_PARTS}[c["scaling"]]
        st.rope = B.make_rope(c["rot"], layout=layout, scaling=scaling, factor=c["factor"],
                              orig_len=_orig_len(c), mscale=_mscale(c))
    if c["op"] != "norm_rope":
        st.pages = B.PagedKV(st.k_pages, st.v_pages, st.table)
    if c["op"] in ("attn", "prefix"):
        st.ws = B.alloc_paged_workspace(st.cfg, c["seqs"], st.tokens, c["shared"])


# --------------------------------------------------------------------------------------- run

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from block_discrete_diffusion_dg_b200 import binding as B
    c = st.case
    if c["op"] == "norm_rope":
        B.dg_qk_norm_rope(st.cfg, c["seqs"], st.new[0], st.qkv, st.kv_len, st.q_gain, st.k_gain,
                          st.rope, st.q, st.k, st.v, st.status)
        return st.q, st.k, st.v
    if c["op"] == "append":
        B.dg_paged_append(st.cfg, c["seqs"], st.tokens, st.seq_off, st.kv_len, st.qkv, st.q_gain,
                          st.k_gain, st.rope, st.pages, st.q, st.status)
        return st.q, st.k_pages, st.v_pages
    if c["op"] == "attn":
        B.dg_paged_attn(st.cfg, c["seqs"], st.tokens, st.seq_off, st.kv_len, st.q, st.pages,
                        c["causal"], st.out, st.ws, st.status)
        return st.out
    B.dg_prefix_attn(st.cfg, c["seqs"], st.tokens, st.seq_off, st.kv_len, c["shared"], st.q,
                     st.pages, c["causal"], st.out, st.ws, st.status)
    return st.out


def _frequencies(case, dev):
    """Angle per position of each pair, in 64 bits."""
    rot = case["rot"]
    j = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    inv = THETA ** (-2.0 * j / rot)
    if case["scaling"] == "linear":
        return inv / case["factor"]
    if case["scaling"] == "by_parts":
        turns = _orig_len(case) * inv / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return inv / case["factor"] * (1.0 - keep) + inv * keep
    return inv


def _norm(x, gain):
    if gain is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain


def _rotate(case, x, cos, sin):
    """x fp32 [tokens, heads, hd]; cos, sin [tokens, 1, rot / 2]."""
    rot = case["rot"]
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _plain_heads(st):
    """q, k and v of the packed rows: heads normed and rotated, rounded once."""
    c = st.case
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    dev = st.qkv.device
    n = torch.tensor(st.new, device=dev)
    seq = torch.repeat_interleave(torch.arange(len(st.new), device=dev), n)
    pos = torch.arange(st.tokens, device=dev) - st.seq_off[seq] + st.kv_len[seq]
    ang = pos.to(torch.float64)[:, None] * _frequencies(c, dev)[None, :]
    cos = (torch.cos(ang) * _mscale(c)).float()[:, None, :]
    sin = (torch.sin(ang) * _mscale(c)).float()[:, None, :]
    x = st.qkv.float().reshape(st.tokens, hq + 2 * hkv, hd)
    q = _rotate(c, _norm(x[:, :hq], st.q_gain), cos, sin).to(st.dt)
    k = _rotate(c, _norm(x[:, hq:hq + hkv], st.k_gain), cos, sin).to(st.dt)
    return q, k, x[:, hq + hkv:].to(st.dt), seq, pos


def _plain_attend(q, k, v, causal_from):
    """q [n, hq, hd], k and v [hkv, keys, hd]; causal_from: cached keys before the first new one,
    or None where every key is visible.  Queries in pieces, so that the scores fit."""
    n, hq, hd = q.shape
    hkv, keys = k.shape[0], k.shape[1]
    rep = hq // hkv
    kf, vf = k.float(), v.float()
    out = torch.empty_like(q)
    step = max(1, min(n, (1 << 29) // (hq * keys)))
    for a in range(0, n, step):
        b = min(n, a + step)
        qf = q[a:b].float().reshape(b - a, hkv, rep, hd).permute(1, 2, 0, 3)
        s = torch.matmul(qf.reshape(hkv, rep * (b - a), hd), kf.transpose(1, 2)) / math.sqrt(hd)
        if causal_from is not None:
            i = torch.arange(a, b, device=q.device)
            hide = torch.arange(keys, device=q.device)[None, :] > causal_from + i[:, None]
            s = s.view(hkv, rep, b - a, keys).masked_fill(hide, float("-inf"))
            s = s.view(hkv, rep * (b - a), keys)
        s = s - s.amax(-1, keepdim=True)
        p = torch.exp(s)
        o = torch.matmul(p, vf) / p.sum(-1, keepdim=True)
        out[a:b] = o.view(hkv, rep, b - a, hd).permute(2, 0, 1, 3).reshape(b - a, hq, hd).to(q.dtype)
    return out


def _run_plain(st):
    c = st.case
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    if c["op"] == "norm_rope":
        q, k, v, _, _ = _plain_heads(st)
        shape = (c["seqs"], st.new[0], hkv, hd)
        return (q.view(c["seqs"], st.new[0], hq, hd), k.reshape(shape).transpose(1, 2).contiguous(),
                v.reshape(shape).transpose(1, 2).contiguous())
    if c["op"] == "append":
        q, k, v, seq, pos = _plain_heads(st)
        where = st.table[seq, pos // page].long()
        st.k_pages[where, :, pos % page] = k
        st.v_pages[where, :, pos % page] = v
        return q, st.k_pages, st.v_pages
    out = torch.empty_like(st.q)
    for s, (n, k) in enumerate(zip(st.new, st.kv)):
        ids = st.table[s, :-(-(n + k) // page)].long()
        kk = st.k_pages[ids].transpose(0, 1).reshape(hkv, -1, hd)[:, :n + k]
        vv = st.v_pages[ids].transpose(0, 1).reshape(hkv, -1, hd)[:, :n + k]
        a, b = st.off[s], st.off[s + 1]
        out[a:b] = _plain_attend(st.q[a:b], kk, vv, k if c["causal"] else None)
    return out


# ------------------------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    c, f64 = case, torch.float64
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    dev = st.seq_off.device
    if c["op"] in ("norm_rope", "append"):
        rot, half = c["rot"], c["rot"] // 2
        heads = st.qkv.to(f64).reshape(st.tokens, -1, hd)
        if c["norm"]:
            for lo, hi, gain in ((0, hq, st.q_gain), (hq, hq + hkv, st.k_gain)):
                part = heads[:, lo:hi]
                size = ((part ** 2).sum(-1, keepdim=True) / hd + EPS) ** 0.5
                heads[:, lo:hi] = part / size * gain.to(f64)
        position = torch.cat([torch.arange(k, k + n, device=dev, dtype=f64)
                              for n, k in zip(st.new, st.kv)])
        slow = []
        for j in range(half):
            w = math.pow(THETA, -2.0 * j / rot)
            if c["scaling"] == "linear":
                w /= c["factor"]
            elif c["scaling"] == "by_parts":
                r = (_orig_len(c) * w / (2.0 * math.pi) - 1.0) / 31.0
                r = min(1.0, max(0.0, r))
                w = w * r + w * (1.0 - r) / c["factor"]
            slow.append(w)
        turn = torch.polar(torch.full((st.tokens, half), _mscale(c), dtype=f64, device=dev),
                           position[:, None] * torch.tensor(slow, dtype=f64, device=dev))
        spun = heads[:, :hq + hkv, :rot]
        if c["layout"] == "half":
            z = torch.complex(spun[..., :half], spun[..., half:]) * turn[:, None]
            spun = torch.cat((z.real, z.imag), -1)
        else:
            z = torch.view_as_complex(spun.reshape(st.tokens, hq + hkv, half, 2).contiguous())
            spun = torch.view_as_real(z * turn[:, None]).reshape(st.tokens, hq + hkv, rot)
        heads[:, :hq + hkv, :rot] = spun
        q, k, v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
        if c["op"] == "norm_rope":
            n = st.new[0]
            return (q.reshape(c["seqs"], n, hq, hd),
                    k.reshape(c["seqs"], n, hkv, hd).permute(0, 2, 1, 3).contiguous(),
                    v.reshape(c["seqs"], n, hkv, hd).permute(0, 2, 1, 3).contiguous())
        pools, pages = [], st.table.tolist()
        for old, rows in ((st.k_pages, k), (st.v_pages, v)):
            pool = old.to(f64)
            for s, (n, have) in enumerate(zip(st.new, st.kv)):
                for p in range(have // page, (have + n - 1) // page + 1):
                    lo, hi = max(have, p * page), min(have + n, (p + 1) * page)
                    src = rows[st.off[s] + lo - have:st.off[s] + hi - have]
                    pool[pages[s][p], :, lo - p * page:hi - p * page] = src.transpose(0, 1)
            pools.append(pool)
        return q, pools[0], pools[1]
    out = torch.empty(st.q.shape, dtype=f64, device=dev)
    rep = hq // hkv
    for s, (n, have) in enumerate(zip(st.new, st.kv)):
        keys = have + n
        ids = st.table[s, :(keys + page - 1) // page].long()
        index = torch.arange(keys, device=dev)
        for g in range(hkv):
            kg = st.k_pages[ids, g].reshape(-1, hd)[:keys].to(f64)
            vg = st.v_pages[ids, g].reshape(-1, hd)[:keys].to(f64)
            rows = st.q[st.off[s]:st.off[s + 1], g * rep:(g + 1) * rep].to(f64)
            piece = max(1, (1 << 27) // (keys * rep))
            for a in range(0, n, piece):
                part = rows[a:a + piece]
                logits = torch.einsum("nrd,kd->nrk", part, kg) * hd ** -0.5
                if c["causal"]:
                    last = have + a + torch.arange(part.shape[0], device=dev)
                    logits[(index[None, :] > last[:, None])[:, None, :].expand_as(logits)] = -math.inf
                w = torch.softmax(logits, -1)
                lo = st.off[s] + a
                out[lo:lo + part.shape[0], g * rep:(g + 1) * rep] = torch.einsum("nrk,kd->nrd", w, vg)
    return out
