"""Parity of the paged-cache operators with their plain 64-bit forms (paged_oracle.py), at the sizes,
masks and layouts where they can go wrong.  Pages hold NaN behind every sequence's last key, page
tables hold ids out of range behind the last page, and buffers hold a marker behind the last row."""
import math
import random
from types import SimpleNamespace

import pytest
import torch

import paged_oracle as P
from block_discrete_diffusion_dg_b200 import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA, EPS = 10000.0, 1e-6
MARK = 7.0


def make_cfg(act, hq, hkv, hd):
    return B.make_config(SimpleNamespace(
        d_model=2048, n_q_heads=hq, n_kv_heads=hkv, head_dim=hd, n_experts=8, top_k=2, d_ff=64,
        vocab=512, canvas=256, n_layers=1, rope_theta=THETA, rms_eps=EPS, act=act, w=act))


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """Pages for sequences of `keys` keys: keys_ [s] holds the stored K, V of sequence s as
    [keys, hkv, hd]; everything else in the pool is NaN."""

    def __init__(self, g, act, hkv, hd, page, keys, shared=0, max_extra=2, empty=False):
        self.page, self.shared = page, shared
        sp = shared // page
        own = [max(0, -(-k // page) - sp) for k in keys]
        n_pages = sp + sum(own) + 2
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        table = torch.full((len(keys), sp + max(own) + max_extra), -1, dtype=torch.int32)
        at = sp
        for s, n in enumerate(own):
            table[s, :sp] = torch.tensor(order[:sp], dtype=torch.int32)
            table[s, sp:sp + n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        shape = (n_pages, hkv, page, hd)
        self.k = torch.full(shape, math.nan, device="cuda").to(DT[act])
        self.v = self.k.clone()
        self.host_table, self.table = table, table.cuda()
        self.kept = []
        for s, n in enumerate(keys):
            if empty:
                break
            kk, vv = randn(g, n, hkv, hd).to(DT[act]), randn(g, n, hkv, hd).to(DT[act])
            if shared and s:
                kk[:shared], vv[:shared] = self.kept[0][0][:shared], self.kept[0][1][:shared]
            pos = torch.arange(n, device="cuda")
            ids = self.table[s][pos // page].long()
            self.k[ids, :, pos % page] = kk
            self.v[ids, :, pos % page] = vv
            self.kept.append((kk, vv))
        self.kv = B.PagedKV(self.k, self.v, self.table)

    def rows(self, pool, s, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        return pool[self.table[s][pos // self.page].long(), :, pos % self.page]


def offsets(new):
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return off


# ------------------------------------------------------------------------------ norms, rotation

ROPES = [
    dict(rot=128, layout="half", scaling="none"),
    dict(rot=64, layout="half", scaling="linear", factor=4.0),
    dict(rot=32, layout="interleaved", scaling="by_parts", factor=8.0, orig_len=4096.0),
    dict(rot=128, layout="interleaved", scaling="none", mscale=1.25),
    dict(rot=0, layout="half", scaling="none"),
    dict(rot=48, layout="half", scaling="by_parts", factor=2.0, orig_len=512.0),
    None,
]


def rope_of(r, hd):
    """(dg_rope or None, arguments of the oracle) of a test's rope, cut to the head."""
    if r is None:
        return None, (P.frequencies(THETA, hd), hd, "half", 1.0)
    rot = min(r["rot"], hd)
    lay = {"half": B.DG_ROPE_HALF, "interleaved": B.DG_ROPE_INTERLEAVED}[r["layout"]]
    sc = {"none": B.DG_ROPE_UNSCALED, "linear": B.DG_ROPE_LINEAR,
          "by_parts": B.DG_ROPE_BY_PARTS}[r["scaling"]]
    f, o, m = r.get("factor", 1.0), r.get("orig_len", 0.0), r.get("mscale", 1.0)
    return (B.make_rope(rot, lay, sc, factor=f, orig_len=o, mscale=m),
            (P.frequencies(THETA, rot, r["scaling"], f, o), rot, r["layout"], m))


def check_rows(got, want, extra, dt):
    assert P.worst(got, want, P.HALF[dt] * want.abs() + extra) <= 1.0


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd", [(16, 8, 128), (7, 1, 64), (2, 1, 32), (3, 3, 128)])
@pytest.mark.parametrize("ri", range(len(ROPES)))
def test_qk_norm_rope(act, hq, hkv, hd, ri):
    dt = DT[act]
    batch, n, pad = 3, 1 + 6 * ri, 16 * (ri % 2)
    g = gen(100 + ri)
    rope, (freq, rot, layout, ms) = rope_of(ROPES[ri], hd)
    width = (hq + 2 * hkv) * hd
    qkv = (3.0 * randn(g, batch * n, width + pad)).to(dt)[:, :width]
    qg = 1 + 0.3 * randn(g, hd) if ri % 3 else None
    kg = 1 + 0.3 * randn(g, hd) if ri % 3 != 1 else None
    lens = [0, 131072 - n, 777]
    q = torch.full((batch, n, hq, hd), MARK, dtype=dt, device="cuda")
    k = torch.full((batch, hkv, n, hd), MARK, dtype=dt, device="cuda")
    v = torch.full_like(k, MARK)
    st = i32([0])
    B.dg_qk_norm_rope(make_cfg(act, hq, hkv, hd), batch, n, qkv, i32(lens), qg, kg, rope, q, k, v, st)
    assert B.dg_read_status(st) == B.DG_OK
    x = qkv.reshape(batch * n, hq + 2 * hkv, hd)
    pos = torch.cat([torch.arange(a, a + n) for a in lens])
    wq, eq = P.norm_rope(x[:, :hq], qg, EPS, pos, freq, rot, layout, ms)
    wk, ek = P.norm_rope(x[:, hq:hq + hkv], kg, EPS, pos, freq, rot, layout, ms)
    check_rows(q.view(batch * n, hq, hd), wq, eq, dt)
    check_rows(k.transpose(1, 2).reshape(batch * n, hkv, hd), wk, ek, dt)
    assert torch.equal(v.transpose(1, 2).reshape(batch * n, hkv, hd), x[:, hq + hkv:])


def test_norm_of_zero_and_huge_rows():
    """A head of zeros stays zero (eps keeps the norm finite), one near fp32's square root of the
    largest value keeps its direction, and NaN stays within its head."""
    cfg = make_cfg("f32", 2, 1, 64)
    qkv = torch.zeros(1, 4 * 64, device="cuda")
    qkv[0, 64:128] = 1e18
    qkv[0, 128:192] = math.nan
    one = torch.ones(64, device="cuda")
    q, k, v = (torch.empty(1, *s, 64, device="cuda") for s in ((1, 2), (1, 1), (1, 1)))
    B.dg_qk_norm_rope(cfg, 1, 1, qkv, i32([0]), one, one, None, q, k, v)
    assert (q[0, 0, 0] == 0).all() and torch.isnan(k).all() and (v == 0).all()
    assert (q[0, 0, 1] - 1).abs().max() < 1e-5


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,page", [(16, 8, 128, 16), (7, 1, 64, 64), (4, 2, 32, 256),
                                            (6, 2, 128, 1024)])
@pytest.mark.parametrize("ri", [0, 2, 5])
def test_paged_append(act, hq, hkv, hd, page, ri):
    dt, g = DT[act], gen(200 + ri)
    rope, (freq, rot, layout, ms) = rope_of(ROPES[ri], hd)
    new, have = [1, 0, 37, 130, 1, 0], [0, 5, page - 1, 3 * page + 2, 900, 0]
    off = offsets(new)
    rows = off[-1] + 3                                   # a padded batch
    c = Cache(g, act, hkv, hd, page, [n + h for n, h in zip(new, have)], empty=True)
    k0, v0 = c.k.clone(), c.v.clone()
    width = (hq + 2 * hkv) * hd
    qkv = randn(g, rows, width).to(dt)
    gain = 1 + 0.3 * randn(g, hd)
    q = torch.full((rows, hq, hd), MARK, dtype=dt, device="cuda")
    st = i32([0])
    B.dg_paged_append(make_cfg(act, hq, hkv, hd), len(new), rows, i32(off), i32(have), qkv, gain, gain,
                      rope, c.kv, q, st)
    assert B.dg_read_status(st) == B.DG_OK
    x = qkv.view(rows, hq + 2 * hkv, hd)[:off[-1]]
    pos = torch.cat([torch.arange(h, h + n) for n, h in zip(new, have)])
    wq, eq = P.norm_rope(x[:, :hq], gain, EPS, pos, freq, rot, layout, ms)
    wk, ek = P.norm_rope(x[:, hq:hq + hkv], gain, EPS, pos, freq, rot, layout, ms)
    check_rows(q[:off[-1]], wq, eq, dt)
    assert (q[off[-1]:].float() == MARK).all()
    for s, (n, h) in enumerate(zip(new, have)):
        a, b = off[s], off[s + 1]
        check_rows(c.rows(c.k, s, h, h + n), wk[a:b], ek[a:b], dt)
        assert torch.equal(c.rows(c.v, s, h, h + n), x[a:b, hq + hkv:])
        p = torch.arange(h, h + n, device="cuda")        # put back what may change, compare the rest
        ids = c.table[s][p // page].long()
        for pool, was in ((c.k, k0), (c.v, v0)):
            pool[ids, :, p % page] = was[ids, :, p % page]
    assert torch.isnan(c.k.float()).all() and torch.isnan(c.v.float()).all()
    # only the cache: q may be left out, and the pages come out the same
    B.dg_paged_append(make_cfg(act, hq, hkv, hd), len(new), rows, i32(off), i32(have), qkv, gain, gain,
                      rope, c.kv, None, st)
    check_rows(c.rows(c.k, 3, have[3], have[3] + new[3]), wk[off[3]:off[4]], ek[off[3]:off[4]], dt)


# ----------------------------------------------------------------------------------- attention

def run_attention(cfg, cache, new, have, q, causal, rows=None, shared=0, ws=None, stream=None):
    rows = q.shape[0] if rows is None else rows
    out = torch.full_like(q, MARK)
    st = i32([0])
    ws = B.alloc_paged_workspace(cfg, len(new), rows, shared) if ws is None else ws
    ws.fill_(0xFF)                                       # NaN bits: nothing stale may be read
    args = (i32(offsets(new)), i32(have)) + ((shared,) if shared else ())
    f = B.dg_prefix_attn if shared else B.dg_paged_attn
    f(cfg, len(new), rows, *args, q, cache.kv, causal, out, ws, st, stream)
    return out, B.dg_read_status(st)


def check_attention(out, q, cache, new, have, causal, act, skip=()):
    off = offsets(new)
    p_bits = 2.0 ** -8 if act == "bf16" else 0.0
    for s, (n, h) in enumerate(zip(new, have)):
        got = out[off[s]:off[s + 1]]
        if s in skip:
            assert (got.float() == MARK).all()
            continue
        if n == 0:
            continue
        k, v = cache.kept[s]
        want, A, e = P.attention(q[off[s]:off[s + 1]], k[:h + n], v[:h + n], causal, h)
        w = P.worst(got, want, P.attention_bound(want, A, e, h + n, q.dtype, p_bits))
        assert w <= 1.0, (s, n, h, w)
    assert (out[off[-1]:].float() == MARK).all()


BATCHES = {
    "one_token_one_key": ([1], [0]),
    "one_token": ([1], [127]),
    "tokens": ([1] * 9, [0, 1, 15, 63, 64, 127, 128, 300, 1031]),
    "prompts": ([1, 130, 0, 67, 257, 16], [0, 0, 0, 0, 0, 0]),
    "chunks": ([5, 33, 128], [250, 64, 1]),
    "long": ([2, 1], [2500, 3001]),
}
HEADS = [("bf16", 16, 8, 128), ("bf16", 14, 2, 64), ("bf16", 5, 1, 128), ("bf16", 64, 1, 64),
         ("bf16", 4, 4, 32), ("f32", 7, 1, 64), ("f32", 2, 2, 128), ("f32", 2, 1, 32)]


@pytest.mark.parametrize("act,hq,hkv,hd", HEADS)
@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("causal", [0, 1])
def test_paged_attn(act, hq, hkv, hd, batch, causal):
    new, have = BATCHES[batch]
    g = gen(1000 * hq + 100 * hkv + hd + len(new))
    page = {"tokens": 16, "prompts": 64, "chunks": 32, "long": 128}.get(batch, 256)
    c = Cache(g, act, hkv, hd, page, [n + h for n, h in zip(new, have)])
    q = (1.5 * randn(g, sum(new) + 2, hq, hd)).to(DT[act])
    out, st = run_attention(make_cfg(act, hq, hkv, hd), c, new, have, q, causal)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, causal, act)


PREFIXED = {
    "tokens": ([1] * 7, [0, 1, 15, 40, 3, 100, 64], 256),
    "canvases": ([16, 16, 64], [0, 70, 200], 512),
    "ragged": ([1, 0, 90, 7], [0, 12, 33, 128], 64),
    "one": ([1], [0], 1024),
}


@pytest.mark.parametrize("act,hq,hkv,hd", HEADS)
@pytest.mark.parametrize("batch", list(PREFIXED))
@pytest.mark.parametrize("causal", [0, 1])
def test_prefix_attn(act, hq, hkv, hd, batch, causal):
    new, own, shared = PREFIXED[batch]
    have = [shared + o for o in own]
    g = gen(len(new))
    c = Cache(g, act, hkv, hd, 64, [n + h for n, h in zip(new, have)], shared=shared)
    q = (1.5 * randn(g, sum(new) + 1, hq, hd)).to(DT[act])
    out, st = run_attention(make_cfg(act, hq, hkv, hd), c, new, have, q, causal, shared=shared)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, causal, act)


def random_batch(rng, seqs, big):
    """New tokens and cached keys of a random batch: single tokens, tails, chunks and prompts."""
    kinds = [lambda: 1, lambda: rng.randint(1, 20), lambda: rng.randint(1, big), lambda: 0]
    new = [rng.choice(kinds)() for _ in range(seqs)]
    have = [rng.choice((0, 1, rng.randint(0, 40), rng.randint(0, 8 * big))) for _ in range(seqs)]
    if sum(new) == 0:
        new[0] = 1
    return new, have


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    """All kinds of work in one call: sequences of many lengths, any head group, page size and mask,
    with and without a shared prefix."""
    rng = random.Random(seed)
    act, hd = rng.choice((("bf16", 128), ("bf16", 64), ("f32", 64)))
    hkv = rng.choice((1, 2, 3))
    hq = hkv * rng.choice((1, 2, 3, 4, 7, 8, 17))
    page = rng.choice((16, 32, 128, 256))
    seqs = rng.choice((1, 5, 40, 140, 400))
    new, have = random_batch(rng, seqs, 300 if seqs < 20 else 30)
    shared = page * rng.randint(1, 4) if seed % 3 == 2 else 0
    have = [shared + h for h in have]
    g = gen(seed)
    c = Cache(g, act, hkv, hd, page, [n + h for n, h in zip(new, have)], shared=shared)
    q = (1.5 * randn(g, sum(new) + 1, hq, hd)).to(DT[act])
    for causal in (0, 1):
        out, st = run_attention(make_cfg(act, hq, hkv, hd), c, new, have, q, causal, shared=shared)
        assert st == B.DG_OK
        check_attention(out, q, c, new, have, causal, act)


@pytest.mark.parametrize("n_new", [1, 40, 200])
def test_pages_past_32_bit_offsets(n_new):
    """A pool of more than 2^31 elements: the sequence's pages lie at its far end."""
    g, hkv, hd, page, have = gen(77), 8, 128, 64, 200
    n_pages = (1 << 31) // (hkv * page * hd) + 64
    pools = [torch.empty(n_pages, hkv, page, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    keys = have + n_new
    used = -(-keys // page)
    table = torch.arange(n_pages - used, n_pages, dtype=torch.int32, device="cuda")[None].contiguous()
    for t in pools:
        t[n_pages - used:] = math.nan
    kv = B.PagedKV(*pools, table)
    cfg = make_cfg("bf16", 16, hkv, hd)
    k, v = (randn(g, keys, hkv, hd).to(torch.bfloat16) for _ in range(2))
    qkv = torch.cat((torch.zeros(keys, 16 * hd, device="cuda", dtype=torch.bfloat16),
                     k.view(keys, -1), v.view(keys, -1)), 1)
    st = i32([0])
    B.dg_paged_append(cfg, 1, keys, i32([0, keys]), i32([0]), qkv, None, None, B.make_rope(0), kv,
                      None, st)
    pos = torch.arange(keys, device="cuda")
    ids = table[0][pos // page].long()
    assert torch.equal(pools[0][ids, :, pos % page], k) and torch.equal(pools[1][ids, :, pos % page], v)
    q = randn(g, n_new, 16, hd).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = B.alloc_paged_workspace(cfg, 1, n_new)
    B.dg_paged_attn(cfg, 1, n_new, i32([0, n_new]), i32([have]), q, kv, 1, out, ws, st)
    assert B.dg_read_status(st) == B.DG_OK
    want, A, e = P.attention(q, k, v, 1, have)
    assert P.worst(out, want, P.attention_bound(want, A, e, keys, torch.bfloat16, 2.0 ** -8)) <= 1.0


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("bf16", 8, 4, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("n", [3, 40, 300])
def test_extreme_scores(act, hq, hkv, hd, n):
    """Scores far apart and growing along the keys: the running maximum moves on again and again and
    late keys take all of the weight, or early ones do; equal scores give the plain mean.  For each
    kind of work (n = 3, 40 and 300 rows of two heads)."""
    g = gen(5)
    new, have = [n], [900]
    c = Cache(g, act, hkv, hd, 64, [900 + n])
    k, v = c.kept[0]
    pos = torch.arange(900 + n, device="cuda")
    ids = c.table[0][pos // 64].long()
    ramp = torch.linspace(-8, 8, 900 + n, device="cuda")[:, None, None]
    k = (torch.ones_like(k, dtype=torch.float32) * ramp).to(k.dtype)
    c.kept[0] = (k, v)
    c.k[ids, :, pos % 64] = k
    q = torch.full((n, hq, hd), 2.0, device="cuda").to(DT[act])
    q[1::3] = -2.0
    q[2::3] = 0.0
    for causal in (0, 1):
        out, st = run_attention(make_cfg(act, hq, hkv, hd), c, new, have, q, causal)
        assert st == B.DG_OK
        check_attention(out, q, c, new, have, causal, act)


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("bf16", 4, 4, 64), ("bf16", 16, 1, 128),
                                           ("bf16", 32, 1, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("shared", [0, 64, 8192])
def test_batches_of_a_few_rows(act, hq, hkv, hd, shared):
    """Calls whose rows all fit few-row items, and the first that do not: one row and several, short
    contexts and ones cut into more pieces than a warp has lanes, with rows of nobody's behind."""
    g, most = gen(19), max(16 * hkv // hq, 1)
    cfg = make_cfg(act, hq, hkv, hd)
    for new, own in (([1], [0]), ([1], [9000]), ([most], [300]), ([most + 1], [300]),
                     ([1] * (most // 2) + [0, most - most // 2], [700] * (most // 2) + [5, 40])):
        have = [shared + o for o in own]
        c = Cache(g, act, hkv, hd, 64, [n + h for n, h in zip(new, have)], shared=shared)
        rows = sum(new)
        for padded in {rows, max(rows, most)}:
            q = randn(g, padded, hq, hd).to(DT[act])
            for causal in (0, 1):
                out, st = run_attention(cfg, c, new, have, q, causal, shared=shared)
                assert st == B.DG_OK
                check_attention(out[:rows], q[:rows], c, new, have, causal, act)
                assert (out[rows:].float() == MARK).all()


@pytest.mark.parametrize("hq,hkv,hd", [(16, 8, 128), (3, 3, 64), (16, 1, 128), (5, 1, 64)])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("kind", ["tokens", "pairs", "one_prompt", "prompts"])
def test_as_many_sequences_as_rows(hq, hkv, hd, causal, kind):
    """Batches that look like single tokens by their sizes, and are, or are prompts among empty
    sequences."""
    g, rng = gen(20), random.Random(hq * 10 + causal)
    new = {"tokens": [1] * 90, "pairs": [2, 0, 1, 1, 0, 2] * 15, "one_prompt": [0] * 40 + [150] + [0] * 120,
           "prompts": [33, 0, 70, 1, 0, 47] + [0] * 150}[kind]
    have = [rng.choice((0, 1, 31, 32, 33, 300, 2500)) for _ in new]
    c = Cache(g, "bf16", hkv, hd, 32, [n + h for n, h in zip(new, have)])
    q = randn(g, sum(new), hq, hd).to(torch.bfloat16)
    out, st = run_attention(make_cfg("bf16", hq, hkv, hd), c, new, have, q, causal)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, causal, "bf16")


@pytest.mark.parametrize("hq,hkv,hd", [(16, 8, 128), (5, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("have", [0, 50])
def test_tokens_prompt_and_idle_slots(hq, hkv, hd, page, have):
    """A serving batch of 256 slots: 199 single tokens over one long context, a prompt of 40 tokens, the
    rest idle.  A worker's range holds several of the prompt's items, each of which sees more pages than
    the one before."""
    g, keys = gen(21), 8192
    c = Cache(g, "bf16", hkv, hd, page, [keys, 40 + have])
    table = torch.full((256, c.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[:199], table[199] = c.table[0], c.table[1]     # (pages may be shared: none is written here)
    c.kv = B.PagedKV(c.k, c.v, table)
    new, lens = [1] * 199 + [40] + [0] * 56, [keys - 1] * 199 + [have] + [0] * 56
    q = (1.5 * randn(g, 239, hq, hd)).to(torch.bfloat16)
    for causal in (1, 0):
        out, st = run_attention(make_cfg("bf16", hq, hkv, hd), c, new, lens, q, causal)
        assert st == B.DG_OK
        for s, rows, h, mask in ((0, slice(0, 199), keys - 1, 0), (1, slice(199, 239), have, causal)):
            k, v = c.kept[s]
            want, A, e = P.attention(q[rows], k, v, mask, h)
            bound = P.attention_bound(want, A, e, k.shape[0], torch.bfloat16, 2.0 ** -8)
            assert P.worst(out[rows], want, bound) <= 1.0


@pytest.mark.parametrize("hq,hkv,hd,page", [(8, 2, 128, 16), (8, 2, 64, 64), (5, 5, 64, 32)])
def test_long_prompt_among_idle_slots(hq, hkv, hd, page):
    g, n = gen(22), 2048
    new, have = [0] * 700 + [n] + [0] * 1347, [0] * 2048
    c = Cache(g, "bf16", hkv, hd, page, [a + h for a, h in zip(new, have)])
    q = (1.5 * randn(g, n, hq, hd)).to(torch.bfloat16)
    out, st = run_attention(make_cfg("bf16", hq, hkv, hd), c, new, have, q, 1)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, 1, "bf16")


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("shared", [0, 1024])
def test_largest_page(act, hq, hkv, hd, shared):
    g, new, own = gen(6), [1, 40, 300], [1500, 0, 1000]
    have = [shared + o for o in own]
    c = Cache(g, act, hkv, hd, 1024, [n + h for n, h in zip(new, have)], shared=shared)
    q = (1.5 * randn(g, sum(new), hq, hd)).to(DT[act])
    out, st = run_attention(make_cfg(act, hq, hkv, hd), c, new, have, q, 1, shared=shared)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, 1, act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [0, 32])
def test_empty_batches_and_rows_before_the_first(act, shared):
    """Offsets that hold no row at all leave the output alone; rows before the first sequence are
    nobody's, and stay too."""
    g, hq, hkv, hd = gen(7), 4, 2, 64
    cfg = make_cfg(act, hq, hkv, hd)
    c = Cache(g, act, hkv, hd, 16, [shared + 40, shared + 90], shared=shared)
    q = randn(g, 12, hq, hd).to(DT[act])
    ws = B.alloc_paged_workspace(cfg, 2, 12, shared)
    for off in ([0, 0, 0], [12, 12, 12], [3, 5, 9]):
        ws.fill_(0xFF)
        out, st = torch.full_like(q, MARK), i32([0])
        have = [shared + 38, shared + 86]
        args = (cfg, 2, 12, i32(off), i32(have)) + ((shared,) if shared else ())
        (B.dg_prefix_attn if shared else B.dg_paged_attn)(*args, q, c.kv, 1, out, ws, st)
        assert B.dg_read_status(st) == B.DG_OK
        assert (out[:off[0]].float() == MARK).all() and (out[off[2]:].float() == MARK).all()
        if off[0] == off[2]:
            continue
        check_attention(out[off[0]:], q[off[0]:], c, [2, 4], have, 1, act)
        qkv = randn(g, 12, (hq + 2 * hkv) * hd).to(DT[act])
        qo = torch.full_like(q, MARK)
        B.dg_paged_append(cfg, 2, 12, i32(off), i32(have), qkv, None, None, B.make_rope(0), c.kv, qo, st)
        assert B.dg_read_status(st) == B.DG_OK
        assert torch.equal(qo[3:9], qkv[3:9, :hq * hd].view(6, hq, hd))
        assert (qo[:3].float() == MARK).all() and (qo[9:].float() == MARK).all()


def test_thousands_of_sequences():
    g, hq, hkv, hd, seqs = gen(13), 4, 2, 64, 3000
    rng = random.Random(4)
    have = [rng.choice((0, 3, 20, 45)) for _ in range(seqs)]
    new = [rng.choice((0, 1, 1, 1, 2)) for _ in range(seqs)]
    c = Cache(g, "bf16", hkv, hd, 16, [n + h for n, h in zip(new, have)])
    q = randn(g, sum(new), hq, hd).to(torch.bfloat16)
    out, st = run_attention(make_cfg("bf16", hq, hkv, hd), c, new, have, q, 1)
    assert st == B.DG_OK
    check_attention(out, q, c, new, have, 1, "bf16")


def test_calls_at_the_same_time():
    """Two streams, each with its own workspace and sequences, over one cache: every result is the one
    that the call gives alone."""
    g, hq, hkv, hd = gen(17), 16, 8, 128
    cfg = make_cfg("bf16", hq, hkv, hd)
    new, have = [1, 1, 90, 300], [2000, 30, 500, 0]
    c = Cache(g, "bf16", hkv, hd, 64, [n + h for n, h in zip(new, have)])
    q = randn(g, sum(new), hq, hd).to(torch.bfloat16)
    want = [run_attention(cfg, c, new, have, q, causal)[0] for causal in (0, 1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [B.alloc_paged_workspace(cfg, 4, sum(new)) for _ in range(2)]
    outs = [[torch.full_like(q, MARK) for _ in range(20)] for _ in range(2)]
    off, lens = i32(offsets(new)), i32(have)
    torch.cuda.synchronize()
    for i in range(20):
        for causal, s in enumerate(streams):
            B.dg_paged_attn(cfg, 4, sum(new), off, lens, q, c.kv, causal, outs[causal][i], ws[causal],
                            None, s)
    torch.cuda.synchronize()
    for causal in (0, 1):
        assert all(torch.equal(o, want[causal]) for o in outs[causal])


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("bf16", 8, 8, 64), ("f32", 4, 2, 64)])
def test_skipped_sequences_leave_their_rows(act, hq, hkv, hd):
    """A sequence past its pages, or shorter than the shared prefix, is skipped and reported; the
    others come out as ever."""
    g = gen(8)
    new, have = [4, 3, 40], [100, 64, 10]
    c = Cache(g, act, hkv, hd, 64, [n + h for n, h in zip(new, have)], max_extra=0)
    q = randn(g, sum(new), hq, hd).to(DT[act])
    cfg = make_cfg(act, hq, hkv, hd)
    over = [100, 127, 10]                                # 130 keys where two pages hold 128
    out, st = run_attention(cfg, c, new, over, q, 1)
    assert st == B.DG_ERR_CAPACITY
    check_attention(out, q, c, new, over, 1, act, skip=(1,))
    qkv = randn(g, sum(new), (hq + 2 * hkv) * hd).to(DT[act])
    k0 = c.k.clone()
    qo = torch.full_like(q, MARK)
    status = i32([0])
    B.dg_paged_append(cfg, 3, sum(new), i32(offsets(new)), i32(over), qkv, None, None,
                      B.make_rope(0), c.kv, qo, status)
    assert B.dg_read_status(status) == B.DG_ERR_CAPACITY
    assert torch.equal(qo, qkv[:, :hq * hd].view_as(qo))
    same = torch.isnan(k0) & torch.isnan(c.k) | (k0 == c.k)
    second = c.table[1].long()
    assert same[second[second >= 0]].all()
    have = [100, 70, 90]
    c = Cache(g, act, hkv, hd, 64, [n + h for n, h in zip(new, have)], shared=64)
    out, st = run_attention(cfg, c, new, [100, 60, 90], q, 1, shared=64)
    assert st == B.DG_ERR_INVALID_ARG
    check_attention(out, q, c, new, [100, 60, 90], 1, act, skip=(1,))


def test_bad_page_ids_are_reported():
    """A page id out of range is never followed: the append skips the row, the attention reports it
    and the other sequences come out as ever."""
    g = gen(9)
    cfg = make_cfg("bf16", 16, 8, 128)
    new, have = [2, 2], [200, 300]
    c = Cache(g, "bf16", 8, 128, 64, [202, 302])
    q = randn(g, 4, 16, 128).to(torch.bfloat16)
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.table[1, 4] = bad
        out, st = run_attention(cfg, c, new, have, q, 1)
        assert st == B.DG_ERR_INVALID_ARG
        keep = c.kept[1]
        check_attention(out[:2], q[:2], c, new[:1], have[:1], 1, "bf16")
        qkv = randn(g, 4, 32 * 128).to(torch.bfloat16)
        status, k0 = i32([0]), c.k.clone()
        B.dg_paged_append(cfg, 2, 4, i32([0, 2, 4]), i32(have), qkv, None, None, None, c.kv, None,
                          status)
        assert B.dg_read_status(status) == B.DG_ERR_INVALID_ARG
        mine = c.host_table[0][c.host_table[0] >= 0].long().cuda()
        rest = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")
        rest[mine] = False
        assert torch.equal(c.k[rest].nan_to_num(9), k0[rest].nan_to_num(9))
        c.kept[0] = (c.rows(c.k, 0, 0, 202), c.rows(c.v, 0, 0, 202))
        c.kept[1] = keep


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("off", [[0, 10, 5, 12], [0, 12, 4], [0, 3, 3, 12, -2], [4, 4, 2]])
def test_descending_offsets_attend_nothing(act, hq, hkv, hd, off):
    """Where offsets descend no row is written, whatever a workspace holds, and every call reports."""
    g, n, seqs, cfg = gen(14), 12, len(off) - 1, make_cfg(act, hq, hkv, hd)
    c = Cache(g, act, hkv, hd, 16, [32 + 40] * seqs, shared=32)
    q = randn(g, n, hq, hd).to(DT[act])
    have, st = [32 + 20] * seqs, i32([0])
    for shared in (0, 32):
        ws = B.alloc_paged_workspace(cfg, seqs, n, shared)
        for fill in (0, 0x7F, 0xBF):
            ws.fill_(fill)
            out = torch.full_like(q, MARK)
            args = (cfg, seqs, n, i32(off), i32(have)) + ((shared,) if shared else ())
            (B.dg_prefix_attn if shared else B.dg_paged_attn)(*args, q, c.kv, 1, out, ws, st)
            assert B.dg_read_status(st) == B.DG_ERR_INVALID_ARG
            B.dg_clear_status(st)
            assert (out.float() == MARK).all()
    B.dg_paged_append(cfg, seqs, n, i32(off), i32(have), randn(g, n, (hq + 2 * hkv) * hd).to(DT[act]),
                      None, None, B.make_rope(0), c.kv, q, st)
    assert B.dg_read_status(st) == B.DG_ERR_INVALID_ARG


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("f32", 4, 4, 32)])
def test_sequences_that_claim_the_same_rows(act, hq, hkv, hd):
    """Offsets that go back and forth: thousands of sequences of 40,000 rows each, whose work adds up
    past 32 bits, are refused as a whole."""
    n, seqs, have = 40000, 8001, 25000
    off = i32([0, n] * (seqs // 2 + 1))
    pages = torch.zeros(2, hkv, 1024, hd, dtype=DT[act], device="cuda")
    kv = B.PagedKV(pages, pages, torch.zeros(seqs, 64, dtype=torch.int32, device="cuda"))
    q = torch.zeros(n, hq, hd, dtype=DT[act], device="cuda")
    out, st, cfg = torch.full_like(q, MARK), i32([0]), make_cfg(act, hq, hkv, hd)
    for shared in (0, 1024):
        ws = B.alloc_paged_workspace(cfg, seqs, n, shared)
        args = (cfg, seqs, n, off, i32([have] * seqs)) + ((shared,) if shared else ())
        (B.dg_prefix_attn if shared else B.dg_paged_attn)(*args, q, kv, 1, out, ws, st)
        assert B.dg_read_status(st) == B.DG_ERR_INVALID_ARG
        B.dg_clear_status(st)
        assert (out.float() == MARK).all()


@pytest.mark.parametrize("off,lens,code", [
    ([20, 30], [5], B.DG_ERR_INVALID_ARG), ([0, 30], [5], B.DG_ERR_INVALID_ARG),
    ([-3, 4], [5], B.DG_ERR_INVALID_ARG), ([0, 4, 8], [5, -1], B.DG_ERR_INVALID_ARG),
    ([0, 4, 8], [5, 1000], B.DG_ERR_CAPACITY), ([0, 4, 4], [5, -1], B.DG_OK),
    ([0, 2, 4, 8, 6], [5] * 4, B.DG_ERR_INVALID_ARG)])
def test_append_reports_what_the_attention_reports(off, lens, code):
    g, n, cfg = gen(15), 8, make_cfg("bf16", 4, 2, 64)
    c = Cache(g, "bf16", 2, 64, 16, [60] * len(lens))
    q, st = torch.empty(n, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([0])
    B.dg_paged_append(cfg, len(lens), n, i32(off), i32(lens), randn(g, n, 8 * 64).to(torch.bfloat16),
                      None, None, None, c.kv, q, st)
    assert B.dg_read_status(st) == code


def test_norm_reports_negative_lengths():
    """A canvas of negative length is skipped, the others come out as ever."""
    g, n, hq, hkv, hd = gen(16), 20, 4, 2, 64
    cfg = make_cfg("bf16", hq, hkv, hd)
    qkv = randn(g, 3 * n, (hq + 2 * hkv) * hd).to(torch.bfloat16)

    def run(lens):
        q = torch.full((3, n, hq, hd), MARK, dtype=torch.bfloat16, device="cuda")
        k = torch.full((3, hkv, n, hd), MARK, dtype=torch.bfloat16, device="cuda")
        v, st = torch.full_like(k, MARK), i32([0])
        B.dg_qk_norm_rope(cfg, 3, n, qkv, i32(lens), None, None, None, q, k, v, st)
        return (q, k, v), B.dg_read_status(st)

    want, st = run([4, 8, 9])
    assert st == B.DG_OK
    got, st = run([4, -8, 9])
    assert st == B.DG_ERR_INVALID_ARG
    for w, t in zip(want, got):
        assert torch.equal(t[0], w[0]) and torch.equal(t[2], w[2])
        assert (t[1].float() == MARK).all()


@pytest.mark.parametrize("hq,hkv", [(6, 2), (5, 1), (14, 2)])
def test_results_do_not_hang_on_the_call_before(hq, hkv):
    """Groups that do not divide a query tile leave rows of it to whatever another call left in shared
    memory; a sequence's neighbours stand in the rows behind its own.  Neither may show in a result."""
    g, hd, n, have = gen(18), 128, 128 // (hq // hkv), 4000
    cfg = make_cfg("bf16", hq, hkv, hd)
    c = Cache(g, "bf16", hkv, hd, 64, [have + n])
    ramp = torch.linspace(0, 1, have + n, device="cuda")[:, None, None]
    k = (ramp + 0.02 * randn(g, have + n, hkv, hd)).to(torch.bfloat16)
    v = c.kept[0][1]
    pos = torch.arange(have + n, device="cuda")
    c.k[c.table[0][pos // 64].long(), :, pos % 64] = k
    c.kept[0] = (k, v)
    # the same sequence many times over, so that items stay whole and pass many key tiles
    seqs = 300
    many = B.PagedKV(c.k, c.v, c.table.repeat(seqs, 1))
    off, lens = i32([i * n for i in range(seqs + 1)]), i32([have] * seqs)
    wide_ws = B.alloc_paged_workspace(cfg, seqs, seqs * n)
    q = (0.2 + 0.02 * randn(g, n, hq, hd)).to(torch.bfloat16)
    qs = q.repeat(seqs, 1, 1)
    big = make_cfg("bf16", 2 * hkv, 2 * hkv, hd)
    pages = torch.ones(2, 2 * hkv, 64, hd, dtype=torch.bfloat16, device="cuda")
    kv = B.PagedKV(pages, pages, torch.zeros(148, 2, dtype=torch.int32, device="cuda"))
    ws = B.alloc_paged_workspace(big, 148, 148 * 100)
    outs = []
    for value in (0.0, 100.0, -3.0):
        qb = torch.full((148 * 100, 2 * hkv, hd), value, dtype=torch.bfloat16, device="cuda")
        B.dg_paged_attn(big, 148, 148 * 100, i32([100 * i for i in range(149)]), i32([0] * 148), qb, kv,
                        0, torch.empty_like(qb), ws)
        outs.append(torch.empty_like(qs))
        B.dg_paged_attn(cfg, seqs, seqs * n, off, lens, qs, many, 0, outs[-1], wide_ws)
    check_attention(outs[0][:n], q, c, [n], [have], 0, "bf16")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ----------------------------------------------------------------------------------- as used

def test_matches_canvas_attention():
    """The paged call and dg_canvas_attn on the same keys, fed by both forms of the norm and
    rotation, agree to their roundings."""
    g = gen(11)
    hq, hkv, hd, n, have, page = 16, 8, 128, 48, 200, 64
    cfg = make_cfg("bf16", hq, hkv, hd)
    qkv = randn(g, n, (hq + 2 * hkv) * hd).to(torch.bfloat16)
    gain = 1 + 0.3 * randn(g, hd)
    c = Cache(g, "bf16", hkv, hd, page, [have + n])
    lens = i32([have])
    q = torch.empty(1, n, hq, hd, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(1, hkv, n, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    B.dg_qk_norm_rope(cfg, 1, n, qkv, lens, gain, gain, None, q, k, v)
    qp = torch.empty(n, hq, hd, dtype=torch.bfloat16, device="cuda")
    B.dg_paged_append(cfg, 1, n, i32([0, n]), lens, qkv, gain, gain, None, c.kv, qp)
    assert torch.equal(qp, q[0])
    assert torch.equal(c.rows(c.k, 0, have, have + n).transpose(0, 1), k[0])
    kc = c.rows(c.k, 0, 0, have).transpose(0, 1).contiguous()[None]
    vc = c.rows(c.v, 0, 0, have).transpose(0, 1).contiguous()[None]
    c.kept[0] = (c.rows(c.k, 0, 0, have + n), c.rows(c.v, 0, 0, have + n))
    for causal in (0, 1):
        ref = torch.empty_like(q)
        B.dg_canvas_attn(cfg, 1, n, q, kc, vc, lens, have, k, v, causal, None, ref,
                         B.alloc_workspace(cfg, 1, n, have))
        out, st = run_attention(cfg, c, [n], [have], qp, causal)
        assert st == B.DG_OK
        want, A, e = P.attention(qp, *c.kept[0], causal, have)
        bound = P.attention_bound(want, A, e, have + n, torch.bfloat16, 2.0 ** -8)
        assert P.worst(out, want, bound) <= 1.0 and P.worst(ref[0], want, bound) <= 1.0


@pytest.mark.parametrize("act,hq,hkv,hd", [("bf16", 16, 8, 128), ("f32", 7, 1, 64)])
def test_prompt_then_tokens_then_canvases(act, hq, hkv, hd):
    """The calls as a server makes them: a long prompt appended and attended once, forked into
    continuations that share its pages, a token each over the shared prefix, then a canvas each;
    every step against the 64-bit forms over all the keys written so far."""
    g, dt, page = gen(21), DT[act], 32
    cfg = make_cfg(act, hq, hkv, hd)
    rng = random.Random(3)
    prompt, forks, canvas = 160, 5, 16
    table = torch.full((forks, 8), -1, dtype=torch.int32)
    table[:, :5] = torch.tensor([9, 3, 11, 0, 7], dtype=torch.int32)
    free = [1, 2, 4, 5, 6, 8, 10, 12, 13, 14]
    for s in range(forks):
        table[s, 5], table[s, 6] = free[2 * s], free[2 * s + 1]
    pools = [torch.full((15, hkv, page, hd), math.nan, device="cuda").to(dt) for _ in range(2)]
    kv = B.PagedKV(*pools, table.cuda())
    gains = [1 + 0.2 * randn(g, hd) for _ in range(2)]
    freq = P.frequencies(THETA, hd)
    rope = B.make_rope(hd)
    status = i32([0])
    keys = [(torch.empty(0, hkv, hd), torch.empty(0, hkv, hd)) for _ in range(forks)]
    lens = [0] * forks

    def step(new, causal, shared):
        off, rows = offsets(new), sum(new)
        qkv = randn(g, rows, (hq + 2 * hkv) * hd).to(dt)
        q = torch.empty(rows, hq, hd, dtype=dt, device="cuda")
        o, n_len = i32(off), i32(lens)
        B.dg_paged_append(cfg, len(new), rows, o, n_len, qkv, gains[0], gains[1], rope, kv, q, status)
        out = torch.empty_like(q)
        ws = B.alloc_paged_workspace(cfg, len(new), rows, shared)
        if shared:
            B.dg_prefix_attn(cfg, len(new), rows, o, n_len, shared, q, kv, causal, out, ws, status)
        else:
            B.dg_paged_attn(cfg, len(new), rows, o, n_len, q, kv, causal, out, ws, status)
        assert B.dg_read_status(status) == B.DG_OK
        x = qkv.view(rows, hq + 2 * hkv, hd)
        for s, n in enumerate(new):
            a, b = off[s], off[s + 1]
            pos = torch.arange(lens[s], lens[s] + n)
            wq, eq = P.norm_rope(x[a:b, :hq], gains[0], EPS, pos, freq, hd, "half", 1.0)
            wk, ek = P.norm_rope(x[a:b, hq:hq + hkv], gains[1], EPS, pos, freq, hd, "half", 1.0)
            check_rows(q[a:b], wq, eq, dt)
            pp = torch.arange(lens[s], lens[s] + n, device="cuda")
            ids = kv.page_table[s][pp // page].long()
            check_rows(pools[0][ids, :, pp % page], wk, ek, dt)
            # the attention on the stored values
            keys[s] = (torch.cat((keys[s][0], pools[0][ids, :, pp % page].float().cpu())),
                       torch.cat((keys[s][1], x[a:b, hq + hkv:].float().cpu())))
            if n:
                want, A, e = P.attention(q[a:b], *keys[s], causal, lens[s])
                bound = P.attention_bound(want, A, e, lens[s] + n, dt, 2.0 ** -8 if act == "bf16" else 0)
                assert P.worst(out[a:b], want, bound) <= 1.0
            lens[s] += n

    step([prompt, 0, 0, 0, 0], 1, 0)
    for s in range(1, forks):
        keys[s], lens[s] = keys[0], lens[0]
    for _ in range(3):
        step([1 if rng.random() < 0.8 else 0 for _ in range(forks)], 1, prompt)
    step([canvas] * forks, 0, prompt)
    step([1] * forks, 1, 0)


def test_captured_step_over_a_shared_prefix():
    """An append and a shared-prefix attention captured together, replayed as the sequences grow."""
    g, hq, hkv, hd, page, shared, seqs = gen(33), 16, 8, 128, 16, 64, 6
    cfg = make_cfg("bf16", hq, hkv, hd)
    c = Cache(g, "bf16", hkv, hd, page, [shared + 60] * seqs, shared=shared)
    for s in range(seqs):                                # only the prefix is there yet
        ids = c.table[s, shared // page:shared // page + 4].long()
        c.k[ids] = math.nan
        c.v[ids] = math.nan
    keys = [[k[:shared].clone(), v[:shared].clone()] for k, v in c.kept]
    rows = 24
    qkv = torch.zeros(rows, (hq + 2 * hkv) * hd, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(rows, hq, hd, dtype=torch.bfloat16, device="cuda")
    out, off, lens, st = torch.empty_like(q), i32([0] * (seqs + 1)), i32([shared] * seqs), i32([0])
    ws = B.alloc_paged_workspace(cfg, seqs, rows, shared)
    rope = B.make_rope(0)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        B.dg_paged_append(cfg, seqs, rows, off, lens, qkv, None, None, rope, c.kv, q, st)
        B.dg_prefix_attn(cfg, seqs, rows, off, lens, shared, q, c.kv, 1, out, ws, st)
    have = [shared] * seqs
    for new in ([1] * 6, [0, 10, 1, 0, 9, 4], [1, 1, 0, 1, 1, 1], [0] * 6, [2, 0, 3, 1, 0, 5]):
        qkv.copy_(randn(g, *qkv.shape).to(torch.bfloat16))
        off.copy_(i32(offsets(new)))
        lens.copy_(i32(have))
        out.fill_(MARK)
        gr.replay()
        assert B.dg_read_status(st) == B.DG_OK
        x = qkv.view(rows, hq + 2 * hkv, hd)
        for s, (a, n) in enumerate(zip(offsets(new), new)):
            keys[s][0] = torch.cat((keys[s][0], x[a:a + n, hq:hq + hkv]))
            keys[s][1] = torch.cat((keys[s][1], x[a:a + n, hq + hkv:]))
        c.kept = [tuple(kv) for kv in keys]
        check_attention(out, x[:, :hq].contiguous(), c, new, have, 1, "bf16")
        have = [h + n for h, n in zip(have, new)]


def test_captured_calls_follow_their_buffers():
    """A captured append and attention replayed with other lengths, offsets and rows in the same
    buffers; two graphs share one workspace in turn; an eager call in between changes nothing."""
    g, hq, hkv, hd, page = gen(31), 16, 8, 128, 16
    cfg = make_cfg("bf16", hq, hkv, hd)
    rows, seqs = 40, 4
    plans = [([1, 1, 1, 1], [30, 100, 7, 0]), ([20, 0, 3, 17], [0, 5, 200, 90]), ([1, 1, 0, 0], [255, 0, 0, 0])]
    c = Cache(g, "bf16", hkv, hd, page, [300] * seqs)
    q = torch.zeros(rows, hq, hd, dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(q), torch.empty_like(q)]
    off, lens, st = i32([0] * (seqs + 1)), i32([0] * seqs), i32([0])
    ws = B.alloc_paged_workspace(cfg, seqs, rows)
    graphs = []
    s = torch.cuda.Stream()
    for causal in (0, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            B.dg_paged_attn(cfg, seqs, rows, off, lens, q, c.kv, causal, outs[causal], ws, st)
        graphs.append(gr)
    for new, have in plans:
        off.copy_(i32(offsets(new)))
        lens.copy_(i32(have))
        q.copy_(randn(g, rows, hq, hd).to(torch.bfloat16))
        for o in outs:
            o.fill_(MARK)
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        B.dg_paged_attn(cfg, seqs, rows, off, lens, q, c.kv, 1, torch.empty_like(q), ws, st)
        torch.cuda.synchronize()
        assert B.dg_read_status(st) == B.DG_OK
        for causal in (0, 1):
            check_attention(outs[causal], q, c, new, have, causal, "bf16")


def test_own_stream_and_repeatable():
    """On a side stream, with a workspace of its own, twice: bit for bit the same."""
    g, hq, hkv, hd = gen(41), 16, 4, 128
    cfg = make_cfg("bf16", hq, hkv, hd)
    new, have = [1, 70, 1, 300], [900, 0, 20, 1000]
    c = Cache(g, "bf16", hkv, hd, 64, [n + h for n, h in zip(new, have)])
    q = randn(g, sum(new), hq, hd).to(torch.bfloat16)
    a, st = run_attention(cfg, c, new, have, q, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, st2 = run_attention(cfg, c, new, have, q, 1)
    s2 = torch.cuda.Stream()
    s2.wait_stream(s)
    out = torch.full_like(q, MARK)
    torch.cuda.synchronize()
    ws = B.alloc_paged_workspace(cfg, 4, sum(new))
    torch.cuda.synchronize()
    B.dg_paged_attn(cfg, 4, sum(new), i32(offsets(new)), i32(have), q, c.kv, 1, out, ws, None, s2)
    torch.cuda.synchronize()
    assert st == B.DG_OK and st2 == B.DG_OK
    assert torch.equal(a, b) and torch.equal(a, out)
    check_attention(a, q, c, new, have, 1, "bf16")
