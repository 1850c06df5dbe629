"""The paged-cache operators restated plainly in 64 bits on the host, with the bounds their results
are held to.

Bounds count roundings (u = 2^-24 for an fp32 operation, h = eps / 2 of the storage type for the one
rounding of a result, e.g. 2^-8 for bf16):
* a normed and rotated element a c - b s: h |o| + (hd + 64) u (|a| + |b|) mscale.  The sum of hd
  squares is off by at most hd u relative, and the square root, the gain, the products and the fp32
  sine (2 ulp, plus 2 u from the angle's own rounding) take fewer than 64 further half steps.
* an attention output: h |o| + c A with A = sum_j p_j |v_j| (p normalised).  A score is off by at most
  e = (hd + 8) u sum |q k| / sqrt(hd), which changes p by a relative e, numerator and denominator
  each; storing p in bf16 for the tensor cores adds h_p = 2^-8 to the numerator; the sums over n keys
  add n 2u each (tensor-core sums may truncate), and the exponentials, rescalings and joins of up to
  128 pieces stay below 2^-16: c = h_p + 2 max e + 4 n u + 2^-16.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def frequencies(theta, rot, scaling="none", factor=1.0, orig_len=0.0, slow=1.0, fast=32.0):
    f = []
    for j in range(rot // 2):
        w = theta ** (-2.0 * j / rot)
        if scaling == "linear":
            w = w / factor
        elif scaling == "by_parts":
            r = (orig_len * w / (2 * math.pi) - slow) / (fast - slow)
            r = min(1.0, max(0.0, r))
            w = w / factor * (1 - r) + w * r
        f.append(w)
    return torch.tensor(f, dtype=torch.float64)


def norm_rope(x, gain, eps, pos, freq, rot, layout, mscale):
    """x [rows, heads, hd] any type, pos [rows]; returns (values, bound without the h |o| term)."""
    x = x.double().cpu()
    hd = x.shape[-1]
    if gain is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * gain.double().cpu()
    y, mag = x.clone(), x.abs()
    ang = pos.double().cpu()[:, None, None] * freq
    c, s = torch.cos(ang) * mscale, torch.sin(ang) * mscale
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(mscale)
    return y, (hd + 64) * U * mag


def attention(q, k, v, causal, have):
    """q [n, hq, hd], k and v [keys, hkv, hd] stored values; `have` keys stand before the first of the
    n new ones.  Returns (values, A, e): see the bound above."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    n, hq, hd = q.shape
    rep = hq // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    s = torch.einsum("nhd,khd->hnk", q, k) / math.sqrt(hd)
    e = torch.einsum("nhd,khd->hnk", q.abs(), k.abs()) / math.sqrt(hd) * (hd + 8) * U
    if causal:
        hide = torch.arange(k.shape[0])[None, :] > have + torch.arange(n)[:, None]
        s = s.masked_fill(hide, -math.inf)
        e = e.masked_fill(hide, 0.0)
    p = torch.softmax(s, -1)
    out = torch.einsum("hnk,khd->nhd", p, v)
    return out, torch.einsum("hnk,khd->nhd", p, v.abs()), e.amax(-1).transpose(0, 1)[..., None]


def attention_bound(out, A, e, keys, dtype, p_bits):
    return HALF[dtype] * out.abs() + (p_bits + 2 * e + 4 * keys * U + 2.0 ** -16) * A


def worst(got, want, bound):
    """Largest error in units of its bound (<= 1 passes; NaN does not)."""
    if want.numel() == 0:
        return 0.0
    d = (got.double().cpu() - want).abs() / (bound + 1e-30)
    return math.inf if torch.isnan(d).any() else float(d.max())
