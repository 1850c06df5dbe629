// Rows of a QKV projection on their way to the attention: per-head RMSNorm of queries and keys, the
// position rotation, and the split into q and either per-canvas K/V or the pages of a cache.
//
// The pages of the method give no position scheme; a canvas continues its cached context
// ("DiffusionGemma Technical Report", Figure 4), so token i of sequence b stands at position
// len[b] + i.  For a head x of q or k (all in fp32, rounded once to the activation type):
//   y = x / sqrt(mean(x^2) + eps) * gain                 (where a gain is given)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)         for each pair (a, b) of the rotated part
// with c, s = mscale * cos, sin(position * f_j).  v passes unchanged.
//
// Bound: HBM (each row is read and written once; about 5 operations a byte).  A lane holds 16
// elements of a head as two 16-byte chunks chosen so that every pair lies within the lane, for
// both pair layouts; hd / 16 lanes make a head, so the norm is 1 to 3 shuffles and a warp works on
// 4 heads of 128 at a time.  A block shares the cosines and sines of its tokens in shared memory,
// each computed once.
//
// The angle is a product of an integer position and a frequency, taken in fp64 as turns and
// reduced to [-1/2, 1/2] before the fp32 sine (an fp32 angle at position 131072 would be off by
// 1e-2 rad); the part of the reduced angle that fp32 drops is added back to first order.
#include <cmath>

#include "dg_common.cuh"
#include "dg_kernels.h"
#include "tc_host.h"

namespace dg {

namespace {

constexpr int Q_THR = 256;
constexpr int Q_TOK = 16;        // tokens per block at most
constexpr int Q_MAX_PAIRS = 64;  // head_dim <= 128

struct QkvArgs {
  const void *qkv;
  long long ld;                  // elements between rows
  int n_tokens, n_seqs, n;       // n > 0: uniform rows per sequence (seq_off unused)
  int block_tokens;              // tokens per block
  const int32_t *seq_off, *len;
  int Hq, Hkv, rot, interleaved;
  float eps, mscale;
  const float *q_gain, *k_gain;
  void *q, *k, *v;               // q [n_tokens][Hq][hd]; uniform: k, v [n_seqs][Hkv][n][hd]
  void *k_pages, *v_pages;
  const int32_t *page_table;
  int n_pages, max_pages, page_shift;
  int32_t *status;
  double turn[Q_MAX_PAIRS];      // frequency of each pair in turns per position
};

template <typename T> struct Chunk;   // 8 elements of an activation type <-> fp32
template <> struct Chunk<bf16> {
  uint4 raw;
  __device__ void load(const bf16 *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
};
template <> struct Chunk<float> {
  float4 a, b;
  __device__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
};

struct TokenSpot {
  int row;               // packed row, -1: none
  long long kv_row;      // K/V row of kv head 0 (in rows of hd), -1: not written
};

// Where packed row t goes, found by one whole warp (32 sequences at a time).
__device__ __forceinline__ TokenSpot packed_spot(const QkvArgs &a, int t, int *pos_out) {
  const int lane = threadIdx.x & 31;
  TokenSpot sp{-1, -1};
  // last sequence that begins at or before row t: 32-way search
  int lo = 0, hi = a.n_seqs;
#pragma unroll 1
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool le = i < hi && (i == lo || a.seq_off[i] <= t);
    const int l = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += l * step;
    hi = min(hi, lo + step);
  }
  const int o0 = a.seq_off[lo], o1 = a.seq_off[lo + 1], have = a.len[lo];
  if (o0 > t || t >= o1) return sp;   // no sequence's row
  if (o0 < 0 || o1 > a.n_tokens || have < 0) return sp;   // (recorded by the thread that checks it)
  sp.row = t;
  // (a position past 2^31 is past every cache: its q is rotated by the wrapped position)
  const int pos = (int)((uint32_t)have + (uint32_t)(t - o0));
  *pos_out = pos;
  if ((long long)have + (o1 - o0) > ((long long)a.max_pages << a.page_shift)) {
    if (lane == 0) set_status(a.status, DG_ERR_CAPACITY);
    return sp;
  }
  const int id = a.page_table[(size_t)lo * a.max_pages + (pos >> a.page_shift)];
  if ((unsigned)id >= (unsigned)a.n_pages) {
    if (lane == 0) set_status(a.status, DG_ERR_INVALID_ARG);
    return sp;
  }
  sp.kv_row = (((long long)id * a.Hkv) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  return sp;
}

template <typename T, int HD>
__global__ void __launch_bounds__(Q_THR) qkv_rows_kernel(const __grid_constant__ QkvArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int LPH = HD / 16;                 // lanes per head
  constexpr int SLOTS = Q_THR / LPH;           // heads in flight in a block
  __shared__ TokenSpot spot[Q_TOK];
  __shared__ int pos_s[Q_TOK];
  // (c, s) of the 8 pairs of lane l: two pairs per float4, entry [token][pair couple][lane]
  __shared__ float4 cs[Q_TOK][4][LPH];
  const int tid = threadIdx.x, t0 = blockIdx.x * a.block_tokens;
  const int head_stride = a.n > 0 ? a.n : 1 << a.page_shift;   // K/V rows between kv heads
  const int l = tid % LPH, slot = tid / LPH;
  const int heads = a.Hq + 2 * a.Hkv;
  // The lane's two chunks of 8 elements: in the rotated part chunk l and its partner half a
  // rotation further on, so that both layouts' pairs stay within the lane; the rest in order.
  const int rl = a.rot / 16;
  const int ca = l < rl ? l : 2 * rl + 2 * (l - rl);
  const int cb = l < rl ? l + rl : ca + 1;
  const int toks = min(a.block_tokens, a.n_tokens - t0), work = toks * heads;
  // The rows are read a step ahead: their place does not depend on the sequences, so the first
  // are under way while those are searched and the angles computed.
  Chunk<T> A, B;
  int tk = slot / heads, h = slot % heads;
  const T *src = (const T *)a.qkv + (size_t)(t0 + tk) * a.ld + (size_t)h * HD;
  if (slot < work) {
    A.load(src + ca * 8);
    B.load(src + cb * 8);
  }
  // Sequences that no row reaches are checked too, a thread each, from the warps that have no token in
  // a small call.
  if (a.n == 0) {
#pragma unroll 1
    for (long long s = (long long)blockIdx.x * Q_THR + Q_THR - 1 - tid; s < a.n_seqs;
         s += (long long)gridDim.x * Q_THR) {
      const int o0 = a.seq_off[s], o1 = a.seq_off[s + 1];
      if (o0 != o1 && (o0 < 0 || o1 < o0 || o1 > a.n_tokens || a.len[s] < 0))
        set_status(a.status, DG_ERR_INVALID_ARG);
    }
  }
  {
    // a warp per token
#pragma unroll 1
    for (int w = tid >> 5; w < toks; w += Q_THR / 32) {
      const int t = t0 + w;
      TokenSpot sp;
      int pos = 0;
      if (a.n > 0) {
        const int b = t / a.n, i = t % a.n;
        const int have = a.len[b];
        sp.row = have < 0 ? -1 : t;
        sp.kv_row = have < 0 ? -1 : (long long)b * a.Hkv * a.n + i;
        if (have < 0 && (tid & 31) == 0) set_status(a.status, DG_ERR_INVALID_ARG);
        pos = (int)((uint32_t)have + (uint32_t)i);
      } else {
        sp = packed_spot(a, t, &pos);
      }
      if ((tid & 31) == 0) {
        spot[w] = sp;
        pos_s[w] = pos;
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int e = tid; e < toks * (a.rot / 2); e += Q_THR) {
    const int k = e / (a.rot / 2), x = e % (a.rot / 2), lane = x / 8, u = x % 8;
    // pair u of rotated lane `lane`
    const int j = !a.interleaved ? 8 * lane + u
                  : u < 4        ? 4 * lane + u
                                 : 4 * (lane + rl) + u - 4;
    const double turns = (double)pos_s[k] * a.turn[j];
    const double r = turns - rint(turns);
    const float rf = (float)r;
    const float d = (float)(r - (double)rf) * 6.283185307179586f;
    float sn, co;
    sincospif(2.f * rf, &sn, &co);
    float *o = reinterpret_cast<float *>(&cs[k][u >> 1][lane]) + 2 * (u & 1);
    o[0] = (co - sn * d) * a.mscale;
    o[1] = (sn + co * d) * a.mscale;
  }
  __syncthreads();

#pragma unroll 1
  for (int w = slot; w < work; w += SLOTS) {
    Chunk<T> A2, B2;
    int h2 = h + SLOTS, tk2 = tk;
    while (h2 >= heads) {
      h2 -= heads;
      ++tk2;
    }
    if (w + SLOTS < work) {
      src = (const T *)a.qkv + (size_t)(t0 + tk2) * a.ld + (size_t)h2 * HD;
      A2.load(src + ca * 8);
      B2.load(src + cb * 8);
    }
    const TokenSpot sp = spot[tk];
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
    const float *gain = is_q ? a.q_gain : is_v ? nullptr : a.k_gain;
    if (!is_v) {
      float x[8], y[8];
      A.get(x);
      B.get(y);
      if (gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
        // the lanes of a head run together: they share w, h and so this branch
        const unsigned mask = ((1u << LPH) - 1u) << ((tid & 31) / LPH * LPH);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float rs = rsqrtf(ss * (1.f / HD) + a.eps);
        Chunk<float> ga, gb;
        float g[8];
        ga.load(gain + ca * 8);
        gb.load(gain + cb * 8);
        ga.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= rs * g[i];
        gb.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= rs * g[i];
      }
      if (l < rl) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 c = cs[tk][i][l];       // (c, s) of pairs 2 i and 2 i + 1
          if (!a.interleaved) {
            const float x0 = x[2 * i], x1 = x[2 * i + 1];
            x[2 * i] = x0 * c.x - y[2 * i] * c.y;
            y[2 * i] = y[2 * i] * c.x + x0 * c.y;
            x[2 * i + 1] = x1 * c.z - y[2 * i + 1] * c.w;
            y[2 * i + 1] = y[2 * i + 1] * c.z + x1 * c.w;
          } else {
            float *z = i < 2 ? x + 4 * i : y + 4 * (i - 2);
            const float z0 = z[0], z2 = z[2];
            z[0] = z0 * c.x - z[1] * c.y;
            z[1] = z[1] * c.x + z0 * c.y;
            z[2] = z2 * c.z - z[3] * c.w;
            z[3] = z[3] * c.z + z2 * c.w;
          }
        }
      }
      A.set(x);
      B.set(y);
    }
    T *dst = nullptr;
    if (is_q) {
      if (sp.row >= 0 && a.q) dst = (T *)a.q + ((size_t)sp.row * a.Hq + h) * HD;
    } else if (sp.kv_row >= 0) {
      const int g = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
      T *base = (T *)(a.n > 0 ? (is_v ? a.v : a.k) : (is_v ? a.v_pages : a.k_pages));
      dst = base + (sp.kv_row + (long long)g * head_stride) * HD;
    }
    if (dst) {
      A.store(dst + ca * 8);
      B.store(dst + cb * 8);
    }
    A = A2;
    B = B2;
    h = h2;
    tk = tk2;
  }
}

// Frequencies theta^(-2j / rot), scaled, in turns per position.  A running product in extended
// precision: 64 factors keep the relative error near 2^-58.
void fill_turns(const RopeSpec &r, double *turn) {
  const long double per_turn = 0.159154943091895335768883763372514L;   // 1 / 2 pi
  const long double ratio = r.rot > 0 ? powl((long double)r.theta, -2.0L / r.rot) : 1.0L;
  long double f = 1.0L;
  for (int j = 0; j < r.rot / 2; ++j, f *= ratio) {
    long double w = f;
    if (r.scaling == DG_ROPE_LINEAR) {
      w = f / r.factor;
    } else if (r.scaling == DG_ROPE_BY_PARTS) {
      // "NTK-by-parts" interpolation (Peng et al., 2023, "YaRN"): pairs that turn more than
      // beta_fast times over the original length keep their frequency, those below beta_slow
      // turns are interpolated, a ramp in between
      const long double turns = r.orig_len * f * per_turn;
      long double keep = (turns - r.beta_slow) / (r.beta_fast - r.beta_slow);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      w = f / r.factor * (1 - keep) + f * keep;
    }
    turn[j] = (double)(w * per_turn);
  }
}

}  // namespace

int launch_qkv_rows(const QkvCall &c, cudaStream_t s) {
  QkvArgs a{};
  a.qkv = c.qkv;
  a.ld = c.ld;
  a.n_tokens = c.n_tokens;
  a.n_seqs = c.n_seqs;
  a.n = c.n;
  a.seq_off = c.seq_off;
  a.len = c.len;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.rot = c.rope.rot;
  a.interleaved = c.rope.interleaved;
  a.eps = (float)c.eps;
  a.mscale = (float)c.rope.mscale;
  a.q_gain = c.q_gain;
  a.k_gain = c.k_gain;
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.k_pages = c.k_pages;
  a.v_pages = c.v_pages;
  a.page_table = c.page_table;
  a.n_pages = c.n_pages;
  a.max_pages = c.max_pages;
  while ((1 << a.page_shift) < c.page_size) ++a.page_shift;
  a.status = c.status;
  fill_turns(c.rope, a.turn);
  // few tokens: a block each, so that every head of a call for single tokens is in flight at once
  // (four blocks fit an SM); many: whole waves of blocks
  const int spread = 4 * num_sms(), waves = (c.n_tokens - 1) / (spread * Q_TOK) + 1;
  a.block_tokens = (c.n_tokens - 1) / (spread * waves) + 1;
  const int grid = (c.n_tokens + a.block_tokens - 1) / a.block_tokens;
  note_launch(s, "qkv_rows");
#define DG_QKV_CASE(T, HD) launch_pdl(qkv_rows_kernel<T, HD>, grid, Q_THR, 0, s, a)
  if (c.act == DG_F32) {
    if (c.hd == 32) DG_QKV_CASE(float, 32);
    else if (c.hd == 64) DG_QKV_CASE(float, 64);
    else DG_QKV_CASE(float, 128);
  } else {
    if (c.hd == 32) DG_QKV_CASE(bf16, 32);
    else if (c.hd == 64) DG_QKV_CASE(bf16, 64);
    else DG_QKV_CASE(bf16, 128);
  }
#undef DG_QKV_CASE
  return check_launch("qkv_rows");
}

}  // namespace dg
