// Attention of packed sequences over a paged K/V cache: the CUDA-core kernel (fp32 activations,
// and bf16 with heads of 32) and the kernels that join partial results.
//
// "DiffusionGemma Technical Report", Figure 4: a prompt is encoded causally into a K/V cache and a
// canvas attends to it bidirectionally; the cache here lies in pages, and sequences of different
// lengths share a launch (paged_plan.cuh splits the work).
//   o = softmax(q K^T / sqrt(hd)) V,  with t = q.k / sqrt(hd) * log2(e):
//   m = max t, l = sum 2^(t - m), O = sum 2^(t - m) v, out = O / l
// and partial results of disjoint key sets join as m = max m_i, l = sum l_i 2^(m_i - m),
// O = sum O_i 2^(m_i - m).  Scores, statistics and O are fp32; the output is rounded once.
#include "dg_common.cuh"
#include "dg_kernels.h"
#include "paged_attn.cuh"
#include "tc_host.h"

namespace dg {

namespace {

constexpr int S_ROWS = 64, S_KT = 64, S_THR = 256;

template <int HD>
constexpr size_t simt_smem() {
  return (size_t)(2 * S_ROWS * (HD + 4) + S_ROWS * (S_KT + 4)) * sizeof(float);
}

// Four consecutive elements as fp32.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const bf16 *p) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162 *>(&v.x);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&v.y);
  return make_float4(__low2float(a), __high2float(a), __low2float(b), __high2float(b));
}

// One CTA walks its range of (item, key tile) units: 64 query rows (token-major, the heads of a
// group within a token) against tiles of 64 keys.  Thread (tx, ty) of 16 x 16 holds rows 4 ty ..
// 4 ty + 3: scores of keys tx + 16 j, then output columns.  K and V take turns in one tile buffer,
// so that two CTAs fit an SM.
template <typename T, int HD>
__global__ void __launch_bounds__(S_THR, 2) paged_attn_simt_kernel(const __grid_constant__ PagedShape p,
                                                                  const __grid_constant__ PagedIO io) {
  pdl_wait();
  pdl_trigger();
  constexpr int LD = HD + 4, LP = S_KT + 4;   // padded rows: conflict-free float4 reads
  constexpr int DPT = HD / 16, VEC = DPT < 4 ? DPT : 4, NV = DPT / VEC;
  extern __shared__ __align__(16) float simt_smem_raw[];
  float *Qs = simt_smem_raw, *KVs = Qs + S_ROWS * LD, *Ps = KVs + S_KT * LD;
  __shared__ PagedStart start[1];
  __shared__ PagedScan scan;
  __shared__ int row_s[2][S_KT];   // rows of a tile's keys in the pool, -1: none (tiles in turn)
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int err = paged_locate<S_THR, 1>(p, blockIdx.x, gridDim.x, 1, start, io.heads, scan);
  __syncthreads();
  const PagedStart st = start[0];
  if (tid == 0 && blockIdx.x == 0) paged_report(io, err);
  const int rep = io.rep;
  const float sl2 = 1.4426950408889634f * rsqrtf((float)HD);
  PagedWalk w;
  for (w.begin(p, PAGED_WIDE, st); w.more(); w.next(p)) {
    const PagedSeg s = w.s;
    const int i0 = w.tok, toks = w.toks, rows = toks * rep, item_keys = w.keys;
    __syncthreads();  // the last piece's readers of Qs and the row list are done
    for (int e = tid; e < S_ROWS * (HD / 4); e += S_THR) {
      const int r = e / (HD / 4), c = e % (HD / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = load4((const T *)io.q + ((size_t)(s.tok0 + i0 + paged_token(io, r)) * io.Hq + w.head * rep +
                                     r - paged_token(io, r) * rep) * HD + c);
      *reinterpret_cast<float4 *>(&Qs[r * LD + c]) = v;
    }
    float o[4][DPT], m[4], l[4];
    int lim[4];  // keys this row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
      lim[i] = s.causal ? s.keys - s.n + i0 + min(paged_token(io, r), toks - 1) + 1 : s.keys;
#pragma unroll
      for (int d = 0; d < DPT; ++d) o[i][d] = 0.f;
    }
    // K and V of a tile pass through registers on their way to the one buffer: V is read while the
    // scores are computed, the next tile's K while P V is; the pages are looked up a tile ahead.
    constexpr int NE = S_KT * (HD / 4) / S_THR;   // 4-element groups of a tile per thread
    float4 pre[NE];
    auto look_up = [&](int t) {
      if (tid < S_KT) {
        const int j = t * S_KT + tid;
        row_s[t & 1][tid] =
            t < w.t1 && j < item_keys ? (int)paged_row(io, p, s.seq, w.head, s.key0 + j) : -1;
      }
    };
    auto fetch = [&](const void *pages, int t) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = tid + i * S_THR, row = row_s[t & 1][e / (HD / 4)];
        pre[i] = row >= 0 ? load4((const T *)pages + (size_t)row * HD + e % (HD / 4) * 4)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    auto put = [&]() {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = tid + i * S_THR;
        *reinterpret_cast<float4 *>(&KVs[e / (HD / 4) * LD + e % (HD / 4) * 4]) = pre[i];
      }
    };
    look_up(w.t0);
    __syncthreads();
    fetch(io.k_pages, w.t0);
    for (int t = w.t0; t < w.t1; ++t) {
      const int j0 = t * S_KT;
      __syncthreads();   // the last P V has read the buffer
      put();
      look_up(t + 1);
      fetch(io.v_pages, t);
      __syncthreads();
      if ((tid >> 5) * 8 < rows) {   // warps without rows only load
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < HD; d += 4) {
          float4 a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4 *>(&Qs[(ty * 4 + i) * LD + d]);
            b[i] = *reinterpret_cast<const float4 *>(&KVs[(tx + 16 * i) * LD + d]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              sc[i][j] = fmaf(a[i].x, b[j].x, sc[i][j]);
              sc[i][j] = fmaf(a[i].y, b[j].y, sc[i][j]);
              sc[i][j] = fmaf(a[i].z, b[j].z, sc[i][j]);
              sc[i][j] = fmaf(a[i].w, b[j].w, sc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mt = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sc[i][j] = j0 + tx + 16 * j < lim[i] ? sc[i][j] * sl2 : -INFINITY;
            mt = fmaxf(mt, sc[i][j]);
          }
#pragma unroll
          for (int b = 8; b > 0; b >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, b));
          const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;
          const float f = exp2f(m[i] - base);
          m[i] = mn;
          float ps = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = exp2f(sc[i][j] - base);
            ps += e;
            Ps[(ty * 4 + i) * LP + tx + 16 * j] = e;
          }
#pragma unroll
          for (int b = 8; b > 0; b >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, b);
          l[i] = l[i] * f + ps;
#pragma unroll
          for (int d = 0; d < DPT; ++d) o[i][d] *= f;
        }
      }
      __syncthreads();   // every thread has read K
      put();
      if (t + 1 < w.t1) fetch(io.k_pages, t + 1);
      __syncthreads();
      if ((tid >> 5) * 8 >= rows) continue;
#pragma unroll 2
      for (int k = 0; k < S_KT; k += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pr[i] = *reinterpret_cast<const float4 *>(&Ps[(ty * 4 + i) * LP + k]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float v[DPT];
#pragma unroll
          for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int y = 0; y < VEC; ++y) v[x * VEC + y] = KVs[(k + kk) * LD + x * 16 * VEC + tx * VEC + y];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pv = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
#pragma unroll
            for (int d = 0; d < DPT; ++d) o[i][d] = fmaf(pv, v[d], o[i][d]);
          }
        }
      }
    }
    const PagedDest dest = paged_dest(p, io, w, blockIdx.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      const int tl = paged_token(io, r), tok = s.tok0 + i0 + tl, h = w.head * rep + r - tl * rep;
      if (dest.kind == PAGED_OUT) {
        const float il = l[i] > 0.f ? 1.f / l[i] : 0.f;
        T *dst = (T *)io.out + ((size_t)tok * io.Hq + h) * HD;
#pragma unroll
        for (int d = 0; d < DPT; ++d)
          dst[d / VEC * 16 * VEC + tx * VEC + d % VEC] = from_f<T>(o[i][d] * il);
      } else {
        const size_t row = paged_part_row(p, io, dest, r, tok, h);
#pragma unroll
        for (int d = 0; d < DPT; ++d)
          io.part_o[row * HD + d / VEC * 16 * VEC + tx * VEC + d % VEC] = o[i][d];
        if (tx == 0) {
          io.part_ml[row] = make_float2(m[i], l[i]);
          if (dest.redirect) paged_redirect(p, io, dest, blockIdx.x, tok, h);
        }
      }
    }
  }
}

// ---- joining ------------------------------------------------------------------------------------

// A row's running state while its partial results are folded in, one warp per row; lane i holds
// columns i V .. i V + V - 1.
template <int HD>
struct Fold {
  static constexpr int V = HD / 32;
  float m = -INFINITY, l = 0.f, acc[V];
  __device__ Fold() {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
  }
  // n partial results, lane i of `ml` holding the i-th's (m, l), `row` its row in part_o.
  __device__ __forceinline__ void add(const float *__restrict__ part_o, int n, float2 ml,
                                      size_t row) {
    const int lane = threadIdx.x & 31;
    constexpr int U = 8;   // rows in flight
    float x[U][V];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const size_t r = __shfl_sync(0xffffffffu, row, min(i0 + i, n - 1));
#pragma unroll
        for (int v = 0; v < V; ++v) x[i][v] = i0 + i < n ? part_o[r * HD + lane * V + v] : 0.f;
      }
    };
    load(0);   // (before the statistics are asked for: one latency, not two)
    const float mn = fmaxf(m, warp_max(lane < n ? ml.x : -INFINITY));
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - base);
    const float c = lane < n ? exp2f(ml.x - base) : 0.f;
    m = mn;
    l = l * f + warp_sum(lane < n ? c * ml.y : 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= f;
    for (int i0 = 0; i0 < n; i0 += U) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float ci = __shfl_sync(0xffffffffu, c, (i0 + i) & 31);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = i0 + i < n ? fmaf(x[i][v], ci, acc[v]) : acc[v];
      }
    }
  }
  // Row r of the item that begins at worker `begin`, its pieces with workers first .. last.
  __device__ __forceinline__ void add_range(const PagedIO &io, int begin, int first, int last, int r) {
    const int lane = threadIdx.x & 31;
    for (int c0 = first; c0 <= last; c0 += 32) {
      const int n = min(32, last - c0 + 1);
      const int c = c0 + min(lane, n - 1);
      const size_t row = paged_slot_row(io, c, c == begin, r);
      add(io.part_o, n, io.part_ml[row], row);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T *dst) const {
    const float il = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) dst[(threadIdx.x & 31) * V + v] = from_f<T>(acc[v] * il);
  }
};

// NR rows at once, each of NS partial results (NR x NS loads in flight).  row[i][k]: rows of
// part_o, on: whether they count; dst[i]: output row, or null.
template <typename T, int HD, int NR, int NS>
__device__ __forceinline__ void join_some(const PagedIO &io, const size_t (&row)[NR][NS],
                                          const bool (&on)[NR][NS], T *const (&dst)[NR]) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31;
  float2 ml[NR][NS];
  float x[NR][NS][V];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      ml[i][k] = io.part_ml[row[i][k]];
#pragma unroll
      for (int v = 0; v < V; ++v) x[i][k][v] = io.part_o[row[i][k] * HD + lane * V + v];
    }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (!dst[i]) continue;
    float m = -INFINITY, l = 0.f, y[V] = {};
#pragma unroll
    for (int k = 0; k < NS; ++k)
      if (on[i][k]) m = fmaxf(m, ml[i][k].x);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      if (!on[i][k]) continue;
      const float c = exp2f(ml[i][k].x - base);
      l = fmaf(ml[i][k].y, c, l);
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = fmaf(x[i][k][v], c, y[v]);
    }
    const float il = l > 0.f ? 1.f / l : 0.f;
    T *d = dst[i] + lane * V;
    if constexpr (V == 4) store4<T>(d, y[0] * il, y[1] * il, y[2] * il, y[3] * il);
    else
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = from_f<T>(y[v] * il);
  }
}

// Joins the items that range boundaries cut.  The workers that go on with an item share its rows:
// of wide items each has two blocks, of narrow ones one, of few-row ones eight have one.  Where an
// item of few rows was cut for many workers (one long context), the warps of a block share the
// pieces of a row and join once more through shared memory; else a warp takes whole rows. (Blocks
// are few on purpose: most have nothing to do, and a thousand of them cost more than the joining.)
struct JoinBlocks {
  int wide, few;   // blocks for wide and few-row items; the rest are for narrow ones
};
template <typename T, int HD>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedIO io, JoinBlocks blocks) {
  pdl_wait();
  pdl_trigger();
  __shared__ float acc_s[8][HD];
  __shared__ float2 ml_s[8];
  constexpr int MANY = 16;   // pieces worth sharing
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blocks: two for each wide worker, one for eight few-row ones, one for each narrow one
  const int b_few = blockIdx.x - blocks.wide, b_narrow = b_few - blocks.few;
  const bool few = b_few >= 0 && b_narrow < 0;
  const int shares = b_few < 0 ? 2 : 1;   // blocks of a wide or narrow worker
  const int c0 = b_few < 0 ? blockIdx.x / 2 : few ? 3 * io.ctas + b_few * 8 : io.ctas + b_narrow;
  const int c = few ? c0 + warp : c0, base = paged_first_worker(io, paged_worker_kind(io, c));
  auto out = [&](const PagedHead &h, int r) {
    const int tl = paged_token(io, r);
    return (T *)io.out + ((size_t)(h.tok0 + tl) * io.Hq + h.head * io.rep + r - tl * io.rep) * HD;
  };
  // few-row items: lane i holds the head of the block's worker i (one after the other, these loads
  // were a good part of a short call's join)
  PagedHead mine{};
  if (few && lane < 8) mine = io.heads[c0 + lane];
  auto head_of = [&](int w) {
    PagedHead h{};
    h.first = __shfl_sync(0xffffffffu, mine.first, w);
    h.last = __shfl_sync(0xffffffffu, mine.last, w);
    h.tok0 = __shfl_sync(0xffffffffu, mine.tok0, w);
    h.tokens = __shfl_sync(0xffffffffu, mine.tokens, w);
    h.head = __shfl_sync(0xffffffffu, mine.head, w);
    return h;
  };
  {
    const PagedHead h = few ? head_of(warp) : io.heads[c];
    const int rows = h.first >= 0 ? h.tokens * io.rep : 0, n = h.last - h.first + 1;
    const int begin = base + h.first;
    // this warp's rows r0, r0 + step, ... of the item's shares
    int r0 = c - begin - 1, step = n - 1;
    if (!few) {
      r0 = (r0 * shares + (shares == 2 ? blockIdx.x & 1 : 0)) * 8 + warp;
      step *= 8 * shares;
    }
    if (n == 2) {
      constexpr int NR = 4;
#pragma unroll 1
      for (; r0 < rows; r0 += NR * step) {
        size_t row[NR][2];
        bool on[NR][2];
        T *dst[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = r0 + i * step, rr = min(r, rows - 1);
          row[i][0] = paged_slot_row(io, begin, true, rr);
          row[i][1] = paged_slot_row(io, begin + 1, false, rr);
          on[i][0] = on[i][1] = true;
          dst[i] = r < rows ? out(h, r) : nullptr;
        }
        join_some<T, HD, NR, 2>(io, row, on, dst);
      }
    } else if (!few || n <= MANY) {
#pragma unroll 1
      for (; r0 < rows; r0 += step) {
        Fold<HD> f;
        f.add_range(io, begin, begin, begin + n - 1, r0);
        f.store(out(h, r0));
      }
    }
  }
  if (!few) return;
  // few-row items of many pieces: this block's part of their rows
  // (once per block and item: with the first of the block's workers that goes on with it)
  unsigned todo = __ballot_sync(0xffffffffu, lane < 8 && mine.first >= 0 && mine.last - mine.first >= MANY &&
                                                 (lane == 0 || base + mine.first >= c0 + lane - 1));
#pragma unroll 1
  for (; todo; todo &= todo - 1) {
    const PagedHead h = head_of(__ffs(todo) - 1);
    const int n = h.last - h.first + 1, begin = base + h.first;
    // blocks that hold such workers
    const int b0 = (begin + 1 - 3 * io.ctas) / 8, b1 = (begin + n - 1 - 3 * io.ctas) / 8;
    const int rows = h.tokens * io.rep, per = (n + 7) / 8;
    const int p0 = min(warp * per, n), p1 = min(p0 + per, n);
    for (int r = (c0 - 3 * io.ctas) / 8 - b0; r < rows; r += b1 - b0 + 1) {
      Fold<HD> f;
      f.add_range(io, begin, begin + p0, begin + p1 - 1, r);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < Fold<HD>::V; ++v) acc_s[warp][lane * Fold<HD>::V + v] = f.acc[v];
      if (lane == 0) ml_s[warp] = make_float2(f.m, f.l);
      __syncthreads();
      if (warp == 0) {
        Fold<HD> g;
        g.add(&acc_s[0][0], 8, ml_s[min(lane, 7)], min(lane, 7));
        g.store(out(h, r));
      }
    }
  }
}

// Joins each row's result over the shared prefix with the one over its own keys; either may have
// been cut into pieces.  A warp takes NR query heads of a packed row.  A small call's time is the
// length of the chain of loads that depend on one another, so its warps take one head each (128
// single tokens over 8192 shared keys, the whole call: 50 us with two heads a warp, 40 with one;
// 1024 tokens: 177 and 181).  The pieces of a row are folded together, up to 32 at once.
template <typename T, int HD, int NR>
__global__ void __launch_bounds__(256, NR == 1 ? 3 : 4) paged_join_prefix_kernel(const __grid_constant__ PagedShape p,
                                                                const __grid_constant__ PagedIO io) {
  pdl_wait();
  pdl_trigger();
  constexpr int NS = 4;
  constexpr unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int groups = (io.Hq + NR - 1) / NR;
  const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int tok = (int)(task / groups), h0 = (int)(task % groups) * NR;
  if (tok >= p.n_tokens) return;
  const int refused = io.heads[0].refused;   // the region was not written then
  // what the region says of the rows, while the sequence is searched
  float2 ml[NR][2];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      ml[i][k] = io.part_ml[paged_region_row(p, io, k, tok, min(h0 + i, io.Hq - 1))];
  // the sequence that holds this row, if it is one the attention took: 32-way search
  int lo = 0, hi = p.n_seqs;
#pragma unroll 1
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool le = i < hi && (i == lo || p.seq_off[i] <= tok);
    const int l = 31 - __clz(__ballot_sync(full, le));
    lo += l * step;
    hi = min(hi, lo + step);
  }
  const PagedSeg s = paged_seg(p, lo + 1);
  if (refused || s.n == 0 || tok < s.tok0 || tok >= s.tok0 + s.n) return;
  // the pieces of each row: over the prefix (k = 0) and over its own keys
  size_t row[NR][NS];
  bool on[NR][NS], many = false;
  T *dst[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int h = min(h0 + i, io.Hq - 1), hr = h % io.rep;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      row[i][2 * k] = row[i][2 * k + 1] = paged_region_row(p, io, k, tok, h);
      on[i][2 * k] = true;
      on[i][2 * k + 1] = ml[i][k].y < 0.f;
      if (ml[i][k].y < 0.f) {  // cut into pieces from this worker on
        const int c = __float_as_int(ml[i][k].x);
        const PagedHead hd = io.heads[c + 1];
        const int r = (tok - hd.tok0) * io.rep + hr;
        many = many || hd.last > hd.first + 1;
        row[i][2 * k] = paged_slot_row(io, c, true, r);
        row[i][2 * k + 1] = paged_slot_row(io, c + 1, false, r);
      }
    }
    dst[i] = h0 + i < io.Hq ? (T *)io.out + ((size_t)tok * io.Hq + h) * HD : nullptr;
  }
  if (!many) {
    join_some<T, HD, NR, NS>(io, row, on, dst);
    return;
  }
#pragma unroll 1
  for (int h = h0; h < min(h0 + NR, io.Hq); ++h) {
    // (the region's entries and the heads again: they are in L1 now, and registers hold fewer warps)
    int first[2], n[2];
    size_t at[2], next[2];   // rows of the first and the second piece
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      at[k] = next[k] = paged_region_row(p, io, k, tok, h);
      first[k] = 0;
      n[k] = 1;
      const float2 e = io.part_ml[at[k]];
      if (e.y < 0.f) {
        first[k] = __float_as_int(e.x);
        const PagedHead hd = io.heads[first[k] + 1];
        const int r = (tok - hd.tok0) * io.rep + h % io.rep;
        n[k] = hd.last - hd.first + 1;
        at[k] = paged_slot_row(io, first[k], true, r);
        next[k] = paged_slot_row(io, first[k] + 1, false, r);
      }
    }
    Fold<HD> f;
#pragma unroll 1
    for (int j0 = 0; j0 < n[0] + n[1]; j0 += 32) {   // the prefix's pieces, then its own
      const int j = min(j0 + lane, n[0] + n[1] - 1), k = j < n[0] ? 0 : 1, i = k ? j - n[0] : j;
      const int kind = paged_worker_kind(io, k ? first[1] : first[0]);
      const size_t later = (k ? next[1] : next[0]) + (size_t)2 * (i - 1) * io.rows[kind];
      const size_t r = i > 0 ? later : k ? at[1] : at[0];
      f.add(io.part_o, min(32, n[0] + n[1] - j0), io.part_ml[r], r);
    }
    f.store((T *)io.out + ((size_t)tok * io.Hq + h) * HD);
  }
}

template <typename T, int HD>
int run_simt(const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  note_launch(s, "paged_attn_simt");
  cudaFuncSetAttribute(paged_attn_simt_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)simt_smem<HD>());
  launch_pdl(paged_attn_simt_kernel<T, HD>, io.ctas, S_THR, simt_smem<HD>(), s, p, io);
  return check_launch("paged_attn_simt");
}

template <typename T, int HD>
int run_join(const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  if (p.shared_len > 0) {
    note_launch(s, "paged_join_prefix");
    // rows that the device holds at once (8 blocks of 8 warps an SM): a head each, else two
    if ((long long)p.n_tokens * io.Hq <= 64LL * num_sms()) {
      const long long tasks = (long long)p.n_tokens * io.Hq;
      launch_pdl(paged_join_prefix_kernel<T, HD, 1>, (unsigned)((tasks + 7) / 8), 256, 0, s, p, io);
    } else {
      const long long tasks = (long long)p.n_tokens * ((io.Hq + 1) / 2);
      launch_pdl(paged_join_prefix_kernel<T, HD, 2>, (unsigned)((tasks + 7) / 8), 256, 0, s, p, io);
    }
    return check_launch("paged_join_prefix");
  }
  // no item of a kind can exist with fewer rows than it takes
  const bool tc = io.workers > io.ctas;
  const bool all_few = tc && paged_all_few(p);
  const JoinBlocks b{!tc || (p.n_tokens > p.qn && !all_few) ? 2 * io.ctas : 0, tc ? io.ctas : 0};
  const int narrow = tc && p.n_tokens > p.qf && !all_few ? 2 * io.ctas : 0;
  note_launch(s, "paged_join");
  launch_pdl(paged_join_kernel<T, HD>, b.wide + b.few + narrow, 256, 0, s, io, b);
  return check_launch("paged_join");
}

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Query rows per item, keys per tile and workers of the kernel that takes the call.
void paged_tiling(const PagedCall &c, PagedShape *p, PagedIO *io) {
  const int rep = c.Hq / c.Hkv;
  const bool tc = paged_tc_supported(c.act, c.hd);
  const int tile = tc ? PAGED_TC_ROWS : S_ROWS;
  p->qt = tile / rep * (tc ? 2 : 1);
  p->qn = tc ? tile / rep : 0;
  p->qf = tc ? PAGED_TC_FEW / rep : 0;
  auto log2 = [](int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
  };
  p->kt_shift[PAGED_WIDE] = p->kt_shift[PAGED_NARROW] = log2(tc ? PAGED_TC_KT : S_KT);
  p->kt_shift[PAGED_FEW] = log2(PAGED_TC_FEW_KT);
  p->start_cost[PAGED_WIDE] = tc ? PAGED_TC_START_WIDE : 0;
  p->start_cost[PAGED_NARROW] = PAGED_TC_START_NARROW;
  p->start_cost[PAGED_FEW] = PAGED_TC_START_FEW;
  io->ctas = num_sms() * (tc ? 1 : 2);
  io->workers = tc ? 11 * io->ctas : io->ctas;
  const long long most = (long long)c.n_tokens * rep;
  for (int k = 0; k < 3; ++k) {
    const int rows = (k == PAGED_WIDE ? p->qt : k == PAGED_NARROW ? p->qn : p->qf) * rep;
    io->rows[k] = rows > most ? (int)most : rows;
  }
  io->region = tc ? paged_slot_row(*io, io->workers, false, 0) : (size_t)2 * io->ctas * io->rows[0];
}

struct PagedLayout {
  size_t heads, part_o, part_ml, total;
};
PagedLayout paged_layout(const PagedCall &c, const PagedIO &io) {
  const size_t rows = io.region + (c.shared_len > 0 ? (size_t)2 * c.n_tokens * c.Hq : 0);
  PagedLayout l;
  l.heads = 0;
  l.part_ml = up256(io.workers * sizeof(PagedHead));
  l.part_o = l.part_ml + up256(rows * sizeof(float2));
  l.total = l.part_o + up256(rows * c.hd * sizeof(float));
  return l;
}

}  // namespace

bool paged_attn_supported(int act, int Hq, int Hkv, int hd) {
  return Hq / Hkv <= S_ROWS && (hd == 32 || hd == 64 || hd == 128);
}

size_t paged_attn_ws_bytes(const PagedCall &c) {
  PagedShape p{};
  PagedIO io{};
  paged_tiling(c, &p, &io);
  return paged_layout(c, io).total;
}

int launch_paged_attn(const PagedCall &c, void *ws, cudaStream_t s) {
  PagedShape p{};
  PagedIO io{};
  paged_tiling(c, &p, &io);
  const PagedLayout l = paged_layout(c, io);
  p.seq_off = c.seq_off;
  p.kv_len = c.kv_len;
  p.n_seqs = c.n_seqs;
  p.n_tokens = c.n_tokens;
  p.Hkv = c.Hkv;
  p.causal = c.causal;
  p.shared_len = c.shared_len;
  p.cap = c.max_pages * c.page_size;
  // Batches of single tokens: every item is taken for few-row, by a kernel without the chains (64
  // tokens over 64 to 16384 keys 123 -> 115 us, 16 over 500 to 1000 keys 20.4 -> 17.9).  Lengths are not
  // known here, so the rule is a row per sequence on average.  A prompt among empty sequences comes out
  // right, but its keys are read once per 16 rows: 512 rows over 4512 keys among 511 empty ones take 171 us
  // where the chains take 45; a prompt of 40 rows beside 199 tokens over 8192 keys costs nothing (1026 us,
  // 1044 with the chains).
  if (p.qf > 0 && (c.n_tokens <= p.qf || (c.shared_len == 0 && c.n_tokens <= c.n_seqs))) {
    PagedShape few = p;
    few.qt = few.qn = few.qf;
    if (paged_cost_bound(few) <= PAGED_COST_LIMIT) p = few;
  }
  if (paged_cost_bound(p) > PAGED_COST_LIMIT) return DG_ERR_UNSUPPORTED;
  io.q = c.q;
  io.out = c.out;
  io.k_pages = c.k_pages;
  io.v_pages = c.v_pages;
  io.page_table = c.page_table;
  io.n_pages = c.n_pages;
  io.max_pages = c.max_pages;
  io.page_shift = 0;
  while ((1 << io.page_shift) < c.page_size) ++io.page_shift;
  io.Hq = c.Hq;
  io.rep = c.Hq / c.Hkv;
  io.rep_mul = (65536 + io.rep - 1) / io.rep;
  io.heads = (PagedHead *)((char *)ws + l.heads);
  io.part_ml = (float2 *)((char *)ws + l.part_ml);
  io.part_o = (float *)((char *)ws + l.part_o);
  io.status = c.status;
  int rc = DG_ERR_UNSUPPORTED;
#define DG_PAGED_CASE(T, HD)              \
  {                                       \
    rc = paged_tc_supported(c.act, HD) ? launch_paged_tc(c, p, io, s) : run_simt<T, HD>(p, io, s); \
    if (rc == DG_OK) rc = run_join<T, HD>(p, io, s); \
  }
  if (c.act == DG_F32) {
    if (c.hd == 32) DG_PAGED_CASE(float, 32)
    else if (c.hd == 64) DG_PAGED_CASE(float, 64)
    else DG_PAGED_CASE(float, 128)
  } else {
    if (c.hd == 32) DG_PAGED_CASE(bf16, 32)
    else if (c.hd == 64) DG_PAGED_CASE(bf16, 64)
    else DG_PAGED_CASE(bf16, 128)
  }
#undef DG_PAGED_CASE
  return rc;
}

}  // namespace dg
