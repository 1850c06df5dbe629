// Attention of packed sequences over a paged K/V cache on the tensor cores (bf16, head_dim 64 and
// 128).  "DiffusionGemma Technical Report", Figure 4; the mathematics and the joining of partial
// results stand in k_paged_attn.cu, the split of the work in paged_plan.cuh.
//
// Query rows are token-major: row r of a tile is token r / rep, head r % rep of one kv head's group,
// so every K/V tile is read once per group and any group size fits a tile of 128 rows.  One CTA per
// SM walks its range of work; an item is
//   wide    two query tiles A and B (up to 256 rows) against the same key tiles, or
//   narrow  one query tile (up to 128 rows: single tokens, short prompts) whose even key tiles go
//           through chain A and odd ones through chain B, joined at the end,
// so that both chains always work and one's softmax overlaps the other's matrix products:
//   S_x = Q_x K^T    (128 x 128 keys x head_dim, bf16 from shared memory)
//   O_x += P_x V     (128 x head_dim x 128 keys, P from tensor memory, V from shared memory)
// Tensor memory (512 columns): S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512); P_x is
// written over S_x.  MMAs of one thread execute in issue order, so S_x of the next key tile is
// issued right behind P_x V.
//
// P is rounded to bf16, as V is given: a relative error up to 2^-8 in each p, independent from key
// to key, which adds to an output about as much as its own rounding does (measured: 0.0024 of the
// outputs' size against 0.0017 for the rounding alone).  Two bf16 parts would cost a second P V
// product, 1.5 times the tensor work.
//
// Warps: 0 copies (one lane per page: each looks its page up and issues that page's TMA boxes into a
// ring of key / value tiles), 1 owns the tensor memory and issues the MMAs, 4-7 are the softmax of
// chain A and 8-11 of chain B, a query row per thread.  What a page holds behind a sequence's last
// key is masked in S and zeroed in V before the product reads it (0 * NaN).
// Every wait is bounded; on expiry the kernel records DG_ERR_TIMEOUT, lets issued copies and MMAs
// finish, frees tensor memory and returns.
#include "dg_common.cuh"
#include "dg_kernels.h"
#include "paged_attn.cuh"
#include "tc_common.cuh"
#include "tc_host.h"

namespace dg {

namespace {

constexpr int P_THR = 384;
constexpr int P_HALF = 128 * 128;          // 128 rows of 64 bf16 (128-byte rows): 16 KB
constexpr uint32_t P_COL_S = 0, P_COL_O = 256, P_TMEM = 512;
constexpr float P_RESCALE = 8.f;           // log2 of the largest P between rescales
constexpr unsigned FULL = 0xffffffffu;
// Registers per thread at launch, and after the split between the copy / MMA warpgroup (LO) and the
// two softmax warpgroups (HI), which hold a whole row of S.
constexpr int P_REGS = 168, P_REGS_LO = 104, P_REGS_HI = 200;
static_assert(128 * P_REGS_LO + 256 * P_REGS_HI <= P_THR * P_REGS, "register split");
static_assert(P_THR * P_REGS <= 65536, "launch registers");

template <int HD>
struct Tc {
  static constexpr int HALVES = HD / 64;
  static constexpr int TILE = HALVES * P_HALF;          // 128 rows x HD
  static constexpr int STAGES = HD == 128 ? 5 : 10;     // key and value tiles in flight
  static constexpr size_t SMEM = 1024 + (size_t)TILE * (2 + STAGES) + 2048;
};

template <int R>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
// 2^x by the hardware approximation (relative error ~2^-22, -inf -> +0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 3-D tiled load of the box at (x = element, y, z).
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *tm, uint64_t *bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// kind::f16 with bf16 A and B, fp32 D, A K-major, B MN-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16_bmn(int M, int N) {
  return tc::idesc_bf16(M, N) | (1u << 16);
}

__device__ __forceinline__ void p_fail(int32_t *st, volatile int *abort_flag) {
  set_status(st, DG_ERR_TIMEOUT);
  *abort_flag = 1;
}

// One piece of a walk in terms of key tiles: tiles [t0, t1) of an item of `keys` keys.
struct Piece {
  bool narrow;
  int t0, t1, keys, toks, i0;
  __device__ __forceinline__ Piece(const PagedShape &p, const PagedWalk &w) {
    toks = paged_item_tokens(p, w.s, w.item);
    narrow = toks <= p.qn;
    keys = paged_item_keys(p, w.s, w.item);
    i0 = w.item * p.qt;
    t0 = narrow ? 2 * w.k0() : w.k0();
    t1 = narrow ? min(2 * w.k1(), (keys + PAGED_TC_KT - 1) / PAGED_TC_KT) : w.k1();
  }
};

template <int HD>
__global__ void __launch_bounds__(P_THR, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedShape p, const __grid_constant__ PagedIO io) {
  pdl_wait();
  pdl_trigger();
  using namespace tc;
  using C = Tc<HD>;
  constexpr int S = C::STAGES, TILE = C::TILE, HALVES = C::HALVES;
  extern __shared__ uint8_t p_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)p_smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sQ = smem;                                   // [2][TILE]
  uint8_t *sKV = sQ + 2 * TILE;                         // [S][TILE], K and V tiles in turn
  uint64_t *q_full = reinterpret_cast<uint64_t *>(sKV + S * TILE);   // [2]
  uint64_t *q_empty = q_full + 2, *full = q_empty + 2, *empty = full + S;
  uint64_t *s_full = empty + S, *p_full = s_full + 2, *pv_done = p_full + 2, *o_empty = pv_done + 2;
  uint64_t *b_done = o_empty + 2, *mma_fin = b_done + 1;
  float2 *b_ml = reinterpret_cast<float2 *>(mma_fin + 1);            // [128] (m, l) of chain B
  PagedStart *start = reinterpret_cast<PagedStart *>(b_ml + 128);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int err;
    const PagedStart st = paged_locate(p, blockIdx.x, gridDim.x, &err);
    if (lane == 0) {
      *start = st;
      if (blockIdx.x == 0) paged_report(io, err);
      paged_write_head(p, io, st, blockIdx.x);
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, P_TMEM);
    tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&o_empty[x], 4);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(b_done, 4);
    mbar_init(mma_fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  } else if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const PagedStart st = *start;
  const int rep = io.rep, qn = p.qn;   // qn tokens of rep heads make a query tile

  PagedWalk w;
  if (warp == 0) {
    // ---- copies
    reg_dec<P_REGS_LO>();
    const int page = 1 << io.page_shift, box = min(page, PAGED_TC_KT);
    uint32_t fill = 0, qs = 0;   // tiles and query tiles loaded so far
    bool ok = true;
    for (w.begin(p, st); ok && w.more(); w.next(p)) {
      const Piece pc(p, w);
      for (int x = 0; x < (pc.narrow ? 1 : 2) && ok; ++x, ++qs) {
        const uint32_t b = qs & 1;
        ok = __all_sync(FULL, mbar_wait(&q_empty[b], ((qs >> 1) & 1) ^ 1));
        if (ok && lane == 0) {
          mbar_expect_tx(&q_full[b], (uint32_t)(rep * qn * HD * 2));
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(sQ + b * TILE + h * P_HALF, &tmQ, &q_full[b], h * 64, w.head * rep,
                        w.s.tok0 + pc.i0 + x * qn);
        }
      }
      // this lane's part of a tile: keys [lane * box, lane * box + box), its page looked up one
      // tile ahead
      auto lookup = [&](int t) -> int {
        const int k = t * PAGED_TC_KT + lane * box;
        if (t >= pc.t1 || lane * box >= PAGED_TC_KT || k >= pc.keys) return -1;
        const int pos = w.s.key0 + k;
        const long long row = paged_row(io, p, w.s.seq, w.head, pos);
        return row < 0 ? io.n_pages * p.Hkv * page : (int)row;   // past the pool: reads zeros
      };
      int y = lookup(pc.t0);
      for (int t = pc.t0; t < pc.t1 && ok; ++t) {
        const int y_next = lookup(t + 1);
        const int boxes = (min(PAGED_TC_KT, pc.keys - t * PAGED_TC_KT) + box - 1) / box;
        for (int kv = 0; kv < 2 && ok; ++kv, ++fill) {
          const uint32_t s = fill % S;
          ok = __all_sync(FULL, mbar_wait(&empty[s], ((fill / S) & 1) ^ 1) && !*abort_flag);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&full[s], (uint32_t)(boxes * box * HD * 2));
          __syncwarp();
          if (y >= 0) {
            const CUtensorMap *tm = kv ? &tmV : &tmK;
            uint8_t *dst = sKV + s * TILE + lane * box * 128;
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_2d(dst + h * P_HALF, tm, &full[s], h * 64, y);
          }
        }
        y = y_next;
      }
    }
    if (!ok && lane == 0) p_fail(io.status, abort_flag);
    // the copies in flight land before the CTA's shared memory can go away
    for (uint32_t f = fill > S ? fill - S : 0; f < fill; ++f) (void)mbar_wait(&full[f % S], (f / S) & 1);
    for (uint32_t f = qs > 2 ? qs - 2 : 0; f < qs; ++f) (void)mbar_wait(&q_full[f & 1], (f >> 1) & 1);
  } else if (warp == 1) {
    // ---- matrix products: the warp waits together, lane 0 issues
    reg_dec<P_REGS_LO>();
    constexpr uint32_t id_s = idesc_bf16(128, PAGED_TC_KT), id_p = idesc_bf16_bmn(128, HD);
    const uint64_t dq = sdesc_sw128(sQ), dk = sdesc_sw128(sKV), dv = sdesc_sw128_mn(sKV, P_HALF);
    uint32_t fill = 0, qs = 0, pieces = 0, pn[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL, mbar_wait(bar, parity));
      fence_after();
    };
    auto issue_s = [&](int x, uint32_t qb, uint32_t ks) {   // S_x = Q K^T
      if (ok && lane == 0) {
        const uint64_t ab = dq + (uint64_t)((qb * TILE) >> 4), bb = dk + (uint64_t)((ks * TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * P_HALF) >> 4) + 2 * (kk & 3);
          mma_bf16(tmem + P_COL_S + x * 128, ab + off, bb + off, id_s, kk > 0 ? 1u : 0u);
        }
        commit(&s_full[x]);
      }
    };
    auto issue_pv = [&](int x, uint32_t vs, bool first) {   // O_x (+)= P_x V
      if (ok && lane == 0) {
        const uint64_t bb = dv + (uint64_t)((vs * TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < PAGED_TC_KT / 16; ++kk)
          mma_f16_ts(tmem + P_COL_O + x * 128, tmem + P_COL_S + x * 128 + kk * 8,
                     bb + (uint64_t)((kk * 16 * 128) >> 4), id_p, kk > 0 || !first ? 1u : 0u);
        commit(&pv_done[x]);
      }
    };
    auto release = [&](uint64_t *bar) {
      if (ok && lane == 0) commit(bar);
    };
    for (w.begin(p, st); ok && w.more(); w.next(p), ++pieces) {
      const Piece pc(p, w);
      const int N = pc.t1 - pc.t0;
      const uint32_t f0 = fill;
      auto k_at = [&](int i) { return f0 + 2 * (uint32_t)i; };       // fill number of K_i; V_i next
      auto wait_fill = [&](uint32_t f) { wait(&full[f % S], (f / S) & 1); };
      // V_i has landed; rows past the item's last key become zeros
      auto wait_v = [&](int i) {
        const uint32_t f = k_at(i) + 1;
        wait_fill(f);
        const int valid = pc.keys - (pc.t0 + i) * PAGED_TC_KT;
        if (ok && valid < PAGED_TC_KT) {
          uint8_t *base = sKV + (f % S) * TILE;
          for (int e = lane; e < (PAGED_TC_KT - valid) * 8; e += 32)   // 8 chunks a row
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              reinterpret_cast<uint4 *>(base + h * P_HALF + valid * 128)[e] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
      };
      const uint32_t qa = qs & 1;
      wait(&q_full[qa], (qs >> 1) & 1);
      if (!pc.narrow) wait(&q_full[qa ^ 1], ((qs + 1) >> 1) & 1);
      const uint32_t qb = pc.narrow ? qa : qa ^ 1;
      wait_fill(k_at(0));
      issue_s(0, qa, k_at(0) % S);
      // a query tile is free once the last S of the piece has read it
      if (pc.narrow) {
        release(&empty[k_at(0) % S]);
        if (N == 1) release(&q_empty[qa]);
        if (N > 1) {
          wait_fill(k_at(1));
          issue_s(1, qa, k_at(1) % S);
          release(&empty[k_at(1) % S]);
          if (N == 2) release(&q_empty[qa]);
        }
        for (int i = 0; i < N && ok; ++i) {
          const int x = i & 1;
          wait_v(i);
          wait(&p_full[x], pn[x] & 1);
          ++pn[x];
          if (i < 2 && pieces > 0) wait(&o_empty[x], (pieces - 1) & 1);
          issue_pv(x, (k_at(i) + 1) % S, i < 2);
          release(&empty[(k_at(i) + 1) % S]);
          if (i + 2 < N) {
            wait_fill(k_at(i + 2));
            issue_s(x, qa, k_at(i + 2) % S);
            release(&empty[k_at(i + 2) % S]);
            if (i + 3 == N) release(&q_empty[qa]);
          }
          if (__any_sync(FULL, *abort_flag != 0)) ok = false;
        }
        if (N == 1 && pieces > 0) wait(&o_empty[1], (pieces - 1) & 1);
        qs += 1;
      } else {
        if (N == 1) release(&q_empty[qa]);
        issue_s(1, qb, k_at(0) % S);
        release(&empty[k_at(0) % S]);
        if (N == 1) release(&q_empty[qb]);
        for (int i = 0; i < N && ok; ++i) {
          const bool more = i + 1 < N;
          wait_v(i);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            wait(&p_full[x], pn[x] & 1);
            ++pn[x];
            if (i == 0 && pieces > 0) wait(&o_empty[x], (pieces - 1) & 1);
            issue_pv(x, (k_at(i) + 1) % S, i == 0);
            if (x == 1) release(&empty[(k_at(i) + 1) % S]);
            if (more) {
              if (x == 0) wait_fill(k_at(i + 1));
              issue_s(x, x ? qb : qa, k_at(i + 1) % S);
              if (x == 1) release(&empty[k_at(i + 1) % S]);
              if (i + 2 == N) release(&q_empty[x ? qb : qa]);
            }
          }
          if (__any_sync(FULL, *abort_flag != 0)) ok = false;
        }
        qs += 2;
      }
      fill += 2 * (uint32_t)N;
    }
    if (lane == 0) {
      if (!ok) p_fail(io.status, abort_flag);
      commit(mma_fin);   // every MMA issued above has completed when this phase does
      (void)mbar_wait(mma_fin, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    reg_dec<P_REGS_LO>();
  } else {
    // ---- softmax of chain x
    reg_inc<P_REGS_HI>();
    const int x = (warp - 4) >> 2;
    const int q4 = warp & 3;                  // tensor-memory lane quarter of this warp
    const int r = q4 * 32 + lane;             // query row of the tile
    const uint32_t lrow = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lrow + P_COL_S + (uint32_t)x * 128;
    const uint32_t tO = tmem + lrow + P_COL_O + (uint32_t)x * 128;
    const float sl2 = 1.4426950408889634f / sqrtf((float)HD);
    uint32_t ns = 0, pieces = 0, narrows = 0; // key tiles, pieces and narrow pieces so far
    bool ok = true;
    for (w.begin(p, st); w.more(); w.next(p), ++pieces) {
      const Piece pc(p, w);
      const int tile0 = pc.narrow ? 0 : x * qn;                 // first token of this chain's tile
      const int toks = pc.narrow ? pc.toks : max(0, min(qn, pc.toks - tile0));
      const int tl = tile0 + min(r / rep, max(toks, 1) - 1);    // this row's token in the item
      const bool row_ok = r < toks * rep;
      const bool warp_on = q4 * 32 < toks * rep;                // any row of this warp
      const int seen = w.s.causal ? w.s.keys - w.s.n + pc.i0 + tl + 1 : pc.keys;
      float m_use = -INFINITY, l = 0.f;
      const int step = pc.narrow ? 2 : 1;
      for (int t = pc.t0 + (pc.narrow ? x : 0); t < pc.t1; t += step, ++ns) {
        if (__any_sync(FULL, *abort_flag != 0)) { ok = false; break; }
        if (!__all_sync(FULL, mbar_wait(&s_full[x], ns & 1))) {
          p_fail(io.status, abort_flag);
          ok = false;
          break;
        }
        fence_after();
        if (warp_on) {
          const int lim = seen - t * PAGED_TC_KT;
          // the row of S: two 64-column loads
          uint32_t sa[64], sb[64];
          tmem_ld64(tS, sa);
          tmem_ld64(tS + 64, sb);
          tmem_ld_wait64(sa);
          tmem_ld_wait64(sb);
          if (__any_sync(FULL, lim < PAGED_TC_KT)) {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              if (j >= lim) sa[j] = __float_as_uint(-INFINITY);
              if (64 + j >= lim) sb[j] = __float_as_uint(-INFINITY);
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto fold_max = [&](const uint32_t (&v)[64]) {
#pragma unroll
            for (int j = 0; j < 64; j += 2)
              m4[(j >> 1) & 3] = max3(m4[(j >> 1) & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
          };
          fold_max(sa);
          fold_max(sb);
          const float m_new = fmaxf(m_use, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2);
          // O is rescaled only when a row's maximum grew by more than 2^8 (P stays below 256, and O
          // and l share their base, so O / l does not change); S of this tile was issued behind the
          // last P V, so O includes it
          if (__any_sync(FULL, m_use != -INFINITY && m_new > m_use + P_RESCALE)) {
            const float f = m_use == -INFINITY ? 1.f : ex2(m_use - m_new);
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(tO + c * 32, o);
            }
            tmem_st_wait();
            l *= f;
            m_use = m_new;
          } else if (m_use == -INFINITY) {
            m_use = m_new;
          }
          const float nb = m_use == -INFINITY ? 0.f : -m_use;
          const float2 sl2v = make_float2(sl2, sl2), nbv = make_float2(nb, nb);
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto emit = [&](const uint32_t (&v)[64], int hf) {
            uint32_t pb[32];
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const float2 t2 = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                           sl2v, nbv);
              const float2 e = make_float2(ex2(t2.x), ex2(t2.y));
              s2[(j >> 1) & 1] = __fadd2_rn(s2[(j >> 1) & 1], e);
              const __nv_bfloat162 b = __floats2bfloat162_rn(e.x, e.y);
              pb[j >> 1] = *reinterpret_cast<const uint32_t *>(&b);
            }
            tmem_st32(tS + hf * 32, pb);
          };
          emit(sa, 0);
          emit(sb, 1);
          l += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
          tmem_st_wait();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // ---- the piece's result
      const int chain_tiles = pc.narrow ? (pc.t1 - pc.t0 + 1 - x) / 2 : pc.t1 - pc.t0;
      if (chain_tiles > 0 && !__all_sync(FULL, mbar_wait(&pv_done[x], (ns - 1) & 1))) {
        p_fail(io.status, abort_flag);
        break;
      }
      fence_after();
      float fa = 1.f, fb = 0.f;   // factors of the two chains' O
      if (pc.narrow) {
        if (x == 1) {
          // chain A stores for both; it is done with the (m, l) handed over before when it has freed
          // the accumulators of the previous piece
          if (pieces > 0 && !__all_sync(FULL, mbar_wait(&o_empty[1], (pieces - 1) & 1))) {
            p_fail(io.status, abort_flag);
            break;
          }
          b_ml[r] = make_float2(m_use, l);
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_done);
          continue;
        }
        if (!__all_sync(FULL, mbar_wait(b_done, narrows & 1))) {
          p_fail(io.status, abort_flag);
          break;
        }
        ++narrows;
        fence_after();
        if (pc.t1 - pc.t0 > 1) {
          const float2 mb = b_ml[r];
          const float m = fmaxf(m_use, mb.x), base = m == -INFINITY ? 0.f : m;
          fa = ex2(m_use - base);
          fb = ex2(mb.x - base);
          l = l * fa + mb.y * fb;
          m_use = m;
        }
      }
      if (warp_on) {
        const bool both = pc.narrow && pc.t1 - pc.t0 > 1;   // O_B holds something
        const PagedDest dest = paged_dest(p, io, w, blockIdx.x);
        const int tok = w.s.tok0 + pc.i0 + tl, h = w.head * rep + r % rep;
        const float il = l > 0.f ? 1.f / l : 0.f;
        bf16 *out = (bf16 *)io.out + ((size_t)tok * io.Hq + h) * HD;
        const size_t prow = paged_part_row(p, io, dest, tile0 * rep + r, tok, h);
        float *part = io.part_o + prow * HD;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait(o);
          if (both) {
            uint32_t ob[32];
            tmem_ld32(tO + 128 + c * 32, ob);
            tmem_ld_wait(ob);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * fa + __uint_as_float(ob[j]) * fb);
          }
          if (!row_ok) continue;   // guards the stores only; every lane reads tensor memory
          if (dest.kind == PAGED_OUT) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(
                    __uint_as_float(o[j + 2 * e]) * il, __uint_as_float(o[j + 2 * e + 1]) * il);
                v[e] = *reinterpret_cast<const uint32_t *>(&b2);
              }
              *reinterpret_cast<uint4 *>(out + c * 32 + j) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4 *>(part + c * 32 + j) =
                  make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
        if (row_ok && dest.kind != PAGED_OUT) {
          io.part_ml[prow] = make_float2(m_use, l);
          if (dest.redirect) paged_redirect(p, io, dest, blockIdx.x, tok, h);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_empty[x]);
        if (pc.narrow) mbar_arrive(&o_empty[1]);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, P_TMEM);
  }
}

template <int HD>
int run_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  using C = Tc<HD>;
  // the register split inside the kernel needs the launch to hold P_REGS registers per thread; a
  // build with fewer would leave setmaxnreg.inc waiting, so it is refused here
  static const int regs = [] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, paged_attn_tc_kernel<HD>) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (regs < P_REGS) return DG_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv;
  const uint64_t rows = (uint64_t)c.n_pages * c.Hkv * c.page_size;
  const uint32_t box = c.page_size < PAGED_TC_KT ? c.page_size : PAGED_TC_KT;
  const CUtensorMapDataType bt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = make_tmap_3d(&tq, bt, 2, c.q, HD, c.Hq, c.n_tokens, 64, io.rep, p.qn);
  if (rc == DG_OK) rc = make_tmap_2d(&tk, bt, 2, c.k_pages, HD, rows, HD * 2, 64, box);
  if (rc == DG_OK) rc = make_tmap_2d(&tv, bt, 2, c.v_pages, HD, rows, HD * 2, 64, box);
  if (rc != DG_OK) return rc;
  note_launch(s, "paged_attn_tc");
  cudaFuncSetAttribute(paged_attn_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)C::SMEM);
  launch_pdl(paged_attn_tc_kernel<HD>, io.ctas, P_THR, C::SMEM, s, tq, tk, tv, p, io);
  return check_launch("paged_attn_tc");
}

}  // namespace

int launch_paged_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  return c.hd == 128 ? run_tc<128>(c, p, io, s) : run_tc<64>(c, p, io, s);
}

}  // namespace dg
