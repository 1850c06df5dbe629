// Attention of packed sequences over a paged K/V cache on the tensor cores (bf16, head_dim 64 and
// 128).  "DiffusionGemma Technical Report", Figure 4; the mathematics and the joining of partial
// results stand in k_paged_attn.cu, the split of the work in paged_plan.cuh.
//
// Query rows are token-major: row r of a tile is token r / rep, head r % rep of one kv head's
// group, so every K/V tile is read once per group and any group size fits a tile of 128 rows.  One
// CTA per SM runs two chains of
//   S_x = Q_x K^T    (128 x 128 keys x head_dim, bf16 from shared memory)
//   P_x = softmax's numerators, O_x += P_x V    (P from tensor memory, V from shared memory)
// so that the softmax of one overlaps the matrix products of the other:
//   wide items     both chains take one query tile each (up to 256 rows) against the same key tiles;
//   narrow items   (short prompts, tails: up to 128 rows) each chain walks a range of its own, so that
//                  the start and end of one's items hide behind the other's work.
// Few-row items (single tokens: up to 16 rows) would leave 7/8 of such a tile empty and pass each
// key tile through a chain of four waits; there each of the eight softmax warps walks a range of
// its own with mma.sync, 32 keys a step, from a ring of its own in the memory that chains would use (a CTA
// serves one kind of work), so that almost all of it is in flight: these items are bound by the bytes of
// their keys.
// Their copies are cp.async, not TMA: a box of one 16-key page takes the TMA unit about 60 cycles
// for 2 KB, and eight warps that each wait for several such boxes waited 3 us before their first
// product.  Calls whose items all are few-row have a kernel of their own without the chains' code
// (one token over 777 keys 12 us, 15 with it).
//
// Tensor memory (512 columns): S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512);
// P_x is written over S_x.  MMAs of one thread execute in issue order, so S_x of the next key tile
// is issued right behind P_x V.
//
// P is rounded to bf16, as V is given: a relative error up to 2^-8 in each p, independent from key
// to key, which adds to an output about as much as its own rounding does (measured: 0.0024 of the
// outputs' size against 0.0017 for the rounding alone).  Two bf16 parts would cost a second P V
// product, 1.5 times the tensor work.
//
// Warps: 0 copies (one lane per page: each looks its page up and issues that page's TMA boxes into
// a ring of key / value tiles), 1 owns the tensor memory and issues the MMAs, 4-7 are the softmax
// of chain A and 8-11 of chain B, a query row per thread.  What a page holds behind a sequence's
// last key is masked in S and zeroed in V before the product reads it (0 * NaN). Every wait is
// bounded; on expiry the kernel records DG_ERR_TIMEOUT, lets issued copies and MMAs finish, frees
// tensor memory and returns.
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
constexpr int P_STAGE = 32 * 32 * 4;       // a softmax warp's 32 rows x 32 columns on their way out
// Registers per thread at launch, and after the split between the copy / MMA warpgroup (LO) and the
// two softmax warpgroups (HI), which hold a whole row of S.
constexpr int P_REGS = 168, P_REGS_LO = 104, P_REGS_HI = 200;
static_assert(128 * P_REGS_LO + 256 * P_REGS_HI <= P_THR * P_REGS, "register split");
static_assert(P_THR * P_REGS <= 65536, "launch registers");

constexpr int F_KT = PAGED_TC_FEW_KT;      // few-row items: keys per step,
constexpr int F_SLOTS = 3;                 // slots of a warp's ring, K and V of a step in turn

template <int HD>
struct Tc {
  static constexpr int HALVES = HD / 64;
  static constexpr int TILE = HALVES * P_HALF;          // 128 rows x HD
  static constexpr int STAGES = HD == 128 ? 4 : 8;      // key and value tiles in flight
  static_assert(8 * F_SLOTS * F_KT * HD * 2 <= (2 + STAGES) * TILE, "few-row rings");
  static constexpr size_t SMEM = 1024 + (size_t)TILE * (2 + STAGES) + 8 * P_STAGE + 2048;
};

// A piece of a few-row item, as the loading side of a warp leaves it for the computing side.
struct FewPiece {
  int tok, toks, head, keys, before, t0, t1, which;
  bool whole;
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
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(p))
               : "memory");
}
// D += A B, m16n8k16, bf16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes from global to shared memory; `on` false: zeros.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
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

// CHAINS false: a call whose items all are few-row; the kernel without what the chains need.
template <int HD, bool CHAINS>
__global__ void __launch_bounds__(P_THR, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedShape p, const __grid_constant__ PagedIO io) {
  pdl_wait();
  pdl_trigger();
  using namespace tc;
  using C = Tc<HD>;
  constexpr int S = C::STAGES, TILE = C::TILE, HALVES = C::HALVES, KT = PAGED_TC_KT;
  extern __shared__ uint8_t p_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)p_smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sQ = smem;                                   // [2][TILE], by chain
  uint8_t *sKV = sQ + 2 * TILE;                         // [S][TILE], K and V tiles in turn
  uint8_t *sOut = sKV + S * TILE;                       // [8][P_STAGE], by softmax warp
  uint64_t *q_full = reinterpret_cast<uint64_t *>(sOut + 8 * P_STAGE);   // [2]
  uint64_t *q_empty = q_full + 2, *full = q_empty + 2, *empty = full + S;
  uint64_t *s_full = empty + S, *p_full = s_full + 2, *pv_done = p_full + 2, *o_empty = pv_done + 2;
  uint64_t *mma_fin = o_empty + 2;
  PagedStart *start = reinterpret_cast<PagedStart *>(mma_fin + 1);   // [PAGED_STARTS]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + PAGED_STARTS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert((4 + 2 * S + 9) * 8 + PAGED_STARTS * sizeof(PagedStart) + 8 <= 2048, "shared memory");

  // (the shuffle tells the compiler that a warp's threads agree on it)
  const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (CHAINS && warp == 1) {
    if (lane == 0) {
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
      mbar_init(mma_fin, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, P_TMEM);
    tmem_relinquish();
  } else if (CHAINS && warp == 2 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // (the scan's scratch lies where rows will leave the kernel much later)
  const int err = paged_locate<P_THR / 3, 3>(p, blockIdx.x, gridDim.x, PAGED_STARTS, start, io.heads,
                                          *reinterpret_cast<PagedScan *>(sOut));
  if constexpr (CHAINS) fence_before();
  __syncthreads();
  if constexpr (CHAINS) fence_after();
  const uint32_t tmem = CHAINS ? __shfl_sync(FULL, *tmem_slot, 0) : 0;
  if (threadIdx.x == 0 && blockIdx.x == 0) paged_report(io, err);
  const int rep = io.rep, qn = p.qn;   // qn tokens of rep heads make a query tile

  if (CHAINS && warp == 0) {
    // ---- copies
    reg_dec<P_REGS_LO>();
    const int page = 1 << io.page_shift, box = min(page, KT);
    uint32_t fill = 0, nq[2] = {0, 0};   // tiles and (by chain) query tiles loaded so far
    bool ok = true;
    // the query tile of chain x: qn tokens from `tok` on
    auto load_q = [&](const PagedWalk &w, int x, int tok) {
      ok = __all_sync(FULL, mbar_wait(&q_empty[x], (nq[x] & 1) ^ 1) && !*abort_flag);
      if (!ok) return;
      if (lane == 0) {
        mbar_expect_tx(&q_full[x], (uint32_t)(rep * qn * HD * 2));
        for (int h = 0; h < HALVES; ++h)
          tma_load_3d(sQ + x * TILE + h * P_HALF, &tmQ, &q_full[x], h * 64, w.head * rep,
                      w.s.tok0 + tok);
      }
      ++nq[x];
    };
    // this lane's part of key tile t: keys [lane * box, lane * box + box); -1: none
    auto lookup = [&](const PagedWalk &w, int t) -> int {
      const int k = t * KT + lane * box;
      if (lane * box >= KT || k >= w.keys) return -1;
      const long long row = paged_row(io, p, w.s.seq, w.head, w.s.key0 + k);
      return row < 0 ? io.n_pages * p.Hkv * page : (int)row;   // past the pool: reads zeros
    };
    auto load = [&](const CUtensorMap *tm, const PagedWalk &w, int t, int y) {
      const int boxes = (min(KT, w.keys - t * KT) + box - 1) / box;
      const uint32_t s = fill % S;
      ok = __all_sync(FULL, mbar_wait(&empty[s], ((fill / S) & 1) ^ 1) && !*abort_flag);
      if (!ok) return;
      if (lane == 0) mbar_expect_tx(&full[s], (uint32_t)(boxes * box * HD * 2));
      __syncwarp();
      if (y >= 0) {
        uint8_t *dst = sKV + s * TILE + lane * box * 128;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) tma_load_2d(dst + h * P_HALF, tm, &full[s], h * 64, y);
      }
      ++fill;
    };
    // Tiles are loaded in the order in which the MMA warp releases them.
    if (start[0].u1 > 0) {
      PagedWalk w;
      for (w.begin(p, PAGED_WIDE, start[0]); ok && w.more(); w.next(p)) {
        int y = lookup(w, w.t0);   // (under way while the query tiles are asked for)
        load_q(w, 0, w.tok);
        if (ok) load_q(w, 1, w.tok + qn);
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          const int y_next = t + 1 < w.t1 ? lookup(w, t + 1) : -1;   // a tile ahead
          load(&tmK, w, t, y);
          if (ok) load(&tmV, w, t, y);
          y = y_next;
        }
      }
    }
    if (start[1].u1 > 0 || start[2].u1 > 0) {
      PagedWalk w[2];
      int t[2] = {0, 0}, y[2] = {0, 0};
      auto load_k = [&](int x) {
        if (!ok || !w[x].more()) return;
        if (t[x] == w[x].t0) load_q(w[x], x, w[x].tok);
        if (ok) load(&tmK, w[x], t[x], y[x]);
      };
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w[x].begin(p, PAGED_NARROW, start[1 + x]);
        if (w[x].more()) y[x] = lookup(w[x], t[x] = w[x].t0);
      }
      load_k(0);
      load_k(1);
      while (ok && (w[0].more() || w[1].more())) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || !w[x].more()) continue;
          load(&tmV, w[x], t[x], y[x]);
          if (++t[x] == w[x].t1) {
            w[x].next(p);
            t[x] = w[x].t0;
          }
          if (w[x].more()) y[x] = lookup(w[x], t[x]);
          load_k(x);
        }
      }
    }
    if (!ok && lane == 0) p_fail(io.status, abort_flag);
    // the copies in flight land before the CTA's shared memory can go away
    for (uint32_t f = fill > S ? fill - S : 0; f < fill; ++f) (void)mbar_wait(&full[f % S], (f / S) & 1);
    for (int x = 0; x < 2; ++x)
      if (nq[x] > 0) (void)mbar_wait(&q_full[x], (nq[x] - 1) & 1);
  } else if (CHAINS && warp == 1) {
    // ---- matrix products: the warp waits together, one lane issues
    reg_dec<P_REGS_LO>();
    constexpr uint32_t id_s = idesc_bf16(128, KT), id_p = idesc_bf16_bmn(128, HD);
    const uint64_t dq = sdesc_sw128(sQ), dk = sdesc_sw128(sKV), dv = sdesc_sw128_mn(sKV, P_HALF);
    // by chain: pieces begun, key tiles whose P was taken
    uint32_t pieces[2] = {0, 0}, pn[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = __all_sync(FULL, mbar_wait(bar, parity));
      fence_after();
    };
    auto wait_fill = [&](uint32_t f) { wait(&full[f % S], (f / S) & 1); };
    const bool leader = elect_one();   // the lane that issues
    auto release = [&](uint64_t *bar) {
      if (ok && leader) commit(bar);
    };
    auto issue_s = [&](int x, uint32_t f) {   // S_x = Q_x K^T, K in fill f
      const uint32_t stage = __shfl_sync(FULL, f % S, 0);
      const uint64_t ab = dq + (uint64_t)((x * TILE) >> 4), bb = dk + (uint64_t)((stage * TILE) >> 4);
      if (ok && leader) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * P_HALF) >> 4) + 2 * (kk & 3);
          mma_bf16(tmem + P_COL_S + x * 128, ab + off, bb + off, id_s, kk > 0 ? 1u : 0u);
        }
        commit(&s_full[x]);
      }
    };
    // O_x (+)= P_x V, V in fill f: waits for P_x, and for O_x where it is begun anew
    auto take_pv = [&](int x, uint32_t f, bool first) {
      wait(&p_full[x], pn[x] & 1);
      ++pn[x];
      if (first && pieces[x] > 1) wait(&o_empty[x], pieces[x] & 1);   // of the piece before
      const uint32_t stage = __shfl_sync(FULL, f % S, 0);
      const uint64_t bb = dv + (uint64_t)((stage * TILE) >> 4);
      if (ok && leader) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_f16_ts(tmem + P_COL_O + x * 128, tmem + P_COL_S + x * 128 + kk * 8,
                     bb + (uint64_t)((kk * 16 * 128) >> 4), id_p, kk > 0 || !first ? 1u : 0u);
        commit(&pv_done[x]);
      }
    };
    // fill f (a value tile) has landed; rows past its `valid` keys become zeros
    auto wait_v = [&](uint32_t f, int valid) {
      wait_fill(f);
      if (ok && valid < KT) {
        uint8_t *base = sKV + (f % S) * TILE + valid * 128;
        for (int e = lane; e < (KT - valid) * 8; e += 32)   // 8 chunks of 16 bytes a row
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            reinterpret_cast<uint4 *>(base + h * P_HALF)[e] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
    };
    auto begin_q = [&](int x) {   // a piece of chain x: its query tile
      wait(&q_full[x], pieces[x] & 1);
      ++pieces[x];
    };
    uint32_t f = 0;   // fills taken so far (wide: the key tile whose S is issued next)
    if (start[0].u1 > 0) {
      PagedWalk w;
      for (w.begin(p, PAGED_WIDE, start[0]); ok && w.more(); w.next(p)) {
        begin_q(0);
        begin_q(1);
        wait_fill(f);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          issue_s(x, f);
          if (w.t0 + 1 == w.t1) release(&q_empty[x]);   // the piece's last S has read it
        }
        release(&empty[f % S]);
        for (int t = w.t0; t < w.t1 && ok; ++t, f += 2) {
          const bool more = t + 1 < w.t1;
          wait_v(f + 1, w.keys - t * KT);
          if (more) wait_fill(f + 2);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            take_pv(x, f + 1, t == w.t0);
            if (x == 1) release(&empty[(f + 1) % S]);
            if (more) {
              issue_s(x, f + 2);
              if (t + 2 == w.t1) release(&q_empty[x]);
              if (x == 1) release(&empty[(f + 2) % S]);
            }
          }
          if (__any_sync(FULL, *abort_flag != 0)) ok = false;
        }
      }
    }
    if (start[1].u1 > 0 || start[2].u1 > 0) {
      PagedWalk w[2];
      int t[2] = {0, 0};
      auto next_s = [&](int x) {
        if (t[x] == w[x].t0) begin_q(x);
        wait_fill(f);
        issue_s(x, f);
        release(&empty[f % S]);
        ++f;
        if (t[x] + 1 == w[x].t1) release(&q_empty[x]);
      };
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w[x].begin(p, PAGED_NARROW, start[1 + x]);
        if (w[x].more()) {
          t[x] = w[x].t0;
          next_s(x);
        }
      }
      while (ok && (w[0].more() || w[1].more())) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || !w[x].more()) continue;
          wait_v(f, w[x].keys - t[x] * KT);
          take_pv(x, f, t[x] == w[x].t0);
          release(&empty[f % S]);
          ++f;
          if (++t[x] == w[x].t1) {
            w[x].next(p);
            t[x] = w[x].t0;
          }
          if (w[x].more()) next_s(x);
        }
        if (__any_sync(FULL, *abort_flag != 0)) ok = false;
      }
    }
    if (leader) {
      if (!ok) p_fail(io.status, abort_flag);
      commit(mma_fin);   // every MMA issued above has completed when this phase does
      (void)mbar_wait(mma_fin, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    if constexpr (CHAINS) reg_dec<P_REGS_LO>();
  } else {
    // ---- softmax of chain x
    if constexpr (CHAINS) reg_inc<P_REGS_HI>();
    const int x = (warp - 4) >> 2;
    const int q4 = warp & 3;                  // tensor-memory lane quarter of this warp
    const int r = q4 * 32 + lane;             // query row of the tile
    const uint32_t lrow = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lrow + P_COL_S + (uint32_t)x * 128;
    const uint32_t tO = tmem + lrow + P_COL_O + (uint32_t)x * 128;
    float4 *stage = reinterpret_cast<float4 *>(sOut + (warp - 4) * P_STAGE);
    const float sl2 = 1.4426950408889634f / sqrtf((float)HD);
    uint32_t ns = 0;                          // key tiles of this chain so far
    bool ok = true;
    for (int kind = 0; CHAINS && kind < 2 && ok; ++kind) {
      if (start[kind == PAGED_WIDE ? 0 : 1 + x].u1 == 0) continue;
      PagedWalk w;
      for (w.begin(p, kind, start[kind == PAGED_WIDE ? 0 : 1 + x]); w.more(); w.next(p)) {
        const int tile0 = kind == PAGED_WIDE ? x * qn : 0;        // first token of the chain's tile
        const int rows = min(qn, w.toks - tile0) * rep;           // at least one token
        const int tl = tile0 + paged_token(io, min(r, rows - 1)); // this row's token in the item
        const bool warp_on = q4 * 32 < rows;                      // any row of this warp
        const int seen = w.s.causal ? w.s.keys - w.s.n + w.tok + tl + 1 : w.keys;
        float m_use = -INFINITY, l = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++ns) {
          if (__any_sync(FULL, *abort_flag != 0)) { ok = false; break; }
          if (!__all_sync(FULL, mbar_wait(&s_full[x], ns & 1))) {
            p_fail(io.status, abort_flag);
            ok = false;
            break;
          }
          fence_after();
          if (warp_on) {
            const int lim = seen - t * KT;
            // the row of S: two 64-column loads
            uint32_t sa[64], sb[64];
            tmem_ld64(tS, sa);
            tmem_ld64(tS + 64, sb);
            tmem_ld_wait64(sa);
            tmem_ld_wait64(sb);
            if (__any_sync(FULL, lim < KT)) {
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
                m4[(j >> 1) & 3] =
                    max3(m4[(j >> 1) & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            };
            fold_max(sa);
            fold_max(sb);
            const float m_new = fmaxf(m_use, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2);
            // O is rescaled only when a row's maximum grew by more than 2^8 (P stays below 256, and
            // O and l share their base, so O / l does not change); S of this tile was issued behind
            // the last P V, so O includes it
            // (rows past the item's last hold another's, or what was in shared memory: not asked, so
            // that results do not depend on them)
            if (__any_sync(FULL, r < rows && m_use != -INFINITY && m_new > m_use + P_RESCALE)) {
              const float g = m_use == -INFINITY ? 1.f : ex2(m_use - m_new);
#pragma unroll 1
              for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * g);
                tmem_st32(tO + c * 32, o);
              }
              tmem_st_wait();
              l *= g;
              m_use = m_new;
            } else if (m_use == -INFINITY) {
              m_use = m_new;
            }
            const float nb = m_use == -INFINITY ? 0.f : -m_use;
            const float2 sl2v = make_float2(sl2, sl2), nbv = make_float2(nb, nb);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto emit = [&](const uint32_t (&v)[64], int hf) {   // P of 64 keys
              uint32_t pb[32];
#pragma unroll
              for (int j = 0; j < 64; j += 2) {
                const float2 t2 = __ffma2_rn(
                    make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sl2v, nbv);
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
        if (!__all_sync(FULL, mbar_wait(&pv_done[x], (ns - 1) & 1))) {
          p_fail(io.status, abort_flag);
          ok = false;
          break;
        }
        fence_after();
        if (warp_on) {
          const int worker =
              paged_first_worker(io, kind) + start[kind == PAGED_WIDE ? 0 : 1 + x].worker;
          const PagedDest dest = paged_dest(p, io, w, worker);
          const int on = min(32, rows - q4 * 32);       // rows of this warp
          const bool out = dest.kind == PAGED_OUT;
          // Rows leave through shared memory, so that 8 lanes write 32 columns of one row together:
          // stored straight from the lanes that hold them, each store touched 32 lines (9000 cycles
          // for 256 rows of 128 fp32 columns).
          const int tok_w = w.s.tok0 + w.tok + tile0, h0 = w.head * rep;
          auto dst_row = [&](int i) {   // of row i of this warp
            const int rr = q4 * 32 + i, tl = paged_token(io, rr);
            return paged_dest_row(io, dest, tile0 * rep + rr, tok_w + tl, h0 + rr - tl * rep);
          };
          const size_t base = paged_dest_base(p, io, dest);
          int row8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) row8[i] = dst_row(i * 4 + (lane >> 3));
          const float g = out ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stage[lane * 8 + (j ^ (lane & 7))] =
                  make_float4(__uint_as_float(o[4 * j]) * g, __uint_as_float(o[4 * j + 1]) * g,
                              __uint_as_float(o[4 * j + 2]) * g, __uint_as_float(o[4 * j + 3]) * g);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3), col = c * 32 + (lane & 7) * 4;
              if (i * 4 >= on) break;
              const float4 v = stage[rr * 8 + ((lane & 7) ^ (rr & 7))];
              if (rr < on) {
                const size_t e = (base + row8[i]) * HD + col;
                if (out) store4<bf16>((bf16 *)io.out + e, v.x, v.y, v.z, v.w);
                else *reinterpret_cast<float4 *>(io.part_o + e) = v;
              }
            }
            __syncwarp();
          }
          if (!out && lane < on) {
            io.part_ml[base + dst_row(lane)] = make_float2(m_use, l);
            if (dest.redirect)
              paged_redirect(p, io, dest, worker, w.s.tok0 + w.tok + tl, h0 + r - (tl - tile0) * rep);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_empty[x]);
      }
    }
    // ---- few-row items
    // A CTA serves one kind of work (paged_share), so a CTA that has few-row items has nothing for its
    // chains: their query tiles and key ring are idle from the start, and hold the rings here.
    __syncwarp();
    const PagedStart &few_start = start[3 + warp - 4];
    if (ok && few_start.u0 < few_start.u1) {
      constexpr int ROW = HD * 2, SLOT = F_KT * ROW;            // a slot: 32 keys, chunks swizzled
      const int fw = warp - 4, gr = lane >> 2, tq = lane & 3;   // fragment row and column pair
      uint8_t *ring = sQ + fw * F_SLOTS * SLOT;
      const int shift = io.page_shift;
      // Copies run F_SLOTS slots ahead of the arithmetic, across items: slot n of the walk is K (n
      // even) or V of a step, one group of cp.async each.  Rows behind the last key are filled
      // with zeros. Each lane holds the place of a page, 32 pages of a sequence at a time
      // (PagedWindow). The loading side walks the items and leaves each piece's description for the
      // computing side.
      PagedFewWalk lw;
      lw.begin(p, few_start);
      PagedWindow win;
      int lt = lw.t0, ids = 0;   // ids: first row (for kv head 0) of the window's page `lane`, -1: none
      bool lv = false;
      uint32_t ls_slot = 0, slot = 0;                           // slots loaded and used next
      FewPiece *pieces = reinterpret_cast<FewPiece *>(stage);   // [4], this warp's
      uint32_t lp = 0, np = 0;                                  // pieces described and computed
      int t = 0, t1 = 0, lead = F_SLOTS;
      bool v_half = false;
      int seen[2] = {0, 0};                                     // keys that rows gr and gr + 8 see
      uint32_t qf[HD / 16][4], ph[2][4], pl[2][4];
      float o[HD / 8][4], m[2], ls[2];
      for (;;) {
        if (lead > 0) {
          --lead;
        } else if (!v_half) {
          if (t == t1) {   // the next piece: Q as the A operand, rows gr and gr + 8
            if (np == lp) break;
            const FewPiece pc = pieces[np & 3];
            const int rows = pc.toks * rep, h0 = pc.head * rep;
            t = pc.t0;
            t1 = pc.t1;
            // (rows past the last repeat it and are not stored)
            const bf16 *q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int rr = min(gr + 8 * i, rows - 1), tl = paged_token(io, rr);
              q[i] = (const bf16 *)io.q + ((size_t)(pc.tok + tl) * io.Hq + h0 + rr - tl * rep) * HD + tq * 2;
              seen[i] = pc.before < 0 ? pc.keys : pc.before + tl + 1;
              m[i] = -INFINITY;
              ls[i] = 0.f;
            }
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                qf[kk][i] = *reinterpret_cast<const uint32_t *>(q[i & 1] + kk * 16 + (i >> 1) * 8);
#pragma unroll
            for (int j = 0; j < HD / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
          }
          const int k0 = t * F_KT;
          cp_wait<F_SLOTS - 1>();
          __syncwarp();
          float s[4][4] = {};
          const uint8_t *K = ring + slot * SLOT;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
              uint32_t b[4];
              const int mi = lane >> 3, key = nn * 16 + (mi >> 1) * 8 + (lane & 7);
              ldsm_x4(b, K + key * ROW + (((kk * 2 + (mi & 1)) ^ (key & 7)) << 4));
              mma_16816(s[2 * nn], qf[kk], b[0], b[1]);
              mma_16816(s[2 * nn + 1], qf[kk], b[2], b[3]);
            }
          // rows gr (i = 0) and gr + 8: mask, running maximum, numerators
          float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + j * 8 + tq * 2 + (e & 1);
              s[j][e] = key < seen[e >> 1] ? s[j][e] * sl2 : -INFINITY;
              mt[e >> 1] = fmaxf(mt[e >> 1], s[j][e]);
            }
          float grow = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mt[i] = fmaxf(mt[i], __shfl_xor_sync(FULL, mt[i], 1));
            mt[i] = fmaxf(mt[i], __shfl_xor_sync(FULL, mt[i], 2));
            if (m[i] == -INFINITY) m[i] = mt[i];
            else grow = fmaxf(grow, mt[i] - m[i]);
          }
          if (__any_sync(FULL, grow > P_RESCALE)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mn = fmaxf(m[i], mt[i]);
              const float g = m[i] == -INFINITY ? 1.f : ex2(m[i] - mn);
              m[i] = mn;
              ls[i] *= g;
#pragma unroll
              for (int j = 0; j < HD / 8; ++j) {
                o[j][2 * i] *= g;
                o[j][2 * i + 1] *= g;
              }
            }
          }
          // P as the A operand in two bf16 parts (16 significant bits; these products are cheap)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float base = m[i] == -INFINITY ? 0.f : m[i];
              const float e0 = ex2(s[j][2 * i] - base), e1 = ex2(s[j][2 * i + 1] - base);
              ls[i] += e0 + e1;
              const __nv_bfloat162 hi = __floats2bfloat162_rn(e0, e1);
              const __nv_bfloat162 lo =
                  __floats2bfloat162_rn(e0 - __low2float(hi), e1 - __high2float(hi));
              ph[j >> 1][2 * (j & 1) + i] = *reinterpret_cast<const uint32_t *>(&hi);
              pl[j >> 1][2 * (j & 1) + i] = *reinterpret_cast<const uint32_t *>(&lo);
            }
          v_half = true;
          slot = slot + 1 == F_SLOTS ? 0 : slot + 1;
        } else {
          cp_wait<F_SLOTS - 1>();
          __syncwarp();
          const uint8_t *V = ring + slot * SLOT;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int nn = 0; nn < HD / 16; ++nn) {
              uint32_t b[4];
              const int mi = lane >> 3, key = kk * 16 + (mi & 1) * 8 + (lane & 7);
              ldsm_x4_t(b, V + key * ROW + (((nn * 2 + (mi >> 1)) ^ (key & 7)) << 4));
              mma_16816(o[2 * nn], ph[kk], b[0], b[1]);
              mma_16816(o[2 * nn], pl[kk], b[0], b[1]);
              mma_16816(o[2 * nn + 1], ph[kk], b[2], b[3]);
              mma_16816(o[2 * nn + 1], pl[kk], b[2], b[3]);
            }
          v_half = false;
          slot = slot + 1 == F_SLOTS ? 0 : slot + 1;
          if (++t == t1) {   // the piece's result
            const FewPiece pc = pieces[np & 3];
            const int rows = pc.toks * rep, h0 = pc.head * rep;
            const int worker = paged_first_worker(io, PAGED_FEW) + few_start.worker;
            const PagedDest dest = paged_dest(p, io, pc.which, pc.t0 == 0, pc.whole, worker);
            const size_t base = paged_dest_base(p, io, dest);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (8 * i >= rows) break;
              ls[i] += __shfl_xor_sync(FULL, ls[i], 1);
              ls[i] += __shfl_xor_sync(FULL, ls[i], 2);
              const int rr = gr + 8 * i;
              if (rr >= rows) continue;
              const int tl = paged_token(io, rr), tok = pc.tok + tl, h = h0 + rr - tl * rep;
              const size_t row = base + paged_dest_row(io, dest, rr, tok, h);
              if (dest.kind == PAGED_OUT) {
                const float il = ls[i] > 0.f ? 1.f / ls[i] : 0.f;
                bf16 *dst = (bf16 *)io.out + row * HD + tq * 2;
#pragma unroll
                for (int j = 0; j < HD / 8; ++j)
                  *reinterpret_cast<__nv_bfloat162 *>(dst + j * 8) =
                      __floats2bfloat162_rn(o[j][2 * i] * il, o[j][2 * i + 1] * il);
              } else {
                float *dst = io.part_o + row * HD + tq * 2;
#pragma unroll
                for (int j = 0; j < HD / 8; ++j)
                  *reinterpret_cast<float2 *>(dst + j * 8) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
                if (tq == 0) {
                  io.part_ml[row] = make_float2(m[i], ls[i]);
                  if (dest.redirect) paged_redirect(p, io, dest, worker, tok, h);
                }
              }
            }
            ++np;
          }
        }
        __syncwarp();   // every lane has read the slot that is loaded now
        if (lw.more()) {
          if (!lv && lt == lw.t0) {   // a piece begins: at most three are described and not yet done
            if (lane == 0)
              pieces[lp & 3] = FewPiece{lw.tok, lw.toks, lw.head, lw.keys, lw.before, lw.t0, lw.t1,
                                        lw.which, lw.whole()};
            ++lp;
          }
          const int pos = lw.key0 + lt * F_KT, pg = pos >> shift, live = lw.keys - lt * F_KT;
          const int pg2 = (pos + 16) >> shift;   // page of the second 16 keys
          if (win.move(lw, pg, pg2)) {
            ids = -1;
            if (win.filled(lw, lane, shift)) {
              const long long row = paged_row(io, p, lw.seq, 0, (pg + lane) << shift);
              ids = row < 0 ? -1 : (int)row;
            }
          }
          const bf16 *pool = (const bf16 *)(lv ? io.v_pages : io.k_pages);
          uint8_t *dst = ring + ls_slot * SLOT;
          constexpr int CPR = HD / 8, RPI = 32 / CPR;   // chunks in a row, rows a warp copies at once
          const int c = lane % CPR, r0 = lane / CPR;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int first = __shfl_sync(FULL, ids, (g ? pg2 : pg) - win.first);
            const int at = first + (lw.head << shift) + ((pos + 16 * g) & ((1 << shift) - 1));
            const bf16 *src = pool + (size_t)(first < 0 ? 0 : at) * HD + c * 8;
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
              const int r = i * RPI + r0, key = 16 * g + r;
              const bool on = first >= 0 && key < live;   // a bad page id, no key: zeros
              cp_async16(dst + key * ROW + ((c ^ (key & 7)) << 4), on ? src + r * HD : pool, on);
            }
          }
          ls_slot = ls_slot + 1 == F_SLOTS ? 0 : ls_slot + 1;
          if (lv && ++lt == lw.t1) {
            lw.next(p);
            lt = lw.t0;
          }
          lv = !lv;
        }
        cp_commit();   // (empty at the end, so that the count of groups in flight stays the same)
      }
    }
  }
  if constexpr (CHAINS) {
    fence_before();
    __syncthreads();
    if (warp == 1) {
      fence_after();
      tmem_dealloc(tmem, P_TMEM);
    }
  }
}

template <int HD, bool CHAINS>
int launch_tc(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PagedShape &p,
              const PagedIO &io, cudaStream_t s) {
  constexpr size_t smem = Tc<HD>::SMEM;
  note_launch(s, "paged_attn_tc");
  cudaFuncSetAttribute(paged_attn_tc_kernel<HD, CHAINS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)smem);
  launch_pdl(paged_attn_tc_kernel<HD, CHAINS>, io.ctas, P_THR, smem, s, tq, tk, tv, p, io);
  return check_launch("paged_attn_tc");
}

template <int HD>
int run_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  // the register split inside the kernel needs the launch to hold P_REGS registers per thread; a
  // build with fewer would leave setmaxnreg.inc waiting, so it is refused here
  static const int regs = [] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, paged_attn_tc_kernel<HD, true>) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (regs < P_REGS) return DG_ERR_UNSUPPORTED;
  CUtensorMap tq{}, tk{}, tv{};
  if (paged_all_few(p)) return launch_tc<HD, false>(tq, tk, tv, p, io, s);
  const uint64_t rows = (uint64_t)c.n_pages * c.Hkv * c.page_size;
  const uint32_t box = c.page_size < PAGED_TC_KT ? c.page_size : PAGED_TC_KT;
  const CUtensorMapDataType bt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = make_tmap_3d(&tq, bt, 2, c.q, HD, c.Hq, c.n_tokens, HD * 2,
                        (uint64_t)c.Hq * HD * 2, 64, io.rep, p.qn);
  if (rc == DG_OK) rc = make_tmap_2d(&tk, bt, 2, c.k_pages, HD, rows, HD * 2, 64, box);
  if (rc == DG_OK) rc = make_tmap_2d(&tv, bt, 2, c.v_pages, HD, rows, HD * 2, 64, box);
  if (rc != DG_OK) return rc;
  return launch_tc<HD, true>(tq, tk, tv, p, io, s);
}

}  // namespace

int launch_paged_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s) {
  return c.hd == 128 ? run_tc<128>(c, p, io, s) : run_tc<64>(c, p, io, s);
}

}  // namespace dg
