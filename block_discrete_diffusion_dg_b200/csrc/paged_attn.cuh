// What the kernels of the paged attention share: pointers, page lookup, and where the result of a
// piece of work goes (see paged_plan.cuh for the pieces).
#pragma once

#include "dg_common.cuh"
#include "paged_plan.cuh"

namespace dg {

struct PagedIO {
  const void *q;                 // [n_tokens][Hq][hd]
  void *out;
  const void *k_pages, *v_pages; // [n_pages][Hkv][page][hd]
  const int32_t *page_table;     // [n_seqs][max_pages]
  int n_pages, max_pages, page_shift;
  int Hq, rep;
  int rep_mul;                   // ceil(2^16 / rep): row / rep by paged_token
  int ctas;
  int workers;                   // of all kinds (see paged_worker)
  int rows[3];                   // rows of a partial result's slot, by kind of item
  PagedHead *heads;              // [workers]
  // rows of fp32 partial results: 2 slots per worker, then (shared prefix) a region
  // [2][n_tokens][Hq]
  size_t region;                 // its first row
  float *part_o;
  float2 *part_ml;               // (m, l) of each row; l < 0 in the region: see paged_redirect
  int32_t *status;
};

// Tensor-core kernel (k_paged_attn_tc.cu): query rows and keys per tile.
constexpr int PAGED_TC_ROWS = 128, PAGED_TC_KT = 128;
constexpr int PAGED_TC_FEW = 16, PAGED_TC_FEW_KT = 32;   // few-row items: rows at most, keys per step
// Starting and storing an item, in key tiles of its kind.
constexpr int PAGED_TC_START_WIDE = 3, PAGED_TC_START_NARROW = 1, PAGED_TC_START_FEW = 1;
inline bool paged_tc_supported(int act, int hd) { return act == DG_BF16 && (hd == 64 || hd == 128); }
struct PagedCall;
int launch_paged_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s);

// Row r of an item is head r % rep of its token r / rep.  The quotient by a multiplication (exact
// for r < 256, rep <= 64: r (rep - 1) < 2^16): rows are turned into tokens and heads in many
// places, and a division is 20 instructions.
__device__ __forceinline__ int paged_token(const PagedIO &io, int r) { return (r * io.rep_mul) >> 16; }

// Row (of hd elements) of key `pos` of a sequence in the page pool, -1 (and the status word set)
// for a page id outside it.
__device__ __forceinline__ long long paged_row(const PagedIO &io, const PagedShape &p, int seq,
                                               int head, int pos) {
  const int id = io.page_table[(size_t)seq * io.max_pages + (pos >> io.page_shift)];
  if ((unsigned)id >= (unsigned)io.n_pages) {
    set_status(io.status, DG_ERR_INVALID_ARG);
    return -1;
  }
  return (((long long)id * p.Hkv + head) << io.page_shift) + (pos & ((1 << io.page_shift) - 1));
}

__device__ __forceinline__ void paged_report(const PagedIO &io, int error) {
  if (error) set_status(io.status, error == 2 ? DG_ERR_CAPACITY : DG_ERR_INVALID_ARG);
}

// ---- destinations
// Workers are numbered through: wide ones [0, ctas), narrow ones (two per CTA) [ctas, 3 ctas), few-row
// ones (eight per CTA) [3 ctas, 11 ctas).
__host__ __device__ inline int paged_first_worker(const PagedIO &io, int kind) {
  return kind == PAGED_WIDE ? 0 : kind == PAGED_NARROW ? io.ctas : 3 * io.ctas;
}
__host__ __device__ inline int paged_worker_kind(const PagedIO &io, int worker) {
  return worker < io.ctas ? PAGED_WIDE : worker < 3 * io.ctas ? PAGED_NARROW : PAGED_FEW;
}
enum { PAGED_OUT = 0, PAGED_REGION = 1, PAGED_SLOT = 2 };
struct PagedDest {
  int kind;
  int which;      // region half: 0 the shared prefix, 1 the sequence's own keys
  size_t slot;    // first row of the slot
  bool redirect;  // the first of several pieces: the region entry points to them
};

// Slots lie kind by kind; paged_slot_row(io, io.workers, false, 0) is their total.
__host__ __device__ inline size_t paged_slot_row(const PagedIO &io, int worker, bool begins, int r) {
  const int kind = paged_worker_kind(io, worker);
  size_t base = 0;
  if (kind >= PAGED_NARROW) base += (size_t)2 * io.ctas * io.rows[PAGED_WIDE];
  if (kind == PAGED_FEW) base += (size_t)4 * io.ctas * io.rows[PAGED_NARROW];
  return base +
         (size_t)(2 * (worker - paged_first_worker(io, kind)) + (begins ? 1 : 0)) * io.rows[kind] + r;
}
__device__ __forceinline__ size_t paged_region_row(const PagedShape &p, const PagedIO &io,
                                                   int which, int tok, int h) {
  return io.region + ((size_t)which * p.n_tokens + tok) * io.Hq + h;
}

// Where a piece goes: a whole item to the output (or its half of the region), a part of one to a
// slot of this worker (slot 1 if the item begins here, slot 0 if it goes on from an earlier
// worker; a range holds at most one of each).
__device__ __forceinline__ PagedDest paged_dest(const PagedShape &p, const PagedIO &io, int which,
                                                bool begins, bool whole, int worker) {
  PagedDest d;
  d.which = which;
  d.kind = !whole ? PAGED_SLOT : p.shared_len > 0 ? PAGED_REGION : PAGED_OUT;
  d.slot = paged_slot_row(io, worker, begins, 0);
  d.redirect = d.kind == PAGED_SLOT && begins && p.shared_len > 0;
  return d;
}
__device__ __forceinline__ PagedDest paged_dest(const PagedShape &p, const PagedIO &io,
                                                const PagedWalk &w, int worker) {
  return paged_dest(p, io, p.shared_len > 0 && w.seg == 0 ? 0 : 1, w.t0 == 0, w.whole(), worker);
}
// Row of the destination that holds packed row (tok, h), row r of the item, without the base.
__device__ __forceinline__ size_t paged_dest_base(const PagedShape &p, const PagedIO &io,
                                                  const PagedDest &d) {
  return d.kind == PAGED_SLOT     ? d.slot
         : d.kind == PAGED_REGION ? paged_region_row(p, io, d.which, 0, 0)
                                  : 0;
}
__device__ __forceinline__ int paged_dest_row(const PagedIO &io, const PagedDest &d, int r, int tok,
                                              int h) {
  return d.kind == PAGED_SLOT ? r : tok * io.Hq + h;
}
__device__ __forceinline__ size_t paged_part_row(const PagedShape &p, const PagedIO &io,
                                                 const PagedDest &d, int r, int tok, int h) {
  return d.kind == PAGED_SLOT ? d.slot + r : paged_region_row(p, io, d.which, tok, h);
}
__device__ __forceinline__ void paged_redirect(const PagedShape &p, const PagedIO &io,
                                               const PagedDest &d, int worker, int tok, int h) {
  io.part_ml[paged_region_row(p, io, d.which, tok, h)] = make_float2(__int_as_float(worker), -1.f);
}

}  // namespace dg
