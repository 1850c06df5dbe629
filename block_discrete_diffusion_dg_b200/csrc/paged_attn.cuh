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
  int rows;                      // rows of a partial result's slot
  int ctas;
  PagedHead *heads;              // [ctas]
  // rows of fp32 partial results: 2 slots per CTA, then (shared prefix) a region [2][n_tokens][Hq]
  float *part_o;
  float2 *part_ml;               // (m, l) of each row; l < 0 in the region: see paged_redirect
  int32_t *status;
};

// Tensor-core kernel (k_paged_attn_tc.cu): query rows and keys per tile.
constexpr int PAGED_TC_ROWS = 128, PAGED_TC_KT = 128;
inline bool paged_tc_supported(int act, int hd) { return act == DG_BF16 && (hd == 64 || hd == 128); }
struct PagedCall;
int launch_paged_tc(const PagedCall &c, const PagedShape &p, const PagedIO &io, cudaStream_t s);

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

// ---- destinations -------------------------------------------------------------------------------
enum { PAGED_OUT = 0, PAGED_REGION = 1, PAGED_SLOT = 2 };
struct PagedDest {
  int kind;
  int which;      // region half: 0 the shared prefix, 1 the sequence's own keys
  size_t slot;    // first row of the slot
  bool redirect;  // the first of several pieces: the region entry points to them
};

__device__ __forceinline__ size_t paged_slot_row(const PagedIO &io, int cta, bool begins, int r) {
  return (size_t)(2 * cta + (begins ? 1 : 0)) * io.rows + r;
}
__device__ __forceinline__ size_t paged_region_row(const PagedShape &p, const PagedIO &io,
                                                   int which, int tok, int h) {
  return (size_t)2 * io.ctas * io.rows + ((size_t)which * p.n_tokens + tok) * io.Hq + h;
}

// Where the current piece of a walk goes: a whole item to the output (or its half of the region),
// a part of one to a slot of this CTA (slot 1 if the item begins here, slot 0 if it goes on from
// an earlier CTA; a range holds at most one of each).
__device__ __forceinline__ PagedDest paged_dest(const PagedShape &p, const PagedIO &io,
                                                const PagedWalk &w, int cta) {
  PagedDest d;
  d.which = p.shared_len > 0 && w.seg == 0 ? 0 : 1;
  const bool begins = w.k0() == 0;
  const bool whole = begins && w.k1() == w.units();
  d.kind = !whole ? PAGED_SLOT : p.shared_len > 0 ? PAGED_REGION : PAGED_OUT;
  d.slot = paged_slot_row(io, cta, begins, 0);
  d.redirect = d.kind == PAGED_SLOT && begins && p.shared_len > 0;
  return d;
}
__device__ __forceinline__ size_t paged_part_row(const PagedShape &p, const PagedIO &io,
                                                 const PagedDest &d, int r, int tok, int h) {
  return d.kind == PAGED_SLOT ? d.slot + r : paged_region_row(p, io, d.which, tok, h);
}
__device__ __forceinline__ void paged_redirect(const PagedShape &p, const PagedIO &io,
                                               const PagedDest &d, int cta, int tok, int h) {
  io.part_ml[paged_region_row(p, io, d.which, tok, h)] = make_float2(__int_as_float(cta), -1.f);
}

// The item that the range of CTA `cta` begins inside, for the join kernels.
__device__ __forceinline__ void paged_write_head(const PagedShape &p, const PagedIO &io,
                                                 const PagedStart &st, int cta) {
  PagedHead h{};
  if (st.u0 < st.u1 && st.u0 > st.item_u0) {
    const PagedSeg s = paged_seg(p, st.seg);
    const long long end = st.item_u0 + paged_item_units(p, s, st.item);
    h.joins = st.u0 - st.item_u0 <= st.per;
    h.last = (int)((end - 1) / st.per);
    h.tok0 = s.tok0 + st.item * p.qt;
    h.tokens = paged_item_tokens(p, s, st.item);
    h.head = st.head;
  }
  io.heads[cta] = h;
}

}  // namespace dg
