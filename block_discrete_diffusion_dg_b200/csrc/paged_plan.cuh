// How the paged attention splits its work over a fixed grid.
//
// Every query tile of a sequence (an "item": the query heads of one kv head times up to `qt`
// consecutive tokens) costs one unit per key tile it visits.  All units of the call, ordered by
// (sequence, kv head, item, key tile), are cut into equal ranges of `per` units, one per CTA, so
// the load is even whatever the lengths are: a batch of short and long sequences, the triangle of
// a causal prompt, or one long context with a few rows.  An item cut by a range boundary leaves
// one partial result per piece, and the pieces are joined afterwards in the order of their keys.
// Lengths live on the device, so each CTA derives its range itself: a warp scans the sequences
// (32 at a time) and searches the item within the sequence.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DG_HD __host__ __device__ __forceinline__
#else
#define DG_HD inline
#endif

namespace dg {

struct PagedShape {
  const int32_t *seq_off;   // [n_seqs + 1] first packed row of each sequence
  const int32_t *kv_len;    // [n_seqs] keys cached before the new tokens
  int n_seqs, n_tokens;     // n_tokens: packed rows of q and out
  int Hkv;
  int qt;                   // tokens per item
  int qn;                   // an item of at most qn tokens is narrow: one unit covers two key tiles
  int kt;                   // keys per tile
  int causal;
  int shared_len;           // > 0: keys [0, shared_len) form segment 0, seen by every token
  int cap;                  // keys a page-table row can address
};

// A run of packed query rows with the keys it sees: one sequence, or (index 0 of a call with a
// shared prefix) all rows over the prefix.
struct PagedSeg {
  int tok0, n;              // packed rows [tok0, tok0 + n); n == 0: nothing to do
  int key0, keys;           // keys [key0, key0 + keys) of the sequence; the last n are the new ones
  int causal;               // when causal
  int seq;                  // page-table row
  int error;                // 0, 1: malformed offsets or lengths, 2: keys past the page table
};

DG_HD int paged_segs(const PagedShape &p) { return p.n_seqs + (p.shared_len > 0 ? 1 : 0); }

DG_HD PagedSeg paged_seg(const PagedShape &p, int index) {
  PagedSeg s;
  s.error = 0;
  if (p.shared_len > 0) {
    if (index == 0) {
      const int last = p.seq_off[p.n_seqs];
      s.tok0 = 0;
      s.n = last < 0 ? 0 : (last > p.n_tokens ? p.n_tokens : last);
      s.key0 = 0;
      s.keys = p.shared_len;
      s.causal = 0;
      s.seq = 0;
      return s;
    }
    --index;
  }
  const int a = p.seq_off[index], b = p.seq_off[index + 1], have = p.kv_len[index];
  s.seq = index;
  s.causal = p.causal;
  s.tok0 = a;
  s.n = b - a;
  s.key0 = p.shared_len;
  s.keys = 0;
  if (a == b) {
    s.n = 0;
  } else if (a < 0 || b < a || b > p.n_tokens || have < p.shared_len) {
    s.n = 0;
    s.error = 1;
  } else if ((long long)have + s.n > p.cap) {
    s.n = 0;
    s.error = 2;
  } else {
    s.keys = have - p.shared_len + s.n;
  }
  return s;
}

// sum_{i < n} floor((a i + b) / m) for a, b >= 0, m > 0.
DG_HD long long floor_sum(long long n, long long m, long long a, long long b) {
  long long r = 0;
  while (n > 0) {
    if (a >= m) {
      r += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      r += n * (b / m);
      b %= m;
    }
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return r;
}

DG_HD int paged_items(const PagedShape &p, const PagedSeg &s) { return (s.n + p.qt - 1) / p.qt; }
DG_HD int paged_item_tokens(const PagedShape &p, const PagedSeg &s, int i) {
  const int left = s.n - i * p.qt;
  return left < p.qt ? left : p.qt;
}
// Keys and key tiles that item i of segment s visits.
DG_HD int paged_item_keys(const PagedShape &p, const PagedSeg &s, int i) {
  if (!s.causal) return s.keys;
  return s.keys - s.n + i * p.qt + paged_item_tokens(p, s, i);
}
DG_HD int paged_item_tiles(const PagedShape &p, const PagedSeg &s, int i) {
  return (paged_item_keys(p, s, i) + p.kt - 1) / p.kt;
}
DG_HD int paged_item_units(const PagedShape &p, const PagedSeg &s, int i) {
  const int t = paged_item_tiles(p, s, i);
  return paged_item_tokens(p, s, i) <= p.qn ? (t + 1) / 2 : t;
}
// Units of the first q items (of one kv head); every item but the last is full and wide.
DG_HD long long paged_units_before(const PagedShape &p, const PagedSeg &s, int q) {
  const int items = paged_items(p, s);
  if (q <= 0 || items == 0) return 0;
  const int wide = q < items ? q : items - 1;
  long long r;
  if (s.causal)
    r = floor_sum(wide, p.kt, p.qt, (long long)s.keys - s.n + p.qt + p.kt - 1);
  else
    r = (long long)wide * ((s.keys + p.kt - 1) / p.kt);
  return q < items ? r : r + paged_item_units(p, s, items - 1);
}
DG_HD long long paged_seg_units(const PagedShape &p, const PagedSeg &s) {
  return s.n > 0 ? p.Hkv * paged_units_before(p, s, paged_items(p, s)) : 0;
}

// One CTA's place in the work: the item it begins in and the unit range it owns.
struct PagedStart {
  long long u0, u1;         // owned units [u0, u1); u0 >= u1: none
  long long item_u0;        // first unit of the item that holds u0
  long long per;            // units per CTA
  int seg, head, item;
};

#ifdef __CUDACC__
// Called by one whole warp.  *error: the largest error code of any sequence, for the caller to
// record.
__device__ inline PagedStart paged_locate(const PagedShape &p, int cta, int ctas, int *error) {
  const int lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  const int segs = paged_segs(p);
  long long total = 0;
  int err = 0;
  for (int b = 0; b < segs; b += 32) {
    long long w = 0;
    if (b + lane < segs) {
      const PagedSeg s = paged_seg(p, b + lane);
      w = paged_seg_units(p, s);
      err = err > s.error ? err : s.error;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(full, w, o);
    total += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const int e = __shfl_xor_sync(full, err, o);
    err = err > e ? err : e;
  }
  *error = err;
  PagedStart r;
  r.per = (total + ctas - 1) / ctas;
  r.u0 = cta * r.per;
  r.u1 = r.u0 + r.per < total ? r.u0 + r.per : total;
  r.seg = r.head = r.item = 0;
  r.item_u0 = 0;
  if (r.u0 >= r.u1) {
    r.u0 = r.u1 = 0;
    return r;
  }
  long long before = 0;
  for (int b = 0; b < segs; b += 32) {
    long long w = 0;
    if (b + lane < segs) w = paged_seg_units(p, paged_seg(p, b + lane));
    long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(full, inc, o);
      if (lane >= o) inc += t;
    }
    const unsigned hit = __ballot_sync(full, before + inc > r.u0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      r.seg = b + l;
      before += __shfl_sync(full, inc - w, l);
      break;
    }
    before += __shfl_sync(full, inc, 31);
  }
  const PagedSeg s = paged_seg(p, r.seg);
  const long long each = paged_units_before(p, s, paged_items(p, s));
  r.head = (int)((r.u0 - before) / each);
  before += r.head * each;
  // the last item whose first unit is <= u0: 32-way search
  int lo = 0, hi = paged_items(p, s);
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool le = i < hi && before + paged_units_before(p, s, i) <= r.u0;
    const int l = 31 - __clz(__ballot_sync(full, le));  // lane 0 always holds
    lo += l * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  r.item = lo;
  r.item_u0 = before + paged_units_before(p, s, lo);
  return r;
}
#endif

// Walks the pieces of a CTA's range [u0, u1) in order: after begin(), while (more()), units
// [k0(), k1()) of the current item of `units()` units.
struct PagedWalk {
  PagedSeg s;
  int seg, head, item, items, n_units;
  long long u, u1, item_u0;

  DG_HD void begin(const PagedShape &p, const PagedStart &st) {
    seg = st.seg;
    head = st.head;
    item = st.item;
    u = st.u0;
    u1 = st.u1;
    item_u0 = st.item_u0;
    if (!more()) return;
    s = paged_seg(p, seg);
    items = paged_items(p, s);
    n_units = paged_item_units(p, s, item);
  }
  DG_HD bool more() const { return u < u1; }
  DG_HD int units() const { return n_units; }
  DG_HD int k0() const { return (int)(u - item_u0); }
  DG_HD int k1() const { return u1 - item_u0 < n_units ? (int)(u1 - item_u0) : n_units; }
  DG_HD void next(const PagedShape &p) {
    item_u0 += n_units;
    u = item_u0;  // past u1 when the piece ended inside its item
    if (!more()) return;
    if (++item == items) {
      item = 0;
      if (++head == p.Hkv) {
        head = 0;
        do {  // units remain, so a later segment has rows
          s = paged_seg(p, ++seg);
        } while (s.n == 0);
        items = paged_items(p, s);
      }
    }
    n_units = paged_item_units(p, s, item);
  }
};

// What CTA c leaves about the item that its range begins in, for joining the pieces.
struct PagedHead {
  int joins;    // 1: the range begins inside an item, and is the first boundary inside it
  int last;     // CTA that holds the item's last unit
  int tok0, tokens, head;   // packed rows and kv head of the item
  int pad[3];
};

}  // namespace dg
