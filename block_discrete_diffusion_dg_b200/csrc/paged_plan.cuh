// How the paged attention splits its work over a fixed grid.
//
// An item is the query heads of one kv head times up to `qt` consecutive tokens of a sequence, against
// the key tiles they see; its cost is the number of those tiles plus a constant for starting and
// storing it.  The costs of all items, ordered by (sequence, kv head, item, key tile), are cut into
// equal ranges, one per worker, so the load is even whatever the lengths are: a batch of short and
// long sequences, the triangle of a causal prompt, or one long context with a few rows.  An item cut
// by a range boundary leaves one partial result per piece, and the pieces are joined afterwards in the
// order of their keys.
// There are three kinds of items, each with workers of its own: wide items (two query tiles that share
// each key tile; a worker is a CTA), narrow ones (a sequence's last item if it has at most `qn` tokens:
// one query tile; a worker is one of a CTA's two chains) and few-row ones (the last item if it has at
// most `qf` tokens: single tokens and short tails; a worker is one of eight warps of a CTA).
// Lengths live on the device, so each worker derives its range itself: a warp scans the sequences
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
  int qn;                   // a last item of at most qn tokens is narrow (0: none is),
  int qf;                   // of at most qf <= qn few-row (0: none is)
  // by kind of item:
  int kt[3];                // keys per tile
  int start_cost[3];        // cost of starting and storing an item, in key tiles
  int least[3];             // least cost worth a worker of its own
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

enum { PAGED_WIDE = 0, PAGED_NARROW = 1, PAGED_FEW = 2 };

// The kind of a segment's last item where it is not wide, else PAGED_WIDE.
DG_HD int paged_tail_kind(const PagedShape &p, const PagedSeg &s) {
  const int tail = s.n % p.qt;
  return tail == 0 || tail > p.qn ? PAGED_WIDE : tail > p.qf ? PAGED_NARROW : PAGED_FEW;
}
// Items of a kind in one kv head of segment s, and the index of the first.
DG_HD int paged_items(const PagedShape &p, const PagedSeg &s, int kind) {
  const int tail = paged_tail_kind(p, s);
  if (kind != PAGED_WIDE) return tail == kind ? 1 : 0;
  return tail == PAGED_WIDE ? (s.n + p.qt - 1) / p.qt : s.n / p.qt;
}
DG_HD int paged_first_item(const PagedShape &p, const PagedSeg &s, int kind) {
  return kind == PAGED_WIDE ? 0 : s.n / p.qt;
}
DG_HD int paged_item_tokens(const PagedShape &p, const PagedSeg &s, int i) {
  const int left = s.n - i * p.qt;
  return left < p.qt ? left : p.qt;
}
// Keys and key tiles that item i of segment s visits.
DG_HD int paged_item_keys(const PagedShape &p, const PagedSeg &s, int i) {
  if (!s.causal) return s.keys;
  return s.keys - s.n + i * p.qt + paged_item_tokens(p, s, i);
}
DG_HD int paged_item_tiles(const PagedShape &p, const PagedSeg &s, int kind, int i) {
  return (paged_item_keys(p, s, i) + p.kt[kind] - 1) / p.kt[kind];
}
// Cost of the first q items of a kind (of one kv head).
DG_HD long long paged_cost_before(const PagedShape &p, const PagedSeg &s, int kind, int q) {
  if (q <= 0) return 0;
  if (kind != PAGED_WIDE)
    return paged_item_tiles(p, s, kind, paged_first_item(p, s, kind)) + p.start_cost[kind];
  const long long start = (long long)q * p.start_cost[kind];
  if (!s.causal) return start + (long long)q * paged_item_tiles(p, s, kind, 0);
  // full items by their sum, the last one (which may have fewer tokens) by itself
  const bool last = q == paged_items(p, s, kind);
  const long long r =
      floor_sum(last ? q - 1 : q, p.kt[kind], p.qt,
                (long long)s.keys - s.n + p.qt + p.kt[kind] - 1);
  return start + (last ? r + paged_item_tiles(p, s, kind, q - 1) : r);
}
DG_HD long long paged_head_cost(const PagedShape &p, const PagedSeg &s, int kind) {
  return s.n > 0 ? paged_cost_before(p, s, kind, paged_items(p, s, kind)) : 0;
}

// A worker's place in the work of a kind: its range [u0, u1) of the total cost (u0 >= u1: none) and
// the item that it begins in.
struct PagedStart {
  long long u0, u1;
  long long item_u0;        // where the item that holds u0 begins
  long long per;            // cost per worker
  int seg, head, item;
};

#ifdef __CUDACC__
// Called by one whole warp.  *error: the largest error code of any sequence, for the caller to
// record.
__device__ inline PagedStart paged_locate(const PagedShape &p, int kind, int worker, int workers,
                                          int *error) {
  const int lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  const int segs = paged_segs(p);
  long long total = 0;
  int err = 0;
  for (int b = 0; b < segs; b += 32) {
    long long w = 0;
    if (b + lane < segs) {
      const PagedSeg s = paged_seg(p, b + lane);
      w = p.Hkv * paged_head_cost(p, s, kind);
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
  r.per = (total + workers - 1) / workers;
  if (r.per < p.least[kind]) r.per = p.least[kind];
  r.u0 = worker * r.per;
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
    if (b + lane < segs) w = p.Hkv * paged_head_cost(p, paged_seg(p, b + lane), kind);
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
  const long long each = paged_head_cost(p, s, kind);
  r.head = (int)((r.u0 - before) / each);
  before += r.head * each;
  // the last item that begins at or before u0: 32-way search
  int lo = 0, hi = paged_items(p, s, kind);
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool le = i < hi && before + paged_cost_before(p, s, kind, i) <= r.u0;
    const int l = 31 - __clz(__ballot_sync(full, le));  // lane 0 always holds
    lo += l * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  r.item = lo;
  r.item_u0 = before + paged_cost_before(p, s, kind, lo);
  return r;
}
#endif

// Walks the pieces of a worker's range in order: after begin(), while (more()), key tiles [t0, t1) of
// item `item` (tokens [tok, tok + toks) of segment s, kv head `head`).  The starting cost of an item
// lies before its first tile, and a range that ends within it leaves the item to the next worker.
struct PagedWalk {
  PagedSeg s;
  int seg, head, index, items;        // index: among the items of the kind
  int item, tok, toks, keys, tiles;   // the current item; keys it visits
  int t0, t1;
  int kind;
  long long u1, item_u0, u;

  DG_HD void begin(const PagedShape &p, int kind_, const PagedStart &st) {
    kind = kind_;
    seg = st.seg;
    head = st.head;
    index = st.item;
    u = st.u0;
    u1 = st.u1;
    item_u0 = st.item_u0;
    if (u >= u1) return;
    s = paged_seg(p, seg);
    items = paged_items(p, s, kind);
    load(p);
    if (t0 >= t1) next(p);
  }
  DG_HD bool more() const { return u < u1; }
  DG_HD bool whole() const { return t0 == 0 && t1 == tiles; }
  DG_HD void load(const PagedShape &p) {
    item = paged_first_item(p, s, kind) + index;
    tok = item * p.qt;
    toks = paged_item_tokens(p, s, item);
    keys = paged_item_keys(p, s, item);
    tiles = (keys + p.kt[kind] - 1) / p.kt[kind];
    const int c = p.start_cost[kind];
    const long long a = u - item_u0 - c, b = u1 - item_u0 - c;
    t0 = a > 0 ? (int)a : 0;
    t1 = b < tiles ? (b > 0 ? (int)b : 0) : tiles;
  }
  DG_HD void next(const PagedShape &p) {
    do {
      item_u0 += tiles + p.start_cost[kind];
      u = item_u0;
      if (!more()) return;
      if (++index == items) {
        index = 0;
        if (++head == p.Hkv) {
          head = 0;
          do {  // cost remains, so a later segment has items
            s = paged_seg(p, ++seg);
            items = s.n > 0 ? paged_items(p, s, kind) : 0;
          } while (items == 0);
        }
      }
      load(p);
    } while (t0 >= t1);
  }
};

// What a worker leaves about the item that its range goes on with, for joining the pieces.
struct PagedHead {
  int joins;    // 1: the range begins inside an item whose first piece lies with the worker before
  int last;     // worker (of the kind) that holds the item's last tile
  int tok0, tokens, head;   // packed rows and kv head of the item
  int pad[3];
};
DG_HD PagedHead paged_head(const PagedShape &p, int kind, const PagedStart &st) {
  PagedHead h = {0, 0, 0, 0, 0, {0, 0, 0}};
  const int c = p.start_cost[kind];
  const long long in = st.u0 - st.item_u0;
  if (st.u0 < st.u1 && in > c) {
    const PagedSeg s = paged_seg(p, st.seg);
    const int item = paged_first_item(p, s, kind) + st.item;
    const long long end = st.item_u0 + c + paged_item_tiles(p, s, kind, item);
    h.joins = in - st.per <= c;
    h.last = (int)((end - 1) / st.per);
    h.tok0 = s.tok0 + item * p.qt;
    h.tokens = paged_item_tokens(p, s, item);
    h.head = st.head;
  }
  return h;
}

}  // namespace dg
