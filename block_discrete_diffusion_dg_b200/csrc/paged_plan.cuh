// How the paged attention splits its work over a fixed grid.
//
// An item is the query heads of one kv head times up to `qt` consecutive tokens of a sequence,
// against the key tiles they see; its cost is the number of those tiles plus a constant for
// starting and storing it.  The costs of all items, ordered by (sequence, kv head, item, key
// tile), are cut into equal ranges, one per worker, so the load is even whatever the lengths are:
// a batch of short and long sequences, the triangle of a causal prompt, or one long context with a
// few rows.  An item cut by a range boundary leaves one partial result per piece, and the pieces
// are joined afterwards in the order of their keys. There are three kinds of items, each with
// workers of its own: wide items (two query tiles that share each key tile; a worker is a CTA),
// narrow ones (a sequence's last item if it has at most `qn` tokens: one query tile; a worker is
// one of a CTA's two chains) and few-row ones (the last item if it has at most `qf` tokens: single
// tokens and short tails; a worker is one of eight warps of a CTA). Lengths live on the device, so
// each CTA derives the ranges of its workers itself: its threads share the sequences out, and a
// warp per worker finds its sequence in a scan over their costs, then the item within it.  All
// costs are 32-bit: a call whose sizes could pass 2^30 is refused on the host.  (In a call for a
// single token this stands in the way of everything else, most of it the fetching of instructions,
// so it is kept short: 64-bit costs and a search by one thread took 11 us.)
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
  int qf;                   // of at most qf <= qn few-row (0: none is; qf == qt: every item is)
  // by kind of item:
  int kt_shift[3];          // keys per tile: 2^kt_shift
  int start_cost[3];        // cost of starting and storing an item, in key tiles
  int least[3];             // least cost worth a worker of its own (0 and 1: any; calls use no more)
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
// Error of a whole call: offsets that descend.  What the costs add up to is only bounded, and a row
// only in one sequence, where they ascend, so nothing is attended then.
constexpr int PAGED_DESCENDS = 3;

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

// Error of the call that segment `index`, found malformed, stands for.
DG_HD int paged_error(const PagedShape &p, int index, int error) {
  const int i = p.shared_len > 0 ? index - 1 : index;   // (the prefix has no error)
  return p.seq_off[i + 1] < p.seq_off[i] ? PAGED_DESCENDS : error;
}

// sum_{i < n} floor((a i + b) / m) for a, b >= 0, m > 0 (each term and the sum below 2^31).
DG_HD int floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint32_t r = 0;
  while (n > 0) {
    if (a >= m) {
      r += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      r += n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return (int)r;
}

enum { PAGED_WIDE = 0, PAGED_NARROW = 1, PAGED_FEW = 2 };

// Full items of a segment (a division is skipped where there are none: single tokens).
DG_HD int paged_full_items(const PagedShape &p, const PagedSeg &s) { return s.n < p.qt ? 0 : s.n / p.qt; }
DG_HD bool paged_all_few(const PagedShape &p) { return p.qf == p.qt; }
// The kind of a segment's last item where it is not wide, else PAGED_WIDE (not asked where every item
// is few-row).
DG_HD int paged_tail_kind(const PagedShape &p, const PagedSeg &s) {
  const int tail = s.n - paged_full_items(p, s) * p.qt;
  return tail == 0 || tail > p.qn ? PAGED_WIDE : tail > p.qf ? PAGED_NARROW : PAGED_FEW;
}
// Items of a kind in one kv head of segment s, and the index of the first.
DG_HD int paged_items(const PagedShape &p, const PagedSeg &s, int kind) {
  if (paged_all_few(p)) return kind != PAGED_FEW ? 0 : s.n <= p.qt ? 1 : (s.n + p.qt - 1) / p.qt;
  const int tail = paged_tail_kind(p, s);
  if (kind != PAGED_WIDE) return tail == kind ? 1 : 0;
  const int full = paged_full_items(p, s);
  return full + (tail == PAGED_WIDE && full * p.qt < s.n ? 1 : 0);
}
DG_HD int paged_first_item(const PagedShape &p, const PagedSeg &s, int kind) {
  return kind == PAGED_WIDE || paged_all_few(p) ? 0 : paged_full_items(p, s);
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
DG_HD int paged_tiles(const PagedShape &p, int kind, int keys) {
  return (keys + (1 << p.kt_shift[kind]) - 1) >> p.kt_shift[kind];
}
DG_HD int paged_item_tiles(const PagedShape &p, const PagedSeg &s, int kind, int i) {
  return paged_tiles(p, kind, paged_item_keys(p, s, i));
}
// Cost of the first q items of a kind (of one kv head).
DG_HD int paged_cost_before(const PagedShape &p, const PagedSeg &s, int kind, int q) {
  if (q <= 0) return 0;
  // a kind other than wide has one item, which sees all of the segment's keys; so has a last one
  if (!s.causal || (q == 1 && s.n <= p.qt) || (kind != PAGED_WIDE && !paged_all_few(p)))
    return q * (paged_tiles(p, kind, s.keys) + p.start_cost[kind]);
  const int last = q * p.qt > s.n ? 1 : 0;   // an item with fewer tokens: by itself
  const int kt = 1 << p.kt_shift[kind];
  const int full = floor_sum(q - last, kt, p.qt, s.keys - s.n + p.qt + kt - 1);
  return full + (last ? paged_tiles(p, kind, s.keys) : 0) + q * p.start_cost[kind];
}
DG_HD int paged_head_cost(const PagedShape &p, const PagedSeg &s, int kind) {
  return s.n > 0 ? paged_cost_before(p, s, kind, paged_items(p, s, kind)) : 0;
}
// At least the total cost of any kind in a call of these sizes.
inline long long paged_cost_bound(const PagedShape &p) {
  long long most = 0;
  for (int kind = 0; kind < 3; ++kind) {
    const long long tiles = (p.cap >> p.kt_shift[kind]) + 1 + p.start_cost[kind];
    const long long tails = (p.n_seqs < p.n_tokens ? p.n_seqs : p.n_tokens) + 1;
    const bool many = kind == PAGED_WIDE || (kind == PAGED_FEW && paged_all_few(p));
    const long long items = many ? 2 * (long long)(p.n_tokens / p.qt) + tails : tails;
    const long long c = p.Hkv * items * tiles;
    most = c > most ? c : most;
  }
  return most;
}
constexpr long long PAGED_COST_LIMIT = 1LL << 30;

// A worker's place in the work of a kind: its range [u0, u1) of the total cost (u0 >= u1: none) and
// the item that it begins in.
struct PagedStart {
  int worker;               // its number among those of the kind
  int u0, u1;
  int item_u0;              // where the item that holds u0 begins
  int per;                  // cost per worker
  int seg, head, item;      // item: among those of the kind
  PagedSeg s;
};

// What a worker leaves about the item that its range goes on with, for joining the pieces.
struct PagedHead {
  int first, last;          // workers (of the kind) that hold its first and last tile; first < 0: the
                            // range does not begin inside an item
  int tok0, tokens, head;   // packed rows and kv head of the item
  int refused;              // nothing is attended (the same in every worker's)
  int pad[2];
};
DG_HD PagedHead paged_head(const PagedShape &p, int kind, const PagedStart &st) {
  PagedHead h = {-1, 0, 0, 0, 0, 0, {0, 0}};
  const int c = p.start_cost[kind];
  if (st.u0 < st.u1 && st.u0 - st.item_u0 > c) {
    const int item = paged_first_item(p, st.s, kind) + st.item;
    const int begin = st.item_u0 + c, end = begin + paged_item_tiles(p, st.s, kind, item);
    h.first = begin / st.per;
    h.last = (end - 1) / st.per;
    h.tok0 = st.s.tok0 + item * p.qt;
    h.tokens = paged_item_tokens(p, st.s, item);
    h.head = st.head;
  }
  return h;
}

// Shares the CTAs out among the kinds that have any cost: kind k gets CTAs [first[k], first[k] +
// count[k]).  Where each CTA took its part of every kind one after the other it paid for a start per
// kind (first loads, code not yet fetched), and the bytes of single tokens did not overlap the matrix
// products of wide items: 128 single tokens over a shared prefix of 8192 keys took 61 us, 49 as they are
// shared out now (41 since the joins got shorter).
// weight: cycles of a CTA per unit of cost on calls of one kind (wide: a key tile of both chains;
// narrow: half of a tile of each chain; few-row: an eighth of 32 keys of each of eight warps, between
// 300, right for many keys per token, and 500, right for a long prefix).
DG_HD void paged_share(const int (&total)[3], int ctas, int (&first)[3], int (&count)[3]) {
  constexpr float weight[3] = {3500.f, 1500.f, 400.f};
  float t[3], sum = 0.f;
  int big = 0;
  for (int k = 0; k < 3; ++k) {
    t[k] = (float)total[k] * weight[k];
    sum += t[k];
    if (t[k] > t[big]) big = k;
  }
  int rest = ctas;
  for (int k = 0; k < 3; ++k) {
    const int c = (int)((float)ctas * (t[k] / (sum > 0.f ? sum : 1.f)));
    count[k] = k == big || total[k] == 0 ? 0 : c > 0 ? c : 1;
    rest -= count[k];
  }
  count[big] = rest;
  first[0] = 0;
  first[1] = count[0];
  first[2] = count[0] + count[1];
}

#ifdef __CUDACC__
// Workers of a kind in one CTA, and their places in the CTA's list of starts.
constexpr int PAGED_STARTS = 11;
__device__ __forceinline__ int paged_cta_workers(int kind) {
  return kind == PAGED_WIDE ? 1 : kind == PAGED_NARROW ? 2 : 8;
}
__device__ __forceinline__ int paged_start_index(int kind) {
  return kind == PAGED_WIDE ? 0 : kind == PAGED_NARROW ? 1 : 3;
}

struct PagedScan {
  int before[3][256];    // by kind and thread: cost of its warp's threads before it
  int sum[3][8];         // by kind and warp
  int error;
};

// Finds the ranges of this CTA's workers of the first KINDS kinds, with GROUP threads for each
// (thread t works for kind t / GROUP; further threads take no part); warp j leaves the j-th
// worker's in start[j] and its head in heads[].  The block synchronises inside, and has to before
// start is read.  Returns the largest error code of any sequence.
template <int GROUP, int KINDS>
__device__ __forceinline__ int paged_locate(const PagedShape &p, int cta, int ctas, int starts,
                                            PagedStart *start, PagedHead *heads, PagedScan &scan) {
  constexpr unsigned full = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31;
  const int segs = paged_segs(p), chunk = (segs + GROUP - 1) / GROUP;
  if (tid == 0) scan.error = 0;
  __syncthreads();
  if (tid < KINDS * GROUP) {
    const int kind = tid / GROUP, t = tid % GROUP;
    uint32_t mine = 0;   // cost of this thread's sequences (past 32 bits only where offsets descend)
    for (int i = t * chunk; i < min((t + 1) * chunk, segs); ++i) {
      const PagedSeg s = paged_seg(p, i);
      if (s.error) atomicMax(&scan.error, paged_error(p, i, s.error));
      mine += (uint32_t)p.Hkv * (uint32_t)paged_head_cost(p, s, kind);
    }
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(full, inc, o);
      if (lane >= o) inc += v;
    }
    scan.before[kind][t] = (int)(inc - mine);
    if (lane == 31) scan.sum[kind][t >> 5] = (int)inc;
  }
  __syncthreads();
  const int j = tid >> 5;   // this warp's worker
  if (j < starts) {
    const int kind = j == 0 ? PAGED_WIDE : j < 3 ? PAGED_NARROW : PAGED_FEW;
    const bool refused = scan.error == PAGED_DESCENDS;
    int totals[3] = {0, 0, 0}, first[3], count[3];
#pragma unroll
    for (int k = 0; k < KINDS; ++k)
      for (int w = 0; w < GROUP / 32; ++w) totals[k] += refused ? 0 : scan.sum[k][w];
    paged_share(totals, ctas, first, count);
    const int n = paged_cta_workers(kind), i = j - paged_start_index(kind);
    const int mine_of = kind == 0 ? count[0] : kind == 1 ? count[1] : count[2];
    const int begin = kind == 0 ? first[0] : kind == 1 ? first[1] : first[2];
    const int total = kind == 0 ? totals[0] : kind == 1 ? totals[1] : totals[2];
    const bool serves = cta >= begin && cta < begin + mine_of;
    // workers are dealt out over the CTAs, so that a small call uses many of them; the numbers of
    // CTAs that serve another kind come last
    const int worker = serves ? i * mine_of + cta - begin
                              : n * mine_of + i * (ctas - mine_of) + (cta < begin ? cta : cta - mine_of);
    PagedStart r{};
    r.worker = worker;
    const uint32_t workers = n * (mine_of > 0 ? mine_of : 1);
    r.per = (int)((uint32_t)(total + workers - 1) / workers);
    if (r.per < p.least[kind]) r.per = p.least[kind];
    if (serves && total > 0 && (uint32_t)worker * (uint32_t)r.per < (uint32_t)total) {
      r.u0 = worker * r.per;
      r.u1 = r.u0 + r.per < total ? r.u0 + r.per : total;
      // the thread whose sequences hold u0: the last that begins at or before it
      int w = 0, at = 0;
      while (r.u0 >= at + scan.sum[kind][w]) at += scan.sum[kind][w++];
      const int mine = at + scan.before[kind][w * 32 + lane];
      const int l = 31 - __clz(__ballot_sync(full, mine <= r.u0));
      r.item_u0 = __shfl_sync(full, mine, l);
      int each;
      for (r.seg = (w * 32 + l) * chunk;; ++r.seg) {
        r.s = paged_seg(p, r.seg);
        each = paged_head_cost(p, r.s, kind);
        if (r.u0 < r.item_u0 + p.Hkv * each) break;
        r.item_u0 += p.Hkv * each;
      }
      r.head = (r.u0 - r.item_u0) / each;
      r.item_u0 += r.head * each;
      // the last item that begins at or before u0: 32-way search
      if (kind == PAGED_WIDE || (paged_all_few(p) && r.s.n > p.qt)) {
        int a = 0, b = paged_items(p, r.s, kind);
#pragma unroll 1
        while (b - a > 1) {
          const int step = (b - a + 31) / 32, i = a + lane * step;
          const bool le = i < b && r.item_u0 + paged_cost_before(p, r.s, kind, i) <= r.u0;
          const int k = 31 - __clz(__ballot_sync(full, le));  // lane 0 always holds
          a += k * step;
          b = b < a + step ? b : a + step;
        }
        r.item = a;
        r.item_u0 += paged_cost_before(p, r.s, kind, a);
      }
    }
    if (lane == 0) {
      start[j] = r;
      PagedHead h = paged_head(p, kind, r);
      h.refused = refused;
      heads[(kind == PAGED_WIDE ? 0 : kind == PAGED_NARROW ? ctas : 3 * ctas) + worker] = h;
    }
  }
  return scan.error;
}
#endif

// Walks the pieces of a worker's range in order: after begin(), while (more()), key tiles [t0, t1)
// of item `item` (tokens [tok, tok + toks) of segment s, kv head `head`).  The starting cost of an
// item lies before its first tile, and a range that ends within it leaves the item to the next
// worker.
struct PagedWalk {
  PagedSeg s;
  int seg, head, index, items;        // index: among the items of the kind
  int item, tok, toks, keys, tiles;   // the current item; keys it visits
  int t0, t1;
  int kind;
  int u1, item_u0, u;

  DG_HD void begin(const PagedShape &p, int kind_, const PagedStart &st) {
    kind = kind_;
    seg = st.seg;
    head = st.head;
    index = st.item;
    u = st.u0;
    u1 = st.u1;
    item_u0 = st.item_u0;
    if (u >= u1) return;
    s = st.s;
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
    tiles = paged_tiles(p, kind, keys);
    const int c = p.start_cost[kind];
    const int a = u - item_u0 - c, b = u1 - item_u0 - c;
    t0 = a > 0 ? a : 0;
    t1 = b < tiles ? (b > 0 ? b : 0) : tiles;
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

// The walk of few-row items alone: a segment mostly has one at most, the same for every kv head, so
// that going on costs a few operations and, at the end of a sequence's heads, the lengths of the next.
struct PagedFewWalk {
  int seq, head, seg, which;          // which: 0 the shared prefix, 1 the sequence's own keys
  int index, items;                   // the current of the segment's items
  int tok, toks;                      // packed rows [tok, tok + toks)
  int key0, keys, tiles;              // keys [key0, key0 + keys)
  int before;                         // keys that the first of the rows sees besides itself; < 0: all
  int seg_end;                        // key behind the segment's last
  int t0, t1, left;                   // tiles of this piece; cost left in the range from its item on

  DG_HD bool more() const { return t0 < t1; }
  DG_HD bool whole() const { return t0 == 0 && t1 == tiles; }
  DG_HD void take(const PagedShape &p, const PagedSeg &s) {
    const int item = paged_first_item(p, s, PAGED_FEW) + index, first = item * p.qt;
    items = paged_items(p, s, PAGED_FEW);
    seq = s.seq;
    tok = s.tok0 + first;
    toks = paged_item_tokens(p, s, item);
    key0 = s.key0;
    keys = paged_item_keys(p, s, item);
    tiles = paged_tiles(p, PAGED_FEW, keys);
    before = s.causal ? keys - toks : -1;
    seg_end = s.key0 + s.keys;
    which = p.shared_len > 0 && seg == 0 ? 0 : 1;
  }
  DG_HD void range(const PagedShape &p, int done) {   // `done`: cost of the item before the range
    const int c = p.start_cost[PAGED_FEW], a = done - c, b = done + left - c;
    t0 = a > 0 ? a : 0;
    t1 = b < tiles ? b : tiles;
  }
  DG_HD void next(const PagedShape &p) {
    t0 = t1 = 0;
    if (left <= 0) return;
    const bool many = items > 1;
    if (++index == items) {
      index = 0;
      ++head;
    }
    if (head == p.Hkv) {
      head = 0;
      PagedSeg s;
      do {  // cost remains, so a later segment has an item
        s = paged_seg(p, ++seg);
      } while (s.n == 0 || paged_items(p, s, PAGED_FEW) == 0);
      take(p, s);
    } else if (many) {
      take(p, paged_seg(p, seg));
    }
    range(p, 0);
    left -= tiles + p.start_cost[PAGED_FEW];
  }
  DG_HD void begin(const PagedShape &p, const PagedStart &st) {
    t0 = t1 = 0;
    left = st.u1 - st.u0;
    if (left <= 0) return;
    seg = st.seg;
    head = st.head;
    index = st.item;
    take(p, st.s);
    range(p, st.u0 - st.item_u0);
    left -= tiles + p.start_cost[PAGED_FEW] - (st.u0 - st.item_u0);
    if (t0 >= t1) next(p);   // (a range that ends within the first item's starting cost ends here)
  }
};

// The pages whose places a warp holds while it copies keys of a few-row walk: PAGED_WINDOW pages of one
// segment from `first` on, as far as the segment has them.  It stays while the walk is in the segment and
// within these pages, from one item to the next too, so it is filled up to the segment's last page: a
// causal segment's next item sees keys that the one which moved the window here did not.
constexpr int PAGED_WINDOW = 32;
struct PagedWindow {
  int seg = -1, first = 0;

  // Moves to page `page` unless pages page .. page2 are in the window; true if it moved.
  DG_HD bool move(const PagedFewWalk &w, int page, int page2) {
    if (w.seg == seg && page >= first && page2 < first + PAGED_WINDOW) return false;
    seg = w.seg;
    first = page;
    return true;
  }
  // Whether the i-th place holds a page of the segment.
  DG_HD bool filled(const PagedFewWalk &w, int i, int page_shift) const {
    return first + i <= (w.seg_end - 1) >> page_shift;
  }
};

}  // namespace dg
