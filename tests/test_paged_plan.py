"""Work split of the paged attention (csrc/paged_plan.cuh), compiled for the host: unit counts against
direct sums, and the walk of every CTA's range against a plain enumeration of all units, for ragged,
empty, causal and shared-prefix batches; malformed lengths get their error codes."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r'''
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "paged_plan.cuh"
using namespace dg;
static unsigned long long x = 88172645463325252ull;
static int rnd(int n) { x ^= x << 13; x ^= x >> 7; x ^= x << 17; return (int)(x % (unsigned)n); }
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

struct Unit { int seg, head, item, k; };

// The range start as paged_locate finds it, by plain counting.
static PagedStart locate(const PagedShape &p, int kind, int worker, int workers) {
  int total = 0;
  for (int i = 0; i < paged_segs(p); ++i) total += p.Hkv * paged_head_cost(p, paged_seg(p, i), kind);
  PagedStart r{};
  r.per = (total + workers - 1) / workers;
  if (r.per < p.least[kind]) r.per = p.least[kind];
  r.u0 = worker * r.per;
  r.u1 = r.u0 + r.per < total ? r.u0 + r.per : total;
  if (r.u0 >= r.u1) { r.u0 = r.u1 = 0; return r; }
  int at = 0;
  for (int i = 0; i < paged_segs(p); ++i) {
    const PagedSeg s = paged_seg(p, i);
    for (int h = 0; s.n > 0 && h < p.Hkv; ++h)
      for (int q = 0; q < paged_items(p, s, kind); ++q) {
        const int n = p.start_cost[kind] + paged_item_tiles(p, s, kind, paged_first_item(p, s, kind) + q);
        if (r.u0 >= at && r.u0 < at + n) { r.seg = i; r.head = h; r.item = q; r.item_u0 = at; r.s = s; return r; }
        at += n;
      }
  }
  return r;
}

int main() {
  for (int t = 0; t < 3000; ++t) {
    const long long n = rnd(60), m = 1 + rnd(200), a = rnd(400), b = rnd(1000);
    long long want = 0;
    for (int i = 0; i < n; ++i) want += (a * i + b) / m;
    CHECK(floor_sum(n, m, a, b) == want);
  }
  for (int t = 0; t < 400; ++t) {
    const int rep = 1 + rnd(9), seqs = 1 + rnd(70), page = 16 << rnd(4);
    const bool wide = rnd(2);
    PagedShape p{};
    p.Hkv = 1 + rnd(4);
    p.kt_shift[0] = p.kt_shift[1] = wide ? 7 : 6;
    p.kt_shift[2] = 5;
    for (int k = 0; k < 3; ++k) p.least[k] = rnd(2) ? rnd(9) : 0;
    p.qt = (wide ? 128 : 64) / rep * (wide ? 2 : 1);
    p.qn = wide ? 128 / rep : 0;
    p.qf = wide && rnd(2) ? 16 / rep : 0;
    const bool few = p.qf > 0 && rnd(2);   // every item few-row
    if (few) p.qt = p.qn = p.qf;
    CHECK(paged_all_few(p) == few);
    p.causal = rnd(2);
    p.shared_len = rnd(3) ? 0 : page * (1 + rnd(20));
    p.cap = p.shared_len + 100000;
    p.start_cost[0] = rnd(4);
    p.start_cost[1] = rnd(4);
    p.start_cost[2] = rnd(4);
    std::vector<int> off(1, 0), kv;
    for (int s = 0; s < seqs; ++s) {
      off.push_back(off.back() + (rnd(4) ? (rnd(2) ? 1 : rnd(700)) : 0));
      kv.push_back(p.shared_len + (rnd(3) ? rnd(3000) : 0));
    }
    p.seq_off = off.data();
    p.kv_len = kv.data();
    p.n_seqs = seqs;
    p.n_tokens = off.back() + rnd(5);
    if (p.n_tokens == 0) p.n_tokens = 1;
    for (int kind = 0; kind < 3; ++kind) {
      std::vector<Unit> all;
      for (int i = 0; i < paged_segs(p); ++i) {
        const PagedSeg s = paged_seg(p, i);
        CHECK(s.error == 0);
        if (s.n == 0) { CHECK(paged_head_cost(p, s, kind) == 0); continue; }
        const int first = paged_first_item(p, s, kind), n = paged_items(p, s, kind);
        if (few) {         // every token in one few-row item
          CHECK(kind == 2 || n == 0);
          int rows = 0;
          for (int q = 0; q < n; ++q) {
            CHECK(paged_item_tokens(p, s, q) > 0 && paged_item_tokens(p, s, q) <= p.qf);
            rows += paged_item_tokens(p, s, q);
          }
          CHECK(first == 0 && rows == (kind == 2 ? s.n : 0));
        } else if (kind == 0) {   // every token in one item of one kind
          int rows = 0;
          for (int q = 0; q < n; ++q) rows += paged_item_tokens(p, s, q);
          const int tail = paged_tail_kind(p, s);
          for (int k = 1; k < 3; ++k) {
            CHECK(paged_items(p, s, k) == (tail == k ? 1 : 0));
            if (tail == k) CHECK(paged_first_item(p, s, k) == n);
          }
          if (tail) {
            const int last = paged_item_tokens(p, s, n);
            CHECK(last > 0 && last <= p.qn && (tail == 2) == (last <= p.qf));
            rows += last;
          } else {
            CHECK(paged_item_tokens(p, s, n - 1) > p.qn);
          }
          CHECK(rows == s.n);
        }
        long long before = 0;
        for (int q = 0; q < n; ++q) {
          CHECK(paged_cost_before(p, s, kind, q) == before);
          const int t = paged_item_tiles(p, s, kind, first + q);
          CHECK(t > 0 && t * (1LL << p.kt_shift[kind]) >= paged_item_keys(p, s, first + q));
          CHECK((t - 1) * (1LL << p.kt_shift[kind]) < paged_item_keys(p, s, first + q));
          before += t + p.start_cost[kind];
        }
        CHECK(paged_cost_before(p, s, kind, n) == before && paged_head_cost(p, s, kind) == before);
        for (int h = 0; h < p.Hkv; ++h)
          for (int q = 0; q < n; ++q)
            for (int k = 0; k < paged_item_tiles(p, s, kind, first + q); ++k)
              all.push_back({i, h, first + q, k});
      }
      long long sum = 0;
      for (int i = 0; i < paged_segs(p); ++i) sum += p.Hkv * (long long)paged_head_cost(p, paged_seg(p, i), kind);
      CHECK(sum <= paged_cost_bound(p));
      const int workers = rnd(2) ? 148 : 1 + rnd(300);
      size_t at = 0;
      std::vector<int> begun(workers, -1);   // the cut item that begins with a worker
      int open = -1, open_tiles = 0;         // worker where the item now being cut began
      long long open_last = -1;
      for (int c = 0; c < workers; ++c) {
        const PagedStart st = locate(p, kind, c, workers);
        const PagedHead hd = paged_head(p, kind, st);
        PagedWalk w;
        int pieces = 0, slots[2] = {0, 0};
        bool goes_on = false;
        for (w.begin(p, kind, st); w.more(); w.next(p)) {
          CHECK(w.t0 < w.t1 && w.t1 <= w.tiles);
          CHECK(w.t0 == 0 || pieces == 0);                       // only the first piece goes on
          if (!w.whole()) ++slots[w.t0 == 0];
          for (int k = w.t0; k < w.t1; ++k, ++at) {
            CHECK(at < all.size());
            CHECK(all[at].seg == w.seg && all[at].head == w.head && all[at].item == w.item && all[at].k == k);
          }
          if (w.t0 > 0) {
            goes_on = true;
            CHECK(open >= 0 && hd.first == open);
            CHECK(hd.tok0 == w.s.tok0 + w.tok && hd.tokens == w.toks && hd.head == w.head);
            if (open_last < 0) open_last = hd.last;
            CHECK(open_last == hd.last);
            if (w.t1 == w.tiles) { CHECK(hd.last == c); open = -1; }
          }
          if (w.t0 == 0 && !w.whole()) {
            CHECK(open < 0);
            open = c; open_last = -1; open_tiles = w.tiles;
          }
          ++pieces;
        }
        (void)open_tiles;
        if (kind == 2) {                       // the short walk sees the same pieces
          PagedFewWalk f;
          f.begin(p, st);
          for (w.begin(p, kind, st); w.more(); w.next(p), f.next(p)) {
            CHECK(f.more() && f.t0 == w.t0 && f.t1 == w.t1 && f.tiles == w.tiles && f.head == w.head);
            CHECK(f.seg == w.seg && f.seq == w.s.seq && f.tok == w.s.tok0 + w.tok && f.toks == w.toks);
            CHECK(f.key0 == w.s.key0 && f.keys == w.keys && f.whole() == w.whole());
            CHECK(f.before == (w.s.causal ? w.s.keys - w.s.n + w.tok : -1));
            CHECK(f.which == (p.shared_len > 0 && w.seg == 0 ? 0 : 1));
          }
          CHECK(!f.more());
        }
        CHECK((hd.first >= 0) == goes_on);
        CHECK(slots[0] <= 1 && slots[1] <= 1);
      }
      CHECK(at == all.size() && open < 0);
    }
  }
  // the CTAs' shares: every kind with work has one at least, none overlap, all are given out
  for (int t = 0; t < 20000; ++t) {
    int total[3], first[3], count[3];
    for (int k = 0; k < 3; ++k) total[k] = rnd(3) ? 0 : rnd(2) ? rnd(50) : rnd(1 << 30);
    const int ctas = 3 + rnd(300);
    paged_share(total, ctas, first, count);
    int at = 0;
    for (int k = 0; k < 3; ++k) {
      CHECK(first[k] == at && count[k] >= (total[k] > 0));
      at += count[k];
    }
    CHECK(at == ctas);
  }
  // error codes
  int off[] = {0, 4, 2, 9, 12, 12}, kv[] = {5, 5, -1, 97, 1000000};
  PagedShape p{};
  p.seq_off = off; p.kv_len = kv; p.n_seqs = 5; p.n_tokens = 12; p.Hkv = 1; p.qt = 64; p.kt_shift[0] = 6; p.cap = 99;
  CHECK(paged_seg(p, 0).error == 0 && paged_seg(p, 0).n == 4 && paged_seg(p, 0).keys == 9);
  CHECK(paged_seg(p, 1).error == 1 && paged_seg(p, 1).n == 0);       // descending offsets
  CHECK(paged_seg(p, 2).error == 1 && paged_seg(p, 2).n == 0);       // negative length
  CHECK(paged_seg(p, 3).error == 2 && paged_seg(p, 3).n == 0);       // 97 + 3 keys past 99
  CHECK(paged_seg(p, 4).error == 0 && paged_seg(p, 4).n == 0);       // empty: lengths do not matter
  p.n_tokens = 8;
  CHECK(paged_seg(p, 2).error == 1);                                 // rows past the buffer
  p.shared_len = 16;
  CHECK(paged_seg(p, 0).n == 8 && paged_seg(p, 0).keys == 16);       // the prefix: rows clamped
  CHECK(paged_seg(p, 1).error == 1);                                 // shorter than the prefix
  kv[0] = 0x7fffffff;
  CHECK(paged_seg(p, 1).error == 2);                                 // no overflow
  std::puts("ok");
  return 0;
}
'''


def test_work_split_covers_every_unit_once(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text(SRC)
    exe = tmp_path / "plan"
    csrc = os.path.join(ROOT, "block_discrete_diffusion_dg_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc, str(src), "-o",
                    str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


WINDOW = SRC.split("int main()")[0] + r'''
// Walks every worker's few-row range as the loading side of a warp does: 32 keys a step, their pages from
// a window that moves with them.  Every 16 keys that a piece has must find their page in it.
static int walk(const PagedShape &p, int page_shift, int workers) {
  for (int c = 0; c < workers; ++c) {
    PagedFewWalk w;
    PagedWindow win;
    int held[PAGED_WINDOW] = {};   // page in each place, -1: none
    for (w.begin(p, locate(p, 2, c, workers)); w.more(); w.next(p)) {
      const PagedSeg s = paged_seg(p, w.seg);
      CHECK(w.seg_end == s.key0 + s.keys);
      for (int t = w.t0; t < w.t1; ++t) {
        const int pos = w.key0 + t * 32, live = w.keys - t * 32;
        const int page[2] = {pos >> page_shift, (pos + 16) >> page_shift};
        if (win.move(w, page[0], page[1])) {
          for (int i = 0; i < PAGED_WINDOW; ++i) {
            held[i] = win.filled(w, i, page_shift) ? page[0] + i : -1;
            // nothing behind the segment's last key is looked up
            CHECK(held[i] < 0 || held[i] << page_shift < s.key0 + s.keys);
          }
        }
        for (int g = 0; g < 2; ++g) {
          const int i = page[g] - win.first;
          CHECK(i >= 0 && i < PAGED_WINDOW);
          CHECK(16 * g >= live || held[i] == page[g]);
        }
      }
    }
  }
  return 0;
}

// A call that takes every item for few-row.
static int batch(int rep, int heads, int page_shift, int causal, int shared, int workers,
                 const std::vector<int> &news, const std::vector<int> &have) {
  std::vector<int> off(1, 0), kv;
  for (size_t s = 0; s < news.size(); ++s) {
    off.push_back(off.back() + news[s]);
    kv.push_back(shared + have[s]);
  }
  PagedShape p{};
  p.Hkv = heads;
  p.kt_shift[0] = p.kt_shift[1] = 7;
  p.kt_shift[2] = 5;
  p.qt = p.qn = p.qf = 16 / rep;
  p.start_cost[2] = 1;
  p.causal = causal;
  p.shared_len = shared;
  p.cap = 1 << 20;
  p.seq_off = off.data();
  p.kv_len = kv.data();
  p.n_seqs = (int)news.size();
  p.n_tokens = off.back() > 0 ? off.back() : 1;
  return walk(p, page_shift, workers);
}

int main() {
  // single tokens over long caches, one short prompt, idle slots
  for (int page_shift = 4; page_shift <= 10; page_shift += 2)
    for (int rep = 1; rep <= 16; rep *= 2)
      for (int have : {0, 10, 50, 500}) {
        std::vector<int> news(199, 1), kv(199, 8191);
        news.push_back(40);
        kv.push_back(have);
        news.resize(256, 0);
        kv.resize(256, 0);
        CHECK(batch(rep, 2, page_shift, 1, 0, 148 * 8, news, kv) == 0);
      }
  // one prompt among empty sequences
  for (int page_shift = 4; page_shift <= 6; ++page_shift) {
    std::vector<int> news(300, 0), kv(300, 0);
    news[7] = 2048;
    CHECK(batch(4, 2, page_shift, 1, 0, 148, news, kv) == 0);
  }
  for (int t = 0; t < 600; ++t) {   // random ones, ranges of any length
    const int seqs = 1 + rnd(40), page_shift = 4 + rnd(7);
    std::vector<int> news, kv;
    for (int s = 0; s < seqs; ++s) {
      news.push_back(rnd(3) ? (rnd(3) ? 1 : rnd(400)) : 0);
      kv.push_back(rnd(3) ? rnd(3000) : 0);
    }
    const int shared = rnd(3) ? 0 : (1 << page_shift) * (1 + rnd(5));
    CHECK(batch(1 + rnd(16), 1 + rnd(3), page_shift, rnd(4) > 0, shared, rnd(2) ? 1 + rnd(12) : 148, news, kv) == 0);
  }
  std::puts("ok");
  return 0;
}
'''


def test_page_window_of_few_row_walks(tmp_path):
    """The places of pages that a few-row warp holds are those of all keys it copies, whatever items of
    a sequence its range goes on with."""
    src = tmp_path / "window.cpp"
    src.write_text(WINDOW)
    exe = tmp_path / "window"
    csrc = os.path.join(ROOT, "block_discrete_diffusion_dg_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc, str(src), "-o",
                    str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
