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
static PagedStart locate(const PagedShape &p, int cta, int ctas) {
  long long total = 0;
  for (int i = 0; i < paged_segs(p); ++i) total += paged_seg_units(p, paged_seg(p, i));
  PagedStart r{};
  r.per = (total + ctas - 1) / ctas;
  r.u0 = cta * r.per;
  r.u1 = r.u0 + r.per < total ? r.u0 + r.per : total;
  if (r.u0 >= r.u1) { r.u0 = r.u1 = 0; return r; }
  long long at = 0;
  for (int i = 0; i < paged_segs(p); ++i) {
    const PagedSeg s = paged_seg(p, i);
    for (int h = 0; s.n > 0 && h < p.Hkv; ++h)
      for (int q = 0; q < paged_items(p, s); ++q) {
        const int n = paged_item_units(p, s, q);
        if (r.u0 >= at && r.u0 < at + n) { r.seg = i; r.head = h; r.item = q; r.item_u0 = at; return r; }
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
    p.kt = wide ? 128 : 64;
    p.qt = (wide ? 128 : 64) / rep * (wide ? 2 : 1);
    p.qn = wide ? 128 / rep : 0;
    p.causal = rnd(2);
    p.shared_len = rnd(3) ? 0 : page * (1 + rnd(20));
    p.cap = p.shared_len + 100000;
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
    std::vector<Unit> all;
    for (int i = 0; i < paged_segs(p); ++i) {
      const PagedSeg s = paged_seg(p, i);
      CHECK(s.error == 0);
      if (s.n == 0) { CHECK(paged_seg_units(p, s) == 0); continue; }
      long long before = 0;
      for (int q = 0; q < paged_items(p, s); ++q) {
        CHECK(paged_units_before(p, s, q) == before);
        CHECK(paged_item_units(p, s, q) > 0);
        const int span = paged_item_tokens(p, s, q) <= p.qn ? 2 * p.kt : p.kt;
        CHECK(paged_item_units(p, s, q) * (long long)span >= paged_item_keys(p, s, q));
        CHECK((paged_item_units(p, s, q) - 1) * (long long)span < paged_item_keys(p, s, q));
        before += paged_item_units(p, s, q);
      }
      CHECK(paged_units_before(p, s, paged_items(p, s)) == before);
      for (int h = 0; h < p.Hkv; ++h)
        for (int q = 0; q < paged_items(p, s); ++q)
          for (int k = 0; k < paged_item_units(p, s, q); ++k) all.push_back({i, h, q, k});
    }
    const int ctas = rnd(2) ? 148 : 1 + rnd(300);
    size_t at = 0;
    for (int c = 0; c < ctas; ++c) {
      const PagedStart st = locate(p, c, ctas);
      PagedWalk w;
      int pieces = 0, cont = 0;
      for (w.begin(p, st); w.more(); w.next(p)) {
        CHECK(w.k0() < w.k1() && w.k1() <= w.units());
        cont += w.k0() > 0;
        CHECK(w.k0() == 0 || pieces == 0);                       // only the first piece goes on
        CHECK(w.k1() == w.units() || w.u + (w.k1() - w.k0()) == st.u1);   // only the last is cut
        for (int k = w.k0(); k < w.k1(); ++k, ++at) {
          CHECK(at < all.size());
          CHECK(all[at].seg == w.seg && all[at].head == w.head && all[at].item == w.item && all[at].k == k);
        }
        ++pieces;
      }
    }
    CHECK(at == all.size());
  }
  // error codes
  int off[] = {0, 4, 2, 9, 12, 12}, kv[] = {5, 5, -1, 97, 1000000};
  PagedShape p{};
  p.seq_off = off; p.kv_len = kv; p.n_seqs = 5; p.n_tokens = 12; p.Hkv = 1; p.qt = 64; p.kt = 64; p.cap = 99;
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
