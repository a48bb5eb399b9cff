// Host-side check of the windowed walk (tva_common.cuh), built with a plain C++ compiler
// like schedule_host.cpp.  For each (prefix, tree, window, sinks), against the definition
// (node at position t sees key s when t - s < window or s < sinks) key by key:
//   - the tiles' valid keys are distinct, lie in the prefix, and are exactly the keys that
//     some node can see (a root, at position P);
//   - a row's mask (window_bits, over every tile) is exactly the keys it sees, and a tile
//     that window_cuts leaves unmasked is seen whole by every row;
//   - window_ancestors finds each node's depth and visible ancestors;
//   - units and row groups found by bisection (stage_sums) are those found by walking;
//   - the walk is no longer than walk_prefix_bound says, and every worker range covers
//     the tiles once (total_units).
// Prints "ok <problems>" or the first violation, and exits non-zero on a violation.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include <cuda_runtime.h>

static uint3 threadIdx = {0, 0, 0};
static dim3 blockDim(1, 1, 1);
template <typename T>
static inline T __ldg(const T* p) { return *p; }
static inline void __syncthreads() {}
static inline int atomicCAS(int* a, int cmp, int v) {
  const int old = *a;
  if (old == cmp) *a = v;
  return old;
}
static inline float __uint_as_float(unsigned u) {
  float f;
  std::memcpy(&f, &u, sizeof f);
  return f;
}

#include "tva_internal.h"

namespace {

int g_problems = 0;

bool fail(const char* what, long long a, long long b) {
  std::printf("FAIL problem %d: %s (%lld, %lld)\n", g_problems, what, a, b);
  return false;
}

bool check(int P, const std::vector<int>& parent, int window, int sinks) {
  ++g_problems;
  const int m = (int)parent.size();
  const int32_t cu_p[3] = {0, 5, 5 + P}, cu_n[3] = {0, 2, 2 + m};  // the second of two sequences
  tva::WinProblem pr{};
  pr.cu_prefix = cu_p;
  pr.cu_nodes = cu_n;
  pr.B = 2;
  pr.Hkv = 1; pr.G = 4; pr.Hq = 4; pr.d = 64; pr.RG = 128; pr.U = 7;
  pr.max_prefix = P > 5 ? P : 5;
  pr.max_nodes = m > 2 ? m : 2;
  pr.kv_capacity = 5 + P;
  pr.node_capacity = 2 + m;
  pr.window = window;
  pr.sinks = sinks;
  const tva::SeqInfo s = tva::seq_info(pr, 1);
  if (!s.ok || s.len != P || s.m != m) return fail("seq_info", s.len, s.m);
  if (s.P > tva::walk_prefix_bound(pr)) return fail("walk longer than its bound", s.P, tva::walk_prefix_bound(pr));
  auto sees = [&](long long t, long long key) { return t - key < window || key < sinks; };
  const int tiles = tva::seq_tiles(s.P);
  std::vector<int> seen(P, 0);
  for (int tile = 1; tile < tiles; ++tile) {
    const int key0 = tva::tile_key0(s, tile), keys = tva::tile_keys(pr, s, tile);
    if (keys < 1 || keys > 128 || key0 < 0 || key0 + keys > P) return fail("tile outside the prefix", key0, keys);
    for (int c = 0; c < keys; ++c) ++seen[key0 + c];
  }
  for (int key = 0; key < P; ++key)
    if (seen[key] != (sees(P, key) ? 1 : 0)) return fail("key covered", key, seen[key]);
  for (int i = 0; i < m; ++i) {
    uint32_t bits[4];
    int depth = -1, want = 0;
    if (!tva::window_ancestors(parent.data(), i, window, sinks, s.len, bits, depth)) return fail("bad tree", i, 0);
    for (int j = parent[i]; j >= 0; j = parent[j]) ++want;
    if (depth != want) return fail("depth", i, depth);
    std::vector<int> anc(m, 0);
    long long dist = 0;
    for (int j = i; j >= 0; j = parent[j], ++dist) anc[j] = sees((long long)P + depth, (long long)P + depth - dist);
    for (int j = 0; j < 128; ++j)
      if ((int)((bits[j >> 5] >> (j & 31)) & 1u) != (j < m ? anc[j] : 0)) return fail("ancestor bit", i, j);
    const int low = tva::window_low(pr, s, depth);
    for (int tile = 1; tile < tiles; ++tile) {
      const int key0 = tva::tile_key0(s, tile), keys = tva::tile_keys(pr, s, tile);
      const bool cut = keys < 128 || tva::window_cuts(pr, s, key0, keys);
      for (int ck = 0; ck < 4; ++ck) {
        const uint32_t w = tva::window_bits(key0 + 32 * ck, keys - 32 * ck, low, pr.sinks);
        for (int c = 0; c < 32; ++c) {
          const bool real = 32 * ck + c < keys, vis = real && sees((long long)P + depth, key0 + 32 * ck + c);
          if ((int)((w >> c) & 1u) != (vis ? 1 : 0)) return fail("mask bit", i, key0 + 32 * ck + c);
          if (!cut && !vis) return fail("unmasked tile hides a key", i, key0 + 32 * ck + c);
        }
      }
    }
  }
  // the schedule over both sequences covers every unit once
  long long covered = 0;
  for (int u = 0; u < pr.U; ++u) {
    long long t0 = 0, t1 = 0;
    tva::worker_range(pr, u, t0, t1, false);
    tva::Segment S;
    long long t = t0;
    while (tva::next_segment(pr, u, t, t1, S, false)) covered += S.n;
  }
  if (covered != tva::total_units(pr)) return fail("units covered", covered, tva::total_units(pr));
  // the same walk with the staged running sums
  int buf[16];
  tva::WinProblem sums = pr;
  tva::stage_sums(sums, buf, 16);
  if (sums.unit_start == nullptr) return fail("no sums", 0, 0);
  if (tva::total_units(sums) != tva::total_units(pr)) return fail("total", tva::total_units(sums), 0);
  for (long long t = 0; t < tva::total_units(pr); ++t) {
    const tva::Loc a = tva::locate_unit(pr, t), b = tva::locate_unit(sums, t);
    if (a.b != b.b || a.g != b.g || a.mp != b.mp || a.tile != b.tile || a.q != b.q || a.start != b.start)
      return fail("unit found by bisection", t, b.b);
  }
  for (long long q = 0;; ++q) {
    const tva::GroupLoc a = tva::locate_group(pr, q), b = tva::locate_group(sums, q);
    if (a.found != b.found || a.T != b.T) return fail("row group found by bisection", q, b.found);
    if (!a.found) break;
    if (a.b != b.b || a.g != b.g || a.mp != b.mp || a.start != b.start || a.tiles != b.tiles)
      return fail("row group by bisection", q, b.b);
  }
  return true;
}

}  // namespace

int main() {
  bool ok = true;
  std::srand(11);
  const int big = 2147483647;
  for (int P : {0, 1, 5, 126, 127, 128, 129, 255, 256, 300, 385, 700})
    for (int window : {1, 2, 7, 127, 128, 129, 256, 300, 701, big})
      for (int sinks : {0, 1, 4, 127, 128, 129, 300, big})
        for (int kind = 0; kind < 3 && ok; ++kind) {
          const int m = kind == 0 ? 1 : 1 + std::rand() % 24;
          std::vector<int> parent(m);
          for (int i = 0; i < m; ++i) parent[i] = kind == 1 ? i - 1 : (i ? std::rand() % (i + 1) - 1 : -1);
          ok = check(P, parent, window, sinks);
        }
  std::vector<int> chain(128);
  for (int i = 0; i < 128; ++i) chain[i] = i - 1;
  for (int P : {0, 3, 200, 513})
    for (int window : {1, 5, 100, 128, 130, 400})
      for (int sinks : {0, 4, 203}) ok = ok && check(P, chain, window, sinks);
  if (ok) std::printf("ok %d\n", g_problems);
  return ok ? 0 : 1;
}
