// k_partials_kv4_rows.cu - attention partials over a 4-bit prefix cache for row groups of at
// most 16 rows (a few tree nodes times the query heads of a KV head: the single tokens and
// short drafts of a serving batch).
//
// What is computed is what k_partials_kv4.cu computes.  There the records are widened into
// shared memory, because that is where tcgen05.mma reads its operands, and a tile passes
// through five hand-overs between warps; with few rows a tile's time is all latency (1.1 us
// a tile and SM, one row or 128).  Here a record is widened in the registers that multiply
// it: mma.sync takes both operands from registers, so 4-bit codes are all that ever reaches
// shared memory, and the warps share nothing but the arrival of tiles.  The tensor work of
// 16 rows is small enough for that path (at 128 rows it would bound the kernel).
//
// How (one CTA per SM, kWarps computing warps and a producer):
//   producer warp: TMA of the raw 128-record tiles into a ring.
//   computing warps: teams of 4 (2) take the tiles in turn, a warp 16 keys at a time.  It holds
//           all rows' Q fragments, its own running maxima, sums and O; the warps' partials
//           meet at a segment's end.
//   S^T = K Q^T, so that the rows are the product's short side (8 or 16 of them, not 16 or
//           32).  The contraction index may run in any order, as long as Q's does too: lane
//           4 g + c takes the whole code words (d / 32) c .. of keys g and g + 8, in one wide
//           load each, and a widened word is half of the A fragments of two k-steps.
//   O^T = V^T P^T: the order of O's columns is free as well.  Lane 4 g + c takes columns
//           (d / 8) g .. of keys 2c, 2c + 1, 2c + 8, 2c + 9, which share a scale; a byte
//           permutation of their codes puts two keys' values into the pairs that the
//           fragments want.  The weights are transposed between the products (movmatrix).
// The tree tile's K / V are 16-bit; their fragments are loaded from global memory.
//
// Measured (bf16, 8 KV heads, d = 128, back to back with the combine; k_partials_kv4.cu in
// brackets): 4 rows over a prefix of 16384 13.8 us (22.7), of 131072 44.6 us (76.5), 32
// sequences of 32768 321 .. 336 us (527).  12 or 16 rows: 63 us (71 .. 75) and 435 us (496 ..
// 527).  32 rows as four blocks spill: 122 us (75), so they stay with that kernel.  (Two blocks
// at d = 128 spill 148 bytes a thread.)
// What bounds it (counters): 131072 rows of one sequence, no unit alone - 58 % of the issue
// slots, DRAM at 3.4 TB/s (each record once), three warps a scheduler; of the 5.6 clocks
// between a warp's instructions 1.1 are fixed latencies, 0.9 another warp's turn, 0.8 a busy
// pipe, 0.7 loads.  The batch of 32, DRAM: 6.5 TB/s (82 % of its peak) of 2.15 GB, for 1.21 GB
// of records.  That is 256 bytes a record of 144: two lines of 128 each, none of them shared
// with the neighbouring KV heads' records, which a batch reads at another time.
//
// P is rounded to q's type for the second product, as in the other kernels; the row sums
// take the unrounded weights, in fp32.
//
// Every wait is bounded (k_partials_tc.cu); a warp that gives up still walks its segments, so
// that the block's barriers stay matched.
#include <cuda.h>

#include <algorithm>

#include "kv4.cuh"
#include "tc_pipeline.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

using namespace ptx;

// NT: 8-row blocks of Q (1 or 2).
template <int D, int NT>
struct Rows {
  // Warps, and how many of them share a tile.  A team sees every kTeams-th tile only: with all
  // 15 warps at every tile, what a tile costs each of them beside its products was a third of
  // the kernel (128k rows, one token: 52.8 us instead of 44.0).  With the producer that is 128
  // registers a thread, or 168 for two blocks (teams of four: 65 us instead of 63).
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kTeam = NT == 1 ? 4 : 2;
  static constexpr int kTeams = kWarps / kTeam;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = 8 * NT;
  static constexpr int kRec = kv4_record_bytes(D);
  static constexpr int kRawBytes = kKeyTile * kRec;
  // A multiple of kTeams: a team then meets its stages in turn, and the parity of a stage's
  // barrier tells its uses apart.  (Nine stages read a batch of 32 sequences slower, 370 us
  // instead of 330.)
  static constexpr int kStages = NT == 1 ? 6 : 8;
  static constexpr int kORow = D + 4;  // floats of a row of a warp's O in shared memory
  static constexpr int kOOff = kStages * kRawBytes;
  static constexpr int kMLOff = kOOff + 4 * kWarps * kRows * kORow;  // [2][kWarps][kRows]
  static constexpr int kParOff = kMLOff + 8 * kWarps * kRows;       // [kWarps][32] parent ids
  static constexpr int kBarOff = kParOff + 128 * kWarps;
  static constexpr int kCuCap = 1024;  // ints: batches up to 511 sequences
  static constexpr int kPrOff = kBarOff + 256;
  static constexpr int kCuOff = kPrOff + 128;
  static constexpr int kSmemBytes = kCuOff + 4 * kCuCap + 128;  // + alignment slack
  static_assert(kStages % kTeams == 0 && kWarps % kTeam == 0, "teams");
  static_assert(kRawBytes % 128 == 0 && kMLOff % 16 == 0 && kBarOff % 16 == 0, "layout");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct RowArgs {
  WinPartialArgs a;
  uint64_t wait_ns;
  int stall;  // test hook: the producer first waits on a barrier nothing completes
};

template <bool kBF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values held as an accumulator's pairs.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, bool kBF16, int NT>
__global__ void __launch_bounds__(Rows<D, NT>::kThreads, 1)
    partials_kv4_rows_kernel(const __grid_constant__ CUtensorMap tm_raw, const RowArgs args) {
  using C = Rows<D, NT>;
  constexpr int kWarps = C::kWarps;
  constexpr int KW = D / 32;  // code words of a key's K that a lane takes
  constexpr int VW = D / 64;  // code words of a key's V that a lane takes
  constexpr int NE = D / 8;   // columns of O that a lane's V words cover
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const WinPartialArgs& a = args.a;
  const int G = a.pr.G;
  WinProblem* pr_s = reinterpret_cast<WinProblem*>(smem + C::kPrOff);
  const WinProblem& pr = *pr_s;
  static_assert(sizeof(WinProblem) <= 128, "staged problem");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = blockIdx.x;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t FULL = sbase + C::kBarOff;        // [kStages]
  const uint32_t EMPTY = FULL + 8 * C::kStages;    // [kStages], the team's warps
  const uint32_t STALL = EMPTY + 8 * C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 16 * C::kStages + 8);

  if (warp == kWarps && lane == 0) {
    prefetch_tmap(&tm_raw);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(FULL + 8 * s, 1);
      mbar_init(EMPTY + 8 * s, C::kTeam);
    }
    mbar_init(STALL, 1);
    *abort_flag = 0;
    fence_mbar_init();
    __threadfence_block();
  }
  pdl_wait();
  pdl_launch_dependents();
  long long t_begin = 0, t_end = 0;
  stage_problem(a.pr, pr_s, reinterpret_cast<int*>(smem + C::kCuOff), C::kCuCap);
  worker_range(pr, u, t_begin, t_end, false);
  if (u == 0 && threadIdx.x == 0) validate_sequences(pr, a.status);
  if (t_begin >= t_end) return;  // uniform over the CTA

  if (warp == kWarps) {
    // ------------------------------------------------------------------ producer
    int raw = 0;
    bool ok = true;
    if (args.stall && !warp_wait(STALL, 0, abort_flag, args.wait_ns)) ok = false;  // test hook
    const uint64_t evict_first = policy_evict_first();  // records are read once
    long long t = t_begin;
    Segment S;
    while (ok && next_segment(pr, u, t, t_end, S, false)) {
      for (int k = S.tile0 == 0 ? 1 : 0; k < S.n; ++k) {
        const int stage = raw % C::kStages, use = raw / C::kStages;
        if (use > 0 && !warp_wait(EMPTY + 8 * stage, (use - 1) & 1, abort_flag, args.wait_ns)) { ok = false; break; }
        int z = S.L.s.p0 + tile_key0(S.L.s, S.tile0 + k);
        if (!TVA_CHECK(z >= 0 && z < S.L.s.p0 + S.L.s.len && z < pr.kv_capacity, a.status)) z = 0;
        mbar_expect_tx_elect(FULL + 8 * stage, C::kRawBytes);
        tma_load_3d_hint_elect(sbase + stage * C::kRawBytes, &tm_raw, 0, S.L.g, z, FULL + 8 * stage, evict_first);
        ++raw;
      }
    }
    // drain: every copy this warp started has landed before shared memory goes away
    for (int i = max(0, raw - C::kStages); i < raw; ++i) drain_wait(FULL + 8 * (i % C::kStages), (i / C::kStages) & 1);
  } else {
    // ------------------------------------------------------------------ computing warps
    const int g = lane >> 2, c = lane & 3;
    const float sl2 = a.scale_log2;
    const bool win = a.pr.window > 0;
    float* const xo = reinterpret_cast<float*>(smem + C::kOOff);
    float* const xm = reinterpret_cast<float*>(smem + C::kMLOff);
    float* const xl = xm + kWarps * C::kRows;
    int* const par = reinterpret_cast<int*>(smem + C::kParOff) + 32 * warp;
    constexpr int kTeams = C::kTeams;
    const int team = warp / C::kTeam;
    uint32_t base = 0;  // tiles of the earlier segments
    bool ok = true;
    long long t = t_begin;
    Segment S;
    while (next_segment(pr, u, t, t_end, S, false)) {
      const Loc& L = S.L;
      const bool tree = S.tile0 == 0;
      const int m = L.s.m;
      const int n_tree = tree ? (m + 15) / 16 : 0;  // 16-key chunks of the tree tile
      // Q: this lane holds row 8 nt + g.
      uint32_t q[NT][D / 16][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + g, nd = row / G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) +
            ((size_t)(L.s.n0 + min(nd, m - 1)) * pr.Hq + L.g * G + row % G) * D + 8 * KW * c);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint4 v = nd < m ? __ldg(src + w) : make_uint4(0u, 0u, 0u, 0u);
          q[nt][2 * w][0] = v.x;
          q[nt][2 * w][1] = v.y;
          q[nt][2 * w + 1][0] = v.z;
          q[nt][2 * w + 1][1] = v.w;
        }
      }
      // Softmax: rows 8 nt + 2c + x.  Ancestor bits where the tree tile is met, depths under a
      // window (m <= 16).
      int node[NT][2], low[NT][2];
      uint32_t anc[NT][2];
      float m_run[NT][2], l_run[NT][2];
      const bool walk = win || warp < n_tree;
      if (walk) {
        __syncwarp();
        if (lane < m) par[lane] = __ldg(a.parent + L.s.n0 + lane);
        __syncwarp();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nd = (8 * nt + 2 * c + x) / G;
          node[nt][x] = nd < m ? nd : -1;
          anc[nt][x] = 0u;
          low[nt][x] = 0;
          m_run[nt][x] = -INFINITY;
          l_run[nt][x] = 0.f;
          if (walk && nd < m) {
            uint32_t bits[4];
            int depth = 0;
            const bool good = win ? window_ancestors(par, nd, pr.window, pr.sinks, L.s.len, bits, depth)
                                  : ancestor_bits_shared(par, nd, bits);
            if (!good) set_status(a.status, kStatusBadTree);
            anc[nt][x] = bits[0];
            if (win) low[nt][x] = window_low(pr, L.s, depth);
          }
        }
      float o[NT][D / 16][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) o[nt][e][0] = o[nt][e][1] = o[nt][e][2] = o[nt][e][3] = 0.f;

      // One chunk of 16 keys: kf(j, w) gives key 8 j + g's K word (d / 32) c + w as four pairs;
      // vf(i, w, odd), of word (d / 64) g + w of V, the even or odd elements, each paired for
      // keys 8 i + 2c and 8 i + 2c + 1; seen(nt, x) the 16 keys that row 8 nt + 2c + x sees.
      auto chunk = [&](auto kf, auto vf, bool masked, auto seen) {
        float s[NT][4], s2[NT][4];  // two chains of products
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint4 k0 = kf(0, w), k1 = kf(1, w);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<kBF16>(s[nt], k0.x, k1.x, k0.y, k1.y, q[nt][2 * w][0], q[nt][2 * w][1]);
            mma16816<kBF16>(s2[nt], k0.z, k1.z, k0.w, k1.w, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
          }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
          if (masked) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t bits = seen(nt, x) >> g;
              if (!(bits & 1u)) s[nt][x] = -INFINITY;
              if (!(bits & 0x100u)) s[nt][2 + x] = -INFINITY;
            }
          }
          // The maximum may lag by 2^8, as in the other kernels (weights stay below 2^8), so
          // most chunks need only ask whether some logit is beyond that.
          float top[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) top[x] = fmaxf(s[nt][x], s[nt][2 + x]) * sl2;
          if (__any_sync(0xffffffffu, top[0] > m_run[nt][0] + 8.0f || top[1] > m_run[nt][1] + 8.0f)) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 4));
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 8));
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 16));
              const float m_new = fmaxf(m_run[nt][x], top[x]);
              const float alpha = m_run[nt][x] == -INFINITY ? 0.f : ex2(m_run[nt][x] - m_new);
              l_run[nt][x] *= alpha;
              m_run[nt][x] = m_new;
#pragma unroll
              for (int e = 0; e < D / 16; ++e) {
                o[nt][e][x] *= alpha;
                o[nt][e][2 + x] *= alpha;
              }
            }
          }
          float pw[4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float nb = m_run[nt][x] == -INFINITY ? 0.f : -m_run[nt][x];
            pw[x] = ex2(fmaf(s[nt][x], sl2, nb));
            pw[2 + x] = ex2(fmaf(s[nt][2 + x], sl2, nb));
            l_run[nt][x] += pw[x] + pw[2 + x];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            p[nt][j] = transpose8(kBF16 ? pack_bf16x2(pw[2 * j], pw[2 * j + 1]) : pack_f16x2(pw[2 * j], pw[2 * j + 1]));
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint4 v0 = vf(0, w, odd), v1 = vf(1, w, odd);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<kBF16>(o[nt][4 * w + 2 * odd], v0.x, v0.y, v1.x, v1.y, p[nt][0], p[nt][1]);
              mma16816<kBF16>(o[nt][4 * w + 2 * odd + 1], v0.z, v0.w, v1.z, v1.w, p[nt][0], p[nt][1]);
            }
          }
      };

      if (warp < n_tree) {  // tree keys 16 warp ..: 16-bit rows, zeros past the tree
        const size_t head = (size_t)L.g * D, step = (size_t)pr.Hkv * D;
        auto row16 = [&](const void* base, int key, int word) -> uint4 {
          if (key >= m) return make_uint4(0u, 0u, 0u, 0u);
          return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) +
                                                      (size_t)(L.s.n0 + key) * step + head + 8 * word));
        };
        chunk([&](int j, int w) { return row16(a.tree_k, 16 * warp + 8 * j + g, KW * c + w); },
              [&](int i, int w, int odd) {
                const uint4 x = row16(a.tree_v, 16 * warp + 8 * i + 2 * c, VW * g + w);
                const uint4 y = row16(a.tree_v, 16 * warp + 8 * i + 2 * c + 1, VW * g + w);
                const uint32_t sel = odd ? 0x7632u : 0x5410u;
                return make_uint4(__byte_perm(x.x, y.x, sel), __byte_perm(x.y, y.y, sel), __byte_perm(x.z, y.z, sel),
                                  __byte_perm(x.w, y.w, sel));
              },
              true,
              [&](int nt, int x) { return anc[nt][x] >> (16 * warp); });
      }
      const int first = tree ? 1 : 0;
      for (int k = first + (team + kTeams - (int)(base % kTeams)) % kTeams; k < S.n; k += kTeams) {
        const uint32_t raw = base + (k - first), stage = raw % C::kStages, phase = raw / C::kStages & 1u;
        if (ok) ok = warp_wait(FULL + 8 * stage, phase, abort_flag, args.wait_ns);
        int key0 = 0, lim = kKeyTile;  // the tile's first key (used under a window) and its keys
        bool cut = false;
        if (win) {
          key0 = tile_key0(L.s, S.tile0 + k);
          lim = tile_keys(pr, L.s, S.tile0 + k);
          cut = window_cuts(pr, L.s, key0, lim);
        } else if (k == S.n - 1) {
          lim = min(kKeyTile, L.s.len - (S.tile0 + k - 1) * kKeyTile);
        }
#pragma unroll 1
        for (int at = 16 * (warp % C::kTeam); at < lim && ok; at += 16 * C::kTeam) {
          const uint32_t rec = sbase + stage * C::kRawBytes + at * C::kRec;
          // all loads first
          uint32_t kc[2][KW], vc[4][VW], ks[2], vs[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t key = rec + (8 * j + g) * C::kRec;
            if constexpr (KW == 4) {
              const uint4 x = ld_shared_v4(key + 16 * c);
              kc[j][0] = x.x; kc[j][1] = x.y; kc[j][2] = x.z; kc[j][3] = x.w;
              ks[j] = ld_shared_u16(key + D + 2 * c);
            } else {
              const uint2 x = ld_shared_v2(key + 8 * c);
              kc[j][0] = x.x; kc[j][1] = x.y;
              ks[j] = ld_shared_u8(key + D + c);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 2 * c + (i & 1) + 8 * (i >> 1);  // key of code i
            const uint32_t key = rec + row * C::kRec;
            if constexpr (VW == 2) {
              const uint2 x = ld_shared_v2(key + D / 2 + 8 * g);
              vc[i][0] = x.x; vc[i][1] = x.y;
              vs[i] = ld_shared_u8(key + D + D / 16 + g);
            } else {
              vc[i][0] = ld_shared(key + D / 2 + 4 * g);
              vs[i] = ld_shared_u8(key + D + D / 16 + (g >> 1));
            }
            if (at + row >= lim) vs[i] = 0u;  // past the tile's last key: another sequence's, or nothing's
          }
          uint32_t s1[2], c1[2], s2[2] = {}, c2[2] = {}, sv[2], cv[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            widen_scale<kBF16>(ks[j], 0, s1[j], c1[j]);
            if constexpr (KW == 4) widen_scale<kBF16>(ks[j], 1, s2[j], c2[j]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) widen_scales<kBF16>(vs[2 * i] | (vs[2 * i + 1] << 16), sv[i], cv[i]);
          chunk([&](int j, int w) { return w < 2 ? widen8<kBF16>(kc[j][w], s1[j], c1[j]) : widen8<kBF16>(kc[j][w], s2[j], c2[j]); },
                [&](int i, int w, int odd) {  // the codes of the two keys' even (odd) elements side by side
                  return widen8<kBF16>(__byte_perm(vc[2 * i][w], vc[2 * i + 1][w], odd ? 0x7632u : 0x5410u), sv[i], cv[i]);
                },
                cut || at + 16 > lim,
                [&](int nt, int x) {
                  return win ? window_bits(key0 + at, lim - at, low[nt][x], pr.sinks) : bits_below(lim - at);
                });
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(EMPTY + 8 * stage);
      }
      base += S.n - first;

      // ---------------------------------------------------------------- the warps' partials
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float l = l_run[nt][x];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          if (g == 0) {
            xm[warp * C::kRows + 8 * nt + 2 * c + x] = m_run[nt][x];
            xl[warp * C::kRows + 8 * nt + 2 * c + x] = l;
          }
        }
      bar_sync(1, 32 * kWarps);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 8 * nt + 2 * c + x;
          float top = -INFINITY, total = 0.f;
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, xm[w * C::kRows + row]);
          for (int w = 0; w < kWarps; ++w) {
            const float mw = xm[w * C::kRows + row];
            total += xl[w * C::kRows + row] * (mw == -INFINITY ? 0.f : ex2(mw - top));
          }
          // under a window a row may see no key of the segment: its partial is 0, log 0
          const float scale = m_run[nt][x] == -INFINITY || total == 0.f ? 0.f : ex2(m_run[nt][x] - top) / total;
          float* dst = xo + (warp * C::kRows + row) * C::kORow + NE * g;
#pragma unroll
          for (int e = 0; e < NE; e += 4) {  // columns e .. e + 3: word e / 8, tiles of its even and odd elements
            const int t0 = e / 8 * 4 + (e / 4 & 1), t1 = t0 + 2;
            *reinterpret_cast<float4*>(dst + e) = make_float4(o[nt][t0][x] * scale, o[nt][t1][x] * scale,
                                                              o[nt][t0][2 + x] * scale, o[nt][t1][2 + x] * scale);
          }
          if (warp == 0 && g == 0 && node[nt][x] >= 0) {
            const size_t slot = (size_t)partial_slot(pr, u, L, false);
            if (slot < (size_t)a.slots) a.lse_part[slot * 128 + row] = top + log2f(total);
          }
        }
      bar_sync(1, 32 * kWarps);
      const size_t slot = (size_t)partial_slot(pr, u, L, false);
      if (slot >= (size_t)a.slots) {  // cannot happen for a consistent layout; never write past it
        if (threadIdx.x == 0) set_status(a.status, kStatusInvalidArg);
        continue;
      }
      const int rows = min(C::kRows, m * G);
      for (int i = threadIdx.x; i < C::kRows * (D / 4); i += 32 * kWarps) {
        const int row = i % C::kRows, cg = i / C::kRows;
        if (row >= rows) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(xo + (w * C::kRows + row) * C::kORow + 4 * cg);
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        *reinterpret_cast<float4*>(a.o_part + o_part_offset(slot, row, cg, 128, D)) = v;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) set_status(a.status, kStatusTimeout);
}

template <int D, bool kBF16, int NT>
cudaError_t launch_typed(const WinPartialArgs& a, cudaStream_t s) {
  auto kernel = partials_kv4_rows_kernel<D, kBF16, NT>;
  const WinProblem& pr = a.pr;
  CUtensorMap mraw;
  if (!make_record_map(&mraw, pr.kv_capacity > 0 ? a.k_cache : a.tree_k, kv4_record_bytes(D), pr.Hkv, pr.kv_capacity))
    return cudaErrorInvalidValue;
  constexpr int smem = Rows<D, NT>::kSmemBytes;
  const cudaError_t e = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                                   "cudaFuncSetAttribute(partials_kv4_rows_kernel)");
  if (e != cudaSuccess) return e;
  RowArgs ra{a, 0, 0};
  tc_wait_settings(&ra.wait_ns, &ra.stall);
  return check_cuda(launch_pdl(kernel, dim3(pr.U), dim3(Rows<D, NT>::kThreads), (size_t)smem, s, mraw, ra),
                    "launch partials_kv4_rows_kernel");
}

template <int NT>
cudaError_t launch_nt(const WinPartialArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) return a.pr.d == 64 ? launch_typed<64, true, NT>(a, s) : launch_typed<128, true, NT>(a, s);
  return a.pr.d == 64 ? launch_typed<64, false, NT>(a, s) : launch_typed<128, false, NT>(a, s);
}

}  // namespace

cudaError_t launch_partials_kv4_rows(const WinPartialArgs& a, int rows, bool bf16, cudaStream_t s) {
  return rows <= 8 ? launch_nt<1>(a, bf16, s) : launch_nt<2>(a, bf16, s);
}

}  // namespace tva
