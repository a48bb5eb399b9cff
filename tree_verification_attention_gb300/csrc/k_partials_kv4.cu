// k_partials_kv4.cu - attention partials over a 4-bit prefix cache (kv4.cuh) on the
// 5th-generation tensor cores; q, the tree's K / V and the output bf16 or fp16.
//
// What is computed is what k_partials_tc.cu computes, for a prefix whose K and V are
// records of 4-bit codes with a scale for 16 of them.  The matrix instructions that take
// 4-bit operands would need Q and P in few bits too, so the records are widened to q's
// type - exactly: a value has at most 7 significant bits - on their way to the tensor
// cores: DRAM and L2 carry 144 bytes a row and head (d = 128) instead of 512.
//
// How (one CTA per SM; Roles gives the warps):
//   producer warp: TMA of Q, and of the raw 128-record tiles (a box of records, 18 KB at
//           d = 128) into a ring of their own.
//   widening warps: thread r widens record r of a tile: 16 bytes of codes become 64 bytes of
//           a K or V tile in the 128-byte-swizzled ring that the MMAs read.  A shift and one
//           and-or put two codes n into the mantissas of 128 + n (fp16: 16 + n), one fused
//           multiply-add takes the offset off and applies the scale.  Rows past a tile's last
//           key are written as zeros, so nothing that a record of another sequence holds can
//           reach a product.  The tree tile's K / V are 16-bit already and fetched by TMA.
//   MMA warp, softmax warps: as in k_partials_tc.cu, two streams of 4 softmax warps.  A
//           softmax warp whose 32 rows are all padding leaves its logits alone.
// TMEM columns: S/P buffers at 0 and 128, O accumulators at 256 and 384 (512 total).
// A window (pr.window > 0) is handled as there too, at run time: it only adds masks to the
// tiles that its lower edge crosses.
//
// Measured (bf16, d = 128, Hkv 8, both launches back to back): 64 nodes, Hq 32, over 65536 rows
// 67 us (the products' floor 35.8); 8 sequences of 4k .. 32k rows, 32 nodes 91 us (31.2); 128
// nodes, Hq 64, over 131072 rows 419 us (286).  No unit is saturated (tensor 46 %, issue slots
// 46 % in the first): what bounds it is the chain of a tile - softmax, products, widening,
// with a hand-over between each two - and issue slots shared by the widening and softmax.  The
// register split spills 80 to 132 bytes a thread (W = 1), 32 to 72 (W = 2).
// Row groups of up to 16 rows go to k_partials_kv4_rows.cu, which has no such chain.
//
// Every wait is bounded as in k_partials_tc.cu.
#include <cuda.h>

#include <algorithm>
#include <cstdio>

#include "kv4.cuh"
#include "tc_pipeline.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

using namespace ptx;

constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 16-bit values (one swizzle span)
// The warps of a kernel for row groups of W M-tiles, and the registers per thread of its
// warpgroups (two of softmax, the widening ones, the rest).  They share what the block is
// launched with (checked before the first launch): a split above that would wait forever.
//   W = 1: a widening warpgroup each for K and V.  A tile's K or V is a chain of about 1300
//          clocks however few rows the tree has; one warpgroup for both took 3000 a tile,
//          more than everything else (8 sequences, 4k..32k: 105 us; 89 when it was split).
//   W = 2: one for both.  The softmax of two M-tiles then bounds a tile and is slowed by
//          every further warp (64k prefix, 64 nodes: 68 us instead of 72).
template <int W>
struct Roles {
  static constexpr int kWidenGroups = W == 1 ? 2 : 1;
  static constexpr int kWidenWarp = 8;
  static constexpr int kProducerWarp = kWidenWarp + 4 * kWidenGroups;
  static constexpr int kMmaWarp = kProducerWarp + 1;
  static constexpr int kThreads = 32 * (kProducerWarp + 4);
  static constexpr int kLaunchRegs = W == 1 ? 96 : 128;
  static constexpr int kSoftmaxRegs = W == 1 ? 152 : 168;
  static constexpr int kWidenRegs = W == 1 ? 56 : 88;
  static constexpr int kOtherRegs = W == 1 ? 64 : 88;
  static_assert(2 * kSoftmaxRegs + kWidenGroups * kWidenRegs + kOtherRegs <= (3 + kWidenGroups) * kLaunchRegs,
                "register split");
};

template <int D, int W>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kStages = (D == 128 ? 3 : 6) + (W == 1 ? 1 : 0);
  static constexpr int kRawBytes = kKeyTile * kv4_record_bytes(D);
  static constexpr int kRaws = D == 128 ? 3 : 6;
  static constexpr int kQBytes = W * kTileBytes;
  static constexpr int kRawOff = kQBytes + kStages * kTileBytes;
  static constexpr int kBarOff = kRawOff + kRaws * kRawBytes;
  static constexpr int kCuOff = 4096;               // staged cu_* arrays inside misc
  static constexpr int kCuCap = 1024;               // ints: batches up to 511 sequences
  static constexpr int kMiscBytes = kCuOff + 4 * kCuCap;
  static constexpr int kSmemBytes = kBarOff + kMiscBytes + 1024;  // + alignment slack
};

struct Kv4Args {
  WinPartialArgs a;
  int npt;  // nodes per M-tile: floor(128 / G)
  // What is fetched of an M-tile's nodes and of the tree tile's rows: no more than the
  // largest tree has.  A TMA copy takes time for each row of its box, so full boxes would
  // hold up the first tiles of small trees.
  int q_nodes, tree_rows;
  uint64_t wait_ns;  // limit of every main-loop wait
  int stall;         // test hook: the MMA thread first waits on a barrier nothing completes
};

// Ring positions of a segment's K and V tiles, after those of the earlier segments.  With
// W = 2: K0 V0 K1 V1 ..; with W = 1: K0, K1, then V_j followed by K_{j+2}.
__device__ __forceinline__ int ring_k(int W, int k) { return W == 2 ? 2 * k : (k < 2 ? k : 2 * k - 1); }
__device__ __forceinline__ int ring_v(int W, int k, int n) {
  return W == 2 ? 2 * k + 1 : (k <= n - 2 ? 2 + 2 * k : 2 * n - 1);
}

// One row's K or V values (codes at `codes`, scales at `scales`, both shared addresses) into
// a swizzled tile whose row starts at `row`, the swizzle's row term already in it.  All loads
// come first.
template <int D, bool kBF16>
__device__ __forceinline__ void widen_row(uint32_t codes, uint32_t scales, uint32_t row) {
  uint4 code[D / 32];
  uint32_t sc1 = 0u, s[D / 16], c[D / 16];
#pragma unroll
  for (int q = 0; q < D / 32; ++q) code[q] = ld_shared_v4(codes + 16 * q);
  const uint32_t sc = ld_shared(scales);
  if constexpr (D == 128) sc1 = ld_shared(scales + 4);
#pragma unroll
  for (int b = 0; b < D / 16; ++b) widen_scale<kBF16>(b < 4 ? sc : sc1, b & 3, s[b], c[b]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // chunk i of a span (of both at d = 128)
    const uint32_t at = row ^ (uint32_t)(i << 4);
    const uint4 v = code[i >> 2];
    const uint32_t w = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    st_shared_v4_at<0>(at, widen8<kBF16>(w, s[i >> 1], c[i >> 1]));
    if constexpr (D == 128) {
      const uint4 v1 = code[2 + (i >> 2)];
      const uint32_t w1 = (i & 3) == 0 ? v1.x : (i & 3) == 1 ? v1.y : (i & 3) == 2 ? v1.z : v1.w;
      st_shared_v4_at<kHalfBytes>(at, widen8<kBF16>(w1, s[4 + (i >> 1)], c[4 + (i >> 1)]));
    }
  }
}

// The 128 logits of this thread's row.
__device__ __forceinline__ void load_row(uint32_t taddr, uint32_t* s) {
  tmem_ld32(taddr, s);
  tmem_ld32(taddr + 32, s + 32);
  tmem_ld32(taddr + 64, s + 64);
  tmem_ld32(taddr + 96, s + 96);
  tmem_wait_ld32(s);
  tie32(s + 32);
  tie32(s + 64);
  tie32(s + 96);
}

__device__ __forceinline__ void mbar_arrive_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}

template <int D, bool kBF16, bool kShare, int W>
__global__ void __launch_bounds__(Roles<W>::kThreads, 1)
    partials_kv4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_raw,
                        const __grid_constant__ CUtensorMap tm_tk, const __grid_constant__ CUtensorMap tm_tv,
                        const Kv4Args args) {
  using C = Cfg<D, W>;
  using R = Roles<W>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const WinPartialArgs& a = args.a;
  WinProblem* pr_s = reinterpret_cast<WinProblem*>(smem + C::kBarOff + C::kCuOff - 128);
  static_assert(sizeof(WinProblem) <= 128, "staged problem");
  const WinProblem& pr = *pr_s;
  const int npt = args.npt, G = a.pr.G;  // kernel parameters: readable before staging
  const uint64_t wait_ns = args.wait_ns;  // main-loop waits; drains use kDrainNs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = blockIdx.x;

  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_s = sbase;
  const uint32_t kv_s = sbase + C::kQBytes;
  const uint32_t raw_s = sbase + C::kRawOff;
  const uint32_t bar0 = sbase + C::kBarOff;
  const uint32_t KV_FULL = bar0;                          // [kStages], 4 widening warps
  const uint32_t KV_EMPTY = KV_FULL + 8 * C::kStages;     // [kStages]
  const uint32_t RAW_FULL = KV_EMPTY + 8 * C::kStages;    // [kRaws]
  const uint32_t RAW_EMPTY = RAW_FULL + 8 * C::kRaws;     // [kRaws], 4 widening warps
  const uint32_t Q_FULL = RAW_EMPTY + 8 * C::kRaws;
  const uint32_t Q_EMPTY = Q_FULL + 8;
  const uint32_t S_FULL = Q_EMPTY + 8;                    // [2]
  const uint32_t P_FULL = S_FULL + 16;                    // [2]
  const uint32_t O_FULL = P_FULL + 16;                    // [2]
  const uint32_t TREE_FULL = O_FULL + 16;                 // [2]: the tree tile's K, V have landed
  const uint32_t TREE_EMPTY = TREE_FULL + 16;             // [2], 4 widening warps: they have been taken
  const uint32_t PAR_READY = TREE_EMPTY + 16;             // [2]
  const uint32_t O_FREE = PAR_READY + 16;
  const uint32_t M1_READY = O_FREE + 8;
  const uint32_t DRAIN = M1_READY + 8;                    // at most 8 x 43 bytes in all
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 448);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 452);
  float* m1_s = reinterpret_cast<float*>(smem + C::kBarOff + 512);  // [2][128]
  float* l1_s = m1_s + 256;                                         // [2][128]
  int* par_s = reinterpret_cast<int*>(smem + C::kBarOff + 2560);    // [2][128] parent ids

  // ---- Set-up that reads nothing an earlier kernel may write (programmatic dependent).
  if (warp == R::kProducerWarp && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_raw);
    prefetch_tmap(&tm_tk);
    prefetch_tmap(&tm_tv);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(KV_FULL + 8 * s, 4);
      mbar_init(KV_EMPTY + 8 * s, 1);
    }
    for (int s = 0; s < C::kRaws; ++s) {
      mbar_init(RAW_FULL + 8 * s, 1);
      mbar_init(RAW_EMPTY + 8 * s, 4 * R::kWidenGroups);
    }
    mbar_init(Q_FULL, 1);
    mbar_init(Q_EMPTY, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(S_FULL + 8 * w, 1);
      mbar_init(P_FULL + 8 * w, 128);
      mbar_init(O_FULL + 8 * w, 1);
      mbar_init(TREE_FULL + 8 * w, 1);
      mbar_init(TREE_EMPTY + 8 * w, 4);
      mbar_init(PAR_READY + 8 * w, 128);
    }
    mbar_init(O_FREE, 256);
    mbar_init(M1_READY, 128);
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
    __threadfence_block();
  }
  pdl_wait();  // launched as a programmatic dependent: inputs are final after this
  pdl_launch_dependents();
  long long t_begin = 0, t_end = 0;
  stage_problem(a.pr, pr_s, reinterpret_cast<int*>(smem + C::kBarOff + C::kCuOff), C::kCuCap);
  worker_range(pr, u, t_begin, t_end, kShare);
  if (u == 0 && threadIdx.x == 0) validate_sequences(pr, a.status);
  if (t_begin >= t_end) return;  // uniform over the CTA

  // The other warps wait for the TMEM allocation on named barrier 1, which the producer
  // warp only arrives at: it goes straight on to its first copies.
  uint32_t tmem = 0;
  if (warp == R::kProducerWarp) {
    __syncwarp();
    bar_arrive(1, R::kThreads);
  } else {
    if (warp == R::kMmaWarp) {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
    tc_fence_before();
    bar_sync(1, R::kThreads);
    tc_fence_after();
    tmem = *tmem_slot;
  }

  if (warp >= R::kProducerWarp) {
    reg_dec<R::kOtherRegs>();
    if (warp == R::kProducerWarp) {
      // ---------------------------------------------------------------- producer
      // All 32 lanes run this role; one elected lane issues each copy and expect-tx.
      int raw = 0, sg = 0;
      int q_loads = 0;  // segments whose Q has been issued
      bool ok = true;
      long long t = t_begin;
      Segment S;
      const uint32_t q_box_bytes = 64u * G * args.q_nodes * 2u;
      const uint64_t evict_first = policy_evict_first();  // records are read once
      while (ok && next_segment(pr, u, t, t_end, S, kShare)) {
        const Loc& L = S.L;
        const int n = S.n;
        const bool tree = S.tile0 == 0;
        const int n_raw = n - (tree ? 1 : 0);
        auto load_q = [&]() -> bool {
          if (sg > 0 && !warp_wait(Q_EMPTY, (sg - 1) & 1, abort_flag, wait_ns)) return false;
          mbar_expect_tx_elect(Q_FULL, (uint32_t)W * C::kHalves * q_box_bytes);
          for (int mt = 0; mt < W; ++mt) {
            int qrow = L.s.n0 + (L.mp * W + mt) * npt;  // past the sequence's nodes: padding rows
            if (!TVA_CHECK(qrow >= L.s.n0 && L.g >= 0 && L.g < pr.Hkv, a.status)) qrow = 0;
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d_elect(q_s + (mt * C::kHalves + h) * kHalfBytes, &tm_q, 64 * h, L.g * G, qrow, Q_FULL);
          }
          ++q_loads;
          return true;
        };
        auto load_raw = [&](int i) -> bool {  // the segment's i-th prefix tile
          const int stage = raw % C::kRaws, use = raw / C::kRaws;
          if (use > 0 && !warp_wait(RAW_EMPTY + 8 * stage, (use - 1) & 1, abort_flag, wait_ns)) return false;
          int z = L.s.p0 + tile_key0(L.s, S.tile0 + (tree ? 1 : 0) + i);
          if (!TVA_CHECK(z >= 0 && z < L.s.p0 + L.s.len && z < pr.kv_capacity, a.status)) z = 0;
          mbar_expect_tx_elect(RAW_FULL + 8 * stage, C::kRawBytes);
          tma_load_3d_hint_elect(raw_s + stage * C::kRawBytes, &tm_raw, 0, L.g, z, RAW_FULL + 8 * stage, evict_first);
          ++raw;
          return true;
        };
        // The first kRaws record tiles wait only for earlier segments, so they may be
        // fetched before this segment's Q; the later ones wait for this segment's own
        // progress, which needs it.
        int i = 0;
        if (sg > 0)
          for (; i < min(n_raw, C::kRaws) && ok; ++i) ok = load_raw(i);
        ok = ok && load_q();
        for (; i < n_raw && ok; ++i) ok = load_raw(i);
        ++sg;
      }
      // drain: every copy this thread started has landed before TMEM / smem go away
      for (int i = max(0, raw - C::kRaws); i < raw; ++i)
        drain_wait(RAW_FULL + 8 * (i % C::kRaws), (i / C::kRaws) & 1);
      if (q_loads > 0) drain_wait(Q_FULL, (q_loads - 1) & 1);
    } else if (warp == R::kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      // All 32 lanes run this role; the *_elect forms issue each MMA / commit from one lane.
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, kBF16);
      constexpr uint32_t idesc_o = idesc_bf16(128, D, true, kBF16);
      int ring = 0, sg = 0;
      uint32_t pbits = 0;  // bit w: parity of the next P_FULL[w] phase
      bool ok = true;
      long long t = t_begin;
      Segment S;
      auto wait_kv = [&](int idx) -> bool {
        if (!warp_wait(KV_FULL + 8 * (idx % C::kStages), (idx / C::kStages) & 1, abort_flag, wait_ns)) return false;
        tc_fence_after();
        return true;
      };
      // Operand descriptors, stepped through their low word.  K / Q are K-major, V MN-major.
      const uint32_t k_hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
      const uint32_t v_hi = (uint32_t)(sdesc_sw128(0, kHalfBytes, 1024) >> 32);
      const uint32_t k_lo = (uint32_t)sdesc_sw128(kv_s, 16, 1024);
      const uint32_t v_lo = (uint32_t)sdesc_sw128(kv_s, kHalfBytes, 1024);
      const uint32_t q_lo = (uint32_t)sdesc_sw128(q_s, 16, 1024);
      auto issue_s = [&](int w, int mt, int idx) {
        const uint32_t kl = k_lo + (uint32_t)((idx % C::kStages) * C::kTileBytes >> 4);
        const uint32_t ql = q_lo + (uint32_t)(mt * C::kTileBytes >> 4);
        const uint32_t dt = tmem + w * 128;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (uint32_t)((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          mma_ss_elect(dt, desc_join(ql + o, k_hi), desc_join(kl + o, k_hi), idesc_s, ks > 0);
        }
        tc_commit_elect(S_FULL + 8 * w);
      };
      auto issue_pv = [&](int w, int idx, bool acc) {
        const uint32_t vl = v_lo + (uint32_t)((idx % C::kStages) * C::kTileBytes >> 4);
        const uint32_t dt = tmem + 256 + w * 128, at = tmem + w * 128;
#pragma unroll
        for (int ks = 0; ks < kKeyTile / 16; ++ks)
          mma_ts_elect(dt, at + ks * 8, desc_join(vl + (uint32_t)(ks * 2048 >> 4), v_hi), idesc_o,
                       (acc || ks > 0) ? 1u : 0u);
      };
      auto wait_p = [&](int w) -> bool {
        if (!warp_wait(P_FULL + 8 * w, (pbits >> w) & 1u, abort_flag, wait_ns)) return false;
        tc_fence_after();
        return true;
      };
      auto wait_ofree = [&]() -> bool {
        if (sg == 0) return true;
        if (!warp_wait(O_FREE, (sg - 1) & 1, abort_flag, wait_ns)) return false;
        tc_fence_after();
        return true;
      };
      auto free_kv = [&](int idx) { tc_commit_elect(KV_EMPTY + 8 * (idx % C::kStages)); };
      if (args.stall && !warp_wait(DRAIN, 0, abort_flag, wait_ns)) ok = false;  // test hook
      while (ok && next_segment(pr, u, t, t_end, S, kShare)) {
        const int n = S.n;
        if (!warp_wait(Q_FULL, sg & 1, abort_flag, wait_ns)) { ok = false; break; }
        tc_fence_after();
        auto rK = [&](int k) { return ring + ring_k(W, k); };
        auto rV = [&](int k) { return ring + ring_v(W, k, n); };
        if (!(ok = wait_kv(rK(0)))) break;
        issue_s(0, 0, rK(0));
        if (W == 2) {
          issue_s(1, 1, rK(0));
          free_kv(rK(0));
          if (n == 1) tc_commit_elect(Q_EMPTY);
          for (int k = 0; k < n && ok; ++k) {
            if (!(ok = wait_kv(rV(k)))) break;
            for (int w = 0; w < 2 && ok; ++w) {
              if (!(ok = wait_p(w))) break;
              if (k == 0 && w == 0 && !(ok = wait_ofree())) break;
              issue_pv(w, rV(k), k > 0);
              pbits ^= 1u << w;
              if (k == n - 1) tc_commit_elect(O_FULL + 8 * w);
              if (w == 1) free_kv(rV(k));
              if (k + 1 < n) {
                if (w == 0 && !(ok = wait_kv(rK(k + 1)))) break;
                issue_s(w, w, rK(k + 1));
                if (w == 1) {
                  free_kv(rK(k + 1));
                  if (k + 1 == n - 1) tc_commit_elect(Q_EMPTY);
                }
              }
            }
          }
        } else {
          free_kv(rK(0));
          if (n > 1) {
            if (!(ok = wait_kv(rK(1)))) break;
            issue_s(1, 0, rK(1));
            free_kv(rK(1));
          }
          if (n <= 2) tc_commit_elect(Q_EMPTY);
          for (int j = 0; j < n && ok; ++j) {
            const int w = j & 1;
            if (!(ok = wait_kv(rV(j)))) break;
            if (!(ok = wait_p(w))) break;
            if (j == 0 && !(ok = wait_ofree())) break;
            issue_pv(w, rV(j), j >= 2);
            pbits ^= 1u << w;
            free_kv(rV(j));
            if (j + 2 >= n) tc_commit_elect(O_FULL + 8 * w);
            if (j + 2 < n) {
              if (!(ok = wait_kv(rK(j + 2)))) break;
              issue_s(w, 0, rK(j + 2));
              free_kv(rK(j + 2));
              if (j + 2 == n - 1) tc_commit_elect(Q_EMPTY);
            }
          }
        }
        ring += 2 * n;
        ++sg;
      }
      // drain: every MMA issued by this thread has completed before TMEM is freed
      tc_commit_elect(DRAIN);
      drain_wait(DRAIN, 0);
    }
  } else if (warp >= R::kWidenWarp) {
    // ------------------------------------------------------------------ widening
    reg_dec<R::kWidenRegs>();
    const int r = threadIdx.x & 127;  // the tile's row (key) of this thread
    const uint32_t row_s = kv_s + r * 128 + ((r & 7) << 4);  // 16-byte chunk c of a span is at c ^ (row mod 8)
    const uint32_t rec_s = raw_s + r * kv4_record_bytes(D);
    const int mine = (warp - R::kWidenWarp) >> 2;  // W = 1: 0 widens K, 1 V
    uint32_t raw = 0, raw_ph = 0;
    int ring = 0, trees = 0, k_loads = 0, v_loads = 0;
    bool ok = true;
    long long t = t_begin;
    Segment S;
    while (ok && next_segment(pr, u, t, t_end, S, kShare)) {
      const int n = S.n;
#pragma unroll 1
      for (int i = 0; i < (R::kWidenGroups == 2 ? n : 2 * n); ++i) {
        const int k = R::kWidenGroups == 2 ? i : i >> 1;
        const bool is_v = (R::kWidenGroups == 2 ? mine : i & 1) != 0;
        const int idx = ring + (is_v ? ring_v(W, k, n) : ring_k(W, k));
        const uint32_t stage = (uint32_t)idx % C::kStages, use = (uint32_t)idx / C::kStages;
        const int tile = S.tile0 + k;
        // The stage's last tile has been used.  (A wait for the phase before a fresh barrier's
        // first returns at once.  With two groups the tiles in between are the other's: its
        // place in the ring is at most three from this group's last one, whose wait implies
        // that every phase but the awaited one is complete - tiles are released in order.)
        if (!(ok = warp_wait(KV_EMPTY + 8 * stage, (use & 1u) ^ 1u, abort_flag, wait_ns))) break;
        int lim;  // rows from here on are written as zeros
        if (tile == 0) {
          // The tree's own K / V are 16-bit already: the group's first warp fetches them into
          // the stage.  (It cannot be the producer warp, which does not follow the ring:
          // a phase of KV_EMPTY that it had not waited for in turn looks like the one two
          // earlier.)  Rows past the tree are another sequence's, or nothing's.
          const uint32_t tree_bar = is_v ? 8 : 0;
          if ((warp & 3) == 0) {
            // TREE_FULL stays one phase ahead: every warp has seen the last tree's
            if (trees > 0 && !(ok = warp_wait(TREE_EMPTY + tree_bar, (trees - 1) & 1, abort_flag, wait_ns))) break;
            int z = S.L.s.n0;
            if (!TVA_CHECK(z >= 0 && z < pr.node_capacity && S.L.s.m > 0, a.status)) z = 0;
            mbar_expect_tx_elect(TREE_FULL + tree_bar, (uint32_t)C::kHalves * 128u * args.tree_rows);
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d_elect(kv_s + stage * C::kTileBytes + h * kHalfBytes, is_v ? &tm_tv : &tm_tk, 64 * h, S.L.g,
                                z, TREE_FULL + tree_bar);
            (is_v ? v_loads : k_loads)++;
          }
          if (!(ok = warp_wait(TREE_FULL + tree_bar, trees & 1, abort_flag, wait_ns))) break;
          mbar_arrive_elect(TREE_EMPTY + tree_bar);
          lim = S.L.s.m;
        } else {
          if (!(ok = warp_wait(RAW_FULL + 8 * raw, raw_ph, abort_flag, wait_ns))) break;
          lim = tile_keys(pr, S.L.s, tile);
          const uint32_t rec = rec_s + raw * C::kRawBytes;
          if (r < lim)
            widen_row<D, kBF16>(rec + (is_v ? D / 2 : 0), rec + D + (is_v ? D / 16 : 0), row_s + stage * C::kTileBytes);
          if (R::kWidenGroups == 2 || is_v) {  // done with the records
            __syncwarp();
            mbar_arrive_elect(RAW_EMPTY + 8 * raw);
            raw = raw + 1 == C::kRaws ? 0 : raw + 1;
            raw_ph ^= raw == 0 ? 1u : 0u;
          }
        }
        if (r >= lim) {
          const uint32_t dst = kv_s + stage * C::kTileBytes + r * 128;
#pragma unroll
          for (int c = 0; c < 8 * C::kHalves; ++c)
            st_shared_v4(dst + (c >> 3) * kHalfBytes + (c & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
        }
        fence_async_shared();  // the MMAs read the stage through the asynchronous proxy
        __syncwarp();
        mbar_arrive_elect(KV_FULL + 8 * stage);
      }
      ring += 2 * n;
      if (S.tile0 == 0) ++trees;
    }
    // drain: the copies that this warp started
    if (k_loads > 0) drain_wait(TREE_FULL, (k_loads - 1) & 1);
    if (v_loads > 0) drain_wait(TREE_FULL + 8, (v_loads - 1) & 1);
  } else {
    // ------------------------------------------------------------------ softmax
    reg_inc<R::kSoftmaxRegs>();
    const int w = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = w * 128, o_col = 256 + w * 128;
    const float sl2 = a.scale_log2;
    const bool win = a.pr.window > 0;
    int cnt = 0, of0 = 0, of1 = 0, sg = 0, pars = 0;
    bool ok = true;
    long long t = t_begin;
    Segment S;
    while (ok && next_segment(pr, u, t, t_end, S, kShare)) {
      const Loc& L = S.L;
      const int n = S.n;
      const int mt = (W == 2) ? w : 0;
      const int node = (L.mp * W + mt) * npt + r / G;  // local node id of this row
      bool row_ok = r < npt * G && node < L.s.m;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      // The tree tile needs the row's ancestor bits; under a window every tile may need its
      // depth.  PAR_READY's even phases complete when the parents are in place, its odd ones
      // when every row of the stream has read them.
      uint32_t anc[4] = {0u, 0u, 0u, 0u};
      int low = 0;  // under a window: the lowest prefix key this row sees through it
      if (win || (S.tile0 == 0 && (W == 2 || w == 0))) {
        int* ps = par_s + w * 128;
        if (pars > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(PAR_READY + 8 * w, 1, abort_flag, wait_ns));
          if (!ok) break;
        }
        if (r < L.s.m) ps[r] = __ldg(a.parent + L.s.n0 + r);
        mbar_arrive(PAR_READY + 8 * w);
        ok = __all_sync(0xffffffffu, mbar_wait(PAR_READY + 8 * w, 0, abort_flag, wait_ns));
        ++pars;
        if (!ok) break;
        if (row_ok) {
          int depth = 0;
          const bool good = win ? window_ancestors(ps, node, pr.window, pr.sinks, L.s.len, anc, depth)
                                : ancestor_bits_shared(ps, node, anc);
          if (!good) set_status(a.status, kStatusBadTree);
          if (win) low = window_low(pr, L.s, depth);
        }
        mbar_arrive(PAR_READY + 8 * w);
      }
      const int n_mine = (W == 2) ? n : (n - w + 1) / 2;
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < n_mine; ++i) {
        const int k = (W == 2) ? i : 2 * i + w;
        const int tile = S.tile0 + k;
        const bool is_tree = tile == 0;
        ok = __all_sync(0xffffffffu, mbar_wait(S_FULL + 8 * w, cnt & 1, abort_flag, wait_ns));
        if (!ok) break;
        tc_fence_after();
        ++cnt;
        if (!warp_ok) {  // only padding rows: what their P and O hold is never read
          tc_fence_before();
          mbar_arrive(P_FULL + 8 * w);
          continue;
        }
        // keys of this tile: [0, lim) exist; the tree tile also needs the ancestor bit
        const int key0 = is_tree ? 0 : tile_key0(L.s, tile);
        const int lim = is_tree ? L.s.m : win ? tile_keys(pr, L.s, tile) : min(kKeyTile, L.s.P - key0);
        if (is_tree || lim < kKeyTile || (win && window_cuts(pr, L.s, key0, lim))) {
          // Rare tiles: rewrite the logits the row does not see to -inf in TMEM, 32 columns
          // at a time, so the two passes below carry no masking code.
#pragma unroll 1
          for (int ck = 0; ck < 4; ++ck) {
            uint32_t sv[32];
            tmem_ld32(tl + s_col + 32 * ck, sv);
            tmem_wait_ld32(sv);
            uint32_t vw;
            if (is_tree) {
              const uint32_t aw = ck == 0 ? anc[0] : ck == 1 ? anc[1] : ck == 2 ? anc[2] : anc[3];
              vw = bits_below(lim - 32 * ck) & (row_ok ? aw : 0u);
            } else if (win) {
              vw = window_bits(key0 + 32 * ck, lim - 32 * ck, low, pr.sinks);
            } else {
              vw = bits_below(lim - 32 * ck);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((vw >> e) & 1u)) sv[e] = kNegInfBits;
            tmem_st32(tl + s_col + 32 * ck, sv);
          }
          tmem_wait_st();
        }
        // pass 1: row maximum; pass 2: p = 2^(s * scale - m).  Each reads the row's 128 logits
        // in one TMEM round trip (keeping them for both costs more registers than there are).
        float mx0 = -INFINITY, mx1 = -INFINITY;
        {
          uint32_t s[128];
          load_row(tl + s_col, s);
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            mx0 = max3(mx0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            mx1 = max3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
          }
        }
        const float m_new = fmaxf(m_run, fmaxf(mx0, mx1) * sl2);
        if (i == 0) {
          m_run = m_new;
        } else {
          const bool need = m_new > m_run + 8.0f;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2(m_run - m_new) : 1.f;
            if (need) {
              l_run *= alpha;
              m_run = m_new;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(tl + o_col + c0, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tl + o_col + c0, o);
            }
            tmem_wait_st();
          }
        }
        const float nb = (m_run == -INFINITY) ? 0.f : -m_run;
        // p packed as 16-bit pairs into the first half of the S buffer; the scaling and the
        // row sum (of the unrounded p, in fp32) run on packed fp32 pairs.
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nbx2 = f2_pack(nb, nb);
        uint64_t lsx2 = f2_pack(0.f, 0.f);
        uint32_t s[128];
        load_row(tl + s_col, s);
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, nbx2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          lsx2 = f2_add(lsx2, f2_pack(p0, p1));
          s[c] = kBF16 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);  // pair c <= 2 c: already read
        }
        tmem_st32(tl + s_col, s);
        tmem_st32(tl + s_col + 32, s + 32);
        float ls0, ls1;
        f2_unpack(lsx2, ls0, ls1);
        l_run += ls0 + ls1;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(P_FULL + 8 * w);
      }
      if (!ok) break;
      // ---------------------------------------------------------------- epilogue
      const size_t slot = (size_t)partial_slot(pr, u, L, kShare);
      if (slot >= (size_t)a.slots) {  // cannot happen for a consistent layout; never write past it
        set_status(a.status, kStatusInvalidArg);
        row_ok = false;
      }
      const int pp = mt * 128 + r;  // padded row: lane = row within a 32-row block
      if (row_ok && !TVA_CHECK(pp < W * 128 && node >= 0 && node < L.s.m, a.status)) row_ok = false;
      float* oblk = a.o_part + o_part_offset(slot, pp, 0, W * 128, D);
      // A row's partial is w0 O_0 (+ w1 O_1); under a window a row may see no key of the
      // segment: its partial is then 0, with log 0.
      float w0, w1 = 0.f, lse;
      bool both = false;
      if (W == 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(O_FULL + 8 * w, (w == 0 ? of0 : of1) & 1, abort_flag, wait_ns));
        if (!ok) break;
        (w == 0 ? of0 : of1)++;
        w0 = l_run > 0.f ? 1.f / l_run : 0.f;
        lse = m_run + log2f(l_run);
      } else if (w == 1) {
        // Stream 1 may own no tile of this segment, so nothing else keeps it from arriving
        // for segment sg before segment sg - 1's release completed: wait for that first.
        if (sg > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(O_FREE, (sg - 1) & 1, abort_flag, wait_ns));
          if (!ok) break;
        }
        m1_s[(sg & 1) * 128 + r] = m_run;
        l1_s[(sg & 1) * 128 + r] = l_run;
        mbar_arrive(M1_READY);
        mbar_arrive(O_FREE);
        ++sg;
        continue;
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(M1_READY, sg & 1, abort_flag, wait_ns));
        if (!ok) break;
        const float m1 = m1_s[(sg & 1) * 128 + r];
        const float l1 = l1_s[(sg & 1) * 128 + r];
        both = n > 1;
        ok = __all_sync(0xffffffffu, mbar_wait(O_FULL, of0 & 1, abort_flag, wait_ns));
        if (!ok) break;
        ++of0;
        if (both) {
          ok = __all_sync(0xffffffffu, mbar_wait(O_FULL + 8, of1 & 1, abort_flag, wait_ns));
          if (!ok) break;
          ++of1;
        }
        const float mm = both ? fmaxf(m_run, m1) : m_run;
        const float a0 = (m_run == -INFINITY) ? 0.f : ex2(m_run - mm);
        const float a1 = (!both || m1 == -INFINITY) ? 0.f : ex2(m1 - mm);
        const float lt = a0 * l_run + a1 * l1;
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        w0 = a0 * inv;
        w1 = a1 * inv;
        lse = mm + log2f(lt);
      }
      tc_fence_after();
      if (warp_ok) {
        const uint32_t oc = tl + (W == 2 ? o_col : 256);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32], o1[32];
          tmem_ld32(oc + c0, o);
          if (both) tmem_ld32(tl + 384 + c0, o1);
          tmem_wait_ld32(o);
          if (both) tie32(o1);
          if (row_ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 v;
              v.x = __uint_as_float(o[e]) * w0 + (both ? __uint_as_float(o1[e]) * w1 : 0.f);
              v.y = __uint_as_float(o[e + 1]) * w0 + (both ? __uint_as_float(o1[e + 1]) * w1 : 0.f);
              v.z = __uint_as_float(o[e + 2]) * w0 + (both ? __uint_as_float(o1[e + 2]) * w1 : 0.f);
              v.w = __uint_as_float(o[e + 3]) * w0 + (both ? __uint_as_float(o1[e + 3]) * w1 : 0.f);
              *reinterpret_cast<float4*>(oblk + (c0 + e) * 32) = v;
            }
          }
        }
      }
      if (row_ok) a.lse_part[slot * (W * 128) + pp] = lse;
      tc_fence_before();
      mbar_arrive(O_FREE);
      ++sg;
    }
  }
  // ------------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) set_status(a.status, kStatusTimeout);
  if (warp == R::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBF16, bool kShare, int W>
cudaError_t launch_typed(const WinPartialArgs& a, int npt, cudaStream_t s) {
  constexpr CUtensorMapDataType type = kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto kernel = partials_kv4_kernel<D, kBF16, kShare, W>;
  const WinProblem& pr = a.pr;
  CUtensorMap mq, mraw, mtk, mtv;
  const int q_nodes = std::min(npt, pr.max_nodes), tree_rows = std::min(kKeyTile, (pr.max_nodes + 7) / 8 * 8);
  if (!make_map(&mq, type, a.q, D, pr.Hq, pr.node_capacity, pr.G, q_nodes) ||
      !make_record_map(&mraw, pr.kv_capacity > 0 ? a.k_cache : a.tree_k, kv4_record_bytes(D), pr.Hkv, pr.kv_capacity) ||
      !make_map(&mtk, type, a.tree_k, D, pr.Hkv, pr.node_capacity, 1, tree_rows) ||
      !make_map(&mtv, type, a.tree_v, D, pr.Hkv, pr.node_capacity, 1, tree_rows))
    return cudaErrorInvalidValue;
  constexpr int smem = Cfg<D, W>::kSmemBytes;
  cudaError_t e = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                             "cudaFuncSetAttribute(partials_kv4_kernel)");
  if (e != cudaSuccess) return e;
  // The warpgroups' register shares must not exceed what the block is launched with.
  static const int regs = [&] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, kernel) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs < Roles<W>::kLaunchRegs) {
    record_error("launch partials_kv4_kernel", regs, "built with fewer registers than its warpgroups share");
    return cudaErrorInvalidConfiguration;
  }
  Kv4Args ka{a, npt, q_nodes, tree_rows, 0, 0};
  tc_wait_settings(&ka.wait_ns, &ka.stall);
  return check_cuda(launch_pdl(kernel, dim3(pr.U), dim3(Roles<W>::kThreads), (size_t)smem, s, mq, mraw, mtk, mtv, ka),
                    "launch partials_kv4_kernel");
}

template <bool kShare, int W>
cudaError_t launch_mode(const WinPartialArgs& a, bool bf16, int npt, cudaStream_t s) {
  if (bf16)
    return a.pr.d == 64 ? launch_typed<64, true, kShare, W>(a, npt, s) : launch_typed<128, true, kShare, W>(a, npt, s);
  return a.pr.d == 64 ? launch_typed<64, false, kShare, W>(a, npt, s) : launch_typed<128, false, kShare, W>(a, npt, s);
}

}  // namespace

cudaError_t launch_partials_kv4(const WinPartialArgs& a, bool bf16, int W, int npt, cudaStream_t s) {
  // Of the largest row group.  Up to 16 rows the other kernel is the faster one (one token over
  // 131072 rows: 44 us instead of 76), from 17 on this one (32 rows: 75 us instead of 122).
  const int rows = a.pr.G * std::min(npt, a.pr.max_nodes);
  if (W == 1 && a.pr.share == 0 && rows <= 16) return launch_partials_kv4_rows(a, rows, bf16, s);
  if (W == 1)
    return a.pr.share != 0 ? launch_mode<true, 1>(a, bf16, npt, s) : launch_mode<false, 1>(a, bf16, npt, s);
  return a.pr.share != 0 ? launch_mode<true, 2>(a, bf16, npt, s) : launch_mode<false, 2>(a, bf16, npt, s);
}

}  // namespace tva
