// k_gdn_chunk.cu - a Gated DeltaNet layer's tokens in chunks of 64 on the tensor cores (bf16).
//
// The recurrence S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, o_t = S_t^T q_t
// ("DFlash-TfM", Method 3) over a chunk of C tokens, from the state S before it.  With G_ij the
// product of alpha over the tokens j+1 .. i, g_i that over the chunk's first tokens up to i, and
//     A = strict_lower(beta_i G_ij k_i.k_j),   T = (I + A)^-1,
// (the page's "(I + X) U = beta V" for a chain) the corrections are U = T diag(beta) r with
// r_i = v_i - g_i S^T k_i, the outputs o_i = g_i S^T q_i + sum_{j <= i} G_ij (q_i.k_j) u_j and
// the state after the chunk S' = g_C S + sum_i G_Ci k_i u_i^T.  What does not depend on the state
// is made ahead of it, so that the chain from state to state is two products deep:
//     W = K^T diag(G_Ci) T diag(beta)    [d x C]      S' = g_C S + W r
//     P = lower(G o Q K^T) T diag(beta)  [C x C]      O  = g o (Q S) + P r
//
// One CTA per (sequence, head, 32 columns of d_v), 13 warps:
//   warps 0-3   (recurrence): X = [K; Q] S (one M = 128 product: lanes 0-63 are K rows, 64-127
//               Q rows), r, then W r and P r.  Thread = TMEM lane; S stays in fp32 in registers,
//               lane = row of d_k.
//   warps 4-11  (two groups of four, chunks in turn): [K; Q] K^T, the decays, T by blocks, W and P,
//               left in TMEM where the recurrence's products read them as their A operand.
//   warp 12     (producer): TMA copies of K and Q tiles into three stages.
// Each group issues its own MMAs from its first warp after a barrier of the group.
//
// Precision: K, Q and V are bf16 inputs and exact.  S, T, W, G o (Q K^T), P and r are fp32 values held
// as two bf16 terms each, so that products have operands of 16 bits or more (a term is off by 2^-17;
// the products of two low terms are left out, 2^-18).  With single terms the outputs would be
// off by 3.5e-3 of their size instead of 1.7e-3 (the rounding of a bf16 output), and by more than
// 5e-3 with keys that repeat: there W r and P r are small sums of large terms.  Sums, decays, T and
// the state are fp32.
//
// Every wait is bounded (as in the attention kernels): when one expires the abort flag is raised,
// the groups leave their loops together at their next barrier, everything in flight is drained
// (again bounded), TMEM is freed and TVA_ERR_TIMEOUT recorded; the state is then not written.
#include <cuda.h>
#include <cuda_bf16.h>

#include "tc_pipeline.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

using namespace ptx;

constexpr int kChunk = 64;
constexpr int kCols = 32;             // columns of d_v per CTA
constexpr int kThreadsCh = 512;      // 13 warps work; the last four share one register budget
constexpr int kProducer = 12;
constexpr int kSpan = kChunk * 128;   // 64 rows of 64 bf16
constexpr int kStagesCh = 3;
constexpr int kLd = kChunk + 4;       // row pitch of A / T in floats
constexpr int kLdX = 36;              // row pitch of the blocks' intermediate product

// TMEM columns: per preparing group 192 ([K; Q] K^T, then G o (Q K^T); W; P; each becomes its hi and lo
// terms in place), then X; once X is read P r goes to its first half and W r to its second.
constexpr uint32_t kTmGroup = 192, kTmW = 64, kTmP = 128, kTmX = 384, kTmD = 416;

template <int D>
struct Ch {
  static constexpr int kHalves = D / 64;
  static constexpr int kStage = kHalves * 2 * kSpan;          // per half: K rows, then Q rows
  static constexpr int kSOff = kStagesCh * kStage;            // S: [D rows][hi 32 | lo 32]
  static constexpr int kROff = kSOff + D * 128;               // r hi, r lo: [64 rows][32, padded to 64]
  static constexpr int kTOff = kROff + 2 * kSpan;             // per group: T hi, lo (for P)
  static constexpr int kZeroOff = kTOff + 2 * 2 * kSpan;      // D = 64: zeros for rows 64 .. 127 of K^T
  static constexpr int kAOff = kZeroOff + (D == 64 ? kSpan : 0);
  // per group: A, then T; then T hi, lo (for W)
  static constexpr int kXOff = kAOff + 2 * kChunk * kLd * 4;
  static constexpr int kGateOff = kXOff + 2 * 32 * kLdX * 4;
  static constexpr int kGate = 4 * kChunk + 8;                // floats per group: alpha, beta, G_Ci; g, g_C
  static constexpr int kBarOff = kGateOff + 2 * kGate * 4;
  static constexpr int kSmem = kBarOff + 256 + 1024;
};

// Barrier `id` over a group of 128 threads; true in all of them when `ok` is in all.
__device__ __forceinline__ bool group_all(int id, bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r != 0;
}

// Two fp32 values as two packed bf16 terms each: hi + lo.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi));
}

struct ChunkArgs {
  GdnUpdateArgs a;
  uint64_t wait_ns;
  int stall;   // test hook: the recurrence first waits on a barrier that nothing completes
};

template <int D>
__global__ void __launch_bounds__(kThreadsCh, 1)
    gdn_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const ChunkArgs args) {
  using C = Ch<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const GdnUpdateArgs& a = args.a;
  const uint64_t wait_ns = args.wait_ns;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t KQ_FULL = bars, KQ_EMPTY = bars + 24, READY = bars + 48, OUT_EMPTY = bars + 64, P_DONE = bars + 80,
                 X_DONE = bars + 96, D_DONE = bars + 104, O_DONE = bars + 112, DRAIN = bars + 120;   // DRAIN [3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 164);

  if (warp == kProducer && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    for (int s = 0; s < kStagesCh; ++s) {
      mbar_init(KQ_FULL + 8 * s, 1);
      mbar_init(KQ_EMPTY + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(READY + 8 * g, 128);
      mbar_init(OUT_EMPTY + 8 * g, 1);
      mbar_init(P_DONE + 8 * g, 1);
    }
    mbar_init(X_DONE, 1);
    mbar_init(D_DONE, 1);
    mbar_init(O_DONE, 1);
    for (int g = 0; g < 3; ++g) mbar_init(DRAIN + 8 * g, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (D == 64) {
    for (int e = tid; e < kSpan / 16; e += kThreadsCh)
      *reinterpret_cast<uint4*>(smem + C::kZeroOff + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_shared();
  }
  pdl_wait();
  pdl_launch_dependents();
  constexpr int CS = D / kCols;
  const int cs = blockIdx.x % CS, bh = blockIdx.x / CS;
  const int b = bh / a.H, h = bh % a.H;
  const int t0 = __ldg(a.cu + b);
  const int n = __ldg(a.cu + b + 1) - t0;
  if (!(t0 >= 0 && n >= 0 && n <= a.max_tokens && (long long)t0 + n <= a.token_capacity)) {
    if (tid == 0) set_status(a.status, kStatusInvalidArg);
    return;   // uniform over the CTA
  }
  if (n == 0) return;
  const int chunks = (n + kChunk - 1) / kChunk;

  if (warp == kProducer) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kProducer) {
    // ------------------------------------------------------------------ producer
    reg_dec<24>();
    bool ok = warp == kProducer;
    int c = 0;
    for (; ok && c < chunks; ++c) {
      const int st = c % kStagesCh, use = c / kStagesCh;
      if (use > 0 && !(ok = warp_wait(KQ_EMPTY + 8 * st, (use - 1) & 1, abort_flag, wait_ns))) break;
      int z = t0 + c * kChunk;
      if (!TVA_CHECK(z >= 0 && z < a.token_capacity, a.status)) z = 0;
      mbar_expect_tx_elect(KQ_FULL + 8 * st, (uint32_t)C::kStage);
      for (int hf = 0; hf < C::kHalves; ++hf) {
        const uint32_t at = sbase + st * C::kStage + hf * 2 * kSpan;
        tma_load_3d_elect(at, &tm_k, 64 * hf, h, z, KQ_FULL + 8 * st);
        tma_load_3d_elect(at + kSpan, &tm_q, 64 * hf, h, z, KQ_FULL + 8 * st);
      }
    }
    for (int i = max(0, c - kStagesCh); i < c; ++i)   // every copy has landed before the CTA ends
      drain_wait(KQ_FULL + 8 * (i % kStagesCh), (i / kStagesCh) & 1);
  } else if (warp >= 4) {
    reg_inc<160>();   // 3 x 128 x 160 + 128 x 24 of the block's 512 x 128 registers
    // ------------------------------------------------------------------ W and P of every other chunk
    const int g = (warp - 4) >> 2, t = (tid - 128) & 127, w = t >> 5;
    const int bar_id = 2 + g;
    const uint32_t tw = tmem + kTmGroup * g;
    const uint32_t lane_base = (uint32_t)(w * 32) << 16;
    float* As = reinterpret_cast<float*>(smem + C::kAOff) + g * kChunk * kLd;
    float* Xs = reinterpret_cast<float*>(smem + C::kXOff) + g * 32 * kLdX;
    float* al_s = reinterpret_cast<float*>(smem + C::kGateOff) + g * C::kGate;   // alpha
    float* be_s = al_s + kChunk;                                                 // beta
    float* en_s = be_s + kChunk;                                                 // G_Ci
    float* ga_s = en_s + kChunk;                                                 // g_i, then g_C
    uint8_t* Tp = smem + C::kTOff + g * 2 * kSpan;
    const uint32_t tp = sbase + C::kTOff + g * 2 * kSpan;
    uint8_t* Tw = reinterpret_cast<uint8_t*>(As);
    const uint32_t tws = sbase + C::kAOff + g * kChunk * kLd * 4;
    static_assert(kChunk * kLd * 4 % 1024 == 0 && kChunk * kLd * 4 >= 2 * kSpan, "T's terms over A");
    constexpr uint32_t idesc_a = idesc_bf16(128, 64, false);                 // [K; Q] K^T: both K-major
    constexpr uint32_t idesc_w = idesc_bf16(128, 64, true) | (1u << 15);     // K^T T: A along M, B along N
    constexpr uint32_t idesc_p = idesc_bf16(128, 64, true);                  // A in TMEM
    const uint32_t kmaj_hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    const uint32_t mnmaj_hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);    // the LBO field is in the low word
    uint32_t ph = 0;   // parity of P_DONE
    bool ok = true;
    const int row = t & 63;         // this lane's token row (of K for t < 64, of Q above)
    for (int c = g; c < chunks; c += 2) {
      const int st = c % kStagesCh, cnt = min(kChunk, n - c * kChunk);
      const uint32_t kq = sbase + st * C::kStage;
      // gates (rows past the sequence's end: no decay, nothing written)
      float al = 1.f, be = 0.f;
      if (t < 64 && t < cnt) {
        const size_t at = (size_t)(t0 + c * kChunk + t) * a.H + h;
        al = __ldg(a.alpha + at);
        be = __ldg(a.beta + at);
      }
      ok = mbar_wait(KQ_FULL + 8 * st, (c / kStagesCh) & 1, abort_flag, wait_ns) && ok;
      if (cnt < kChunk) {
        // rows of K and Q past the end belong to other sequences or to none: zeros instead
        for (int e = t; e < C::kHalves * 2 * 8 * (kChunk - cnt); e += 128) {
          const int r = cnt + (e >> 3) % (kChunk - cnt), part = (e >> 3) / (kChunk - cnt);
          *reinterpret_cast<uint4*>(smem + st * C::kStage + part * kSpan + r * 128 + (e & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_shared();
      }
      if (t < 64) {
        al_s[t] = al;
        be_s[t] = be;
      }
      ok = group_all(bar_id, ok);
      if (!ok) break;
      if (w == 0) {
        tc_fence_after();
        const uint32_t lo = (uint32_t)sdesc_sw128(kq, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (uint32_t)((ks >> 2) * 2 * kSpan + (ks & 3) * 32) >> 4;
          mma_ss_elect(tw, desc_join(lo + o, kmaj_hi), desc_join(lo + o, kmaj_hi), idesc_a, ks > 0);
        }
        tc_commit_elect(P_DONE + 8 * g);
      }
      // products of the decays from the chunk's start and to its end: 64 threads, a scan each way
      float pre = al, suf = 1.f;
      if (t < 64) {
        suf = t < 63 ? al_s[t + 1] : 1.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_up_sync(0xffffffffu, pre, o), y = __shfl_down_sync(0xffffffffu, suf, o);
          if (lane >= o) pre *= x;
          if (lane + o < 32) suf *= y;
        }
        // across the two warps: the other one's 32 factors, multiplied by every lane's share
        float other = t < 32 ? al_s[32 + lane] : al_s[lane];
        if (t < 32 && lane == 0) other = 1.f;   // al_s[32] is already in warp 0's suffixes
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) other *= __shfl_xor_sync(0xffffffffu, other, o);
        if (t < 32) suf *= other;
        else pre *= other;
        en_s[t] = suf;
      }
      ok = mbar_wait(P_DONE + 8 * g, ph, abort_flag, wait_ns);
      ph ^= 1;
      tc_fence_after();
      {
        uint32_t d[64];
        tmem_ld32(tw + lane_base, d);
        tmem_ld32(tw + lane_base + 32, d + 32);
        tmem_wait_ld32(d);
        tie32(d + 32);
        // row `row` of beta_i G_ij k_i.k_j (j < i), or of G_ij q_i.k_j (j <= i)
        const bool qrow = t >= 64;
        float p = qrow ? 1.f : be;
        const int last = qrow ? row : row - 1;
#pragma unroll
        for (int j4 = 60; j4 >= 0; j4 -= 4) {
          const float4 a4 = *reinterpret_cast<const float4*>(al_s + j4);
          const float next = j4 < 60 ? al_s[j4 + 4] : 1.f;
          const float f[4] = {a4.y, a4.z, a4.w, next};   // alpha of token j + 1
#pragma unroll
          for (int e = 3; e >= 0; --e) {
            const int j = j4 + e;
            if (j < row) p *= f[e];
            d[j] = j <= last ? __float_as_uint(__uint_as_float(d[j]) * p) : 0u;
          }
        }
        if (!qrow) {
#pragma unroll
          for (int j = 0; j < 64; j += 4)
            *reinterpret_cast<uint4*>(As + row * kLd + j) = make_uint4(d[j], d[j + 1], d[j + 2], d[j + 3]);
#pragma unroll
          for (int j = 0; j < 64; ++j) d[j] = 0u;
        } else {
          uint32_t o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            split2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]), d[j], o[j]);
#pragma unroll
          for (int j = 0; j < 32; ++j) d[32 + j] = o[j];
        }
        tmem_st32(tw + lane_base, d);   // lower(G o Q K^T) in lanes 64 .. 127, zeros above
        tmem_st32(tw + lane_base + 32, d + 32);
        tmem_wait_st();
        tc_fence_before();
      }
      ok = group_all(bar_id, ok);
      if (!ok) break;
      // ---- T = (I + A)^-1: 16-row diagonal blocks by substitution (a column per lane), then the
      // blocks below them, T21 = -T22 (A21 T11), at 16 and at 32 rows
      {
        const int o = 16 * w, cc = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s0 = i == cc ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
          for (int j = 0; j < i; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(As + (o + i) * kLd + o + j);
            s0 = fmaf(-v.x, x[j], s0);
            if (j + 1 < i) s1 = fmaf(-v.y, x[j + 1], s1);
            if (j + 2 < i) s0 = fmaf(-v.z, x[j + 2], s0);
            if (j + 3 < i) s1 = fmaf(-v.w, x[j + 3], s1);
          }
          x[i] = s0 + s1;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) As[(o + i) * kLd + o + cc] = x[i];
        }
      }
      group_all(bar_id, true);
      {
        const int o = 32 * (w >> 1), tt = t & 63, i = tt >> 2, c4 = 4 * (tt & 3);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float x = As[(o + 16 + i) * kLd + o + k];
          const float4 v = *reinterpret_cast<const float4*>(As + (o + k) * kLd + o + c4);
          s.x = fmaf(x, v.x, s.x); s.y = fmaf(x, v.y, s.y); s.z = fmaf(x, v.z, s.z); s.w = fmaf(x, v.w, s.w);
        }
        float* X = Xs + (w >> 1) * 16 * kLdX;
        *reinterpret_cast<float4*>(X + i * kLdX + c4) = s;
        group_all(bar_id, true);
        s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float x = -As[(o + 16 + i) * kLd + o + 16 + k];
          const float4 v = *reinterpret_cast<const float4*>(X + k * kLdX + c4);
          s.x = fmaf(x, v.x, s.x); s.y = fmaf(x, v.y, s.y); s.z = fmaf(x, v.z, s.z); s.w = fmaf(x, v.w, s.w);
        }
        *reinterpret_cast<float4*>(As + (o + 16 + i) * kLd + o + c4) = s;
      }
      group_all(bar_id, true);
      {
        // 32 x 32 x 32: rows i and i + 16, four columns a thread, on packed pairs of columns
        const int i = t >> 3, c4 = 4 * (t & 7);
        auto product = [&](const float* L, const float* R, int ldr, float sign, float4& o0, float4& o1) {
          uint64_t s00 = 0, s01 = 0, s10 = 0, s11 = 0;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 x0 = *reinterpret_cast<const float4*>(L + i * kLd + k);
            const float4 x1 = *reinterpret_cast<const float4*>(L + (i + 16) * kLd + k);
            const float y0[4] = {x0.x, x0.y, x0.z, x0.w}, y1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(R + (k + e) * ldr + c4);
              const uint64_t p0 = f2_pack(y0[e], y0[e]), p1 = f2_pack(y1[e], y1[e]);
              s00 = f2_fma(p0, v.x, s00);
              s01 = f2_fma(p0, v.y, s01);
              s10 = f2_fma(p1, v.x, s10);
              s11 = f2_fma(p1, v.y, s11);
            }
          }
          f2_unpack(s00, o0.x, o0.y);
          f2_unpack(s01, o0.z, o0.w);
          f2_unpack(s10, o1.x, o1.y);
          f2_unpack(s11, o1.z, o1.w);
          o0.x *= sign; o0.y *= sign; o0.z *= sign; o0.w *= sign;
          o1.x *= sign; o1.y *= sign; o1.z *= sign; o1.w *= sign;
        };
        float4 o0, o1;
        product(As + 32 * kLd, As, kLd, 1.f, o0, o1);                 // A21 T11
        *reinterpret_cast<float4*>(Xs + i * kLdX + c4) = o0;
        *reinterpret_cast<float4*>(Xs + (i + 16) * kLdX + c4) = o1;
        group_all(bar_id, true);
        product(As + 32 * kLd + 32, Xs, kLdX, -1.f, o0, o1);          // -T22 (A21 T11)
        *reinterpret_cast<float4*>(As + (32 + i) * kLd + c4) = o0;
        *reinterpret_cast<float4*>(As + (48 + i) * kLd + c4) = o1;
      }
      group_all(bar_id, true);
      {
        // T diag(beta) (for P) and diag(G_Ci) T diag(beta) (for W, over A's place), two terms each:
        // row i is the products' k = i, its columns lie along N
        const int i = t >> 1, j0 = 32 * (t & 1);
        const float en = en_s[i];
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(As + i * kLd + j0 + j);
          const float4 bb = *reinterpret_cast<const float4*>(be_s + j0 + j);
          x[j] = v.x * bb.x; x[j + 1] = v.y * bb.y; x[j + 2] = v.z * bb.z; x[j + 3] = v.w * bb.w;
        }
        group_all(bar_id, true);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t hi[4], lo[4];
          const int at = i * 128 + (((j0 >> 3) + q) ^ (i & 7)) * 16;
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], lo[e]);
          *reinterpret_cast<uint4*>(Tp + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(Tp + kSpan + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(x[8 * q + 2 * e] * en, x[8 * q + 2 * e + 1] * en, hi[e], lo[e]);
          *reinterpret_cast<uint4*>(Tw + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(Tw + kSpan + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async_shared();
      }
      // the recurrence is done with this group's previous W, P and decays
      if (c >= 2) ok = mbar_wait(OUT_EMPTY + 8 * g, ((c >> 1) - 1) & 1, abort_flag, wait_ns);
      ok = group_all(bar_id, ok);
      if (!ok) break;
      if (w == 0) {
        tc_fence_after();
        const uint32_t lbo = D == 128 ? 2u * kSpan : sbase + C::kZeroOff - kq;   // rows 64 .. of K^T
        const uint32_t klo = (uint32_t)sdesc_sw128(kq, lbo, 1024);
        const uint32_t wlo = (uint32_t)sdesc_sw128(tws, 16, 1024), plo = (uint32_t)sdesc_sw128(tp, 16, 1024);
#pragma unroll
        for (int part = 0; part < 2; ++part)   // hi and lo terms
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss_elect(tw + kTmW, desc_join(klo + (ks * 2048 >> 4), mnmaj_hi),
                         desc_join(wlo + ((part * kSpan + ks * 2048) >> 4), mnmaj_hi), idesc_w, part > 0 || ks > 0);
#pragma unroll
        for (int part = 0; part < 3; ++part)   // hi hi, hi lo, lo hi
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ts_elect(tw + kTmP, tw + (part == 2 ? 32 : 0) + ks * 8,
                         desc_join(plo + (((part == 1 ? kSpan : 0) + ks * 2048) >> 4), mnmaj_hi), idesc_p,
                         part > 0 || ks > 0);
        tc_commit_elect(P_DONE + 8 * g);
      }
      if (t < 64) ga_s[t] = pre;
      if (t == 63) ga_s[64] = pre;
      ok = mbar_wait(P_DONE + 8 * g, ph, abort_flag, wait_ns);
      ph ^= 1;
      tc_fence_after();
      {
        uint32_t d[64], o[32];
        tmem_ld32(tw + kTmW + lane_base, d);
        tmem_ld32(tw + kTmW + lane_base + 32, d + 32);
        tmem_wait_ld32(d);
        tie32(d + 32);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          split2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]), d[j], o[j]);
        tmem_st32(tw + kTmW + lane_base, d);
        tmem_st32(tw + kTmW + lane_base + 32, o);
        tmem_ld32(tw + kTmP + lane_base, d);
        tmem_ld32(tw + kTmP + lane_base + 32, d + 32);
        tmem_wait_ld32(d);
        tie32(d + 32);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          split2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]), d[j], o[j]);
        tmem_st32(tw + kTmP + lane_base, d);
        tmem_st32(tw + kTmP + lane_base + 32, o);
        tmem_wait_st();
        tc_fence_before();
      }
      mbar_arrive(READY + 8 * g);
    }
    if (w == 0) {
      tc_commit_elect(DRAIN + 8 * g);
      drain_wait(DRAIN + 8 * g, 0);
    }
  } else {
    // ------------------------------------------------------------------ recurrence
    reg_inc<160>();
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const bool krow = tid < 64;
    const int row = tid & 63;
    constexpr uint32_t idesc_x = idesc_bf16(128, 64, true);
    constexpr uint32_t idesc_d = idesc_bf16(128, kCols, true);
    const uint32_t hi_word = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    const uint32_t s_lo = (uint32_t)sdesc_sw128(sbase + C::kSOff, 16, 1024);
    const uint32_t r_lo = (uint32_t)sdesc_sw128(sbase + C::kROff, 16, 1024);
    const size_t hs = (size_t)a.H * D;
    float* Sg = a.state + (((size_t)b * a.H + h) * D + (tid < D ? tid : 0)) * D + cs * kCols;
    float S[kCols];
#pragma unroll
    for (int j = 0; j < kCols; j += 4) {
      const float4 v = tid < D ? *reinterpret_cast<const float4*>(Sg + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
    }
    const __nv_bfloat16* Vg = static_cast<const __nv_bfloat16*>(a.v) + (size_t)t0 * hs + (size_t)h * D + cs * kCols;
    __nv_bfloat16* Og = static_cast<__nv_bfloat16*>(a.out) + (size_t)t0 * hs + (size_t)h * D + cs * kCols;
    uint4 vr[4];
    auto fetch_v = [&](int c) {   // this lane's row of chunk c's V (K lanes)
      if (krow && c * kChunk + row < n) {
        const uint4* src = reinterpret_cast<const uint4*>(Vg + (size_t)(c * kChunk + row) * hs);
#pragma unroll
        for (int q = 0; q < 4; ++q) vr[q] = __ldg(src + q);
      }
    };
    // this lane's row of S in two terms, as k = row of a product, columns along N: hi 32, lo 32
    auto stage_s = [&]() {
      if (tid < D) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(S[8 * q + 2 * e], S[8 * q + 2 * e + 1], hi[e], lo[e]);
          uint8_t* at = smem + C::kSOff + tid * 128;
          *reinterpret_cast<uint4*>(at + ((q ^ (tid & 7)) * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + (((4 + q) ^ (tid & 7)) * 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_shared();
    };
    fetch_v(0);
    stage_s();
    float oq[kCols];        // Q lanes: g_i S^T q_i of the chunk
    uint32_t od[kCols];     // and its P r
    // Test hook: DRAIN's phase completes only through this group's own commit below.
    bool ok = args.stall ? mbar_wait(DRAIN + 16, 0, abort_flag, wait_ns) : true;
    auto write_out = [&](int c) {
      if (krow || c * kChunk + row >= n) return;
      uint4* dst = reinterpret_cast<uint4*>(Og + (size_t)(c * kChunk + row) * hs);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * q + 2 * e;
          p[e] = pack_bf16x2(oq[j] + __uint_as_float(od[j]), oq[j + 1] + __uint_as_float(od[j + 1]));
        }
        dst[q] = make_uint4(p[0], p[1], p[2], p[3]);
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const int g = c & 1, st = c % kStagesCh, cnt = min(kChunk, n - c * kChunk);
      const float* ga_s = reinterpret_cast<const float*>(smem + C::kGateOff) + g * C::kGate + 3 * kChunk;
      const uint32_t tw = tmem + kTmGroup * g;
      ok = mbar_wait(READY + 8 * g, (c >> 1) & 1, abort_flag, wait_ns) && ok;
      ok = group_all(1, ok);
      if (!ok) break;
      if (warp == 0) {
        tc_fence_after();
        const uint32_t kq = (uint32_t)sdesc_sw128(sbase + st * C::kStage, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (uint32_t)((ks >> 2) * 2 * kSpan + (ks & 3) * 32) >> 4;
          mma_ss_elect(tmem + kTmX, desc_join(kq + o, hi_word), desc_join(s_lo + (ks * 2048 >> 4), hi_word), idesc_x, ks > 0);
        }
        tc_commit_elect(X_DONE);
      }
      if (c > 0) write_out(c - 1);   // while the product runs
      const float ga = ga_s[row], gc = ga_s[64];
      ok = mbar_wait(X_DONE, c & 1, abort_flag, wait_ns);
      tc_fence_after();
      {
        uint32_t x[64];
        tmem_ld32(tmem + kTmX + lane_base, x);
        tmem_ld32(tmem + kTmX + lane_base + 32, x + 32);
        tmem_wait_ld32(x);
        tie32(x + 32);
        if (krow) {
          const bool live = row < cnt;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t hi[4], lo[4];
            const uint32_t vw[4] = {vr[q].x, vr[q].y, vr[q].z, vr[q].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * q + 2 * e;
              const float x0 = __uint_as_float(x[j]) + __uint_as_float(x[32 + j]);
              const float x1 = __uint_as_float(x[j + 1]) + __uint_as_float(x[33 + j]);
              const float r0 = live ? fmaf(-ga, x0, bf16_lo(vw[e])) : 0.f;
              const float r1 = live ? fmaf(-ga, x1, bf16_hi(vw[e])) : 0.f;
              split2(r0, r1, hi[e], lo[e]);
            }
            uint8_t* at = smem + C::kROff + row * 128 + ((q ^ (row & 7)) * 16);
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(at + kSpan) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          fence_async_shared();
          fetch_v(c + 1);
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j) oq[j] = ga * (__uint_as_float(x[j]) + __uint_as_float(x[32 + j]));
        }
      }
      tc_fence_before();
      ok = group_all(1, ok);
      if (!ok) break;
      if (warp == 0) {
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < 3; ++part) {   // W_hi r_hi, W_hi r_lo, W_lo r_hi
          const uint32_t at = tw + kTmW + (part == 2 ? 32 : 0), rb = r_lo + (part == 1 ? kSpan >> 4 : 0);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ts_elect(tmem + kTmD, at + ks * 8, desc_join(rb + (ks * 2048 >> 4), hi_word), idesc_d, part > 0 || ks > 0);
        }
        tc_commit_elect(D_DONE);
#pragma unroll
        for (int part = 0; part < 3; ++part) {   // P likewise
          const uint32_t at = tw + kTmP + (part == 2 ? 32 : 0), rb = r_lo + (part == 1 ? kSpan >> 4 : 0);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ts_elect(tmem + kTmX, at + ks * 8, desc_join(rb + (ks * 2048 >> 4), hi_word), idesc_d, part > 0 || ks > 0);
        }
        tc_commit_elect(O_DONE);
        tc_commit_elect(OUT_EMPTY + 8 * g);
        tc_commit_elect(KQ_EMPTY + 8 * st);
      }
      ok = mbar_wait(D_DONE, c & 1, abort_flag, wait_ns);
      tc_fence_after();
      {
        uint32_t x[32];
        tmem_ld32(tmem + kTmD + lane_base, x);
        tmem_wait_ld32(x);
#pragma unroll
        for (int j = 0; j < kCols; ++j) S[j] = fmaf(gc, S[j], __uint_as_float(x[j]));
      }
      stage_s();
      ok = mbar_wait(O_DONE, c & 1, abort_flag, wait_ns) && ok;
      tc_fence_after();
      tmem_ld32(tmem + kTmX + lane_base, od);
      tmem_wait_ld32(od);
      tc_fence_before();
    }
    ok = group_all(1, ok && !*abort_flag);
    if (ok) {
      write_out(chunks - 1);
      if (tid < D) {
#pragma unroll
        for (int j = 0; j < kCols; j += 4)
          *reinterpret_cast<float4*>(Sg + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      }
    }
    if (warp == 0) {
      tc_commit_elect(DRAIN + 16);
      drain_wait(DRAIN + 16, 0);
    }
  }
  // ------------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(a.status, kStatusTimeout);
  if (warp == kProducer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_chunk_typed(const GdnUpdateArgs& a, cudaStream_t s) {
  CUtensorMap mq, mk;
  if (!make_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, D, a.H, a.token_capacity, 1, kChunk) ||
      !make_map(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k, D, a.H, a.token_capacity, 1, kChunk))
    return cudaErrorInvalidValue;
  constexpr int smem = Ch<D>::kSmem;
  static_assert(smem <= 232448, "shared memory of one CTA");
  cudaError_t e = check_cuda(cudaFuncSetAttribute(gdn_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                             "cudaFuncSetAttribute(gdn_chunk_kernel)");
  if (e != cudaSuccess) return e;
  ChunkArgs ca{a, 0, 0};
  tc_wait_settings(&ca.wait_ns, &ca.stall);
  return check_cuda(launch_pdl(gdn_chunk_kernel<D>, dim3((unsigned)((long long)a.B * a.H * (D / kCols))),
                               dim3(kThreadsCh), (size_t)smem, s, mq, mk, ca),
                    "launch gdn_chunk_kernel");
}

}  // namespace

cudaError_t launch_gdn_chunk(const GdnUpdateArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_chunk_typed<64>(a, s) : launch_chunk_typed<128>(a, s);
}

}  // namespace tva
