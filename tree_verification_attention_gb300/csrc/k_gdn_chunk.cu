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
// Two kernels.  The first makes W and P of every (sequence, head, chunk), all at once, one CTA of
// eight warps each (four resident per SM), and leaves them in the workspace as the second's shared
// memory will hold them (48 KB at d = 128).  The second walks a sequence's chunks, one CTA per (sequence,
// head, 64 or 32 columns of d_v): a producer warp fetches K, Q, W and P a chunk ahead, a warp issues the
// products, and the others hold the state in registers (fp32; thread = row of d_k = TMEM lane, 16 columns):
//     X = [K; Q] S (one M = 128 product: lanes 0-63 are K rows, 64-127 Q rows) -> r -> W r, P r.
// Long prompts go in segments of chunks, a pair of launches each, so that the workspace stays bounded; a
// segment is prepared beside the walk through the one before it.
//
// What bounds it, measured at 32 heads, d = 128 (GB300, CUDA events): 4096 tokens 138 us, 32768 tokens 969 us
// (1.12 TB/s and 106 TFLOP/s of the recurrence's own products; floor 160 us, its bytes).  The walk is a chain of
// some 2350 clocks a chunk: X 640 (eight MMAs of 39 clocks, then their latency, commit and wake-up), r 370, W r
// 580, the state's update and split 340, two hand-overs of 170 and 120; no unit is busy (tensor 24 %, issue 23 %).
// The preparation of 2048 (head, chunk) pairs takes 47 us, 49 % of the issue slots, 44 % of the shared-memory
// pipe: some 11500 warp instructions each, half of them splits and layouts.
// Steps (4096 / 32768 tokens): one kernel that made W and P beside the walk, each CTA for its own columns,
// 374 / 2942 us (four times the preparation, and 108 KB of code that ran at the rate of its instruction
// fetches); two kernels 254 / 1922; the products issued by a warp of their own, no barrier among the state's
// holders 190 / 1402; images out by bulk copies, T read without bank conflicts 181 / 1330; 16 columns a thread, 32
// a CTA where each has an SM 148 / 1080; the inverse's blocks on mma.sync 141 / 1042; a segment prepared
// beside the walk before it 140 / 987; eight warps a preparing CTA 138 / 969.
//
// Precision: K, Q and V are bf16 inputs and exact.  S, T, W, G o (Q K^T), P and r are fp32 values held
// as two bf16 terms each, so that products have operands of 16 bits or more (a term is off by 2^-17;
// the products of two low terms are left out, 2^-18).  With single terms the outputs would be
// off by 3.5e-3 of their size instead of 1.7e-3 (the rounding of a bf16 output), and by more than
// 5e-3 with keys that repeat: there W r and P r are small sums of large terms.  Sums, decays, T and
// the state are fp32.
//
// Every wait is bounded (as in the attention kernels): when one expires the abort flag is raised, every
// warp leaves its loop at its next wait, everything in flight is drained (again bounded), TMEM is
// freed and TVA_ERR_TIMEOUT recorded; the state is then not written.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "tc_pipeline.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

using namespace ptx;

constexpr int kChunk = 64;
constexpr int kSpan = kChunk * 128;   // 64 rows of 64 bf16: one 128-byte swizzle span
constexpr int kLd = kChunk + 4;       // row pitch of A / T in floats
constexpr int kLdX = 36;              // row pitch of the blocks' intermediate product

// What the first kernel leaves for the second, per (sequence, head, chunk): W hi, W lo [D rows of 64
// tokens], P hi, P lo [64 rows of 64 tokens], K-major and swizzled, then g_i (64 floats).
template <int D>
struct Image {
  static constexpr int kW = D * 128;
  static constexpr int kP = 2 * kW;
  static constexpr int kG = kP + 2 * kSpan;
  static constexpr int kBytes = kG + kChunk * 4;
};

// Two fp32 values as two packed bf16 terms each: hi + lo.
__device__ __forceinline__ void split2(uint64_t x2, uint32_t& hi, uint32_t& lo) {
  float a, b;
  f2_unpack(x2, a, b);
  hi = pack_bf16x2(a, b);
  f2_unpack(f2_fma(f2_pack(bf16_lo(hi), bf16_hi(hi)), f2_pack(-1.f, -1.f), x2), a, b);
  lo = pack_bf16x2(a, b);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) { split2(f2_pack(a, b), hi, lo); }

// Block barrier; true when `ok` is in every thread.  The vote tells the compiler that the answer is the
// same throughout a warp, so that what follows keeps its operands in uniform registers.
__device__ __forceinline__ bool all_threads(bool ok) { return __all_sync(0xffffffffu, __syncthreads_and(ok)); }

struct ChunkArgs {
  GdnUpdateArgs a;
  uint8_t* images;       // [B][segment][H]
  int chunk0, span;      // first chunk and chunks of each sequence in this pair of launches
  int segment;           // images a sequence and head has room for
  uint64_t wait_ns;
  int stall;   // test hook: the state kernel first waits on a barrier that nothing completes
};

__device__ __forceinline__ bool sequence_ok(const GdnUpdateArgs& a, int t0, int n) {
  return t0 >= 0 && n >= 0 && n <= a.max_tokens && (long long)t0 + n <= a.token_capacity;
}

// ------------------------------------------------------------------ W and P of one chunk

constexpr int kThreadsPr = 256;   // TMEM lane t % 128, columns (of 64) 32 (t / 128) ..
constexpr uint32_t kTmWork = 64;   // TMEM: [K; Q] K^T, then G o (Q K^T) hi and lo, at 0; then W, then P

template <int D>
struct Pr {
  static constexpr int kHalves = D / 64;
  static constexpr int kKQ = kHalves * 2 * kSpan;       // per half: K rows, then Q rows
  static constexpr int kAOff = kKQ;                     // A, then T; then T hi, lo (for W)
  // T hi, lo (for P) over Q, whose products are done by then.  On their way out: W hi over K, W lo
  // over T's terms for W, P over T's terms for P
  static constexpr int kTHi = kSpan, kTLo = D == 128 ? 3 * kSpan : kAOff + kChunk * kLd * 4;
  static constexpr int kXOff = kAOff + kChunk * kLd * 4 + (D == 128 ? 0 : kSpan);
  static constexpr int kGateOff = kXOff + 32 * kLdX * 4;   // alpha, beta, G_Ci, products from token 33 on
  static constexpr int kBarOff = kGateOff + 4 * kChunk * 4;
  static constexpr int kSmem = kBarOff + 64 + 1024;
  static_assert(kChunk * kLd * 4 % 1024 == 0 && kChunk * kLd * 4 >= 2 * kSpan, "T's terms over A");
};

// d += L R over k0 <= k < k1 for a 16 x 8 product (L: 16 rows of pitch ldl, R: rows k of pitch ldr), by
// one warp: lane 4 g + t holds rows g, g + 8 and columns 2 t, 2 t + 1.  Operands are too small for the
// tcgen05 forms' 128 rows.  Three tf32 products of two terms each (the first holds the top 11 bits,
// the second the rest, of which the product takes 11; low times low, 2^-22, is left out): as good as
// fp32, and a third of the shared-memory reads of fp32 products from registers, which bounded the kernel.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], const float (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                 "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}
__device__ __forceinline__ float top11(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }
__device__ __forceinline__ void block_product(const float* L, int ldl, const float* R, int ldr, int k0, int k1, int lane,
                                              float (&d)[4]) {
  const float* l = L + (lane >> 2) * ldl + (lane & 3);
  const float* r = R + (lane & 3) * ldr + (lane >> 2);
#pragma unroll 2
  for (int k = k0; k < k1; k += 8) {
    const float a[4] = {l[k], l[8 * ldl + k], l[k + 4], l[8 * ldl + k + 4]};
    const float b[2] = {r[k * ldr], r[(k + 4) * ldr]};
    float ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) { ah[e] = top11(a[e]); al[e] = a[e] - ah[e]; }
#pragma unroll
    for (int e = 0; e < 2; ++e) { bh[e] = top11(b[e]); bl[e] = b[e] - bh[e]; }
    mma_tf32(d, al, bh);
    mma_tf32(d, ah, bl);
    mma_tf32(d, ah, bh);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsPr, 4)
    gdn_chunk_prepare_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                             const ChunkArgs args) {
  using C = Pr<D>;
  using I = Image<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const GdnUpdateArgs& a = args.a;
  const uint64_t wait_ns = args.wait_ns;
  const int t = threadIdx.x, w = t >> 5, lane = t & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t KQ_FULL = sbase + C::kBarOff, P_DONE = KQ_FULL + 8, DRAIN = KQ_FULL + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 28);

  // The first segment waits for what stands before the call.  A later one needs nothing of the walk that
  // is still at work on the segment before it - the call's inputs are final, and its images go to
  // the other half of the workspace, last read by the walk before that one, which this one has waited for - so it
  // starts beside it, on what that leaves free; but the grid ends after that walk, because the next
  // one, which waits for this grid alone, continues its state: the last CTA sees to that.
  const bool early = args.chunk0 != 0, last_cta = early && blockIdx.x == gridDim.x - 1;
  if (!early) pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x % a.H, bc = blockIdx.x / a.H;
  const int b = bc / args.span, c = args.chunk0 + bc % args.span;
  const int t0 = __ldg(a.cu + b), n = __ldg(a.cu + b + 1) - t0;
  if (!sequence_ok(a, t0, n) || c * kChunk >= n) {   // the state kernel reports bad bounds
    if (last_cta) pdl_wait();
    return;
  }
  const int cnt = min(kChunk, n - c * kChunk);

  if (w == 0) {   // the copies start before anything else
    if (lane == 0) {
      mbar_init(KQ_FULL, 1);
      mbar_init(P_DONE, 1);
      mbar_init(DRAIN, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    int z = t0 + c * kChunk;
    if (!TVA_CHECK(z >= 0 && z < a.token_capacity, a.status)) z = 0;
    mbar_expect_tx_elect(KQ_FULL, (uint32_t)C::kKQ);
    for (int hf = 0; hf < C::kHalves; ++hf) {
      tma_load_3d_elect(sbase + hf * 2 * kSpan, &tm_k, 64 * hf, h, z, KQ_FULL);
      tma_load_3d_elect(sbase + hf * 2 * kSpan + kSpan, &tm_q, 64 * hf, h, z, KQ_FULL);
    }
  }
  float* As = reinterpret_cast<float*>(smem + C::kAOff);
  float* Xs = reinterpret_cast<float*>(smem + C::kXOff);
  float* al_s = reinterpret_cast<float*>(smem + C::kGateOff);   // alpha
  float* be_s = al_s + kChunk;                                  // beta
  float* en_s = be_s + kChunk;                                  // G_Ci
  float* mid_s = en_s + kChunk;                                 // product of alpha over tokens 33 .. i
  // gates (rows past the sequence's end: no decay, nothing written)
  float al = 1.f, be = 0.f;
  if (t < cnt) {
    const size_t at = (size_t)(t0 + c * kChunk + t) * a.H + h;
    al = __ldg(a.alpha + at);
    be = __ldg(a.beta + at);
  }
  if (t < kChunk) {
    al_s[t] = al;
    be_s[t] = be;
  }
  if (w == 1) {
    tmem_alloc(smem_u32(tmem_slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half = t >> 7;
  const uint32_t lane_base = (uint32_t)((w & 3) * 32) << 16;
  constexpr uint32_t idesc_a = idesc_bf16(128, 64, false);                 // [K; Q] K^T: both K-major
  constexpr uint32_t idesc_w = idesc_bf16(128, 64, true) | (1u << 15);     // K^T T: A along M, B along N
  constexpr uint32_t idesc_p = idesc_bf16(128, 64, true);                  // A in TMEM
  const uint32_t desc_hi = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);     // the LBO field is in the low word
  // products of the decays from the chunk's start and to its end: 64 threads, a scan each way
  float pre = al;
  if (t < 64) {
    float suf = t < 63 ? al_s[t + 1] : 1.f, mid = lane == 0 ? 1.f : al;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, pre, o), y = __shfl_down_sync(0xffffffffu, suf, o);
      const float z = __shfl_up_sync(0xffffffffu, mid, o);
      if (lane >= o) { pre *= x; mid *= z; }
      if (lane + o < 32) suf *= y;
    }
    mid_s[t] = t < 32 ? 1.f : mid;
    // across the two warps: the other one's 32 factors, multiplied by every lane's share
    float other = t < 32 ? al_s[32 + lane] : al_s[lane];
    if (t < 32 && lane == 0) other = 1.f;   // al_s[32] is already in warp 0's suffixes
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) other *= __shfl_xor_sync(0xffffffffu, other, o);
    if (t < 32) suf *= other;
    else pre *= other;
    en_s[t] = suf;
  }
  bool ok = mbar_wait(KQ_FULL, 0, abort_flag, wait_ns);
  if (cnt < kChunk) {
    // rows of K and Q past the end belong to other sequences or to none: zeros instead
    for (int e = t; e < C::kHalves * 2 * 8 * (kChunk - cnt); e += kThreadsPr) {
      const int r = cnt + (e >> 3) % (kChunk - cnt), part = (e >> 3) / (kChunk - cnt);
      *reinterpret_cast<uint4*>(smem + part * kSpan + r * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  ok = all_threads(ok);
  if (ok && w == 0) {
    tc_fence_after();
    const uint32_t lo = (uint32_t)sdesc_sw128(sbase, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t o = (uint32_t)((ks >> 2) * 2 * kSpan + (ks & 3) * 32) >> 4;
      mma_ss_elect(tmem, desc_join(lo + o, desc_hi), desc_join(lo + o, desc_hi), idesc_a, ks > 0);
    }
    tc_commit_elect(P_DONE);
  }
  const int row = t & 63;   // this lane's token row (of K for lanes below 64, of Q above)
  const bool qrow = (t & 64) != 0;
  if (ok) ok = mbar_wait(P_DONE, 0, abort_flag, wait_ns);
  tc_fence_after();
  {
    // this thread's half of row `row` of beta_i G_ij k_i.k_j (j < i), or of G_ij q_i.k_j (j <= i)
    uint32_t d[32];
    tmem_ld32(tmem + lane_base + 32 * half, d);
    const int j0 = 32 * half, last = qrow ? row : row - 1;
    // G_row,31 but for alpha of token 32, which the walk below multiplies in, where the walk starts there
    float p = (qrow ? 1.f : be_s[row]) * (half == 0 ? mid_s[row] : 1.f);
    tmem_wait_ld32(d);
#pragma unroll
    for (int j4 = 28; j4 >= 0; j4 -= 4) {
      const float4 a4 = *reinterpret_cast<const float4*>(al_s + j0 + j4);
      const float next = al_s[min(j0 + j4 + 4, kChunk - 1)];
      const float f[4] = {a4.y, a4.z, a4.w, next};   // alpha of token j + 1 (never used past token 63)
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        const int j = j0 + j4 + e;
        if (j < row) p *= f[e];
        d[j4 + e] = j <= last ? __float_as_uint(__uint_as_float(d[j4 + e]) * p) : 0u;
      }
    }
    uint32_t lo[16];
    if (!qrow) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4*>(As + row * kLd + j0 + j) = make_uint4(d[j], d[j + 1], d[j + 2], d[j + 3]);
#pragma unroll
      for (int j = 0; j < 16; ++j) d[j] = lo[j] = 0u;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        split2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]), d[j], lo[j]);
    }
    tc_fence_before();
    __syncthreads();   // every column is read
    tc_fence_after();
    tmem_st16(tmem + lane_base + 16 * half, d);   // lower(G o Q K^T) in lanes 64 .. 127, zeros above: hi
    tmem_st16(tmem + lane_base + 32 + 16 * half, lo);
    tmem_wait_st();
    tc_fence_before();
  }
  // ---- T = (I + A)^-1: 16-row diagonal blocks by substitution (a column per lane), then the
  // blocks below them, T21 = -T22 (A21 T11), at 16 and at 32 rows
  if (w < 4) {
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
  __syncthreads();
  const int gq = lane >> 2, tq = 2 * (lane & 3);   // this lane's first row and columns of a 16 x 8 product
  {
    const int o = 32 * ((w >> 1) & 1), n0 = 8 * (w & 1);   // two blocks of 32 rows; columns of their 16
    float* Xb = Xs + ((w >> 1) & 1) * 16 * kLdX + n0;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    if (w < 4) {
      block_product(As + (o + 16) * kLd + o, kLd, As + o * kLd + o + n0, kLd, 0, 16, lane, d);   // A21 T11
      *reinterpret_cast<float2*>(Xb + gq * kLdX + tq) = make_float2(d[0], d[1]);
      *reinterpret_cast<float2*>(Xb + (gq + 8) * kLdX + tq) = make_float2(d[2], d[3]);
    }
    __syncthreads();
    if (w < 4) {
      d[0] = d[1] = d[2] = d[3] = 0.f;
      block_product(As + (o + 16) * kLd + o + 16, kLd, Xb, kLdX, 0, 16, lane, d);
      float* T21 = As + (o + 16 + gq) * kLd + o + n0 + tq;
      *reinterpret_cast<float2*>(T21) = make_float2(-d[0], -d[1]);
      *reinterpret_cast<float2*>(T21 + 8 * kLd) = make_float2(-d[2], -d[3]);
    }
  }
  __syncthreads();
  {
    // 32 x 32 x 32: warp w takes 16 rows and 8 columns; T11 has nothing above, T22 nothing right of, its
    // diagonal
    const int m0 = 16 * (w & 1), n0 = 8 * (w >> 1);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    block_product(As + (32 + m0) * kLd, kLd, As + n0, kLd, n0, 32, lane, d);   // A21 T11
    float* X = Xs + (m0 + gq) * kLdX + n0 + tq;
    *reinterpret_cast<float2*>(X) = make_float2(d[0], d[1]);
    *reinterpret_cast<float2*>(X + 8 * kLdX) = make_float2(d[2], d[3]);
    __syncthreads();
    d[0] = d[1] = d[2] = d[3] = 0.f;
    block_product(As + (32 + m0) * kLd + 32, kLd, Xs + n0, kLdX, 0, m0 + 16, lane, d);   // -T22 (A21 T11)
    float* T21 = As + (32 + m0 + gq) * kLd + n0 + tq;
    *reinterpret_cast<float2*>(T21) = make_float2(-d[0], -d[1]);
    *reinterpret_cast<float2*>(T21 + 8 * kLd) = make_float2(-d[2], -d[3]);
  }
  __syncthreads();
  {
    // T diag(beta) (for P) and diag(G_Ci) T diag(beta) (for W, over A's place), two terms each:
    // row i is the products' k = i, its columns lie along N
    const int i = t & 63, j0 = 16 * (t >> 6);
    const float en = en_s[i];
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(As + i * kLd + j0 + j);
      const float4 bb = *reinterpret_cast<const float4*>(be_s + j0 + j);
      x[j] = v.x * bb.x; x[j + 1] = v.y * bb.y; x[j + 2] = v.z * bb.z; x[j + 3] = v.w * bb.w;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t hi[4], lo[4];
      const int at = i * 128 + (((j0 >> 3) + q) ^ (i & 7)) * 16;
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], lo[e]);
      *reinterpret_cast<uint4*>(smem + C::kTHi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(smem + C::kTLo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[8 * q + 2 * e] * en, x[8 * q + 2 * e + 1] * en, hi[e], lo[e]);
      *reinterpret_cast<uint4*>(smem + C::kAOff + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(smem + C::kAOff + kSpan + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_async_shared();
  }
  ok = all_threads(ok);
  if (ok && w == 0) {
    tc_fence_after();
    // rows 64 .. 127 of K^T: the second half (d = 64: Q's, whose products are not read)
    const uint32_t klo = (uint32_t)sdesc_sw128(sbase, D == 128 ? 2 * kSpan : kSpan, 1024);
    const uint32_t wlo = (uint32_t)sdesc_sw128(sbase + C::kAOff, 16, 1024);
#pragma unroll
    for (int part = 0; part < 2; ++part)   // hi and lo terms
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss_elect(tmem + kTmWork, desc_join(klo + (ks * 2048 >> 4), desc_hi),
                     desc_join(wlo + ((part * kSpan + ks * 2048) >> 4), desc_hi), idesc_w, part > 0 || ks > 0);
    tc_commit_elect(P_DONE);
  }
  if (ok) ok = mbar_wait(P_DONE, 1, abort_flag, wait_ns);
  tc_fence_after();
  uint32_t d[32];
  tmem_ld32(tmem + kTmWork + lane_base + 32 * half, d);
  tmem_wait_ld32(d);
  tc_fence_before();
  ok = all_threads(ok);
  if (ok && w == 0) {   // P while W is written out
    tc_fence_after();
    const uint32_t plo = (uint32_t)sdesc_sw128(sbase, 16, 1024);
#pragma unroll
    for (int part = 0; part < 3; ++part)   // hi hi, hi lo, lo hi
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ts_elect(tmem + kTmWork, tmem + (part == 2 ? 32 : 0) + ks * 8,
                     desc_join(plo + (((part == 1 ? C::kTLo : C::kTHi) + ks * 2048) >> 4), desc_hi), idesc_p, part > 0 || ks > 0);
    tc_commit_elect(P_DONE);
  }
  // this thread's 32 tokens of a row in two terms
  auto write_row = [&](uint8_t* hi_row, uint8_t* lo_row, int r) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split2(__uint_as_float(d[8 * q + 2 * e]), __uint_as_float(d[8 * q + 2 * e + 1]), hi[e], lo[e]);
      const int at = ((4 * half + q) ^ (r & 7)) * 16;
      *reinterpret_cast<uint4*>(hi_row + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(lo_row + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  const int r128 = t & 127;
  if (r128 < D) write_row(smem + (r128 < 64 ? 0 : 2 * kSpan) + row * 128, smem + C::kAOff + r128 * 128, r128);
  if (t < kChunk) al_s[t] = pre;
  if (ok) ok = mbar_wait(P_DONE, 0, abort_flag, wait_ns);
  tc_fence_after();
  if (qrow) {   // P is in lanes 64 .. 127
    tmem_ld32(tmem + kTmWork + lane_base + 32 * half, d);
    tmem_wait_ld32(d);
    write_row(smem + C::kTHi + row * 128, smem + C::kTLo + row * 128, row);
  }
  fence_async_shared();
  tc_fence_before();
  ok = all_threads(ok);
  if (!ok && w == 0) {   // a wait ran out: what is in flight lands before the CTA ends
    tc_commit_elect(DRAIN);
    drain_wait(DRAIN, 0);
    drain_wait(KQ_FULL, 0);
    if (t == 0) set_status(a.status, kStatusTimeout);
  }
  if (!ok) __syncthreads();   // uniform over the CTA
  if (ok && t == 0) {
    uint8_t* image = args.images + (((size_t)b * args.segment + (c - args.chunk0)) * a.H + h) * I::kBytes;
    for (int hf = 0; hf < C::kHalves; ++hf) bulk_store(image + hf * kSpan, sbase + hf * 2 * kSpan, kSpan);
    bulk_store(image + I::kW, sbase + C::kAOff, I::kW);
    bulk_store(image + I::kP, sbase + C::kTHi, kSpan);
    bulk_store(image + I::kP + kSpan, sbase + C::kTLo, kSpan);
    bulk_store(image + I::kG, sbase + C::kGateOff, kChunk * 4);
    bulk_stores_done();
  }
  if (w == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
  if (last_cta) pdl_wait();
}

// ------------------------------------------------------------------ the walk from state to state

constexpr uint32_t kTmX = 0, kTmD = 64, kTmO = 128;   // TMEM columns: X, W r, P r

// NS columns of d_v per CTA, 16 per thread.  With 64 columns S and r are two tiles, of the hi and the lo
// terms (rows of 64 columns).  With 32 a row of one tile holds both, so that one product of N = 64 does for
// both (an MMA of N = 32 takes as long: reading its A operand bounds it) and their sums are added after.
template <int D, int NS>
struct St {
  static constexpr bool kPair = NS == 32;
  static constexpr int kHolders = 8 * NS;   // threads that hold the state
  static constexpr int kProducer = kHolders / 32, kMma = kProducer + 1, kThreads = kHolders + 64;
  static constexpr int kHalves = D / 64;
  static constexpr int kKQ = kHalves * 2 * kSpan;
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kStage = (kKQ + Image<D>::kBytes + 1023) / 1024 * 1024;
  static constexpr int kSOff = kStages * kStage;                      // S: [D rows of d_k]
  static constexpr int kROff = kSOff + (kPair ? 1 : 2) * D * 128;     // r: [64 tokens]
  static constexpr int kBarOff = kROff + (kPair ? 1 : 2) * kSpan;
  static constexpr int kSmem = kBarOff + 128 + 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

template <int D, int NS>
__global__ void __launch_bounds__(St<D, NS>::kThreads, 1)
    gdn_chunk_state_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const ChunkArgs args) {
  using C = St<D, NS>;
  using I = Image<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const GdnUpdateArgs& a = args.a;
  const uint64_t wait_ns = args.wait_ns;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t FULL = bars, EMPTY = bars + 24, X_DONE = bars + 48, D_DONE = bars + 56, O_DONE = bars + 64,
                 DRAIN = bars + 72, S_READY = bars + 80, R_READY = bars + 88;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 96);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 100);

  if (tid == C::kProducer * 32) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(FULL + 8 * s, 1);
      mbar_init(EMPTY + 8 * s, 1);
    }
    mbar_init(X_DONE, 1);
    mbar_init(D_DONE, 1);
    mbar_init(O_DONE, 1);
    mbar_init(DRAIN, 1);
    mbar_init(S_READY, C::kHolders);
    mbar_init(R_READY, C::kHolders);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  constexpr int CS = D / NS;
  const int cs = blockIdx.x % CS, bh = blockIdx.x / CS;
  const int b = bh / a.H, h = bh % a.H;
  const int t0 = __ldg(a.cu + b);
  const int n = __ldg(a.cu + b + 1) - t0;
  if (!sequence_ok(a, t0, n)) {
    if (tid == 0) set_status(a.status, kStatusInvalidArg);
    return;   // uniform over the CTA
  }
  const int chunks = min(args.span, (n + kChunk - 1) / kChunk - args.chunk0);   // in this segment
  if (chunks <= 0) return;
  const int first = args.chunk0 * kChunk;   // the segment's first token
  if (warp == C::kProducer) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::kProducer) {
    // ------------------------------------------------------------------ producer
    bool ok = true;
    int c = 0;
    const uint8_t* image = args.images + ((size_t)b * args.segment * a.H + h) * I::kBytes;
    for (; c < chunks; ++c) {
      const int st = c % C::kStages, use = c / C::kStages;
      if (use > 0 && !(ok = warp_wait(EMPTY + 8 * st, (use - 1) & 1, abort_flag, wait_ns))) break;
      int z = t0 + first + c * kChunk;
      if (!TVA_CHECK(z >= 0 && z < a.token_capacity, a.status)) z = 0;
      const uint32_t at = sbase + st * C::kStage;
      mbar_expect_tx_elect(FULL + 8 * st, (uint32_t)(C::kKQ + I::kBytes));
      for (int hf = 0; hf < C::kHalves; ++hf) {
        tma_load_3d_elect(at + hf * 2 * kSpan, &tm_k, 64 * hf, h, z, FULL + 8 * st);
        tma_load_3d_elect(at + hf * 2 * kSpan + kSpan, &tm_q, 64 * hf, h, z, FULL + 8 * st);
      }
      bulk_load_elect(at + C::kKQ, image + (size_t)c * a.H * I::kBytes, I::kBytes, FULL + 8 * st);
    }
    for (int i = max(0, c - C::kStages); i < c; ++i)   // every copy has landed before the CTA ends
      drain_wait(FULL + 8 * (i % C::kStages), (i / C::kStages) & 1);
  } else if (warp == C::kMma) {
    // ------------------------------------------------------------------ MMA issuer
    // A converged warp of its own: issued from one of the state's warps, between its barriers, an MMA
    // took 55 to 100 clocks to issue instead of about as long as it runs.
    constexpr uint32_t idesc = idesc_bf16(128, 64, true);   // A K-major, B along N
    const uint32_t hi_word = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    const uint32_t s_lo = (uint32_t)sdesc_sw128(sbase + C::kSOff, 16, 1024);
    const uint32_t r_lo = (uint32_t)sdesc_sw128(sbase + C::kROff, 16, 1024);
    const uint32_t st_lo = (uint32_t)sdesc_sw128(sbase, 16, 1024);
    // W (or P) r, W and r in two terms each: hi hi, hi lo, lo hi. A pair's other columns take lo lo with the
    // last: the same time as half its columns alone, and the state a seventh nearer (6.1e-6 to 5.2e-6 off).
    auto issue_r = [&](uint32_t d_tmem, uint32_t a_lo, int a_bytes) {
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        if (C::kPair && part == 1) continue;   // in the first product's other columns
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss_elect(d_tmem, desc_join(a_lo + (uint32_t)(((part == 2 ? a_bytes : 0) + ks * 32) >> 4), hi_word),
                       desc_join(r_lo + (uint32_t)(((part == 1 ? kSpan : 0) + ks * 2048) >> 4), hi_word),
                       idesc, part > 0 || ks > 0);
      }
    };
    // Test hook: DRAIN's phase completes only through this warp's own commit below.
    bool ok = !(args.stall && !warp_wait(DRAIN, 0, abort_flag, wait_ns));
    for (int c = 0; ok && c < chunks; ++c) {
      const int st = c % C::kStages;
      const uint32_t stage = st_lo + (uint32_t)(st * C::kStage >> 4);
      if (!(ok = warp_wait(FULL + 8 * st, (c / C::kStages) & 1, abort_flag, wait_ns))) break;
      if (!(ok = warp_wait(S_READY, c & 1, abort_flag, wait_ns))) break;
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < (C::kPair ? 1 : 2); ++part)   // S hi, S lo
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (uint32_t)((ks >> 2) * 2 * kSpan + (ks & 3) * 32) >> 4;
          mma_ss_elect(tmem + kTmX, desc_join(stage + o, hi_word),
                       desc_join(s_lo + (uint32_t)((part * D * 128 + ks * 2048) >> 4), hi_word), idesc,
                       part > 0 || ks > 0);
        }
      tc_commit_elect(X_DONE);
      if (!(ok = warp_wait(R_READY, c & 1, abort_flag, wait_ns))) break;
      tc_fence_after();
      const uint32_t w_lo = stage + (C::kKQ >> 4);
      issue_r(tmem + kTmD, w_lo, I::kW);
      tc_commit_elect(D_DONE);
      // P stands in rows 64 .. 127 of its operand; the bytes before it make rows that are not read
      issue_r(tmem + kTmO, w_lo + ((I::kP - kSpan) >> 4), kSpan);
      tc_commit_elect(O_DONE);
      tc_commit_elect(EMPTY + 8 * st);
    }
    tc_commit_elect(DRAIN);
    drain_wait(DRAIN, 0);
  } else {
    // ------------------------------------------------------------------ the state's holders
    // No barrier among them: what a thread reads of TMEM or writes to shared memory is ordered by the
    // products' own barriers.  X is issued when all have staged S (S_READY), so have read the
    // last X and W r; P r is overwritten once all have staged r (R_READY), so have read it.
    const int wg = warp >> 2, r128 = tid & 127;   // columns 16 wg .. of the slice; row of d_k and TMEM lane
    const uint32_t lane_base = ((uint32_t)((warp & 3) * 32) << 16) + 16 * wg;
    const bool krow = r128 < 64;
    const int row = r128 & 63;
    const size_t hs = (size_t)a.H * D;
    const int col = cs * NS + 16 * wg;
    float* Sg = a.state + (((size_t)b * a.H + h) * D + (r128 < D ? r128 : 0)) * D + col;
    uint64_t S2[8];   // this row's 16 columns, in pairs
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = r128 < D ? __ldcg(reinterpret_cast<const float4*>(Sg + 4 * q)) : make_float4(0.f, 0.f, 0.f, 0.f);
      S2[2 * q] = f2_pack(v.x, v.y);
      S2[2 * q + 1] = f2_pack(v.z, v.w);
    }
    const __nv_bfloat16* Vg = static_cast<const __nv_bfloat16*>(a.v) + (size_t)(t0 + first) * hs + (size_t)h * D + col;
    __nv_bfloat16* Og = static_cast<__nv_bfloat16*>(a.out) + (size_t)(t0 + first) * hs + (size_t)h * D + col;
    const int left = n - first;   // tokens from the segment's first one on
    uint4 vr[2];
    auto fetch_v = [&](int c) {   // this lane's row of chunk c's V (K lanes)
      if (krow && c < chunks && c * kChunk + row < left) {
        const uint4* src = reinterpret_cast<const uint4*>(Vg + (size_t)(c * kChunk + row) * hs);
        vr[0] = __ldg(src);
        vr[1] = __ldg(src + 1);
      }
    };
    // 16 columns of a row in two terms: the row is the products' k, its columns lie along N
    auto stage_row = [&](int off, int lo_off, int r, const uint64_t* x2) {
      uint8_t* at = smem + off + r * 128;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x2[4 * q + e], hi[e], lo[e]);
        const int ch = 2 * wg + q;
        *reinterpret_cast<uint4*>(at + ((ch ^ (r & 7)) * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + (C::kPair ? ((ch + 4) ^ (r & 7)) * 16 : lo_off + ((ch ^ (r & 7)) * 16))) =
            make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_shared();
    };
    // 16 columns of a product (the two halves' sum where S or r stood side by side), in pairs
    auto load = [&](uint32_t tm, uint64_t* x2) {
      uint32_t x[16];
      tmem_ld16(tmem + tm + lane_base, x);
      if constexpr (C::kPair) {
        uint32_t y[16];
        tmem_ld16(tmem + tm + 32 + lane_base, y);
        tmem_wait_ld16(x);
        tie16(y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x2[j] = f2_add(f2_pack(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                         f2_pack(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])));
      } else {
        tmem_wait_ld16(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x2[j] = f2_pack(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
      }
    };
    fetch_v(0);
    if (r128 < D) stage_row(C::kSOff, D * 128, r128, S2);
    bool ok = true;
    tc_fence_before();
    mbar_arrive(S_READY);
    uint64_t oq[8];   // Q lanes: g_i S^T q_i
    auto write_out = [&](int c) {   // the chunk's outputs: its P r added
      uint64_t x2[8];
      load(kTmO, x2);
      if (krow || c * kChunk + row >= left) return;
      uint4* dst = reinterpret_cast<uint4*>(Og + (size_t)(c * kChunk + row) * hs);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          f2_unpack(f2_add(oq[4 * q + e], x2[4 * q + e]), lo, hi);
          w[e] = pack_bf16x2(lo, hi);
        }
        dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int st = c % C::kStages;
      if (c > 0) {   // the last chunk's outputs, while X is computed
        ok = __all_sync(0xffffffffu, mbar_wait(O_DONE, (c - 1) & 1, abort_flag, wait_ns));
        if (!ok) break;
        tc_fence_after();
        write_out(c - 1);
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, mbar_wait(FULL + 8 * st, (c / C::kStages) & 1, abort_flag, wait_ns));
      if (!ok) break;
      const float* ga_s = reinterpret_cast<const float*>(smem + st * C::kStage + C::kKQ + I::kG);
      const float ga = ga_s[row], gc = ga_s[kChunk - 1];
      ok = __all_sync(0xffffffffu, mbar_wait(X_DONE, c & 1, abort_flag, wait_ns));
      if (!ok) break;
      tc_fence_after();
      uint64_t x2[8];
      load(kTmX, x2);
      if (krow) {   // uniform over the warp
        const uint64_t g2 = f2_pack(-ga, -ga);
        const uint32_t vw[8] = {vr[0].x, vr[0].y, vr[0].z, vr[0].w, vr[1].x, vr[1].y, vr[1].z, vr[1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x2[j] = f2_fma(g2, x2[j], f2_pack(bf16_lo(vw[j]), bf16_hi(vw[j])));
        if (c * kChunk + row >= left) {   // past the end: K holds other rows there
#pragma unroll
          for (int j = 0; j < 8; ++j) x2[j] = 0;
        }
        stage_row(C::kROff, kSpan, row, x2);
      } else {
        const uint64_t g2 = f2_pack(ga, ga);
#pragma unroll
        for (int j = 0; j < 8; ++j) oq[j] = f2_mul(g2, x2[j]);
      }
      tc_fence_before();
      mbar_arrive(R_READY);
      fetch_v(c + 1);
      ok = __all_sync(0xffffffffu, mbar_wait(D_DONE, c & 1, abort_flag, wait_ns));
      if (!ok) break;
      tc_fence_after();
      load(kTmD, x2);
      const uint64_t gc2 = f2_pack(gc, gc);
#pragma unroll
      for (int j = 0; j < 8; ++j) S2[j] = f2_fma(gc2, S2[j], x2[j]);
      if (r128 < D) stage_row(C::kSOff, D * 128, r128, S2);
      tc_fence_before();
      if (c + 1 < chunks) mbar_arrive(S_READY);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(O_DONE, (chunks - 1) & 1, abort_flag, wait_ns));
    if (ok && __all_sync(0xffffffffu, !*abort_flag)) {
      tc_fence_after();
      write_out(chunks - 1);
      if (r128 < D) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4 v;
          f2_unpack(S2[2 * q], v.x, v.y);
          f2_unpack(S2[2 * q + 1], v.z, v.w);
          *reinterpret_cast<float4*>(Sg + 4 * q) = v;
        }
      }
    }
  }
  // ------------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(a.status, kStatusTimeout);
  if (warp == C::kProducer) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Chunks of each sequence per pair of launches: all of them when that takes no more than kSlots
// images (0.4 GB at d = 128), else as many as that allows, but at least 8 (32768 tokens of 32 heads:
// segments of 32, 64, 128 and 256 chunks 1086, 1016, 984 and 987 us; without the overlap of a segment's preparation
// and the walk before it 1201, 1123, 1070 and 1045).
constexpr int kSms = 152;
constexpr long long kSlots = 8192;
int segment_chunks(int B, int H, int max_tokens) {
  const int all = (max_tokens + kChunk - 1) / kChunk;
  return (int)std::min<long long>(all, std::max<long long>(8, kSlots / ((long long)B * H)));
}

template <int D, int NS>
cudaError_t launch_state(const ChunkArgs& ca, const CUtensorMap& mq, const CUtensorMap& mk, cudaStream_t s) {
  using C = St<D, NS>;
  const cudaError_t e = check_cuda(
      cudaFuncSetAttribute(gdn_chunk_state_kernel<D, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem),
      "cudaFuncSetAttribute(gdn_chunk_state_kernel)");
  if (e != cudaSuccess) return e;
  return check_cuda(launch_pdl(gdn_chunk_state_kernel<D, NS>, dim3((unsigned)((long long)ca.a.B * ca.a.H * (D / NS))),
                               dim3(C::kThreads), (size_t)C::kSmem, s, mq, mk, ca),
                    "launch gdn_chunk_state_kernel");
}

template <int D>
cudaError_t launch_chunk_typed(const GdnUpdateArgs& a, void* workspace, cudaStream_t s) {
  CUtensorMap mq, mk;
  if (!make_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, D, a.H, a.token_capacity, 1, kChunk) ||
      !make_map(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k, D, a.H, a.token_capacity, 1, kChunk))
    return cudaErrorInvalidValue;
  cudaError_t e = check_cuda(cudaFuncSetAttribute(gdn_chunk_prepare_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  Pr<D>::kSmem),
                             "cudaFuncSetAttribute(gdn_chunk_prepare_kernel)");
  if (e != cudaSuccess) return e;
  const int all = (a.max_tokens + kChunk - 1) / kChunk, segment = segment_chunks(a.B, a.H, a.max_tokens);
  // A chunk takes a CTA of 32 columns less time than one of 64, but not half of it: 32 columns while
  // every CTA then has an SM of its own (32 heads, d = 128, 32 / 64 columns: 1 prompt of 2048 tokens 75 / 93 us, 2 of
  // 1024 78 / 63, 8 266 / 234; d = 64, 1 of 2048 61 / 79, 3 of 1024 79 / 64).
  const bool narrow = (long long)a.B * a.H * (D / 32) <= kSms;
  ChunkArgs ca{a, nullptr, 0, 0, segment, 0, 0};
  tc_wait_settings(&ca.wait_ns, &ca.stall);
  const size_t half = (size_t)a.B * a.H * segment * Image<D>::kBytes;   // segments take the halves in turn
  for (int c0 = 0, i = 0; c0 < all; c0 += segment, ++i) {
    ca.images = static_cast<uint8_t*>(workspace) + (i & 1) * half;
    ca.chunk0 = c0;
    ca.span = std::min(segment, all - c0);
    e = check_cuda(launch_pdl(gdn_chunk_prepare_kernel<D>, dim3((unsigned)((long long)a.B * a.H * ca.span)),
                              dim3(kThreadsPr), (size_t)Pr<D>::kSmem, s, mq, mk, ca),
                   "launch gdn_chunk_prepare_kernel");
    if (e != cudaSuccess) return e;
    e = narrow ? launch_state<D, 32>(ca, mq, mk, s) : launch_state<D, 64>(ca, mq, mk, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t gdn_chunk_workspace(int B, int H, int d, int max_tokens) {
  const int segment = segment_chunks(B, H, max_tokens);
  return (size_t)B * H * segment * (segment * kChunk < max_tokens ? 2 : 1) * (d == 64 ? Image<64>::kBytes : Image<128>::kBytes);
}

cudaError_t launch_gdn_chunk(const GdnUpdateArgs& a, void* workspace, cudaStream_t s) {
  return a.d == 64 ? launch_chunk_typed<64>(a, workspace, s) : launch_chunk_typed<128>(a, workspace, s);
}

}  // namespace tva
