// k_gdn_update.cu - the Gated DeltaNet recurrence token by token: a sequence's tokens
// (gdn_update_varlen) or the accepted path of a draft tree (commit_accepted_gdn), with the
// state updated in place.
//
//     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t
//
// ("DFlash-TfM", Method 3, the update that its tree verification defers).  With x = S_{t-1}^T k_t
// and w = beta_t (v_t - alpha_t x) a step is S_t = alpha_t S_{t-1} + k_t w^T and
// o_t = alpha_t S_{t-1}^T q_t + (q_t . k_t) w, so both products read the state before the step
// and their sums over the key rows are taken together.  Columns of S (of d_v) never meet.
//
// A block of two warps takes 32 columns of one head's state (16 with sixteen row groups).  A warp's columns
// x D rows stay in its registers from the first token to the last: lane = 4 rg + c4 holds columns 4 c4 ..
// 4 c4 + 3 of the rows 32 i + 4 rg + e (e < 4), packed in pairs of rows (e, e + 1), so that a 16-byte read
// of k or q from shared memory is two such pairs and the products and the update run on packed fp32
// pairs.  The eight row groups are summed by a butterfly of shuffles.  (With sixteen: lane = 2 rg + c4, rows
// 64 i + 4 rg + e.)  Tokens are staged kTile at a time; the next tile's rows are on their way from memory
// while the current one is computed.  All arithmetic is fp32 (bf16 rows are widened as they are staged, the
// output rounded once).
//
// Few tokens are bound by the state's traffic: it is read and written once, with streaming hints (64
// sequences of 32 heads, d = 128, 272 MB: one token 41.9 us, 6.5 TB/s, without the hints 45.9; the commit of
// 64 paths of 0 to 8 nodes 46.3 and 52.1 us, and 57.6 without a bound on the registers that lets eight
// blocks share a SM).  Many tokens are bound by the chain from token to token: the products and the update
// (136 packed multiply-adds of two clocks each, on the one scheduler that a warp has), three shuffles, the
// correction; some 310 clocks (777 tokens of single precision 125 us, with sixteen row groups 104).  Tried
// and not kept: the state scaled lazily by the product of the decays (one multiply-add an element instead of
// two, but a division a token: no shorter), the outputs' sums behind the update.
#include <cuda_bf16.h>

#include <type_traits>

#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

using namespace ptx;

constexpr int kThreadsUp = 64;
constexpr int kTile = 8;     // tokens staged together

__device__ __forceinline__ float4 up_load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 up_load4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void up_store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void up_store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// kPath: the tokens are the nodes of an accepted path and there is no output.  RG: row groups, 8 or 16.
template <int D, typename T, bool kPath, int RG>
__global__ void __launch_bounds__(kThreadsUp, kPath ? 8 : 6) gdn_recurrent_kernel(GdnUpdateArgs a) {
  constexpr int C4 = 32 / RG;          // lanes side by side
  constexpr int kColsUp = 8 * C4;      // columns of d_v per block, half of them per warp
  constexpr int CS = D / kColsUp;      // blocks per (sequence, head)
  constexpr int NI = D / (4 * RG);     // row quadruples per lane
  constexpr bool kOut = !kPath;
  __shared__ __align__(16) float sk[2][kTile][D];
  __shared__ __align__(16) float sq[2][kOut ? kTile : 1][D];
  __shared__ __align__(16) float sv[2][kTile][kColsUp];
  __shared__ float s_alpha[2][kTile], s_beta[2][kTile];
  __shared__ int s_path[kPath ? kMaxNodes : 1];

  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = blockIdx.x % CS, bh = blockIdx.x / CS;
  const int b = bh / a.H, h = bh % a.H;
  const int rg = lane / C4, c4 = lane % C4;
  const int c0 = cs * kColsUp;                    // this block's first column
  const int col = c0 + 4 * (C4 * warp + c4);      // this lane's
  float* S = a.state + ((size_t)b * a.H + h) * D * D + col;

  // which rows: checked before anything is written
  const int t0 = __ldg(a.cu + b);
  const int m = __ldg(a.cu + b + 1) - t0;
  int n = kPath ? __ldg(a.accept_len + b) : m;
  bool ok = t0 >= 0 && m >= 0 && m <= a.max_tokens && (long long)t0 + m <= a.token_capacity;
  if constexpr (kPath) {
    ok = ok && n >= 0 && n <= m;
    for (int j = tid; ok && j < n; j += kThreadsUp) {
      const int p = __ldg(a.accept_path + t0 + j);
      if (p < 0 || p >= m) ok = false;
      s_path[j] = p;
    }
    ok = __syncthreads_and(ok);
  }
  if (!ok) {
    if (tid == 0) set_status(a.status, kStatusInvalidArg);
    return;
  }
  if (n == 0) return;

  // the state, in flight while the first tile is
  float4 s4[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s4[i][e] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(4 * (RG * i + rg) + e) * D));

  const size_t hs = (size_t)a.H * D;
  constexpr int kVecs = kTile * (D / 4) / kThreadsUp;   // 16-byte pieces of k (of q) per thread and tile
  float4 pk[kVecs], pq[kOut ? kVecs : 1], pv;
  float pa = 1.f, pb = 0.f;
  constexpr int kVPieces = kTile * (kColsUp / 4);   // of v per tile, at most one a thread
  static_assert(kVPieces <= kThreadsUp, "v");
  auto row_of = [&](int j) -> size_t { return (size_t)t0 + (kPath ? s_path[j] : j); };
  auto fetch = [&](int j0) {
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      const int e = tid + x * kThreadsUp, j = j0 + e / (D / 4);
      if (j < n) {
        const size_t at = row_of(j) * hs + (size_t)h * D + 4 * (e % (D / 4));
        pk[x] = up_load4(static_cast<const T*>(a.k) + at);
        if constexpr (kOut) pq[x] = up_load4(static_cast<const T*>(a.q) + at);
      }
    }
    const int j = j0 + tid / (kColsUp / 4);
    if (tid < kVPieces && j < n)
      pv = up_load4(static_cast<const T*>(a.v) + row_of(j) * hs + (size_t)h * D + c0 + 4 * (tid % (kColsUp / 4)));
    if (tid < kTile && j0 + tid < n) {
      pa = __ldg(a.alpha + row_of(j0 + tid) * a.H + h);
      pb = __ldg(a.beta + row_of(j0 + tid) * a.H + h);
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      const int e = tid + x * kThreadsUp;
      *reinterpret_cast<float4*>(&sk[buf][e / (D / 4)][4 * (e % (D / 4))]) = pk[x];
      if constexpr (kOut) *reinterpret_cast<float4*>(&sq[buf][e / (D / 4)][4 * (e % (D / 4))]) = pq[x];
    }
    if (tid < kVPieces) *reinterpret_cast<float4*>(&sv[buf][tid / (kColsUp / 4)][4 * (tid % (kColsUp / 4))]) = pv;
    if (tid < kTile) { s_alpha[buf][tid] = pa; s_beta[buf][tid] = pb; }
  };
  fetch(0);
  stage(0);
  __syncthreads();

  uint64_t s2[2 * NI][4];   // [row pair][column]
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      s2[2 * i + p][0] = f2_pack(s4[i][2 * p].x, s4[i][2 * p + 1].x);
      s2[2 * i + p][1] = f2_pack(s4[i][2 * p].y, s4[i][2 * p + 1].y);
      s2[2 * i + p][2] = f2_pack(s4[i][2 * p].z, s4[i][2 * p + 1].z);
      s2[2 * i + p][3] = f2_pack(s4[i][2 * p].w, s4[i][2 * p + 1].w);
    }

  for (int j0 = 0, buf = 0; j0 < n; j0 += kTile, buf ^= 1) {
    const bool more = j0 + kTile < n;   // uniform over the block
    if (more) fetch(j0 + kTile);
    const int cnt = min(kTile, n - j0);
    constexpr int kUnroll = kOut ? 4 : 1;   // single precision prompts 133 -> 125 us; a path's few nodes lose by it
#pragma unroll kUnroll
    for (int j = 0; j < cnt; ++j) {
      uint64_t k2[2 * NI];
      uint64_t x2[4], y2[4], z2 = 0;   // S^T k, S^T q, q.k (0 bits: a pair of zeros)
#pragma unroll
      for (int c = 0; c < 4; ++c) x2[c] = y2[c] = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const ulonglong2 kv = *reinterpret_cast<const ulonglong2*>(&sk[buf][j][4 * (RG * i + rg)]);
        k2[2 * i] = kv.x;
        k2[2 * i + 1] = kv.y;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x2[c] = f2_fma(s2[2 * i][c], kv.x, x2[c]);
          x2[c] = f2_fma(s2[2 * i + 1][c], kv.y, x2[c]);
        }
        if constexpr (kOut) {
          const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(&sq[buf][j][4 * (RG * i + rg)]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y2[c] = f2_fma(s2[2 * i][c], qv.x, y2[c]);
            y2[c] = f2_fma(s2[2 * i + 1][c], qv.y, y2[c]);
          }
          z2 = f2_fma(qv.x, kv.x, z2);
          z2 = f2_fma(qv.y, kv.y, z2);
        }
      }
      float x[4], y[4], z = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float lo, hi;
        f2_unpack(x2[c], lo, hi);
        x[c] = lo + hi;
        if constexpr (kOut) {
          f2_unpack(y2[c], lo, hi);
          y[c] = lo + hi;
        }
      }
      if constexpr (kOut) {
        float lo, hi;
        f2_unpack(z2, lo, hi);
        z = lo + hi;
      }
#pragma unroll
      for (int o = C4; o < 32; o <<= 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], o);
        if constexpr (kOut) {
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] += __shfl_xor_sync(0xffffffffu, y[c], o);
          z += __shfl_xor_sync(0xffffffffu, z, o);
        }
      }
      const float al = s_alpha[buf][j], be = s_beta[buf][j];
      const float4 vv = *reinterpret_cast<const float4*>(&sv[buf][j][4 * (C4 * warp + c4)]);
      float w[4];
      w[0] = be * (vv.x - al * x[0]);
      w[1] = be * (vv.y - al * x[1]);
      w[2] = be * (vv.z - al * x[2]);
      w[3] = be * (vv.w - al * x[3]);
      const uint64_t a2 = f2_pack(al, al);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint64_t w2 = f2_pack(w[c], w[c]);
#pragma unroll
        for (int i = 0; i < 2 * NI; ++i) s2[i][c] = f2_fma(a2, s2[i][c], f2_mul(k2[i], w2));
      }
      if constexpr (kOut) {
        if (rg == 0)
          up_store4(static_cast<T*>(a.out) + row_of(j0 + j) * hs + (size_t)h * D + col,
                    make_float4(fmaf(z, w[0], al * y[0]), fmaf(z, w[1], al * y[1]), fmaf(z, w[2], al * y[2]),
                                fmaf(z, w[3], al * y[3])));
      }
    }
    if (more) stage(buf ^ 1);
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float lo[4], hi[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) f2_unpack(s2[2 * i + p][c], lo[c], hi[c]);
      float* at = S + (size_t)(4 * (RG * i + rg) + 2 * p) * D;
      __stcs(reinterpret_cast<float4*>(at), make_float4(lo[0], lo[1], lo[2], lo[3]));
      __stcs(reinterpret_cast<float4*>(at + D), make_float4(hi[0], hi[1], hi[2], hi[3]));
    }
}

template <int D, typename T, bool kPath, int RG>
cudaError_t launch_recurrent_rows(const GdnUpdateArgs& a, cudaStream_t s) {
  return check_cuda(launch_pdl(gdn_recurrent_kernel<D, T, kPath, RG>, dim3((unsigned)((long long)a.B * a.H * (D * RG / 256))),
                               dim3(kThreadsUp), 0, s, a),
                    "launch gdn_recurrent_kernel");
}

// Sixteen row groups: twice the warps, each with half of a token's products and a fourth shuffle.  They pay when
// there is a scheduler for every warp and more than a few tokens (fp32, 5 sequences of up to 777 tokens, 6
// heads: 104 us against 125), not otherwise (one token of 1 sequence 2.7 against 2.4 us, of 64 57 against 42).
constexpr int kSchedulers = 608;
constexpr int kFewTokens = 8;

template <int D, typename T>
cudaError_t launch_recurrent_typed(const GdnUpdateArgs& a, cudaStream_t s) {
  if (a.accept_len != nullptr) return launch_recurrent_rows<D, T, true, 8>(a, s);
  if (a.max_tokens > kFewTokens && (long long)a.B * a.H * (D / 8) <= kSchedulers)
    return launch_recurrent_rows<D, T, false, 16>(a, s);
  return launch_recurrent_rows<D, T, false, 8>(a, s);
}

}  // namespace

cudaError_t launch_gdn_recurrent(const GdnUpdateArgs& a, cudaStream_t s) {
  if (a.bf16)
    return a.d == 64 ? launch_recurrent_typed<64, __nv_bfloat16>(a, s) : launch_recurrent_typed<128, __nv_bfloat16>(a, s);
  return a.d == 64 ? launch_recurrent_typed<64, float>(a, s) : launch_recurrent_typed<128, float>(a, s);
}

}  // namespace tva
