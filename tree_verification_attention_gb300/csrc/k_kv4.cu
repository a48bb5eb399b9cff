// k_kv4.cu - writing K / V rows into the 4-bit cache, and reading its values back
// (kv4.cuh, include/tva.h "4-bit cache").
//
// append: row i of k, v [n, Hkv, d] is quantised into record row slot[i].
// commit: the accepted path's rows of tree_k, tree_v ("Faster decoding", "The scheduler
//         must plan speculative work"), as commit_accepted_kv copies them.
// read:   the values that record rows stand for.
//
// A thread quantises one block of 16 values: it loads them, finds the scale, and stores
// eight bytes of codes; four threads put their scale bytes together into one word.  The
// blocks of a row are numbered K before V and head by head, so neighbouring threads load
// neighbouring 32 (fp32: 64) bytes.
#include "kv4.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ float to_f(T v) { return (float)v; }

// Quantises the 16 values at `src` (aligned to their size) into codes and a scale byte.
template <typename T>
__device__ __forceinline__ int quantise16(const T* src, uint32_t code[2]) {
  alignas(16) T x[16];
  const uint4* s4 = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint4*>(x)[i] = __ldg(s4 + i);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(to_f(x[i])));
  const int byte = kv4_scale_byte(amax);
  const float s = kv4_scale_value(byte), inv = byte > 0 ? 1.0f / s : 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t c = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) c |= (uint32_t)(kv4_round(to_f(x[8 * w + e]), s, inv) + 8) << kv4_shift(e);
    code[w] = c;
  }
  return byte;
}

// One block (half 0: K, 1: V; block `blk` of head `head`) of a row into its record.  Called
// by whole groups of four lanes with consecutive blocks (d / 16 is a multiple of 4).
template <typename T>
__device__ __forceinline__ void store_block(const T* src, uint8_t* rec, int d, int half, int blk) {
  uint32_t code[2];
  const int byte = quantise16(src, code);
  *reinterpret_cast<uint2*>(rec + half * (d / 2) + blk * 8) = make_uint2(code[0], code[1]);
  const int lane = threadIdx.x & 31;
  const uint32_t group = 0xfu << (lane & ~3);
  uint32_t w = (uint32_t)byte << (8 * (lane & 3));
  w |= __shfl_xor_sync(group, w, 1);
  w |= __shfl_xor_sync(group, w, 2);
  if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(rec + d + half * (d / 16) + blk) = w;
  const int pad = 9 * d / 8;
  if (pad != kv4_record_bytes(d) && half == 1 && blk == d / 16 - 1)
    *reinterpret_cast<uint2*>(rec + pad) = make_uint2(0u, 0u);
}

// Item t of a row: its K blocks, then its V blocks.
template <typename T>
__device__ __forceinline__ void quantise_item(const T* k, const T* v, uint8_t* cache, long long src_row,
                                              long long dst_row, int Hkv, int d, int t) {
  const int nb = d / 16, per = Hkv * nb;
  const int half = t >= per ? 1 : 0;
  const int in_row = t - half * per;
  const int head = in_row / nb, blk = in_row % nb;
  const T* src = (half ? v : k) + src_row * (long long)Hkv * d + in_row * 16;
  uint8_t* rec = cache + (dst_row * Hkv + head) * (long long)kv4_record_bytes(d);
  store_block<T>(src, rec, d, half, blk);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(Kv4RowArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int per_row = 2 * a.Hkv * (a.d / 16);
  const long long total = (long long)a.rows * per_row;
  for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < total; e += (long long)gridDim.x * kThreads) {
    const long long row = e / per_row;
    const int t = (int)(e - row * per_row);
    const long long slot = __ldg(a.slot + row);
    if (slot < 0) continue;
    if (slot >= a.kv_capacity) {
      if (t == 0) set_status(a.status, kStatusInvalidArg);
      continue;
    }
    quantise_item<T>(static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.cache, row, slot, a.Hkv, a.d, t);
  }
}

constexpr int kRowsPerBlock = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads) commit_kv4_kernel(CommitArgs a, int Hkv, int d) {
  __shared__ int s_path[kMaxNodes];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int b = blockIdx.x, y = blockIdx.y;
  const int n0 = __ldg(a.cu_nodes + b);
  const int m = __ldg(a.cu_nodes + b + 1) - n0;
  const int L = __ldg(a.accept_len + b);
  const long long dst = __ldg(a.dst_row + b);
  bool ok = n0 >= 0 && m >= 0 && m <= a.max_nodes && (long long)n0 + m <= a.node_capacity && L >= 0 && L <= m &&
            dst >= 0 && dst + L <= a.kv_capacity;
  // every path id of the sequence, not only this block's rows
  for (int j = threadIdx.x; ok && j < L; j += kThreads) {
    const int p = __ldg(a.accept_path + n0 + j);
    if (p < 0 || p >= m) ok = false;
    s_path[j] = p;
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (y == 0 && threadIdx.x == 0) set_status(a.status, kStatusInvalidArg);
    return;
  }
  const int j0 = y * kRowsPerBlock, j1 = min(L, j0 + kRowsPerBlock);
  const int per_row = 2 * Hkv * (d / 16);
  for (int e = threadIdx.x; e < (j1 - j0) * per_row; e += kThreads) {
    const int j = j0 + e / per_row;
    quantise_item<T>(static_cast<const T*>(a.tree_k), static_cast<const T*>(a.tree_v),
                     static_cast<uint8_t*>(a.k_cache), (long long)n0 + s_path[j], dst + j, Hkv, d, e % per_row);
  }
}

// Eight values of code word `w` at scale byte `byte`.
__device__ __forceinline__ void values8(uint32_t w, int byte, float x[8]) {
  const float s = kv4_scale_value(byte);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)((int)((w >> kv4_shift(e)) & 15u) - 8) * s;
}

__device__ __forceinline__ void store8(float* dst, const float x[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float x[8]) {  // exact
  *reinterpret_cast<uint4*>(dst) = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                                              ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(__half* dst, const float x[8]) {  // exact
  *reinterpret_cast<uint4*>(dst) = make_uint4(ptx::pack_f16x2(x[0], x[1]), ptx::pack_f16x2(x[2], x[3]),
                                              ptx::pack_f16x2(x[4], x[5]), ptx::pack_f16x2(x[6], x[7]));
}

// A thread reads one code word (8 values), numbered as the destination's elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(Kv4RowArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int words = a.d / 8, per_half = a.Hkv * words;
  const long long total = (long long)a.rows * per_half * 2;
  for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < total; e += (long long)gridDim.x * kThreads) {
    const long long row = e / (2 * per_half);
    const int t = (int)(e - row * 2 * per_half);
    const int half = t >= per_half ? 1 : 0, in_row = t - half * per_half;
    const int head = in_row / words, i = in_row % words;
    const long long slot = a.slot != nullptr ? (long long)__ldg(a.slot + row) : row;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (slot >= a.kv_capacity) {
      if (t == 0) set_status(a.status, kStatusInvalidArg);
    } else if (slot >= 0) {
      const uint8_t* rec = a.cache + (slot * a.Hkv + head) * (long long)kv4_record_bytes(a.d);
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(rec + half * (a.d / 2)) + i);
      values8(w, __ldg(rec + a.d + half * (a.d / 16) + i / 2), x);
    }
    T* dst = static_cast<T*>(const_cast<void*>(half ? a.v : a.k)) + (row * per_half + in_row) * 8;
    store8(dst, x);
  }
}

unsigned blocks_for(long long items) {
  const long long b = (items + kThreads - 1) / kThreads;
  return (unsigned)(b < 1 ? 1 : (b < 152 * 64 ? b : 152 * 64));
}

template <typename T>
cudaError_t run_append(const Kv4RowArgs& a, cudaStream_t s) {
  const long long items = (long long)a.rows * 2 * a.Hkv * (a.d / 16);
  return check_cuda(launch_pdl(append_kernel<T>, dim3(blocks_for(items)), dim3(kThreads), 0, s, a),
                    "launch append_kernel");
}

template <typename T>
cudaError_t run_read(const Kv4RowArgs& a, cudaStream_t s) {
  const long long items = (long long)a.rows * 2 * a.Hkv * (a.d / 8);
  return check_cuda(launch_pdl(read_kernel<T>, dim3(blocks_for(items)), dim3(kThreads), 0, s, a), "launch read_kernel");
}

template <typename T>
cudaError_t run_commit(const CommitArgs& a, int Hkv, int d, cudaStream_t s) {
  const dim3 grid((unsigned)a.B, (unsigned)((a.max_nodes + kRowsPerBlock - 1) / kRowsPerBlock));
  return check_cuda(launch_pdl(commit_kv4_kernel<T>, grid, dim3(kThreads), 0, s, a, Hkv, d),
                    "launch commit_kv4_kernel");
}

}  // namespace

cudaError_t launch_append_kv4(const Kv4RowArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? run_append<float>(a, s) : dtype == 2 ? run_append<__half>(a, s) : run_append<__nv_bfloat16>(a, s);
}

cudaError_t launch_read_kv4(const Kv4RowArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? run_read<float>(a, s) : dtype == 2 ? run_read<__half>(a, s) : run_read<__nv_bfloat16>(a, s);
}

cudaError_t launch_commit_kv4(const CommitArgs& a, int Hkv, int d, int dtype, cudaStream_t s) {
  return dtype == 1   ? run_commit<float>(a, Hkv, d, s)
         : dtype == 2 ? run_commit<__half>(a, Hkv, d, s)
                      : run_commit<__nv_bfloat16>(a, Hkv, d, s);
}

}  // namespace tva
