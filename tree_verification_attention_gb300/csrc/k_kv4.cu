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
// neighbouring 32 (fp32: 64) bytes.  A thread block takes a few whole rows, so that the
// numbers of its items stay small and dividing them by a row's items is one multiplication.
// What they must read and write, they do once; what bounds them is instructions.  32768 rows
// of 8 heads, d = 128, bf16 (172 MB each way): append 34.2 us (5.0 TB/s, 70 % of the issue
// slots), read 36.4 us (65 %); the copy peak would be 25 us.  The commit of 64 sequences takes
// 3.4 us back to back (6.9 cold), latency: the lengths, the path, then its rows.
#include <type_traits>

#include "kv4.cuh"
#include "tc_ptx.cuh"
#include "tva_internal.h"

namespace tva {
namespace {

constexpr int kThreads = 256;
constexpr int kItemsPerBlock = 2048;

// t / d for t < 2^16, d <= 2^16 as a multiplication: with m = ceil(2^32 / d) the error of
// t m / 2^32 is below t / 2^32 < 1 / d.
__host__ __device__ inline uint32_t small_inverse(uint32_t d) { return (uint32_t)(((1ull << 32) + d - 1) / d); }
__device__ __forceinline__ int small_div(int t, uint32_t inverse) { return (int)__umulhi((uint32_t)t, inverse); }

template <typename T> __device__ __forceinline__ float to_f(T v) { return (float)v; }

// The general form: any values of any type.
template <typename T>
__device__ __noinline__ int quantise16_any(const T* x, uint32_t code[2]) {
  float amax = 0.0f;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(to_f(x[i])));  // (a NaN is passed over)
  const int byte = kv4_scale_byte(amax);
  const float s = kv4_scale_value(byte), inv = byte > 0 ? 1.0f / s : 0.0f;
  code[0] = code[1] = 0u;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) code[i >> 3] |= (uint32_t)(kv4_round(to_f(x[i]), s, inv) + 8) << kv4_shift(i & 7);
  return byte;
}

// The two values of a packed 16-bit pair.
template <typename T> __device__ __forceinline__ float2 pair_f(uint32_t w);
template <> __device__ __forceinline__ float2 pair_f<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <> __device__ __forceinline__ float2 pair_f<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Quantises the 16 values at `src` (16-byte aligned) into codes and a scale byte.
//
// 16-bit values with a normal scale below the largest take a short way.  A quotient x / s
// (11 significant bits over 4, below 7.5) that is not halfway between two whole numbers is
// at least 2^-8 / 30 > 2^-13 away from it, so it may be rounded to a multiple of 2^-15
// first - which one fused multiply-add onto 384 does, taking up the errors of 1 / s as
// well - and that exactly representable value to the nearest whole number by a second
// addition, onto 3 * 2^22, whose low bits are then the code.  No limit is needed: the scale
// is at least 16/17 of amax / 7, so |x / s| <= 7.4375.
template <typename T>
__device__ __forceinline__ int quantise16(const T* src, uint32_t code[2]) {
  if constexpr (sizeof(T) == 4) {
    alignas(16) T x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(x)[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    const int byte = kv4_scale_byte(amax);
    const float s = kv4_scale_value(byte), inv = byte > 0 ? 1.0f / s : 0.0f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t c = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) c |= (uint32_t)(kv4_round(x[8 * w + e], s, inv) + 8) << kv4_shift(e);
      code[w] = c;
    }
    return byte;
  } else {
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src)), hi = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t m = w[0] & 0x7fff7fffu;  // the order of magnitudes is that of their bits
#pragma unroll
    for (int i = 1; i < 8; ++i) m = ptx::max_s16x2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    const int byte = kv4_scale_byte(pair_f<T>(m).x);
    if (m >= kInf || byte < 8 || byte >= kKv4MaxScale) return quantise16_any(src, code);
    const float inv = __fdividef(1.0f, kv4_scale_value(byte));
    const uint64_t inv2 = ptx::f2_pack(inv, inv), near2 = ptx::f2_pack(384.0f, 384.0f);
    const uint64_t whole2 = ptx::f2_pack(12582536.0f, 12582536.0f);  // 3 * 2^22 - 384 + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c = 0u - 0x4b400000u * 0x11111111u;  // what the eight sums' exponent bits add up to
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 p = pair_f<T>(w[4 * h + e / 2]);
        float z0, z1;
        ptx::f2_unpack(ptx::f2_add(ptx::f2_fma(ptx::f2_pack(p.x, p.y), inv2, near2), whole2), z0, z1);
        c += __float_as_uint(z0) << kv4_shift(e);
        c += __float_as_uint(z1) << kv4_shift(e + 1);
      }
      code[h] = c;
    }
    return byte;
  }
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
  __syncwarp(group);
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
  const int shift = d == 128 ? 3 : 2;  // d / 16 blocks a head
  const int per = Hkv << shift;
  const int half = t >= per ? 1 : 0;
  const int in_row = t - half * per;
  const int head = in_row >> shift, blk = in_row & ((1 << shift) - 1);
  const T* src = (half ? v : k) + src_row * (long long)Hkv * d + in_row * 16;
  uint8_t* rec = cache + (dst_row * Hkv + head) * (long long)kv4_record_bytes(d);
  store_block<T>(src, rec, d, half, blk);
}

// rows_per_block whole rows a block; `inverse` is small_inverse(items of a row).
template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(Kv4RowArgs a, int rows_per_block, uint32_t inverse) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int per_row = 2 * a.Hkv * (a.d / 16);
  const long long row0 = (long long)blockIdx.x * rows_per_block;
  const int rows = (int)min((long long)rows_per_block, a.rows - row0);
  for (int e = threadIdx.x; e < rows * per_row; e += kThreads) {
    const int i = rows_per_block > 1 ? small_div(e, inverse) : 0;
    const int t = e - i * per_row;
    const long long slot = __ldg(a.slot + row0 + i);
    if (slot < 0) continue;
    if (slot >= a.kv_capacity) {
      if (t == 0) set_status(a.status, kStatusInvalidArg);
      continue;
    }
    quantise_item<T>(static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.cache, row0 + i, slot, a.Hkv, a.d, t);
  }
}

constexpr int kRowsPerBlock = 2;  // of the commit: few rows, so many small blocks

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
  for (int j = j0; j < j1; ++j)
    for (int t = threadIdx.x; t < per_row; t += kThreads)
      quantise_item<T>(static_cast<const T*>(a.tree_k), static_cast<const T*>(a.tree_v),
                       static_cast<uint8_t*>(a.k_cache), (long long)n0 + s_path[j], dst + j, Hkv, d, t);
}

// The eight values of code word `w` at scale byte `byte`, exactly, in each type: by pairs, as
// the attention widens them (value by value the conversions bound the kernel).
__device__ __forceinline__ void store8(__nv_bfloat16* dst, uint32_t w, uint32_t byte) {
  uint32_t s, c;
  widen_scale<true>(byte, 0, s, c);
  *reinterpret_cast<uint4*>(dst) = widen8<true>(w, s, c);
}
__device__ __forceinline__ void store8(__half* dst, uint32_t w, uint32_t byte) {
  uint32_t s, c;
  widen_scale<false>(byte, 0, s, c);
  *reinterpret_cast<uint4*>(dst) = widen8<false>(w, s, c);
}
__device__ __forceinline__ void store8(float* dst, uint32_t w, uint32_t byte) {
  uint32_t s, c;
  widen_scale<false>(byte, 0, s, c);
  const uint4 h = widen8<false>(w, s, c);
  const float2 x0 = pair_f<__half>(h.x), x1 = pair_f<__half>(h.y), x2 = pair_f<__half>(h.z), x3 = pair_f<__half>(h.w);
  reinterpret_cast<float4*>(dst)[0] = make_float4(x0.x, x0.y, x1.x, x1.y);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x2.x, x2.y, x3.x, x3.y);
}

// A thread reads one code word (8 values), numbered as the destination's elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(Kv4RowArgs a, int rows_per_block, uint32_t inverse) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int shift = a.d == 128 ? 4 : 3;  // d / 8 words a head
  const int per_half = a.Hkv << shift, per_row = 2 * per_half;
  const long long row0 = (long long)blockIdx.x * rows_per_block;
  const int rows = (int)min((long long)rows_per_block, a.rows - row0);
  for (int e = threadIdx.x; e < rows * per_row; e += kThreads) {
    const int r = rows_per_block > 1 ? small_div(e, inverse) : 0;
    const int t = e - r * per_row;
    const long long row = row0 + r;
    const int half = t >= per_half ? 1 : 0, in_row = t - half * per_half;
    const int head = in_row >> shift, i = in_row & ((1 << shift) - 1);
    const long long slot = a.slot != nullptr ? (long long)__ldg(a.slot + row) : row;
    uint32_t word = 0u, byte = 0u;  // at scale 0 every code is 0
    if (slot >= a.kv_capacity) {
      if (t == 0) set_status(a.status, kStatusInvalidArg);
    } else if (slot >= 0) {
      const uint8_t* rec = a.cache + (slot * a.Hkv + head) * (long long)kv4_record_bytes(a.d);
      word = __ldg(reinterpret_cast<const uint32_t*>(rec + half * (a.d / 2)) + i);
      byte = __ldg(rec + a.d + half * (a.d / 16) + i / 2);
    }
    T* dst = static_cast<T*>(const_cast<void*>(half ? a.v : a.k)) + (row * per_half + in_row) * 8;
    store8(dst, word, byte);
  }
}

// Rows a block and blocks for rows of `per_row` items; more than 2^16 items a row (never
// numbered by small_div then) get a block each.
template <typename K>
cudaError_t launch_rows(K kernel, const Kv4RowArgs& a, int per_row, cudaStream_t s, const char* what) {
  // about 2048 items a block, but no fewer than 8 blocks an SM's worth while the rows last
  // (each block then holds a thread's worth of items or a row)
  const long long spread = a.rows / (152 * 8) + 1, least = (kThreads + per_row - 1) / per_row;
  const long long most = per_row >= kItemsPerBlock ? 1 : kItemsPerBlock / per_row;
  const int rows_per_block = (int)(spread < least ? least : spread < most ? spread : most);
  const long long blocks = ((long long)a.rows + rows_per_block - 1) / rows_per_block;
  return check_cuda(launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, rows_per_block,
                               small_inverse((uint32_t)per_row)),
                    what);
}

template <typename T>
cudaError_t run_append(const Kv4RowArgs& a, cudaStream_t s) {
  return launch_rows(append_kernel<T>, a, 2 * a.Hkv * (a.d / 16), s, "launch append_kernel");
}

template <typename T>
cudaError_t run_read(const Kv4RowArgs& a, cudaStream_t s) {
  return launch_rows(read_kernel<T>, a, 2 * a.Hkv * (a.d / 8), s, "launch read_kernel");
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
