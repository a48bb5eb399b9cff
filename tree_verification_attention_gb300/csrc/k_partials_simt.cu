// k_partials_simt.cu - attention partials on the CUDA cores (float32 inputs).
//
// One CTA per worker of the unit decomposition in tva_common.cuh.  For every segment
// (a contiguous run of key tiles of one row group) the CTA walks the row group in
// blocks of 32 rows; per block it streams the segment's keys in sub-tiles of 32 (each
// thread's share fetched as 16-byte vectors one sub-tile ahead, so the loads of the
// next sub-tile overlap the work on this one) and keeps a running maximum / sum per
// row (online softmax, base 2), so each segment
// yields the partial output O and log-sum-exp LSE of the LongSpec aggregation
// ("Fast Tree Attention", Aggregation).  The tree tile is masked with the
// ancestor-or-self bits of each row's node (LongSpec's tree mask; "Faster decoding",
// "Chains and trees consume work differently").
//
// Shared-memory reads bound a busy CTA: 5 sequences of up to 3001 rows, 13 nodes, d = 64
// under a window take 34.6 us with the combine (62 with scalar reads, 45 with one row a
// thread).  That call has 136 units for 456 CTAs, so each busy one passes its unit's 128 keys
// twice (32 rows and 7) while the others idle: finer units would shorten it.  At d = 128 two
// rows a thread spill (28 bytes; 64 under a window) and win all the same: 16384 rows, 8 nodes,
// Hq 32, Hkv 8, no window 117 us instead of 174 (d = 64: 62 instead of 91).
//
// This path carries the float32 dtype (head_dim 64 or 128).  bfloat16 inputs go to
// the tensor-core kernel.
#include <type_traits>

#include "tva_internal.h"

namespace tva {
namespace {

constexpr int kRB = 32;       // rows per block
constexpr int kKT = 32;       // keys per sub-tile
constexpr int kRows = 2;      // rows per thread, kRB / kRows apart
constexpr int kThreads = 128; // 8 threads per kRows rows: 4 keys each for QK, D/8 columns for PV

// Four consecutive elements of a row (16-byte aligned: rows are D floats and the base
// pointers are 16-byte aligned).
__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

template <int D>
constexpr size_t simt_smem_bytes() {
  return sizeof(float) * (kRB * D + kKT * D + kKT * D + kRB * (kKT + 4)) + sizeof(uint32_t) * kMaxNodes * 4;
}

template <int D, bool kWin>
__global__ void __launch_bounds__(kThreads, 3) partials_simt_kernel(PartialArgsOf<std::conditional_t<kWin, WinProblem, Problem>> a) {
  extern __shared__ float smem[];
  // The products' shared-memory reads bound the kernel: they are 16 bytes wide, and a thread
  // uses each K and V value for two rows.  Chunk c (4 floats) of row r of qs is at c ^ (r mod 8), of key r of ks
  // at c ^ (r / 4 mod 8): the rows that a warp reads together are then in different banks.
  float* qs = smem;                          // [kRB][D]
  float* ks = qs + kRB * D;                  // [kKT][D]
  float* vs = ks + kKT * D;                  // [kKT][D]
  float* ps = vs + kKT * D;                  // [kRB][kKT+4]
  uint32_t* masks = reinterpret_cast<uint32_t*>(ps + kRB * (kKT + 4));  // [128][4]
  __shared__ int tree_bad;
  __shared__ int par_s[kMaxNodes];           // parent ids of the current tree
  __shared__ int low_s[kWin ? kMaxNodes : 1];  // kWin: lowest prefix key each node sees through its window

  __shared__ int cu_buf[512];
  auto pr = a.pr;
  stage_cu(pr, cu_buf, 512);
  const float* __restrict__ q = static_cast<const float*>(a.q);
  const int tid = threadIdx.x;
  const int r_loc = tid >> 3;  // first row of this thread inside the block
  const int kg = tid & 7;      // key group (QK) / column phase (PV)
  const int u = blockIdx.x;
  if (u == 0 && tid == 0) validate_sequences(pr, a.status);
  long long t = 0, t_end = 0;
  worker_range(pr, u, t, t_end, pr.share != 0);
  const size_t kv_stride = (size_t)pr.Hkv * D;

  Segment S;
  while (next_segment(pr, u, t, t_end, S, pr.share != 0)) {
    const Loc L = S.L;
    const int tile0 = S.tile0;
    const int tile1 = S.tile0 + S.n;
    const bool has_tree = tile0 == 0;   // the tree tile is a row group's first unit
    const SeqInfo s = L.s;
    const long long slot = partial_slot(pr, u, L, pr.share != 0);
    const bool slot_ok = slot < a.slots;  // cannot fail for a consistent layout
    if (!slot_ok && tid == 0) set_status(a.status, kStatusInvalidArg);

    if (has_tree || kWin) {
      __syncthreads();
      if (tid == 0) tree_bad = 0;
      __syncthreads();
      for (int i = tid; i < s.m; i += kThreads) par_s[i] = __ldg(a.parent + s.n0 + i);  // one round of loads
      __syncthreads();
      for (int i = tid; i < s.m; i += kThreads) {
        uint32_t bits[4];
        if constexpr (kWin) {
          int depth;
          if (!window_ancestors(par_s, i, pr.window, pr.sinks, s.len, bits, depth)) tree_bad = 1;
          low_s[i] = window_low(pr, s, depth);
        } else {
          if (!ancestor_bits_shared(par_s, i, bits)) tree_bad = 1;
        }
        masks[i * 4 + 0] = bits[0]; masks[i * 4 + 1] = bits[1];
        masks[i * 4 + 2] = bits[2]; masks[i * 4 + 3] = bits[3];
      }
      __syncthreads();
      if (tid == 0 && tree_bad) set_status(a.status, kStatusBadTree);
    }

    const int rows_total = s.m * pr.G;
    const int row_begin = L.mp * pr.RG;
    const int row_end = min(rows_total, row_begin + pr.RG);
    for (int rb = row_begin; rb < row_end; rb += kRB) {
      __syncthreads();
      {
        // all of the thread's loads first (one round of latency), then the stores
        constexpr int kN = kRB * D / 4 / kThreads;
        float4 qv[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int idx = (tid + i * kThreads) * 4, r = idx / D, dd = idx % D, row = rb + r;
          qv[i] = row < row_end
                      ? load4(q + ((size_t)(s.n0 + row / pr.G) * pr.Hq + L.g * pr.G + row % pr.G) * D + dd)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int idx = (tid + i * kThreads) * 4, r = idx / D, dd = idx % D;
          *reinterpret_cast<float4*>(qs + r * D + (dd ^ ((r & 7) * 4))) = qv[i];
        }
      }
      int my_row[kRows], my_node[kRows];
      bool row_ok[kRows];
      float m_run[kRows], l_run[kRows], o[kRows][D / 8];
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        my_row[x] = rb + r_loc + x * (kRB / kRows);
        row_ok[x] = my_row[x] < row_end;
        my_node[x] = row_ok[x] ? my_row[x] / pr.G : 0;
        m_run[x] = -INFINITY;
        l_run[x] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) o[x][k] = 0.f;
      }

      for (int tile = tile0; tile < tile1; ++tile) {
        const bool is_tree = tile == 0;
        int key0 = (tile - 1) * kKeyTile, nkeys = is_tree ? s.m : min(kKeyTile, s.P - key0), sinks = 0;
        if constexpr (kWin) {
          sinks = pr.sinks;
          if (!is_tree) {
            key0 = tile_key0(s, tile);
            nkeys = tile_keys(pr, s, tile);
          }
        }
        int low[kRows];
#pragma unroll
        for (int x = 0; x < kRows; ++x) low[x] = kWin && !is_tree ? low_s[my_node[x]] : 0;  // my_node < m
        const float* kb = static_cast<const float*>(is_tree ? a.tree_k : a.k_cache);
        const float* vb = static_cast<const float*>(is_tree ? a.tree_v : a.v_cache);
        const size_t first = is_tree ? (size_t)s.n0 : (size_t)s.p0 + (size_t)key0;
        kb += first * kv_stride + (size_t)L.g * D;
        vb += first * kv_stride + (size_t)L.g * D;
        // The sub-tile's K / V are loaded into registers one sub-tile ahead: the loads
        // of sub-tile k0 + kKT are in flight while sub-tile k0 is computed.
        constexpr int kN = kKT * D / 4 / kThreads;
        float4 kr[kN], vr[kN];
        auto fetch = [&](int k0) {
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int idx = (tid + i * kThreads) * 4, key = idx / D, dd = idx % D;
            const bool valid = k0 + key < nkeys;
            kr[i] = valid ? load4(kb + (size_t)(k0 + key) * kv_stride + dd) : make_float4(0.f, 0.f, 0.f, 0.f);
            vr[i] = valid ? load4(vb + (size_t)(k0 + key) * kv_stride + dd) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        };
        fetch(0);
        for (int k0 = 0; k0 < nkeys; k0 += kKT) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int idx = (tid + i * kThreads) * 4, key = idx / D, dd = idx % D;
            *reinterpret_cast<float4*>(ks + key * D + (dd ^ (((key >> 2) & 7) * 4))) = kr[i];
            *reinterpret_cast<float4*>(vs + key * D + dd) = vr[i];
          }
          if (k0 + kKT < nkeys) fetch(k0 + kKT);
          __syncthreads();
          float sc[kRows][4];
#pragma unroll
          for (int x = 0; x < kRows; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[x][k] = 0.f;
#pragma unroll 2
          for (int dd = 0; dd < D; dd += 4) {
            float4 qv[kRows];
#pragma unroll
            for (int x = 0; x < kRows; ++x) {
              const int r = r_loc + x * (kRB / kRows);
              qv[x] = *reinterpret_cast<const float4*>(qs + r * D + (dd ^ ((r & 7) * 4)));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 kv = *reinterpret_cast<const float4*>(ks + (kg * 4 + k) * D + (dd ^ (kg * 4)));
#pragma unroll
              for (int x = 0; x < kRows; ++x) {
                sc[x][k] = fmaf(qv[x].x, kv.x, sc[x][k]);
                sc[x][k] = fmaf(qv[x].y, kv.y, sc[x][k]);
                sc[x][k] = fmaf(qv[x].z, kv.z, sc[x][k]);
                sc[x][k] = fmaf(qv[x].w, kv.w, sc[x][k]);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < kRows; ++x) {
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = k0 + kg * 4 + k;
              bool vis = row_ok[x] && key < nkeys;
              if (kWin && !is_tree) vis = vis && (key0 + key >= low[x] || key0 + key < sinks);
              if (is_tree && vis) vis = (masks[my_node[x] * 4 + (key >> 5)] >> (key & 31)) & 1u;
              sc[x][k] = vis ? sc[x][k] * a.scale_log2 : -INFINITY;
              mx = fmaxf(mx, sc[x][k]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            const float m_new = fmaxf(m_run[x], mx);
            const float alpha = (m_new == -INFINITY) ? 1.f : exp2f(m_run[x] - m_new);
            float psum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float p = (sc[x][k] == -INFINITY) ? 0.f : exp2f(sc[x][k] - m_new);
              ps[(r_loc + x * (kRB / kRows)) * (kKT + 4) + kg * 4 + k] = p;
              psum += p;
            }
            psum += __shfl_xor_sync(0xffffffffu, psum, 4);
            psum += __shfl_xor_sync(0xffffffffu, psum, 2);
            psum += __shfl_xor_sync(0xffffffffu, psum, 1);
            l_run[x] = l_run[x] * alpha + psum;
            m_run[x] = m_new;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) o[x][k] *= alpha;
          }
          __syncwarp();
#pragma unroll 2
          for (int j = 0; j < kKT; j += 4) {  // this thread's columns: 4 kg .. 4 kg + 3 of every 32
            float pj[kRows][4];
#pragma unroll
            for (int x = 0; x < kRows; ++x) {
              const float4 pv = *reinterpret_cast<const float4*>(ps + (r_loc + x * (kRB / kRows)) * (kKT + 4) + j);
              pj[x][0] = pv.x; pj[x][1] = pv.y; pj[x][2] = pv.z; pj[x][3] = pv.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(vs + (j + e) * D + 32 * k + 4 * kg);
#pragma unroll
                for (int x = 0; x < kRows; ++x) {
                  o[x][4 * k] = fmaf(pj[x][e], v.x, o[x][4 * k]);
                  o[x][4 * k + 1] = fmaf(pj[x][e], v.y, o[x][4 * k + 1]);
                  o[x][4 * k + 2] = fmaf(pj[x][e], v.z, o[x][4 * k + 2]);
                  o[x][4 * k + 3] = fmaf(pj[x][e], v.w, o[x][4 * k + 3]);
                }
              }
          }
        }
      }
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        if (!row_ok[x] || !slot_ok) continue;
        // under a window a row may see no key of the segment: its partial is 0, log 0
        const float inv = kWin && l_run[x] == 0.f ? 0.f : 1.f / l_run[x];
        const int rr = my_row[x] - row_begin, MT = mtile_rows(pr.G);
        const int pp = rr / MT * 128 + rr % MT;  // padded row (see o_part_offset)
        const int RGP = padded_group_rows(pr.RG, pr.G);
        if (TVA_CHECK(pp < RGP, a.status)) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            *reinterpret_cast<float4*>(a.o_part + o_part_offset(slot, pp, 8 * k + kg, RGP, D)) =
                make_float4(o[x][4 * k] * inv, o[x][4 * k + 1] * inv, o[x][4 * k + 2] * inv, o[x][4 * k + 3] * inv);
          if (kg == 0) a.lse_part[(size_t)slot * RGP + pp] = m_run[x] + log2f(l_run[x]);
        }
      }
    }
  }
}

template <int D, bool kWin>
cudaError_t launch_simt_typed(const PartialArgsOf<std::conditional_t<kWin, WinProblem, Problem>>& a, cudaStream_t s) {
  constexpr size_t smem = simt_smem_bytes<D>();
  cudaError_t e = check_cuda(cudaFuncSetAttribute(partials_simt_kernel<D, kWin>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem),
                             "cudaFuncSetAttribute(partials_simt_kernel)");
  if (e != cudaSuccess) return e;
  partials_simt_kernel<D, kWin><<<a.pr.U, kThreads, smem, s>>>(a);
  return check_cuda(cudaGetLastError(), "launch partials_simt_kernel");
}

}  // namespace

int simt_workers_per_sm() { return 3; }

cudaError_t launch_partials_simt(const PartialArgs& a, int dtype, cudaStream_t s) {
  if (dtype != 1) {  // bf16 runs on the tensor-core kernel
    record_error("launch_partials_simt", 0, "float32 only");
    return cudaErrorInvalidValue;
  }
  return a.pr.d == 64 ? launch_simt_typed<64, false>(a, s) : launch_simt_typed<128, false>(a, s);
}

cudaError_t launch_partials_simt(const WinPartialArgs& a, int dtype, cudaStream_t s) {
  if (dtype != 1) {
    record_error("launch_partials_simt", 0, "float32 only");
    return cudaErrorInvalidValue;
  }
  return a.pr.d == 64 ? launch_simt_typed<64, true>(a, s) : launch_simt_typed<128, true>(a, s);
}

}  // namespace tva
