// Building blocks of the kernels that work on whole token rows (norms, rotary positions).  A row
// is owned by a group of W warps; thread t of the group holds V pieces of E neighbouring channels
// of every row it meets: pieces t, t + 32 W, ...  Rows to come are fetched by asynchronous copies
// into slots of shared memory that only the thread itself reads, so that fetching ahead costs
// neither registers nor barriers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace rola {

constexpr int kVec = 8;              // channels of a vector
constexpr int kMaxRowChannels = 8192;
constexpr int kRowSMs = 148;

// Threads of a row: W warps with V pieces each.  More pieces per thread mean fewer threads to
// reduce over; among the V whose last warp is not much emptier, the largest is taken (two pieces
// instead of one: backward of qk_norm_rope on 1536 bf16 channels 154 us, not 201; gated_norm on
// 5120, bound by memory, the same).
struct RowShape {
  int V, W, G, threads;   // G groups in a block
};
inline RowShape row_shape(int C, int E, int max_v, int max_warps) {
  const int pieces = C / E;
  RowShape s{1, (pieces + 31) / 32, 1, 0};
  for (int v = 2; v <= max_v; v *= 2) {
    const int w = (pieces + 32 * v - 1) / (32 * v);
    if (s.W > max_warps || 8ll * v * w <= 9ll * s.V * s.W) s.V = v, s.W = w;
  }
  s.G = s.W == 1 ? 4 : 1;   // groups of several warps have the block's barrier to themselves
  s.threads = 32 * s.W * s.G;
  return s;
}

// Lets a kernel take `smem` bytes of dynamic shared memory.  The limit is state of the kernel on the
// device, which calls from several host threads share: it is set to kMost, the most that any call
// of this instance takes, and never to the call's own size, so that no launch finds it lowered.
constexpr size_t kMostSharedMemory = 227 * 1024;   // of a block, with its static part
template <size_t kMost, typename K>
cudaError_t allow_shared_memory(K kern, size_t smem) {
  if (smem > kMost) return cudaErrorInvalidValue;
  if (smem <= 40 * 1024) return cudaSuccess;       // with the static part within the default
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
}

// E neighbouring channels of type T, as a thread moves them: 16 bytes, or 8 where bf16 stands
// beside fp32.  E is 8 where all tensors are bf16 and 4 where one is fp32, so that a warp's access
// always covers whole 32-byte sectors (8 fp32 channels as two 16-byte halves would touch every
// sector twice, and write each in two parts).
template <typename T, int E>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const uint4& a, float* v) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // the one rounding of an output: round to nearest even
  static __device__ __forceinline__ uint4 put(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Piece<__nv_bfloat16, 4> {
  using Raw = uint2;
  static __device__ __forceinline__ void get(const uint2& a, float* v) {
    v[0] = __uint_as_float(a.x << 16);
    v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16);
    v[3] = __uint_as_float(a.y & 0xffff0000u);
  }
  static __device__ __forceinline__ uint2 put(const float* v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]), g = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&h), *reinterpret_cast<const uint32_t*>(&g));
  }
};
template <>
struct Piece<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void get(const float4& a, float* v) {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  static __device__ __forceinline__ float4 put(const float* v) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <int E, typename T>
__device__ __forceinline__ void load_piece(const T* p, float* v) {
  Piece<T, E>::get(*reinterpret_cast<const typename Piece<T, E>::Raw*>(p), v);
}
template <int E, typename T>
__device__ __forceinline__ void store_piece(T* p, const float* v) {
  *reinterpret_cast<typename Piece<T, E>::Raw*>(p) = Piece<T, E>::put(v);
}
template <int E, typename T>
__host__ __device__ constexpr int piece_bytes() { return E * (int)sizeof(T); }
// E fp32 values (gains, modulations, partial sums).
template <int E>
__device__ __forceinline__ void load_floats(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < E; i += 4) load_piece<4>(p + i, v + i);
}
template <int E>
__device__ __forceinline__ void store_floats(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < E; i += 4) store_piece<4>(p + i, v + i);
}
// 8 channels of either type.
__device__ __forceinline__ void load8(const float* p, float* v) { load_floats<8>(p, v); }
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) { load_piece<8>(p, v); }
__device__ __forceinline__ void store8(float* p, const float* v) { store_floats<8>(p, v); }
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) { store_piece<8>(p, v); }

// Asynchronous copies into shared memory, waited for in groups: `keep` may still be in flight.
template <int bytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_addr(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(sm100::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int keep>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(keep) : "memory");
}
// A piece of T into the thread's slot of a plane [threads], and out of it.
template <int E, typename T>
__device__ __forceinline__ void fetch_piece(uint8_t* plane, const T* src) {
  constexpr int n = piece_bytes<E, T>();
  copy_async<n>(plane + threadIdx.x * n, src);
}
template <int E, typename T>
__device__ __forceinline__ void read_piece(const uint8_t* plane, float* v) {
  Piece<T, E>::get(reinterpret_cast<const typename Piece<T, E>::Raw*>(plane)[threadIdx.x], v);
}

// A thread's place in its group.
struct RowGroup {
  int W, g, wi, lane, t;   // warps of the group, group in the block, warp in it, lane, thread in it
  __device__ __forceinline__ explicit RowGroup(int warps) : W(warps) {
    const int warp = threadIdx.x >> 5;
    g = warp / W;
    wi = warp - g * W;
    lane = threadIdx.x & 31;
    t = 32 * wi + lane;
  }
  __device__ __forceinline__ void sync() const {
    if (W == 1)
      __syncwarp();
    else
      __syncthreads();   // the group is the block
  }
};

// Sums over the group, to every thread, in a fixed order: a butterfly in each warp (two values
// share one: each half of the lanes goes on with one of them), then the warps' sums one after
// the other.  A barrier as well.  `buf` holds W values (pairs) of the group; two
// reductions in a row use two buffers.
__device__ __forceinline__ float group_sum(const RowGroup& rg, float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (rg.W == 1) {
    __syncwarp();
    return v;
  }
  if (rg.lane == 0) buf[rg.wi] = v;
  rg.sync();
  v = buf[0];
  for (int w = 1; w < rg.W; ++w) v += buf[w];
  return v;
}
__device__ __forceinline__ float2 group_sum(const RowGroup& rg, float a, float b, float* buf) {
  const bool low = rg.lane < 16;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (rg.W == 1) return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  if ((rg.lane & 15) == 0) buf[2 * rg.wi + (rg.lane >> 4)] = v;
  rg.sync();
  const float2* p = reinterpret_cast<const float2*>(buf);
  float2 s = p[0];
  for (int w = 1; w < rg.W; ++w) {
    s.x += p[w].x;
    s.y += p[w].y;
  }
  return s;
}

// out[c] = sum over `parts` partial rows, `stride` floats apart, of the `fold` columns c, c + cols,
// ... : 128 threads take every 128th of the parts * fold values, eight loads at a time, then a fixed
// tree.  A block has 8 columns (one sector of a row) x 128 threads: with 32 x 32, a thousand columns
// were 32 blocks that each waited for a chain of loads (2331 rows of 1000: 15 us, now 11).
constexpr int kSumCols = 8, kSumRows = 128;
__device__ __forceinline__ void column_sum(const float* __restrict__ part, unsigned parts, size_t stride, int cols,
                                           unsigned fold, float* __restrict__ out) {
  __shared__ float sum[32][kSumCols + 1];
  const int col = blockIdx.x * kSumCols + threadIdx.x, y = threadIdx.y;
  const int lane = (y * kSumCols + threadIdx.x) & 31, warp = y / (32 / kSumCols);
  float s = 0.f;
  if (col < cols) {
    const unsigned rows = kSumRows / fold, more = kSumRows - rows * fold;   // 128 values on
    unsigned row = y / fold, f = y - row * fold;
    while (row < parts) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[u] = row < parts ? part[row * stride + (size_t)f * cols + col] : 0.f;
        row += rows;
        f += more;
        if (f >= fold) f -= fold, ++row;
      }
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
#pragma unroll
  for (int o = 16; o >= kSumCols; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane < kSumCols) sum[warp][lane] = s;
  __syncthreads();
  if (warp >= kSumCols) return;
  s = sum[lane][warp];                 // column `warp` of the block
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int at = blockIdx.x * kSumCols + warp;
  if (lane == 0 && at < cols) out[at] = s;
}

}  // namespace rola
