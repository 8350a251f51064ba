// Building blocks of the kernels that work on whole token rows (norms, rotary positions): a
// row is owned by a group of W warps, every thread of which holds the same 8 channels of each
// row it meets.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace rola {

constexpr int kVec = 8;              // channels of a thread
constexpr int kMaxRowChannels = 8192;
constexpr int kMaxRowWarps = kMaxRowChannels / kVec / 32;
constexpr int kRowSMs = 148;

// Shape of a launch over rows of C channels: W warps own a row, a block holds G such groups.
struct RowShape {
  int W, G, threads, blocks;
};
inline RowShape row_shape(long long rows, int C, int threads_per_sm) {
  RowShape s;
  s.W = (C / kVec + 31) / 32;
  s.G = s.W >= 8 ? 1 : 8 / s.W;
  s.threads = 32 * s.W * s.G;
  long long want = (rows + s.G - 1) / s.G;
  int per_sm = threads_per_sm / s.threads;
  const long long most = (long long)kRowSMs * (per_sm < 1 ? 1 : per_sm);
  s.blocks = (int)(want < most ? want : most);
  return s;
}

template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// The one rounding of an output (round to nearest even; fp32 is stored as it is).
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
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
    if (W == 1) {
      __syncwarp();
    } else {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(32 * W) : "memory");
    }
  }
};

// Sums of NV values over the group, to every thread, in a fixed order: a butterfly in each
// warp, then the warps' sums one after the other.  `buf` is [kMaxRowWarps][NV] of the group;
// two reductions in a row use two buffers (one barrier then keeps them apart).
template <int NV>
__device__ __forceinline__ void group_sum(const RowGroup& rg, float (&v)[NV], float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (rg.W == 1) {
    __syncwarp();
    return;
  }
  if (rg.lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[rg.wi * NV + i] = v[i];
  rg.sync();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = rg.lane < rg.W ? buf[rg.lane * NV + i] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

}  // namespace rola
