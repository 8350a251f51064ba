// Joins the parts of a cross attention whose long axis was split over blocks.
//
//   out = sum_s exp(lse_s - lse) out_s,  lse = log sum_s exp(lse_s)      (forward)
//   dx  = sum_s dx_s                                                     (gradients)
//
// in the parts' order, in fp32, rounded once.  Bound by memory: every part is read once.
#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

// A row (b, n, h) of d channels: d / 8 threads.
template <typename T>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ CrossArgs a, int splits,
                                                         const float* __restrict__ part,
                                                         const float* __restrict__ plse, T* __restrict__ out,
                                                         float* __restrict__ lse) {
  const int per = a.d / kVec;
  const long long rows = (long long)a.B * a.Nq * a.H, e = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = e / per;
  if (row >= rows) return;
  const int c = (int)(e - row * per) * kVec, h = (int)(row % a.H);
  const long long bn = row / a.H;
  const int b = (int)(bn / a.Nq), n = (int)(bn - (long long)b * a.Nq);
  const size_t zat = ((size_t)b * a.H + h) * a.Nq + n, zs = (size_t)a.B * a.H * a.Nq;
  float top = -INFINITY;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, __ldg(plse + s * zs + zat));
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[kVec] = {};
  for (int s = 0; s < splits; ++s) {
    const float w = expf(__ldg(plse + s * zs + zat) - ref);
    sum += w;
    if (w == 0.f) continue;            // a part without a valid key holds zeros
    float v[kVec];
    load8(part + ((size_t)s * rows + row) * a.d + c, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] *= inv;
  store8(out + row * a.d + c, acc);
  if (c == 0 && lse) lse[zat] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename T>
__global__ void __launch_bounds__(256) cross_sum_kernel(int parts, size_t n, size_t stride,
                                                        const float* __restrict__ part, T* __restrict__ out) {
  const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * kVec;
  if (at >= n) return;
  float acc[kVec] = {};
  for (int s = 0; s < parts; ++s) {
    float v[kVec];
    load8(part + s * stride + at, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] += v[i];
  }
  store8(out + at, acc);
}

}  // namespace

cudaError_t launch_cross_join(const CrossArgs& a, rola_dtype dt, int splits, const float* part, const float* plse,
                              void* out, float* lse, cudaStream_t st) {
  const long long threads = (long long)a.B * a.Nq * a.H * (a.d / kVec);
  const unsigned grid = (unsigned)((threads + 255) / 256);
  if (dt == ROLA_F32)
    cross_join_kernel<float><<<grid, 256, 0, st>>>(a, splits, part, plse, (float*)out, lse);
  else
    cross_join_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, splits, part, plse, (__nv_bfloat16*)out, lse);
  return cudaGetLastError();
}

cudaError_t launch_cross_sum(rola_dtype dt, int parts, size_t n, size_t stride, const float* part, void* out,
                             cudaStream_t st) {
  const unsigned grid = (unsigned)((n / kVec + 255) / 256);
  if (dt == ROLA_F32)
    cross_sum_kernel<float><<<grid, 256, 0, st>>>(parts, n, stride, part, (float*)out);
  else
    cross_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(parts, n, stride, part, (__nv_bfloat16*)out);
  return cudaGetLastError();
}

}  // namespace rola
