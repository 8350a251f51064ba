// Dense attention to an encoder's states on the FMA pipe (fp32 products and sums): the fp32
// configuration of cross_attend and of its gradients.
//
//   S = scale q k^T,  P = exp(S - lse),  O = P v
//   D = rowsum(dO * O);  dS = P * (dO v^T - D);  dq = scale dS k;  dk = scale dS^T q;  dv = P^T dO
//
// Tiles of 64 queries x 64 keys, 256 threads as 16 x 16: a thread holds 4 x 4 entries of S (rows
// 4 ty + i, columns tx + 16 j) and 4 rows x d/16 columns of each product, two columns per packed
// FMA.  Rows in shared memory are padded by 16 bytes, so that 16 threads that read 16 rows at the
// same channel touch all banks.  Long axes that too few tiles share are split over blocks: keys
// in the forward and for dq, queries for dk and dv; the parts are joined in a fixed order.
#include "block_internal.cuh"
#include "row_ops.cuh"
#include "sm100_ptx.cuh"

namespace rola {
namespace {

using sm100::fma2;

constexpr int kTile = 64;
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Keys of sample b that may be valid: the first `len`.
__device__ __forceinline__ int key_count(const CrossArgs& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ bool key_valid(const CrossArgs& a, int b, int m, int len) {
  return m < len && (!a.key_mask || __ldg(a.key_mask + (size_t)b * a.Nk + m) != 0);
}

// Rows m0 .. m0 + 63 of head h into a padded tile; rows that `ok` refuses become zeros.
template <typename T, int D, typename F>
__device__ __forceinline__ void load_tile(float* tile, const T* x, const rola_strides& s, int b, int h, int m0,
                                          const F& ok) {
  const T* base = x + b * s.b + h * s.h;
  for (int e = threadIdx.x; e < kTile * D / 4; e += kThreads) {
    const int row = e / (D / 4), c = 4 * (e % (D / 4));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ok(m0 + row)) v = load4(base + (long long)(m0 + row) * s.n + c);
    *reinterpret_cast<float4*>(tile + row * (D + 4) + c) = v;
  }
}

// s[i][j] = a_row(4 ty + i) . b_row(tx + 16 j), over D channels.
template <int D>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int ty, int tx, float (&s)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
  float t[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) t[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * (D + 4) + c);
      y[i] = *reinterpret_cast<const float4*>(b + (tx + 16 * i) * (D + 4) + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // even and odd channels in the two lanes of a packed FMA
        fma2(s[i][j], t[i][j], x[i].x, x[i].y, y[j].x, y[j].y, s[i][j], t[i][j]);
        fma2(s[i][j], t[i][j], x[i].z, x[i].w, y[j].z, y[j].w, s[i][j], t[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] += t[i][j];
}

// acc[i][c] += sum_m p[4 ty + i][m] x[m][cols], cols 4 tx + 64 j.
template <int D>
__device__ __forceinline__ void mul_rows(const float* p, const float* x, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 2
  for (int m = 0; m < kTile; m += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (4 * ty + i) * (kTile + 4) + m);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(x + (m + e) * (D + 4) + 4 * tx + 64 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
          float* o = acc[i] + 4 * j;
          fma2(o[0], o[1], f, f, y.x, y.y, o[0], o[1]);
          fma2(o[2], o[3], f, f, y.z, y.w, o[2], o[3]);
        }
      }
  }
}

// acc[i][c] += sum_q p[q][4 ty + i] x[q][cols]: the transposed product.
template <int D>
__device__ __forceinline__ void mul_cols(const float* p, const float* x, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 4
  for (int q = 0; q < kTile; ++q) {
    const float4 w = *reinterpret_cast<const float4*>(p + q * (kTile + 4) + 4 * ty);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(x + q * (D + 4) + 4 * tx + 64 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        float* o = acc[i] + 4 * j;
        fma2(o[0], o[1], f, f, y.x, y.y, o[0], o[1]);
        fma2(o[2], o[3], f, f, y.z, y.w, o[2], o[3]);
      }
    }
  }
}

// Max / sum over the 16 threads that share a row.
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
struct Tiles {
  static constexpr int kRow = D + 4;
  static constexpr int kX = kTile * kRow;           // floats of a padded q, k, v or dO tile
  static constexpr int kP = kTile * (kTile + 4);    // of a padded P or dS tile
};

// Forward.  grid (q tiles, H * splits, B); split s takes every key tile of its run.  With one
// split `out` and lse are the results; else the split's own softmax in part, plse.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_simt_kernel(const __grid_constant__ CrossArgs a, int splits,
                                                              const T* __restrict__ q, const T* __restrict__ k,
                                                              const T* __restrict__ v, T* __restrict__ out,
                                                              float* __restrict__ lse, float* __restrict__ part,
                                                              float* __restrict__ plse) {
  using L = Tiles<D>;
  extern __shared__ float sm[];
  float *sq = sm, *sk = sq + L::kX, *sv = sk + L::kX, *sp = sv + L::kX;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, q0 = blockIdx.x * kTile;
  const int len = key_count(a, b), tiles = (len + kTile - 1) / kTile;
  const int run = ((a.Nk + kTile - 1) / kTile + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = min(tiles, t0 + run);
  load_tile<T, D>(sq, q, a.q, b, h, q0, [&](int n) { return n < a.Nq; });
  float m[4], l[4], o[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    const int m0 = t * kTile;
    auto ok = [&](int n) { return key_valid(a, b, n, len); };
    __syncthreads();
    load_tile<T, D>(sk, k, a.k, b, h, m0, ok);
    load_tile<T, D>(sv, v, a.v, b, h, m0, ok);
    bool valid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
    __syncthreads();
    float s[4][4];
    dot_tile<D>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = valid[j] ? s[i][j] * a.scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      const float now = fmaxf(m[i], max16(top)), ref = now == -INFINITY ? 0.f : now;
      const float keep = expf(m[i] - ref);
      m[i] = now;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[i][j] - ref);
        sum += p;
        sp[(4 * ty + i) * (kTile + 4) + tx + 16 * j] = p;
      }
      l[i] = l[i] * keep + sum16(sum);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= keep;
    }
    __syncwarp();                      // a row of P is made and read by one half-warp
    mul_rows<D>(sp, sv, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q0 + 4 * ty + i;
    if (n >= a.Nq) continue;
    // a row without a valid key: out 0, lse -inf
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const float z = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    const size_t at = (((size_t)b * a.Nq + n) * a.H + h) * D, zat = ((size_t)b * a.H + h) * a.Nq + n;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 r = make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                                   o[i][4 * j + 3] * inv);
      if (splits == 1)
        store4(out + at + 4 * tx + 64 * j, r);
      else
        store4(part + (size_t)sp_i * a.B * a.Nq * a.H * D + at + 4 * tx + 64 * j, r);
    }
    if (tx == 0) {
      if (splits > 1)
        plse[(size_t)sp_i * a.B * a.H * a.Nq + zat] = z;
      else if (lse)
        lse[zat] = z;
    }
  }
}

// D = rowsum(dO * O), [B, H, Nq]: one warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_rowdot_kernel(const __grid_constant__ CrossArgs a,
                                                           const T* __restrict__ dout, const T* __restrict__ out,
                                                           float* __restrict__ drow) {
  const long long rows = (long long)a.B * a.Nq * a.H;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int h = (int)(row % a.H);
  const long long bn = row / a.H;
  const int b = (int)(bn / a.Nq), n = (int)(bn - (long long)b * a.Nq);
  float s = 0.f;
  const T* x = dout + b * a.dout.b + n * a.dout.n + h * a.dout.h;
  const T* y = out + row * D;
  if (4 * lane < D) {
    const float4 u = load4(x + 4 * lane), w = load4(y + 4 * lane);
    s = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, u.w * w.w)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) drow[((size_t)b * a.H + h) * a.Nq + n] = s;
}

// P and dS of a tile pair (rows of queries, columns of keys) from S and dO v^T.  A row without a
// valid key has lse = -inf: its P is zero, as is that of rows past Nq.
template <int D, bool kNeedP>
__device__ __forceinline__ void score_tile(const CrossArgs& a, const float* sq, const float* sk, const float* sdo,
                                           const float* sv, int q0, const float* lse, const float* drow, size_t zat,
                                           const bool (&valid)[4], int ty, int tx, float* sp, float* sds) {
  float s[4][4], dp[4][4];
  dot_tile<D>(sq, sk, ty, tx, s);
  dot_tile<D>(sdo, sv, ty, tx, dp);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q0 + 4 * ty + i;
    const float z = n < a.Nq ? __ldg(lse + zat + n) : -INFINITY, dr = n < a.Nq ? __ldg(drow + zat + n) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool on = valid[j] && z != -INFINITY;
      const float p = on ? expf(fmaf(s[i][j], a.scale, -z)) : 0.f;
      const int at = (4 * ty + i) * (kTile + 4) + tx + 16 * j;
      if (kNeedP) sp[at] = p;
      sds[at] = on ? p * (dp[i][j] - dr) * a.scale : 0.f;
    }
  }
}

// dq.  grid (q tiles, H * splits, B): keys split as in the forward.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_simt_dq_kernel(
    const __grid_constant__ CrossArgs a, int splits, const T* __restrict__ dout, const T* __restrict__ q,
    const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ lse, const float* __restrict__ drow,
    T* __restrict__ dq, float* __restrict__ part) {
  using L = Tiles<D>;
  extern __shared__ float sm[];
  float *sq = sm, *sdo = sq + L::kX, *sk = sdo + L::kX, *sv = sk + L::kX, *sds = sv + L::kX;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, q0 = blockIdx.x * kTile;
  const int len = key_count(a, b), tiles = (len + kTile - 1) / kTile;
  const int run = ((a.Nk + kTile - 1) / kTile + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = min(tiles, t0 + run);
  const size_t zat = ((size_t)b * a.H + h) * a.Nq;
  auto row = [&](int n) { return n < a.Nq; };
  load_tile<T, D>(sq, q, a.q, b, h, q0, row);
  load_tile<T, D>(sdo, dout, a.dout, b, h, q0, row);
  float acc[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
  for (int t = t0; t < t1; ++t) {
    const int m0 = t * kTile;
    auto ok = [&](int n) { return key_valid(a, b, n, len); };
    __syncthreads();
    load_tile<T, D>(sk, k, a.k, b, h, m0, ok);
    load_tile<T, D>(sv, v, a.v, b, h, m0, ok);
    bool valid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
    __syncthreads();
    score_tile<D, false>(a, sq, sk, sdo, sv, q0, lse, drow, zat, valid, ty, tx, nullptr, sds);
    __syncwarp();                      // a row of dS is made and read by one half-warp
    mul_rows<D>(sds, sk, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q0 + 4 * ty + i;
    if (n >= a.Nq) continue;
    const size_t at = (((size_t)b * a.Nq + n) * a.H + h) * D + 4 * tx;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 r = make_float4(acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]);
      if (splits == 1)
        store4(dq + at + 64 * j, r);
      else
        store4(part + (size_t)sp_i * a.B * a.Nq * a.H * D + at + 64 * j, r);
    }
  }
}

// dk, dv.  grid (key tiles, H * splits, B): split s takes a run of query tiles.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_simt_dkv_kernel(
    const __grid_constant__ CrossArgs a, int splits, const T* __restrict__ dout, const T* __restrict__ q,
    const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ lse, const float* __restrict__ drow,
    T* __restrict__ dk, T* __restrict__ dv, float* __restrict__ part) {
  using L = Tiles<D>;
  extern __shared__ float sm[];
  float *sq = sm, *sdo = sq + L::kX, *sk = sdo + L::kX, *sv = sk + L::kX, *sp = sv + L::kX, *sds = sp + L::kP;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, m0 = blockIdx.x * kTile;
  const int len = key_count(a, b), qtiles = (a.Nq + kTile - 1) / kTile, run = (qtiles + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = m0 < len ? min(qtiles, t0 + run) : t0;   // no valid key: zeros
  const size_t zat = ((size_t)b * a.H + h) * a.Nq;
  auto ok = [&](int n) { return key_valid(a, b, n, len); };
  load_tile<T, D>(sk, k, a.k, b, h, m0, ok);
  load_tile<T, D>(sv, v, a.v, b, h, m0, ok);
  bool valid[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
  float ak[4][D / 16], av[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
  for (int t = t0; t < t1; ++t) {
    const int q0 = t * kTile;
    auto row = [&](int n) { return n < a.Nq; };
    __syncthreads();
    load_tile<T, D>(sq, q, a.q, b, h, q0, row);
    load_tile<T, D>(sdo, dout, a.dout, b, h, q0, row);
    __syncthreads();
    score_tile<D, true>(a, sq, sk, sdo, sv, q0, lse, drow, zat, valid, ty, tx, sp, sds);
    __syncthreads();
    mul_cols<D>(sp, sdo, ty, tx, av);
    mul_cols<D>(sds, sq, ty, tx, ak);
  }
  const size_t total = (size_t)a.B * a.Nk * a.H * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = m0 + 4 * ty + i;
    if (n >= a.Nk) continue;
    const size_t at = (((size_t)b * a.Nk + n) * a.H + h) * D + 4 * tx;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 rk = make_float4(ak[i][4 * j], ak[i][4 * j + 1], ak[i][4 * j + 2], ak[i][4 * j + 3]);
      const float4 rv = make_float4(av[i][4 * j], av[i][4 * j + 1], av[i][4 * j + 2], av[i][4 * j + 3]);
      if (splits == 1) {
        store4(dk + at + 64 * j, rk);
        store4(dv + at + 64 * j, rv);
      } else {
        store4(part + (2 * (size_t)sp_i) * total + at + 64 * j, rk);
        store4(part + (2 * (size_t)sp_i + 1) * total + at + 64 * j, rv);
      }
    }
  }
}

template <typename K>
cudaError_t opt_in(K kern, size_t smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <typename T, int D>
cudaError_t forward(const CrossArgs& a, int splits, const void* q, const void* k, const void* v, void* out, float* lse,
                    float* part, cudaStream_t st) {
  using L = Tiles<D>;
  constexpr size_t smem = sizeof(float) * (3 * L::kX + L::kP);
  cudaError_t e = opt_in(cross_simt_kernel<T, D>, smem);
  if (e != cudaSuccess) return e;
  float* plse = part + (size_t)splits * a.B * a.Nq * a.H * D;
  cross_simt_kernel<T, D><<<dim3((a.Nq + kTile - 1) / kTile, a.H * splits, a.B), kThreads, smem, st>>>(
      a, splits, (const T*)q, (const T*)k, (const T*)v, (T*)out, lse, part, plse);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return launch_cross_join(a, sizeof(T) == 2 ? ROLA_BF16 : ROLA_F32, splits, part, plse, out, lse, st);
}

template <typename T, int D>
cudaError_t backward(const CrossArgs& a, int sq, int sk, const void* dout, const void* q, const void* k, const void* v,
                     const void* out, const float* lse, void* dq, void* dk, void* dv, float* drow, float* part,
                     cudaStream_t st) {
  using L = Tiles<D>;
  constexpr rola_dtype dt = sizeof(T) == 2 ? ROLA_BF16 : ROLA_F32;
  constexpr size_t smem_q = sizeof(float) * (4 * L::kX + L::kP), smem_k = sizeof(float) * (4 * L::kX + 2 * L::kP);
  cudaError_t e = opt_in(cross_simt_dq_kernel<T, D>, smem_q);
  if (e == cudaSuccess) e = opt_in(cross_simt_dkv_kernel<T, D>, smem_k);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.Nq * a.H;
  cross_rowdot_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(a, (const T*)dout, (const T*)out, drow);
  cross_simt_dq_kernel<T, D><<<dim3((a.Nq + kTile - 1) / kTile, a.H * sk, a.B), kThreads, smem_q, st>>>(
      a, sk, (const T*)dout, (const T*)q, (const T*)k, (const T*)v, lse, drow, (T*)dq, part);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t nq = (size_t)rows * D, nk = (size_t)a.B * a.Nk * a.H * D;
  if (sk > 1) {   // the parts are read before dk, dv's take their place (one stream)
    e = launch_cross_sum(dt, sk, nq, nq, part, dq, st);
    if (e != cudaSuccess) return e;
  }
  cross_simt_dkv_kernel<T, D><<<dim3((a.Nk + kTile - 1) / kTile, a.H * sq, a.B), kThreads, smem_k, st>>>(
      a, sq, (const T*)dout, (const T*)q, (const T*)k, (const T*)v, lse, drow, (T*)dk, (T*)dv, part);
  e = cudaGetLastError();
  if (e != cudaSuccess || sq == 1) return e;
  e = launch_cross_sum(dt, sq, nk, 2 * nk, part, dk, st);
  return e != cudaSuccess ? e : launch_cross_sum(dt, sq, nk, 2 * nk, part + nk, dv, st);
}

}  // namespace

cudaError_t launch_cross_simt(const CrossArgs& a, rola_dtype dt, int splits, const void* q, const void* k,
                              const void* v, void* out, float* lse, float* part, cudaStream_t st) {
  if (dt == ROLA_F32)
    return a.d == 64 ? forward<float, 64>(a, splits, q, k, v, out, lse, part, st)
                     : forward<float, 128>(a, splits, q, k, v, out, lse, part, st);
  return a.d == 64 ? forward<__nv_bfloat16, 64>(a, splits, q, k, v, out, lse, part, st)
                   : forward<__nv_bfloat16, 128>(a, splits, q, k, v, out, lse, part, st);
}

cudaError_t launch_cross_simt_backward(const CrossArgs& a, rola_dtype dt, int splits_q, int splits_k, const void* dout,
                                       const void* q, const void* k, const void* v, const void* out, const float* lse,
                                       void* dq, void* dk, void* dv, float* drow, float* part, cudaStream_t st) {
  if (dt == ROLA_F32)
    return a.d == 64
               ? backward<float, 64>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow, part, st)
               : backward<float, 128>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow, part, st);
  return a.d == 64 ? backward<__nv_bfloat16, 64>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow,
                                                 part, st)
                   : backward<__nv_bfloat16, 128>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow,
                                                  part, st);
}

}  // namespace rola
