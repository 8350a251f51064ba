// Dense attention to an encoder's states on the FMA pipe (fp32 products and sums): the fp32
// configuration of cross_attend and of its gradients.
//
//   S = scale q k^T,  P = exp(S - lse),  O = P v
//   D = rowsum(dO * O);  dS = P * (dO v^T - D);  dq = scale dS k;  dk = scale dS^T q;  dv = P^T dO
//
// Tiles of 64 queries x 64 keys, 256 threads as 16 x 16: a thread holds 4 x 4 entries of S (rows
// 4 ty + i, columns tx + 16 j) and 4 rows x d/16 columns of each product, two sums per packed FMA.
// Rows in shared memory are padded by 16 bytes, so that 16 threads that read 16 rows at the same
// channel touch all banks.  A tile's successor is fetched as soon as its last product is done,
// under the products of the other tile.  Long axes that too few tiles share are split over blocks:
// keys in the forward and for dq, queries for dk and dv; the parts are joined in a fixed order.
//
// Measured: 777 x 333 keys, 2 x 3 heads of 64, masked: 24 us and 7 for the join.  Gradients of
// 1000 x 257, 12 heads of 128: D 5 us, dq 100 and 6 for the sum, dk and dv 134 and 2 x 4: 1.5 and
// 2.0 GFMA, 0.41 of the FMA pipe's rate.  What bounds it are the waits of eight warps an SM (four
// tiles of 64 x 128 fill its shared memory) for shared memory and at barriers.
#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;

// Keys of sample b that may be valid: the first `len`.
__device__ __forceinline__ int key_count(const CrossArgs& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ bool key_valid(const CrossArgs& a, int b, int m, int len) {
  return m < len && (!a.key_mask || __ldg(a.key_mask + (size_t)b * a.Nk + m) != 0);
}

// Fetches rows m0 .. m0 + 63 of head h into a padded tile; rows that `ok` refuses become zeros.
template <int D, typename F>
__device__ __forceinline__ void fetch_tile(float* tile, const float* x, const rola_strides& s, int b, int h, int m0,
                                           const F& ok) {
  const float* base = x + b * s.b + h * s.h;
#pragma unroll 4
  for (int e = threadIdx.x; e < kTile * D / 4; e += kThreads) {
    const int row = e / (D / 4), c = 4 * (e % (D / 4));
    const bool on = ok(m0 + row);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_addr(tile + row * (D + 4) + c)),
                 "l"(on ? base + (long long)(m0 + row) * s.n + c : x), "r"(on ? 16 : 0)
                 : "memory");
  }
  copy_commit();
}
// Every thread's copies but the last `keep` tiles' have landed.
template <int keep>
__device__ __forceinline__ void tiles_ready() {
  copy_wait<keep>();
  __syncthreads();
}

__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

// s[i][j] = a_row(4 ty + i) . b_row(tx + 16 j), over D channels.
template <int D>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int ty, int tx, float (&s)[4][4]) {
  float2 t[4][4];                      // even and odd channels
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) t[i][j] = make_float2(0.f, 0.f);
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
      for (int j = 0; j < 4; ++j) {
        t[i][j] = __ffma2_rn(lo2(x[i]), lo2(y[j]), t[i][j]);
        t[i][j] = __ffma2_rn(hi2(x[i]), hi2(y[j]), t[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = t[i][j].x + t[i][j].y;
}

// Sums of a thread: 4 rows x D/16 columns, as pairs: columns 4 tx + 64 j + (0, 1), (2, 3).
template <int D>
struct Acc {
  float2 v[4][D / 32];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) v[i][j] = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void add(int i, float f, int j, const float4& y) {
    const float2 ff = make_float2(f, f);
    v[i][2 * j] = __ffma2_rn(ff, lo2(y), v[i][2 * j]);
    v[i][2 * j + 1] = __ffma2_rn(ff, hi2(y), v[i][2 * j + 1]);
  }
  __device__ __forceinline__ float4 at(int i, int j, float f) const {
    return make_float4(v[i][2 * j].x * f, v[i][2 * j].y * f, v[i][2 * j + 1].x * f, v[i][2 * j + 1].y * f);
  }
};

// acc row i += sum_m p[4 ty + i][m] x[m].
template <int D>
__device__ __forceinline__ void mul_rows(const float* p, const float* x, int ty, int tx, Acc<D>& acc) {
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
        for (int i = 0; i < 4; ++i) acc.add(i, e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w, j, y);
      }
  }
}

// acc row i += sum_q p[q][4 ty + i] x[q]: the transposed product.
template <int D>
__device__ __forceinline__ void mul_cols(const float* p, const float* x, int ty, int tx, Acc<D>& acc) {
#pragma unroll 4
  for (int q = 0; q < kTile; ++q) {
    const float4 w = *reinterpret_cast<const float4*>(p + q * (kTile + 4) + 4 * ty);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(x + q * (D + 4) + 4 * tx + 64 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc.add(i, i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w, j, y);
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
template <int D>
__global__ void __launch_bounds__(kThreads) cross_simt_kernel(const __grid_constant__ CrossArgs a, int splits,
                                                              const float* __restrict__ q,
                                                              const float* __restrict__ k,
                                                              const float* __restrict__ v, float* __restrict__ out,
                                                              float* __restrict__ lse, float* __restrict__ part,
                                                              float* __restrict__ plse) {
  using L = Tiles<D>;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sk = sq + L::kX, *sv = sk + L::kX, *sp = sv + L::kX;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, q0 = blockIdx.x * kTile;
  const int len = key_count(a, b), tiles = (len + kTile - 1) / kTile;
  const int run = ((a.Nk + kTile - 1) / kTile + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = min(tiles, t0 + run);
  auto ok = [&](int n) { return key_valid(a, b, n, len); };
  fetch_tile<D>(sq, q, a.q, b, h, q0, [&](int n) { return n < a.Nq; });
  if (t0 < t1) {
    fetch_tile<D>(sk, k, a.k, b, h, t0 * kTile, ok);
    fetch_tile<D>(sv, v, a.v, b, h, t0 * kTile, ok);
  }
  float m[4], l[4];
  Acc<D> o;
  o.zero();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    const int m0 = t * kTile;
    bool valid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
    tiles_ready<1>();                  // q and K (V may be in flight)
    float s[4][4];
    dot_tile<D>(sq, sk, ty, tx, s);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sk, k, a.k, b, h, m0 + kTile, ok);
    else
      copy_commit();
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
      for (int c = 0; c < D / 32; ++c) o.v[i][c] = __fmul2_rn(o.v[i][c], make_float2(keep, keep));
    }
    tiles_ready<1>();                  // V (the next K may be in flight), and P
    mul_rows<D>(sp, sv, ty, tx, o);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sv, v, a.v, b, h, m0 + kTile, ok);
    else
      copy_commit();
  }
  copy_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q0 + 4 * ty + i;
    if (n >= a.Nq) continue;
    // a row without a valid key: out 0, lse -inf
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const float z = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    const size_t at = (((size_t)b * a.Nq + n) * a.H + h) * D + 4 * tx, zat = ((size_t)b * a.H + h) * a.Nq + n;
    float* dst = splits == 1 ? out + at : part + (size_t)sp_i * a.B * a.Nq * a.H * D + at;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) *reinterpret_cast<float4*>(dst + 64 * j) = o.at(i, j, inv);
    if (tx == 0) {
      if (splits > 1)
        plse[(size_t)sp_i * a.B * a.H * a.Nq + zat] = z;
      else if (lse)
        lse[zat] = z;
    }
  }
}

// D = rowsum(dO * O), [B, H, Nq]: D / 4 threads per row.
template <int D>
__global__ void __launch_bounds__(256) cross_rowdot_kernel(const __grid_constant__ CrossArgs a,
                                                           const float* __restrict__ dout,
                                                           const float* __restrict__ out, float* __restrict__ drow) {
  constexpr int kPer = D / 4;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x, row = e / kPer;
  const int c = 4 * (int)(e - row * kPer), h = (int)(row % a.H);
  const long long bn = row / a.H;
  const int b = (int)(bn / a.Nq), n = (int)(bn - (long long)b * a.Nq);
  float s = 0.f;
  if (b < a.B) {
    const float4 u = *reinterpret_cast<const float4*>(dout + b * a.dout.b + n * a.dout.n + h * a.dout.h + c);
    const float4 w = *reinterpret_cast<const float4*>(out + row * D + c);
    s = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, u.w * w.w)));
  }
#pragma unroll
  for (int o = kPer / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (c == 0 && b < a.B) drow[((size_t)b * a.H + h) * a.Nq + n] = s;
}

// P and dS of a tile pair (rows of queries, columns of keys) from S and dP = dO v^T.  A row without
// a valid key has lse = -inf: its P is zero, as is that of rows past Nq.
struct RowStats {
  float z[4], d[4];
  __device__ __forceinline__ RowStats(const CrossArgs& a, const float* lse, const float* drow, size_t zat, int n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = n0 + i < a.Nq ? __ldg(lse + zat + n0 + i) : -INFINITY;
      d[i] = n0 + i < a.Nq ? __ldg(drow + zat + n0 + i) : 0.f;
    }
  }
};
template <bool kNeedP>
__device__ __forceinline__ void score_tile(const CrossArgs& a, const float (&s)[4][4], const float (&dp)[4][4],
                                           const RowStats& r, const bool (&valid)[4], int ty, int tx, float* sp,
                                           float* sds) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool on = valid[j] && r.z[i] != -INFINITY;
      const float p = on ? expf(fmaf(s[i][j], a.scale, -r.z[i])) : 0.f;
      const int at = (4 * ty + i) * (kTile + 4) + tx + 16 * j;
      if (kNeedP) sp[at] = p;
      sds[at] = on ? p * (dp[i][j] - r.d[i]) * a.scale : 0.f;
    }
}

// dq.  grid (q tiles, H * splits, B): keys split as in the forward.
template <int D>
__global__ void __launch_bounds__(kThreads) cross_simt_dq_kernel(
    const __grid_constant__ CrossArgs a, int splits, const float* __restrict__ dout, const float* __restrict__ q,
    const float* __restrict__ k, const float* __restrict__ v, const float* __restrict__ lse,
    const float* __restrict__ drow, float* __restrict__ dq, float* __restrict__ part) {
  using L = Tiles<D>;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sdo = sq + L::kX, *sk = sdo + L::kX, *sv = sk + L::kX, *sds = sv + L::kX;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, q0 = blockIdx.x * kTile;
  const int len = key_count(a, b), tiles = (len + kTile - 1) / kTile;
  const int run = ((a.Nk + kTile - 1) / kTile + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = min(tiles, t0 + run);
  auto ok = [&](int n) { return key_valid(a, b, n, len); };
  auto row = [&](int n) { return n < a.Nq; };
  const RowStats stats(a, lse, drow, ((size_t)b * a.H + h) * a.Nq, q0 + 4 * ty);
  fetch_tile<D>(sdo, dout, a.dout, b, h, q0, row);
  if (t0 < t1) fetch_tile<D>(sv, v, a.v, b, h, t0 * kTile, ok);
  fetch_tile<D>(sq, q, a.q, b, h, q0, row);
  if (t0 < t1) fetch_tile<D>(sk, k, a.k, b, h, t0 * kTile, ok);
  Acc<D> acc;
  acc.zero();
  for (int t = t0; t < t1; ++t) {
    const int m0 = t * kTile;
    bool valid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
    float s[4][4], dp[4][4];
    if (t == t0)
      tiles_ready<2>();                // dO and V (q and K may be in flight)
    else
      tiles_ready<1>();                // V (K may be in flight)
    dot_tile<D>(sdo, sv, ty, tx, dp);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sv, v, a.v, b, h, m0 + kTile, ok);
    else
      copy_commit();
    tiles_ready<1>();                  // q and K (the next V may be in flight)
    dot_tile<D>(sq, sk, ty, tx, s);
    score_tile<false>(a, s, dp, stats, valid, ty, tx, nullptr, sds);
    __syncwarp();                      // a row of dS is made and read by one half-warp
    mul_rows<D>(sds, sk, ty, tx, acc);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sk, k, a.k, b, h, m0 + kTile, ok);
    else
      copy_commit();
  }
  copy_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = q0 + 4 * ty + i;
    if (n >= a.Nq) continue;
    const size_t at = (((size_t)b * a.Nq + n) * a.H + h) * D + 4 * tx;
    float* dst = splits == 1 ? dq + at : part + (size_t)sp_i * a.B * a.Nq * a.H * D + at;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) *reinterpret_cast<float4*>(dst + 64 * j) = acc.at(i, j, 1.f);
  }
}

// dk, dv.  grid (key tiles, H * splits, B): split s takes a run of query tiles.
template <int D>
__global__ void __launch_bounds__(kThreads) cross_simt_dkv_kernel(
    const __grid_constant__ CrossArgs a, int splits, const float* __restrict__ dout, const float* __restrict__ q,
    const float* __restrict__ k, const float* __restrict__ v, const float* __restrict__ lse,
    const float* __restrict__ drow, float* __restrict__ dk, float* __restrict__ dv, float* __restrict__ part) {
  using L = Tiles<D>;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sdo = sq + L::kX, *sk = sdo + L::kX, *sv = sk + L::kX, *sp = sv + L::kX, *sds = sp + L::kP;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.z, h = blockIdx.y / splits, sp_i = blockIdx.y - h * splits, m0 = blockIdx.x * kTile;
  const int len = key_count(a, b), qtiles = (a.Nq + kTile - 1) / kTile, run = (qtiles + splits - 1) / splits;
  const int t0 = sp_i * run, t1 = m0 < len ? min(qtiles, t0 + run) : t0;   // no valid key: zeros
  const size_t zat = ((size_t)b * a.H + h) * a.Nq;
  auto ok = [&](int n) { return key_valid(a, b, n, len); };
  auto row = [&](int n) { return n < a.Nq; };
  fetch_tile<D>(sv, v, a.v, b, h, m0, ok);
  if (t0 < t1) fetch_tile<D>(sdo, dout, a.dout, b, h, t0 * kTile, row);
  fetch_tile<D>(sk, k, a.k, b, h, m0, ok);
  if (t0 < t1) fetch_tile<D>(sq, q, a.q, b, h, t0 * kTile, row);
  bool valid[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) valid[j] = ok(m0 + tx + 16 * j);
  Acc<D> ak, av;
  ak.zero();
  av.zero();
  for (int t = t0; t < t1; ++t) {
    const int q0 = t * kTile;
    const RowStats stats(a, lse, drow, zat, q0 + 4 * ty);
    float s[4][4], dp[4][4];
    if (t == t0)
      tiles_ready<2>();                // v and dO (k and Q may be in flight)
    else
      tiles_ready<1>();                // dO (Q may be in flight)
    dot_tile<D>(sdo, sv, ty, tx, dp);
    tiles_ready<0>();                  // k and Q
    dot_tile<D>(sq, sk, ty, tx, s);
    score_tile<true>(a, s, dp, stats, valid, ty, tx, sp, sds);
    __syncthreads();
    mul_cols<D>(sp, sdo, ty, tx, av);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sdo, dout, a.dout, b, h, q0 + kTile, row);
    else
      copy_commit();
    mul_cols<D>(sds, sq, ty, tx, ak);
    __syncthreads();
    if (t + 1 < t1)
      fetch_tile<D>(sq, q, a.q, b, h, q0 + kTile, row);
    else
      copy_commit();
  }
  copy_wait<0>();
  const size_t total = (size_t)a.B * a.Nk * a.H * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = m0 + 4 * ty + i;
    if (n >= a.Nk) continue;
    const size_t at = (((size_t)b * a.Nk + n) * a.H + h) * D + 4 * tx;
    float* k_dst = splits == 1 ? dk + at : part + 2 * (size_t)sp_i * total + at;
    float* v_dst = splits == 1 ? dv + at : part + (2 * (size_t)sp_i + 1) * total + at;
    // a key that does not count has sums of 0 * dO and 0 * q, which may be NaN
    const bool counts = ok(n);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      *reinterpret_cast<float4*>(k_dst + 64 * j) = counts ? ak.at(i, j, 1.f) : zero;
      *reinterpret_cast<float4*>(v_dst + 64 * j) = counts ? av.at(i, j, 1.f) : zero;
    }
  }
}

template <typename K>
cudaError_t opt_in(K kern, size_t smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <int D>
cudaError_t forward(const CrossArgs& a, int splits, const float* q, const float* k, const float* v, float* out,
                    float* lse, float* part, cudaStream_t st) {
  using L = Tiles<D>;
  constexpr size_t smem = sizeof(float) * (3 * L::kX + L::kP);
  cudaError_t e = opt_in(cross_simt_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  float* plse = part + (size_t)splits * a.B * a.Nq * a.H * D;
  cross_simt_kernel<D><<<dim3((a.Nq + kTile - 1) / kTile, a.H * splits, a.B), kThreads, smem, st>>>(
      a, splits, q, k, v, out, lse, part, plse);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return launch_cross_join(a, ROLA_F32, splits, part, plse, out, lse, st);
}

template <int D>
cudaError_t backward(const CrossArgs& a, int sq, int sk, const float* dout, const float* q, const float* k,
                     const float* v, const float* out, const float* lse, float* dq, float* dk, float* dv, float* drow,
                     float* part, cudaStream_t st) {
  using L = Tiles<D>;
  constexpr size_t smem_q = sizeof(float) * (4 * L::kX + L::kP), smem_k = sizeof(float) * (4 * L::kX + 2 * L::kP);
  cudaError_t e = opt_in(cross_simt_dq_kernel<D>, smem_q);
  if (e == cudaSuccess) e = opt_in(cross_simt_dkv_kernel<D>, smem_k);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.Nq * a.H;
  cross_rowdot_kernel<D><<<(unsigned)((rows * (D / 4) + 255) / 256), 256, 0, st>>>(a, dout, out, drow);
  cross_simt_dq_kernel<D><<<dim3((a.Nq + kTile - 1) / kTile, a.H * sk, a.B), kThreads, smem_q, st>>>(
      a, sk, dout, q, k, v, lse, drow, dq, part);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t nq = (size_t)rows * D, nk = (size_t)a.B * a.Nk * a.H * D;
  if (sk > 1) {   // the parts are read before dk, dv's take their place (one stream)
    e = launch_cross_sum(ROLA_F32, sk, nq, nq, part, dq, st);
    if (e != cudaSuccess) return e;
  }
  cross_simt_dkv_kernel<D><<<dim3((a.Nk + kTile - 1) / kTile, a.H * sq, a.B), kThreads, smem_k, st>>>(
      a, sq, dout, q, k, v, lse, drow, dk, dv, part);
  e = cudaGetLastError();
  if (e != cudaSuccess || sq == 1) return e;
  e = launch_cross_sum(ROLA_F32, sq, nk, 2 * nk, part, dk, st);
  return e != cudaSuccess ? e : launch_cross_sum(ROLA_F32, sq, nk, 2 * nk, part + nk, dv, st);
}

}  // namespace

cudaError_t launch_cross_simt(const CrossArgs& a, int splits, const float* q, const float* k, const float* v,
                              float* out, float* lse, float* part, cudaStream_t st) {
  return a.d == 64 ? forward<64>(a, splits, q, k, v, out, lse, part, st)
                   : forward<128>(a, splits, q, k, v, out, lse, part, st);
}

cudaError_t launch_cross_simt_backward(const CrossArgs& a, int splits_q, int splits_k, const float* dout,
                                       const float* q, const float* k, const float* v, const float* out,
                                       const float* lse, float* dq, float* dk, float* dv, float* drow, float* part,
                                       cudaStream_t st) {
  return a.d == 64 ? backward<64>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow, part, st)
                   : backward<128>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, drow, part, st);
}

}  // namespace rola
