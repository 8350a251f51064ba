// RMS norm of q and k with rotary positions on three axes, and its gradients.
//
//   u = x * w * rstd,  rstd = 1 / sqrt(mean(x^2) + eps);   y = R(p) u
//   g = R(p)^T dy;  dw = sum over tokens of g * x * rstd;  h = g * w;
//   dx = rstd * (h - x * rstd^2 * mean(h * x))
//
// Bound by memory: every element is read once and written once, so a token's row stays in
// registers between the statistics and the rotation.  A group of warps owns the rows of one
// tensor (q or k); a thread has up to four pieces of E channels, at the same channels of their
// heads (a group's width is a multiple of the head), so that one set of E/2 angles serves them
// all and 1/rms is folded into it.  Angles are formed in fp64 turns, reduced to one turn (exact to
// 2^-53 of the position), then sincospi in fp32: for a grid whose axes fit, once per block into a
// table in shared memory (t + h + w positions instead of t * h * w); else per token, one token
// ahead, by the first threads of the group.
//
// Measured, bf16 with token norm and a grid: 32760 tokens x 40 heads of 128, q and k, 223 us for
// 1.34 GB (6.0 TB/s, 0.92 of a plain copy).  The backward of 12 heads, 131 to 137 us for 0.60 GB
// (0.68 to 0.71 of a copy): there the instructions set the pace, about 430 per warp and row of 512
// channels at 0.6 of the issue slots (unpacking three bf16 operands, the rotation, two dots, two
// sums over the group), with 15 warps an SM at 127 registers and the block's barrier in every row.
// The same with fp32 gradients, 198 us for 0.81 GB (0.62); of 40 heads, 533 us with bf16 gradients
// (0.58) and 570 with fp32 (0.72).  Small calls (2 x 1000 tokens of 2 heads) take the launch's 11 us.
#include <cmath>
#include <type_traits>

#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kAhead = 3;       // token rows in flight per thread
constexpr int kMaxGroups = 4;
constexpr int kThreadsPerSM = 1024;            // resident threads that a grid is sized for
constexpr int kBackThreadsPerSM = 512;         // of the backward with a norm, at 128 registers (1024: 141 us, now 131)
constexpr int kMaxV = 4;                       // pieces of a thread
constexpr int kMaxThreads = 512;                // 8192 channels, pieces of 4
constexpr int kMaxWarps = kMaxThreads / 32;

template <bool kAngles>
struct Shared {
  alignas(16) float2 cs[kAngles ? 3 : 1][kMaxGroups][kAngles ? 64 : 1];   // written one token ahead: three in turn
  alignas(16) float red[2][kMaxGroups][2 * kMaxWarps];
};

// cos and sin of an angle given in turns.
__device__ __forceinline__ float2 cos_sin(double turn) {
  turn -= rint(turn);
  float2 v;
  sincospif(2.f * (float)turn, &v.y, &v.x);
  return v;
}

constexpr int kTableMost = 4096;   // entries: 32 KB
__host__ __device__ inline long long table_entries(const NormRopeArgs& a) {
  const RotArgs& r = a.rot;
  return (long long)r.gt * r.pt + (long long)r.gh * r.ph + (long long)r.gw * (a.d / 2 - r.pt - r.ph);
}

// The table of a grid's angles: axis by axis, [position][pair of the axis].
__device__ __forceinline__ void write_table(const NormRopeArgs& a, float2* tab) {
  const RotArgs& r = a.rot;
  const int pw = a.d / 2 - r.pt - r.ph;
  const int n[3] = {r.gt, r.gh, r.gw}, c[3] = {r.pt, r.ph, pw}, s[3] = {r.st, r.sh, r.sw};
  for (int axis = 0, first = 0; axis < 3; ++axis) {
    for (int e = threadIdx.x; e < n[axis] * c[axis]; e += blockDim.x) {
      const int p = e / c[axis], i = e - p * c[axis];
      tab[e] = cos_sin((double)((long long)p + s[axis]) * r.turns[first + i]);
    }
    tab += n[axis] * c[axis];
    first += c[axis];
  }
}

// A thread's walk over that table: tokens n, n + step, ... of the grid, E/2 pairs from pair c on.
template <int E>
struct Walker {
  int t, y, x, dt, dy, dx;
  int axis[E / 2], at[E / 2];
  __device__ __forceinline__ Walker(const NormRopeArgs& a, int c, int n, int step) {
    const RotArgs& r = a.rot;
    const int hw = r.gh * r.gw;
    t = n / hw, y = n % hw / r.gw, x = n % r.gw;
    dt = step / hw, dy = step % hw / r.gw, dx = step % r.gw;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const int p = c + i;
      axis[i] = p < r.pt ? 0 : p < r.pt + r.ph ? 1 : 2;
      at[i] = axis[i] == 0 ? p : axis[i] == 1 ? r.gt * r.pt + p - r.pt : r.gt * r.pt + r.gh * r.ph + p - r.pt - r.ph;
    }
  }
  __device__ __forceinline__ void load(const NormRopeArgs& a, const float2* tab, float2 (&cs)[E / 2]) const {
    const RotArgs& r = a.rot;
    const int rt = t * r.pt, ry = y * r.ph, rx = x * (a.d / 2 - r.pt - r.ph);
#pragma unroll
    for (int i = 0; i < E / 2; ++i)   // past the grid: not turned
      cs[i] = t < r.gt ? tab[at[i] + (axis[i] == 0 ? rt : axis[i] == 1 ? ry : rx)] : make_float2(1.f, 0.f);
  }
  __device__ __forceinline__ void next(const NormRopeArgs& a) {
    x += dx;
    y += dy;
    t += dt;
    if (x >= a.rot.gw) x -= a.rot.gw, ++y;
    if (y >= a.rot.gh) y -= a.rot.gh, ++t;
  }
};

enum Rot { kNoRot = 0, kPerToken = 1, kTable = 2 };

// The angles of a thread: pairs t and t + threads of the group.
struct Turner {
  double turns[2];
  int axis[2], pair[2];
  __device__ __forceinline__ Turner(const NormRopeArgs& a, int t, int threads) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = t + i * threads;
      pair[i] = c < (a.d >> 1) ? c : -1;
      axis[i] = c < a.rot.pt ? 0 : c < a.rot.pt + a.rot.ph ? 1 : 2;
      turns[i] = pair[i] >= 0 ? a.rot.turns[c] : 0.0;
    }
  }
  // cos and sin of token n's pairs into cs[0 .. d/2)
  __device__ __forceinline__ void write(const NormRopeArgs& a, int b, int n, float2* cs) const {
    if (pair[0] < 0) return;
    const RotArgs& r = a.rot;
    int tt = 0, y = 0, x = 0;
    if (r.pos == ROLA_POS_GRID) {
      const unsigned hw = r.gh * r.gw;
      tt = (unsigned)n / hw;
      const unsigned rem = n - tt * hw;
      y = rem / (unsigned)r.gw;
      x = rem - y * r.gw;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (pair[i] < 0) return;
      long long p;
      if (r.pos == ROLA_POS_GIVEN)
        p = __ldg(r.positions + ((size_t)(r.batched ? b : 0) * a.N + n) * 3 + axis[i]);
      else if (tt >= r.gt)
        p = 0;                         // past the grid: not turned
      else
        p = axis[i] == 0 ? (long long)tt + r.st : axis[i] == 1 ? (long long)y + r.sh : (long long)x + r.sw;
      cs[pair[i]] = cos_sin((double)p * turns[i]);
    }
  }
};

// A piece as E/2 rotary pairs, two fp32 lanes to an instruction.
template <typename T, int E>
__device__ __forceinline__ void read_pairs(const uint8_t* plane, float2 (&v)[E / 2]) {
  float f[E];
  read_piece<E, T>(plane, f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <int E, typename T>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&v)[E / 2]) {
  float f[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
  store_piece<E>(p, f);
}
// v = R u (kBack: R^T u).
template <bool kBack, int P>
__device__ __forceinline__ void rotate(const float2 (&cs)[P], float2 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float c = cs[i].x, s = kBack ? -cs[i].y : cs[i].y;
    v[i] = make_float2(fmaf(v[i].x, c, -v[i].y * s), fmaf(v[i].x, s, v[i].y * c));
  }
}
template <int P>
__device__ __forceinline__ float dot(const float2 (&a)[P], const float2 (&b)[P]) {
  float2 s = __fmul2_rn(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < P; ++i) s = __ffma2_rn(a[i], b[i], s);
  return s.x + s.y;
}
template <int E>
__device__ __forceinline__ void load_turns(const float2* p, float2 (&cs)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; i += 2) {
    const float4 a = *reinterpret_cast<const float4*>(p + i);
    cs[i] = make_float2(a.x, a.y);
    cs[i + 1] = make_float2(a.z, a.w);
  }
}

// Sum over the threads that hold one head's channels (d/E neighbouring lanes: 8, 16 or 32).
template <int E>
__device__ __forceinline__ float head_sum(float v, int d) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  if (d > 8 * E) v += __shfl_xor_sync(0xffffffffu, v, 8);
  if (d > 16 * E) v += __shfl_xor_sync(0xffffffffu, v, 16);
  return v;
}

// The gains of channels c .. c + E - 1 of head h (1 where there are none).
template <int NORM, int P>
__device__ __forceinline__ void load_gain(const NormRopeArgs& a, const float* __restrict__ w, int h, int c,
                                          float2 (&gain)[P]) {
  const float* p = NORM == ROLA_NORM_HEAD ? w + c : w + (size_t)h * a.d + c;
#pragma unroll
  for (int i = 0; i < P; ++i)
    gain[i] = NORM != ROLA_NORM_NONE && h < a.H ? __ldg(reinterpret_cast<const float2*>(p) + i) : make_float2(1.f, 1.f);
}

// grid (token groups, B, q | k).
template <typename T, int E, int NORM, int ROT, int V>
__global__ void __launch_bounds__(E == 4 ? kMaxThreads : 256)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int W, const T* q,
                                                        const T* k, const float* __restrict__ wq,
                                                        const float* __restrict__ wk, T* qo, T* ko) {
  constexpr int P = E / 2;
  constexpr int kRow = V * piece_bytes<E, T>();   // bytes of a row per thread
  __shared__ Shared<ROT == kPerToken> sh;
  extern __shared__ __align__(16) uint8_t ring[];   // [kAhead][V][tensors][threads] pieces
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), b = blockIdx.y, nt = blockDim.x;
  const bool is_k = blockIdx.z;
  const rola_strides si = is_k ? a.k : a.q, so = is_k ? a.ko : a.qo;
  const float* w = is_k ? wk : wq;
  const int h0 = (E * rg.t) >> a.head_shift, c = (E * rg.t) & (a.d - 1), hs = (E * 32 * W) >> a.head_shift;
  const T* src = (is_k ? k : q) + b * si.b + h0 * si.h + c;
  T* dst = (is_k ? ko : qo) + b * so.b + h0 * so.h + c;
  const int64_t hx = hs * si.h, ho = hs * so.h;
  float2 gain[V][P];
#pragma unroll
  for (int j = 0; j < V; ++j) load_gain<NORM>(a, w, h0 + j * hs, c, gain[j]);
  const Turner turner(a, ROT == kPerToken ? rg.t : a.d, 32 * W);
  float2* tab = reinterpret_cast<float2*>(ring + kAhead * kRow * nt);
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? a.H * a.d : a.d);
  const int first = blockIdx.x * G + rg.g, step = gridDim.x * G;
  src += first * si.n;
  dst += first * so.n;
  const int64_t dx = step * si.n, dout = step * so.n;
  unsigned ahead = first;              // the next row to fetch
  auto fetch = [&](int s) {
    if (ahead < (unsigned)a.N) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (h0 + j * hs < a.H) fetch_piece<E>(ring + (s * kRow + j * piece_bytes<E, T>()) * nt, src + j * hx);
    }
    copy_commit();
    ahead += step;
    src += dx;
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(s);
  if (ROT == kPerToken && first < a.N) turner.write(a, b, first, sh.cs[0][rg.g]);
  Walker<E> walk(a, c >> 1, first, step);
  if (ROT == kTable) {
    write_table(a, tab);
    __syncthreads();
  }
  int slot = 0, turn = 0, it = 0;
  for (long long n = first; n < a.N; n += step, ++it) {
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    copy_wait<kAhead - 1>();
    float2 x[V][P];
    float sum = 0.f, rms[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool on = h0 + j * hs < a.H;
      read_pairs<T, E>(ring + (slot * kRow + j * piece_bytes<E, T>()) * nt, x[j]);
      const float s = NORM != ROLA_NORM_NONE && on ? dot(x[j], x[j]) : 0.f;
      sum += s;
      if (NORM == ROLA_NORM_HEAD) rms[j] = rsqrtf(fmaf(head_sum<E>(s, a.d), inv, a.eps));
    }
    const int next = turn == 2 ? 0 : turn + 1;
    if (ROT == kPerToken && n + step < a.N) turner.write(a, b, (int)(n + step), sh.cs[next][rg.g]);
    float unit = 1.f;
    if (NORM == ROLA_NORM_TOKEN)
      unit = rsqrtf(fmaf(group_sum(rg, sum, sh.red[it & 1][rg.g]), inv, a.eps));
    else if (ROT == kPerToken)
      rg.sync();
    float2 cs[P];
    if (ROT) {
      if (ROT == kTable) {
        walk.load(a, tab, cs);
        walk.next(a);
      } else {
        load_turns<E>(sh.cs[turn][rg.g] + (c >> 1), cs);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) cs[i] = make_float2(cs[i].x * unit, cs[i].y * unit);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (h0 + j * hs >= a.H) continue;
      const float f = (NORM == ROLA_NORM_HEAD ? rms[j] : 1.f) * (ROT ? 1.f : unit);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (NORM != ROLA_NORM_NONE) x[j][i] = __fmul2_rn(x[j][i], gain[j][i]);
        if (NORM == ROLA_NORM_HEAD || (NORM == ROLA_NORM_TOKEN && !ROT))
          x[j][i] = __fmul2_rn(x[j][i], make_float2(f, f));
      }
      if (ROT) rotate<false>(cs, x[j]);
      store_pairs<E>(dst + j * ho, x[j]);
    }
    dst += dout;
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    turn = next;
  }
  copy_wait<0>();
}

// Backward.  dq, dk are contiguous.  part: [gridDim.x * B * G][2][H * d] partial sums of dw.
template <typename T, typename TG, int E, int NORM, int ROT, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_rope_backward_kernel(
    const __grid_constant__ NormRopeArgs a, int W, const TG* dqo, const TG* dko, const T* __restrict__ q,
    const T* __restrict__ k, const float* __restrict__ wq, const float* __restrict__ wk, T* dq, T* dk,
    float* __restrict__ part) {
  constexpr int P = E / 2;
  constexpr int kBg = piece_bytes<E, TG>(), kBx = NORM == ROLA_NORM_NONE ? 0 : piece_bytes<E, T>();
  constexpr int kRow = V * (kBg + kBx);            // bytes of a row per thread
  __shared__ Shared<ROT == kPerToken> sh;
  extern __shared__ __align__(16) uint8_t ring[];   // [kAhead][V][tensors][threads] pieces
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), b = blockIdx.y, nt = blockDim.x, C = a.H * a.d;
  const bool is_k = blockIdx.z;
  const rola_strides si = is_k ? a.k : a.q, su = is_k ? a.ko : a.qo;
  const float* w = is_k ? wk : wq;
  const int h0 = (E * rg.t) >> a.head_shift, c = (E * rg.t) & (a.d - 1), hs = (E * 32 * W) >> a.head_shift;
  const T* src = NORM == ROLA_NORM_NONE ? nullptr : (is_k ? k : q) + b * si.b + h0 * si.h + c;
  const TG* up = (is_k ? dko : dqo) + b * su.b + h0 * su.h + c;
  const int64_t hx = hs * si.h, hu = hs * su.h;
  T* dst = (is_k ? dk : dq) + ((size_t)b * a.N * a.H + h0) * a.d + c;
  float2 gain[V][P], acc[V][P];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    load_gain<NORM>(a, w, h0 + j * hs, c, gain[j]);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[j][i] = make_float2(0.f, 0.f);
  }
  const Turner turner(a, ROT == kPerToken ? rg.t : a.d, 32 * W);
  float2* tab = reinterpret_cast<float2*>(ring + kAhead * kRow * nt);
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? C : a.d);
  const int first = blockIdx.x * G + rg.g, step = gridDim.x * G;
  const int64_t dx = step * si.n, du = step * su.n, dout = (int64_t)step * C;
  const int64_t ho = (int64_t)hs * a.d;
  if (NORM != ROLA_NORM_NONE) src += first * si.n;
  up += first * su.n;
  dst += (int64_t)first * C;
  unsigned ahead = first;              // the next row to fetch
  auto fetch = [&](int s) {
    if (ahead < (unsigned)a.N) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (h0 + j * hs < a.H) {
          uint8_t* at = ring + (s * kRow + j * (kBg + kBx)) * nt;
          fetch_piece<E>(at, up + j * hu);
          if (NORM != ROLA_NORM_NONE) fetch_piece<E>(at + kBg * nt, src + j * hx);
        }
    }
    copy_commit();
    ahead += step;
    up += du;
    if (NORM != ROLA_NORM_NONE) src += dx;
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(s);
  if (ROT == kPerToken && first < a.N) turner.write(a, b, first, sh.cs[0][rg.g]);
  Walker<E> walk(a, c >> 1, first, step);
  if (ROT == kTable) {
    write_table(a, tab);
    __syncthreads();
  }
  if (ROT == kPerToken) rg.sync();
  int slot = 0, turn = 0, it = 0;
  for (long long n = first; n < a.N; n += step, ++it) {
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    copy_wait<kAhead - 1>();
    float2 cs[P];
    if (ROT == kTable) {
      walk.load(a, tab, cs);
      walk.next(a);
    } else if (ROT) {
      load_turns<E>(sh.cs[turn][rg.g] + (c >> 1), cs);
    }
    float2 g[V][P];
    float s0 = 0.f, s1 = 0.f, r[V], m[V];   // sums of x^2 and of h x;  r = 1/rms, m = mean(h x r)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool on = h0 + j * hs < a.H;
      const uint8_t* at = ring + (slot * kRow + j * (kBg + kBx)) * nt;
      read_pairs<TG, E>(at, g[j]);
      if (ROT) rotate<true>(cs, g[j]);
      if (NORM != ROLA_NORM_NONE) {
        float2 x[P], h[P];             // x is read again below: cheaper than V x E more registers
        read_pairs<T, E>(at + kBg * nt, x);
        const float t0 = on ? dot(x, x) : 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) h[i] = __fmul2_rn(g[j][i], gain[j][i]);
        const float t1 = on ? dot(h, x) : 0.f;
        s0 += t0;
        s1 += t1;
        if (NORM == ROLA_NORM_HEAD) {
          r[j] = rsqrtf(fmaf(head_sum<E>(t0, a.d), inv, a.eps));
          m[j] = head_sum<E>(t1, a.d) * inv * r[j];
        }
      }
    }
    const int next = turn == 2 ? 0 : turn + 1;
    if (ROT == kPerToken && n + step < a.N) turner.write(a, b, (int)(n + step), sh.cs[next][rg.g]);
    if (NORM == ROLA_NORM_TOKEN) {
      const float2 s = group_sum(rg, s0, s1, sh.red[it & 1][rg.g]);
      if (ROT == kPerToken && W == 1) __syncwarp();
      r[0] = rsqrtf(fmaf(s.x, inv, a.eps));
      m[0] = s.y * inv * r[0];
#pragma unroll
      for (int j = 1; j < V; ++j) r[j] = r[0], m[j] = m[0];
    } else if (ROT == kPerToken) {
      rg.sync();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (h0 + j * hs >= a.H) continue;
      if (NORM != ROLA_NORM_NONE) {
        float2 x[P];
        read_pairs<T, E>(ring + (slot * kRow + j * (kBg + kBx) + kBg) * nt, x);
        const float2 rr = make_float2(r[j], r[j]), mm = make_float2(-m[j], -m[j]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 xh = __fmul2_rn(x[i], rr);               // x / rms
          acc[j][i] = __ffma2_rn(g[j][i], xh, acc[j][i]);
          g[j][i] = __fmul2_rn(__ffma2_rn(xh, mm, __fmul2_rn(g[j][i], gain[j][i])), rr);
        }
      }
      store_pairs<E>(dst + j * ho, g[j]);
    }
    dst += dout;
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    turn = next;
  }
  copy_wait<0>();
  if (NORM != ROLA_NORM_NONE) {
    const size_t group = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * G + rg.g;
    float* p = part + (group * 2 + is_k) * C + (size_t)h0 * a.d + c;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (h0 + j * hs < a.H) store_floats<E>(p + (size_t)j * hs * a.d, &acc[j][0].x);
  }
}

// dw of q and k (blockIdx.y) from the partial sums; per head, over the heads too.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int parts, int C, int cols,
                                                            float* __restrict__ dwq, float* __restrict__ dwk) {
  column_sum(part + (size_t)blockIdx.y * C, parts, 2 * (size_t)C, cols, C / cols, blockIdx.y ? dwk : dwq);
}

// Blocks of token groups: the SMs full with the rows of both tensors and all samples.
int token_blocks(const RowShape& s, int B, int N, int tensors, int per_sm = kThreadsPerSM) {
  const long long fill = (long long)kRowSMs * (per_sm / s.threads);
  long long x = (fill + (long long)B * tensors - 1) / ((long long)B * tensors);
  const long long most = ((long long)N + s.G - 1) / s.G;
  return (int)(x < most ? x : most);
}

// Backward: a thread's sums of dw stay in registers, so half as many channels per thread.
RowShape backward_shape(int C, int E) { return row_shape(C, E, 16 / E, kMaxWarps); }

// The most dynamic shared memory of an instance: the widest block's ring, and the largest table.
template <int ROT>
constexpr size_t most_smem(int row_bytes) {
  return (size_t)kAhead * row_bytes * kMaxThreads + (ROT == kTable ? sizeof(float2) * kTableMost : 0);
}

// The table pays where the blocks' copies of it hold fewer angles than their tokens (backward of
// 32760 tokens of 12 heads on a 21 x 30 x 52 grid, 2184 entries: 141 us with it, 154 without; 40
// heads forward: 223 and 232).
bool use_table(const NormRopeArgs& a, int blocks) {
  if (a.rot.pos != ROLA_POS_GRID) return false;
  const long long n = table_entries(a);
  return n <= kTableMost && n * blocks <= (long long)a.N * (a.d / 2);
}

// Channels of a piece.
template <typename... Ts>
constexpr int kE = (std::is_same_v<Ts, float> || ...) ? 4 : 8;

template <typename T, int NORM, int ROT, int V>
cudaError_t forward_v(const NormRopeArgs& a, const RowShape& s, const void* q, const void* k, const float* wq,
                      const float* wk, void* qo, void* ko, cudaStream_t st) {
  constexpr int kRow = V * piece_bytes<kE<T>, T>();
  constexpr size_t kMost = most_smem<ROT>(kRow);
  static_assert(kMost + sizeof(Shared<ROT == kPerToken>) <= kMostSharedMemory, "the widest rows fit");
  const size_t smem = (size_t)kAhead * kRow * s.threads + (ROT == kTable ? sizeof(float2) * table_entries(a) : 0);
  const int tensors = k ? 2 : 1;
  cudaError_t e = allow_shared_memory<kMost>(norm_rope_kernel<T, kE<T>, NORM, ROT, V>, smem);
  if (e != cudaSuccess) return e;
  norm_rope_kernel<T, kE<T>, NORM, ROT, V>
      <<<dim3(token_blocks(s, a.B, a.N, tensors), a.B, tensors), s.threads, smem, st>>>(
          a, s.W, (const T*)q, (const T*)k, wq, wk, (T*)qo, (T*)ko);
  return cudaGetLastError();
}

template <typename T, int NORM>
cudaError_t forward(const NormRopeArgs& a, const void* q, const void* k, const float* wq, const float* wk, void* qo,
                    void* ko, cudaStream_t st) {
  const RowShape s = row_shape(a.H * a.d, kE<T>, kMaxV, kMaxWarps);
  auto go = [&](auto rot) {
    constexpr int R = decltype(rot)::value;
    return s.V == 1   ? forward_v<T, NORM, R, 1>(a, s, q, k, wq, wk, qo, ko, st)
           : s.V == 2 ? forward_v<T, NORM, R, 2>(a, s, q, k, wq, wk, qo, ko, st)
                      : forward_v<T, NORM, R, 4>(a, s, q, k, wq, wk, qo, ko, st);
  };
  if (a.rot.pos == ROLA_POS_NONE) return go(std::integral_constant<int, kNoRot>{});
  return use_table(a, token_blocks(s, a.B, a.N, k ? 2 : 1)) ? go(std::integral_constant<int, kTable>{})
                                                            : go(std::integral_constant<int, kPerToken>{});
}

template <int NORM>
int back_blocks(const RowShape& s, int B, int N, int tensors) {
  return token_blocks(s, B, N, tensors, NORM == ROLA_NORM_NONE ? kThreadsPerSM : kBackThreadsPerSM);
}

template <typename T, typename TG, int NORM, int ROT, int V>
cudaError_t backward_v(const NormRopeArgs& a, const RowShape& s, const void* dqo, const void* dko, const void* q,
                       const void* k, const float* wq, const float* wk, void* dq, void* dk, float* dwq, float* dwk,
                       float* part, cudaStream_t st) {
  constexpr int E = kE<T, TG>;
  constexpr int kRow = V * (piece_bytes<E, TG>() + (NORM ? piece_bytes<E, T>() : 0));
  constexpr size_t kMost = most_smem<ROT>(kRow);
  static_assert(kMost + sizeof(Shared<ROT == kPerToken>) <= kMostSharedMemory, "the widest rows fit");
  const size_t smem = (size_t)kAhead * kRow * s.threads + (ROT == kTable ? sizeof(float2) * table_entries(a) : 0);
  const int tensors = dko ? 2 : 1, C = a.H * a.d, blocks = back_blocks<NORM>(s, a.B, a.N, tensors);
  cudaError_t e = allow_shared_memory<kMost>(norm_rope_backward_kernel<T, TG, E, NORM, ROT, V>, smem);
  if (e != cudaSuccess) return e;
  norm_rope_backward_kernel<T, TG, E, NORM, ROT, V><<<dim3(blocks, a.B, tensors), s.threads, smem, st>>>(
      a, s.W, (const TG*)dqo, (const TG*)dko, (const T*)q, (const T*)k, wq, wk, (T*)dq, (T*)dk, part);
  e = cudaGetLastError();
  if (e != cudaSuccess || NORM == ROLA_NORM_NONE) return e;
  const int cols = NORM == ROLA_NORM_HEAD ? a.d : C;
  norm_rope_dw_kernel<<<dim3((cols + kSumCols - 1) / kSumCols, tensors), dim3(kSumCols, kSumRows), 0, st>>>(
      part, blocks * a.B * s.G, C, cols, dwq, dwk);
  return cudaGetLastError();
}

template <typename T, typename TG, int NORM>
cudaError_t backward(const NormRopeArgs& a, const void* dqo, const void* dko, const void* q, const void* k,
                     const float* wq, const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                     cudaStream_t st) {
  const RowShape s = backward_shape(a.H * a.d, kE<T, TG>);
  auto go = [&](auto rot) {
    constexpr int R = decltype(rot)::value;
    if constexpr (kE<T, TG> == 4)
      if (s.V == 4)
        return backward_v<T, TG, NORM, R, 4>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
    return s.V == 1 ? backward_v<T, TG, NORM, R, 1>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st)
                    : backward_v<T, TG, NORM, R, 2>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  };
  if (a.rot.pos == ROLA_POS_NONE) return go(std::integral_constant<int, kNoRot>{});
  return use_table(a, back_blocks<NORM>(s, a.B, a.N, dko ? 2 : 1)) ? go(std::integral_constant<int, kTable>{})
                                                                   : go(std::integral_constant<int, kPerToken>{});
}

template <typename T, typename TG, typename... A>
cudaError_t backward_norm(rola_qk_norm norm, const A&... x) {
  if (norm == ROLA_NORM_NONE) return backward<T, TG, ROLA_NORM_NONE>(x...);
  if (norm == ROLA_NORM_TOKEN) return backward<T, TG, ROLA_NORM_TOKEN>(x...);
  return backward<T, TG, ROLA_NORM_HEAD>(x...);
}
template <typename T, typename... A>
cudaError_t forward_norm(rola_qk_norm norm, const A&... x) {
  if (norm == ROLA_NORM_NONE) return forward<T, ROLA_NORM_NONE>(x...);
  if (norm == ROLA_NORM_TOKEN) return forward<T, ROLA_NORM_TOKEN>(x...);
  return forward<T, ROLA_NORM_HEAD>(x...);
}

}  // namespace

int norm_rope_parts(int B, int N, int C, int tensors) {
  int most = 0;
  for (int e : {4, 8}) {               // for either type of piece
    const RowShape s = backward_shape(C, e);
    const int n = back_blocks<ROLA_NORM_TOKEN>(s, B, N, tensors) * B * s.G;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, rola_dtype dt, rola_qk_norm norm, const void* q, const void* k,
                             const float* wq, const float* wk, void* qo, void* ko, cudaStream_t st) {
  if (dt == ROLA_F32) return forward_norm<float>(norm, a, q, k, wq, wk, qo, ko, st);
  return forward_norm<__nv_bfloat16>(norm, a, q, k, wq, wk, qo, ko, st);
}

cudaError_t launch_norm_rope_backward(const NormRopeArgs& a, rola_dtype dt, rola_dtype gdt, rola_qk_norm norm,
                                      const void* dqo, const void* dko, const void* q, const void* k, const float* wq,
                                      const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                                      cudaStream_t st) {
  if (dt == ROLA_F32) return backward_norm<float, float>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  if (gdt == ROLA_F32)
    return backward_norm<__nv_bfloat16, float>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  return backward_norm<__nv_bfloat16, __nv_bfloat16>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
}

}  // namespace rola
