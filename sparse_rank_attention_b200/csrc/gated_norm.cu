// Gated residual with the modulated norm of the sum, and its gradients.
//
//   r = x + gate * branch;  xhat = (r - mean) * rstd  (or r * rstd);  y = xhat * A + B
//   with A, B = 1 + scale, shift  or  weight, bias.
//   g = dy * A;  dx = dr + rstd * (g - mean(g) - xhat * mean(g * xhat))  (rms: no mean(g))
//   dbranch = gate * dx;  dgate = sum dx * branch;  dA = sum dy * xhat;  dB = sum dy,
//   the sums over the tokens that share a row of the modulation (all tokens for weight, bias).
//
// Bound by memory: each tensor is read or written once.  A group of warps owns a token, a
// thread the same 8 channels of every token it meets, so that the modulation stays in registers
// while the tokens share it and the column sums of the backward are private to a thread.  The
// variance is taken about the mean of the values held in registers (a second sum, not
// E[x^2] - E[x]^2, which loses everything when the mean is large).
#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kThreadsPerSM = 1536;   // resident threads that the forward's grid is sized for
constexpr int kGroupsMost = 8;
constexpr int kRed = kMaxRowWarps * 2 + kGroupsMost * 2;

__device__ __forceinline__ void load8f(const float* p, float* v) {
  Raw8<float> r;
  r.load(p);
  r.get(v);
}

template <typename TX, typename TY, bool LAYER>
__global__ void __launch_bounds__(1024) gated_norm_kernel(const __grid_constant__ GatedNormArgs a, int W,
                                                          const TX* x, const TY* __restrict__ branch,
                                                          const float* __restrict__ gate,
                                                          const float* __restrict__ scale,
                                                          const float* __restrict__ shift,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ bias, TX* r, TY* __restrict__ y) {
  __shared__ float red[2][kRed];
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W);
  const int c = kVec * rg.t;
  const bool on = c < a.C;
  const long long rows = (long long)a.B * a.N, step = (long long)gridDim.x * G;
  const float inv = 1.f / a.C;
  float mg[kVec], ma[kVec], mb[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    mg[i] = 1.f;
    ma[i] = weight && on ? __ldg(weight + c + i) : 1.f;
    mb[i] = bias && on ? __ldg(bias + c + i) : 0.f;
  }
  long long held = -1;                 // the modulation row in registers
  Raw8<TX> nx;
  Raw8<TY> nb;
  nx.zero();
  nb.zero();
  auto fetch = [&](long long row) {
    if (row < rows && on) {
      nx.load(x + row * a.C + c);
      if (branch) nb.load(branch + row * a.C + c);
    }
  };
  long long row = (long long)blockIdx.x * G + rg.g;
  fetch(row);
  for (; row < rows; row += step) {
    const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N), t = n / a.per;
    const long long mod = (long long)b * a.T + t;
    if (mod != held && on) {
      held = mod;
      if (gate) load8f(gate + b * a.gate_b + t * a.gate_t + c, mg);
      if (scale) {
        load8f(scale + b * a.scale_b + t * a.scale_t + c, ma);
        load8f(shift + b * a.shift_b + t * a.shift_t + c, mb);
#pragma unroll
        for (int i = 0; i < kVec; ++i) ma[i] += 1.f;
      }
    }
    float v[kVec], u[kVec];
    nx.get(v);
    nb.get(u);
    fetch(row + step);
    if (branch) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = fmaf(mg[i], u[i], v[i]);
      if (on) store8(r + row * a.C + c, v);
    }
    if (LAYER) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < kVec; ++i) s[0] += v[i];
      group_sum<1>(rg, s, red[0] + rg.g * (W + 1));
      const float mean = s[0] * inv;
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = on ? v[i] - mean : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kVec; ++i) s[0] = fmaf(v[i], v[i], s[0]);
    group_sum<1>(rg, s, red[1] + rg.g * (W + 1));
    if (!LAYER) rg.sync();             // red[1] is written again by the next row
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    if (on) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = fmaf(v[i] * rstd, ma[i], mb[i]);
      store8(y + row * a.C + c, v);
    }
  }
}

// A group takes one segment after the other: a chunk of the tokens that share a modulation
// row.  A segment's column sums go to msum, [segments][3][C] (dgate, dscale, dshift): the
// gradients themselves where a modulation row is one segment (outputs given), else partial
// sums.  The sums of weight and bias run over all segments of the group: wsum [groups][2][C].
template <typename TX, typename TY, bool LAYER>
__global__ void __launch_bounds__(1024) gated_norm_backward_kernel(
    const __grid_constant__ GatedNormArgs a, int W, const TY* __restrict__ dy, const TX* dr,
    const TX* __restrict__ r, const TY* __restrict__ branch, const float* __restrict__ gate,
    const float* __restrict__ scale, const float* __restrict__ weight, TX* dx, TY* __restrict__ dbranch,
    float* __restrict__ dgate, float* __restrict__ dscale, float* __restrict__ dshift, int64_t sum_stride,
    float* __restrict__ wsum) {
  __shared__ float red[2][kRed];
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W);
  const int c = kVec * rg.t;
  const bool on = c < a.C;
  const float inv = 1.f / a.C;
  const long long segs = (long long)a.B * a.T * a.chunks, groups = (long long)gridDim.x * G;
  const long long group = (long long)blockIdx.x * G + rg.g;
  float mg[kVec], ma[kVec], sg[kVec], sa[kVec], sb[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    mg[i] = 1.f;
    ma[i] = weight && on ? __ldg(weight + c + i) : 1.f;
    sg[i] = sa[i] = sb[i] = 0.f;
  }
  for (long long seg = group; seg < segs; seg += groups) {
    const int mod = (int)(seg / a.chunks), ch = (int)(seg - (long long)mod * a.chunks);
    const int b = mod / a.T, t = mod - b * a.T;
    const int n0 = t * a.per + ch * a.chunk, n1 = min(n0 + a.chunk, (t + 1) * a.per);
    if (on) {
      if (gate) load8f(gate + b * a.gate_b + t * a.gate_t + c, mg);
      if (scale) {
        load8f(scale + b * a.scale_b + t * a.scale_t + c, ma);
#pragma unroll
        for (int i = 0; i < kVec; ++i) ma[i] += 1.f;
      }
    }
    for (int n = n0; n < n1; ++n) {
      const size_t at = ((size_t)b * a.N + n) * a.C + c;
      Raw8<TX> xr, xd;
      Raw8<TY> xy, xb;
      xr.zero(); xd.zero(); xy.zero(); xb.zero();
      if (on) {
        xr.load(r + at);
        xy.load(dy + at);
        if (dr) xd.load(dr + at);
        if (branch) xb.load(branch + at);
      }
      float v[kVec], g[kVec], d[kVec];
      xr.get(v);
      xy.get(d);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        g[i] = d[i] * ma[i];
        s[0] += v[i];
        s[1] += g[i];
      }
      float gm = 0.f;
      if (LAYER) {
        group_sum<2>(rg, s, red[0] + rg.g * (W + 1) * 2);
        const float mean = s[0] * inv;
        gm = s[1] * inv;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = on ? v[i] - mean : 0.f;
      }
      float q[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        q[0] = fmaf(v[i], v[i], q[0]);
        q[1] = fmaf(g[i], v[i], q[1]);
      }
      group_sum<2>(rg, q, red[1] + rg.g * (W + 1) * 2);
      if (!LAYER) rg.sync();           // red[1] is written again by the next row
      const float rstd = rsqrtf(fmaf(q[0], inv, a.eps));
      const float proj = q[1] * inv * rstd;          // mean(g * xhat)
      float o[kVec], e[kVec];
      xd.get(o);
      xb.get(e);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float xh = v[i] * rstd;
        sa[i] = fmaf(d[i], xh, sa[i]);
        sb[i] += d[i];
        o[i] = fmaf(rstd, g[i] - gm - xh * proj, o[i]);
        sg[i] = fmaf(o[i], e[i], sg[i]);
      }
      if (on) {
        store8(dx + at, o);
        if (branch) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) o[i] *= mg[i];
          store8(dbranch + at, o);
        }
      }
    }
    if (on && gate) {
      store8(dgate + seg * sum_stride + c, sg);
#pragma unroll
      for (int i = 0; i < kVec; ++i) sg[i] = 0.f;
    }
    if (on && scale) {
      store8(dscale + seg * sum_stride + c, sa);
      store8(dshift + seg * sum_stride + c, sb);
#pragma unroll
      for (int i = 0; i < kVec; ++i) sa[i] = sb[i] = 0.f;
    }
  }
  if (weight && on) {
    store8(wsum + group * 2 * a.C + c, sa);
    store8(wsum + (group * 2 + 1) * a.C + c, sb);
  }
}

// out_z[c] = sum over `parts` consecutive partial rows; a partial row holds `sums` vectors of C
// (blockIdx.y picks one and its output), gridDim.z output rows.  Fixed order: 8 threads take
// every eighth part, then their sums in order.
__global__ void __launch_bounds__(256) gated_norm_reduce_kernel(const float* __restrict__ part, long long parts,
                                                                int sums, int C, float* o0, float* o1, float* o2) {
  __shared__ float sum[8][32];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  const float* p = part + ((size_t)blockIdx.z * parts * sums + blockIdx.y) * C;
  float s = 0.f;
  if (c < C)
    for (long long i = y; i < parts; i += 8) s += p[(size_t)i * sums * C + c];
  sum[y][threadIdx.x] = s;
  __syncthreads();
  if (y == 0 && c < C) {
    for (int i = 1; i < 8; ++i) s += sum[i][threadIdx.x];
    out[(size_t)blockIdx.z * C + c] = s;
  }
}

template <typename TX, typename TY>
cudaError_t forward(const GatedNormArgs& a, rola_norm_kind kind, const void* x, const void* branch, const float* gate,
                    const float* scale, const float* shift, const float* weight, const float* bias, void* r, void* y,
                    cudaStream_t st) {
  const RowShape s = row_shape((long long)a.B * a.N, a.C, kThreadsPerSM);
  auto* kern = kind == ROLA_LAYER ? gated_norm_kernel<TX, TY, true> : gated_norm_kernel<TX, TY, false>;
  kern<<<s.blocks, s.threads, 0, st>>>(a, s.W, (const TX*)x, (const TY*)branch, gate, scale, shift, weight, bias,
                                       (TX*)r, (TY*)y);
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t backward(const GatedNormArgs& a, rola_norm_kind kind, const void* dy, const void* dr, const void* r,
                     const void* branch, const float* gate, const float* scale, const float* weight, void* dx,
                     void* dbranch, float* dgate, float* dscale, float* dshift, float* dweight, float* dbias,
                     float* part, cudaStream_t st) {
  const RowShape s = row_shape((long long)a.B * a.T * a.chunks, a.C, kThreadsPerSM);
  auto* kern = kind == ROLA_LAYER ? gated_norm_backward_kernel<TX, TY, true> : gated_norm_backward_kernel<TX, TY, false>;
  const long long mods = (long long)a.B * a.T;
  const bool direct = a.chunks == 1;   // a segment's sums are the gradients
  float* msum = part;
  float* wsum = part + (direct || !(gate || scale) ? 0 : mods * a.chunks * 3 * a.C);
  kern<<<s.blocks, s.threads, 0, st>>>(
      a, s.W, (const TY*)dy, (const TX*)dr, (const TX*)r, (const TY*)branch, gate, scale, weight, (TX*)dx,
      (TY*)dbranch, direct ? dgate : msum, direct ? dscale : msum + a.C, direct ? dshift : msum + 2 * a.C,
      (direct ? 1 : 3) * (int64_t)a.C, wsum);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned cols = (a.C + 31) / 32;
  for (long long z = 0; z < mods && !direct && (gate || scale); z += 65535) {
    const long long left = mods - z < 65535 ? mods - z : 65535;
    auto at = [&](float* p) { return p ? p + z * a.C : nullptr; };
    gated_norm_reduce_kernel<<<dim3(cols, 3, (unsigned)left), dim3(32, 8), 0, st>>>(
        msum + z * a.chunks * 3 * a.C, a.chunks, 3, a.C, at(dgate), at(dscale), at(dshift));
  }
  if (weight)
    gated_norm_reduce_kernel<<<dim3(cols, 2, 1), dim3(32, 8), 0, st>>>(wsum, (long long)s.blocks * s.G, 2, a.C, dweight,
                                                                     dbias, nullptr);
  return cudaGetLastError();
}

}  // namespace

// Chunks of the tokens that share a modulation row: a segment for every group of a full grid,
// and no more (each costs a row of partial sums).
void gated_norm_chunks(const rola_gated_norm_params& p, int* chunks, int* chunk) {
  const RowShape s = row_shape((long long)p.B * p.N, p.C, kThreadsPerSM);
  const int per = p.N / p.T;
  const long long mods = (long long)p.B * p.T;
  long long want = ((long long)s.blocks * s.G + mods - 1) / mods;
  if (want > per) want = per;
  *chunk = (int)((per + want - 1) / want);
  *chunks = (per + *chunk - 1) / *chunk;
}

size_t gated_norm_workspace(const rola_gated_norm_params& p) {
  int chunks, chunk;
  gated_norm_chunks(p, &chunks, &chunk);
  const long long segs = (long long)p.B * p.T * chunks;
  const RowShape s = row_shape(segs, p.C, kThreadsPerSM);
  return sizeof(float) * (size_t)p.C * ((chunks > 1 ? 3 * segs : 0) + 2 * (long long)s.blocks * s.G);
}

cudaError_t launch_gated_norm(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind, const void* x,
                              const void* branch, const float* gate, const float* scale, const float* shift,
                              const float* weight, const float* bias, void* r, void* y, cudaStream_t st) {
  if (xt == ROLA_BF16)
    return forward<__nv_bfloat16, __nv_bfloat16>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
  if (yt == ROLA_BF16)
    return forward<float, __nv_bfloat16>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
  return forward<float, float>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
}

cudaError_t launch_gated_norm_backward(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind,
                                       const void* dy, const void* dr, const void* r, const void* branch,
                                       const float* gate, const float* scale, const float* weight, void* dx,
                                       void* dbranch, float* dgate, float* dscale, float* dshift, float* dweight,
                                       float* dbias, float* part, cudaStream_t st) {
  if (xt == ROLA_BF16)
    return backward<__nv_bfloat16, __nv_bfloat16>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate,
                                                  dscale, dshift, dweight, dbias, part, st);
  if (yt == ROLA_BF16)
    return backward<float, __nv_bfloat16>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate, dscale,
                                          dshift, dweight, dbias, part, st);
  return backward<float, float>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate, dscale, dshift,
                                dweight, dbias, part, st);
}

}  // namespace rola
