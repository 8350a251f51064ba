// What the tcgen05 kernels of the cross attention share: tile sizes, work items, key validity.
#pragma once

#include "block_internal.cuh"
#include "sm100_ptx.cuh"
#include "softmax_exp.cuh"

namespace rola {

constexpr int kTile = 128;                    // queries of a tile, keys of a tile
constexpr uint32_t kBox = 128 * 128;          // bytes of a box: 128 rows x 64 channels

// One work item: a pair of query tiles of one head over a run of key tiles.
struct Item {
  int b, h, q0, streams, t0, t1, split;
};
// n / d for 0 <= n < 2^31 without a division: (hi(n m) + n) >> s with m = floor(2^32 (2^s - d) / d) + 1,
// s = ceil(log2 d).
struct Divisor {
  uint32_t d, m, s;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {d, (uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ int quotient(int n, const Divisor& d) {
  return (int)((__umulhi((uint32_t)n, d.m) + (uint32_t)n) >> d.s);
}
struct Work {
  int pairs, splits, run, items;
  Divisor per_head, per_pair, per_sample;     // pairs * splits, splits, H
  int padded;                                 // backward: rows of a head's statistics
};
__device__ __forceinline__ int key_count(const CrossArgs& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ Item item_at(const CrossArgs& a, const Work& w, int i) {
  Item x;
  const int bh = quotient(i, w.per_head), rest = i - bh * (int)w.per_head.d;
  const int pair = quotient(rest, w.per_pair);
  x.split = rest - pair * w.splits;
  x.b = quotient(bh, w.per_sample);
  x.h = bh - x.b * a.H;
  x.q0 = pair * 2 * kTile;
  x.streams = x.q0 + kTile < a.Nq ? 2 : 1;
  x.t0 = x.split * w.run;
  x.t1 = max(x.t0, min((key_count(a, x.b) + kTile - 1) / kTile, x.t0 + w.run));
  return x;
}
inline void set_divisors(Work* w, int H) {
  w->per_head = divisor((uint32_t)w->pairs * w->splits);
  w->per_pair = divisor(w->splits);
  w->per_sample = divisor(H);
}
// The next item at or after i that has key tiles (all others need no products), or one past the end.
__device__ __forceinline__ int next_item(const CrossArgs& a, const Work& w, int i, Item* x) {
  for (; i < w.items; i += gridDim.x) {
    *x = item_at(a, w, i);
    if (x->t1 > x->t0) return i;
  }
  return w.items;
}

// The 128 validity bits of key tile t (warp-collective): word e holds keys 32e .. 32e + 31.
__device__ __forceinline__ void tile_bits(const CrossArgs& a, int b, int len, int t, int lane, uint32_t (&bits)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int m = t * kTile + 32 * e + lane;
    bool ok = m < len;
    if (a.key_mask && ok) ok = __ldg(a.key_mask + (size_t)b * a.Nk + m) != 0;
    bits[e] = __ballot_sync(0xffffffffu, ok);
  }
}
__device__ __forceinline__ bool all_set(const uint32_t (&bits)[4]) {
  return (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
}

// Zeros the rows of a [128][64 kBoxes] tile (128-byte rows per box) whose bit is not set.
template <int kBoxes>
__device__ __forceinline__ void clear_rows(uint8_t* tile, const uint32_t (&bits)[4], int lane) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!((bits[e] >> lane) & 1u))
      for (int c = 0; c < kBoxes; ++c)
#pragma unroll
        for (int o = 0; o < 8; ++o)
          *reinterpret_cast<uint4*>(tile + c * kBox + (32 * e + lane) * 128 + 16 * o) = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A bounded wait of a converged warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t& m, uint32_t parity, const sm100::WaitCtl& w) {
  return __all_sync(0xffffffffu, sm100::mbar_wait(sm100::smem_addr(&m), parity, w));
}
// The lane that issues products and commits in a converged warp (always the same one).
__device__ __forceinline__ bool elect_leader() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}
// columns `col` = A (smem, K-major [128][D]) x B (smem, K-major [128][D])^T
template <int D>
__device__ __forceinline__ void product_ss(uint32_t col, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = sm100::idesc_f16(1, 128, 128, 0, 0);
  const uint64_t da = sm100::sdesc_sw128(a, 16, 1024), db = sm100::sdesc_sw128(b, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {   // 32 bytes inside a box, boxes 16 KB apart
    const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
    sm100::mma_f16_ss(col, da + off, db + off, idesc, kk > 0);
  }
}
// columns `col` (+)= A (tensor memory, 128 rows x 128, its halves `half` columns apart) x B (smem,
// [128 rows][D])
template <int D>
__device__ __forceinline__ void product_ts(uint32_t col, uint32_t a, uint32_t half, uint32_t b, bool add) {
  constexpr uint32_t idesc = sm100::idesc_f16(1, 128, D, 0, 1);
  const uint64_t db = sm100::sdesc_sw128(b, kBox, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)          // 16 rows of B: 8 columns of A, 2048 bytes of B
    sm100::mma_f16_ts(col, a + (kk >> 2) * half + (kk & 3) * 8, db + 128 * kk, idesc, add || kk > 0);
}

// Reads and clears a status word in device memory of the current device.
inline cudaError_t take_status(int (&symbol)[1], int* word, cudaStream_t st) {
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, symbol);
  if (e == cudaSuccess) e = cudaMemcpyAsync(word, at, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess || *word == 0) return e;
  e = cudaMemsetAsync(at, 0, sizeof(int), st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace rola
