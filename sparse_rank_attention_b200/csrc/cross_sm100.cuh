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
struct Work {
  int pairs, splits, run, items;
  int padded;                                 // backward: rows of a head's statistics
};
__device__ __forceinline__ int key_count(const CrossArgs& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ Item item_at(const CrossArgs& a, const Work& w, int i) {
  Item x;
  const int bh = i / (w.pairs * w.splits), rest = i - bh * w.pairs * w.splits;
  const int pair = rest / w.splits;
  x.split = rest - pair * w.splits;
  x.b = bh / a.H;
  x.h = bh - x.b * a.H;
  x.q0 = pair * 2 * kTile;
  x.streams = x.q0 + kTile < a.Nq ? 2 : 1;
  x.t0 = x.split * w.run;
  x.t1 = max(x.t0, min((key_count(a, x.b) + kTile - 1) / kTile, x.t0 + w.run));
  return x;
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
