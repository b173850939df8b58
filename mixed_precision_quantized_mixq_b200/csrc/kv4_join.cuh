// Joining the partial results that attention over the KV cache leaves where an item (rows of one
// kv head) is cut between CTAs.
#pragma once

#include "kv4.h"
#include "kv4_ptx.cuh"

namespace mixq {

struct Kv4Join {  // an item that starts in a CTA and ends in a later one
  int last;               // CTA of the last part, -1: no such item
  int row0, first, rows;  // q row of the sequence's first row; first row and rows of the item
  int head, pad[3];
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One row by one warp, parts in their order.  A part is [rows][D] sums, then its `rows` maxima,
// then its sums of weights; part(c) is that of CTA c.  32 parts at a time: a lane a part for the
// maximum and the factors, then all lanes for the sums, so that few loads follow one another.
template <int D, typename T, typename F>
__device__ __forceinline__ void kv4_join_row(F part, int c0, int last, int rows, int r, int lane, T *op) {
  constexpr int V = D / 32;
  float mx = -1e30f, sum = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int c = c0; c <= last; c += 32) {
    const bool in = c + lane <= last;
    const float m = in ? part(c + lane)[rows * D + r] : -1e30f, l = in ? part(c + lane)[rows * D + rows + r] : 0.f;
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, mx);
    const float old = ex2f(mx - top), f = ex2f(m - top);
    mx = top;
    float fl = in ? f * l : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, o);
    sum = fmaf(sum, old, fl);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= old;
    const int n = min(32, last - c + 1);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float w = __shfl_sync(0xffffffffu, f, k);
      const float *p = part(c + k) + r * D + lane * V;
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]), acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t *>(op + lane * V + i) =
        kv4_bits<uint32_t>(Kv4Type<T>::from2(acc[i] * inv, acc[i + 1] * inv));
}

}  // namespace mixq
