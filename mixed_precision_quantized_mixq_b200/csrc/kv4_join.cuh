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

// Rows of a part's slot: what an item of each kernel has at most.
constexpr int kKv4TileRows = 256, kKv4StepRows = 16;
__host__ __device__ constexpr size_t kv4_slot_floats(int rows, int d) { return rows * (static_cast<size_t>(d) + 2); }

// One row by one warp, for many parts: 32 at a time, a lane a part for the maximum and the factors,
// then all lanes for the sums, so that few loads follow one another.
template <int D, int ROWS, typename T, typename F>
__device__ __forceinline__ void kv4_join_row(F part, int c0, int last, int r, int lane, T *op) {
  constexpr int V = D / 32;
  float mx = -1e30f, sum = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int c = c0; c <= last; c += 32) {
    const bool in = c + lane <= last;
    const float m = in ? part(c + lane)[ROWS * D + r] : -1e30f, l = in ? part(c + lane)[ROWS * D + ROWS + r] : 0.f;
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
        Kv4Type<T>::held2(acc[i] * inv, acc[i + 1] * inv);
}

// Joins the items of `ctas` CTAs that were cut, N rows a warp, parts in their order.  A CTA has two
// slots in `work`, of the item that goes on from the CTA before and of the one that goes on after
// it; a slot is [ROWS][D] sums, then ROWS maxima, then ROWS sums of weights.  i: the warp's number
// among those of this call, `per` a CTA.  With few parts four rows at once hide the loads (four
// 7B prompts: 9 us against 15 of a row a warp); with 18 parts 20 us against 10.
template <int D, int ROWS, int N, typename T>
__device__ __forceinline__ void kv4_join(const Kv4AttnArgs &a, const float *work, int ctas, int i, int per) {
  constexpr int V = D / 32;
  const int c0 = i / per, r0 = (i % per) * N, lane = threadIdx.x & 31;
  const Kv4Join x = reinterpret_cast<const Kv4Join *>(work)[c0];
  if (x.last < 0 || r0 >= x.rows) return;
  const float *slots = work + ctas * (sizeof(Kv4Join) / 4);
  auto place = [&](int r) {
    const int rr = x.first + r, qi = rr / a.group;
    return static_cast<T *>(a.out) + (x.row0 + static_cast<int64_t>(qi)) * a.o_row +
           (static_cast<int64_t>(x.head) * a.group + (rr - qi * a.group)) * a.o_head;
  };
  auto part = [&](int c) { return slots + (2 * static_cast<size_t>(c) + (c == c0)) * kv4_slot_floats(ROWS, D); };
  if (N > 1 && x.last - c0 < 4) {
    float mx[N], sum[N], acc[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      mx[n] = -1e30f, sum[n] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[n][v] = 0.f;
    }
#pragma unroll 2
    for (int c = c0; c <= x.last; ++c) {
      const float *p = part(c);
      float m[N], l[N], o[N][V];
#pragma unroll
      for (int n = 0; n < N; ++n) m[n] = p[ROWS * D + r0 + n], l[n] = p[ROWS * D + ROWS + r0 + n];
#pragma unroll
      for (int n = 0; n < N; ++n) {  // rows past the item's last hold whatever was there, and are not stored
        const float *q = p + (r0 + n) * D + lane * V;
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4 *>(q);
          o[n][0] = f.x, o[n][1] = f.y, o[n][2] = f.z, o[n][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2 *>(q);
          o[n][0] = f.x, o[n][1] = f.y;
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float top = fmaxf(mx[n], m[n]), old = ex2f(mx[n] - top), f = ex2f(m[n] - top);
        mx[n] = top;
        sum[n] = fmaf(sum[n], old, f * l[n]);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[n][v] = fmaf(acc[n][v], old, f * o[n][v]);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (r0 + n >= x.rows) break;
      const float inv = sum[n] == 0.f ? 0.f : 1.f / sum[n];
      T *op = place(r0 + n) + lane * V;
#pragma unroll
      for (int v = 0; v < V; v += 2)
        *reinterpret_cast<uint32_t *>(op + v) = Kv4Type<T>::held2(acc[n][v] * inv, acc[n][v + 1] * inv);
    }
    return;
  }
#pragma unroll 1
  for (int r = r0; r < min(r0 + N, x.rows); ++r) kv4_join_row<D, ROWS>(part, c0, x.last, r, lane, place(r));
}

}  // namespace mixq
