// The 4-bit KV cache: page format constants, the launch arguments of its
// kernels (kv4.cu: append and read; kv4_attn.cu: attention) and the device
// helpers they share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mixq {

// Tokens per record.  A record is [16][D/2] K bytes, the interleaved V bytes
// (16*D/2) and one 4-byte (s, lo) pair per token for K, then for V.
constexpr int kKv4Rec = 16;
__host__ __device__ constexpr int kv4_rec_bytes(int d) { return kKv4Rec * (d + 8); }

struct Kv4Cache {
  uint8_t *pages;
  int64_t page_stride;  // bytes between pages
  int n_pages;
  int recs_per_page;
  int page_shift;  // log2(recs_per_page), -1 if that is not a power of two
  int n_kv;
  int d;     // 64 or 128
  int bf16;  // type of the rows and of the (s, lo) pairs
};

struct Kv4Batch {
  int n_seqs;
  const int32_t *table;  // [n_seqs][table_width]
  int table_width;
  int64_t table_stride;
  const int32_t *lens;  // append, attention: tokens stored after the call; read: first position (or null)
  const int32_t *cu;    // [n_seqs + 1] row offsets, null: one row per sequence
  int rows;             // rows in the row tensors
};

struct Kv4Rows {  // K and V rows [rows][n_kv][d]; strides in elements
  const void *k, *v;
  int64_t k_row, k_head, v_row, v_head;
};

// Keys of a sequence that attention can see at most: no position, rounded up to a tile of either
// kernel and a tile further, leaves 32 bits.
constexpr int kKv4MaxKeys = 0x7fffffff - 255;

struct Kv4AttnArgs {
  Kv4Cache c;
  Kv4Batch b;
  const void *q;
  void *out;
  int64_t q_row, q_head, o_row, o_head;
  int n_q;    // query heads
  int group;  // n_q / n_kv
  int64_t max_rows;    // bound on a sequence's rows of a kv head (new tokens x group)
  int room;            // keys that a row of the table has room for, kKv4MaxKeys at most
  int64_t tile_above;  // sequences with more rows than this belong to the tile kernel
  float scale;
  int window, sinks;  // window 0: all keys up to the query's position
  float *work;       // step kernel's parts
  float *work_tile;  // tile kernel's parts
  int num_sms;
  int stall;  // the variants whose pipelines stop (timeout test; fp16, d 64)
  int32_t *status;
};

cudaError_t launch_kv4_append(const Kv4Cache &c, const Kv4Batch &b, const Kv4Rows &r,
                              int32_t *status, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &b, const Kv4Rows &r,
                            int32_t *status, cudaStream_t stream);
size_t kv4_step_workspace(int d, int num_sms);
size_t kv4_tile_workspace(int d, int num_sms);
// More rows (new tokens x group) of a kv head than this: tile kernel.  16 sequences of 4096 tokens, 64 / 8
// heads of 128, fp16, us by the step / the tile kernel: 16 rows 60 / 107, 32 rows 80 / 109, 40 rows
// 92 / 109, 48 rows 105 / 109, 64 rows 132 / 110; bf16 57 / 111 up to 116 / 113; D 64 41 / 95 up to
// 95 / 97.  One sequence alone: 35 / 35 at 16 rows, 31 / 37 at 64.
constexpr int kKv4TileAbove = 32;
// Decode steps and small row counts (kv4_attn.cu), many rows (kv4_tile.cu); the
// first launches the second where it is needed, and the join of what both cut (kv4_join.cuh).
cudaError_t launch_kv4_attn(Kv4AttnArgs a, cudaStream_t stream);
cudaError_t launch_kv4_tile(const Kv4AttnArgs &a, cudaStream_t stream);

#ifdef __CUDACC__

// Row range of sequence s in the row tensors; a range that is not ordered or
// leaves the tensor counts as empty.  bad: such a range was seen.
__device__ __forceinline__ int2 kv4_row_range(const Kv4Batch &b, int s, bool *bad) {
  if (!b.cu) return make_int2(s, s + 1);
  const int r0 = __ldg(b.cu + s), r1 = __ldg(b.cu + s + 1);
  if (r0 < 0 || r1 < r0 || r1 > b.rows) {
    *bad = true;
    return make_int2(0, 0);
  }
  return make_int2(r0, r1);
}

// An (s, lo) pair as two fp32 values.
template <bool BF16>
__device__ __forceinline__ float2 kv4_pair(uint32_t p) {
  if (BF16) return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
  __half2 h;
  memcpy(&h, &p, 4);
  return __half22float2(h);
}

template <typename T>
struct Kv4Type;
template <>
struct Kv4Type<__half> {
  using T2 = __half2;
  static constexpr bool bf16 = false;
  static __device__ __forceinline__ float2 f2(__half2 v) { return __half22float2(v); }
  static __device__ __forceinline__ __half2 from2(float a, float b) { return __floats2half2_rn(a, b); }
  // the same, but held at the largest finite value (NaN stays): outputs of attention.  A mean of V rows
  // can pass it, as 15 s + lo can (s is rounded) and as rounded weights need not sum to what divides them.
  static __device__ __forceinline__ uint32_t held2(float a, float b) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
  static constexpr float max_finite = 65504.f;
};
template <>
struct Kv4Type<__nv_bfloat16> {
  using T2 = __nv_bfloat162;
  static constexpr bool bf16 = true;
  static __device__ __forceinline__ float2 f2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ __nv_bfloat162 from2(float a, float b) {
    return __floats2bfloat162_rn(a, b);
  }
  static __device__ __forceinline__ uint32_t held2(float a, float b) {
    uint32_t d;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
  static constexpr float max_finite = 3.3895313892515355e38f;
};

template <typename A, typename B>
__device__ __forceinline__ A kv4_bits(B b) {
  static_assert(sizeof(A) == sizeof(B), "same size");
  A a;
  memcpy(&a, &b, sizeof a);
  return a;
}

#endif  // __CUDACC__

}  // namespace mixq
