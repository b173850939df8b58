// Append and read of the 4-bit KV cache (QServe W4A8KV4 notes: each token and
// head of K and V is its own 4-bit asymmetric group).
//
//   append: lo = min x, hi = max x, s = T((hi - lo) / 15),
//           c = min(rint((x - lo) * (1 / s)), 15)           (fp32, each step rounded once)
//   read:   x^ = c * s + lo                                  (fp32, rounded once to T)
//
// Both passes are bound by HBM: 4*D bytes of rows against D + 8 bytes of cache
// per token and kv head.  A warp owns one 16-token record of one kv head.  A
// row of D values is held by D/8 lanes, 16 bytes each, so rows move in whole
// 128- or 256-byte segments, a row's range takes log2(D/8) shuffles, and K's
// eight 4-bit codes of a lane are exactly one word of the record.  The V words
// of a record hold four tokens (2t, 2t+8, 2t+1, 2t+9), which one group of D/8
// lanes loads as four rows; a 4x4 byte transpose in registers turns their codes
// into whole words.
//
// What they measured (B200): 107 MB of rows of six 7B prompts written in 34.5 us
// (3.9 TB/s with the codes; 1860 instructions a record and head, 73 % of the issue
// slots: the instructions bound it, not HBM) and read back in 27 (5.1 TB/s); eight
// prefixes of up to 16384 tokens, 389 MB, read in 65 (6.0 TB/s, 91 % of the measured
// copy rate; issue slots 72 %).  A fourth block per SM (64 registers) brought 2 us of the
// write, asking for the page beside the rows 2 more.
#include <cuda_runtime.h>

#include "kv4.h"
#include "kv4_ptx.cuh"

namespace mixq {
namespace {

constexpr int kWarps = 8;

// First sequence of the virtual record index v.  Sequence s owns the indexes
// from floor(cu[s] / 16) + 2 s: at least one more than the records its rows can
// touch, so every record has an index and the search needs cu alone.
__device__ __forceinline__ int find_seq(const Kv4Batch &b, int v, int lane) {
  int lo = 0, hi = b.n_seqs - 1;  // answer in [lo, hi]: last s with start(s) <= v
  while (lo < hi) {
    // 32 probes split the range: last probe whose start is <= v
    const int n = hi - lo;
    const int step = (n + 31) / 32;
    const int s = min(lo + (lane + 1) * step, hi);
    const int start = (__ldg(b.cu + s) >> 4) + 2 * s;
    const unsigned m = __ballot_sync(0xffffffffu, start <= v);
    const int k = __popc(m);  // starts do not fall, so m is a prefix of the lanes
    const int nlo = k == 0 ? lo : min(lo + k * step, hi);
    hi = k == 32 ? hi : min(lo + (k + 1) * step - 1, hi);
    lo = nlo;
    hi = max(hi, lo);
  }
  return lo;
}

// The first blocks of a call with offsets look at all of them, a sequence a thread: offsets that fall
// may hide a sequence from the search.  Blocks of their own, as values held beside the search cost
// the others registers (prefixes 65 -> 68 us).
__device__ __forceinline__ void check_offsets(const Kv4Batch &b, int32_t *status) {
  const unsigned s = blockIdx.x * (kWarps * 32) + threadIdx.x;
  bool bad = false;
  if (blockIdx.y == 0 && s < b.n_seqs) kv4_row_range(b, s, &bad);
  if (bad) record_error(status, kErrInvalidArg);
}

struct Place {
  int row0;       // row of the record's token 0 (may lie before the range)
  int t0, t1;     // tokens [t0, t1) of the record belong to the call
  int page;       // of the record; not checked
  int64_t off;    // of the record of kv head 0 in its page
};

// The record itself, null if its page is not usable.
__device__ __forceinline__ uint8_t *record(const Kv4Cache &c, const Place &p, int lane, int32_t *status) {
  if (p.page < 0 || p.page >= c.n_pages) {
    if (lane == 0) record_error(status, kErrInvalidArg);
    return nullptr;
  }
  return c.pages + p.page * c.page_stride + p.off;
}

// The record that virtual index v stands for, or t0 == t1.
__device__ __forceinline__ Place locate(const Kv4Cache &c, const Kv4Batch &b, int v, int lane,
                                        bool append, int32_t *status) {
  Place p{0, 0, 0, -1, 0};
  int s, local;
  if (b.cu) {
    s = find_seq(b, v, lane);
    local = v - ((__ldg(b.cu + s) >> 4) + 2 * s);
  } else {
    s = v;
    local = 0;
  }
  bool bad = false;
  const int2 r = kv4_row_range(b, s, &bad);
  const int n = r.y - r.x;
  if (bad && lane == 0) record_error(status, kErrInvalidArg);
  if (n == 0) return p;
  // positions [first, first + n)
  const int first = append ? __ldg(b.lens + s) - n : (b.lens ? __ldg(b.lens + s) : 0);
  const int from = max(first, 0);
  if (first + static_cast<int64_t>(n) <= from) return p;
  const int rec = (from >> 4) + local;
  const int64_t base = static_cast<int64_t>(rec) * 16;
  const int64_t t0 = max(static_cast<int64_t>(from) - base, static_cast<int64_t>(0));
  const int64_t t1 = min(first + static_cast<int64_t>(n) - base, static_cast<int64_t>(16));
  if (t1 <= t0) return p;
  const int slot = rec / c.recs_per_page;
  p.page = slot < b.table_width ? __ldg(b.table + s * b.table_stride + slot) : -1;
  p.t0 = static_cast<int>(t0);
  p.t1 = static_cast<int>(t1);
  p.row0 = static_cast<int>(r.x + (base - first));
  p.off = static_cast<int64_t>(rec - slot * c.recs_per_page) * kv4_rec_bytes(c.d);
  return p;
}

// Transpose of a 4x4 byte matrix held as four words.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, b, 0x5410);
  w[1] = __byte_perm(a, b, 0x7632);
  w[2] = __byte_perm(c, d, 0x5410);
  w[3] = __byte_perm(c, d, 0x7632);
}

// Token that byte i of a V word of quad t belongs to.
__device__ __forceinline__ int quad_token(int t, int i) { return 2 * t + (i >> 1) + 8 * (i & 1); }

// x / 15, rounded to nearest: the quotient from the rounded reciprocal, corrected once with
// its exact remainder (P. Markstein, IBM J. Res. Dev. 34, 1990).  x is 0 or the difference of
// two 16-bit values, so nothing here underflows inexactly.
__device__ __forceinline__ float div15(float x) {
  constexpr float r = 1.f / 15.f;
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-15.f, q, x), r, q);
}

// 1 / s, rounded to nearest, for a normal s with an 11-bit significand whose reciprocal is
// normal: one such correction (same source) of an approximation within a unit in the last place.
__device__ __forceinline__ float reciprocal(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return __fmaf_rn(__fmaf_rn(-s, y, 1.f), y, y);
}

// The eight codes of a lane (one row spread over LANES lanes) as a word, and the row's (s, lo)
// pair.  K: nibble p = dim 2p, nibble p + 4 = dim 2p + 1; else nibbles 0..7 = dims 0..7.
template <typename T, int LANES, bool K>
__device__ __forceinline__ uint32_t quantize8(const uint4 &raw, uint32_t *pair) {
  using X = Kv4Type<T>;
  using T2 = typename X::T2;
  const T2 x[4] = {kv4_bits<T2>(raw.x), kv4_bits<T2>(raw.y), kv4_bits<T2>(raw.z),
                   kv4_bits<T2>(raw.w)};
  // the *_nan forms keep a NaN, so a row with one ends as (NaN, NaN)
  T2 mn = __hmin2_nan(__hmin2_nan(x[0], x[1]), __hmin2_nan(x[2], x[3]));
  T2 mx = __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
  // (min x, min -x) in one register: one shuffle per step serves both ends
  const uint32_t a = kv4_bits<uint32_t>(mn), z = kv4_bits<uint32_t>(mx);
  T2 e = __hmin2_nan(kv4_bits<T2>(__byte_perm(a, z, 0x5410) ^ 0x80000000u),
                     kv4_bits<T2>(__byte_perm(a, z, 0x7632) ^ 0x80000000u));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    e = __hmin2_nan(e, kv4_bits<T2>(__shfl_xor_sync(0xffffffffu, kv4_bits<uint32_t>(e), o)));
  const float2 ends = X::f2(e);
  const float lo = ends.x, hi = -ends.y;
  const float range = __fsub_rn(hi, lo);
  const T2 sl = X::from2(div15(range), lo);
  float s = X::f2(sl).x;
  if (s < 1.17549435e-38f) s = 0.f;  // a bf16 subnormal's reciprocal may not be finite
  const bool finite = range - range == 0.f;  // neither end NaN or infinite, nor their distance
  const float inv = s > 0.f ? reciprocal(s) : 0.f;
  // 1.5 * 2^23 + (x - lo) * inv, each step rounded once: the last rounds half to even and leaves
  // the code in the low bits
  const uint64_t nlo = f32x2(-lo, -lo), inv2 = f32x2(inv, inv);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = X::f2(x[i]);
    const float2 u = from_f32x2(mul_f32x2(add_f32x2(f32x2(f.x, f.y), nlo), inv2));
    // one at a time: ptxas joins the packed product and sum into one rounding
    c[2 * i] = __float_as_uint(__fadd_rn(u.x, 12582912.f));
    c[2 * i + 1] = __float_as_uint(__fadd_rn(u.y, 12582912.f));
  }
  // s is range / 15 to within a small part unless it is subnormal in T; only then can a code pass 15
  if (__builtin_expect(__any_sync(0xffffffffu, __fmul_rn(range, inv) >= 15.5f), 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = min(c[i], 0x4b40000fu);
  }
  // c[i] = 0x4b400000 + code: codes times their places add up, and the constant parts in one word
  constexpr uint32_t kBits = 0x4b400000u;
  uint32_t w;
  if (K) {
    const uint32_t even = c[0] + c[2] * 16 + c[4] * 256 + c[6] * 4096, odd = c[1] + c[3] * 16 + c[5] * 256 + c[7] * 4096;
    w = even + odd * 65536 - kBits * 0x1111u * 0x10001u;
  } else {
    w = c[0] + c[1] * 16 + c[2] * 256 + c[3] * 4096 + (c[4] + c[5] * 16 + c[6] * 256 + c[7] * 4096) * 65536 -
        kBits * 0x11111111u;
  }
  *pair = finite ? kv4_bits<uint32_t>(X::from2(s, lo)) : 0x7fff7fffu;
  return w;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 4)
    kv4_append_kernel(Kv4Cache c, Kv4Batch b, Kv4Rows r, int32_t *status, unsigned checks) {
  constexpr int LANES = D / 8, RPW = 32 / LANES;  // lanes per row, rows per warp load
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x < checks) return check_offsets(b, status);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kWarps + warp;
  if (h >= c.n_kv) return;
  const Place p = locate(c, b, blockIdx.x - checks, lane, true, status);
  if (p.t0 >= p.t1) return;
  const int sub = lane / LANES, l = lane % LANES;
  uint8_t *rec = nullptr;
  const T *k = static_cast<const T *>(r.k) + h * r.k_head + l * 8;
  const T *v = static_cast<const T *>(r.v) + h * r.v_head + l * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  // Rows come in V's quad order for both K and V: one lane group loads the four
  // tokens of a quad.  All loads of a half record are issued before their use.
#pragma unroll
  for (int it = 0; it < 4 / RPW; ++it) {
    const int t = it * RPW + sub;
    uint4 kr[4], vr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = quad_token(t, i);
      const bool in = tok >= p.t0 && tok < p.t1;
      const int64_t row = p.row0 + tok;
      kr[i] = in ? __ldg(reinterpret_cast<const uint4 *>(k + row * r.k_row)) : zero;
      vr[i] = in ? __ldg(reinterpret_cast<const uint4 *>(v + row * r.v_row)) : zero;
    }
    if (it == 0) {  // only here, so that the page's look-up and the rows' loads overlap
      rec = record(c, p, lane, status);
      if (!rec) return;
      rec += h * static_cast<int64_t>(c.recs_per_page) * kv4_rec_bytes(D);
    }
    uint32_t vw[4];
    int valid = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = quad_token(t, i);
      const bool in = tok >= p.t0 && tok < p.t1;
      uint32_t kp, vp;
      const uint32_t kc = quantize8<T, LANES, true>(kr[i], &kp);
      vw[i] = quantize8<T, LANES, false>(vr[i], &vp);
      if (in) {
        valid |= 1 << i;
        reinterpret_cast<uint32_t *>(rec + tok * (D / 2))[l] = kc;
        if (l == 0) {
          reinterpret_cast<uint32_t *>(rec + 16 * D)[tok] = kp;
          reinterpret_cast<uint32_t *>(rec + 16 * D + 64)[tok] = vp;
        }
      }
    }
    transpose4(vw);  // word j: byte column 4 l + j, byte i = token i of the quad
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint8_t *w = rec + 8 * D + (l >> 3) * 512 + (4 * (l & 1) + j) * 64 + t * 16 + ((l >> 1) & 3) * 4;
      if (valid == 15) {
        *reinterpret_cast<uint32_t *>(w) = vw[j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (valid >> i & 1) w[i] = static_cast<uint8_t>(vw[j] >> (8 * i));
      }
    }
  }
}

// A word of eight codes and the row's pair -> eight values of T (word orders as in quantize8).
template <typename T, bool K>
__device__ __forceinline__ uint4 dequantize8(uint32_t w, float2 sl) {
  using X = Kv4Type<T>;
  // 2^23 + code * 16^p as bits, exact, for the four nibbles of a half; c * s is exact, so the sum
  // rounds once (s / 16^p is exact as well: s has 11 bits and is normal, or 0, in fp32)
  const uint64_t s01 = f32x2(sl.x, sl.x * 0.0625f), s23 = f32x2(sl.x * 0.00390625f, sl.x * 0.000244140625f),
                 lo = f32x2(sl.y, sl.y), down = f32x2(-8388608.f, -8388608.f);
  float v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = h ? w >> 16 : w;
    const uint64_t a = f32x2(__uint_as_float(0x4b000000u | (u & 0xfu)), __uint_as_float(0x4b000000u | (u & 0xf0u)));
    const uint64_t b = f32x2(__uint_as_float(0x4b000000u | (u & 0xf00u)), __uint_as_float(0x4b000000u | (u & 0xf000u)));
    const float2 x = from_f32x2(fma_f32x2(add_f32x2(a, down), s01, lo)), y = from_f32x2(fma_f32x2(add_f32x2(b, down), s23, lo));
    v[K ? h : 4 * h] = x.x, v[K ? 2 + h : 4 * h + 1] = x.y;
    v[K ? 4 + h : 4 * h + 2] = y.x, v[K ? 6 + h : 4 * h + 3] = y.y;
  }
  // s was rounded, so 15 s + lo can pass the type's largest value: hold it there (NaN passes)
  if (__builtin_expect(fmaf(15.f, sl.x, sl.y) > X::max_finite, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] > X::max_finite ? X::max_finite : v[i];
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = kv4_bits<uint32_t>(X::from2(v[2 * i], v[2 * i + 1]));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 5)
    kv4_read_kernel(Kv4Cache c, Kv4Batch b, Kv4Rows r, int32_t *status, unsigned checks) {
  constexpr int LANES = D / 8, RPW = 32 / LANES;
  constexpr bool BF = Kv4Type<T>::bf16;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x < checks) return check_offsets(b, status);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kWarps + warp;
  if (h >= c.n_kv) return;
  const Place p = locate(c, b, blockIdx.x - checks, lane, false, status);
  if (p.t0 >= p.t1) return;
  const int sub = lane / LANES, l = lane % LANES;
  const uint8_t *rec = record(c, p, lane, status);
  if (!rec) return;
  rec += h * static_cast<int64_t>(c.recs_per_page) * kv4_rec_bytes(D);
  T *k = const_cast<T *>(static_cast<const T *>(r.k)) + h * r.k_head + l * 8;
  T *v = const_cast<T *>(static_cast<const T *>(r.v)) + h * r.v_head + l * 8;
  uint32_t kw[4 / RPW][4], vw[4 / RPW][4], kp[4 / RPW][4], vp[4 / RPW][4];
#pragma unroll
  for (int it = 0; it < 4 / RPW; ++it) {
    const int t = it * RPW + sub;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = quad_token(t, i);
      kw[it][i] = __ldcs(reinterpret_cast<const uint32_t *>(rec + tok * (D / 2)) + l);
      vw[it][i] = __ldcs(reinterpret_cast<const uint32_t *>(rec + 8 * D + (l >> 3) * 512 +
                                                      (4 * (l & 1) + i) * 64 + t * 16 + ((l >> 1) & 3) * 4));
      kp[it][i] = reinterpret_cast<const uint32_t *>(rec + 16 * D)[tok];
      vp[it][i] = reinterpret_cast<const uint32_t *>(rec + 16 * D + 64)[tok];
    }
  }
#pragma unroll
  for (int it = 0; it < 4 / RPW; ++it) {
    const int t = it * RPW + sub;
    transpose4(vw[it]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = quad_token(t, i);
      if (tok < p.t0 || tok >= p.t1) continue;
      const int64_t row = p.row0 + tok;
      // codes and rows pass through once: 2 us of 70 by the streaming hints
      __stcs(reinterpret_cast<uint4 *>(k + row * r.k_row), dequantize8<T, true>(kw[it][i], kv4_pair<BF>(kp[it][i])));
      __stcs(reinterpret_cast<uint4 *>(v + row * r.v_row), dequantize8<T, false>(vw[it][i], kv4_pair<BF>(vp[it][i])));
    }
  }
}

template <typename K>
cudaError_t launch(K kernel, const Kv4Cache &c, const Kv4Batch &b, const Kv4Rows &r,
                   int32_t *status, cudaStream_t stream) {
  // virtual records: one per sequence, or the last start plus the last sequence's own
  const unsigned records = b.cu ? b.rows / 16 + 2u * b.n_seqs : b.n_seqs;
  const unsigned checks = b.cu ? (b.n_seqs + kWarps * 32 - 1) / (kWarps * 32) : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(records + checks, (c.n_kv + kWarps - 1) / kWarps, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, c, b, r, status, checks);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache &c, const Kv4Batch &b, const Kv4Rows &r,
                              int32_t *status, cudaStream_t stream) {
  if (c.bf16)
    return c.d == 128 ? launch(kv4_append_kernel<__nv_bfloat16, 128>, c, b, r, status, stream)
                      : launch(kv4_append_kernel<__nv_bfloat16, 64>, c, b, r, status, stream);
  return c.d == 128 ? launch(kv4_append_kernel<__half, 128>, c, b, r, status, stream)
                    : launch(kv4_append_kernel<__half, 64>, c, b, r, status, stream);
}

cudaError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &b, const Kv4Rows &r,
                            int32_t *status, cudaStream_t stream) {
  if (c.bf16)
    return c.d == 128 ? launch(kv4_read_kernel<__nv_bfloat16, 128>, c, b, r, status, stream)
                      : launch(kv4_read_kernel<__nv_bfloat16, 64>, c, b, r, status, stream);
  return c.d == 128 ? launch(kv4_read_kernel<__half, 128>, c, b, r, status, stream)
                    : launch(kv4_read_kernel<__half, 64>, c, b, r, status, stream);
}

}  // namespace mixq
