// Attention over the 4-bit KV cache for many query rows (prompts and chunks of
// prompts), on the 5th-generation tensor cores.
//
// One CTA takes up to 256 query rows of one (sequence, kv head): rows are (new
// token, head of the group) pairs, so grouped heads fill the tiles.  The rows are
// two 128-row MMA tiles that take turns: while the softmax of one runs, the
// tensor core works for the other.  Per 128 keys and row tile
//   S = Q C^T   (C: K's codes, exact in the 16-bit type), 128 x 128 x D, in TMEM
//   t = scale log2(e) (s_k S + lo_k sum(q)),  P = 2^(t - m)
//   O += P V^   (V^: V's rows as they read back, rounded once to the type)
// with P written over S in TMEM as the second product's A operand.
//
// Roles: warps 0-7 softmax (thread = query row = TMEM lane; no reduction crosses
// lanes), warps 8-15 unpack the cache straight from global memory into the
// swizzled operand tiles (one 16-token record a warp and tile, the next tile's
// bytes already in registers), warp 16 issues the MMAs.  K stays in codes because
// a rounded K would move every score; the pairs act on S instead.  V is rounded
// to the type like any 16-bit V, which leaves the softmax no work per V row.
//
// The running maximum moves only when a score passes it by 2^8, so O (in TMEM) is
// rarely rescaled; P carries 2^6 more so that fp16 keeps 11 bits down to 2^-20 of
// the row's largest weight.
#include <cuda_runtime.h>

#include <atomic>

#include "kv4.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace mixq {
namespace {

constexpr int kThreads = 640;  // 8 softmax, 8 unpack, 1 MMA warp (and 3 that complete its group)
constexpr int kRows = 256;     // query rows per CTA
constexpr int kKeys = 128;     // keys per tile
constexpr float kNegBig = -1e30f;
constexpr uint64_t kWaitNs = 2000000000ull;

// registers per thread after the split; 2*128*176 + 2*128*48 + 128*24 = 60416 of the
// 640 * 96 = 61440 the CTA starts with
constexpr int kRegsSoftmax = 176, kRegsUnpack = 48, kRegsMma = 24;

template <int D>
struct TileSmem {
  alignas(1024) uint8_t q[2][128 * D * 2];
  alignas(1024) uint8_t k[2][kKeys * D * 2];
  alignas(1024) uint8_t v[2][kKeys * D * 2];
  alignas(16) float4 kp[4][kKeys / 2];  // per pair of keys: s0 s1 lo0 lo1, times scale log2(e)
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], par_full[4], s_full[2], p_full[2], o_full[2];
  uint32_t hidden[4];  // records of the tile whose page is not usable
  uint32_t tmem;
  int dead;
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a));
  return f;
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D(tmem, fp32) (+)= A(tmem, 16-bit: lane = row, two K values per column) * B(smem)^T
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Bounded wait; once one has run out, none waits any more and the CTA winds up.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, volatile int *dead, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!*dead) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *dead = 1;
      record_error(status, kErrTimeout);
    }
  }
}

template <typename T>
struct Codes;
template <>
struct Codes<__half> {
  // 1024 + c, then - 1024; the second nibble as 1024 + 16 c, then / 16 - 64: exact
  static __device__ __forceinline__ void pairs(uint32_t w, __half2 (&o)[4]) {
    const uint32_t h = w >> 8;
    const __half2 k1024 = __float2half2_rn(1024.f), k16 = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.f);
    o[0] = __hsub2(kv4_bits<__half2>((w & 0x000f000fu) | 0x64006400u), k1024);
    o[1] = __hfma2(kv4_bits<__half2>((w & 0x00f000f0u) | 0x64006400u), k16, k64);
    o[2] = __hsub2(kv4_bits<__half2>((h & 0x000f000fu) | 0x64006400u), k1024);
    o[3] = __hfma2(kv4_bits<__half2>((h & 0x00f000f0u) | 0x64006400u), k16, k64);
  }
};
template <>
struct Codes<__nv_bfloat16> {
  // 128 + c, then - 128: exact
  static __device__ __forceinline__ void pairs(uint32_t w, __nv_bfloat162 (&o)[4]) {
    const __nv_bfloat162 k128 = __float2bfloat162_rn(128.f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = __hsub2(kv4_bits<__nv_bfloat162>(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u), k128);
  }
};

// The CTA's rows and key tiles.
struct Job {
  int seq, row0, len, pos0;  // sequence, its first q row, its keys, position of its first new token
  int first, rows;           // rows of the kv head: first of this CTA, how many
  int tiles;                 // key tiles to visit
  int sink_tiles, skip;      // tile i >= sink_tiles is key tile i + skip
  __device__ __forceinline__ int key0(int i) const {
    return (i + (i >= sink_tiles ? skip : 0)) * kKeys;
  }
};

// Virtual row tile v belongs to the last sequence s with floor(cu[s] G / 256) + s
// <= v: every sequence owns at least as many as its rows fill, and the search
// needs cu alone.  A sequence's last rows come first (they see the most keys).
// rows == 0: nothing to do.
__device__ __forceinline__ Job find_job(const Kv4AttnArgs &a, int v, int lane) {
  Job j{};
  int lo = 0, hi = a.b.n_seqs - 1;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int s = min(lo + (lane + 1) * step, hi);
    const int64_t row = a.b.cu ? __ldg(a.b.cu + s) : s;
    const int64_t start = row * a.group / kRows + s;
    const int k = __popc(__ballot_sync(0xffffffffu, start <= v));
    const int nlo = min(lo + k * step, hi);
    hi = k == 32 ? hi : max(nlo, min(lo + (k + 1) * step - 1, hi));
    lo = nlo;
  }
  bool bad = false;
  const int2 r = kv4_row_range(a.b, lo, &bad);
  const int full = __ldg(a.b.lens + lo);
  const int64_t cap = static_cast<int64_t>(a.b.table_width) * a.c.recs_per_page * kKv4Rec;
  if (threadIdx.x == 0 && (bad || full < 0 || full > cap)) record_error(a.status, kErrInvalidArg);
  if (bad) return j;
  const int64_t all = static_cast<int64_t>(r.y - r.x) * a.group;
  const int n_tiles = static_cast<int>((all + kRows - 1) / kRows);
  const int64_t local = v - (static_cast<int64_t>(r.x) * a.group / kRows + lo);
  if (all <= a.tile_above || local < 0 || local >= n_tiles) return j;
  j.seq = lo;
  j.row0 = r.x;
  j.first = static_cast<int>(n_tiles - 1 - local) * kRows;
  j.rows = static_cast<int>(min(static_cast<int64_t>(kRows), all - j.first));
  j.len = static_cast<int>(min(static_cast<int64_t>(max(full, 0)), cap));
  j.pos0 = full - (r.y - r.x);
  const int pmin = j.pos0 + j.first / a.group, pmax = j.pos0 + (j.first + j.rows - 1) / a.group;
  const int total = (max(0, min(j.len, pmax + 1)) + kKeys - 1) / kKeys;
  j.sink_tiles = total;
  j.tiles = total;
  if (a.window > 0) {
    const int w0 = min(max(0, max(pmin, 0) - a.window + 1) / kKeys, total);
    j.sink_tiles = min((min(a.sinks, j.len) + kKeys - 1) / kKeys, w0);
    j.skip = w0 - j.sink_tiles;
    j.tiles = total - j.skip;
  }
  return j;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_tile_kernel(const Kv4AttnArgs a) {
  using S = TileSmem<D>;
  using X = Kv4Type<T>;
  using T2 = typename X::T2;
  constexpr bool BF = X::bf16;
  constexpr int REC = kv4_rec_bytes(D), WORDS = D / 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S &sm = *reinterpret_cast<S *>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int head = blockIdx.x;

  griddep_wait();
  griddep_launch_dependents();
  const Job job = find_job(a, blockIdx.y, lane);
  if (job.rows == 0) return;
  if (tid == 0) {
    sm.dead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 128);
      mbar_init(&sm.k_full[i], 8);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 8);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.par_full[i], 8);
      sm.hidden[i] = 0;
    }
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const uint32_t tm_s[2] = {tmem, tmem + 128}, tm_o[2] = {tmem + 256, tmem + 256 + D};
  const int row_tiles = job.rows > 128 ? 2 : 1;
  const int n = job.tiles;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    reg_inc<kRegsSoftmax>();
    const int i = warp / 4, row = tid & 127, r = i * 128 + row;
    if (i < row_tiles) {
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 TMEM lanes per warp
      const bool valid = r < job.rows;
      const int qi = (job.first + r) / a.group, g = job.first + r - qi * a.group;
      const int64_t head_q = static_cast<int64_t>(head) * a.group + g;
      const int p = job.pos0 + qi;
      // ---- the thread's query row into the operand tile, and its sum
      float qsum = 0.f;
      {
        const T *qp = static_cast<const T *>(a.q) + (job.row0 + static_cast<int64_t>(qi)) * a.q_row + head_q * a.q_head;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = valid ? __ldg(reinterpret_cast<const uint4 *>(qp) + c) : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = X::f2(kv4_bits<T2>(u[e]));
            qsum += f.x;
            qsum += f.y;
          }
          *reinterpret_cast<uint4 *>(sm.q[i] + (c / 8) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x;
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full[i]);
      }
      const uint64_t qs2 = pack2(qsum, qsum);
      // key j is visible when j < vis and (j >= wlo or j < sinks)
      const int vis = valid ? min(p + 1, job.len) : job.len;
      const int wlo = valid && a.window > 0 ? p - a.window + 1 : -0x7fffffff;
      const int tmin = job.pos0 + (job.first + i * 128) / a.group;
      const int tmax = job.pos0 + (job.first + min(i * 128 + 128, job.rows) - 1) / a.group;
      float m = kNegBig;
      uint64_t l2 = pack2(0.f, 0.f);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int k0 = job.key0(j);
        wait(&sm.par_full[j & 3], (j >> 2) & 1, &sm.dead, a.status);
        const float4 *kp = sm.kp[j & 3];
        const uint32_t hid = sm.hidden[j & 3];
        wait(&sm.s_full[i], j & 1, &sm.dead, a.status);
        tc_fence_after();
        union {
          uint32_t u[4][32];
          float f[128];
          uint64_t d[64];
        } t;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tm_s[i] + lanes + c * 32, t.u[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float4 x = kp[c];
          t.d[c] = fma2(t.d[c], pack2(x.x, x.y), mul2(pack2(x.z, x.w), qs2));
        }
        const bool whole = hid == 0 && k0 + kKeys <= min(tmin + 1, job.len) &&
                           (a.window <= 0 || k0 > tmax - a.window || k0 + kKeys <= a.sinks);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const int key = k0 + c;
            if (key >= vis || (key < wlo && key >= a.sinks) || (hid >> (c / 16) & 1)) t.f[c] = -INFINITY;
          }
        }
        float mx = t.f[0];
#pragma unroll
        for (int c = 1; c < 128; ++c) mx = fmaxf(mx, t.f[c]);
        if (__any_sync(0xffffffffu, mx > m + 8.f)) {
          const float nm = fmaxf(m, mx);
          const float al = ex2f(m - nm);
          m = nm;
          l2 = mul2(l2, pack2(al, al));
          if (j > 0) {
            wait(&sm.o_full[i], (j - 1) & 1, &sm.dead, a.status);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tm_o[i] + lanes + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tmem_st16(tm_o[i] + lanes + c * 16, o);
            }
            tmem_st_wait();
          }
        }
        const uint64_t shift = pack2(6.f - m, 6.f - m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 x = unpack2(add2(t.d[h * 32 + c], shift));
            const float p0 = ex2f(x.x), p1 = ex2f(x.y);
            l2 = add2(l2, pack2(p0, p1));
            w[c] = kv4_bits<uint32_t>(X::from2(p0, p1));
          }
          tmem_st32(tm_s[i] + lanes + h * 32, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[i]);
      }
      // ---- the row's result.  Column c of O is dim 2c, column D/2 + c dim 2c + 1.
      float inv = 0.f;
      if (n > 0) {
        const float2 l = unpack2(l2);
        const float sum = l.x + l.y;
        inv = sum == 0.f ? 0.f : 1.f / sum;
        wait(&sm.o_full[i], (n - 1) & 1, &sm.dead, a.status);
        tc_fence_after();
      }
      T *op = static_cast<T *>(a.out) + (job.row0 + static_cast<int64_t>(qi)) * a.o_row + head_q * a.o_head;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t e0[16], e1[16];
        if (n > 0) {
          tmem_ld16(tm_o[i] + lanes + c * 16, e0);
          tmem_ld16(tm_o[i] + lanes + D / 2 + c * 16, e1);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) e0[e] = e1[e] = 0;
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = kv4_bits<uint32_t>(X::from2(__uint_as_float(e0[e]) * inv, __uint_as_float(e1[e]) * inv));
        if (valid) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4 *>(op)[c * 4 + e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
      tc_fence_before();
    }
  } else if (warp < 16) {
    // -------------------------------------------------------------- unpack
    reg_dec<kRegsUnpack>();
    const int rw = warp - 8, g = lane >> 2, t = lane & 3;
    const float sl2 = a.scale * 1.4426950408889634f;
    const uint8_t *base = a.c.pages + static_cast<int64_t>(head) * a.c.recs_per_page * REC;
    const int32_t *table = a.b.table + job.seq * a.b.table_stride;
    uint4 k[2], v[D / 64];
    uint32_t pr = 0;  // lane's (s, lo): token lane % 16, of K below lane 16 and V above
    int state = 0;    // of the loaded record: 0 beyond the keys, 1 loaded, 2 page not usable
    int page = -1;
    auto load_page = [&](int j) {
      page = -1;
      if (j >= n) return;
      const int key = job.key0(j) + rw * 16;
      if (key < job.len) page = __ldg(table + key / 16 / a.c.recs_per_page);
    };
    auto load = [&](int j) {
      k[0] = k[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) v[c] = make_uint4(0, 0, 0, 0);
      pr = 0;
      state = 0;
      if (j >= n) return;
      const int key = job.key0(j) + rw * 16;
      if (key >= job.len) return;
      if (page < 0 || page >= a.c.n_pages) {
        state = 2;
        if (lane == 0) record_error(a.status, kErrInvalidArg);
        return;
      }
      state = 1;
      const uint8_t *rec = base + page * a.c.page_stride + (key / 16 % a.c.recs_per_page) * REC;
      if (D == 128) {
        k[0] = __ldg(reinterpret_cast<const uint4 *>(rec) + lane);
        k[1] = __ldg(reinterpret_cast<const uint4 *>(rec + 512) + lane);
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(rec) + lane);
        const uint2 y = __ldg(reinterpret_cast<const uint2 *>(rec + 256) + lane);
        k[0] = make_uint4(x.x, x.y, y.x, y.y);
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) v[c] = __ldg(reinterpret_cast<const uint4 *>(rec + 8 * D + c * 512) + lane);
      pr = __ldg(reinterpret_cast<const uint32_t *>(rec + 16 * D) + lane);
    };
    load_page(0);
    load(0);
    load_page(1);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int st = j & 1;
      // pairs: a row whose own K or V pair is not finite scores NaN and has V = 0, so that
      // only queries that see it become NaN
      float2 own = kv4_pair<BF>(pr);
      const bool fin = (own.x + own.y) - (own.x + own.y) == 0.f;
      const bool both = __shfl_xor_sync(0xffffffffu, static_cast<int>(fin), 16) && fin;
      if (j >= 2) wait(&sm.k_empty[st], (j / 2 - 1) & 1, &sm.dead, a.status);
      if (lane < 16) {
        float *kp = reinterpret_cast<float *>(&sm.kp[j & 3][rw * 8 + lane / 2]) + (lane & 1);
        kp[0] = both ? own.x * sl2 : 0.f;
        kp[2] = both ? own.y * sl2 : NAN;
      }
      if (state == 2 && lane == 0) atomicOr(&sm.hidden[j & 3], 1u << rw);
      if (state != 2 && lane == 0) atomicAnd(&sm.hidden[j & 3], ~(1u << rw));
      // ---- K codes: lane (g, t) has dims [t D/4, (t+1) D/4) of keys g and g + 8
      uint8_t *kt = sm.k[st];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = rw * 16 + h * 8 + g;
        uint32_t w[WORDS];
        if (D == 128) {
          w[0] = k[h].x, w[1] = k[h].y, w[WORDS - 2] = k[h].z, w[WORDS - 1] = k[h].w;
        } else {
          w[0] = h ? k[0].z : k[0].x, w[1] = h ? k[0].w : k[0].y;
        }
#pragma unroll
        for (int x = 0; x < WORDS; ++x) {
          // lanes t >= 2 take their words in another order: eight lanes of a 16-byte store then hit
          // eight different 16-byte banks
          const int y = D == 128 ? x ^ (t & 2) : x;
          uint32_t word = w[x];
          if (D == 128) word = (t & 2) ? w[x ^ 2] : w[x];
          T2 c[4];
          Codes<T>::pairs(word, c);
          const int chunk = t * WORDS + y;  // 16-byte chunk of the row: 8 dims
          *reinterpret_cast<uint4 *>(kt + (chunk / 8) * 16384 + key * 128 + (((chunk & 7) ^ g) << 4)) =
              make_uint4(kv4_bits<uint32_t>(c[0]), kv4_bits<uint32_t>(c[1]), kv4_bits<uint32_t>(c[2]),
                         kv4_bits<uint32_t>(c[3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.k_full[st]);
        mbar_arrive(&sm.par_full[j & 3]);
      }
      // ---- V rows, transposed: tile row = dim (2b at b, 2b + 1 at D/2 + b), 64 keys per 128-byte atom
      if (j >= 2) wait(&sm.v_empty[st], (j / 2 - 1) & 1, &sm.dead, a.status);
      {
        // (s, lo) of this lane's tokens 2t, 2t+1 and 2t+8, 2t+9 in the type
        const uint32_t use = both ? pr : 0u;
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = __shfl_sync(0xffffffffu, use, 16 + 2 * t + (e & 1) + 8 * (e >> 1));
        const T2 s0 = kv4_bits<T2>(__byte_perm(q[0], q[1], 0x5410)), l0 = kv4_bits<T2>(__byte_perm(q[0], q[1], 0x7632));
        const T2 s1 = kv4_bits<T2>(__byte_perm(q[2], q[3], 0x5410)), l1 = kv4_bits<T2>(__byte_perm(q[2], q[3], 0x7632));
        const T2 top = X::from2(X::max_finite, X::max_finite);
        uint8_t *vt = sm.v[st] + (rw / 4) * (D * 128) + 4 * t;
        const int c0 = (rw & 3) * 2;  // chunk of tokens 0..7 of the record
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            T2 o[4];  // (dim 2b, tokens 2t..), (2b + 1, 2t..), (2b, 2t+8..), (2b + 1, 2t+8..)
            Codes<T>::pairs(w[x], o);
            uint8_t *row = vt + (c * 32 + x * 8 + g) * 128;
            const int at0 = (c0 ^ g) << 4, at1 = ((c0 + 1) ^ g) << 4;
            // 15 s + lo can pass the type's largest value (s is rounded): hold it there
            *reinterpret_cast<T2 *>(row + at0) = __hmin2(__hfma2(o[0], s0, l0), top);
            *reinterpret_cast<T2 *>(row + D * 64 + at0) = __hmin2(__hfma2(o[1], s0, l0), top);
            *reinterpret_cast<T2 *>(row + at1) = __hmin2(__hfma2(o[2], s1, l1), top);
            *reinterpret_cast<T2 *>(row + D * 64 + at1) = __hmin2(__hfma2(o[3], s1, l1), top);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[st]);
      load(j + 1);
      load_page(j + 2);
    }
  } else {
    // ----------------------------------------------------------------- MMA
    reg_dec<kRegsMma>();
    if (warp == 16 && lane == 0 && n > 0) {
      constexpr uint32_t kind = BF ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t id_qk = idesc_f16_f32(128, kKeys) | kind, id_pv = idesc_f16_f32(128, D) | kind;
      auto qk = [&](int i, int j) {
        const uint64_t qd = sw128_kmajor_desc(smem_u32(sm.q[i])), kd = sw128_kmajor_desc(smem_u32(sm.k[j & 1]));
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint64_t adv = (x / 4) * (16384 >> 4) + (x % 4) * 2;
          mma_f16(tm_s[i], qd + adv, kd + adv, id_qk, x > 0);
        }
        mma_commit(&sm.s_full[i]);
      };
      auto pv = [&](int i, int j) {
        const uint64_t vd = sw128_kmajor_desc(smem_u32(sm.v[j & 1]));
#pragma unroll
        for (int x = 0; x < kKeys / 16; ++x) {
          const uint64_t adv = (x / 4) * ((D * 128) >> 4) + (x % 4) * 2;
          mma_f16_ts(tm_o[i], tm_s[i] + x * 8, vd + adv, id_pv, j > 0 || x > 0);
        }
        mma_commit(&sm.o_full[i]);
      };
      wait(&sm.k_full[0], 0, &sm.dead, a.status);
      for (int i = 0; i < row_tiles; ++i) {
        wait(&sm.q_full[i], 0, &sm.dead, a.status);
        tc_fence_after();
        qk(i, 0);
      }
      mma_commit(&sm.k_empty[0]);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        for (int i = 0; i < row_tiles; ++i) {
          if (i == 0) wait(&sm.v_full[j & 1], (j / 2) & 1, &sm.dead, a.status);
          wait(&sm.p_full[i], j & 1, &sm.dead, a.status);
          tc_fence_after();
          pv(i, j);
          if (i == row_tiles - 1) mma_commit(&sm.v_empty[j & 1]);
          if (j + 1 < n) {
            if (i == 0) {
              wait(&sm.k_full[(j + 1) & 1], ((j + 1) / 2) & 1, &sm.dead, a.status);
              tc_fence_after();
            }
            qk(i, j + 1);
            if (i == row_tiles - 1) mma_commit(&sm.k_empty[(j + 1) & 1]);
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D>
cudaError_t launch(const Kv4AttnArgs &a, cudaStream_t stream) {
  auto kernel = kv4_tile_kernel<T, D>;
  const int smem = static_cast<int>(sizeof(TileSmem<D>));
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t v = static_cast<int64_t>(a.b.rows) * a.group / kRows + a.b.n_seqs;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.c.n_kv, static_cast<unsigned>(v), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv4_tile(const Kv4AttnArgs &a, cudaStream_t stream) {
  if (a.c.bf16)
    return a.c.d == 128 ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
  return a.c.d == 128 ? launch<__half, 128>(a, stream) : launch<__half, 64>(a, stream);
}

}  // namespace mixq
