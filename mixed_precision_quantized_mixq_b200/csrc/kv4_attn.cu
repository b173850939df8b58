// Attention over the 4-bit KV cache for few query rows (decode steps, and any
// call the tile kernel does not take).
//
//   S_j = scale * (s_k (q . c_j) + lo_k sum(q)),  o = sum_j p_j (s_v c_j + lo_v) / sum_j p_j
//
// so the 4-bit codes themselves are matrix operands and the (s, lo) pairs act on
// the 16 scores and weights of a record instead of its 16*D values.  A code c is
// used as the fp16 subnormal c * 2^-24 (low nibble of a 16-bit lane) or
// c * 2^-20 (second nibble): a mask per pair of codes, no conversion, exact
// products, and the powers of two come out again in fp32.
//
// Tokens are the M side of the matrix instructions (m16n8k16) and query rows
// the N side, so the 8 or 16 rows a decode step has per kv head fill the
// instruction.  Everything a warp touches of a record is contiguous per lane
// (layout in kv4.h): two 16-byte shared loads for K, two for V.
//
// The cache is read once: HBM bounds the kernel.  Each warp keeps its own ring
// of records in flight (one bulk copy each, one mbarrier per slot), so no warp
// waits for another in the loop.  The records of all (sequence, head, row
// tile) items are one line, cut into equal parts over a persistent grid: the
// load is even whatever the lengths, and the host needs to know none of them.
// An item cut by such a boundary leaves fp32 partial results in the workspace,
// which a second, dependent launch joins in the order of the parts.
#include <cuda_runtime.h>

#include <atomic>

#include "kv4.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace mixq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kNegBig = -1e30f;  // running maximum before the first visible key
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMinQuota = 16;  // records: below two a warp, a cut costs more than it spreads
constexpr int kMaxRows = 16;

struct Desc {  // item whose last part is not in the CTA that starts it
  int seq, item, last, pad;
};

__host__ __device__ constexpr size_t slot_floats(int d) { return kMaxRows * static_cast<size_t>(d) + 2 * kMaxRows; }

// What the walk needs to know of a sequence.
struct Seq {
  int row0, nq;     // query rows in the q tensor
  int len;          // keys that exist (bounded by the table)
  int pos0;         // position of the first new token
  int tiles;        // row tiles per kv head
  int n_rec;        // records visited per item (at least 1 if there are rows)
  int skip_at, skip_by;  // record index i >= skip_at means record i + skip_by
};

template <int R>
__device__ __forceinline__ Seq load_seq(const Kv4AttnArgs &a, int s) {
  Seq q{};
  bool bad = false;
  const int2 r = kv4_row_range(a.b, s, &bad);
  q.row0 = r.x;
  q.nq = r.y - r.x;
  const int full = __ldg(a.b.lens + s);
  const int64_t cap = static_cast<int64_t>(a.b.table_width) * a.c.recs_per_page * kKv4Rec;
  q.len = static_cast<int>(min(static_cast<int64_t>(max(full, 0)), cap));
  if (bad || full < 0 || full > cap) {
    if (threadIdx.x == 0) record_error(a.status, kErrInvalidArg);
  }
  q.pos0 = full - q.nq;
  const int64_t rows = static_cast<int64_t>(q.nq) * a.group;
  q.tiles = rows > a.tile_above ? 0 : static_cast<int>((rows + R - 1) / R);
  const int total = (q.len + kKv4Rec - 1) / kKv4Rec;
  q.skip_at = total;
  q.skip_by = 0;
  q.n_rec = total;
  if (a.window > 0) {
    const int first = max(0, max(q.pos0, 0) - a.window + 1) / kKv4Rec;  // first record of the window
    const int sink = min((min(a.sinks, q.len) + kKv4Rec - 1) / kKv4Rec, first);
    q.skip_at = sink;
    q.skip_by = min(first, total) - sink;
    q.n_rec = total - q.skip_by;
  }
  q.n_rec = max(q.n_rec, 1);
  return q;
}

__device__ __forceinline__ int64_t seq_cost(const Seq &q, int n_kv) {
  return static_cast<int64_t>(q.tiles) * n_kv * q.n_rec;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  return kv4_bits<uint32_t>(__floats2half2_rn(a, b));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Position on the line of records, relative to the CTA's first record.
template <int R>
struct Walk {
  Seq q;
  int seq, item, start;  // start of the item

  __device__ __forceinline__ int items(const Kv4AttnArgs &a) const { return q.tiles * a.c.n_kv; }
  // to the item that holds position i (the caller keeps i below the CTA's end)
  __device__ __forceinline__ void seek(const Kv4AttnArgs &a, int i) {
    while (i >= start + q.n_rec) {
      start += q.n_rec;
      if (++item >= items(a)) {
        item = 0;
        do {
          q = load_seq<R>(a, ++seq);
        } while (q.tiles == 0 && seq + 1 < a.b.n_seqs);
      }
    }
  }
  __device__ __forceinline__ int head(const Kv4AttnArgs &) const { return item / q.tiles; }
  __device__ __forceinline__ int record(int i) const {
    const int r = i - start;
    return r + (r >= q.skip_at ? q.skip_by : 0);
  }
};

template <int D, int NT, int SLOTS>
struct Smem {
  static constexpr int REC = kv4_rec_bytes(D);
  static constexpr int R = 8 * NT;
  static constexpr int OROW = D + 4;  // padded row: float2 stores of the four t lanes hit other banks
  alignas(128) uint8_t ring[kWarps][SLOTS][REC];
  alignas(16) float o[kWarps][R][OROW];
  float m[kWarps][R], l[kWarps][R];
  uint64_t full[kWarps][SLOTS];
  int ok[kWarps][SLOTS];
  long long scan[kWarps + 1];
  int found_seq;
  long long found_start;
};

template <typename T, int D, int NT, int SLOTS>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv4_attn_kernel(const Kv4AttnArgs a) {
  constexpr int R = 8 * NT, WORDS = D / 32, MT = D / 16, REC = kv4_rec_bytes(D);
  constexpr bool BF = Kv4Type<T>::bf16;
  using S = Smem<D, NT, SLOTS>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S &sm = *reinterpret_cast<S *>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane >> 2, t = lane & 3;

  if (tid < kWarps * SLOTS) mbar_init(&sm.full[tid / SLOTS][tid % SLOTS], 1);
  fence_mbar_init();
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's part of the line
  long long mine = 0;
  for (int s = tid; s < a.b.n_seqs; s += kThreads) mine += seq_cost(load_seq<R>(a, s), a.c.n_kv);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sm.scan[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sm.scan[w];
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long quota = per > kMinQuota ? per : kMinQuota;
  const long long lo = min(static_cast<long long>(blockIdx.x) * quota, total);
  const int mylen = static_cast<int>(min(quota, total - lo));
  Desc *desc = reinterpret_cast<Desc *>(a.work);
  float *slots = a.work + gridDim.x * (sizeof(Desc) / 4);
  if (mylen == 0) {
    if (tid == 0) desc[blockIdx.x].seq = -1;
    return;
  }
  // the sequence that holds position lo
  long long base = 0;
  for (int s0 = 0; s0 < a.b.n_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    const long long cost = s < a.b.n_seqs ? seq_cost(load_seq<R>(a, s), a.c.n_kv) : 0;
    long long incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    long long before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.scan[w];
      all += sm.scan[w];
    }
    const long long start = before + incl - cost;
    if (lo >= start && lo < start + cost) {
      sm.found_seq = s;
      sm.found_start = start;
    }
    base += all;
    if (base > lo) break;
  }
  __syncthreads();

  Walk<R> cur;
  cur.seq = sm.found_seq;
  cur.q = load_seq<R>(a, cur.seq);
  {
    const long long in = lo - sm.found_start;
    cur.item = static_cast<int>(in / cur.q.n_rec);
    cur.start = static_cast<int>(static_cast<long long>(cur.item) * cur.q.n_rec - in);
  }

  // ---- the warp's ring.  Two steps ahead of the copy: the page of the next
  // record is loaded one turn before its copy is issued.
  Walk<R> pre = cur;
  int pre_i = warp;       // position whose page is in pre_page
  int pre_page = -1;
  int64_t pre_off = 0;
  uint32_t issued = 0;
  const uint64_t policy = policy_evict_first();
  auto load_page = [&]() {
    pre_page = -1;
    if (pre_i >= mylen) return;
    pre.seek(a, pre_i);
    const int rec = pre.record(pre_i);
    if (rec * kKv4Rec >= pre.q.len) return;
    const int slot = a.c.page_shift >= 0 ? rec >> a.c.page_shift : rec / a.c.recs_per_page;
    pre_page = __ldg(a.b.table + pre.seq * a.b.table_stride + slot);
    pre_off = (static_cast<int64_t>(pre.head(a)) * a.c.recs_per_page + (rec - slot * a.c.recs_per_page)) * REC;
  };
  auto issue = [&]() {
    if (pre_i < mylen) {
      if (lane == 0) {
        const int slot = issued % SLOTS;
        uint64_t *bar = &sm.full[warp][slot];
        const bool ok = pre_page >= 0 && pre_page < a.c.n_pages;
        sm.ok[warp][slot] = ok;
        if (ok) {
          mbar_arrive_expect_tx(bar, REC);
          bulk_load(sm.ring[warp][slot], a.c.pages + pre_page * a.c.page_stride + pre_off, REC, bar, policy);
        } else {
          if (pre.q.len > 0 && pre.record(pre_i) * kKv4Rec < pre.q.len) record_error(a.status, kErrInvalidArg);
          mbar_arrive(bar);
        }
      }
      ++issued;
      pre_i += kWarps;
    }
    load_page();
  };
  load_page();
#pragma unroll 1
  for (int i = 0; i < SLOTS; ++i) issue();

  uint32_t used = 0;
  bool dead = false;
  const float sl2 = a.scale * 1.4426950408889634f;

#pragma unroll 1
  for (int pos = 0; pos < mylen;) {
    cur.seek(a, pos);
    const int seg_end = min(cur.start + cur.q.n_rec, mylen);
    const int head = cur.head(a), tile = cur.item - head * cur.q.tiles;
    const int row_first = tile * R, rows_all = cur.q.nq * a.group;

    // ---- query fragments: column n = query row, lane t holds dims [t D/4, (t+1) D/4)
    uint32_t qf[NT][WORDS][4];
    float cs[NT][2], qs[NT][2];
    int vis[NT][2], wlo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row_first + nt * 8 + g;
      const bool valid = r < rows_all;
      const int qi = r / a.group;
      const T *qp = static_cast<const T *>(a.q) + (cur.q.row0 + static_cast<int64_t>(qi)) * a.q_row +
                    (static_cast<int64_t>(head) * a.group + (r - qi * a.group)) * a.q_head + t * (D / 4);
      uint4 raw[WORDS];
#pragma unroll
      for (int w = 0; w < WORDS; ++w)
        raw[w] = valid ? __ldg(reinterpret_cast<const uint4 *>(qp) + w) : make_uint4(0, 0, 0, 0);
      float sum = 0.f;
      int e = 0;
      if (BF) {
        // bf16 rows go to fp16 under a power of two that puts the row's largest
        // value into [2^13, 2^14): exact down to 2^-30 of it
        float mx = 0.f;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          const uint32_t u[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(u[i] << 16)),
                                 fabsf(__uint_as_float(u[i] & 0xffff0000u))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
        e = max(-100, ex - 13);
      }
      const float down = BF ? pow2(-e) : 1.f;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        const uint32_t u[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          if (BF) {
            x = __uint_as_float(u[i] << 16) * down;
            y = __uint_as_float(u[i] & 0xffff0000u) * down;
            qf[nt][w][i] = pack_half2(x, y);
          } else {
            const float2 f = __half22float2(kv4_bits<__half2>(u[i]));
            x = f.x;
            y = f.y;
            qf[nt][w][i] = u[i];
          }
          sum += x;
          sum += y;
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float up = sl2 * (BF ? pow2(e) : 1.f);
      const float mycs = up * 16777216.f, myqs = up * sum;
      const int p = cur.q.pos0 + qi;
      const int myvis = valid ? min(p + 1, cur.q.len) : 0x7fffffff;
      const int mywlo = valid && a.window > 0 ? max(p, 0) - a.window + 1 : -0x7fffffff;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int src = (2 * t + j) * 4;
        cs[nt][j] = __shfl_sync(0xffffffffu, mycs, src);
        qs[nt][j] = __shfl_sync(0xffffffffu, myqs, src);
        vis[nt][j] = __shfl_sync(0xffffffffu, myvis, src);
        wlo[nt][j] = __shfl_sync(0xffffffffu, mywlo, src);
      }
    }
    // positions of the tile's first and last row
    const int pmin = cur.q.pos0 + row_first / a.group;
    const int pmax = cur.q.pos0 + (min(row_first + R, rows_all) - 1) / a.group;
    // keys up to these lie before the window of the first and of the last row (a row at a
    // negative position sees nothing: 0 stands for it, and no difference leaves 32 bits)
    const int edge_min = max(pmin, 0) - a.window, edge_max = max(pmax, 0) - a.window;

    float o[NT][MT][4], m[NT][2], l[NT][2], z[NT][2];
    float sig = pow2(100);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = kNegBig;
        l[nt][j] = 0.f;
        z[nt][j] = 0.f;
      }
    }

    // ---- the warp's records of this segment
#pragma unroll 1
    for (int i = pos + ((warp - pos) & (kWarps - 1)); i < seg_end; i += kWarps) {
      const int slot = used % SLOTS;
      if (!dead && !mbar_wait(&sm.full[warp][slot], (used / SLOTS) & 1, kWaitNs)) {
        dead = true;
        if (lane == 0) record_error(a.status, kErrTimeout);
      }
      ++used;
      const uint8_t *rec = sm.ring[warp][slot];
      const bool ok = sm.ok[warp][slot] && !dead;
      const int j0 = cur.record(i) * kKv4Rec;
      const bool none = !ok || j0 > pmax || (a.window > 0 && j0 + kKv4Rec <= edge_min + 1 && j0 >= a.sinks);
      if (!none) {
        uint32_t ka[WORDS], kb[WORDS], vw[WORDS * 2];
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4 *>(rec + lane * 16);
          const uint4 y = *reinterpret_cast<const uint4 *>(rec + 512 + lane * 16);
          ka[0] = x.x, ka[1] = x.y, ka[WORDS - 2] = x.z, ka[WORDS - 1] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[WORDS - 2] = y.z, kb[WORDS - 1] = y.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(rec + lane * 8);
          const uint2 y = *reinterpret_cast<const uint2 *>(rec + 256 + lane * 8);
          ka[0] = x.x, ka[1] = x.y, kb[0] = y.x, kb[1] = y.y;
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 x = *reinterpret_cast<const uint4 *>(rec + 8 * D + c * 512 + lane * 16);
          vw[4 * c] = x.x, vw[4 * c + 1] = x.y, vw[4 * c + 2] = x.z, vw[4 * c + 3] = x.w;
        }
        const uint32_t *pk = reinterpret_cast<const uint32_t *>(rec + 16 * D);
        float2 kp0 = kv4_pair<BF>(pk[g]), kp1 = kv4_pair<BF>(pk[g + 8]);
        // an infinite pair makes the score NaN, not one more hidden key at -inf
        kp0.x = fmaf(kp0.x + kp0.y, 0.f, kp0.x);
        kp1.x = fmaf(kp1.x + kp1.y, 0.f, kp1.x);
        const float2 v0 = kv4_pair<BF>(pk[16 + g]), v1 = kv4_pair<BF>(pk[24 + g]);

        // scores of tokens g and g + 8 for columns 2t, 2t + 1
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < WORDS; ++w) {
            const uint32_t a8 = ka[w] >> 8, b8 = kb[w] >> 8;
            mma16816(x, ka[w] & 0x000f000fu, kb[w] & 0x000f000fu, a8 & 0x000f000fu,
                     b8 & 0x000f000fu, qf[nt][w][0], qf[nt][w][2]);
            mma16816(y, ka[w] & 0x00f000f0u, kb[w] & 0x00f000f0u, a8 & 0x00f000f0u,
                     b8 & 0x00f000f0u, qf[nt][w][1], qf[nt][w][3]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 k = j < 2 ? kp0 : kp1;
            const float raw = fmaf(y[j], 0.0625f, x[j]);
            s[nt][j] = fmaf(raw * k.x, cs[nt][j & 1], k.y * qs[nt][j & 1]);
          }
        }
        const bool whole = j0 + kKv4Rec <= min(pmin + 1, cur.q.len) &&
                           (a.window <= 0 || j0 > edge_max || j0 + kKv4Rec <= a.sinks);
        float s0 = v0.x, s1 = v1.x, l0 = v0.y, l1 = v1.y;
        if (!whole) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = j0 + g + (j < 2 ? 0 : 8);
              if (key >= vis[nt][j & 1] || (key < wlo[nt][j & 1] && key >= a.sinks)) s[nt][j] = -INFINITY;
            }
          // tokens that no row of the tile sees may hold anything
          const int k0 = j0 + g, k1 = k0 + 8, last = min(pmax, cur.q.len - 1);
          if (k0 > last || (a.window > 0 && k0 <= edge_min && k0 >= a.sinks)) s0 = 0.f, l0 = 0.f;
          if (k1 > last || (a.window > 0 && k1 <= edge_min && k1 >= a.sinks)) s1 = 0.f, l1 = 0.f;
        }

        // ---- running maximum, moved only when a score passes it by 2^8
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) grow |= s[nt][j] > m[nt][j & 1] + 8.f;
        // V scales go to [2^6, 2^7) of the largest seen, so weights times scale
        // stay below 2^15 and keep fp16's 11 bits down to 2^-21 of the largest
        const float smax = fmaxf(s0, s1);
        const bool rescale = smax * sig >= 128.f;
        if (__any_sync(0xffffffffu, grow || rescale)) {
          float f = 1.f;
          float mx = smax < INFINITY ? fmaxf(smax, 0.f) : 0.f;
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx * sig >= 128.f) {
            const float nsig = pow2(6 + 127 - static_cast<int>(__float_as_uint(mx) >> 23));
            f = nsig / sig;
            sig = nsig;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float al[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float n = fmaxf(s[nt][j], s[nt][j + 2]);
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16));
              n = fmaxf(n, m[nt][j]);
              al[j] = ex2(m[nt][j] - n);
              m[nt][j] = n;
              l[nt][j] *= al[j];
              z[nt][j] *= al[j];
              al[j] *= f;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][0] *= al[0];
              o[nt][i][1] *= al[1];
              o[nt][i][2] *= al[0];
              o[nt][i][3] *= al[1];
            }
          }
        }

        // ---- weights, their sums, and the products with V
        s0 *= sig;
        s1 *= sig;
        uint32_t p0[NT], p1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ex2(s[nt][j] - m[nt][j & 1]);
            l[nt][j & 1] += p[j];
          }
          float w[4];
          if (whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[nt][j & 1] = fmaf(p[j], j < 2 ? l0 : l1, z[nt][j & 1]);
              w[j] = p[j] * (j < 2 ? s0 : s1);
            }
          } else {
            // a key hidden from this row must not reach it through 0 * NaN
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool hid = s[nt][j] == -INFINITY;
              z[nt][j & 1] += hid ? 0.f : p[j] * (j < 2 ? l0 : l1);
              w[j] = hid ? 0.f : p[j] * (j < 2 ? s0 : s1);
            }
          }
          p0[nt] = transpose8x8(pack_half2(w[0], w[1]));
          p1[nt] = transpose8x8(pack_half2(w[2], w[3]));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t v8 = vw[i] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[nt][i], vw[i] & 0x000f000fu, vw[i] & 0x00f000f0u, v8 & 0x000f000fu,
                     v8 & 0x00f000f0u, p0[nt], p1[nt]);
        }
      }
      __syncwarp();
      issue();
    }

    // ---- join the warps.  Rows 8 m + g of the products are dims 2 (8 m + g) (x 2^-24)
    // and 2 (8 m + g) + 1 (x 2^-20).
    const float un = 1.f / sig;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float lj = l[nt][j], zj = z[nt][j];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          lj += __shfl_xor_sync(0xffffffffu, lj, x);
          zj += __shfl_xor_sync(0xffffffffu, zj, x);
        }
        const int col = nt * 8 + 2 * t + j;
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<float2 *>(&sm.o[warp][col][2 * (8 * i + g)]) =
              make_float2(fmaf(o[nt][i][j] * 16777216.f, un, zj), fmaf(o[nt][i][j + 2] * 1048576.f, un, zj));
        if (g == 0) {
          sm.m[warp][col] = m[nt][j];
          sm.l[warp][col] = lj;
        }
      }
    __syncthreads();
    const bool begins = cur.start >= 0, ends = cur.start + cur.q.n_rec <= mylen;
    float *part = slots + (2 * blockIdx.x + (begins ? 1 : 0)) * slot_floats(D);
    for (int e = tid; e < R * D / 4; e += kThreads) {
      const int r = e / (D / 4), d = (e % (D / 4)) * 4;
      if (row_first + r >= rows_all) continue;
      float mx = sm.m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][r]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(sm.m[w][r] - mx);
        const float4 x = *reinterpret_cast<const float4 *>(&sm.o[w][r][d]);
        sum = fmaf(f, sm.l[w][r], sum);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      if (begins && ends) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int rr = row_first + r, qi = rr / a.group;
        T *op = static_cast<T *>(a.out) + (cur.q.row0 + static_cast<int64_t>(qi)) * a.o_row +
                (static_cast<int64_t>(head) * a.group + (rr - qi * a.group)) * a.o_head + d;
        using X = Kv4Type<T>;
        uint2 v;
        v.x = kv4_bits<uint32_t>(X::from2(acc.x * inv, acc.y * inv));
        v.y = kv4_bits<uint32_t>(X::from2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2 *>(op) = v;
      } else {
        *reinterpret_cast<float4 *>(part + r * D + d) = acc;
        if (d == 0) {
          part[kMaxRows * D + r] = mx;
          part[kMaxRows * D + kMaxRows + r] = sum;
        }
      }
    }
    __syncthreads();
    if (tid == 0 && seg_end == mylen) {
      Desc x{-1, 0, 0, 0};
      if (begins && !ends) {
        const long long end = lo + cur.start + cur.q.n_rec;
        x = Desc{cur.seq, cur.item, static_cast<int>((end - 1) / quota), 0};
      }
      desc[blockIdx.x] = x;
    }
    pos = seg_end;
  }
  // after a wait that ran out, do not leave while copies may still land here
  if (dead)
    for (uint32_t i = used > SLOTS ? used - SLOTS : 0; i < issued; ++i)
      mbar_wait(&sm.full[warp][i % SLOTS], (i / SLOTS) & 1, kWaitNs / 16);
}

// Joins the parts of the item that starts in part blockIdx.x and ends later.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads) kv4_join_kernel(const Kv4AttnArgs a) {
  constexpr int R = 8 * NT;
  griddep_wait();
  griddep_launch_dependents();
  const Desc *desc = reinterpret_cast<const Desc *>(a.work);
  const float *slots = a.work + gridDim.x * (sizeof(Desc) / 4);
  const Desc x = desc[blockIdx.x];
  if (x.seq < 0) return;
  const Seq q = load_seq<R>(a, x.seq);
  const int head = x.item / q.tiles, row_first = (x.item - head * q.tiles) * R;
  const int rows_all = q.nq * a.group, c0 = blockIdx.x;
  for (int e = threadIdx.x; e < R * D / 4; e += kThreads) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    const int rr = row_first + r;
    if (rr >= rows_all) continue;
    float mx = kNegBig, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0; c <= x.last; ++c)
      mx = fmaxf(mx, slots[(2 * c + (c == c0)) * slot_floats(D) + kMaxRows * D + r]);
#pragma unroll 4
    for (int c = c0; c <= x.last; ++c) {
      const float *p = slots + (2 * c + (c == c0)) * slot_floats(D);
      const float f = ex2(p[kMaxRows * D + r] - mx);
      const float4 v = *reinterpret_cast<const float4 *>(p + r * D + d);
      sum = fmaf(f, p[kMaxRows * D + kMaxRows + r], sum);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int qi = rr / a.group;
    T *op = static_cast<T *>(a.out) + (q.row0 + static_cast<int64_t>(qi)) * a.o_row +
            (static_cast<int64_t>(head) * a.group + (rr - qi * a.group)) * a.o_head + d;
    using X = Kv4Type<T>;
    uint2 o;
    o.x = kv4_bits<uint32_t>(X::from2(acc.x * inv, acc.y * inv));
    o.y = kv4_bits<uint32_t>(X::from2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(op) = o;
  }
}

template <typename T, int D, int NT>
cudaError_t launch(const Kv4AttnArgs &a, cudaStream_t stream) {
  constexpr int SLOTS = NT == 1 ? 4 : 6;
  auto kernel = kv4_attn_kernel<T, D, NT, SLOTS>;
  const int smem = static_cast<int>(sizeof(Smem<D, NT, SLOTS>));
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.num_sms * (NT == 1 ? 2 : 1), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, D, NT>, a);
}

template <typename T, int D>
cudaError_t pick(const Kv4AttnArgs &a, cudaStream_t stream) {
  // 8 rows per tile while a sequence's rows of a kv head fit one such tile
  return a.max_rows <= 8 ? launch<T, D, 1>(a, stream) : launch<T, D, 2>(a, stream);
}

}  // namespace

size_t kv4_step_workspace(int d, int num_sms) {
  const size_t ctas = 2 * static_cast<size_t>(num_sms);
  return ctas * sizeof(Desc) + ctas * 2 * slot_floats(d) * sizeof(float);
}

cudaError_t launch_kv4_attn(Kv4AttnArgs a, cudaStream_t stream) {
  // A sequence with more than kKv4TileAbove rows per kv head goes to the tile kernel; the lengths are
  // on the device, so a call whose bound allows both kinds launches both, and each skips the other's.
  a.tile_above = INT64_MAX;
  if (a.max_rows > kKv4TileAbove) {
    a.tile_above = kKv4TileAbove;
    const cudaError_t e = launch_kv4_tile(a, stream);
    if (e != cudaSuccess) return e;
    a.max_rows = kKv4TileAbove;
  }
  if (a.c.bf16)
    return a.c.d == 128 ? pick<__nv_bfloat16, 128>(a, stream) : pick<__nv_bfloat16, 64>(a, stream);
  return a.c.d == 128 ? pick<__half, 128>(a, stream) : pick<__half, 64>(a, stream);
}

}  // namespace mixq
