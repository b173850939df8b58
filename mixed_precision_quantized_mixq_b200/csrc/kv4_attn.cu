// Attention over the 4-bit KV cache for few query rows (decode steps, and any
// call the tile kernel does not take).
//
//   S_j = scale * (s_k (q . c_j) + lo_k sum(q)),  o = sum_j p_j (s_v c_j + lo_v) / sum_j p_j
//
// so the 4-bit codes themselves are matrix operands and the (s, lo) pairs act on
// the 16 scores and weights of a record instead of its 16*D values.  A code c is
// used as the fp16 subnormal c * 2^-24 (low nibble of a 16-bit lane) or
// c * 2^-20 (second nibble): a mask per pair of codes, no conversion, exact
// products, and the powers of two are made up for in q or come out again in fp32.
//
// Tokens are the M side of the matrix instructions (m16n8k16) and query rows
// the N side, so the 8 or 16 rows a decode step has per kv head fill the
// instruction.  Everything a warp touches of a record is contiguous per lane
// (layout in kv4.h): two 16-byte shared loads for K, two for V.
//
// The cache is read once: HBM bounds the kernel, if the instructions per record
// stay few.  So a warp takes units of two records, looks pages up for 16 units at
// a time (a record a lane), and checks the running maximum by the sum of the
// weights.  Each warp keeps its own ring of units in flight (a bulk copy a record,
// one mbarrier per slot).  The units of all (sequence, head, row tile) items are
// one line, cut into equal parts over a persistent grid and each CTA's part again
// over its warps: the load is even whatever the lengths, the host needs to know
// none of them, and no warp waits for another before its span is done.
// An item cut between warps is joined in shared memory at the CTA's end; one cut
// between CTAs leaves fp32 partial results in the workspace, which a last,
// dependent launch joins in the order of the parts, those of the tile kernel too.
//
// What it measured (B200, warm launches, us against the bytes at the measured copy
// rate): 16 sequences of up to 4096 tokens, 32 / 32 heads, fp16 50 (30); 64 of up to
// 8192, 64 / 8 heads, bf16 85 (54); two of 131071, 64 / 8 heads, fp16 82 (44); a
// window of 4096 over 16 sequences, 32 / 8 heads 35 (11).  With the arithmetic left
// out the second takes 67, with the copies left out about as long as whole: about 260
// instructions a record and warp, 88 of them masks and shifts, at 0.55 issues a
// cycle (four warps a scheduler; more would need fewer than the 128 registers that
// the sums and queries take).  About 14 us of each call are before the first data
// and after the last: the look-up chain length -> page -> record, the join of the
// warps, and the second launch.  A spill in the loop costs most of all: 74 bytes of
// it made the second 184.  One warp's units next to each other (spans) against units
// dealt out in turn: 50 against 75 for the first, as no barrier is left between items.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "kv4.h"
#include "kv4_join.cuh"
#include "kv4_ptx.cuh"
#include "tma_host.h"

namespace mixq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kNegBig = -1e30f;  // running maximum before the first visible key
constexpr uint64_t kWaitNs = 2000000000ull, kStallWaitNs = 20000000ull;
constexpr int kUnit = 2;       // records
constexpr int kUnitKeys = kUnit * kKv4Rec;
constexpr int kMinQuota = 8;   // units: below one a warp, a cut costs more than it spreads
constexpr int kMaxRows = kKv4StepRows;

__host__ __device__ constexpr size_t slot_floats(int d) { return kv4_slot_floats(kMaxRows, d); }

// What the walk needs to know of a sequence.
struct Seq {
  int row0, nq;     // query rows in the q tensor
  int len;          // keys that exist (bounded by the table)
  int pos0;         // position of the first new token
  int tiles;        // row tiles per kv head
  int n_unit;       // units visited per item (at least 1 if there are rows)
  int skip_at, skip_by;  // unit index i >= skip_at means unit i + skip_by
};

// wrong: set if the sequence's offsets or length are not usable
template <int R>
__device__ __forceinline__ Seq load_seq(const Kv4AttnArgs &a, int s, bool *wrong = nullptr) {
  Seq q{};
  bool bad = false;
  const int2 r = kv4_row_range(a.b, s, &bad);
  q.row0 = r.x;
  q.nq = r.y - r.x;
  const int full = __ldg(a.b.lens + s);
  q.len = min(max(full, 0), a.room);
  if (wrong) *wrong = bad || full < 0 || full > a.room;
  q.pos0 = full - q.nq;
  const int64_t rows = static_cast<int64_t>(q.nq) * a.group;
  q.tiles = rows > a.tile_above ? 0 : static_cast<int>((rows + R - 1) / R);
  const int total = static_cast<int>((static_cast<unsigned>(q.len) + kUnitKeys - 1) / kUnitKeys);
  q.skip_at = total;
  q.skip_by = 0;
  q.n_unit = total;
  if (a.window > 0) {
    const int first = max(0, max(q.pos0, 0) - a.window + 1) / kUnitKeys;  // first unit of the window
    const int sink = min(static_cast<int>((static_cast<unsigned>(min(a.sinks, q.len)) + kUnitKeys - 1) / kUnitKeys), first);
    q.skip_at = sink;
    q.skip_by = min(first, total) - sink;
    q.n_unit = total - q.skip_by;
  }
  q.n_unit = max(q.n_unit, 1);
  return q;
}

__device__ __forceinline__ int64_t seq_cost(const Seq &q, int n_kv) {
  return static_cast<int64_t>(q.tiles) * n_kv * q.n_unit;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  return kv4_bits<uint32_t>(__floats2half2_rn(a, b));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Position on the line of units, relative to the CTA's first unit.
template <int R>
struct Walk {
  Seq q;
  int seq, item, start;  // start of the item

  __device__ __forceinline__ int items(const Kv4AttnArgs &a) const { return q.tiles * a.c.n_kv; }
  // to the item that holds position i (the caller keeps i below the CTA's end)
  __device__ __forceinline__ void seek(const Kv4AttnArgs &a, int i) {
    while (i >= start + q.n_unit) {
      const int by = min((i - start) / q.n_unit, items(a) - item);
      start += by * q.n_unit;
      item += by;
      if (item == items(a)) {
        item = 0;
        do {
          q = load_seq<R>(a, ++seq);
        } while (q.tiles == 0 && seq + 1 < a.b.n_seqs);
      }
    }
  }
  __device__ __forceinline__ int head(const Kv4AttnArgs &) const { return item / q.tiles; }
  __device__ __forceinline__ int unit(int i) const {
    const int r = i - start;
    return r + (r >= q.skip_at ? q.skip_by : 0);
  }
};

struct Place {  // of a part of an item
  int end;  // where the item ends in the CTA's part of the line
  int head, row0, row_first, rows;  // first q row of the sequence, first row and number of rows of the item
};

template <int D, int R, int SLOTS>
struct Smem {
  static constexpr int REC = kv4_rec_bytes(D);
  static constexpr int OROW = D + 4;  // padded row: float2 stores of the four t lanes hit other banks
  alignas(128) uint8_t ring[kWarps][SLOTS][kUnit][REC];
  float m[2][kWarps][R], l[2][kWarps][R];  // [0]: the item that a warp's span begins in, [1]: the one it ends in
  // bit 0: the first is there, 1: and ends here, 4: and is in the ring; 2: the second is there; 3: no span
  int part[kWarps];
  Place place[2][kWarps];
  uint64_t full[kWarps][SLOTS];
  int ok[kWarps][SLOTS];  // a bit per record
  int died[kWarps];       // slot * 2 + phase of the unit that did not come
  long long scan[kWarps + 1];
  int found_seq;
  long long found_start;
  long long lo, quota;
};

// R rows of an item: 16, 8, or 4 that take the 8 columns of a product twice.  STALL (a test): each
// warp's first unit is never asked for, and waits are short.
template <typename T, int D, int R, int SLOTS, bool STALL>
__global__ void __launch_bounds__(kThreads, R <= 8 ? 2 : 1) kv4_attn_kernel(const Kv4AttnArgs a) {
  constexpr int NT = (R + 7) / 8, WORDS = D / 32, MT = D / 16, REC = kv4_rec_bytes(D);
  constexpr bool BF = Kv4Type<T>::bf16;
  constexpr bool TWICE = R == 4;      // columns 4..7 are the second parts of rows 0..3
  constexpr bool PARTS = !BF && R > 4;  // second parts have products of their own
  using S = Smem<D, R, SLOTS>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S &sm = *reinterpret_cast<S *>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane >> 2, t = lane & 3;

  if (tid < kWarps * SLOTS) mbar_init(&sm.full[tid / SLOTS][tid % SLOTS], 1);
  fence_mbar_init();
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's part of the line
  long long total = 0, cost = 0, start = 0;  // of the thread's last sequence
  auto scan = [&](int s0) {
    const int s = s0 + tid;
    bool wrong = false;
    cost = s < a.b.n_seqs ? seq_cost(load_seq<R>(a, s, &wrong), a.c.n_kv) : 0;
    // here, where every sequence is looked at, those without work too
    if (wrong && blockIdx.x == 0) record_error(a.status, kErrInvalidArg);
    long long incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    start = total + incl - cost;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) start += sm.scan[w];
      total += sm.scan[w];
    }
  };
  for (int s0 = 0; s0 < a.b.n_seqs; s0 += kThreads) scan(s0);
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long quota = per > kMinQuota ? per : kMinQuota;
  const long long lo = min(static_cast<long long>(blockIdx.x) * quota, total);
  const int mylen = static_cast<int>(min(quota, total - lo));
  Kv4Join *desc = reinterpret_cast<Kv4Join *>(a.work);
  auto slots = [&]() { return a.work + gridDim.x * (sizeof(Kv4Join) / 4); };
  auto heads = [&]() { return slots() + 2 * gridDim.x * slot_floats(D) + static_cast<size_t>(blockIdx.x) * kWarps * R * D; };
  if (tid == 0) sm.lo = lo, sm.quota = quota;  // kept there, not in registers
  if (mylen == 0) {
    if (tid == 0) desc[blockIdx.x].last = -1;
    return;
  }
  // the sequence that holds position lo
  auto find = [&](int s0) {
    if (lo >= start && lo < start + cost) {
      sm.found_seq = s0 + tid;
      sm.found_start = start;
    }
  };
  if (a.b.n_seqs <= kThreads) {
    find(0);
  } else {
    total = 0;
    for (int s0 = 0; total <= lo; s0 += kThreads) {
      scan(s0);
      find(s0);
    }
  }
  __syncthreads();

  Walk<R> cur;
  cur.seq = sm.found_seq;
  cur.q = load_seq<R>(a, cur.seq);
  {
    const long long in = lo - sm.found_start;
    cur.item = static_cast<int>(in / cur.q.n_unit);
    cur.start = static_cast<int>(static_cast<long long>(cur.item) * cur.q.n_unit - in);
  }

  // ---- the warp's span [w0, w1) of the part, and its ring.  Lane 2 u + r has the place of record r of
  // the u-th unit of a batch of 16, and the page of the same one of the next batch.
  // Warp 0 always has one.
  const int w0 = static_cast<int>((static_cast<int64_t>(mylen) * warp + kWarps - 1) / kWarps),
            w1 = static_cast<int>((static_cast<int64_t>(mylen) * (warp + 1) + kWarps - 1) / kWarps);
  int pre_i = w0 + lane / kUnit;
  int pre_page = -1;
  int64_t pre_off = -1, place = -1;  // -1: beyond the keys, -2: the page is not usable
  const uint64_t policy = policy_evict_first();
  auto look_up = [&]() {
    pre_off = -1;
    if (pre_i < w1) {
      Walk<R> pre = cur;  // at most a batch and a ring behind
      pre.seek(a, pre_i);
      const int64_t rec = static_cast<int64_t>(pre.unit(pre_i)) * kUnit + lane % kUnit;
      if (rec * kKv4Rec < pre.q.len) {
        const int r = static_cast<int>(rec), slot = a.c.page_shift >= 0 ? r >> a.c.page_shift : r / a.c.recs_per_page;
        pre_page = __ldg(a.b.table + pre.seq * a.b.table_stride + slot);
        pre_off = (static_cast<int64_t>(pre.head(a)) * a.c.recs_per_page + (r - slot * a.c.recs_per_page)) * REC;
      }
    }
    pre_i += 32 / kUnit;
  };
  auto issue = [&](int n, int slot) {  // the span's n-th unit
    if (STALL && n == 0) return;
    const int u = n % (32 / kUnit);
    if (u == 0) {
      place = pre_off;
      if (pre_off >= 0) {
        place = pre_page >= 0 && pre_page < a.c.n_pages ? pre_page * a.c.page_stride + pre_off : -2;
        if (place < 0) record_error(a.status, kErrInvalidArg);
      }
      look_up();
    }
    const int64_t p0 = __shfl_sync(0xffffffffu, place, kUnit * u), p1 = __shfl_sync(0xffffffffu, place, kUnit * u + 1);
    if (elect_one()) {
      uint64_t *bar = &sm.full[warp][slot];
      uint8_t(*dst)[REC] = sm.ring[warp][slot];
      sm.ok[warp][slot] = (p0 >= 0 ? 1 : 0) | (p1 >= 0 ? 2 : 0);
      if (p0 >= 0 && p1 == p0 + REC) {  // neighbours in a page
        mbar_arrive_expect_tx(bar, 2 * REC);
        bulk_load(dst[0], a.c.pages + p0, 2 * REC, bar, policy);
      } else {
        const uint32_t bytes = (p0 >= 0 ? REC : 0) + (p1 >= 0 ? REC : 0);
        if (bytes)
          mbar_arrive_expect_tx(bar, bytes);
        else
          mbar_arrive(bar);
        if (p0 >= 0) bulk_load(dst[0], a.c.pages + p0, REC, bar, policy);
        if (p1 >= 0) bulk_load(dst[1], a.c.pages + p1, REC, bar, policy);
      }
    }
    __syncwarp();
  };
  look_up();
#pragma unroll 1
  for (int i = 0; i < SLOTS; ++i)
    if (w0 + i < w1) issue(i, i);

  // A wait that runs out is the whole warp's: lanes that disagreed about it would part before the
  // products.  After it the warp waits no more and asks for nothing.
  constexpr uint64_t wait_ns = STALL ? kStallWaitNs : kWaitNs;
  bool dead = false;
  int slot = 0;
  uint32_t phase = 0;
  const float sl2 = a.scale * 1.4426950408889634f;

  int parts = w0 < w1 ? 0 : 8;
#pragma unroll 1
  for (int pos = w0; pos < w1;) {
    cur.seek(a, pos);
    const int seg_end = min(cur.start + cur.q.n_unit, w1);
    const int head = cur.head(a), tile = cur.item - head * cur.q.tiles;
    const int row_first = tile * R, rows_all = cur.q.nq * a.group;

    // ---- query fragments: column n = query row, lane t holds dims [t D/4, (t+1) D/4)
    uint32_t qf[NT][WORDS][4];
    float cs[NT][2], qs[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row_first + (TWICE ? g & 3 : nt * 8 + g);
      const bool valid = r < rows_all;
      const int qi = r / a.group;
      const T *qp = static_cast<const T *>(a.q) + (cur.q.row0 + static_cast<int64_t>(qi)) * a.q_row +
                    (static_cast<int64_t>(head) * a.group + (r - qi * a.group)) * a.q_head + t * (D / 4);
      uint4 raw[WORDS];
#pragma unroll
      for (int w = 0; w < WORDS; ++w)
        raw[w] = valid ? __ldg(reinterpret_cast<const uint4 *>(qp) + w) : make_uint4(0, 0, 0, 0);
      // rows go to fp16 under a power of two that puts the row's largest value into [2^13, 2^14);
      // dims whose codes are c * 2^-20 divided by 16, so that all products have one scale: exact
      // down to 2^-24 of the largest
      float2 f[WORDS][4];
      float mx = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        const uint32_t u[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[w][i] = kv4_pair<BF>(u[i]);
          mx = fmaxf(mx, fmaxf(fabsf(f[w][i].x), fabsf(f[w][i].y)));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = max(-100, static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 13);
      const float down = pow2(-e);
#pragma unroll
      for (int w = 0; w < WORDS; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = f[w][i].x * down, y = f[w][i].y * down;
          qf[nt][w][i] = i & 1 ? pack_half2(x * 0.0625f, y * 0.0625f) : pack_half2(x, y);
          sum += x;
          sum += y;
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float up = sl2 * pow2(e);
      const float mycs = up * 16777216.f, myqs = up * sum;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int src = (2 * t + j) * 4;
        cs[nt][j] = __shfl_sync(0xffffffffu, mycs, src);
        qs[nt][j] = __shfl_sync(0xffffffffu, myqs, src);
      }
    }
    // positions of the tile's first and last row
    const int pmin = cur.q.pos0 + row_first / a.group;
    const int pmax = cur.q.pos0 + (min(row_first + R, rows_all) - 1) / a.group;
    // keys up to these lie before the window of the first and of the last row (a row at a
    // negative position sees nothing: 0 stands for it, and no difference leaves 32 bits)
    const int edge_min = max(pmin, 0) - a.window, edge_max = max(pmax, 0) - a.window;

    float o[NT][MT][4], e[NT][4], m[NT][2], l[NT][2], z[NT][2];  // e: 7 times the weights' sums, as o sums them
    float lim[NT][2];  // a sum of weights above this moves the maximum m (0 before the first key)
    float sig = pow2(100);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) e[nt][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = 0.f;
        lim[nt][j] = -1.f;
        l[nt][j] = 0.f;
        z[nt][j] = 0.f;
      }
    }

    // positions [from, to): units whose keys all rows see
    const int to = cur.start + min(max(pmin + 1, 0), cur.q.len) / kUnitKeys - cur.q.skip_by;
    const int from = a.window > 0 ? cur.start + max((max(edge_max, -1) + kUnitKeys) / kUnitKeys - cur.q.skip_by, cur.q.skip_at)
                                  : cur.start;

    // ---- the warp's units of this segment
#pragma unroll 1
    for (int i = pos; i < seg_end; ++i) {
      if (!dead && __any_sync(0xffffffffu, !mbar_wait(&sm.full[warp][slot], phase, wait_ns))) {
        dead = true;
        if (lane == 0) {
          record_error(a.status, kErrTimeout);
          sm.died[warp] = slot * 2 + phase;
        }
      }
      const int ok = dead ? 0 : sm.ok[warp][slot];
      const bool whole = i >= from && i < to && ok == 3;
      int j0 = 0;
      bool none = false;
      if (!whole) {
        j0 = cur.unit(i) * kUnitKeys;
        none = !ok || j0 > pmax || (a.window > 0 && j0 + kUnitKeys <= edge_min + 1 && j0 >= a.sinks);
      }
      if (!none) {
        // scores, less the maxima, of tokens g and g + 8 of each record for columns 2t, 2t + 1
        float s[kUnit][NT][4], vs[kUnit][2], vl[kUnit][2];
#pragma unroll
        for (int r = 0; r < kUnit; ++r) {
          const uint8_t *rec = sm.ring[warp][slot][r];
          uint32_t ka[WORDS], kb[WORDS];
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
          const uint32_t *pk = reinterpret_cast<const uint32_t *>(rec + 16 * D);
          float2 kp0 = kv4_pair<BF>(pk[g]), kp1 = kv4_pair<BF>(pk[g + 8]);
          // an infinite pair makes the score NaN, not one more hidden key at -inf
          kp0.x = fmaf(kp0.x + kp0.y, 0.f, kp0.x);
          kp1.x = fmaf(kp1.x + kp1.y, 0.f, kp1.x);
          const float2 v0 = kv4_pair<BF>(pk[16 + g]), v1 = kv4_pair<BF>(pk[24 + g]);
          vs[r][0] = v0.x, vs[r][1] = v1.x, vl[r][0] = v0.y, vl[r][1] = v1.y;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
              const uint32_t a8 = ka[w] >> 8, b8 = kb[w] >> 8;
              mma16816(x, ka[w] & 0x000f000fu, kb[w] & 0x000f000fu, a8 & 0x000f000fu,
                       b8 & 0x000f000fu, qf[nt][w][0], qf[nt][w][2]);
              mma16816(x, ka[w] & 0x00f000f0u, kb[w] & 0x00f000f0u, a8 & 0x00f000f0u,
                       b8 & 0x00f000f0u, qf[nt][w][1], qf[nt][w][3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 k = j < 2 ? kp0 : kp1;
              s[r][nt][j] = fmaf(x[j] * k.x, cs[nt][j & 1], fmaf(k.y, qs[nt][j & 1], -m[nt][j & 1]));
            }
          }
        }
        if (!whole) {
          const int last = min(pmax, cur.q.len - 1);
          // a column's row sees key j when j < vis and (j >= wlo or j < sinks); columns without a row
          // see all
          int vis[NT][2], wlo[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int rr = row_first + (TWICE ? 2 * (t & 1) : nt * 8 + 2 * t) + j, p = cur.q.pos0 + rr / a.group;
              const bool valid = rr < rows_all;
              vis[nt][j] = valid ? min(p + 1, cur.q.len) : 0x7fffffff;
              wlo[nt][j] = valid && a.window > 0 ? max(p, 0) - a.window + 1 : 0;
            }
#pragma unroll
          for (int r = 0; r < kUnit; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = j0 + r * kKv4Rec + h * 8 + g;
              const bool gone = !(ok >> r & 1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (gone || key >= vis[nt][j] || (key < wlo[nt][j] && key >= a.sinks)) s[r][nt][2 * h + j] = -INFINITY;
              // tokens that no row of the tile sees may hold anything
              if (gone || key > last || (a.window > 0 && key <= edge_min && key >= a.sinks)) vs[r][h] = 0.f, vl[r][h] = 0.f;
            }
        }

        // ---- weights.  No weight is above its column's sum, so the sums tell whether a maximum has
        // to move: when a score passes it by about 2^8.  V scales go to [2^6, 2^7) of the largest
        // seen, so weights times scale stay below 2^15 and keep fp16's 11 bits down to 2^-21 of
        // the largest.
        float p[kUnit][NT][4], sum[NT][2];
        auto weigh = [&]() -> bool {
          bool over = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int r = 0; r < kUnit; ++r) {
                p[r][nt][j] = ex2f(s[r][nt][j]);
                p[r][nt][j + 2] = ex2f(s[r][nt][j + 2]);
              }
              sum[nt][j] = (p[0][nt][j] + p[0][nt][j + 2]) + (p[1][nt][j] + p[1][nt][j + 2]);
              over |= sum[nt][j] > lim[nt][j];
            }
          return over;
        };
        const float smax = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
        const bool over = weigh();
        if (__any_sync(0xffffffffu, over || smax * sig >= 128.f)) {
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
              float n = fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]), fmaxf(s[1][nt][j], s[1][nt][j + 2]));
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
              n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16));
              const bool seen = lim[nt][j] > 0.f;
              const float d = n > (seen ? 0.f : -INFINITY) ? n : 0.f;
              al[j] = seen ? ex2f(-d) : 1.f;  // nothing to scale before the first key
              if (n > -INFINITY) lim[nt][j] = 256.f;
              m[nt][j] += d;
#pragma unroll
              for (int r = 0; r < kUnit; ++r) {
                s[r][nt][j] -= d;
                s[r][nt][j + 2] -= d;
              }
              l[nt][j] *= al[j];
              z[nt][j] *= al[j];
              al[j] *= f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) e[nt][j] *= al[j & 1];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][0] *= al[0];
              o[nt][i][1] *= al[1];
              o[nt][i][2] *= al[0];
              o[nt][i][3] *= al[1];
            }
          }
          weigh();
        }

        // ---- their sums, and the products with V
        // a key hidden from this row must not reach it through 0 * NaN
        auto products = [&](auto hides) {
#pragma unroll
          for (int r = 0; r < kUnit; ++r) {
            const float s0 = vs[r][0] * sig, s1 = vs[r][1] * sig;
            if (!BF) {
              vl[r][0] = fmaf(7.f, vs[r][0], vl[r][0]);
              vl[r][1] = fmaf(7.f, vs[r][1], vl[r][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool hid = hides.value && s[r][nt][j] == -INFINITY;
                z[nt][j & 1] = hid ? z[nt][j & 1] : fmaf(p[r][nt][j], vl[r][j / 2], z[nt][j & 1]);
                p[r][nt][j] = hid ? 0.f : p[r][nt][j] * (j < 2 ? s0 : s1);
              }
          }
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] += sum[nt][0];
          l[nt][1] += sum[nt][1];
        }
        if (whole)
          products(std::false_type{});
        else
          products(std::true_type{});
        // Codes are all positive, so what the products lose does not cancel against lo's part of the
        // row, and the mean over a long context is small beside both.  A bf16 result is rounded far
        // enough to hide that (16384 tokens: 1.01 to 1.08 of the rounding's own error; 131071: 1.09).
        // For fp16 caches
        //   weights go in as two fp16 parts (22 bits); with four rows the columns 4..7 hold the second
        //   parts, else they are a product of their own (8 % of the kernel);
        //   a row of sevens among the codes sums what the same instructions make of the weights, which
        //   takes out, with 7 s beside lo, what their sums lose by being cut off (131072 tokens: 8e-4
        //   of the result otherwise).
#pragma unroll
        for (int r = 0; r < kUnit; ++r) {
          uint32_t p0[NT], p1[NT], q0[NT], q1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t h0 = pack_half2(p[r][nt][0], p[r][nt][1]), h1 = pack_half2(p[r][nt][2], p[r][nt][3]);
            const float2 f0 = __half22float2(kv4_bits<__half2>(h0)), f1 = __half22float2(kv4_bits<__half2>(h1));
            uint32_t d0 = 0, d1 = 0;
            if (TWICE || PARTS) {
              d0 = pack_half2(p[r][nt][0] - f0.x, p[r][nt][1] - f0.y);
              d1 = pack_half2(p[r][nt][2] - f1.x, p[r][nt][3] - f1.y);
            }
            p0[nt] = transpose8x8(TWICE && t >= 2 ? d0 : h0);
            p1[nt] = transpose8x8(TWICE && t >= 2 ? d1 : h1);
            if (PARTS) {
              q0[nt] = transpose8x8(d0);
              q1[nt] = transpose8x8(d1);
            }
          }
          if (!BF) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(e[nt], 0x00070007u, 0x00700070u, 0x00070007u, 0x00700070u, p0[nt], p1[nt]);
              if (PARTS) mma16816(e[nt], 0x00070007u, 0x00700070u, 0x00070007u, 0x00700070u, q0[nt], q1[nt]);
            }
          }
          const uint8_t *rec = sm.ring[warp][slot][r];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(rec + 8 * D + c * 512 + lane * 16);
            const uint32_t vw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v8 = vw[i] >> 8, a0 = vw[i] & 0x000f000fu, a1 = vw[i] & 0x00f000f0u, a2 = v8 & 0x000f000fu,
                             a3 = v8 & 0x00f000f0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[nt][4 * c + i], a0, a1, a2, a3, p0[nt], p1[nt]);
                if (PARTS) mma16816(o[nt][4 * c + i], a0, a1, a2, a3, q0[nt], q1[nt]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (!dead && i + SLOTS < w1) issue(i + SLOTS - w0, slot);
      if (++slot == SLOTS) slot = 0, phase ^= 1;
    }

    // ---- the segment's result.  Rows 8 i + g of the products are dims 2 (8 i + g) (x 2^-24) and
    // 2 (8 i + g) + 1 (x 2^-20).
    const float un = 1.f / sig;
    if (TWICE) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[0][i][j] += __shfl_xor_sync(0xffffffffu, o[0][i][j], 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[0][j] += __shfl_xor_sync(0xffffffffu, e[0][j], 2);
    }
    if (!BF) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] -= e[nt][j];
    }
    const bool begins = cur.start >= w0, ends = cur.start + cur.q.n_unit <= w1;
    // a part that ends the span waits in the ring, which is empty by then
    const int which = begins ? 1 : 0;
    const bool at_end = seg_end == w1;
    float *part = at_end ? reinterpret_cast<float *>(sm.ring[warp]) : heads() + warp * (R * D);
    const int pitch = at_end ? S::OROW : D;
    if (!begins) parts |= (ends ? 3 : 1) | (at_end ? 16 : 0);
    if (begins && !ends) parts |= 4;
    if (lane == 0 && !(begins && ends))
      sm.place[which][warp] = Place{cur.start + cur.q.n_unit, head, cur.q.row0, row_first,
                                    min(R, rows_all - row_first)};
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
        const int col = nt * 8 + 2 * t + j, rr = row_first + col;
        if (rr >= rows_all || (TWICE && t >= 2)) continue;
        if (begins && ends) {
          const float inv = lj == 0.f ? 0.f : 1.f / lj;
          const int qi = rr / a.group;
          T *op = static_cast<T *>(a.out) + (cur.q.row0 + static_cast<int64_t>(qi)) * a.o_row +
                  (static_cast<int64_t>(head) * a.group + (rr - qi * a.group)) * a.o_head + 2 * g;
#pragma unroll
          for (int i = 0; i < MT; ++i)
            *reinterpret_cast<uint32_t *>(op + 16 * i) =
                Kv4Type<T>::held2(fmaf(o[nt][i][j] * 16777216.f, un, zj) * inv, fmaf(o[nt][i][j + 2] * 1048576.f, un, zj) * inv);
        } else {
#pragma unroll
          for (int i = 0; i < MT; ++i)
            *reinterpret_cast<float2 *>(part + col * pitch + 2 * (8 * i + g)) =
                make_float2(fmaf(o[nt][i][j] * 16777216.f, un, zj), fmaf(o[nt][i][j + 2] * 1048576.f, un, zj));
          if (g == 0) {
            sm.m[which][warp][col] = lim[nt][j] > 0.f ? m[nt][j] : kNegBig;
            sm.l[which][warp][col] = lj;
          }
        }
      }
    pos = seg_end;
  }
  if (lane == 0) sm.part[warp] = parts;

  // ---- join the warps, a warp an item: those that begin in warp b's span, or in the CTA before
  // (b == -1), and go on
  if (tid == 0) desc[blockIdx.x].last = -1;
  __syncthreads();
#pragma unroll 1
  for (int b = warp - 1; b < kWarps; b += kWarps) {
    if (!(b < 0 ? sm.part[0] & 1 : sm.part[b] & 4)) continue;
    int last = b;  // last warp with a part
    bool ends = false;
    for (int w = b + 1; w < kWarps && !ends; ++w)
      if (sm.part[w] & 1) {
        last = w;
        ends = sm.part[w] & 2;
      } else if (!(sm.part[w] & 8)) {
        break;
      }
    const Place x = b < 0 ? sm.place[0][0] : sm.place[1][b];
    const bool full = b >= 0 && ends;
    if (b >= 0 && !ends && lane == 0)
      desc[blockIdx.x] = Kv4Join{static_cast<int>((sm.lo + x.end - 1) / sm.quota), x.row0, x.row_first, x.rows, x.head, {}};
    float *part = slots() + (2 * static_cast<size_t>(blockIdx.x) + (b < 0 ? 0 : 1)) * slot_floats(D);
#pragma unroll 1
    for (int e = lane; e < x.rows * (D / 4); e += 32) {
      const int r = e / (D / 4), d = (e % (D / 4)) * 4;
      float mx = b < 0 ? kNegBig : sm.m[1][b][r];
      for (int w = b + 1; w <= last; ++w)
        if (sm.part[w] & 1) mx = fmaxf(mx, sm.m[0][w][r]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int w = max(b, 0); w <= last; ++w) {
        const bool second = w == b;
        if (!second && !(sm.part[w] & 1)) continue;
        const float *p = second || sm.part[w] & 16 ? reinterpret_cast<const float *>(sm.ring[w]) + r * S::OROW
                                                   : heads() + w * (R * D) + r * D;
        const float4 o = *reinterpret_cast<const float4 *>(p + d);
        const float f = ex2f(sm.m[second][w][r] - mx);
        sum = fmaf(f, sm.l[second][w][r], sum);
        acc.x = fmaf(f, o.x, acc.x);
        acc.y = fmaf(f, o.y, acc.y);
        acc.z = fmaf(f, o.z, acc.z);
        acc.w = fmaf(f, o.w, acc.w);
      }
      if (full) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int rr = x.row_first + r, qi = rr / a.group;
        T *op = static_cast<T *>(a.out) + (x.row0 + static_cast<int64_t>(qi)) * a.o_row +
                (static_cast<int64_t>(x.head) * a.group + (rr - qi * a.group)) * a.o_head + d;
        using X = Kv4Type<T>;
        uint2 v;
        v.x = X::held2(acc.x * inv, acc.y * inv);
        v.y = X::held2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(op) = v;
      } else {
        *reinterpret_cast<float4 *>(part + r * D + d) = acc;
        if (d == 0) {
          part[kMaxRows * D + r] = mx;
          part[kMaxRows * D + kMaxRows + r] = sum;
        }
      }
    }
  }
  // after a wait that ran out, do not leave while copies may still land here: the ring's, from the
  // slot that did not come on (one that was never asked for costs its limit)
  if (dead) {
    slot = sm.died[warp] / 2, phase = sm.died[warp] & 1;
    for (int n = 0; n < SLOTS; ++n) {
      mbar_wait(&sm.full[warp][slot], phase, wait_ns / 16);
      if (++slot == SLOTS) slot = 0, phase ^= 1;
    }
  }
}

// Joins what both kernels cut: first the tile kernel's items (tile_ctas 0: none), then those here.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) kv4_join_kernel(const Kv4AttnArgs a, int tile_ctas, int ctas) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x * kWarps + threadIdx.x / 32, tiles = tile_ctas * (kKv4TileRows / 4);
  if (i < tiles)
    kv4_join<D, kKv4TileRows, 4, T>(a, a.work_tile, tile_ctas, i, kKv4TileRows / 4);
  else if (i - tiles < ctas * R)
    kv4_join<D, kMaxRows, 1, T>(a, a.work, ctas, i - tiles, R);
}

template <typename T, int D, int R, bool STALL = false>
cudaError_t launch(const Kv4AttnArgs &a, cudaStream_t stream) {
  constexpr int SLOTS = D == 64 ? 5 : R <= 8 ? 3 : 5;  // units in flight: two CTAs fit an SM, or one with 16 rows
  auto kernel = kv4_attn_kernel<T, D, R, SLOTS, STALL>;
  const int smem = static_cast<int>(sizeof(Smem<D, R, SLOTS>));
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.num_sms * (R <= 8 ? 2 : 1), 1, 1);
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
  const int ctas = cfg.gridDim.x, tile_ctas = a.tile_above < INT64_MAX ? a.num_sms : 0;
  cfg.gridDim = dim3((tile_ctas * (kKv4TileRows / 4) + ctas * R + kWarps - 1) / kWarps, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, D, R>, a, tile_ctas, ctas);
}

template <typename T, int D>
cudaError_t pick(const Kv4AttnArgs &a, cudaStream_t stream) {
  if constexpr (!Kv4Type<T>::bf16 && D == 64)
    if (a.stall) return launch<T, D, 8, true>(a, stream);
  // the fewest rows per item that take a sequence's rows of a kv head at once; four only where
  // weights have second parts (16 sequences of up to 4096, 32 / 32 heads of 128, one row each, by items
  // of 4 / 8 / 16 rows: fp16 50 / 54 / 80 us, bf16 - / 49 / 70)
  if constexpr (!Kv4Type<T>::bf16)
    if (a.max_rows <= 4) return launch<T, D, 4>(a, stream);
  return a.max_rows <= 8 ? launch<T, D, 8>(a, stream) : launch<T, D, 16>(a, stream);
}

}  // namespace

size_t kv4_step_workspace(int d, int num_sms) {
  const size_t ctas = 2 * static_cast<size_t>(num_sms);
  // an item's first and last part of each CTA, and 8 rows that each warp leaves for its CTA (or half
  // the CTAs with 16)
  return ctas * sizeof(Kv4Join) + ctas * 2 * slot_floats(d) * sizeof(float) + ctas * kWarps * 8 * d * sizeof(float);
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
