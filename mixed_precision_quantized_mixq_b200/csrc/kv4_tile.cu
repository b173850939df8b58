// Attention over the 4-bit KV cache for many query rows (prompts and chunks of
// prompts), on the 5th-generation tensor cores.
//
// Work is up to 256 query rows of one (sequence, kv head) against its visible
// keys, 128 at a time; rows are (new token, head of the group) pairs, so grouped
// heads fill the tiles.  The rows are two 128-row MMA tiles that take turns: while
// the softmax of one runs, the tensor core works for the other.  Per key tile
//   S = Q C^T   (C: K's codes, exact in the 16-bit type), 128 x 128 x D, in TMEM
//   t = scale log2(e) (s_k S + lo_k sum(q)),  P = 2^(t - m)
//   O += P V^   (V^: V's rows as they read back, rounded once to fp16, or to bf16 where a
//                bf16 cache's values do not fit fp16)
// with P written over S in TMEM as the second product's A operand.
//
// Roles: warps 0-7 softmax (thread = query row = TMEM lane; no reduction crosses
// lanes); warps 8-15 unpack K's codes and warps 16-23 V's rows straight from global
// memory into the swizzled operand tiles, one 16-token record a warp and tile, the
// next tile's bytes already in registers; warp 24 issues the MMAs; warp 25 walks the
// work ahead of them and hands out items and the places of records.  K stays in codes
// because a rounded K would move every score; the pairs act on S instead.  V is
// rounded like any 16-bit V, which leaves the softmax no work per V row.
//
// The key tiles of all (sequence, 256 rows, head) items, and places for the turn to
// each, are one line, cut into equal parts over a persistent grid of one CTA per SM:
// the load is even whatever the lengths and however few items there are.  The roles
// run on from item to item: the next item's query rows are fetched during the last
// tile of this one, and its first scores are computed beside this one's last product.
// An item cut by a boundary leaves fp32 partial results, which the call's last launch
// joins in their order.
//
// The running maximum moves only when a score passes it by 2^8, so O (in TMEM) is
// rarely rescaled, and by whole powers of two, which is exact; P carries 2^6 more so
// that fp16 keeps 11 bits down to 2^-20 of the row's largest weight.  Weights and V are rounded to 11
// bits each: an error of 3.5e-4 of the result for fp16, where rounding the result alone gives 2.1e-4.
// Weights as two fp16 parts, the second in the TMEM columns that their scores leave, brought 2.9e-4
// and cost a fifth (four prompts 187 -> 226 us, windowed chunks 99 -> 113): left out.
//
// What bounds it (B200, 1024 tokens over 15360, 64 / 8 heads of 128, bf16: 772 us, 690
// TFLOP/s, 42 % of the measured matrix peak; four ragged prompts of up to 2048 tokens,
// 32 heads: 188 us, 356 TFLOP/s): no unit alone.  A pair of row tiles takes about 6100
// cycles a key tile; the matrix products and the exponentials need 2048 each, the
// issue slots 2600 (a third of them the unpacking), and shared memory 3700: the
// operands of the products 1560, (s, lo) of the keys for eight warps 1280, the
// unpacked tiles 550.  Prompts lose the rest to tiles on the diagonal and to items of
// few tiles.  Measured and left out: two threads a row on 16 softmax warps (776 us
// against 742), 16 x 256-bit TMEM fragments that read (s, lo) a quarter as often (757
// to 837), the first half of P handed over early (741), maxima from the weights' sums
// (742), unrolled further (794: the roles share the instruction cache), the next chunk's
// scores computed beside this one's exponentials (783 against 773).
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "kv4.h"
#include "kv4_join.cuh"
#include "kv4_ptx.cuh"
#include "tma_host.h"

namespace mixq {
namespace {

constexpr int kThreads = 896;  // softmax 0-7, K 8-15, V 16-23, MMA 24, walk 25 (26, 27 complete its group)
constexpr int kRows = kKv4TileRows;  // query rows per CTA
constexpr int kKeys = 128;     // keys per tile
constexpr int kSeqChunk = 64;  // sequences the search for a CTA's part looks at together
// What the turn to an item costs, in key tiles.  With 1 / 2 / 3, us: four prompts of 32 heads, D 128
// 193 / 187 / 194 in fp16 and 206 / 200 / 207 in bf16, D 64 155 / 159 / 164 and 165 / 169 / 174; 70B
// chunk 775 / 771 / 774; windowed chunks, D 64 99 / 99 / 101, D 128 117 / 115 / 117.
constexpr int kTurn = 2;
constexpr int kMinTiles = 4;   // key tiles per part: below, joining costs more than the cut spreads
constexpr float kNegBig = -1e30f;
constexpr uint64_t kWaitNs = 2000000000ull, kStallWaitNs = 20000000ull;

constexpr int kItems = 8;      // items the walk may be ahead

// registers per thread after the split; 256*144 + 512*40 + 128*56 = 64512, the 896 * 72 the CTA
// starts with
constexpr int kRegsSoftmax = 144, kRegsUnpack = 40, kRegsMma = 56;

// A part of an item: key tiles [t0, t0 + n) of a block of rows.  n == 0: no more.
struct Item {
  int n, t0, tiles, sinks, skip;  // tiles of the whole item; tile i is key tile i, from sinks on i + skip
  int row0, rows, len, pos0;      // rows: of this block
  int first, head;                // first row of the block within the sequence's rows
  int n0;                         // tiles [t0, t0 + n0) concern the first row tile: n, or n - 1 where it sees no key of the last
};

template <int D>
struct TileSmem {
  alignas(1024) uint8_t q[2][128 * D * 2];
  alignas(1024) uint8_t k[2][kKeys * D * 2];
  alignas(1024) uint8_t v[2][kKeys * D * 2];
  alignas(16) float4 kp[4][kKeys / 2];  // per pair of keys: s0 s1 lo0 lo1, times scale log2(e)
  alignas(8) uint8_t hidden[4][8];  // of the tile's records: bit 0: the page is not usable, bit 1: bf16 products with V
  alignas(16) int4 sight[kRows];  // of a row: key j is seen when j < x and (j >= y or j < sinks); z, w: of its row tile
  Item item[kItems];
  int64_t src[2][32];  // records of four tiles: offset in the pages, -1 beyond the keys, -2 page not usable, -3 no more tiles
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], par_full[4], s_full[2], p_full[2], o_full[2];
  uint64_t item_full[kItems], item_empty[kItems], src_full[2], src_empty[2], done;
  long long cost[kSeqChunk];
  int found;
  long long found_start;
  uint32_t tmem;
  int dead;
};

// Bounded wait; once one has run out, none waits any more and the CTA winds up.
template <bool STALL>
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, volatile int *dead, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!*dead) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return;
    if (globaltimer_ns() - t0 > (STALL ? kStallWaitNs : kWaitNs)) {
      *dead = 1;
      record_error(status, kErrTimeout);
    }
  }
}

// The n lowest bits, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n) {
  n = min(max(n, 0), 32);
  return static_cast<uint32_t>((1ull << n) - 1);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Whether fp16 would hold a row of V with this bf16 pair worse than bf16: it reaches 2^15, or s or
// lo is not exact in fp16, or s is so small that fp16's smallest step (2^-24) shows beside it.
__device__ __forceinline__ bool past_half(float2 v) {
  const float s = fabsf(v.x), lo = fabsf(v.y), top = fmaxf(lo, fabsf(fmaf(15.f, v.x, v.y)));
  return !(top < 32768.f) || (s < 1.220703125e-4f && s > 0.f) || (lo < 7.62939453125e-6f && lo > 0.f);
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

// A sequence as the walk sees it.
struct Rows {
  int row0, len, pos0;  // first q row, keys that exist, position of the first new token
  int rows;             // query rows of a kv head
  int blocks;           // of 256 rows; 0: the sequence is not this kernel's
};

__device__ __forceinline__ Rows load_rows(const Kv4AttnArgs &a, int s) {
  Rows q{};
  bool bad = false;
  const int2 r = kv4_row_range(a.b, s, &bad);
  const int full = __ldg(a.b.lens + s);
  if ((threadIdx.x & 31) == 0 && (bad || full < 0 || full > a.room)) record_error(a.status, kErrInvalidArg);
  q.row0 = r.x;
  q.len = min(max(full, 0), a.room);
  q.pos0 = full - (r.y - r.x);
  q.rows = (r.y - r.x) * a.group;
  q.blocks = q.rows > a.tile_above ? (q.rows + kRows - 1) / kRows : 0;
  return q;
}

// The key tiles that a block of rows visits: tile i is key tile i, from `sinks` on i + skip.
struct Keys {
  int tiles, sinks, skip;
  __device__ __forceinline__ int key0(int i) const { return (i + (i >= sinks ? skip : 0)) * kKeys; }
};

__device__ __forceinline__ Keys keys_of(const Kv4AttnArgs &a, const Rows &q, int block) {
  const int first = block * kRows, last = min(first + kRows, q.rows) - 1;
  const int total = (max(0, min(q.len, q.pos0 + last / a.group + 1)) + kKeys - 1) / kKeys;
  Keys k{total, total, 0};
  if (a.window > 0) {
    const int w0 = min(max(0, max(q.pos0 + first / a.group, 0) - a.window + 1) / kKeys, total);
    k.sinks = min((min(a.sinks, q.len) + kKeys - 1) / kKeys, w0);
    k.skip = w0 - k.sinks;
    k.tiles = total - k.skip;
  }
  k.tiles = max(k.tiles, 1);  // rows that see nothing still get their zeros, from a tile without keys
  return k;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Length on the line of sequence s over all its blocks and heads (whole warp): an item is kTurn
// places for the turn to it and a place for each key tile.
__device__ __forceinline__ long long seq_length(const Kv4AttnArgs &a, int s, int lane) {
  const Rows q = load_rows(a, s);
  long long n = 0;
  for (int b = lane; b < q.blocks; b += 32) n += keys_of(a, q, b).tiles + kTurn;
  return warp_sum(n) * a.c.n_kv;
}

// A CTA's part of the line, one item after another.
struct Walk {
  Rows q;
  Keys k;
  int seq, block, head;
  int t0, t1;       // tiles of the item that belong to the part
  int left;         // places of the part from `from` on
  int from;         // place in the item that the part begins at
  long long start;  // of the item on the line

  __device__ __forceinline__ void set() {
    t0 = max(from - kTurn, 0);
    t1 = min(k.tiles, max(from + left - kTurn, 0));
  }
  __device__ __forceinline__ int length() const { return k.tiles + kTurn; }
  __device__ __forceinline__ bool more() const { return left - (length() - from) > kTurn; }  // with a tile of it
  __device__ __forceinline__ void next(const Kv4AttnArgs &a) {
    left -= length() - from;
    start += length();
    from = 0;
    if (++head == a.c.n_kv) {
      head = 0;
      if (++block >= q.blocks) {
        block = 0;
        do {
          q = load_rows(a, ++seq);
        } while (q.blocks == 0);
      }
      k = keys_of(a, q, block);
    }
    set();
  }
  __device__ __forceinline__ int rows() const { return min(kRows, q.rows - block * kRows); }
};

using Desc = Kv4Join;

__host__ __device__ constexpr size_t slot_floats(int d) { return kv4_slot_floats(kRows, d); }

// STALL (a test): the CTA's second tile of V never arrives, and waits are short.
template <typename T, int D, bool STALL>
__global__ void __launch_bounds__(kThreads, 1) kv4_tile_kernel(const Kv4AttnArgs a) {
  using S = TileSmem<D>;
  using X = Kv4Type<T>;
  using T2 = typename X::T2;
  constexpr bool BF = X::bf16;
  constexpr int REC = kv4_rec_bytes(D), WORDS = D / 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S &sm = *reinterpret_cast<S *>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;

  if (tid == 0) {
    sm.dead = 0;
    mbar_init(&sm.done, 1);
    for (int i = 0; i < kItems; ++i) {
      sm.item[i].n = 0;
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 9);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.src_full[i], 1);
      mbar_init(&sm.src_empty[i], 16);
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.k_full[i], 8);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 8);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.par_full[i], 8);
    fence_mbar_init();
  }
  if (tid < 64) sm.src[tid / 32][tid % 32] = -1;
  if (warp == 24) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's part [lo, lo + span) of the line
  long long total = 0;
  for (int s0 = 0; s0 < a.b.n_seqs; s0 += kSeqChunk) {
    __syncthreads();
    for (int s = warp; s < kSeqChunk; s += kThreads / 32) {
      const long long c = s0 + s < a.b.n_seqs ? seq_length(a, s0 + s, lane) : 0;
      if (lane == 0) sm.cost[s] = c;
    }
    __syncthreads();
    total += warp_sum(sm.cost[lane] + sm.cost[lane + 32]);
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long quota = max(per, static_cast<long long>(kMinTiles));
  const long long lo = min(static_cast<long long>(blockIdx.x) * quota, total);
  const int span = static_cast<int>(min(quota, total - lo));
  Desc *desc = reinterpret_cast<Desc *>(a.work_tile);
  float *slots = a.work_tile + gridDim.x * (sizeof(Desc) / 4);
  Walk w{};
  if (span > 0) {
    long long base = 0;
    for (int s0 = 0; s0 < a.b.n_seqs; s0 += kSeqChunk) {
      if (a.b.n_seqs > kSeqChunk) {  // else the costs are there
        __syncthreads();
        for (int s = warp; s < kSeqChunk; s += kThreads / 32) {
          const long long c = s0 + s < a.b.n_seqs ? seq_length(a, s0 + s, lane) : 0;
          if (lane == 0) sm.cost[s] = c;
        }
        __syncthreads();
      }
      if (tid == 0) {
        sm.found = -1;
        long long at = base;
        for (int s = 0; s < kSeqChunk; ++s) {
          if (lo >= at && lo < at + sm.cost[s]) {
            sm.found = s0 + s;
            sm.found_start = at;
          }
          at += sm.cost[s];
        }
      }
      base += warp_sum(sm.cost[lane] + sm.cost[lane + 32]);
      __syncthreads();
      if (sm.found >= 0) break;
    }
    w.seq = sm.found;
    w.q = load_rows(a, w.seq);
    // the block: its heads' places begin at or before lo and end after it
    long long in = lo - sm.found_start, at = 0;
    for (int b0 = 0; b0 < w.q.blocks; b0 += 32) {
      const long long c = b0 + lane < w.q.blocks ? static_cast<long long>(keys_of(a, w.q, b0 + lane).tiles + kTurn) * a.c.n_kv : 0;
      long long incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, in < at + incl);
      if (hit) {
        const int f = __ffs(hit) - 1;
        w.block = b0 + f;
        in -= at + __shfl_sync(0xffffffffu, incl - c, f);
        break;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.k = keys_of(a, w.q, w.block);
    w.head = static_cast<int>(in / w.length());
    w.from = static_cast<int>(in - static_cast<long long>(w.head) * w.length());
    w.start = lo - w.from;
    w.left = span;
    w.set();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);  // the same in every lane
  auto tm_s = [tmem](int i) { return tmem + i * 128; };
  auto tm_o = [tmem](int i) { return tmem + 256 + i * D; };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    reg_inc<kRegsSoftmax>();
    const int i = warp / 4, row = tid & 127, r = i * 128 + row;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 TMEM lanes per warp
    int jt = 0;  // key tiles of the CTA so far
    int jn = 0;  // those of this row tile (its barriers' phases)
    // After items that had nothing for this row tile it is ahead of the keys, and the phase of their
    // barrier then says nothing (two phases back looks like done).
    bool ahead = false;
    float qsum = 0.f;
    // The warp's 32 query rows of an item into the operand tile, D/8 lanes a row; then, once they
    // are there, each lane's sum over its own row.
    auto fetch_q = [&](const Item &x) {
      if (i * 128 >= x.rows) return;
      const int rr = x.first + r, qi = rr / a.group;
      const int64_t at = (x.row0 + static_cast<int64_t>(qi)) * a.q_row +
                         (static_cast<int64_t>(x.head) * a.group + (rr - qi * a.group)) * a.q_head;
      constexpr int LANES = D / 8, RPW = 32 / LANES;
      const int l = lane % LANES;
#pragma unroll 4
      for (int y = 0; y < 32; y += RPW) {
        const int z = y + lane / LANES, tr = (warp & 3) * 32 + z;
        const int64_t from = __shfl_sync(0xffffffffu, at, z);
        const bool valid = i * 128 + tr < x.rows;
        cp_async16(smem_u32(sm.q[i]) + (l / 8) * 16384 + tr * 128 + (((l & 7) ^ (tr & 7)) << 4),
                   static_cast<const T *>(a.q) + (valid ? from : 0) + l * 8, valid ? 16 : 0);
      }
    };
    auto have_q = [&](const Item &x) {
      if (i * 128 >= x.rows) return;
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[i]);
      uint64_t sum = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x4 = *reinterpret_cast<const uint4 *>(sm.q[i] + (c / 8) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        const uint32_t u[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = X::f2(kv4_bits<T2>(u[e]));
          sum = add_f32x2(sum, f32x2(f.x, f.y));
        }
      }
      const float2 f = from_f32x2(sum);
      qsum = f.x + f.y;
    };
    wait<STALL>(&sm.item_full[0], 0, &sm.dead, a.status);
    // an item after a wait that ran out may be half written, and its rows lie anywhere
    auto there = [&](const Item &x) { return !__any_sync(0xffffffffu, x.n == 0 || sm.dead); };
    if (there(sm.item[0])) {
      fetch_q(sm.item[0]);
      have_q(sm.item[0]);
    }
#pragma unroll 1
    for (int it = 0;; ++it) {
      const Item &x = sm.item[it % kItems], &nx = sm.item[(it + 1) % kItems];  // x has arrived already
      if (!there(x)) break;  // the lanes leave together
      const int n = i ? x.n : x.n0;  // of this row tile
      const bool active = i * 128 < x.rows;
      uint64_t la = f32x2(0.f, 0.f), lb = la;
      float base = 0.f;         // what is added to t: 6 - m, m a whole number, once a key was seen
      float limit = -INFINITY;  // t + base above this moves the maximum
      if (active) {
        {
          // z: keys that all rows of the tile may see, w: the last row's position; in shared memory, as
          // the registers are the scores'
          const bool valid = r < x.rows;
          const int p = x.pos0 + (x.first + r) / a.group;
          sm.sight[r] = make_int4(valid ? min(p + 1, x.len) : x.len, valid && a.window > 0 ? max(max(p, 0) - a.window + 1, 0) : 0,
                                  min(x.pos0 + (x.first + i * 128) / a.group + 1, x.len),
                                  max(x.pos0 + (x.first + min(i * 128 + 128, x.rows) - 1) / a.group, 0));
        }
        const uint64_t qs2 = f32x2(qsum, qsum);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int st = (jt + j) & 3;
          if (ahead) {  // the keys are there when the scores are
            wait<STALL>(&sm.s_full[i], jn & 1, &sm.dead, a.status);
            ahead = false;
          }
          wait<STALL>(&sm.par_full[st], ((jt + j) >> 2) & 1, &sm.dead, a.status);
          const float4 *kp = sm.kp[st];
          const uint2 hid = *reinterpret_cast<const uint2 *>(sm.hidden[st]);
          const int k0 = (x.t0 + j + (x.t0 + j >= x.sinks ? x.skip : 0)) * kKeys;
          const bool whole = ((hid.x | hid.y) & 0x01010101u) == 0 && k0 + kKeys <= sm.sight[r].z &&
                             (a.window <= 0 || k0 > sm.sight[r].w - a.window || k0 + kKeys <= a.sinks);
          wait<STALL>(&sm.s_full[i], (jn + j) & 1, &sm.dead, a.status);
          tc_fence_after();
          if (j + 1 == n) {  // the last scores are there, so the operand tile is free for the next rows
            wait<STALL>(&sm.item_full[(it + 1) % kItems], (it + 1) / kItems & 1, &sm.dead, a.status);
            if (there(nx)) fetch_q(nx);
          }
          union Chunk {
            uint32_t u[32];
            float f[32];
            uint64_t d[16];
          };
          // t + base of 32 keys in place of their scores, and the largest
          auto scores = [&](Chunk &t, int c) -> float {
            const uint64_t b2 = f32x2(base, base);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 x = kp[c * 16 + e];
              t.d[e] = fma_f32x2(t.d[e], f32x2(x.x, x.y), fma_f32x2(f32x2(x.z, x.w), qs2, b2));
            }
            if (__builtin_expect(!whole, 0)) {
              // one bit per key, so that no lane branches
              const int kc = k0 + c * 32;
              const uint32_t off = (c < 2 ? hid.x : hid.y) >> ((c & 1) * 16);
              const uint32_t seen = low_bits(sm.sight[r].x - kc) & (~low_bits(sm.sight[r].y - kc) | low_bits(a.sinks - kc)) &
                                    ~((off & 1u) * 0xffffu | (off >> 8 & 1u) * 0xffff0000u);
#pragma unroll
              for (int e = 0; e < 32; ++e) t.f[e] = seen & (1u << e) ? t.f[e] : -INFINITY;
            }
            float m0 = max3(t.f[0], t.f[1], t.f[2]), m1 = max3(t.f[3], t.f[4], t.f[5]);
#pragma unroll
            for (int e = 6; e < 30; e += 4) {
              m0 = max3(m0, t.f[e], t.f[e + 1]);
              m1 = max3(m1, t.f[e + 2], t.f[e + 3]);
            }
            return max3(m0, m1, fmaxf(t.f[30], t.f[31]));
          };
          // moves the maximum: the chunk, and what the row has in O, the sums and this tile's
          // first c chunks of weights
          auto grow = [&](Chunk &t, int c, float mx) {
            const bool need = mx > limit;
            const float d = need ? 6.f - ceilf(mx) : 0.f;
            const float al = limit > -INFINITY ? ex2f(d) : 1.f;  // a power of two; nothing to scale before the first key
            if (need) limit = 14.f;
            base += d;
            const uint64_t d2 = f32x2(d, d), al2 = f32x2(al, al);
#pragma unroll
            for (int e = 0; e < 16; ++e) t.d[e] = add_f32x2(t.d[e], d2);
            la = mul_f32x2(la, al2);
            lb = mul_f32x2(lb, al2);
            if (j > 0) {
              wait<STALL>(&sm.o_full[i], (jn + j - 1) & 1, &sm.dead, a.status);
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < D / 16; ++x) {
                uint32_t o[16];
                tmem_ld16(tm_o(i) + lanes + x * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st16(tm_o(i) + lanes + x * 16, o);
              }
            }
            if (c > 0) {
              tmem_st_wait();
#pragma unroll 1
              for (int x = 0; x < c; ++x) {
                uint32_t o[16];
                tmem_ld16(tm_s(i) + lanes + x * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 f = __half22float2(kv4_bits<__half2>(o[e]));
                  o[e] = kv4_bits<uint32_t>(__floats2half2_rn(f.x * al, f.y * al));
                }
                tmem_st16(tm_s(i) + lanes + x * 16, o);
              }
            }
            tmem_st_wait();
          };
          // 32 keys at a time.  P of keys [32c, 32c + 32) takes TMEM columns [16c, 16c + 16), whose
          // scores have been read.  Not unrolled further: the roles share the instruction cache.
#pragma unroll 2
          for (int c = 0; c < 4; ++c) {
            Chunk t;
            tmem_ld32(tm_s(i) + lanes + c * 32, t.u);
            tmem_ld_wait();
            const float mx = scores(t, c);
            if (__builtin_expect(__any_sync(0xffffffffu, mx > limit), 0)) grow(t, c, mx);
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = from_f32x2(t.d[e]);
              const float p0 = ex2f(y.x), p1 = ex2f(y.y);
              if (e & 1) lb = add_f32x2(lb, f32x2(p0, p1));
              else la = add_f32x2(la, f32x2(p0, p1));
              p[e] = kv4_bits<uint32_t>(__floats2half2_rn(p0, p1));
            }
            tmem_st16(tm_s(i) + lanes + c * 16, p);
          }
          tmem_st_wait();
          // Weights of bf16 products.  Which records those are shows only here: the conversion beside the
          // exponentials would be in every tile's code.  Rounded from fp16 they are off by 2^-12 more beside
          // bf16's own 2^-9.
          if (BF && __builtin_expect((hid.x | hid.y) & 0x02020202u, 0)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = (c < 2 ? hid.x : hid.y) >> ((c & 1) * 16);
              uint32_t o[16];
              tmem_ld16(tm_s(i) + lanes + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (w >> (e / 8 * 8 + 1) & 1)
                  o[e] = kv4_bits<uint32_t>(__float22bfloat162_rn(__half22float2(kv4_bits<__half2>(o[e]))));
              tmem_st16(tm_s(i) + lanes + c * 16, o);
            }
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[i]);
        }
        jn += n;
      } else {
        ahead = true;
        wait<STALL>(&sm.item_full[(it + 1) % kItems], (it + 1) / kItems & 1, &sm.dead, a.status);
        if (there(nx)) fetch_q(nx);
      }
      jt += x.n;
      if (there(nx)) have_q(nx);
      // ---- the result.  Column c of O is dim 2c, column D/2 + c dim 2c + 1.
      if (active) {
        const float2 l0 = from_f32x2(la), l1 = from_f32x2(lb);
        const float sum = (l0.x + l0.y) + (l1.x + l1.y);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const bool valid = r < x.rows, begins = x.t0 == 0, full = begins && x.t0 + x.n == x.tiles;
        const int rr = x.first + r, qi = rr / a.group;
        T *op = static_cast<T *>(a.out) + (x.row0 + static_cast<int64_t>(qi)) * a.o_row +
                (static_cast<int64_t>(x.head) * a.group + (rr - qi * a.group)) * a.o_head;
        float *part = slots + (2 * static_cast<size_t>(blockIdx.x) + (begins ? 1 : 0)) * slot_floats(D);
        wait<STALL>(&sm.o_full[i], (jn - 1) & 1, &sm.dead, a.status);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t e0[16], e1[16];
          tmem_ld16(tm_o(i) + lanes + c * 16, e0);
          tmem_ld16(tm_o(i) + lanes + D / 2 + c * 16, e1);
          tmem_ld_wait();
          if (valid && full) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t y[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                y[z] = X::held2(__uint_as_float(e0[4 * e + z]) * inv, __uint_as_float(e1[4 * e + z]) * inv);
              reinterpret_cast<uint4 *>(op)[c * 4 + e] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4 *>(part + r * D)[c * 8 + e] = make_uint4(e0[2 * e], e1[2 * e], e0[2 * e + 1], e1[2 * e + 1]);
          }
        }
        if (valid && !full) {
          part[kRows * D + r] = limit > -INFINITY ? -base : kNegBig;
          part[kRows * D + kRows + r] = sum;
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[it % kItems]);
    }
    cp_async_wait_all();  // rows that were asked for before a wait ran out
  } else if (warp < 24) {
    // -------------------------------------------------------------- unpack
    // One record a warp and tile: its K codes and pairs (warps 8-15), its V rows (16-23).
    reg_dec<kRegsUnpack>();
    const int rw = warp & 7, g = lane >> 2, t = lane & 3;
    const bool for_k = warp < 16;
    uint4 x[D / 64];
    uint32_t pr = 0;    // lane's (s, lo): token lane % 16, of K below lane 16 and V above
    bool gone = false;  // the record's page is not usable
    bool end = false;   // no more tiles
    auto load = [&](int j) {
      const int b = j >> 2;
      if ((j & 3) == 0) wait<STALL>(&sm.src_full[b & 1], b >> 1 & 1, &sm.dead, a.status);
      const int64_t off = sm.src[b & 1][(j & 3) * 8 + rw];
      end = __any_sync(0xffffffffu, off == -3 || sm.dead);  // the lanes leave together
      if ((j & 3) == 3) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.src_empty[b & 1]);
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) x[c] = make_uint4(0, 0, 0, 0);
      pr = 0;
      gone = off == -2;
      if (off < 0) return;
      const uint8_t *rec = a.c.pages + off;
      if (!for_k) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) x[c] = __ldg(reinterpret_cast<const uint4 *>(rec + 8 * D + c * 512) + lane);
      } else if (D == 128) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) x[c] = __ldg(reinterpret_cast<const uint4 *>(rec + c * 512) + lane);
      } else {
        const uint2 y = __ldg(reinterpret_cast<const uint2 *>(rec) + lane), z = __ldg(reinterpret_cast<const uint2 *>(rec + 256) + lane);
        x[0] = make_uint4(y.x, y.y, z.x, z.y);
      }
      pr = __ldg(reinterpret_cast<const uint32_t *>(rec + 16 * D) + lane);
    };
    // A row whose own K or V pair is not finite scores NaN and has V = 0, so that only queries
    // that see it become NaN.
    auto finite = [&](float2 own) -> bool {
      const bool fin = (own.x + own.y) - (own.x + own.y) == 0.f;
      return __shfl_xor_sync(0xffffffffu, static_cast<int>(fin), 16) && fin;
    };
    load(0);
    if (for_k) {
      const float sl2 = a.scale * 1.4426950408889634f;
#pragma unroll 1
      for (int j = 0; !end; ++j) {
        const int st = j & 1;
        const float2 own = kv4_pair<BF>(pr);
        const bool both = finite(own);
        if (j >= 2) wait<STALL>(&sm.k_empty[st], (j / 2 - 1) & 1, &sm.dead, a.status);
        if (lane < 16) {
          float *kp = reinterpret_cast<float *>(&sm.kp[j & 3][rw * 8 + lane / 2]) + (lane & 1);
          kp[0] = both ? own.x * sl2 : 0.f;
          kp[2] = both ? own.y * sl2 : NAN;
        }
        const bool wide = BF && __any_sync(0xffffffffu, lane >= 16 && both && past_half(own));
        if (lane == 0) sm.hidden[j & 3][rw] = (gone ? 1 : 0) | (wide ? 2 : 0);
        // ---- K codes: lane (g, t) has dims [t D/4, (t+1) D/4) of keys g and g + 8
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint8_t *kt = sm.k[st] + (rw * 16 + h * 8 + g) * 128;
          uint32_t word[WORDS];
          if constexpr (D == 128) {
            // lanes t >= 2 take their words in another order: eight lanes of a 16-byte store then
            // hit eight different 16-byte banks
            const bool swap = t & 2;
            word[0] = swap ? x[0].z : x[0].x, word[1] = swap ? x[0].w : x[0].y;
            word[WORDS - 2] = swap ? x[0].x : x[0].z, word[WORDS - 1] = swap ? x[0].y : x[0].w;
            x[0] = x[D / 64 - 1];  // then keys g + 8
          } else {
            word[0] = h ? x[0].z : x[0].x, word[1] = h ? x[0].w : x[0].y;
          }
#pragma unroll
          for (int y = 0; y < WORDS; ++y) {
            T2 c[4];
            Codes<T>::pairs(word[y], c);
            const int chunk = t * WORDS + (D == 128 ? y ^ (t & 2) : y);  // 16-byte chunk of the row: 8 dims
            *reinterpret_cast<uint4 *>(kt + (chunk / 8) * 16384 + (((chunk & 7) ^ g) << 4)) =
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
        load(j + 1);
      }
    } else {
#pragma unroll 1
      for (int j = 0; !end; ++j) {
        const int st = j & 1;
        const float2 own = kv4_pair<BF>(pr);
        const bool both = finite(own);
        if (j >= 2) wait<STALL>(&sm.v_empty[st], (j / 2 - 1) & 1, &sm.dead, a.status);
        // transposed: tile row = dim (2b at b, 2b + 1 at D/2 + b), 64 keys per 128-byte atom
        // (s, lo) of this lane's tokens 2t, 2t+1 and 2t+8, 2t+9
        const uint32_t use = both ? pr : 0u;
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = __shfl_sync(0xffffffffu, use, 16 + 2 * t + (e & 1) + 8 * (e >> 1));
        const int c0 = (rw & 3) * 2;  // chunk of tokens 0..7 of the record
        uint8_t *v0 = sm.v[st] + (rw / 4) * (D * 128) + g * 128 + 4 * t + ((c0 ^ g) << 4);
        uint8_t *v1 = sm.v[st] + (rw / 4) * (D * 128) + g * 128 + 4 * t + (((c0 + 1) ^ g) << 4);
        // o = (dim 2b, tokens 2t..), (2b + 1, 2t..), (2b, 2t+8..), (2b + 1, 2t+8..)
        auto rows = [&](auto type, auto rare, const auto (&sc)[2], const auto (&of)[2]) {
          using U = decltype(type);
          using U2 = typename Kv4Type<U>::T2;
          const U2 top = Kv4Type<U>::from2(Kv4Type<U>::max_finite, Kv4Type<U>::max_finite);
#pragma unroll(rare.value ? 1 : D / 64)
          for (int c = 0; c < D / 64; ++c) {
            const uint4 xc = rare.value && c ? x[D / 64 - 1] : x[rare.value ? 0 : c];
            const uint32_t y[4] = {xc.x, xc.y, xc.z, xc.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              U2 o[4];
              Codes<U>::pairs(y[e], o);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                o[z] = __hfma2(o[z], sc[z / 2], of[z / 2]);
                if (rare.value) o[z] = __hmax2(__hmin2(o[z], top), __hneg2(top));
                *reinterpret_cast<U2 *>((z < 2 ? v0 : v1) + (c * 32 + e * 8) * 128 + (z & 1) * D * 64) = o[z];
              }
            }
          }
        };
        // bf16 rows go in as fp16, which holds them eight times as exactly, while they are in its
        // range.  15 s + lo can pass the type's largest value (s is rounded), and the bytes of a record
        // that no token has written may say anything, s < 0 too: values are held within the type, as
        // a hidden key's weight of 0 must meet no infinity.  (Zeros for what lies behind the last key
        // instead cost all records 1 to 2 %: four prompts 186 -> 190 us.)
        const bool wide = BF && __any_sync(0xffffffffu, lane >= 16 && both && past_half(own));
        if (BF && __builtin_expect(!wide, 1)) {
          __half2 sc[2], of[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 u = kv4_pair<BF>(q[2 * h]), w = kv4_pair<BF>(q[2 * h + 1]);
            sc[h] = __floats2half2_rn(u.x, w.x);
            of[h] = __floats2half2_rn(u.y, w.y);
          }
          rows(__half{}, std::false_type{}, sc, of);
        } else {
          T2 sc[2], of[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sc[h] = kv4_bits<T2>(__byte_perm(q[2 * h], q[2 * h + 1], 0x5410));
            of[h] = kv4_bits<T2>(__byte_perm(q[2 * h], q[2 * h + 1], 0x7632));
          }
          if (BF || __builtin_expect(__any_sync(0xffffffffu, fabsf(fmaf(15.f, own.x, own.y)) > X::max_finite), 0))
            rows(T{}, std::true_type{}, sc, of);
          else
            rows(T{}, std::false_type{}, sc, of);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !(STALL && j == 1)) mbar_arrive(&sm.v_full[st]);
        load(j + 1);
      }
    }
  } else {
    reg_dec<kRegsMma>();
    if (warp == 24) {
      // --------------------------------------------------------------- MMA
      constexpr uint32_t kind = BF ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t id_qk = idesc_f16_f32(128, kKeys) | kind, id_pv = idesc_f16_f32(128, D);
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(sm.q)), k_desc = sw128_kmajor_desc(smem_u32(sm.k)),
                     v_desc = sw128_kmajor_desc(smem_u32(sm.v));
      constexpr uint32_t kStage = 128 * D * 2 >> 4;  // an operand tile, in the descriptors' units
      auto qk = [&](int i, int jt) {
        const uint64_t qd = q_desc + i * kStage, kd = k_desc + (jt & 1) * kStage;
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint64_t adv = (x / 4) * (16384 >> 4) + (x % 4) * 2;
            mma_f16(tm_s(i), qd + adv, kd + adv, id_qk, x > 0);
          }
          mma_commit(&sm.s_full[i]);
        }
        __syncwarp();
      };
      auto pv = [&](int i, int jt, bool add) {
        const uint64_t vd = v_desc + (jt & 1) * kStage;
        // a byte per record, that is per 16 keys
        const uint64_t wide = BF ? *reinterpret_cast<const uint64_t *>(sm.hidden[jt & 3]) & 0x0202020202020202ull : 0;
        if (elect_one()) {
          if (BF && __builtin_expect(wide != 0, 0)) {
#pragma unroll 1
            for (int x = 0; x < kKeys / 16; ++x)
              mma_f16_ts(tm_o(i), tm_s(i) + x * 8, vd + (x / 4) * ((D * 128) >> 4) + (x % 4) * 2,
                         wide >> (8 * x) & 2 ? id_pv | kind : id_pv, add || x > 0);
          } else {
#pragma unroll
            for (int x = 0; x < kKeys / 16; ++x)
              mma_f16_ts(tm_o(i), tm_s(i) + x * 8, vd + (x / 4) * ((D * 128) >> 4) + (x % 4) * 2, id_pv, add || x > 0);
          }
          mma_commit(&sm.o_full[i]);
        }
        __syncwarp();
      };
      // Per key tile and row tile: O += P V, then S of the next key tile, which may be the next item's.
      int it = 0, j = 0, n = 0, n0 = 0, row_tiles = 0;  // of the tile whose P V comes next
      uint32_t p_phase = 0, q_phase = 0;  // a bit per row tile
#pragma unroll 1
      for (int jt = -1;; ++jt) {
        int next_n = n, next_n0 = n0, next_tiles = row_tiles;
        const bool turn = j + 1 >= n;  // the next scores are another item's
        if (turn) {
          const int slot = (n ? it + 1 : it) % kItems;
          wait<STALL>(&sm.item_full[slot], (n ? it + 1 : it) / kItems & 1, &sm.dead, a.status);
          next_n = sm.item[slot].n;
          next_n0 = sm.item[slot].n0;
          next_tiles = __any_sync(0xffffffffu, next_n == 0 || sm.dead) ? 0 : sm.item[slot].rows > 128 ? 2 : 1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
        }
        if (row_tiles) wait<STALL>(&sm.v_full[jt & 1], (jt / 2) & 1, &sm.dead, a.status);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i < row_tiles && (i || j < n0)) {
            wait<STALL>(&sm.p_full[i], p_phase >> i & 1, &sm.dead, a.status);
            p_phase ^= 1u << i;
            tc_fence_after();
            pv(i, jt, j > 0);
          }
          if (i == 0 && next_tiles) wait<STALL>(&sm.k_full[(jt + 1) & 1], ((jt + 1) / 2) & 1, &sm.dead, a.status);
          if (i < next_tiles && (i || (turn ? 0 : j + 1) < next_n0)) {
            if (turn) {
              wait<STALL>(&sm.q_full[i], q_phase >> i & 1, &sm.dead, a.status);
              q_phase ^= 1u << i;
            }
            tc_fence_after();
            qk(i, jt + 1);
          }
        }
        if (row_tiles && elect_one()) mma_commit(&sm.v_empty[jt & 1]);
        __syncwarp();
        if (!next_tiles) break;
        if (elect_one()) mma_commit(&sm.k_empty[(jt + 1) & 1]);
        __syncwarp();
        if (turn) {
          if (n) ++it;
          j = 0;
        } else {
          ++j;
        }
        n = next_n;
        n0 = next_n0;
        row_tiles = next_tiles;
      }
      if (elect_one()) mma_commit(&sm.done);  // nothing in flight when the CTA gives its memory back
      mbar_wait(&sm.done, 0, kWaitNs);
    } else if (warp == 25) {
      // -------------------------------------------------------------- walk
      // Items and the places of records, four tiles (32 lanes) at a time, ahead of the other roles.
      int it = 0, pj = 0;
      auto publish = [&](bool end) {
        if (it >= kItems) wait<STALL>(&sm.item_empty[it % kItems], (it / kItems - 1) & 1, &sm.dead, a.status);
        const int n = end ? 0 : w.t1 - w.t0, first = w.block * kRows;
        const int seen0 = min(w.q.len, w.q.pos0 + (first + min(127, w.rows() - 1)) / a.group + 1);
        const bool less = n > 1 && w.k.key0(w.t1 - 1) >= seen0;
        if (lane == 0)
          sm.item[it % kItems] = Item{n, w.t0, w.k.tiles, w.k.sinks, w.k.skip, w.q.row0, w.rows(),
                                      w.q.len, w.q.pos0, first, w.head, less ? n - 1 : n};
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_full[it % kItems]);
        ++it;
      };
      Desc d{-1, 0, 0, 0, 0, {}};
      bool going = span > 0 && w.t1 > w.t0;
      const bool any = going;
      if (any) publish(false);
#pragma unroll 1
      for (int b = 0; b == 0 || going; ++b) {
        int key = 0, len = 0, seq = 0, head = 0;
        bool tile = false;  // the lane's place has one
#pragma unroll 1
        for (int x = 0; x < 4; ++x, ++pj) {
          if (going && pj == w.t1 - w.t0) {
            going = w.more();
            if (going) {
              w.next(a);
              pj = 0;
              publish(false);
            }
          }
          if (going && lane / 8 == x) {
            tile = true;
            key = w.k.key0(w.t0 + pj) + (lane & 7) * 16;
            len = w.q.len;
            seq = w.seq;
            head = w.head;
          }
        }
        int64_t off = tile ? -1 : -3;
        if (key < len) {
          const int rec = key / 16;
          const int slot = a.c.page_shift >= 0 ? rec >> a.c.page_shift : rec / a.c.recs_per_page;
          const int page = __ldg(a.b.table + seq * a.b.table_stride + slot);
          if (page < 0 || page >= a.c.n_pages) {
            off = -2;
            record_error(a.status, kErrInvalidArg);
          } else {
            off = page * a.c.page_stride + (static_cast<int64_t>(head) * a.c.recs_per_page + (rec - slot * a.c.recs_per_page)) * REC;
          }
        }
        if (b >= 2) wait<STALL>(&sm.src_empty[b & 1], (b / 2 - 1) & 1, &sm.dead, a.status);
        sm.src[b & 1][lane] = off;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.src_full[b & 1]);
      }
      if (any && w.t0 == 0 && w.t1 < w.k.tiles)
        d = Desc{static_cast<int>((w.start + w.length() - 1) / quota), w.q.row0, w.block * kRows, w.rows(), w.head, {}};
      publish(true);
      if (lane == 0) desc[blockIdx.x] = d;
    }
  }
  __syncthreads();
  if (warp == 24) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool STALL = false>
cudaError_t launch(const Kv4AttnArgs &a, cudaStream_t stream) {
  auto kernel = kv4_tile_kernel<T, D, STALL>;
  const int smem = static_cast<int>(sizeof(TileSmem<D>));
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.num_sms, 1, 1);
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

size_t kv4_tile_workspace(int d, int num_sms) {
  return num_sms * sizeof(Desc) + num_sms * 2 * slot_floats(d) * sizeof(float);
}

cudaError_t launch_kv4_tile(const Kv4AttnArgs &a, cudaStream_t stream) {
  if (a.stall && !a.c.bf16 && a.c.d == 64) return launch<__half, 64, true>(a, stream);
  if (a.c.bf16)
    return a.c.d == 128 ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
  return a.c.d == 128 ? launch<__half, 128>(a, stream) : launch<__half, 64>(a, stream);
}

}  // namespace mixq
