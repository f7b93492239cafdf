// What the window and tree attention kernels share: the call's parameters, which rows
// and tokens a block works on, and which of them see each other.
#pragma once

#include <cuda_bf16.h>

#include "attention_mma.cuh"
#include "common.cuh"
#include "kv_layout.cuh"

namespace idx {

constexpr int kTile = 64;                        // tokens
constexpr int kPieces = kKvDim / 64;             // 128-byte pieces of a token's bf16 row
constexpr uint64_t kWaitLimitNs = 2000000000ull;
// log2 of what P may reach before O is rescaled. P, l and O are floating point, so their relative precision does not
// depend on the reference; with 2^31 tokens of values below 2^17, O stays below 2^88.
constexpr float kRescaleStep = 40.0f;
constexpr int kAhead = 4;                        // tiles between the L2 prefetch and the loads
constexpr int kMaxSplitRequests = 160;           // of a call whose contexts are split
constexpr int kJoinTiles = 3;                    // a part's extra stores and the join, in tiles

// Bit 0: a visible page outside the table or the cache (its tokens are skipped). Bit 1: a wait expired.
static __device__ unsigned int g_paged_error = 0;

struct PagedParams {
  const __nv_bfloat16* q;
  int64_t ld_q, ld_qh;  // elements between rows, between heads
  const uint8_t* cache;
  int num_blocks, block_size;
  int64_t block_stride;
  const int32_t* block_table;
  int64_t ld_bt;
  int n_pages;
  const int32_t* cu_rows;
  const int32_t* ctx_lens;
  int B;
  int window, sinks;     // of the window attention
  const int32_t* mask;   // of the tree attention
  int64_t ld_mask;
  int words;
  int T, H;
  float scale_log2;  // softmax_scale * log2(e)
  __nv_bfloat16* out;
  int64_t ld_out, ld_oh;
  float* lse;
  int64_t ld_lse;
  int page_shift;              // log2(block_size)
  int head_blocks, heads;      // groups of heads, and the heads of one
  int tokens;                  // query rows of a unit
  int capacity;                // parts that there is room for; 0: contexts are not split
  int2* ws_sched;              // [B]: first part of a request and its parts a unit
  float2* ws_ml;               // [capacity, rows of a part]: maximum (log2 units) and sum
  float* ws_o;                 // [capacity, rows of a part, dims of a part]: accumulators
};

// A unit of work: consecutive query rows of one request with one group of heads, and a range of the tiles of the
// tokens that they see together.
struct Unit {
  int request, row0, rows;  // q rows [row0, row0 + rows)
  int head0, heads;
  int half;                 // which half of the dims, where a unit is one of two
  int pos0;                 // position of the first row
  int base, ctx;            // tokens of the request before its new rows, and with them
  int lo, hi;               // tokens in [0, first) or [lo, hi] are seen by a row
  int first;
  int skip;                 // tiles from 0 that hold the first tokens; the others start at tile_lo
  int tile_lo;
  int tile0, tiles;         // this part's range
  int part, parts;          // global number of the part (of a split context), and the parts of the unit
};

__device__ __forceinline__ int row_at(const PagedParams& p, int b) {
  return min(max(__ldg(p.cu_rows + b), 0), p.T);
}

// Tokens that the table has pages for.
__device__ __forceinline__ int table_tokens(const PagedParams& p) {
  return static_cast<int>(min(static_cast<int64_t>(p.n_pages) << p.page_shift, static_cast<int64_t>(INT32_MAX)));
}

// Which tokens rows [first, last] of the unit's request see together, and the number of their tiles.
template <bool kTree>
__device__ __forceinline__ int seen_tiles(const PagedParams& p, int first, int last, Unit& u) {
  if (kTree) {
    u.hi = u.ctx - 1;
    u.lo = 0;
    u.first = 0;
  } else {
    u.hi = u.base + last;
    u.lo = u.base + first >= p.window ? u.base + first - p.window + 1 : 0;
    u.first = min(p.sinks, u.hi + 1);
  }
  u.hi = min(u.hi, table_tokens(p) - 1);
  u.tile_lo = u.lo / kTile;
  u.skip = min((u.first + kTile - 1) / kTile, u.tile_lo);
  if (u.hi < 0) return u.skip = 0;
  return u.skip + max(u.hi / kTile - u.tile_lo + 1, 0);
}

// No unit of a request with n new rows has more tiles.
template <bool kTree>
__device__ __forceinline__ int most_tiles(const PagedParams& p, int n, int ctx) {
  const int all = (min(ctx, table_tokens(p)) + kTile - 1) / kTile;
  if (kTree) return max(all, 1);
  const int64_t near = (static_cast<int64_t>(p.window) + min(p.tokens, n) - 2) / kTile + 2;
  return max(static_cast<int>(min(static_cast<int64_t>(all), near + (min(p.sinks, ctx) + kTile - 1) / kTile)), 1);
}

// The block's (pair's) unit, found by every warp for itself; false: there is none. `kHalves`: units that share
// their rows. All lanes get the same.
template <bool kTree, int kHalves>
__device__ __forceinline__ bool find_unit(const PagedParams& p, int index, Unit& u) {
  const int lane = threadIdx.x & 31;
  const int U = p.tokens;
  int group, at, n;
  if (p.capacity == 0) {
    // Groups of U rows of all requests have numbers: those of request b start at floor(cu_rows[b] / U) + b, which
    // leaves room for its last, part-filled one.
    u.half = index % kHalves;
    u.head0 = index / kHalves % p.head_blocks * p.heads;
    const int g = index / kHalves / p.head_blocks;
    int lo = 0, hi = p.B;  // the last b with a first group <= g, 32 candidates a round
    while (true) {
      const int step = (hi - lo + 31) / 32, b = lo + lane * step;
      int first = 0, next = 0, ctx = 0;
      if (b < hi) {
        first = row_at(p, b);
        if (step == 1) {  // the last round: what is needed of the request comes along
          next = row_at(p, b + 1);
          ctx = __ldg(p.ctx_lens + b);
        }
      }
      const int src = __popc(__ballot_sync(0xFFFFFFFFu, b < hi && first / U + b <= g)) - 1;
      if (src < 0) return false;
      lo += src * step;
      if (step == 1) {
        at = __shfl_sync(0xFFFFFFFFu, first, src);
        n = __shfl_sync(0xFFFFFFFFu, next, src) - at;
        u.ctx = __shfl_sync(0xFFFFFFFFu, ctx, src);
        break;
      }
      hi = min(lo + step, hi);
    }
    u.request = lo;
    group = g - at / U - lo;
    u.part = 0;
    u.parts = 1;
  } else {
    // Every request's units are cut into parts of `per` tiles, `per` the same for all and about the smallest with
    // which one wave has room for all parts.
    constexpr int kPer = kMaxSplitRequests / 32;
    int first[kPer], rows[kPer], ctxs[kPer], units[kPer], most[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int b = 32 * k + lane;
      first[k] = rows[k] = ctxs[k] = 0;
      if (b < p.B) {
        first[k] = row_at(p, b);
        rows[k] = row_at(p, b + 1);
        ctxs[k] = __ldg(p.ctx_lens + b);
      }
    }
    int64_t sum = 0;
    int longest = 1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      rows[k] -= first[k];
      units[k] = most[k] = 0;
      if (rows[k] > 0) {
        units[k] = (rows[k] + U - 1) / U * p.head_blocks * kHalves;
        most[k] = most_tiles<kTree>(p, rows[k], max(ctxs[k], 0));
      }
      sum += static_cast<int64_t>(units[k]) * most[k];
      longest = max(longest, most[k]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    int per = static_cast<int>(min(max((sum + p.capacity - 1) / p.capacity, int64_t{1}), static_cast<int64_t>(longest)));
    int count[kPer];
    while (true) {
      if (per + kJoinTiles >= longest) per = longest;  // whole contexts cost less than parts and their join
      int total = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        count[k] = (most[k] + per - 1) / per;
        total += units[k] * count[k];
      }
      total = __reduce_add_sync(0xFFFFFFFFu, total);
      if (total <= p.capacity || per == longest) break;
      per += max(per / 8, 1);
    }
    int before = 0, found_at = 0, found_units = 0, found_parts = 0;
    u.request = -1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int mine = units[k] * count[k];
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
      }
      const int start = before + upto - mine;
      if (index == 0 && threadIdx.x < 32 && 32 * k + lane < p.B) p.ws_sched[32 * k + lane] = make_int2(start, count[k]);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, index >= start && index < start + mine);
      if (who) {
        const int src = __ffs(who) - 1;
        u.request = 32 * k + src;
        found_at = __shfl_sync(0xFFFFFFFFu, start, src);
        found_units = __shfl_sync(0xFFFFFFFFu, units[k], src);
        found_parts = __shfl_sync(0xFFFFFFFFu, count[k], src);
        at = __shfl_sync(0xFFFFFFFFu, first[k], src);
        n = __shfl_sync(0xFFFFFFFFu, rows[k], src);
        u.ctx = __shfl_sync(0xFFFFFFFFu, ctxs[k], src);
      }
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (u.request < 0) return false;
    const int in = index - found_at, unit = in % found_units;  // units vary fastest: they read the same tokens
    u.half = unit % kHalves;
    u.head0 = unit / kHalves % p.head_blocks * p.heads;
    group = unit / kHalves / p.head_blocks;
    u.part = index;
    u.parts = found_parts;
    u.tile0 = in / found_units * per;
    u.tiles = per;
  }
  const int start = group * U;
  if (start >= n) return false;
  u.row0 = at + start;
  u.rows = min(U, n - start);
  u.heads = min(p.heads, p.H - u.head0);
  u.ctx = max(u.ctx, 0);
  u.base = u.ctx - n;
  u.pos0 = u.base + start;
  const int all = seen_tiles<kTree>(p, start, start + u.rows - 1, u);
  if (u.ctx > table_tokens(p) && threadIdx.x == 0) atomicOr(&g_paged_error, 1u);
  if (p.capacity == 0) {
    u.tile0 = 0;
    u.tiles = all;
  } else {
    u.tiles = max(min(u.tiles, all - u.tile0), 0);
  }
  return true;
}

// First token of the part's tile i.
__device__ __forceinline__ int tile_start(const Unit& u, int i) {
  const int t = u.tile0 + i;
  return (t < u.skip ? t : t - u.skip + u.tile_lo) * kTile;
}

// Whether a row of the unit sees token j.
__device__ __forceinline__ bool unit_sees(const Unit& u, int j) { return j <= u.hi && (j >= u.lo || j < u.first); }

// The table's entry for token j, as it stands there; -1 if no row sees the token or the table has no such page. Nothing
// here waits for the entry, so that it can be asked for long before its use.
__device__ __forceinline__ int entry_of(const PagedParams& p, const Unit& u, int j) {
  const int page = j >> p.page_shift;
  return unit_sees(u, j) && page < p.n_pages ? __ldg(p.block_table + u.request * p.ld_bt + page) : -1;
}

__device__ __forceinline__ bool is_block(const PagedParams& p, int entry) {
  return static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_blocks);
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Bit c: whether row t of the unit sees token x + c.
template <bool kTree>
__device__ __forceinline__ uint32_t row_sees(const PagedParams& p, const Unit& u, int t, int x) {
  if (t >= u.rows) return 0;
  if (kTree) {
    uint32_t bits = low_bits(u.base - x);
    const int node = x - u.base;  // of bit 0
    if (node > -32 && bits != 0xFFFFFFFFu) {
      const int w = node >> 5;  // rounded down
      const int32_t* row = p.mask + (u.row0 + t) * p.ld_mask;
      const uint32_t a = w >= 0 && w < p.words ? static_cast<uint32_t>(__ldg(row + w)) : 0u;
      const uint32_t b = w + 1 >= 0 && w + 1 < p.words ? static_cast<uint32_t>(__ldg(row + w + 1)) : 0u;
      bits |= __funnelshift_r(a, b, node & 31);
    }
    return bits & low_bits(u.ctx - x);
  } else {
    const int pos = u.pos0 + t;
    const int from = pos >= p.window ? pos - p.window + 1 : 0;
    return low_bits(pos - x + 1) & (~low_bits(from - x) | low_bits(p.sinks - x));
  }
}

// One look at the codes of a token's four scales: a word of multiplier exponents, all zero for a token
// that is not finite (kKvNanScaleCode). Multiplied by zero it leaves no trace in the products; the softmax makes the
// rows that see it NaN by a flag, so that it cannot reach the others through 0 * NaN.
__device__ __forceinline__ bool codes_finite(uint32_t codes) {
  return __vcmpgtu4(codes, kKvMaxScaleCode * 0x01010101u) == 0u;
}
__device__ __forceinline__ uint32_t multiplier_bytes(uint32_t codes) {
  return codes_finite(codes) ? __vadd4(codes, 0x78787878u) : 0u;  // exponent field code + 120, as kv_dequant_multiplier
}

// Bounded wait. A wait that takes two seconds marks the block dead and raises the device
// flag; from then on no wait blocks, every role runs its remaining iterations on whatever it
// finds (all addresses stay in bounds), and the block ends in order.
template <class S>
__device__ __forceinline__ void wait_for(S& sh, uint64_t* bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) {
    const uint64_t t0 = global_timer_ns();
    while (!sh.dead && !mbar_try_wait(bar, parity)) {
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_paged_error, 2u);
        sh.dead = 1;
      }
    }
  }
  __syncwarp();
}

}  // namespace idx
