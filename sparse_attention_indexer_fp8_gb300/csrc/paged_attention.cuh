// What the window and tree attention kernel works on: the call's parameters, how its work is cut into units and shared
// out, which rows and tokens a unit has and which of them see each other.
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
// Requests of a call whose work is shared out: a warp holds their lengths, five a lane. With ten a lane, the kernel's
// registers fell out so that every call took 8-10 % longer.
constexpr int kMaxSharedRequests = 160;
constexpr int kUnitTiles = 6;                    // a unit's start and end, in tiles
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
  int workers;                 // blocks that share the units; 0: a block a unit
  bool cut;                    // shares are even, and may begin and end within a unit; else whole units in turn
  struct Cut* ws_cuts;         // [workers]
  float2* ws_ml;               // [2 workers, 64 rows]: maximum (log2 units) and sum of a part
  float* ws_o;                 // [2 workers, 64 rows, 512]: accumulators
};

// The unit that the end of a worker's share cuts, if the worker has its first part: for the join.
struct alignas(16) Cut {
  int row0, rows, head0, heads;
  int parts;  // 0: none
  int unused[3];
};

// A unit of work: consecutive query rows of one request with one group of heads, and a range of the tiles of the
// tokens that they see together.
struct alignas(16) Unit {
  int request;
  int lo, hi;               // tokens in [0, first) or [lo, hi] are seen by a row
  int first;
  int skip;                 // tiles from 0 that hold the first tokens; the others start at tile_lo
  int tile_lo;
  int tile0, tiles;         // this part's range
  int row0, rows;           // q rows [row0, row0 + rows)
  int head0, heads;
  int pos0;                 // position of the first row
  int base, ctx;            // tokens of the request before its new rows, and with them
  int part;                 // number of the part; -1: the unit is whole
  int parts;                // of the unit
  bool any;                 // false: there is no unit left
};

// Where a unit's tokens lie, out of shared memory: eight words that need not stay in registers.
__device__ __forceinline__ Unit tokens_of(uint32_t unit) {
  const uint4 a = ld_shared16(unit), b = ld_shared16(unit + 16);
  Unit u;
  u.request = static_cast<int>(a.x);
  u.lo = static_cast<int>(a.y);
  u.hi = static_cast<int>(a.z);
  u.first = static_cast<int>(a.w);
  u.skip = static_cast<int>(b.x);
  u.tile_lo = static_cast<int>(b.y);
  u.tile0 = static_cast<int>(b.z);
  u.tiles = static_cast<int>(b.w);
  return u;
}

__device__ __forceinline__ int row_at(const PagedParams& p, int b) {
  return min(max(__ldg(p.cu_rows + b), 0), p.T);
}

// Tokens that the table has pages for.
__device__ __forceinline__ int table_tokens(const PagedParams& p) {
  return static_cast<int>(min(static_cast<int64_t>(p.n_pages) << p.page_shift, static_cast<int64_t>(INT32_MAX)));
}

// Tiles of n tokens, of as many as 32 bits count.
__device__ __forceinline__ int tiles_of(int n) { return n / kTile + (n % kTile > 0); }

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
  u.skip = min(tiles_of(u.first), u.tile_lo);
  if (u.hi < 0) return u.skip = 0;
  return u.skip + max(u.hi / kTile - u.tile_lo + 1, 0);
}

// No unit of a request with n new rows has more tiles.
template <bool kTree>
__device__ __forceinline__ int most_tiles(const PagedParams& p, int n, int ctx) {
  const int all = tiles_of(min(ctx, table_tokens(p)));
  if (kTree) return max(all, 1);
  const int64_t near = (static_cast<int64_t>(p.window) + min(p.tokens, n) - 2) / kTile + 2;
  return max(static_cast<int>(min(static_cast<int64_t>(all), near + tiles_of(min(p.sinks, ctx)))), 1);
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Whether one of `rows` masks, every `step`-th from `row` on, has a bit of nodes [from, to). Asked only where a page is
// missing, to say whether that is an error; not inlined, so that it takes no registers from the loops around it.
static __device__ __noinline__ bool nodes_seen(const int32_t* masks, int64_t ld_mask, int words, int row, int rows, int step,
                                               int from, int to) {
  for (; row < rows; row += step) {
    for (int w = from >> 5; w < words && 32 * w < to; ++w) {
      const uint32_t in = ~low_bits(from - 32 * w) & low_bits(to - 32 * w);
      if (static_cast<uint32_t>(__ldg(masks + row * ld_mask + w)) & in) return true;
    }
  }
  return false;
}

// Completes a unit of rows from `start` on, of a request whose n new rows begin at row `at`; its tiles are [u.tile0,
// u.tile0 + u.tiles) as far as there are as many. False: it has no row, or, where cu_rows does not ascend, none of the
// request's.
template <bool kTree>
__device__ __forceinline__ bool complete_unit(const PagedParams& p, int at, int n, int start, Unit& u) {
  if (start < 0 || start >= n) return false;
  u.row0 = at + start;
  u.rows = min(p.tokens, n - start);
  u.heads = min(p.heads, p.H - u.head0);
  u.ctx = max(u.ctx, 0);
  u.base = u.ctx - n;
  u.pos0 = u.base + start;
  const int all = seen_tiles<kTree>(p, start, start + u.rows - 1, u);
  const int known = table_tokens(p);
  if (u.ctx > known) {  // the last of a window's rows sees the last token, of nodes their masks tell
    const int lane = threadIdx.x & 31;
    const bool seen = !kTree || u.base > known ||
                      nodes_seen(p.mask + u.row0 * p.ld_mask, p.ld_mask, p.words, lane, u.rows, 32, max(known - u.base, 0), n);
    if (seen) atomicOr(&g_paged_error, 1u);
  }
  u.tiles = max(min(u.tiles, all - u.tile0), 0);
  return true;
}

// Unit number `index` of the grid; false: there is none. All lanes get the same.
template <bool kTree>
__device__ __forceinline__ bool find_unit(const PagedParams& p, int index, Unit& u) {
  const int lane = threadIdx.x & 31, U = p.tokens;
  // Groups of U rows of all requests have numbers: those of request b start at floor(cu_rows[b] / U) + b, which
  // leaves room for its last, part-filled one.
  const int g = index / p.head_blocks;
  u.head0 = (index - g * p.head_blocks) * p.heads;
  int at, n, lo = 0, hi = p.B;  // the last b with a first group <= g, 32 candidates a round
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
  u.part = -1;
  u.tile0 = 0;
  u.tiles = INT32_MAX;
  return complete_unit<kTree>(p, at, n, (g - at / U - lo) * U, u);
}

// All units of a call in one line, request after request, computed by one warp from the lengths, which the host does not
// know. Where shares are even, a unit is as long as its tiles, and where there are more units than workers, as what its
// start and end cost besides; every worker gets the same share of the line, and only the line's cuts split a unit. Where
// whole units are taken in turn, each is one long.
template <bool kTree>
struct Line {
  static constexpr int kPer = kMaxSharedRequests / 32;  // requests of a lane: b = 32 k + lane
  int first[kPer], rows[kPer], ctxs[kPer], units[kPer], length[kPer];
  int start[kPer];   // of the request's units
  int total, share;
  int extra;         // of a unit's length, the part that is not tiles

  __device__ __forceinline__ explicit Line(const PagedParams& p) {
    const int lane = threadIdx.x & 31, used = (p.B + 31) / 32;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      first[k] = rows[k] = ctxs[k] = 0;
      const int b = 32 * k + lane;
      if (b < p.B) {
        first[k] = row_at(p, b);
        rows[k] = row_at(p, b + 1);
        ctxs[k] = __ldg(p.ctx_lens + b);
      }
    }
    int longest = 1, all = 0, sum = 0;  // the host lets no call in whose sums are near 32 bits
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      units[k] = length[k] = 0;
      if (k >= used) continue;
      rows[k] -= first[k];
      if (rows[k] > 0) {
        units[k] = (rows[k] + p.tokens - 1) / p.tokens * p.head_blocks;
        length[k] = p.cut ? most_tiles<kTree>(p, rows[k], max(ctxs[k], 0)) : 1;
      }
      all += units[k];
      sum += units[k] * length[k];
      longest = max(longest, length[k]);
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    extra = p.cut && all > p.workers ? kUnitTiles : 0;
    sum = __reduce_add_sync(0xFFFFFFFFu, sum) + all * extra;
    longest += extra;
#pragma unroll
    for (int k = 0; k < kPer; ++k) length[k] += extra;
    // A share is the workers' part of the line, or where the 128 KB that every part stores and the join reads (0.04 us at
    // 6.6 TB/s) cost as much as one more tile for each (1.5 us).
    share = max((sum + p.workers - 1) / p.workers, static_cast<int>(0.5f + sqrtf(0.025f * static_cast<float>(sum))));
    // With fewer units than workers, a share may begin in one unit and end in another, and has two starts and ends. Where
    // that costs more, units are lengthened to whole numbers of shares: of `per` tiles, the fewest with which all have room,
    // or all of the longest.
    int per = 0;
    if (p.cut && all <= p.workers) {
      per = min(share, longest);
      while (true) {
        if (per + kJoinTiles >= longest) per = longest;  // whole contexts cost less than parts and their join
        int parts = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          if (k < used) parts += units[k] * ((length[k] + per - 1) / per);
        }
        parts = __reduce_add_sync(0xFFFFFFFFu, parts);
        if (parts <= p.workers || per == longest) break;
        per += max(per / 8, 1);
      }
      if (per > share + kUnitTiles) per = 0;
    }
    if (per) share = per;
    int before = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      start[k] = 0;
      if (k >= used) continue;
      if (per) length[k] = (length[k] + per - 1) / per * per;
      const int mine = units[k] * length[k];
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
      }
      start[k] = before + upto - mine;
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    total = min(before, INT32_MAX / 2);  // as the host knows it of ranges that ascend; a worker steps beyond it
  }

  // The unit at `at` of the line: where it starts there, and its length. Sets the unit's request, ctx and heads;
  // `row`, `n` and `from` are the request's first row, its rows, and the unit's first of them.
  __device__ __forceinline__ int unit_at(const PagedParams& p, int at, Unit& u, int& len, int& row, int& n, int& from) const {
    const int used = (p.B + 31) / 32;
    int begin = 0;
    u.request = 0;
    len = 1;
    row = n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (k >= used) continue;
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, at >= start[k] && at - start[k] < units[k] * length[k]);
      if (who) {
        const int src = __ffs(who) - 1;
        u.request = 32 * k + src;
        begin = __shfl_sync(0xFFFFFFFFu, start[k], src);
        len = __shfl_sync(0xFFFFFFFFu, length[k], src);
        row = __shfl_sync(0xFFFFFFFFu, first[k], src);
        n = __shfl_sync(0xFFFFFFFFu, rows[k], src);
        u.ctx = __shfl_sync(0xFFFFFFFFu, ctxs[k], src);
      }
    }
    const int unit = (at - begin) / len, group = unit / p.head_blocks;
    u.head0 = (unit - group * p.head_blocks) * p.heads;
    from = group * p.tokens;
    return begin + unit * len;
  }
};

// A worker's place on the line, and the end of its share; pos < 0 at first.
struct Place {
  int pos, end;
};

// The worker's next unit, or part of one, found by one warp. False: there is none left.
template <bool kTree>
__device__ __forceinline__ bool next_unit(const PagedParams& p, int worker, Place& place, Unit& u) {
  const bool at_first = place.pos < 0;
  if (p.workers == 0) {
    place.pos = 0;
    return at_first && find_unit<kTree>(p, worker, u);
  }
  if (p.cut && !at_first && place.pos >= place.end) return false;
  const Line<kTree> line(p);
  int len, row, n, from;
  if (!p.cut) {
    place.pos = at_first ? worker : place.pos + p.workers;
    if (place.pos >= line.total) return false;
    // windows from the last rows on: of causal rows these see most, and what is long should not begin last
    line.unit_at(p, kTree ? place.pos : line.total - 1 - place.pos, u, len, row, n, from);
    u.tile0 = 0;
    u.tiles = INT32_MAX;
    u.part = -1;
    return complete_unit<kTree>(p, row, n, from, u);
  }
  if (at_first) {
    // as many shares as there are workers cover the line, and little more
    place.pos = worker * line.share;
    place.end = min(place.pos + line.share, line.total);
    if (place.pos >= place.end) return false;
  }
  const int pos = place.pos;
  const int begin = line.unit_at(p, pos, u, len, row, n, from);
  const int stop = min(begin + len, place.end);
  u.tile0 = max(pos - begin - line.extra, 0);
  u.tiles = max(stop - begin - line.extra, 0) - u.tile0;
  // A unit's first part is its worker's last, any other its worker's first.
  u.part = pos == begin && stop == begin + len ? -1 : pos == begin ? 2 * worker + 1 : 2 * worker;
  u.parts = min((begin + len - 1) / line.share, p.workers - 1) - worker + 1;  // where this is the first
  place.pos = stop;
  return complete_unit<kTree>(p, row, n, from, u);
}

// One warp finds the worker's unit and leaves it in `unit`; `unit.any` is false after the last.
template <bool kTree>
__device__ __forceinline__ void find_next(const PagedParams& p, int worker, bool first, Place& place, Unit& unit) {
  Unit u;
  Place at = first ? Place{-1, 0} : place;
  u.any = next_unit<kTree>(p, worker, at, u);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    unit = u;
    place = at;
    if (p.cut) {
      if (first) p.ws_cuts[worker].parts = 0;
      if (u.any && u.part == 2 * worker + 1) p.ws_cuts[worker] = Cut{u.row0, u.rows, u.head0, u.heads, u.parts, {0, 0, 0}};
    }
  }
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

// Tokens [lo, hi] are all seen by row t of the unit; most tiles lie within.
template <bool kTree>
__device__ __forceinline__ int2 all_seen(const PagedParams& p, const Unit& u, bool have, int t) {
  if (!have) return make_int2(0, -1);
  if (kTree) return make_int2(0, u.base - 1);
  const int pos = u.pos0 + t;
  return make_int2(pos >= p.window ? pos - p.window + 1 : 0, pos);
}

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

// Multiplier exponents of a token's four scales, code + 120 as in kv_dequant_multiplier; all zero for a token that is
// not finite (kKvNanScaleCode). Multiplied by zero it leaves no trace in the products; the softmax makes the rows that
// see it NaN by a flag, so that it cannot reach the others through 0 * NaN.
__device__ __forceinline__ uint32_t multiplier_bytes(uint32_t codes) {
  return __vcmpgtu4(codes, kKvMaxScaleCode * 0x01010101u) == 0u ? __vadd4(codes, 0x78787878u) : 0u;
}

// Two values at once: a * b + c, and a + b.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The largest of 32 logits v * unit, in four chains.
__device__ __forceinline__ float softmax_top(const uint32_t (&v)[32], float unit) {
  float top[4];
  if (unit >= 0.f) {
#pragma unroll
    for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(v[c]);
#pragma unroll
    for (int c = 4; c < 32; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(v[c]));
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * unit;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(v[c]);
#pragma unroll
  for (int c = 4; c < 32; ++c) top[c & 3] = fminf(top[c & 3], __uint_as_float(v[c]));
  return fminf(fminf(top[0], top[1]), fminf(top[2], top[3])) * unit;
}

// The weights 2^(v * unit - ref) of 32 logits, in pairs as bf16, and their sum before that rounding.
__device__ __forceinline__ float softmax_weights(uint32_t (&v)[32], float unit, float ref, uint32_t (&w)[16]) {
  const uint64_t unit2 = pack2(unit, unit), ref2 = pack2(-ref, -ref);
  float x[32];
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    unpack2(fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), unit2, ref2), x[c], x[c + 1]);
  }
#pragma unroll
  for (int c = 0; c < 32; ++c) x[c] = exp2_approx(x[c]);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(x[c], x[c + 1]));
    const __nv_bfloat162 e = __floats2bfloat162_rn(x[c], x[c + 1]);
    w[c / 2] = *reinterpret_cast<const uint32_t*>(&e);
  }
  float a, b;
  unpack2(add2(sum[0], sum[1]), a, b);
  return a + b;
}

// Eight e4m3 dims to bf16, times the multiplier.
__device__ __forceinline__ uint4 dequant8(const uint2& x, uint32_t mul) {
  uint4 w;
  kv_dequant4_signs(x.x, mul, w.x, w.y);
  kv_dequant4_signs(x.y, mul, w.z, w.w);
  return w;
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
