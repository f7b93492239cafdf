// The kernel of window and tree attention: a block takes units of up to 64 query rows (a row is one head of one token)
// and some of the tokens that they see, all 512 dims of the values.
#pragma once

#include "paged_attention.cuh"

namespace idx {
namespace block {

// ---------------------------------------------------------------------------
// Per tile of 64 tokens
//   S = Q K^T   64 rows x 64 tokens, 36 steps of K = 16 over the 576 dims
//   P = exp2(S * scale - m)    the running maximum m of each row in registers
//   O += P V    64 rows x 512 dims, 4 steps of K = 16 over the 64 tokens, two halves of N = 256
// with tcgen05.mma.ws (M = 64) in bf16 x bf16 -> fp32, the form and the roles of the sparse attention: warps 4-19 load
// and dequantise the tokens' latents, warps 21-22 copy their position dims and prefetch (22 also finds the next unit and
// copies its Q), warp 20 issues the matrix instructions, warps 0-3 do the softmax; all but 20-22 store the result. Keys
// and values are one copy in shared memory: a token is a row of nine 128-byte swizzled pieces (64 dims each), read along
// the dims as the K-major B operand of S and along the tokens as the N-major one of O. Two groups of eight loader warps
// own a stage each, and hold the next tile in registers.
//
// What differs: tokens lie in pages, so eight of a warp share one block and one address; rows of several query tokens
// see different tokens, so each thread of the softmax has its own mask of a tile; and parts of a context are found on
// the device from the lengths, which the host does not know.
//
// What bounds it: a tile takes some 3000 clocks (1.43 us where few blocks run, 1.54 us with all), the products' 2176
// among them: M = 64 has half of the tensor cores' rate. Shared memory is nearer its limit: 1408 accesses of 128 bytes
// by the tensor core (72 KB of keys, 64 of values, 24 of Q, P twice) and 1140 by the warps (72 KB of keys stored, P, and
// waits of either for the other) are 2550 a tile. With 64 rows one copy of a token serves no more. The chain of a stage
// (store 2000 clocks, S 1200, softmax 1300, O 850, and the other stage's S between) takes what two tiles take. A block's
// first unit starts in some 8000 clocks (lengths, table, first tokens and Q are four round trips), a later one in 4300,
// and a unit ends in some 5000.
// Measured: four chunks of 256 to 512 rows, 128 heads, a window of 1024: 629 us (37 % of the bf16 rate); 64 trees of 4
// to 8 nodes, 64 heads, contexts of 4096 to 8192: 443 us (44 %); one tree of 8 nodes, 128 heads, 32768 tokens: 103 us
// (37 %). Pairs of blocks on one product of M = 256 with half of the values' dims each (full rate, but S twice) took
// 703, 488 and 97 us, and lost more in units that are not full. Copies of Q and position dims by the threads added 1 %
// to the chunks (a 16-byte copy is an access for every 32 bytes), S and O in halves that overlap the stores 2 %, results
// stored by bulk copies 1 %.
// ---------------------------------------------------------------------------
constexpr int kRows = 64;                        // of a unit
constexpr int kQBytes = kPieces * kPieceBytes;
constexpr int kStageBytes = kPieces * kPieceBytes;
constexpr int kStages = 2;
constexpr int kLoaderWarps = 16;
constexpr int kGroupWarps = kLoaderWarps / kStages;  // each stage has its own group of loader warps
constexpr int kTokensPerWarp = kTile / kGroupWarps;
static_assert(kTokensPerWarp == 8, "a loader warp's tokens are eight rows of the swizzle, within one page");
constexpr int kMmaWarp = 4 + kLoaderWarps;
constexpr int kRopeWarp = kMmaWarp + 1;          // one per stage
constexpr int kThreads = (kRopeWarp + kStages) * 32;
constexpr int kOCols = 256;                      // tensor-memory columns of O; S0 and S1 (32 each) follow
constexpr int kQCols = 320;                      // and the first kQTmemPieces pieces of Q
constexpr int kQTmemPieces = 6;
constexpr int kTmemCols = 512;
static_assert(kQCols + kQTmemPieces * 32 <= kTmemCols, "tensor memory of one block");

struct Shared {
  uint64_t q_full, q_free, drained;              // Q is in place; S of the last tile is complete
  uint64_t k_full[kStages];                      // a stage's tokens are stored
  uint64_t s_full[kStages];                      // S of the tile is complete
  uint64_t p_full[kStages];                      // P is stored
  uint64_t o_done[kStages];                      // the tile's share of O is complete: P and the stage are free
  uint32_t tmem;
  volatile uint32_t dead;                        // a wait expired: no further wait blocks
  alignas(8) uint8_t there[kStages][kGroupWarps];   // bit j of byte w: token 8 w + j of the tile is there
  alignas(8) uint8_t poison[kStages][kGroupWarps];  // and not finite
  alignas(8) uint64_t q_here;                    // Q of the next unit: these three live as long as the block
  uint64_t rope_here[kStages];                   // a tile's position dims
  float xchg[2][128];
  float inv[kRows];                              // 1 / sum of each row
  Unit units[2];                                 // this one and the next
  Place place;
};

constexpr int kSmemBytes = kQBytes + kStages * kStageBytes + kPieceBytes + 1024 + static_cast<int>(sizeof(Shared));
static_assert(kSmemBytes <= 232448, "shared memory of one block");

__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 2, %0;" ::"n"(kMmaWarp * 32) : "memory"); }

// The softmax warps and the matrix warp: tensor memory is there (and every row of Q copied).
__device__ __forceinline__ void tmem_bar() { asm volatile("bar.sync 3, 160;" ::: "memory"); }

// The two warps with either half of a tile's tokens for the same 32 rows.
__device__ __forceinline__ void row_bar(int which) { asm volatile("bar.sync %0, 64;" ::"r"(4 + which) : "memory"); }

// Tokens of one copy of position dims: within a page and half a tile.
__host__ __device__ constexpr int copy_tokens_of(int block_size) { return block_size < 32 ? block_size : 32; }

// A copy that was asked for always arrives; should it not, the wait ends all the same, as every other.
__device__ __forceinline__ void wait_copy(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(&g_paged_error, 2u);
      return;
    }
  }
}

// All that a block does for a unit; `started`: barriers and tensor memory are there from an earlier one.
template <bool kTree>
__device__ __forceinline__ void run_unit(const PagedParams& p, const CUtensorMap* rope_map, uint8_t* smem, Shared& sh, int turn,
                                         const Unit& u, bool& started, uint32_t& copies) {
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + kQBytes;
  uint8_t* p_s = k_s + kStages * kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = u.tiles;
  // query row r of the unit: head r % heads of token r / heads
  auto q_row_of = [&](int r) { return r / p.heads; };

  if (tiles == 0) {
    if (u.part >= 0) {
      if (tid < kRows) p.ws_ml[static_cast<int64_t>(u.part) * kRows + tid] = make_float2(-INFINITY, 0.f);
    } else {
      for (int i = tid; i < u.rows * u.heads * (kKvLatent / 8); i += kThreads) {
        const int r = i / (kKvLatent / 8);
        *reinterpret_cast<uint4*>(p.out + (u.row0 + r / u.heads) * p.ld_out + (u.head0 + r % u.heads) * p.ld_oh +
                                  8 * (i % (kKvLatent / 8))) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (p.lse && tid < u.rows * u.heads) p.lse[(u.row0 + tid / u.heads) * p.ld_lse + u.head0 + tid % u.heads] = -INFINITY;
    }
    return;
  }

  // Barriers and tensor memory are set up by the matrix warp; every role first does what needs neither.
  uint32_t tmem = 0;
  auto setup = [&]() {
    tc_fence_before();
    __syncwarp();
    asm volatile("bar.sync 0;" ::: "memory");
    tc_fence_after();
    tmem = sh.tmem;
  };

  if (warp >= 4 && warp < kMmaWarp) {
    // ---------------------------------------------------------------- loaders
    const int group = (warp - 4) / kGroupWarps, lw = (warp - 4) % kGroupWarps;  // this group's tiles: group, group + 2, ...
    const int r0 = kTokensPerWarp * lw;  // the warp's first token of a tile
    // Lane l stores unit l % 8 of piece l / 8 and of piece 4 + l / 8: it holds the eight dims of either half
    // that the swizzle puts there. So the loads' addresses depend on the row, and the stores', which
    // would take registers, do not.
    uint2 raw[kTokensPerWarp][2];
    // A tile's block is looked up one tile of the group before its tokens are loaded, and they two before their
    // conversion: nothing between two tiles' loads waits for an address.
    uint32_t mults = 0, next_codes = 0, found_codes = 0;
    uint32_t there = 0;  // bit j: token j of the found tile is loaded
    const uint8_t* latent = nullptr;  // of the warp's first token
    // of a lane's own token, lane % 8; the warp's tokens that a row sees share one block
    const uint32_t unit_at = smem_u32(&sh.units[turn]);
    auto tokens = [&]() {
      if constexpr (kTree) return u; else return tokens_of(unit_at);
    };
    auto lookup = [&](int tile) {
      if (tile >= tiles) return -1;
      const Unit v = tokens();
      return entry_of(p, v, tile_start(v, tile) + r0 + (lane & 7));
    };
    auto find = [&](int tile, int block) {  // the lane's token is in `block`
      const bool mine = is_block(p, block);
      there = __ballot_sync(0xFFFFFFFFu, mine) & 0xFFu;
      const int blk = there ? __shfl_sync(0xFFFFFFFFu, block, __ffs(there) - 1) : 0;
      found_codes = 0;
      if (there) {
        const int off = (tile_start(tokens(), tile) + r0) & (p.block_size - 1);
        const uint8_t* base = p.cache + blk * p.block_stride;
        latent = base + off * kKvLatent;
        if (mine) {
          found_codes = __ldg(reinterpret_cast<const uint32_t*>(base + p.block_size * kKvScaleAt) + off + (lane & 7));
        }
      }
    };
    auto load = [&]() {
      int own = lane;
      asm volatile("" : "+r"(own));  // eight offsets would take eight registers through the loop
#pragma unroll
      for (int j = 0; j < kTokensPerWarp; ++j) {
        const bool ok = (there >> j) & 1u;
        raw[j][0] = load8_if(latent + kKvLatent * j + 8 * (own ^ j), ok);  // r0 is a multiple of eight: row j of the swizzle
        raw[j][1] = load8_if(latent + kKvLatent * j + 256 + 8 * (own ^ j), ok);
      }
    };
    // eight dims in half h of the token with these multipliers
    auto word_of = [&](int j) { return __shfl_sync(0xFFFFFFFFu, mults, j); };
    auto mul_of = [&](uint32_t word, uint32_t h) { return __byte_perm(word, 0u, 0x4440u + 2 * h + (lane >> 4)) * 0x00800080u; };
    const uint32_t unit = smem_u32(k_s) + group * kStageBytes + (lane >> 3) * kPieceBytes + r0 * 128 + 16 * (lane & 7);

    int next_block;
    uint32_t now;  // `there` of the tile in the registers
    {
      const int here = lookup(group);
      next_block = lookup(group + kStages);
      find(group, here);
      load();
      next_codes = found_codes;
      now = there;
      if (group + kStages < tiles) find(group + kStages, next_block);
      next_block = lookup(group + 2 * kStages);
    }
    if (group >= tiles) setup();
    for (int i = group; i < tiles; i += kStages) {
      mults = multiplier_bytes(next_codes);
      const uint32_t bad = __ballot_sync(0xFFFFFFFFu, mults == 0u) & now;
      // The window form has registers to convert one of a warp's sixteen before the stage is free, with where the unit's
      // tokens lie in shared memory: 626 us for the chunks above instead of 643. Two or more, or any in the tree form, spill
      // (64 trees: 450 us instead of 446).
      constexpr bool kAheadOne = !kTree;
      uint4 ready;
      if (kAheadOne) ready = dequant8(raw[0][0], mul_of(word_of(0), 0));
      if (i >= kStages) wait_for(sh, &sh.o_done[group], ((i >> 1) - 1) & 1);
      if (kAheadOne) st_shared16(unit, ready);
#pragma unroll
      for (int j = 0; j < kTokensPerWarp; ++j) {
        const uint32_t word = word_of(j);
#pragma unroll
        for (int h = kAheadOne && j == 0 ? 1 : 0; h < 2; ++h) {
          st_shared16(unit + 4 * h * kPieceBytes + j * 128, dequant8(raw[j][h], mul_of(word, h)));
        }
      }
      if (lane == 0) {
        // O of tile i - 2, waited for above, was issued once its softmax had read this place
        sh.there[group][lw] = static_cast<uint8_t>(now);
        sh.poison[group][lw] = static_cast<uint8_t>(bad);
      }
      fence_proxy_async_smem();
      if (i == group) setup();  // the first tile is converted while Q is on its way
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[group]);
      if (i + kStages < tiles) {
        load();
        next_codes = found_codes;
        now = there;
        if (i + 2 * kStages < tiles) find(i + 2 * kStages, next_block);
        next_block = lookup(i + 3 * kStages);
      }
    }
  } else if (warp >= kRopeWarp) {
    // ---------------------------------------------------------------- position dims, and L2 prefetch
    // Position dims are bf16 in the cache as in the tile: bulk copies of the tile's pages, as soon as S of the tile
    // before is complete. Tokens that no row sees come along or leave what was there: their scores are not read. Lane l
    // locates tokens l and 32 + l. The same warp reports missing pages, and brings the records of the tile kAhead further on
    // into L2.
    const int group = warp - kRopeWarp;
    auto entry = [&](int tile, int h) { return tile < tiles ? entry_of(p, u, tile_start(u, tile) + 32 * h + lane) : -1; };
    // 32 tokens: each lane's own position dims and codes, and 8 x 4 lines of latents an instruction
    auto prefetch = [&](int tile, int h, int block) {
      if (tile >= tiles) return;
      const int off = (tile_start(u, tile) + 32 * h + lane) & (p.block_size - 1);
      const uint8_t* latent = nullptr;
      if (is_block(p, block)) {
        const uint8_t* base = p.cache + block * p.block_stride;
        latent = base + off * kKvLatent;
        prefetch_l2(base + p.block_size * kKvRopeAt + off * (2 * kKvRope));
        if ((lane & 15) == 0) prefetch_l2(base + p.block_size * kKvScaleAt + 4 * off);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = shfl_ptr(latent, 8 * k + (lane >> 2));
        if (src) prefetch_l2(src + 128 * (lane & 3));
      }
      __syncwarp();
    };
    int here[2], ahead[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      here[h] = entry(group, h);
      ahead[h] = entry(group + kAhead, h);
    }
    const uint32_t piece = smem_u32(k_s) + group * kStageBytes + (kPieces - 1) * kPieceBytes;
    const int copy_tokens = copy_tokens_of(p.block_size);
    if (group >= tiles) setup();
    for (int i = group; i < tiles; i += kStages) {
      // a page, or 32 tokens of one, are a copy, made by the first lane with a token in it
      int block[2];
      uint32_t first[2];
      int copied = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = tile_start(u, i) + 32 * h + lane;
        block[h] = here[h];
        const bool mine = is_block(p, block[h]);
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, mine);
        const uint32_t page = copy_tokens == 32 ? 0xFFFFFFFFu : lane < 16 ? 0xFFFFu : 0xFFFF0000u;
        first[h] = __ballot_sync(0xFFFFFFFFu, mine && lane == __ffs(have & page) - 1);
        copied += __popc(first[h]);
        if (!mine && unit_sees(u, j)) {
          const int node = j - u.base;
          if (!kTree || node < 0 ||
              nodes_seen(p.mask + u.row0 * p.ld_mask, p.ld_mask, p.words, 0, u.rows, 1, node, node + 1)) {
            atomicOr(&g_paged_error, 1u);
          }
        }
        here[h] = entry(i + kStages, h);
      }
      // only S reads position dims, so their piece is free long before the stage is
      if (i >= kStages) wait_for(sh, &sh.s_full[group], ((i >> 1) - 1) & 1);
      if (copied) {
        if (lane == 0) mbar_arrive_expect_tx(&sh.rope_here[group], copied * copy_tokens * (2 * kKvRope));
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if ((first[h] >> lane) & 1u) {
            const int at = 32 * h + (lane & ~(copy_tokens - 1));  // in the tile
            tma_load_3d(piece + at * 128, rope_map, &sh.rope_here[group], 0, (tile_start(u, i) + at) & (p.block_size - 1),
                      block[h]);
          }
        }
      }
      if (i == group) {
        for (int k = group + kStages; k < kAhead && k < tiles; k += kStages) {  // the first tile's are on their way
          prefetch(k, 0, entry(k, 0));
          prefetch(k, 1, entry(k, 1));
        }
        setup();
      }
      if (copied) wait_copy(&sh.rope_here[group], copies++ & 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[group]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        prefetch(i + kAhead, h, ahead[h]);
        ahead[h] = entry(i + kAhead + kStages, h);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      if (started) {
        // nobody waits any more: all warps have passed the last unit's end
        for (uint64_t* bar = &sh.q_full; bar < reinterpret_cast<uint64_t*>(&sh.tmem); ++bar) mbar_inval(bar);
      } else {
        sh.dead = 0;
      }
      mbar_init(&sh.q_full, 4);
      mbar_init(&sh.q_free, 1);
      mbar_init(&sh.drained, 1);
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sh.k_full[i], kGroupWarps + 1);
        mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.p_full[i], 4);
        mbar_init(&sh.o_done[i], 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
    if (!started) {
      tmem_alloc(&sh.tmem, kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    tmem_bar();
    setup();
    // ---------------------------------------------------------------- matrix instructions
    // Whichever of the next S and the next O product has its operands goes first, O before S.
    uint32_t lead;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(lead));
    const uint64_t q_desc = sw128_kmajor_desc(smem_u32(q_s));
    const uint64_t p_desc = sw128_kmajor_desc(smem_u32(p_s));
    const uint64_t k_desc = sw128_kmajor_desc(smem_u32(k_s));
    const uint64_t v_desc = sw128_nmajor_desc(smem_u32(k_s));
    wait_for(sh, &sh.q_full, 0);
    tc_fence_after();
    const int total = __shfl_sync(0xFFFFFFFFu, tiles, 0);
    int s_next = 0, o_next = 0;
    uint64_t t0 = global_timer_ns();
    int idle = 0;
    while (o_next < total) {
      const bool can_o = o_next < s_next && mbar_test(&sh.p_full[o_next & 1], (o_next >> 1) & 1);
      if (__all_sync(0xFFFFFFFFu, can_o)) {
        tc_fence_after();
        const int st = o_next & 1;
        const uint64_t v = v_desc + st * (kStageBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            mma_ws_bf16(tmem + half * (kOCols / 2), p_desc + 2 * ks, v + ((4 * half * kPieceBytes + 2048 * ks) >> 4),
                        idesc_bf16(64, 256, true), o_next > 0 || ks > 0, lead);
          }
        }
        commit_if(&sh.o_done[st], lead);
        ++o_next;
        idle = 0;
        continue;
      }
      const bool can_s = s_next < total && s_next - o_next < kStages &&
                         mbar_test(&sh.k_full[s_next & 1], (s_next >> 1) & 1);
      if (__all_sync(0xFFFFFFFFu, can_s)) {
        tc_fence_after();
        const int st = s_next & 1;
        const uint64_t k = k_desc + st * (kStageBytes >> 4);
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t b = k + ((c * kPieceBytes) >> 4) + 2 * ks;
            if (c < kQTmemPieces) {
              mma_ws_bf16_ta(tmem + kOCols + st * 32, tmem + kQCols + 32 * c + 8 * ks, b, idesc_bf16(64, 64, false),
                             c > 0 || ks > 0, lead);
            } else {
              mma_ws_bf16(tmem + kOCols + st * 32, q_desc + ((c * kPieceBytes) >> 4) + 2 * ks, b,
                          idesc_bf16(64, 64, false), 1, lead);
            }
          }
        }
        commit_if(&sh.s_full[st], lead);
        if (++s_next == total) commit_if(&sh.q_free, lead);
        idle = 0;
        continue;
      }
      // nothing was ready: the limit of two seconds runs from the first such pass
      if (idle++ == 0) t0 = global_timer_ns();
      bool expired = sh.dead != 0;
      if (!expired && (idle & 63) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
        expired = true;
        atomicOr(&g_paged_error, 2u);
        sh.dead = 1;
      }
      if (__any_sync(0xFFFFFFFFu, expired)) break;
    }
    if (o_next < total) {  // given up: whatever was issued finishes before the tensor memory is freed
      commit_if(&sh.drained, lead);
      t0 = global_timer_ns();
      while (!mbar_test(&sh.drained, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- softmax
    // Q was copied by the warp that found the unit; rows past its last one hold anything, and give results that nobody
    // reads. As many pieces as there are columns go into tensor memory: S reads less of the shared memory that the loaders
    // and O want too.
    wait_copy(&sh.q_here, copies & 1);
    ++copies;
    tmem_bar();
    tc_fence_after();
    tmem = sh.tmem;
    const int r = tid & 63, half = tid >> 6;          // row of the unit, and half of the tile's tokens
    const int t = q_row_of(r), h = r - t * p.heads;
    const bool have = t < u.rows && h < u.heads;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t own_row = smem_u32(q_s) + r * 128;
#pragma unroll 2
    for (int x = 0; x < 8 * kQTmemPieces; x += 4) {
      uint32_t w[16];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint4 v = ld_shared16(own_row + (x >> 3) * kPieceBytes + ((((x + y) & 7) ^ (r & 7)) << 4));
        w[4 * y] = v.x;
        w[4 * y + 1] = v.y;
        w[4 * y + 2] = v.z;
        w[4 * y + 3] = v.w;
      }
      tmem_st16(lanes + kQCols + 4 * x, w);
    }
    tmem_wait_st();
    setup();
    auto arrive = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    arrive(&sh.q_full);

    const int2 all = all_seen<kTree>(p, u, have, t);
    float m = -INFINITY, l = 0.f;                     // maximum (log2 units) that P and O refer to; this half's sum
    bool poisoned = false;                            // the row sees a token that is not finite
    for (int i = 0; i < tiles; ++i) {
      const int st = i & 1;
      const int x = tile_start(u, i) + 32 * half;
      uint32_t seen = 0xFFFFFFFFu;
      if (x < all.x || x + 31 > all.y) seen = have ? row_sees<kTree>(p, u, t, x) : 0u;
      wait_for(sh, &sh.s_full[st], (i >> 1) & 1);
      wait_for(sh, &sh.k_full[st], (i >> 1) & 1);  // long complete: `there` is written
      tc_fence_after();
      uint32_t v[32];
      tmem_ld_x32(lanes + kOCols + st * 32, v);
      seen &= *reinterpret_cast<const uint32_t*>(&sh.there[st][4 * half]);
      const uint32_t bad = *reinterpret_cast<const uint32_t*>(&sh.poison[st][4 * half]);
      poisoned |= (seen & bad) != 0u;
      seen &= ~bad;
      tmem_wait_ld(v);
      // v * unit is the logit in log2 units: the raw products as they are where every token counts, or
      // scaled here with -inf for the others
      float unit = p.scale_log2;
      if (seen != 0xFFFFFFFFu) {
        unit = 1.0f;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          v[c] = (seen >> c) & 1u ? __float_as_uint(__uint_as_float(v[c]) * p.scale_log2) : 0xFF800000u;
        }
      }
      float top = softmax_top(v, unit);
      sh.xchg[st][tid] = top;
      row_bar(warp & 1);
      top = fmaxf(top, sh.xchg[st][tid ^ 64]);
      // P and O keep an old reference until the maximum has risen by 2^40, so hardly a tile rescales O
      const bool rise = top > m + kRescaleStep || (m == -INFINITY && top > -INFINITY);
      const float m_new = rise ? top : m;
      if (i > 0) {
        // O is complete up to the last tile (for a rescaling), and with it the only P is free
        const float f = rise && m != -INFINITY ? exp2_approx(m - m_new) : 1.0f;  // without a reference, l and O are 0
        const bool scale_o = __any_sync(0xFFFFFFFFu, f != 1.0f);
        wait_for(sh, &sh.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
        if (scale_o) {
          tc_fence_after();
          l *= f;
#pragma unroll 1
          for (int c = 0; c < kOCols; c += 16) {
            uint32_t o[16];
            tmem_ld16(lanes + c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(lanes + c, o);
          }
          tmem_wait_st();
        }
      }
      m = m_new;
      // The weights are rounded to bf16 for the product: its operands have one type, and bf16 is the one that holds every
      // token exactly. l sums them unrounded, so lse keeps its 32 bits.
      const float ref = m == -INFINITY ? 0.f : m;
      uint32_t w[16];
      l += softmax_weights(v, unit, ref, w);
      const uint32_t p_row = smem_u32(p_s) + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        st_shared16(p_row + (((4 * half + c) ^ (r & 7)) << 4), make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
      }
      arrive(&sh.p_full[st]);
    }
    if (poisoned) l = __int_as_float(0x7FC00000);
    row_bar(warp & 1);
    sh.xchg[0][tid] = l;
    row_bar(warp & 1);
    l += sh.xchg[0][tid ^ 64];
    if (half == 0) {
      const bool split = u.part >= 0;
      sh.inv[r] = split ? 1.0f : l == 0.f ? 0.f : 1.0f / l;
      if (split) {
        p.ws_ml[static_cast<int64_t>(u.part) * kRows + r] = make_float2(m, l);
      } else if (p.lse && have) {
        p.lse[(u.row0 + t) * p.ld_lse + u.head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      }
    }
  }
  if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- epilogue
    // The loaders, four to a lane quarter and 64 columns each, write O (bf16, or the sums of a part) into the
    // stages' memory, a row of it per query row, and all warps store whole rows.
    constexpr int kPitchBf16 = kKvLatent * 2 + 16, kPitchF32 = kKvLatent * 4 + 16;  // eight rows' stores fall into different banks
    static_assert(kRows * kPitchF32 <= kStages * kStageBytes, "the rows fit the stages");
    // Only the softmax warps may wait for the last O by its parity: they have followed every phase of both o_done
    // barriers. The loader warps are ordered behind O by the block barrier and the fences around it.
    if (warp < 4) {
      wait_for(sh, &sh.o_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);
      tc_fence_after();
      tc_fence_before();
    }
    epilogue_bar();
    tc_fence_after();
    const volatile Unit& e = sh.units[turn];
    const bool split = e.part >= 0;
    tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    if (warp >= 4) {
      const int quarter = warp & 3, r = (32 * quarter + lane) & 63, half = quarter >> 1;
      const float inv = sh.inv[r];
#pragma unroll 1
      for (int c = 64 * ((warp - 4) >> 2); c < 64 * ((warp - 4) >> 2) + 64; c += 32) {
        uint32_t o[32];
        tmem_ld_x32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + c, o);
        tmem_wait_ld(o);
        // A product has 256 dims, 128 to each lane half.
        const int dim = (c / 128) * 256 + half * 128 + (c % 128);
        if (split) {
          const uint32_t at = smem_u32(k_s) + r * kPitchF32 + dim * 4;
#pragma unroll
          for (int j = 0; j < 8; ++j) st_shared16(at + 16 * j, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        } else {
          const uint32_t at = smem_u32(k_s) + r * kPitchBf16 + dim * 2;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[8 * j + 2 * x]) * inv,
                                                             __uint_as_float(o[8 * j + 2 * x + 1]) * inv);
              w[x] = *reinterpret_cast<const uint32_t*>(&b);
            }
            st_shared16(at + 16 * j, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
    }
    epilogue_bar();
    // a warp stores a row at a time
    const int rows = e.rows * p.heads, row0 = e.row0, heads = e.heads, head0 = e.head0, part = e.part;
    for (int r = warp; r < rows; r += kMmaWarp) {
      const int t = q_row_of(r), h = r - t * p.heads;
      if (h >= heads) continue;
      const uint32_t from = smem_u32(k_s) + 16 * lane;
      if (split) {
        float* dst = p.ws_o + (static_cast<int64_t>(part) * kRows + r) * kKvLatent + 4 * lane;
#pragma unroll
        for (int x = 0; x < kKvLatent / 128; ++x) {
          *reinterpret_cast<uint4*>(dst + 128 * x) = ld_shared16(from + r * kPitchF32 + 512 * x);
        }
      } else {
        __nv_bfloat16* dst = p.out + (row0 + t) * p.ld_out + (head0 + h) * p.ld_oh + 8 * lane;
#pragma unroll
        for (int x = 0; x < kKvLatent / 256; ++x) {
          *reinterpret_cast<uint4*>(dst + 256 * x) = ld_shared16(from + r * kPitchBf16 + 512 * x);
        }
      }
    }
  }
  started = true;
}

// The next unit, found by one warp, and its Q, copied once S of the last tile has left the place.
template <bool kTree>
__device__ __forceinline__ void prepare_unit(const PagedParams& p, const CUtensorMap* q_map, uint8_t* smem, Shared& sh, int turn,
                                             bool first, bool busy) {
  Unit& next = sh.units[turn];
  find_next<kTree>(p, blockIdx.x, first, sh.place, next);
  __syncwarp();
  if (!next.any || next.tiles == 0) return;
  if (busy) wait_for(sh, &sh.q_free, 0);
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_arrive_expect_tx(&sh.q_here, kPieces * p.heads * p.tokens * 128);
  __syncwarp();
  if (lane < kPieces) tma_load_3d(smem_u32(smem) + lane * kPieceBytes, q_map, &sh.q_here, 64 * lane, next.head0, next.row0);
}

template <bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
paged_block_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap rope_map, const PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Shared& sh = *reinterpret_cast<Shared*>(smem + kQBytes + kStages * kStageBytes + kPieceBytes);

  if (p.cut) asm volatile("griddepcontrol.launch_dependents;");  // the join may be set up meanwhile
  const bool finder = threadIdx.x / 32 == kThreads / 32 - 1;
  if (finder && (threadIdx.x & 31) == 0) {
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&rope_map);
    mbar_init(&sh.q_here, 1);
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.rope_here[i], 1);
    fence_mbar_init();
  }
  bool started = false;   // barriers and tensor memory are there
  uint32_t copies = 0;    // that the warp has waited for: Q, or a stage's position dims
  for (int turn = 1, first = 1;; turn ^= 1, first = 0) {
    bool busy = false;
    if (!first) {
      const Unit u = sh.units[turn];
      if (!u.any) break;
      busy = u.tiles > 0;
      run_unit<kTree>(p, &rope_map, smem, sh, turn, u, started, copies);
    }
    // the last tiles' position dims are copied: this warp finds the next unit while the others finish theirs
    if (finder) prepare_unit<kTree>(p, &q_map, smem, sh, turn ^ 1, first, busy);
    fence_proxy_async_smem();  // the stages held results, and take copies again
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
  }
  if (started && threadIdx.x / 32 == kMmaWarp) tmem_dealloc(sh.tmem, kTmemCols);
}

}  // namespace block
}  // namespace idx
