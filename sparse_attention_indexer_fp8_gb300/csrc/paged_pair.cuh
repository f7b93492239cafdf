// Window and tree attention of many rows a request: a pair of blocks (a cluster of two) per unit of up to
// 256 query rows (a row is one head of one token) and half of the value dims.
#pragma once

#include "paged_attention.cuh"

namespace idx {
namespace pair {

// ---------------------------------------------------------------------------
// Per tile of 64 tokens, each block of the pair with 128 of the rows:
//   S = Q K^T   256 rows x 64 tokens, 36 steps of K = 16 over the 576 dims
//   P = exp2(S * scale - m)    the running maximum m of each row in registers
//   O += P V    256 rows x 256 dims, 4 steps of K = 16 over the 64 tokens
// with tcgen05.mma.cta_group::2 (M = 256) in bf16 x bf16 -> fp32, issued by the first block for both.
//
// Why this form. 128 rows a block fill the lanes of tensor memory, and then 512 dims of O in fp32 fill its columns
// and leave none for S. So a unit has 256 of the dims, and S is computed for either half: 832 multiplications a
// row and token instead of 544 (x 2), at the full rate. (64 rows a block with all dims, the other form that fits, run
// at half the rate, and dequantise every token twice as often.) With two blocks on one product each keeps half of
// the B operand: of a tile the keys of 32 tokens and 128 value dims of all 64, so a block dequantises 20480 values a
// tile instead of 32768 and reads half as much of shared memory for B.
//
// Tensor memory: O 256 columns, S of two tiles 128, four of the nine pieces (64 dims) of Q 128. Shared memory: the rest
// of Q 80 KB, keys of two tiles (36 KB each), values of three (16 KB), P 16 KB.
//
// Roles: warps 0-7 do the softmax (row and half of the tile's tokens a thread), 8-23 load and dequantise, in two
// groups that take turns, 24 issues the matrix instructions (in the first block), 25-26 copy position dims and prefetch.
// ---------------------------------------------------------------------------
constexpr int kRows = 256;                       // of a unit
constexpr int kBlockRows = 128;
constexpr int kHalves = 2;
constexpr int kDims = kKvLatent / kHalves;       // of a unit's values
constexpr int kOwn = kTile / 2;                  // tokens of a tile whose keys a block holds
constexpr int kStages = 2;                       // of keys and S
constexpr int kValueStages = 3;
constexpr int kRing = 4;
constexpr int kKeyPiece = kOwn * 128;
constexpr int kKeyBytes = kPieces * kKeyPiece;
constexpr int kValuePieces = kDims / 2 / 64;     // of a block
constexpr int kValueBytes = kValuePieces * kPieceBytes;
constexpr int kQTmemPieces = 4;
constexpr int kQPiece = kBlockRows * 128;
constexpr int kQBytes = (kPieces - kQTmemPieces) * kQPiece;
constexpr int kPBytes = kBlockRows * 128;
constexpr int kSoftmaxWarps = 8;
constexpr int kLoaderWarps = 16;
constexpr int kGroups = 2;                       // of loader warps
constexpr int kGroupWarps = kLoaderWarps / kGroups;
constexpr int kPerWarp = kOwn / kGroupWarps;     // tokens of a warp: this many own ones, and as many of the other block's
static_assert(kPerWarp == 4, "a loader warp's own tokens are half of the swizzle's rows, within one page");
constexpr int kFirstLoader = kSoftmaxWarps;
constexpr int kMmaWarp = kFirstLoader + kLoaderWarps;
constexpr int kRopeWarp = kMmaWarp + 1;
constexpr int kThreads = (kRopeWarp + kGroups) * 32;
constexpr int kSCol = 256;                       // tensor-memory columns: O, S, Q
constexpr int kQCol = kSCol + kStages * kTile;
constexpr int kTmemCols = 512;
static_assert(kQCol + kQTmemPieces * 32 <= kTmemCols, "tensor memory of one block");

struct Shared {
  // waited for by the first block's matrix warp; both blocks' warps arrive
  uint64_t k_full[kStages];                      // a tile's keys and values are stored
  uint64_t s_free[kStages];                      // S is in registers
  uint64_t p_full;                               // P is stored
  // of either block; the matrix instructions arrive
  uint64_t s_full[kStages];                      // S of the tile is complete: the keys are free
  uint64_t o_done[kValueStages];                 // the tile's share of O is complete: P and the values are free
  uint64_t drained;
  uint64_t flags[kRing];                         // `there` is written
  uint32_t tmem;
  volatile uint32_t dead;                        // a wait expired: no further wait blocks
  alignas(16) uint8_t there[kRing][kTile / 4]; // of four tokens each: low bits, the token is there; high, and not finite
  float xchg[2][2 * kBlockRows];
  float inv[kBlockRows];                         // 1 / sum of each row
  Unit unit;
  Place place;
};

constexpr int kSmemBytes =
    kQBytes + kStages * kKeyBytes + kValueStages * kValueBytes + kPBytes + 1024 + static_cast<int>(sizeof(Shared));
static_assert(kSmemBytes <= 232448, "shared memory of one block");

// Issued by the lane with `issue` set, for both blocks; the warp passes converged.
__device__ __forceinline__ void mma2_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                          uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc),
      "r"(issue)
      : "memory");
}

// The same with A in either block's tensor memory.
__device__ __forceinline__ void mma2_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                             uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc),
      "r"(issue)
      : "memory");
}

// Arrives on the barrier of both blocks once everything issued so far is complete.
__device__ __forceinline__ void commit2(uint64_t* bar, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "mov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(issue)
      : "memory");
}

__device__ __forceinline__ uint32_t first_block_addr(const void* ptr) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(ptr)));
  return a;
}

// Arrives on the first block's barrier. What it announces was written to this block's own shared or tensor memory for
// the tensor core of this SM, and the fences before it have made it visible there.
__device__ __forceinline__ void arrive_first(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The two warps that share a row of tensor-memory lanes: either half of a tile's tokens for the same 32 rows.
__device__ __forceinline__ void row_bar(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(4 + quarter) : "memory"); }

// The softmax warps and the matrix warp: tensor memory is there.
__device__ __forceinline__ void tmem_bar() { asm volatile("bar.sync 3, %0;" ::"n"(kSoftmaxWarps * 32 + 32) : "memory"); }

__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 2, %0;" ::"n"(kMmaWarp * 32) : "memory"); }

template <bool kTree>
__global__ void __launch_bounds__(kThreads, 1) paged_pair_kernel(const PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + kQBytes;
  uint8_t* v_s = k_s + kStages * kKeyBytes;
  uint8_t* p_s = v_s + kValueStages * kValueBytes;
  Shared& sh = *reinterpret_cast<Shared*>(p_s + kPBytes);

  if (p.workers) asm volatile("griddepcontrol.launch_dependents;");  // the join may be set up meanwhile
  bool started = false;
  for (bool first = true;; first = false) {
  const Unit u = fetch_unit<kTree, kHalves>(p, sh, blockIdx.x / 2, first, cluster_rank() == 0);
  if (!u.any) break;
  const int tid = thread_number(), warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int tiles = u.tiles;
  // row r of the block: head r % heads of token first_token + r / heads
  const int first_token = rank * (p.tokens / 2);
  const int64_t part_row = static_cast<int64_t>(u.part) * kRows + rank * kBlockRows;

  if (tiles == 0) {
    if (u.part >= 0) {
      if (tid < kBlockRows) p.ws_ml[part_row + tid] = make_float2(-INFINITY, 0.f);
    } else {
      const int rows = max(min(u.rows - first_token, p.tokens / 2), 0) * u.heads;
      for (int i = tid; i < rows * (kDims / 8); i += kThreads) {
        const int r = i / (kDims / 8);
        *reinterpret_cast<uint4*>(p.out + (u.row0 + first_token + r / u.heads) * p.ld_out +
                                  (u.head0 + r % u.heads) * p.ld_oh + u.half * kDims + 8 * (i % (kDims / 8))) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      if (p.lse && u.half == 0 && tid < rows) {
        p.lse[(u.row0 + first_token + tid / u.heads) * p.ld_lse + u.head0 + tid % u.heads] = -INFINITY;
      }
    }
    __syncthreads();
    continue;
  }

  // Barriers and tensor memory are set up by the matrix warp; every role first does what needs neither. Both blocks'
  // barriers exist behind it, and Q is in its place.
  uint32_t tmem = 0;
  auto setup = [&]() {
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    tmem = sh.tmem;
  };

  if (warp >= kFirstLoader && warp < kMmaWarp) {
    // ---------------------------------------------------------------- loaders
    const int group = (warp - kFirstLoader) / kGroupWarps, lw = (warp - kFirstLoader) % kGroupWarps;
    const int r0 = kPerWarp * lw;                          // the warp's first row of the keys
    const int own_at = rank * kOwn + r0, other_at = (rank ^ 1) * kOwn + r0;  // and its tokens of the tile
    const int which = lane & 7;                            // lanes 0-3 locate the own tokens, 4-7 the other's
    const int mine = which < kPerWarp ? own_at + which : other_at + which - kPerWarp;
    uint2 raw[kPerWarp][2];    // eight dims in either half of each own token
    uint2 raw_other[2];        // eight of the block's value dims of tokens 0, 1 (by half warp) and 2, 3
    uint32_t mults = 0, next_codes = 0, found_codes = 0;
    uint32_t there = 0;        // bit j: token j of the found tile is loaded
    const uint8_t *own = nullptr, *other = nullptr;  // the first own token's latent; the lane's values of tokens 0, 1
    auto lookup = [&](int tile) { return tile < tiles ? entry_of(p, u, tile_start(u, tile) + mine) : -1; };
    const uint32_t value_at = kDims * u.half + kDims / 2 * rank;  // bytes into a latent
    auto find = [&](int tile, int block) {  // the lane's token is in `block`
      there = __ballot_sync(0xFFFFFFFFu, is_block(p, block)) & 0xFFu;
      const int x = tile_start(u, tile);
      const uint32_t low = there & 0xFu, high = there >> 4;
      if (low) {
        const int blk = __shfl_sync(0xFFFFFFFFu, block, __ffs(low) - 1);
        own = p.cache + blk * p.block_stride + ((x + own_at) & (p.block_size - 1)) * kKvLatent;
      }
      if (high) {
        const int blk = __shfl_sync(0xFFFFFFFFu, block, __ffs(high) + 3);
        other = p.cache + blk * p.block_stride + ((x + other_at) & (p.block_size - 1)) * kKvLatent + value_at;
      }
      found_codes = 0;
      if (is_block(p, block)) {
        const uint8_t* base = p.cache + block * p.block_stride + p.block_size * kKvScaleAt;
        found_codes = __ldg(reinterpret_cast<const uint32_t*>(base) + ((x + mine) & (p.block_size - 1)));
      }
    };
    // Lane l stores unit l % 8 of a piece: it holds the eight dims that the swizzle puts there. So the loads'
    // addresses depend on the row, and the stores' do not.
    const int swizzle = r0 & 7;  // of the warp's first token, 0 or 4
    auto load = [&]() {
#pragma unroll
      for (int j = 0; j < kPerWarp; ++j) {
        const bool ok = (there >> j) & 1u;
        const uint8_t* src = own + kKvLatent * j + 8 * (lane ^ (swizzle | j));
        raw[j][0] = load8_if(src, ok);
        raw[j][1] = load8_if(src + 256, ok);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = 2 * k + (lane >> 4);
        raw_other[k] = load8_if(other + kKvLatent * j + 8 * ((lane & 15) ^ (swizzle | j)), (there >> (4 + j)) & 1u);
      }
    };
    const uint32_t keys = smem_u32(k_s) + group * kKeyBytes + (lane >> 3) * kKeyPiece + r0 * 128 + 16 * (lane & 7);
    // the lanes that hold own tokens' value dims, and where those and the others' go
    const bool value_lane = (lane >> 4) == rank;
    const uint32_t values = smem_u32(v_s) + ((lane >> 3) & 1) * kPieceBytes + 16 * (lane & 7);
    const uint32_t own_values = values + own_at * 128, other_values = values + (other_at + (lane >> 4)) * 128;
    const uint32_t k_bar = first_block_addr(&sh.k_full[group]);

    uint32_t now = 0;  // `there` of the tile in the registers
    int v_st = group;
    int next_block = -1;
    {
      const int here = lookup(group);
      next_block = lookup(group + kGroups);
      find(group, here);
      load();
      next_codes = found_codes;
      now = there;
      if (group + kGroups < tiles) find(group + kGroups, next_block);
      next_block = lookup(group + 2 * kGroups);
    }
    setup();
    for (int i = group; i < tiles; i += kGroups) {
      mults = multiplier_bytes(next_codes);
      const uint32_t bad = __ballot_sync(0xFFFFFFFFu, mults == 0u) & now;
      if (i >= kStages) wait_for(sh, &sh.s_full[group], ((i >> 1) - 1) & 1);
      // Of the values' stage, which the groups take in turn, a wait by parity needs the barrier to be in the phase of tile
      // i - 3 or the next. It is not further: that is this tile's. It is not before: of the group's last tile, O of i - 5 was
      // waited for, which was issued after the softmax had seen O of i - 6 complete.
      if (i >= kValueStages) wait_for(sh, &sh.o_done[v_st], (i / kValueStages - 1) & 1);
      const uint32_t v_off = v_st * kValueBytes;
#pragma unroll
      for (int j = 0; j < kPerWarp; ++j) {
        const uint32_t word = __shfl_sync(0xFFFFFFFFu, mults, j);
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[h] = dequant8(raw[j][h], __byte_perm(word, 0u, 0x4440u + 2 * h + (lane >> 4)) * 0x00800080u);
          st_shared16(keys + 4 * h * kKeyPiece + j * 128, w[h]);
        }
        if (value_lane) st_shared16(own_values + v_off + j * 128, u.half ? w[1] : w[0]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t word = __shfl_sync(0xFFFFFFFFu, mults, kPerWarp + 2 * k + (lane >> 4));
        st_shared16(other_values + v_off + 2 * k * 128,
                    dequant8(raw_other[k], __byte_perm(word, 0u, 0x4440u + 2 * u.half + rank) * 0x00800080u));
      }
      if (lane == 0) {
        // S of tile i - 2 is complete; it was issued once the softmax of tile i - 4 had read this place
        sh.there[i % kRing][own_at / 4] = static_cast<uint8_t>((now & 0xFu) | ((bad & 0xFu) << 4));
        sh.there[i % kRing][other_at / 4] = static_cast<uint8_t>((now >> 4) | (bad & 0xF0u));
        mbar_arrive(&sh.flags[i % kRing]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_first(k_bar);
      v_st = v_st == 0 ? 2 : v_st - 1;  // of tile i + 2
      if (i + kGroups < tiles) {
        load();
        next_codes = found_codes;
        now = there;
      }
      if (i + 2 * kGroups < tiles) find(i + 2 * kGroups, next_block);
      next_block = lookup(i + 3 * kGroups);
    }
  } else if (warp >= kRopeWarp) {
    // ---------------------------------------------------------------- position dims, and L2 prefetch
    // Position dims are bf16 in the cache as in the keys: copied asynchronously. Lane l locates the block's
    // token l. The same warp brings the records of the tile kAhead further on into L2; the other block
    // does the same with the other tokens.
    const int mine = rank * kOwn + lane;
    auto entry = [&](int tile) { return tile < tiles ? entry_of(p, u, tile_start(u, tile) + mine) : -1; };
    auto prefetch = [&](int tile, int blk) {
      if (tile >= tiles) return;
      const int off = (tile_start(u, tile) + mine) & (p.block_size - 1);
      const uint8_t* latent = nullptr;
      if (is_block(p, blk)) {
        const uint8_t* base = p.cache + blk * p.block_stride;
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
    const int group = warp - kRopeWarp;
    int here = entry(group), ahead = entry(group + kAhead);
    for (int i = group; i < kAhead && i < tiles; i += kGroups) prefetch(i, entry(i));
    const uint32_t k_bar = first_block_addr(&sh.k_full[group]);
    const uint32_t piece = smem_u32(k_s) + group * kKeyBytes + (kPieces - 1) * kKeyPiece;
    setup();
    for (int i = group; i < tiles; i += kGroups) {
      const int j = tile_start(u, i) + mine;
      const uint8_t* rope = nullptr;
      if (is_block(p, here)) {
        rope = p.cache + here * p.block_stride + p.block_size * kKvRopeAt + (j & (p.block_size - 1)) * (2 * kKvRope);
      } else if (unit_sees(u, j)) {
        atomicOr(&g_paged_error, 1u);
      }
      here = entry(i + kGroups);
      if (i >= kStages) wait_for(sh, &sh.s_full[group], ((i >> 1) - 1) & 1);
#pragma unroll
      for (int c = 0; c < kOwn / 4; ++c) {
        const int t = 4 * c + (lane >> 3), x = lane & 7;
        const uint8_t* from = shfl_ptr(rope, t);
        copy16_if(piece + t * 128 + ((x ^ (t & 7)) << 4), from ? from + 16 * x : p.cache, from != nullptr);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_first(k_bar);
      prefetch(i + kAhead, ahead);
      ahead = entry(i + kAhead + kGroups);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      if (started) {
        // nobody waits or arrives any more: all warps of both blocks have passed the last unit's end
        for (uint64_t* bar = &sh.k_full[0]; bar < reinterpret_cast<uint64_t*>(&sh.tmem); ++bar) mbar_inval(bar);
      } else {
        sh.dead = 0;
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sh.k_full[i], 2 * (kGroupWarps + 1));
        mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.s_free[i], 2 * kSoftmaxWarps);
      }
      for (int i = 0; i < kValueStages; ++i) mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.p_full, 2 * kSoftmaxWarps);
      for (int i = 0; i < kRing; ++i) mbar_init(&sh.flags[i], kGroupWarps);
      mbar_init(&sh.drained, 1);
      fence_mbar_init();
    }
    __syncwarp();
    if (!started) asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                 "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(&sh.tmem)), "r"(kTmemCols)
                 : "memory");
    tc_fence_before();
    tmem_bar();
    setup();
    if (rank == 0) {
      // -------------------------------------------------------------- matrix instructions
      uint32_t lead;
      asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(lead));
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(q_s));
      const uint64_t p_desc = sw128_kmajor_desc(smem_u32(p_s));
      const uint64_t k_desc = sw128_kmajor_desc(smem_u32(k_s));
      const uint64_t v_desc = sw128_nmajor_desc(smem_u32(v_s));
      const int total = __shfl_sync(0xFFFFFFFFu, tiles, 0);
      // Whichever of the next S and the next O product has its operands goes first, O before S.
      int s_next = 0, o_next = 0, o_st = 0;
      uint64_t t0 = global_timer_ns();
      int idle = 0;
      while (o_next < total) {
        if (o_next < s_next && __all_sync(0xFFFFFFFFu, mbar_test(&sh.p_full, o_next & 1))) {
          tc_fence_after();
          const uint64_t v = v_desc + o_st * (kValueBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            mma2_bf16(tmem, p_desc + 2 * ks, v + ((2048 * ks) >> 4), idesc_bf16(kRows, kDims, true), o_next > 0 || ks > 0,
                      lead);
          }
          commit2(&sh.o_done[o_st], lead);
          ++o_next;
          if (++o_st == kValueStages) o_st = 0;
          idle = 0;
          continue;
        }
        const int st = s_next & 1;
        const uint32_t par = (s_next >> 1) & 1;
        if (s_next < total && __all_sync(0xFFFFFFFFu, mbar_test(&sh.k_full[st], par) &&
                                                          (s_next < kStages || mbar_test(&sh.s_free[st], par ^ 1u)))) {
          tc_fence_after();
          const uint64_t k = k_desc + st * (kKeyBytes >> 4);
          const uint32_t s = tmem + kSCol + st * kTile;
#pragma unroll
          for (int c = 0; c < kPieces; ++c) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint64_t b = k + ((c * kKeyPiece) >> 4) + 2 * ks;
              if (c < kQTmemPieces) {
                mma2_bf16_ta(s, tmem + kQCol + 32 * c + 8 * ks, b, idesc_bf16(kRows, kTile, false), c > 0 || ks > 0, lead);
              } else {
                mma2_bf16(s, q_desc + (((c - kQTmemPieces) * kQPiece) >> 4) + 2 * ks, b, idesc_bf16(kRows, kTile, false), 1,
                          lead);
              }
            }
          }
          commit2(&sh.s_full[st], lead);
          ++s_next;
          idle = 0;
          continue;
        }
        // nothing was ready: the limit of two seconds runs from the first such pass
        if (idle++ == 0) t0 = global_timer_ns();
        __nanosleep(32);  // the other warps of the scheduler need its slots
        bool expired = sh.dead != 0;
        if (!expired && (idle & 63) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
          expired = true;
          atomicOr(&g_paged_error, 2u);
          sh.dead = 1;
        }
        if (__any_sync(0xFFFFFFFFu, expired)) break;
      }
      if (o_next < total) {  // given up: whatever was issued finishes before the tensor memory is freed
        commit2(&sh.drained, lead);
        t0 = global_timer_ns();
        while (!mbar_test(&sh.drained, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
        __syncwarp();
      }
    }
  } else if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax
    const int quarter = warp & 3, half = warp >> 2;  // lanes of tensor memory, half of the tile's tokens
    const int r = 32 * quarter + lane;
    const int t = first_token + r / p.heads, h = r % p.heads;
    const bool have = r / p.heads < p.tokens / 2 && t < u.rows && h < u.heads;
    // Q, sixteen rows a warp, rows past the unit's last one zero, all copies out at once: the pieces for tensor memory
    // into the keys' place for now. Lane l < 16 finds row l.
    {
      const int qr = kBlockRows / kSoftmaxWarps * warp + (lane & 15), qt = qr / p.heads, qh = qr - qt * p.heads;
      const bool in = qt < p.tokens / 2 && first_token + qt < u.rows && qh < u.heads;
      const uint8_t* src = in ? reinterpret_cast<const uint8_t*>(p.q + (u.row0 + first_token + qt) * p.ld_q + (u.head0 + qh) * p.ld_qh)
                              : nullptr;
      const uint32_t to = (lane >> 3) * kQPiece + kBlockRows / kSoftmaxWarps * warp * 128;
#pragma unroll 4
      for (int x = 0; x < kBlockRows / kSoftmaxWarps; ++x) {
        const uint8_t* row = shfl_ptr(src, x);
        const bool have_row = row != nullptr;
        const uint8_t* from = (have_row ? row : reinterpret_cast<const uint8_t*>(p.q)) + 16 * lane;
        const uint32_t at = to + x * 128 + (((lane & 7) ^ (x & 7)) << 4);
        copy16_if(smem_u32(k_s) + at, from, have_row);
        copy16_if(smem_u32(q_s) + at, from + 512, have_row);
        if (lane < 8) copy16_if(smem_u32(q_s) + 4 * kQPiece + at, from + 1024, have_row);
      }
    }
    static_assert(kQTmemPieces == 4, "half of the latent pieces");
    asm volatile("cp.async.wait_all;" ::: "memory");
    tmem_bar();
    tc_fence_after();
    tmem = sh.tmem;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll 2
    for (int x = 16 * half; x < 16 * half + 16; x += 4) {  // either thread of a row half of its units
      uint32_t w[16];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint4 v = ld_shared16(smem_u32(k_s) + ((x + y) >> 3) * kQPiece + r * 128 + ((((x + y) & 7) ^ (r & 7)) << 4));
        w[4 * y] = v.x;
        w[4 * y + 1] = v.y;
        w[4 * y + 2] = v.z;
        w[4 * y + 3] = v.w;
      }
      tmem_st16(lanes + kQCol + 4 * x, w);
    }
    tmem_wait_st();
    fence_proxy_async_smem();
    const uint32_t s_free = first_block_addr(&sh.s_free[0]), p_full = first_block_addr(&sh.p_full);
    setup();

    const int2 all = all_seen<kTree>(p, u, have, t);
    float m = -INFINITY, l = 0.f;                     // maximum (log2 units) that P and O refer to; this half's sum
    bool poisoned = false;                            // the row sees a token that is not finite
    int last = kValueStages - 1;                      // stage of the last tile's values
    uint32_t last_par = 1;
    for (int i = 0; i < tiles; ++i) {
      const int st = i & 1;
      const uint32_t par = (i >> 1) & 1;
      const int x = tile_start(u, i) + 32 * half;
      uint32_t seen = 0xFFFFFFFFu;
      if (x < all.x || x + 31 > all.y) seen = have ? row_sees<kTree>(p, u, t, x) : 0u;
      wait_for(sh, &sh.s_full[st], par);
      tc_fence_after();
      uint32_t v[32];
      tmem_ld_x32(lanes + kSCol + st * kTile + 32 * half, v);
      wait_for(sh, &sh.flags[i % kRing], (i / kRing) & 1);  // long complete
      const uint2 there = *reinterpret_cast<const uint2*>(&sh.there[i % kRing][8 * half]);
      tmem_wait_ld(v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(s_free + 8 * st);
      if (there.x != 0x0F0F0F0Fu || there.y != 0x0F0F0F0Fu) {
        uint32_t valid = 0, bad = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t b = (k < 4 ? there.x : there.y) >> (8 * (k & 3));
          valid |= (b & 0xFu) << (4 * k);
          bad |= (b >> 4 & 0xFu) << (4 * k);
        }
        seen &= valid;
        poisoned |= (seen & bad) != 0u;
        seen &= ~bad;
      }
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
      sh.xchg[i & 1][tid] = top;
      row_bar(quarter);
      top = fmaxf(top, sh.xchg[i & 1][tid ^ kBlockRows]);
      // P and O keep an old reference until the maximum has risen by 2^40, so hardly a tile rescales O. (With 2^8 a tenth of
      // a warp's tiles did, for 1400 clocks, and each held up the other warps of both blocks.)
      const bool rise = top > m + kRescaleStep || (m == -INFINITY && top > -INFINITY);
      const float m_new = rise ? top : m;
      const float f = rise && m != -INFINITY ? exp2_approx(m - m_new) : 1.0f;  // without a reference, l and O are 0
      l *= f;
      m = m_new;
      // The weights are rounded to bf16 for the product: its operands have one type, and bf16 is the one that holds every
      // token exactly. l sums them unrounded, so lse keeps its 32 bits.
      const float ref = m == -INFINITY ? 0.f : m;
      uint32_t w[16];
      l += softmax_weights(v, unit, ref, w);
      if (i > 0) {
        // O is complete up to the last tile (for a rescaling), and with it P is free
        wait_for(sh, &sh.o_done[last], last_par);
        if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
          tc_fence_after();
          // either thread of a row has half of its columns
#pragma unroll 1
          for (int c = kDims / 2 * half; c < kDims / 2 * half + kDims / 2; c += 16) {
            uint32_t o[16];
            tmem_ld16(lanes + c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(lanes + c, o);
          }
          tmem_wait_st();
        }
      }
      const uint32_t p_row = smem_u32(p_s) + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        st_shared16(p_row + (((4 * half + c) ^ (r & 7)) << 4), make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(p_full);
      if (++last == kValueStages) last = 0, last_par ^= 1;
    }
    if (poisoned) l = __int_as_float(0x7FC00000);
    row_bar(quarter);
    sh.xchg[0][tid] = l;
    row_bar(quarter);
    l += sh.xchg[0][tid ^ kBlockRows];
    if (half == 0) {
      const bool split = u.part >= 0;
      sh.inv[r] = split ? 1.0f : l == 0.f ? 0.f : 1.0f / l;
      if (split) {
        p.ws_ml[part_row + r] = make_float2(m, l);
      } else if (p.lse && have && u.half == 0) {
        p.lse[(u.row0 + t) * p.ld_lse + u.head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      }
    }
    // Only the softmax warps may wait for the last O by its parity: they have followed every phase. The loader warps
    // are ordered behind it by the block barrier and the fences around it.
    wait_for(sh, &sh.o_done[last], last_par);
    tc_fence_after();
    tc_fence_before();
  }
  if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- epilogue
    // The loaders, four to a lane quarter and 64 columns each, write O (bf16, or the sums of a part) into the
    // stages' memory, a row of it per query row, and all warps store whole rows.
    constexpr int kPitchBf16 = kDims * 2 + 16, kPitchF32 = kDims * 4 + 16;  // eight rows' stores fall into different banks
    static_assert(kBlockRows * kPitchF32 <= kStages * kKeyBytes + kValueStages * kValueBytes + kPBytes, "the rows fit behind Q");
    epilogue_bar();
    tc_fence_after();
    const volatile Unit& e = sh.unit;
    const bool split = e.part >= 0;
    tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    if (warp >= kFirstLoader) {
      const int quarter = warp & 3, r = 32 * quarter + lane;
      const float inv = sh.inv[r];
#pragma unroll 1
      for (int c = 64 * ((warp - kFirstLoader) >> 2); c < 64 * ((warp - kFirstLoader) >> 2) + 64; c += 32) {
        uint32_t o[32];
        tmem_ld_x32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + c, o);
        tmem_wait_ld(o);
        if (split) {
          const uint32_t at = smem_u32(k_s) + r * kPitchF32 + c * 4;
#pragma unroll
          for (int j = 0; j < 8; ++j) st_shared16(at + 16 * j, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        } else {
          const uint32_t at = smem_u32(k_s) + r * kPitchBf16 + c * 2;
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
    const int first = static_cast<int>(cluster_rank()) * (p.tokens / 2);
    const int rows = max(min(e.rows - first, p.tokens / 2), 0) * p.heads, row0 = e.row0 + first;
    const int heads = e.heads, head0 = e.head0, dim0 = e.half * kDims;
    const int64_t part = static_cast<int64_t>(e.part) * kRows + cluster_rank() * kBlockRows;
    for (int r = warp; r < rows; r += kMmaWarp) {
      const int t = r / p.heads, h = r - t * p.heads;
      if (h >= heads) continue;
      const uint32_t from = smem_u32(k_s) + 16 * lane;
      if (split) {
        float* dst = p.ws_o + (part + r) * kDims + 4 * lane;
#pragma unroll
        for (int x = 0; x < kDims / 128; ++x) {
          *reinterpret_cast<uint4*>(dst + 128 * x) = ld_shared16(from + r * kPitchF32 + 512 * x);
        }
      } else {
        *reinterpret_cast<uint4*>(p.out + (row0 + t) * p.ld_out + (head0 + h) * p.ld_oh + dim0 + 8 * lane) =
            ld_shared16(from + r * kPitchBf16);
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  // neither block goes on while the other may still arrive in it or read its operands
  cluster_sync();
  tc_fence_after();
  started = true;
  }
  if (started && threadIdx.x / 32 == kMmaWarp) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace pair
}  // namespace idx
