// Attention of every query row over the tokens selected for it, read from the
// attention cache through their slots.
//
// "DeepSeek V3.2 稀疏注意力 DSA 推理流程图解", data-flow items 2-3: the selection hands
// the main attention a list of cache slots per query row; all heads of the row
// attend to the same list and share the token's one latent (key: its 512 latent
// and 64 position dims, value: the latent).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attention_mma.cuh"
#include "common.cuh"
#include "kv_layout.cuh"

namespace idx {
namespace {

// Bit 0: a slot outside the cache (the entry is skipped). Bit 1: a wait expired.
__device__ unsigned int g_attention_error = 0;

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t ld_q, ld_qh;  // elements between rows, between heads
  const uint8_t* cache;
  int num_blocks, block_size, block_span;
  uint32_t span_magic, span_shift;  // slot / block_span = (slot * span_magic >> 32) >> span_shift
  int64_t block_stride;
  const int32_t* slots;
  int64_t ld_slots;
  int k;
  const int32_t* n_sel;
  int T, H;
  float scale_log2;  // softmax_scale * log2(e)
  __nv_bfloat16* out;
  int64_t ld_out, ld_oh;
  float* lse;
  int64_t ld_lse;
  int head_blocks, parts, part_tiles;  // groups of 64 heads; parts of a row's list, and the tiles of one
  float2* ws_ml;                       // [T, head_blocks, parts, 64]: maximum (log2 units) and sum
  float* ws_o;                         // [T, head_blocks, parts, 64, 512]: accumulators
};

// ---------------------------------------------------------------------------
// The kernel
//
// One block per (row, group of 64 heads, part of the row's list), one block per SM.
// Per tile of 64 tokens:
//   S = Q K^T   64 heads x 64 tokens, 36 steps of K = 16 over the 576 dims
//   P = exp2(S * scale - m)    the running maximum m of each head in registers
//   O += P V    64 heads x 512 dims, 4 steps of K = 16 over the 64 tokens, two halves of N = 256
// with tcgen05.mma.ws (M = 64) in bf16 x bf16 -> fp32. The weight-stationary form is taken
// because its M = 64 fills all 128 tensor-memory lanes (row r, column half c / (N / 2) in lane
// r + 64 (c / (N / 2))): O takes 256 columns, where the plain form would take all 512 and leave none
// for S, and runs at five eighths of the rate (N = 256: 128 clocks against 80 on a GB300).
//
// Roles: warps 4-19 gather and dequantise the tokens' latents, warps 21-22 copy their position
// dims and prefetch, warp 20 issues the matrix instructions, warps 0-3 load Q and do the
// softmax; all but 20-22 store the result.
//
// Keys and values are one copy in shared memory: a token is a row of nine 128-byte swizzled
// pieces (64 dims each). Read along the dims it is the K-major B operand of S, read along the
// tokens the N-major B operand of O. Two tiles of 72 KB are in flight beside Q (72 KB) and P (8 KB).
//
// Two groups of eight loader warps own a stage each. A group converts and stores its tile, then issues
// every load of its next one at once, into registers: memory latency runs under the other group's
// conversion and the matrix work, with no staging buffer. (There was no room for one beside all of Q;
// since two thirds of Q went to tensor memory, 48 KB of its place are read by nobody once it is there.)
// (One group that refilled each register right after its conversion measured 7000 clocks a tile: loads of
// two tiles shared scoreboards, so every conversion waited for the newest load.) What a warp keeps in
// flight is limited whatever it asks for: random 512-byte rows read by 8 warps an SM came at 3.2 TB/s, by
// 16 at 5.4 TB/s, by 32 at 6.4 TB/s, with 8 or 16 rows asked for by each; hence sixteen, and the prefetch
// into L2.
//
// What bounds it: no counter is full. A tile takes 1.45 us (16 heads) to 1.48 us (64) of a block's time,
// some 2950 clocks: the slope from lists of 2048 to lists of 4096 entries, 128 rows. ncu counts per tile
// 1408 wavefronts of shared memory by the tensor core (S 768, O 640; S would take 1152 without Q's larger
// part in tensor memory) and 1830 by loads and stores (stores, shuffles and P 1170, the loads 660), 39 %
// and 51 % of the 3580 clocks that a tile takes with its share of a block's start and end. Their sum is
// more than the slope, so the two overlap and neither is the bound. Leaving out any one kind of work in a
// copy saved 5 to 11 %. That fits a chain: tile i + 2 may be stored only after O of tile i, and then its
// conversion, S, softmax and O follow in a row. 128 rows x 16 heads x 2048 tokens: 57 us where rows share
// eight contexts of 32 K tokens (the records of the entries take 26 us at the measured HBM rate, the
// distinct ones 16), 64 us where each row has 96 K tokens of its own (25 us); 1024 rows x 128 heads: 763
// us (763 TFLOP/s). Pairs of blocks that shared a tile's tokens (cta_group::2, M = 128) read less but
// measured 867 us there: values that cross between two SMs came at 10 bytes a clock, and gathered twice
// they cost what was saved.
// ---------------------------------------------------------------------------
constexpr int kHeadsPerBlock = 64;
constexpr int kTile = 64;
constexpr int kPieces = kKvDim / 64;             // 128-byte pieces of a token's bf16 row
constexpr int kQBytes = kPieces * kPieceBytes;
constexpr int kStageBytes = kPieces * kPieceBytes;
constexpr int kStages = 2;
constexpr int kLoaderWarps = 16;
constexpr int kGroupWarps = kLoaderWarps / kStages;  // each stage has its own group of loader warps
constexpr int kTokensPerWarp = kTile / kGroupWarps;
static_assert(kTokensPerWarp == 8, "a loader warp's tokens are eight rows of the swizzle");
constexpr int kEarly = 3;  // of a warp's tokens, those converted while the stage is still in use
constexpr int kMmaWarp = 4 + kLoaderWarps;
constexpr int kRopeWarp = kMmaWarp + 1;          // one per stage
constexpr int kThreads = (kRopeWarp + kStages) * 32;
constexpr int kValidRing = 4;
constexpr int kAhead = 4;                        // tiles between the L2 prefetch and the loads
constexpr int kOCols = 256;                      // tensor-memory columns of O; S0 and S1 (32 each) follow
constexpr int kQCols = 320;                      // and the first kQTmemPieces pieces of Q
constexpr int kQTmemPieces = 6;
constexpr int kTmemCols = 512;
static_assert(kQCols + kQTmemPieces * 32 <= kTmemCols, "tensor memory of one block");
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescaleStep = 8.0f;             // log2: P may reach 2^8 before O is rescaled

struct Shared {
  uint64_t q_full, drained;
  uint64_t k_full[kStages];                      // a stage's tokens are stored
  uint64_t s_full[kStages];                      // S of the tile is complete
  uint64_t p_full[kStages];                      // P is stored
  uint64_t o_done[kStages];                      // the tile's share of O is complete: P and the stage are free
  uint64_t flags[kValidRing];                    // `valid` is written
  uint32_t tmem;
  volatile uint32_t dead;                        // a wait expired: no further wait blocks
  uint32_t valid[kValidRing][2];                 // bit t: token t of the tile counts
  float xchg[2][128];
  float inv[kHeadsPerBlock];                     // 1 / sum of each head
};

constexpr int kSmemBytes = kQBytes + kStages * kStageBytes + kPieceBytes + 1024 + static_cast<int>(sizeof(Shared));
static_assert(kSmemBytes <= 232448, "shared memory of one block");

// Bounded wait. A wait that takes two seconds marks the block dead and raises the device
// flag; from then on no wait blocks, every role runs its remaining iterations on whatever it
// finds (all addresses stay in bounds), and the block ends in order.
__device__ __forceinline__ void wait_bar(Shared& sh, uint64_t* bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) {
    const uint64_t t0 = global_timer_ns();
    while (!sh.dead && !mbar_try_wait(bar, parity)) {
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_attention_error, 2u);
        sh.dead = 1;
      }
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 2, %0;" ::"n"(kMmaWarp * 32) : "memory"); }

// The softmax warps and the matrix warp: tensor memory is there (and every row of Q copied).
__device__ __forceinline__ void tmem_bar() { asm volatile("bar.sync 3, 160;" ::: "memory"); }

__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Where the token of a list entry lies; all null for an entry that does not count.
struct Token {
  const uint8_t* latent;
  const uint8_t* rope;
  const uint32_t* codes;
};

__device__ __forceinline__ Token locate(const AttnParams& p, int slot) {
  Token t{nullptr, nullptr, nullptr};
  if (slot < 0) return t;
  const int blk = static_cast<int>(__umulhi(static_cast<uint32_t>(slot), p.span_magic) >> p.span_shift);
  const int off = slot - blk * p.block_span;
  if (blk >= p.num_blocks || off >= p.block_size) {
    atomicOr(&g_attention_error, 1u);
    return t;
  }
  const uint8_t* base = p.cache + blk * p.block_stride;
  t.latent = base + off * kKvLatent;
  t.rope = base + p.block_size * kKvRopeAt + off * (2 * kKvRope);
  t.codes = reinterpret_cast<const uint32_t*>(base + p.block_size * kKvScaleAt + 4 * off);
  return t;
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + kQBytes;
  uint8_t* p_s = k_s + kStages * kStageBytes;
  Shared& sh = *reinterpret_cast<Shared*>(p_s + kPieceBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kSplit) asm volatile("griddepcontrol.launch_dependents;");  // the join may be set up meanwhile
  // head groups vary fastest: the blocks that read the same tokens run side by side
  const int hb = blockIdx.x % p.head_blocks;
  const int part = kSplit ? (blockIdx.x / p.head_blocks) % p.parts : 0;
  const int row = blockIdx.x / (p.head_blocks * p.parts);
  const int h0 = hb * kHeadsPerBlock;
  int n = p.k;
  if (p.n_sel) n = min(n, max(__ldg(p.n_sel + row), 0));
  const int first = part * p.part_tiles * kTile;  // of this block's entries
  if (kSplit) n = min(n, first + p.part_tiles * kTile);
  const int tiles = n > first ? (n - first + kTile - 1) / kTile : 0;

  const int64_t ws_row = (static_cast<int64_t>(row) * p.head_blocks + hb) * p.parts + part;
  if (tiles == 0) {
    if (kSplit) {
      if (tid < kHeadsPerBlock) p.ws_ml[ws_row * kHeadsPerBlock + tid] = make_float2(-INFINITY, 0.f);
    } else {
      const int heads = min(kHeadsPerBlock, p.H - h0);
      for (int i = tid; i < heads * (kKvLatent / 8); i += kThreads) {
        const int h = h0 + i / (kKvLatent / 8);
        *reinterpret_cast<uint4*>(p.out + row * p.ld_out + h * p.ld_oh + 8 * (i % (kKvLatent / 8))) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      if (p.lse && tid < heads) p.lse[row * p.ld_lse + h0 + tid] = -INFINITY;
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
    const int32_t* list = p.slots + row * p.ld_slots + first;
    const int count = n - first;
    const int mine = r0 + lane % kTokensPerWarp;  // entry of a tile that this lane locates
    const int left = count - mine;      // entries from its first one on
    const int32_t* my_list = list + mine;
    auto entry = [&](int tile) { return tile * kTile < left ? __ldg(my_list + tile * kTile) : -1; };

    // Lane l stores unit l % 8 of piece l / 8 and of piece 4 + l / 8: it holds the eight dims of either half
    // that the swizzle puts there. So the loads' addresses depend on the row, and the stores', which
    // would take registers, do not.
    uint2 raw[kTokensPerWarp][2];
    // Tokens are located two tiles of the group ahead of their conversion, and their slots read one more
    // ahead: nothing between two tiles' loads waits for an address.
    uint32_t codes = 0, next_codes = 0, found_codes = 0;
    int next_slot = -1;
    const uint8_t* latent = nullptr;
    auto find = [&](int tile) {
      const Token tok = locate(p, next_slot);
      latent = tok.latent;
      next_slot = entry(tile + kStages);
      found_codes = 0;
      if (latent) found_codes = __ldg(tok.codes);
    };
    auto load = [&]() {
#pragma unroll
      for (int j = 0; j < kTokensPerWarp; ++j) {
        const uint8_t* src = shfl_ptr(latent, j);
        raw[j][0] = load8_if(src + 8 * (lane ^ j), src != nullptr);  // r0 is a multiple of eight: row j of the swizzle
        raw[j][1] = load8_if(src + 256 + 8 * (lane ^ j), src != nullptr);
      }
    };
    // eight dims in half h of the token with these scale codes
    auto word_of = [&](int j) { return __shfl_sync(0xFFFFFFFFu, codes, j); };
    auto convert = [&](const uint2& x, uint32_t word, uint32_t h) {
      const uint32_t mul = kv_multiplier_of(__byte_perm(word, 0u, 0x4440u + 2 * h + (lane >> 4)));
      uint4 w;
      kv_dequant4_even_odd(x.x, mul, w.x, w.y);
      kv_dequant4_even_odd(x.y, mul, w.z, w.w);
      return w;
    };
    const uint32_t unit = smem_u32(k_s) + group * kStageBytes + (lane >> 3) * kPieceBytes + r0 * 128 + 16 * (lane & 7);

    if (group < tiles) {
      next_slot = entry(group);
      find(group);
      load();
      next_codes = found_codes;
      find(group + kStages);
    }
    setup();
    for (int i = group; i < tiles; i += kStages) {
      codes = __vminu4(next_codes, kKvCodeLimit * 0x01010101u);
      uint4 early[kEarly][2];
#pragma unroll
      for (int j = 0; j < kEarly; ++j) {
        const uint32_t word = word_of(j);
        early[j][0] = convert(raw[j][0], word, 0);
        early[j][1] = convert(raw[j][1], word, 1);
      }
      if (i >= kStages) wait_bar(sh, &sh.o_done[group], ((i >> 1) - 1) & 1);
#pragma unroll
      for (int j = 0; j < kTokensPerWarp; ++j) {
        const uint32_t word = j < kEarly ? 0u : word_of(j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          st_shared16(unit + 4 * h * kPieceBytes + j * 128, j < kEarly ? early[j % kEarly][h] : convert(raw[j][h], word, h));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[group]);
      if (i + kStages < tiles) load();
      next_codes = found_codes;
      find(i + 2 * kStages);
    }
  } else if (warp >= kRopeWarp) {
    // ---------------------------------------------------------------- position dims, and L2 prefetch
    // Position dims are bf16 in the cache as in the tile: copied asynchronously, as soon as S of the tile
    // before is complete (with the rest of the stage, after O, they held every tile up: 880 against 785 us
    // for 1024 rows x 128 heads).
    // Lane l locates tokens l and 32 + l. The same warp brings the records of the tile kAhead further
    // on into L2: a random token comes out of HBM in some 2900 clocks, out of L2 in 1200, and the
    // loaders' registers hold one tile.
    const int group = warp - kRopeWarp;
    const int32_t* list = p.slots + row * p.ld_slots + first;
    const int count = n - first;
    auto entry = [&](int tile, int h) {
      const int e = tile * kTile + 32 * h + lane;
      return e < count ? __ldg(list + e) : -1;
    };
    // 32 tokens: each lane's own position dims and codes, and 8 x 4 lines of latents an instruction
    auto prefetch = [&](int slot) {
      const Token t = locate(p, slot);
      if (t.latent) {
        prefetch_l2(t.rope);
        prefetch_l2(t.codes);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = shfl_ptr(t.latent, 8 * k + (lane >> 2));
        if (src) prefetch_l2(src + 128 * (lane & 3));
      }
      __syncwarp();
    };
    for (int i = group; i < kAhead && i < tiles; i += kStages) {
      prefetch(entry(i, 0));
      prefetch(entry(i, 1));
    }
    int s0 = entry(group, 0), s1 = entry(group, 1);
    int a0 = entry(group + kAhead, 0), a1 = entry(group + kAhead, 1);
    const uint32_t piece = smem_u32(k_s) + group * kStageBytes + (kPieces - 1) * kPieceBytes;
    setup();
    for (int i = group; i < tiles; i += kStages) {
      const uint8_t* src[2] = {locate(p, s0).rope, locate(p, s1).rope};
      s0 = entry(i + kStages, 0);
      s1 = entry(i + kStages, 1);
      // only S reads position dims, so their piece is free long before the stage is
      if (i >= kStages) wait_bar(sh, &sh.s_full[group], ((i >> 1) - 1) & 1);
#pragma unroll
      for (int c = 0; c < kTile / 4; ++c) {
        const int t = 4 * c + (lane >> 3), u = lane & 7;
        const uint8_t* from = shfl_ptr(src[c / 8], t & 31);
        copy16_if(piece + t * 128 + ((u ^ (t & 7)) << 4), from ? from + 16 * u : p.cache, from != nullptr);
      }
      const uint32_t v0 = __ballot_sync(0xFFFFFFFFu, src[0] != nullptr);
      const uint32_t v1 = __ballot_sync(0xFFFFFFFFu, src[1] != nullptr);
      if (lane == 0) {
        // S of tile i - 2, waited for above, was issued after O of tile i - 4, hence after entry i - 4 was read
        sh.valid[i % kValidRing][0] = v0;
        sh.valid[i % kValidRing][1] = v1;
        mbar_arrive(&sh.flags[i % kValidRing]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full[group]);
      if (i + kAhead < tiles) {
        prefetch(a0);
        prefetch(a1);
        a0 = entry(i + kStages + kAhead, 0);
        a1 = entry(i + kStages + kAhead, 1);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      mbar_init(&sh.q_full, 4);
      mbar_init(&sh.drained, 1);
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sh.k_full[i], kGroupWarps + 1);
        mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.p_full[i], 4);
        mbar_init(&sh.o_done[i], 1);
      }
      for (int i = 0; i < kValidRing; ++i) mbar_init(&sh.flags[i], 1);
      sh.dead = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(&sh.tmem, kTmemCols);
    tmem_relinquish();
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
    wait_bar(sh, &sh.q_full, 0);
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
        ++s_next;
        idle = 0;
        continue;
      }
      // nothing was ready: the limit of two seconds runs from the first such pass
      if (idle++ == 0) t0 = global_timer_ns();
      bool expired = sh.dead != 0;
      if (!expired && (idle & 63) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
        expired = true;
        atomicOr(&g_attention_error, 2u);
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
    // Q, sixteen rows a warp, rows of heads past the last one zero, all copies out at once. The latent dims
    // are then put into the loaders' order, 0, 2, 1, 3 of every four, and as many of them as there are columns
    // into tensor memory: S reads less of the shared memory that the loaders and O want too.
    const uint32_t q_row = smem_u32(q_s) + 16 * warp * 128;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int qh = h0 + 16 * warp + i;
      const bool have = qh < p.H;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q + row * p.ld_q + (have ? qh * p.ld_qh : 0));
      const uint32_t at = q_row + i * 128 + (((lane & 7) ^ (i & 7)) << 4);
      copy16_if(at + (lane >> 3) * kPieceBytes, src + 16 * lane, have);
      copy16_if(at + (4 + (lane >> 3)) * kPieceBytes, src + 512 + 16 * lane, have);
      if (lane < 8) copy16_if(at + 8 * kPieceBytes, src + 1024 + 16 * lane, have);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tmem_bar();
    tc_fence_after();
    tmem = sh.tmem;
    const int r = tid & 63, half = tid >> 6;          // head of the group, and half of the tile's tokens
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    auto reorder = [](const uint4& v) {
      return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x5410),
                        __byte_perm(v.z, v.w, 0x7632));
    };
    const uint32_t own_row = smem_u32(q_s) + r * 128;
#pragma unroll 1
    for (int u = 0; u < 8 * kQTmemPieces; u += 4) {
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 v = reorder(ld_shared16(own_row + (u >> 3) * kPieceBytes + ((((u + x) & 7) ^ (r & 7)) << 4)));
        w[4 * x] = v.x;
        w[4 * x + 1] = v.y;
        w[4 * x + 2] = v.z;
        w[4 * x + 3] = v.w;
      }
      tmem_st16(lanes + kQCols + 4 * u, w);
    }
    // of the latent pieces that stay in shared memory, each thread has half a row
#pragma unroll
    for (int c = kQTmemPieces; c < kKvLatent / 64; ++c) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t at = own_row + c * kPieceBytes + (((4 * half + u) ^ (r & 7)) << 4);
        st_shared16(at, reorder(ld_shared16(at)));
      }
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

    float m = -INFINITY, l = 0.f;                     // maximum (log2 units) that P and O refer to; this half's sum
    for (int i = 0; i < tiles; ++i) {
      const int st = i & 1;
      wait_bar(sh, &sh.s_full[st], (i >> 1) & 1);
      wait_bar(sh, &sh.flags[i % kValidRing], (i / kValidRing) & 1);  // long complete
      tc_fence_after();
      uint32_t v[32];
      tmem_ld_x32(lanes + kOCols + st * 32, v);
      const uint32_t valid = sh.valid[i % kValidRing][half];
      tmem_wait_ld(v);
      // v * unit is the logit in log2 units: the raw products as they are where every token counts, or
      // scaled here with -inf for the others
      float unit = p.scale_log2;
      float top = -INFINITY;
      if (valid != 0xFFFFFFFFu) {
        unit = 1.0f;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          v[c] = (valid >> c) & 1u ? __float_as_uint(__uint_as_float(v[c]) * p.scale_log2) : 0xFF800000u;
        }
      }
      if (unit >= 0.f) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) top = fmaxf(top, fmaxf(__uint_as_float(v[c]), __uint_as_float(v[c + 1])));
      } else {
        top = INFINITY;
#pragma unroll
        for (int c = 0; c < 32; c += 2) top = fminf(top, fminf(__uint_as_float(v[c]), __uint_as_float(v[c + 1])));
      }
      top *= unit;
      sh.xchg[st][tid] = top;
      softmax_bar();
      top = fmaxf(top, sh.xchg[st][tid ^ 64]);
      // P and O keep an old reference until the maximum has risen by 2^8: P stays finite and
      // its relative precision is the same, and most tiles leave O alone
      const bool rise = top > m + kRescaleStep || (m == -INFINITY && top > -INFINITY);
      const float m_new = rise ? top : m;
      if (i > 0) {
        // O is complete up to the last tile (for a rescaling), and with it the only P is free
        const bool scale_o = __any_sync(0xFFFFFFFFu, rise);
        wait_bar(sh, &sh.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
        if (scale_o) {
          tc_fence_after();
          const float f = rise ? exp2_approx(m - m_new) : 1.0f;  // m = -inf: 0, and O is 0
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
      // token exactly. l sums them unrounded, so lse keeps its 32 bits, and out differs from the exact value by 2.1e-3
      // (norm) where its own rounding alone makes 1.65e-3. A second product with the rest would cost O again.
      const float ref = m == -INFINITY ? 0.f : m;
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float e0 = exp2_approx(fmaf(__uint_as_float(v[c]), unit, -ref));
        const float e1 = exp2_approx(fmaf(__uint_as_float(v[c + 1]), unit, -ref));
        l += e0 + e1;
        const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
        w[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      const uint32_t p_row = smem_u32(p_s) + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        st_shared16(p_row + (((4 * half + c) ^ (r & 7)) << 4), make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
      }
      arrive(&sh.p_full[st]);
    }
    softmax_bar();
    sh.xchg[0][tid] = l;
    softmax_bar();
    l += sh.xchg[0][tid ^ 64];
    const int h = h0 + r;
    if (half == 0) {
      sh.inv[r] = l == 0.f ? 0.f : 1.0f / l;
      if (kSplit) {
        p.ws_ml[ws_row * kHeadsPerBlock + r] = make_float2(m, l);
      } else if (p.lse && h < p.H) {
        p.lse[row * p.ld_lse + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      }
    }
  }
  if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- epilogue
    // The loaders, four to a lane quarter and 64 columns each, write O (bf16, or the sums of a part) into the
    // stages' memory, a row of it per head, and all warps store whole rows. (Stored from the registers, 16
    // bytes of a row each, the rows of 64 heads took 5500 clocks, 10500 in fp32; as bulk copies, whose
    // end the block has to wait for, 2300 to 5800.)
    constexpr int kRowBytes = kKvLatent * (kSplit ? 4 : 2);
    constexpr int kPitch = kRowBytes + 16;  // eight rows' stores fall into different banks
    static_assert(kHeadsPerBlock * kPitch <= kStages * kStageBytes, "the rows fit the stages");
    // Only the softmax warps may wait for the last O by its parity: they have followed every phase of both o_done
    // barriers. A loader warp has followed its own stage's only, and from three tiles on could take an earlier phase
    // of the other for the last one. It is ordered behind O by the block barrier and the fences around it.
    if (warp < 4) {
      wait_bar(sh, &sh.o_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);
      tc_fence_after();
      tc_fence_before();
    }
    epilogue_bar();
    tc_fence_after();
    if (warp >= 4) {
      const int quarter = warp & 3, r = (32 * quarter + lane) & 63, half = quarter >> 1;
      const float inv = sh.inv[r];
#pragma unroll 1
      for (int c = 64 * ((warp - 4) >> 2); c < 64 * ((warp - 4) >> 2) + 64; c += 32) {
        uint32_t o[32];
        tmem_ld_x32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + c, o);
        tmem_wait_ld(o);
        // A product has 256 dims, 128 to each lane half. Dims 1 and 2 of every four have changed places.
        const int dim = (c / 128) * 256 + half * 128 + (c % 128);
        const uint32_t at = smem_u32(k_s) + r * kPitch + dim * (kSplit ? 4 : 2);
        if (kSplit) {
#pragma unroll
          for (int j = 0; j < 8; ++j) st_shared16(at + 16 * j, make_uint4(o[4 * j], o[4 * j + 2], o[4 * j + 1], o[4 * j + 3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int e = 8 * j + 4 * (x >> 1) + (x & 1);  // dims 2 x, 2 x + 1 lie two columns apart
              const __nv_bfloat162 b =
                  __floats2bfloat162_rn(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 2]) * inv);
              w[x] = *reinterpret_cast<const uint32_t*>(&b);
            }
            st_shared16(at + 16 * j, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
    }
    epilogue_bar();
    constexpr int kUnits = kRowBytes / 16;
    const int heads = min(kHeadsPerBlock, p.H - h0);
    for (int i = tid; i < heads * kUnits; i += kMmaWarp * 32) {
      const int r = i / kUnits, u = i % kUnits;
      uint8_t* dst = kSplit ? reinterpret_cast<uint8_t*>(p.ws_o + (ws_row * kHeadsPerBlock + r) * kKvLatent)
                            : reinterpret_cast<uint8_t*>(p.out + row * p.ld_out + (h0 + r) * p.ld_oh);
      *reinterpret_cast<uint4*>(dst + 16 * u) = ld_shared16(smem_u32(k_s) + r * kPitch + 16 * u);
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the parts of each (row, head): weights 2^(m_i - max m), a part without a valid token skipped (its
// accumulators were never written). A head is the work of kWarps warps, each of which takes every kWarps-th
// part, two at a time, 16 dims a lane: all heads of a batch run at once, and the eight loads of two parts
// are in flight together. The maxima and sums are few enough for every warp to reduce them itself.
constexpr int kJoinWarps = 8;   // of a block
constexpr int kMaxParts = 128;

template <int kWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const AttnParams p) {
  constexpr int kHeads = kJoinWarps / kWarps;  // of a block
  __shared__ float4 sums[kHeads][kWarps > 1 ? kWarps - 1 : 1][kKvLatent / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp / kWarps, g = warp % kWarps;
  const uint32_t heads = static_cast<uint32_t>(p.H), head = blockIdx.x * kHeads + sub;
  const bool have = head < static_cast<uint32_t>(p.T) * heads;
  const uint32_t row = have ? head / heads : 0u, h = have ? head - row * heads : 0u;
  const int64_t base = (static_cast<int64_t>(row) * p.head_blocks + h / kHeadsPerBlock) * p.parts * kHeadsPerBlock +
                       h % kHeadsPerBlock;
  const float2* ml = p.ws_ml + base;  // of part i: ml[64 i], o[64 * 128 i]
  const float4* o = reinterpret_cast<const float4*>(p.ws_o + base * kKvLatent) + lane;
  constexpr int kStep = kHeadsPerBlock * kKvLatent / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every part is complete and visible

  float2 mine[kMaxParts / 32];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < kMaxParts / 32; ++c) {
    mine[c] = 32 * c + lane < p.parts ? __ldcg(ml + (32 * c + lane) * kHeadsPerBlock) : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, mine[c].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll
  for (int c = 0; c < kMaxParts / 32; ++c) {
    if (mine[c].y != 0.f) l = fmaf(exp2f(mine[c].x - m), mine[c].y, l);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);

  float4 acc[4] = {};
  for (int i = g; i < p.parts; i += 2 * kWarps) {
    float2 x[2];
    float4 v[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int part = i + j * kWarps;
      x[j] = make_float2(-INFINITY, 0.f);
      if (part >= p.parts) continue;
      x[j] = __ldcg(ml + part * kHeadsPerBlock);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[j][c] = __ldcg(o + static_cast<int64_t>(part) * kStep + 32 * c);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (x[j].y == 0.f) continue;
      const float w = exp2f(x[j].x - m);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c].x = fmaf(w, v[j][c].x, acc[c].x);
        acc[c].y = fmaf(w, v[j][c].y, acc[c].y);
        acc[c].z = fmaf(w, v[j][c].z, acc[c].z);
        acc[c].w = fmaf(w, v[j][c].w, acc[c].w);
      }
    }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (g > 0) sums[sub][g - 1][lane + 32 * c] = acc[c];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < kWarps - 1; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = sums[sub][i][lane + 32 * c];
        acc[c].x += v.x;
        acc[c].y += v.y;
        acc[c].z += v.z;
        acc[c].w += v.w;
      }
    }
  }
  if (!have) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  __nv_bfloat16* dst = p.out + row * p.ld_out + h * p.ld_oh + 4 * lane;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    *reinterpret_cast<uint2*>(dst + 128 * c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (p.lse && lane == 0) {
    p.lse[row * p.ld_lse + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

// Parts that a list of k entries is split into: as many as one wave of blocks has room for, if that
// is cheaper than whole rows. In units of a tile (1.46 us on a GB300) a block's start and end cost some seven with the
// launch, whole or part, and the join four. Lists of 2048, 64 heads, in parts against whole: one row 14 us (32 parts) and
// 57 us, 16 rows 22 (8) and 57, 64 rows 41 (2) and 58. A second wave of parts does not pay: 100 rows
// measured 80 us in three parts and 59 whole.
int attention_parts(int64_t blocks, int k, int sms) {
  const int tiles = (k + kTile - 1) / kTile;
  if (sms <= 0 || tiles <= 1 || 2 * blocks > sms) return 1;
  const int room = static_cast<int>(std::min<int64_t>(sms / blocks, kMaxParts));
  const int per = (tiles + room - 1) / room;         // tiles of a part
  const int parts = (tiles + per - 1) / per;         // none without tiles
  return per + 4 < tiles ? parts : 1;
}

int64_t part_bytes() { return kHeadsPerBlock * (static_cast<int64_t>(kKvLatent) * 4 + 8); }

}  // namespace

unsigned int attention_read_and_clear_error(cudaStream_t stream, cudaError_t* err) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  *err = cudaStreamSynchronize(stream);
  if (*err != cudaSuccess) return 0;
  *err = cudaMemcpyFromSymbol(&v, g_attention_error, sizeof(v));
  if (*err != cudaSuccess) return 0;
  if (v) *err = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(zero));
  return v;
}

}  // namespace idx

using namespace idx;

extern "C" size_t idx_sparse_attention_workspace_bytes(int32_t T, int32_t H, int32_t k) {
  if (T <= 0 || H <= 0 || k <= 0 || k > (1 << 30)) return 0;
  const int64_t blocks = static_cast<int64_t>(T) * ((H + kHeadsPerBlock - 1) / kHeadsPerBlock);
  const int parts = attention_parts(blocks, k, device_sm_count());
  return parts == 1 ? 0 : static_cast<size_t>(blocks * parts * part_bytes());
}

extern "C" idx_status_t idx_sparse_attention(const void* q, int64_t ld_q, int64_t ld_qh, const uint8_t* cache,
                                             int32_t num_blocks, int32_t block_size, int64_t block_stride_bytes,
                                             int32_t block_span, const int32_t* slots, int64_t ld_slots, int32_t k,
                                             const int32_t* n_sel, int32_t T, int32_t H, float softmax_scale,
                                             void* out, int64_t ld_out, int64_t ld_oh, float* lse, int64_t ld_lse,
                                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  const char* fn = "idx_sparse_attention";
  if (T < 0 || H < 0 || k < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (k > (1 << 30)) return fail(IDX_ERR_UNSUPPORTED, "%s: lists of %d entries", fn, k);
  if (H > IDX_ATTENTION_MAX_HEADS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d heads", fn, H);
  if (ld_slots < k || ld_q < kKvDim || ld_qh < kKvDim || ld_out < kKvLatent || ld_oh < kKvLatent || (lse && ld_lse < H)) {
    return fail(IDX_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  }
  if (!std::isfinite(softmax_scale * 1.4426950408889634f)) return fail(IDX_ERR_INVALID_ARG, "%s: softmax_scale is not finite", fn);
  if (T == 0 || H == 0) return IDX_OK;
  if (!q || !cache || !out || (!slots && k > 0)) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  idx_status_t st = check_kv_cache(fn, cache, num_blocks, block_size, block_stride_bytes);
  if (st != IDX_OK) return st;
  if (block_span < block_size) return fail(IDX_ERR_UNSUPPORTED, "%s: block_span %d < block_size", fn, block_span);
  if (!aligned(q, 16) || ld_q % 8 != 0 || ld_qh % 8 != 0 || !aligned(out, 16) || ld_out % 8 != 0 || ld_oh % 8 != 0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: q and out rows must be 16-byte aligned", fn);
  }
  if (ws && !aligned(ws, 16)) return fail(IDX_ERR_UNSUPPORTED, "%s: the workspace is not 16-byte aligned", fn);
  const int sms = device_sm_count();
  if (sms <= 0) return fail(IDX_ERR_CUDA, "%s: cannot query the SM count", fn);
  AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ld_q = ld_q;
  p.ld_qh = ld_qh;
  p.cache = cache;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.block_span = block_span;
  // Division of n < 2^31 by d by one multiplication: with 2^(s - 1) < d <= 2^s and m = floor(2^(31 + s) / d) + 1,
  // m d exceeds 2^(31 + s) by at most d <= 2^s, so n m / 2^(31 + s) exceeds n / d by less than 1 / d.
  uint32_t log = 1;
  while ((int64_t{1} << log) < block_span) ++log;
  p.span_magic = static_cast<uint32_t>((uint64_t{1} << (31 + log)) / static_cast<uint32_t>(block_span) + 1);
  p.span_shift = log - 1;
  p.block_stride = block_stride_bytes;
  p.slots = slots;
  p.ld_slots = ld_slots;
  p.k = k;
  p.n_sel = n_sel;
  p.T = T;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ld_out = ld_out;
  p.ld_oh = ld_oh;
  p.lse = lse;
  p.ld_lse = ld_lse;
  p.head_blocks = (H + kHeadsPerBlock - 1) / kHeadsPerBlock;
  const int64_t blocks = static_cast<int64_t>(T) * p.head_blocks;
  p.parts = ws ? attention_parts(blocks, k, sms) : 1;
  const int tiles = (k + kTile - 1) / kTile;
  p.part_tiles = (tiles + p.parts - 1) / p.parts;
  if (blocks * p.parts > INT32_MAX || static_cast<int64_t>(T) * H > INT32_MAX) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: %d rows of %d heads", fn, T, H);
  }
  const unsigned grid = static_cast<unsigned>(blocks * p.parts);
  if (p.parts > 1) {
    if (ws_bytes < static_cast<size_t>(blocks * p.parts * part_bytes())) {
      return fail(IDX_ERR_INVALID_ARG, "%s: the workspace has %zu bytes, %lld are needed", fn, ws_bytes,
                  static_cast<long long>(blocks * p.parts * part_bytes()));
    }
    p.ws_o = static_cast<float*>(ws);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + blocks * p.parts * kHeadsPerBlock * kKvLatent);
  }
  auto* kernel = p.parts > 1 ? attention_kernel<true> : attention_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  kernel<<<grid, kThreads, kSmemBytes, stream>>>(p);
  st = check_launch(fn);
  if (st != IDX_OK || p.parts == 1) return st;
  // launched while the parts run: its blocks wait at their first reads for the parts' end; a warp takes four parts
  const int warps = p.parts <= 4 ? 1 : p.parts <= 8 ? 2 : p.parts <= 16 ? 4 : 8;
  auto* join = warps == 1   ? attention_join_kernel<1>
               : warps == 2 ? attention_join_kernel<2>
               : warps == 4 ? attention_join_kernel<4>
                            : attention_join_kernel<8>;
  const int heads = kJoinWarps / warps;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(T) * H + heads - 1) / heads));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t ej = cudaLaunchKernelEx(&cfg, join, p);
  if (ej != cudaSuccess) {
    cudaGetLastError();
    return fail(IDX_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(ej));
  }
  return check_launch(fn);
}
