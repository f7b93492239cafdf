// Attention over whole contexts of the paged attention cache: within a sliding
// window and over a few first tokens (idx_window_attention), and of trees of drafted
// tokens (idx_tree_attention).
#include <algorithm>
#include <cmath>

#include "paged_attention.cuh"
#include "paged_block.cuh"

namespace idx {
namespace {

// How a call's rows are cut into units, and the workers among whom they are shared out.
struct Plan {
  int head_blocks, heads, tokens, workers;
  int64_t units;
};

// Joins the parts of the units that the workers' shares cut: weights 2^(m_i - max m), a part without a visible token
// skipped (its accumulators were never written). The rows of all cut units are dealt out to the warps, or where there
// are few to groups of up to eight warps, each of which takes its share of the parts, four at a time. The first part of a
// unit is its worker's last (2 worker + 1), every other its worker's first (2 worker). At most 40 MB are read, mostly from
// L2; it adds some 4 us to a call.
constexpr int kJoinWarps = 8;   // of a block
constexpr int kJoinBlocks = 2;  // of an SM
constexpr int kMaxWorkers = kJoinWarps * 32;

__global__ void __launch_bounds__(kJoinWarps * 32, kJoinBlocks) paged_join_kernel(const PagedParams p) {
  constexpr int kVecs = kKvLatent / 128;
  __shared__ int ends[kMaxWorkers];  // rows of the cut units up to and with each worker's
  __shared__ float4 sums[kJoinWarps][kKvLatent / 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every part is complete and visible
  const int cuts = min(p.workers, kMaxWorkers);
  int mine = 0;
  if (tid < cuts && __ldcg(&p.ws_cuts[tid].parts) > 0) mine = __ldcg(&p.ws_cuts[tid].rows) * __ldcg(&p.ws_cuts[tid].heads);
  if (!__syncthreads_or(mine)) return;
  ends[tid] = mine;
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int k = 0; k < kMaxWorkers; k += 32) {
      int upto = ends[k + lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
      }
      ends[k + lane] = before + upto;
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
  __syncthreads();
  const int total = ends[kMaxWorkers - 1];
  int team = kJoinWarps;  // warps of a row
  while (team > 1 && static_cast<int64_t>(total) * team > static_cast<int64_t>(gridDim.x) * kJoinWarps) team >>= 1;
  const int teams = kJoinWarps / team, g = warp % team;
  for (int base = blockIdx.x * teams; base < total; base += gridDim.x * teams) {  // the same for all warps
    const int item = base + warp / team;
    const bool have = item < total;
    Cut cut{};
    int worker = 0, r = 0, t = 0, h = 0;
    if (have) {
      int lo = 0, hi = kMaxWorkers - 1;  // the first worker with ends > item
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > item) hi = mid; else lo = mid + 1;
      }
      worker = lo;
      const int4* c = reinterpret_cast<const int4*>(p.ws_cuts + worker);
      const int4 c0 = __ldcg(c), c1 = __ldcg(c + 1);
      cut = Cut{c0.x, c0.y, c0.z, c0.w, c1.x, {0, 0, 0}};
      const int in = item - (lo > 0 ? ends[lo - 1] : 0);
      t = in / cut.heads;
      h = in - t * cut.heads;
      r = t * p.heads + h;
    }
    auto place = [&](int i) { return static_cast<int64_t>(2 * (worker + i) + (i == 0 ? 1 : 0)) * block::kRows + r; };
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < cut.parts; i += 32) {
      const float2 x = __ldcg(p.ws_ml + place(i));
      const float top = fmaxf(m, x.x);
      if (l != 0.f) l *= exp2f(m - top);
      if (x.y != 0.f) l += x.y * exp2f(x.x - top);
      m = top;
    }
    float top = m;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    if (l != 0.f) l *= exp2f(m - top);
    m = top;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    float4 acc[kVecs] = {};
    for (int i0 = g; i0 < cut.parts; i0 += 4 * team) {
      float2 x[4];
      float4 v[4][kVecs];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * team;
        x[j] = make_float2(-INFINITY, 0.f);
        if (i >= cut.parts) continue;
        x[j] = __ldcg(p.ws_ml + place(i));
        const float4* o = reinterpret_cast<const float4*>(p.ws_o + place(i) * kKvLatent) + lane;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) v[j][c] = __ldcg(o + 32 * c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (x[j].y == 0.f) continue;
        const float w = exp2f(x[j].x - m);
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
          acc[c].x = fmaf(w, v[j][c].x, acc[c].x);
          acc[c].y = fmaf(w, v[j][c].y, acc[c].y);
          acc[c].z = fmaf(w, v[j][c].z, acc[c].z);
          acc[c].w = fmaf(w, v[j][c].w, acc[c].w);
        }
      }
    }
    if (team > 1) {
      __syncthreads();  // the last row's sums are read
#pragma unroll
      for (int c = 0; c < kVecs; ++c) sums[warp][lane + 32 * c] = acc[c];
      __syncthreads();
      if (g > 0) continue;
      for (int i = 1; i < team; ++i) {
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
          const float4 v = sums[warp + i][lane + 32 * c];
          acc[c].x += v.x;
          acc[c].y += v.y;
          acc[c].z += v.z;
          acc[c].w += v.w;
        }
      }
    }
    if (!have) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int64_t q = cut.row0 + t;
    __nv_bfloat16* dst = p.out + q * p.ld_out + (cut.head0 + h) * p.ld_oh + 4 * lane;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
      *reinterpret_cast<uint2*>(dst + 128 * c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    if (p.lse && lane == 0) {
      p.lse[q * p.ld_lse + cut.head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

Plan plan_of(int32_t T, int32_t B, int32_t H) {
  Plan plan{};
  plan.head_blocks = (H + block::kRows - 1) / block::kRows;
  plan.heads = (H + plan.head_blocks - 1) / plan.head_blocks;
  plan.tokens = block::kRows / plan.heads;
  plan.units = (T / plan.tokens + static_cast<int64_t>(B)) * plan.head_blocks;
  plan.workers = B <= kMaxSharedRequests ? std::min(device_sm_count(), kMaxWorkers) : 0;
  return plan;
}

int64_t plan_bytes(const Plan& plan) {
  return plan.workers * (static_cast<int64_t>(sizeof(Cut)) + 2 * block::kRows * (kKvLatent * 4 + 8));
}

// How many tiles a row may see: the host knows only how much the table or the window has room for.
int64_t most_tiles_of(const PagedParams& p, const Plan& plan, bool tree) {
  const int64_t tokens = std::min(static_cast<int64_t>(p.n_pages) * p.block_size, static_cast<int64_t>(INT32_MAX));
  return (tree ? tokens : std::min(tokens, static_cast<int64_t>(p.window) + p.sinks + plan.tokens)) / kTile;
}

// Whether even shares can gain what they cost: the parts' stores, the join, and a start and an end more for a block (some
// 6 us). Few units are cut: 8 requests of 4 rows and 16 heads take 16.6 us shared and 19.1 us plain with 8 tiles, 15.3 and
// 13.2 with 4; 76 windows of 4096 tokens and 64 heads 69 and 104 us, 16 of 1024 21 and 33 us. Of more units only the uneven
// ends are gained, and windows are as long as one another (128 of 4096 tokens: 120 and 107 us). 64 requests of 8 rows and
// 64 heads take 443 and 505 us with 128 tiles at most, 148 and 146 with 32, 100 and 85 with 16.
bool worth_cutting(const PagedParams& p, const Plan& plan, bool tree) {
  const int64_t units = std::min(static_cast<int64_t>(p.T) * plan.head_blocks, plan.units);
  const bool few = 2 * units <= plan.workers;
  if (most_tiles_of(p, plan, tree) < (few ? 8 : 32) || !(tree || few)) return false;
  // the line's sums stay far within 32 bits
  return most_tiles_of(p, plan, true) + 1 + kUnitTiles <= (int64_t{1} << 29) / std::max<int64_t>(units, plan.workers);
}

// Whether a block for each SM, which takes units in turn and finds the next while it finishes one, is faster than a block
// for each unit: chunks of four prompts, 128 heads, a window of 1024 take 629 us, and some 5 % more with a block each;
// four prompts of 512 rows 266 and 307 us. Long contexts are left to the order in which blocks become free: 64 trees of 8 nodes and 64
// heads with up to 128 tiles take 539 us in turn and 506 with a block each, with 16 tiles 83 and 86, with 8 tiles 51 and 58.
bool worth_sharing(const PagedParams& p, const Plan& plan, bool tree) {
  return plan.units > plan.workers && (!tree || most_tiles_of(p, plan, tree) < 32);
}

// What both calls check and launch; `p` holds what they were given.
idx_status_t paged_attention(const char* fn, PagedParams& p, float softmax_scale, void* ws, size_t ws_bytes, bool tree,
                             cudaStream_t stream) {
  if (p.T < 0 || p.H < 0 || p.B < 0 || p.n_pages < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (p.H > IDX_ATTENTION_MAX_HEADS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d heads", fn, p.H);
  if (p.ld_bt < p.n_pages || p.ld_q < kKvDim || p.ld_qh < kKvDim || p.ld_out < kKvLatent || p.ld_oh < kKvLatent ||
      (p.lse && p.ld_lse < p.H)) {
    return fail(IDX_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  }
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  if (!std::isfinite(p.scale_log2)) return fail(IDX_ERR_INVALID_ARG, "%s: softmax_scale is not finite", fn);
  if (p.T == 0 || p.H == 0 || p.B == 0) return IDX_OK;
  if (!p.q || !p.cache || !p.out || !p.cu_rows || !p.ctx_lens || (!p.block_table && p.n_pages > 0)) {
    return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  }
  const idx_status_t st = check_kv_cache(fn, p.cache, p.num_blocks, p.block_size, p.block_stride);
  if (st != IDX_OK) return st;
  if (!aligned(p.q, 16) || p.ld_q % 8 != 0 || p.ld_qh % 8 != 0 || !aligned(p.out, 16) || p.ld_out % 8 != 0 || p.ld_oh % 8 != 0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: q and out rows must be 16-byte aligned", fn);
  }
  constexpr int64_t kMostBytes = int64_t{1} << 40;  // between two rows, heads or blocks: what a tensor map holds
  if ((p.T > 1 && p.ld_q >= kMostBytes / 2) || (p.H > 1 && p.ld_qh >= kMostBytes / 2) ||
      (p.num_blocks > 1 && p.block_stride >= kMostBytes)) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: a stride of 2^40 bytes or more", fn);
  }
  if (ws && !aligned(ws, 16)) return fail(IDX_ERR_UNSUPPORTED, "%s: the workspace is not 16-byte aligned", fn);
  if (device_sm_count() <= 0) return fail(IDX_ERR_CUDA, "%s: cannot query the SM count", fn);
  const Plan plan = plan_of(p.T, p.B, p.H);
  if (plan.units > INT32_MAX / 2 || static_cast<int64_t>(p.T) * p.H > INT32_MAX / 2) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: %d rows of %d heads in %d requests", fn, p.T, p.H, p.B);
  }
  p.page_shift = p.block_size == 16 ? 4 : p.block_size == 32 ? 5 : p.block_size == 64 ? 6 : 7;
  p.head_blocks = plan.head_blocks;
  p.heads = plan.heads;
  p.tokens = plan.tokens;
  p.cut = ws && plan.workers && worth_cutting(p, plan, tree);
  p.workers = p.cut || worth_sharing(p, plan, tree) ? plan.workers : 0;
  if (ws && ws_bytes < static_cast<size_t>(plan_bytes(plan))) {
    return fail(IDX_ERR_INVALID_ARG, "%s: the workspace has %zu bytes, %lld are needed", fn, ws_bytes,
                static_cast<long long>(plan_bytes(plan)));
  }
  if (p.cut) {
    p.ws_cuts = static_cast<Cut*>(ws);
    p.ws_o = reinterpret_cast<float*>(p.ws_cuts + p.workers);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + 2 * static_cast<int64_t>(p.workers) * block::kRows * kKvLatent);
  }
  // Q as a unit reads it, 64 dims of its heads and rows a copy, and the position dims of the cache's pages. Strides of one
  // row, head or block may be anything.
  CUtensorMap q_map, rope_map;
  const uint64_t q_dims[3] = {kKvDim, static_cast<uint64_t>(p.H), static_cast<uint64_t>(p.T)};
  const uint64_t q_strides[2] = {p.H > 1 ? 2 * static_cast<uint64_t>(p.ld_qh) : 2 * kKvDim,
                                 p.T > 1 ? 2 * static_cast<uint64_t>(p.ld_q) : 2 * kKvDim};
  const uint32_t q_box[3] = {64, static_cast<uint32_t>(plan.heads), static_cast<uint32_t>(plan.tokens)};
  idx_status_t made = encode_tensor_map(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q, q_dims, q_strides, q_box,
                                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (made != IDX_OK) return made;
  const uint64_t rope_dims[3] = {kKvRope, static_cast<uint64_t>(p.block_size), static_cast<uint64_t>(std::max(p.num_blocks, 1))};
  const uint64_t rope_strides[2] = {2 * kKvRope, static_cast<uint64_t>(p.num_blocks > 1 ? p.block_stride : p.block_size * IDX_KV_TOKEN_BYTES)};
  const uint32_t rope_box[3] = {kKvRope, static_cast<uint32_t>(block::copy_tokens_of(p.block_size)), 1};
  made = encode_tensor_map(&rope_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.cache + p.block_size * kKvRopeAt, rope_dims,
                           rope_strides, rope_box, CU_TENSOR_MAP_SWIZZLE_128B);
  if (made != IDX_OK) return made;
  const unsigned units = static_cast<unsigned>(p.workers ? p.workers : plan.units);
  auto* kernel = tree ? block::paged_block_kernel<true> : block::paged_block_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, block::kSmemBytes);
  if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  kernel<<<units, block::kThreads, block::kSmemBytes, stream>>>(q_map, rope_map, p);
  if (e == cudaSuccess && p.cut && p.workers > 1) {
    const idx_status_t launched = check_launch(fn);
    if (launched != IDX_OK) return launched;
    // launched while the parts run: its blocks wait at their first reads for the parts' end
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(kJoinBlocks * device_sm_count()));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_join_kernel, static_cast<const PagedParams>(p));
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(IDX_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  }
  return check_launch(fn);
}

}  // namespace

unsigned int paged_attention_read_and_clear_error(cudaStream_t stream, cudaError_t* err) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  *err = cudaStreamSynchronize(stream);
  if (*err != cudaSuccess) return 0;
  *err = cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v));
  if (*err != cudaSuccess) return 0;
  if (v) *err = cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(zero));
  return v;
}

}  // namespace idx

using namespace idx;

extern "C" size_t idx_paged_attention_workspace_bytes(int32_t T, int32_t B, int32_t H) {
  if (T <= 0 || B <= 0 || H <= 0 || H > IDX_ATTENTION_MAX_HEADS) return 0;
  return static_cast<size_t>(plan_bytes(plan_of(T, B, H)));
}

extern "C" idx_status_t idx_window_attention(const void* q, int64_t ld_q, int64_t ld_qh, const uint8_t* cache,
                                             int32_t num_blocks, int32_t block_size, int64_t block_stride_bytes,
                                             const int32_t* block_table, int64_t ld_bt, int32_t n_pages,
                                             const int32_t* cu_rows, const int32_t* ctx_lens, int32_t B,
                                             int32_t window, int32_t sinks, int32_t T, int32_t H,
                                             float softmax_scale, void* out, int64_t ld_out, int64_t ld_oh, float* lse,
                                             int64_t ld_lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const char* fn = "idx_window_attention";
  if (window < 1 || sinks < 0) return fail(IDX_ERR_INVALID_ARG, "%s: window %d, sinks %d", fn, window, sinks);
  PagedParams p{static_cast<const __nv_bfloat16*>(q), ld_q, ld_qh, cache, num_blocks, block_size, block_stride_bytes,
                block_table, ld_bt, n_pages, cu_rows, ctx_lens, B, window, sinks, nullptr, 0, 0, T, H, 0.f,
                static_cast<__nv_bfloat16*>(out), ld_out, ld_oh, lse, ld_lse};
  return paged_attention(fn, p, softmax_scale, ws, ws_bytes, false, stream);
}

extern "C" idx_status_t idx_tree_attention(const void* q, int64_t ld_q, int64_t ld_qh, const uint8_t* cache,
                                           int32_t num_blocks, int32_t block_size, int64_t block_stride_bytes,
                                           const int32_t* block_table, int64_t ld_bt, int32_t n_pages,
                                           const int32_t* cu_rows, const int32_t* ctx_lens, int32_t B,
                                           const int32_t* mask, int64_t ld_mask, int32_t words, int32_t T, int32_t H,
                                           float softmax_scale, void* out, int64_t ld_out, int64_t ld_oh, float* lse,
                                           int64_t ld_lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const char* fn = "idx_tree_attention";
  if (words < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (words > IDX_TREE_MAX_WORDS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d words", fn, words);
  if (ld_mask < words) return fail(IDX_ERR_INVALID_ARG, "%s: ld_mask is smaller than words", fn);
  if (T > 0 && words > 0 && !mask) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  PagedParams p{static_cast<const __nv_bfloat16*>(q), ld_q, ld_qh, cache, num_blocks, block_size, block_stride_bytes,
                block_table, ld_bt, n_pages, cu_rows, ctx_lens, B, 0, 0, mask, ld_mask, words, T, H, 0.f,
                static_cast<__nv_bfloat16*>(out), ld_out, ld_oh, lse, ld_lse};
  return paged_attention(fn, p, softmax_scale, ws, ws_bytes, true, stream);
}
