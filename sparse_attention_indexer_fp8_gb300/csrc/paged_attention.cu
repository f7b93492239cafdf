// Attention over whole contexts of the paged attention cache: within a sliding
// window and over a few first tokens (idx_window_attention), and of trees of drafted
// tokens (idx_tree_attention).
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "paged_attention.cuh"
#include "paged_block.cuh"
#include "paged_pair.cuh"

namespace idx {
namespace {

// How a call's rows are cut into units, and whether their contexts are split: where one wave has room for more parts
// than there are units.
struct Plan {
  bool pairs;
  int head_blocks, heads, tokens, capacity;
  int64_t units;
  int64_t part_floats, part_rows;  // of a part: accumulators, maxima and sums
};

// Joins the parts of each row (one head of one token), of a unit with half of the dims each half by itself: weights
// 2^(m_i - max m), a part without a visible token skipped (its accumulators were never written). That is the work of
// kWarps warps, each of which takes every kWarps-th part, two at a time: all rows of a batch run at once, and the loads
// of two parts are in flight together. Rows whose context was not split are complete already.
constexpr int kJoinWarps = 8;   // of a block
constexpr int kMaxParts = 160;

template <bool kPair, int kWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedParams p) {
  constexpr int kItems = kJoinWarps / kWarps;  // of a block
  constexpr int kHalves = kPair ? pair::kHalves : 1;
  constexpr int kDims = kKvLatent / kHalves, kVecs = kDims / 128;
  constexpr int kPartRows = kPair ? pair::kRows : block::kRows;
  __shared__ float4 sums[kItems][kWarps > 1 ? kWarps - 1 : 1][kDims / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp / kWarps, g = warp % kWarps;
  const uint32_t heads = static_cast<uint32_t>(p.H), item = blockIdx.x * kItems + sub;
  const int d = static_cast<int>(item % kHalves);
  const uint32_t head = item / kHalves;
  bool have = head < static_cast<uint32_t>(p.T) * heads;
  const int row = have ? static_cast<int>(head / heads) : 0, h = have ? static_cast<int>(head % heads) : 0;
  int lo = 0, hi = p.B;  // the last b with cu_rows[b] <= row
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const bool before = b < hi && (lane == 0 || row_at(p, b) <= row);
    lo += (__popc(__ballot_sync(0xFFFFFFFFu, before)) - 1) * step;
    hi = min(lo + step, hi);
  }
  const int at = row_at(p, lo), n = row_at(p, lo + 1) - at, in = row - at;
  have = have && in >= 0 && in < n;
  const int units = (n + p.tokens - 1) / p.tokens * p.head_blocks * kHalves;
  const int unit = (in / p.tokens * p.head_blocks + h / p.heads) * kHalves + d;
  int r = in % p.tokens;
  if (kPair) {
    const int own = p.tokens / 2;
    r = r / own * pair::kBlockRows + r % own * p.heads + h % p.heads;
  } else {
    r = r * p.heads + h % p.heads;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every part is complete and visible
  const int2 sched = have ? __ldcg(p.ws_sched + lo) : make_int2(0, 1);
  const int parts = min(sched.y, kMaxParts);
  have = have && parts > 1;
  const int64_t step = static_cast<int64_t>(units) * kPartRows;
  const int64_t first = static_cast<int64_t>(sched.x + unit) * kPartRows + r;
  const float2* ml = p.ws_ml + first;  // of part i: ml[step * i]
  const float4* o = reinterpret_cast<const float4*>(p.ws_o + first * kDims) + lane;

  float4 acc[kVecs] = {};
  float m = -INFINITY, l = 0.f;
  if (have) {
    float2 mine[kMaxParts / 32];
#pragma unroll
    for (int c = 0; c < kMaxParts / 32; ++c) {
      mine[c] = 32 * c + lane < parts ? __ldcg(ml + (32 * c + lane) * step) : make_float2(-INFINITY, 0.f);
      m = fmaxf(m, mine[c].x);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
#pragma unroll
    for (int c = 0; c < kMaxParts / 32; ++c) {
      if (mine[c].y != 0.f) l = fmaf(exp2f(mine[c].x - m), mine[c].y, l);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    for (int i = g; i < parts; i += 2 * kWarps) {
      float2 x[2];
      float4 v[2][kVecs];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int part = i + j * kWarps;
        x[j] = make_float2(-INFINITY, 0.f);
        if (part >= parts) continue;
        x[j] = __ldcg(ml + part * step);
#pragma unroll
        for (int c = 0; c < kVecs; ++c) v[j][c] = __ldcg(o + part * step * (kDims / 4) + 32 * c);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
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
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      if (g > 0) sums[sub][g - 1][lane + 32 * c] = acc[c];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < kWarps - 1; ++i) {
#pragma unroll
      for (int c = 0; c < kVecs; ++c) {
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
  __nv_bfloat16* dst = p.out + row * p.ld_out + h * p.ld_oh + d * kDims + 4 * lane;
#pragma unroll
  for (int c = 0; c < kVecs; ++c) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    *reinterpret_cast<uint2*>(dst + 128 * c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (p.lse && lane == 0 && d == 0) {
    p.lse[row * p.ld_lse + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, unsigned blocks, cudaStream_t stream) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 2;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(pair::kThreads);
  cfg.dynamicSmemBytes = pair::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Pairs that the current device runs at once; 0 when it cannot be queried.
int device_pairs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  auto* kernel = pair::paged_pair_kernel<false>;
  int n = 0;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pair_config(attr, 2, nullptr);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pair::kSmemBytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

Plan plan_of(int32_t T, int32_t B, int32_t H) {
  Plan plan{};
  const int per_request = T / B;  // query tokens, on average
  const char* env = getenv("IDX_PAIR");
  plan.pairs = env ? atoi(env) : static_cast<int64_t>(per_request) * H >= 192;
  const int rows = plan.pairs ? pair::kBlockRows : block::kRows;
  plan.head_blocks = (H + rows - 1) / rows;
  plan.heads = (H + plan.head_blocks - 1) / plan.head_blocks;
  plan.tokens = rows / plan.heads * (plan.pairs ? 2 : 1);
  const int each = plan.head_blocks * (plan.pairs ? pair::kHalves : 1);  // units of a group of tokens
  const int64_t groups = T / plan.tokens + static_cast<int64_t>(B);
  plan.units = groups * each;
  // no more groups hold rows: each request's last one may be part-filled
  const int64_t filled = std::min<int64_t>(T, groups) * each;
  const int room = plan.pairs ? device_pairs() : device_sm_count();
  plan.capacity = filled < room && B <= kMaxSplitRequests ? std::min(room, kMaxParts) : 0;
  plan.part_rows = plan.pairs ? pair::kRows : block::kRows;
  plan.part_floats = plan.part_rows * (plan.pairs ? pair::kDims : kKvLatent);
  return plan;
}

int64_t sched_bytes(int32_t B) { return (static_cast<int64_t>(B) * sizeof(int2) + 15) / 16 * 16; }

int64_t plan_bytes(const Plan& plan, int32_t B) {
  return plan.capacity ? sched_bytes(B) + plan.capacity * (plan.part_floats * 4 + plan.part_rows * 8) : 0;
}

template <bool kPair>
auto* join_kernel(int warps) {
  return warps == 1   ? paged_join_kernel<kPair, 1>
         : warps == 2 ? paged_join_kernel<kPair, 2>
         : warps == 4 ? paged_join_kernel<kPair, 4>
                      : paged_join_kernel<kPair, 8>;
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
  p.capacity = ws ? plan.capacity : 0;
  if (p.capacity) {
    const int64_t need = plan_bytes(plan, p.B);
    if (ws_bytes < static_cast<size_t>(need)) {
      return fail(IDX_ERR_INVALID_ARG, "%s: the workspace has %zu bytes, %lld are needed", fn, ws_bytes,
                  static_cast<long long>(need));
    }
    p.ws_sched = static_cast<int2*>(ws);
    p.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sched_bytes(p.B));
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + p.capacity * plan.part_floats);
  }
  const unsigned units = static_cast<unsigned>(p.capacity ? p.capacity : plan.units);
  cudaLaunchAttribute attr[1];
  cudaError_t e;
  if (plan.pairs) {
    auto* kernel = tree ? pair::paged_pair_kernel<true> : pair::paged_pair_kernel<false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pair::kSmemBytes);
    if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
    const cudaLaunchConfig_t cfg = pair_config(attr, 2 * units, stream);
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedParams>(p));
  } else {
    auto* kernel = tree ? block::paged_block_kernel<true> : block::paged_block_kernel<false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, block::kSmemBytes);
    if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
    kernel<<<units, block::kThreads, block::kSmemBytes, stream>>>(p);
    e = cudaSuccess;
  }
  if (e == cudaSuccess && p.capacity) {
    const idx_status_t launched = check_launch(fn);
    if (launched != IDX_OK) return launched;
    // Launched while the parts run: its blocks wait at their first reads for the parts' end. A warp takes some four of
    // the parts that a row has on average.
    const int64_t each = p.head_blocks * (plan.pairs ? pair::kHalves : 1);
    const int64_t parts = p.capacity / std::max<int64_t>(std::min<int64_t>(p.T, plan.units / each) * each, 1);
    const int warps = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;
    auto* join = plan.pairs ? join_kernel<true>(warps) : join_kernel<false>(warps);
    const int64_t items = static_cast<int64_t>(p.T) * p.H * (plan.pairs ? pair::kHalves : 1), per = kJoinWarps / warps;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((items + per - 1) / per));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join, static_cast<const PagedParams>(p));
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
  return static_cast<size_t>(plan_bytes(plan_of(T, B, H), B));
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
