// Attention over whole contexts of the paged attention cache: within a sliding
// window and over a few first tokens (idx_window_attention), and of trees of drafted
// tokens (idx_tree_attention).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv_layout.cuh"

namespace idx {
namespace {

// Bit 0: a visible page outside the table or the cache (its tokens are skipped). Bit 1: a wait expired.
__device__ unsigned int g_paged_error = 0;

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
};

// ---------------------------------------------------------------------------
// One block per row and group of eight heads: tiles of 32 tokens dequantised into shared memory, a thread per
// (head, token) for the logits, two dims of every head a thread for the sums.
// ---------------------------------------------------------------------------
constexpr int kHeadsPerBlock = 8;
constexpr int kTile = 32;
constexpr int kThreads = 256;
constexpr int kPitch = kKvDim + 1;

struct Shared {
  float q[kHeadsPerBlock][kKvDim];
  float k[kTile][kPitch];
  float p[kHeadsPerBlock][kTile];
  int see[kTile];
};

template <bool kTree>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, h0 = blockIdx.y * kHeadsPerBlock;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_rows + mid) <= row) lo = mid; else hi = mid;
  }
  const int b = lo, first = __ldg(p.cu_rows + b), end = __ldg(p.cu_rows + b + 1);
  if (row < first || row >= end) return;
  const int64_t ctx = __ldg(p.ctx_lens + b), base = ctx - (end - first), pos = base + (row - first);
  // tokens [0, a) and [c, d) may be seen
  int64_t a, c, d;
  if (kTree) {
    a = 0, c = 0, d = ctx;
  } else {
    d = pos + 1;
    c = max(pos - p.window + 1, int64_t{0});
    a = min(static_cast<int64_t>(p.sinks), min(c, d));
  }
  for (int i = tid; i < kHeadsPerBlock * kKvDim; i += kThreads) {
    const int h = h0 + i / kKvDim;
    sh.q[i / kKvDim][i % kKvDim] =
        h < p.H ? __bfloat162float(p.q[row * p.ld_q + h * p.ld_qh + i % kKvDim]) * p.scale_log2 : 0.f;
  }
  float m = -INFINITY, l = 0.f;  // of head `warp`
  float acc[kHeadsPerBlock][2] = {};
  const int64_t n = a + max(d - c, int64_t{0});
  for (int64_t t0 = 0; t0 < n; t0 += kTile) {
    __syncthreads();
    for (int t = warp; t < kTile; t += kThreads / 32) {
      const int64_t i = t0 + t, j = i < a ? i : c + i - a;
      bool see = i < n;
      if (kTree && see && j >= base) {
        const int64_t node = j - base;
        see = node < 32 * p.words && (__ldg(p.mask + row * p.ld_mask + node / 32) >> (node % 32) & 1);
      }
      int blk = -1;
      if (see) {
        const int64_t page = j / p.block_size;
        if (page < p.n_pages) blk = __ldg(p.block_table + b * p.ld_bt + page);
        if (blk < 0 || blk >= p.num_blocks) {
          see = false;
          if (lane == 0) atomicOr(&g_paged_error, 1u);
        }
      }
      if (lane == 0) sh.see[t] = see;
      if (!see) {
        for (int x = lane; x < kKvDim; x += 32) sh.k[t][x] = 0.f;
        continue;
      }
      const int off = static_cast<int>(j % p.block_size);
      const uint8_t* base_ptr = p.cache + blk * p.block_stride;
      const uint32_t* lat = reinterpret_cast<const uint32_t*>(base_ptr + off * kKvLatent);
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(base_ptr + p.block_size * kKvScaleAt + 4 * off);
      const uint32_t* pe = reinterpret_cast<const uint32_t*>(base_ptr + p.block_size * kKvRopeAt + off * (2 * kKvRope));
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t w[2];
        kv_dequant4(lat[32 * x + lane], kv_dequant_multiplier((codes >> (8 * x)) & 0xFFu), w[0], w[1]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          sh.k[t][128 * x + 4 * lane + y] = __uint_as_float(y & 1 ? w[y / 2] & 0xFFFF0000u : w[y / 2] << 16);
        }
      }
      const uint32_t w = pe[lane];
      sh.k[t][kKvLatent + 2 * lane] = __uint_as_float(w << 16);
      sh.k[t][kKvLatent + 2 * lane + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
    __syncthreads();
    float s = 0.f;
    for (int x = 0; x < kKvDim; ++x) s = fmaf(sh.q[warp][x], sh.k[lane][x], s);
    if (!sh.see[lane]) s = -INFINITY;
    float top = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float m_new = fmaxf(m, top), ref = m_new == -INFINITY ? 0.f : m_new;
    const float f = exp2f(m - ref), e = exp2f(s - ref);
    m = m_new;
    float sum = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    l = l * f + sum;
    sh.p[warp][lane] = e;
    __shared__ float scale[kHeadsPerBlock];
    if (lane == 0) scale[warp] = f;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeadsPerBlock; ++h) {
      acc[h][0] *= scale[h];
      acc[h][1] *= scale[h];
    }
    for (int t = 0; t < kTile; ++t) {
      if (!sh.see[t]) continue;
      const float v0 = sh.k[t][2 * tid], v1 = sh.k[t][2 * tid + 1];
#pragma unroll
      for (int h = 0; h < kHeadsPerBlock; ++h) {
        acc[h][0] = fmaf(sh.p[h][t], v0, acc[h][0]);
        acc[h][1] = fmaf(sh.p[h][t], v1, acc[h][1]);
      }
    }
  }
  __shared__ float total[kHeadsPerBlock];
  if (lane == 0) {
    total[warp] = l;
    if (p.lse && h0 + warp < p.H) {
      p.lse[row * p.ld_lse + h0 + warp] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  for (int h = 0; h < kHeadsPerBlock && h0 + h < p.H; ++h) {
    const float inv = total[h] == 0.f ? 0.f : 1.0f / total[h];
    *reinterpret_cast<__nv_bfloat162*>(p.out + row * p.ld_out + (h0 + h) * p.ld_oh + 2 * tid) =
        __floats2bfloat162_rn(acc[h][0] * inv, acc[h][1] * inv);
  }
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
  (void)ws_bytes;
  auto* kernel = tree ? paged_attention_kernel<true> : paged_attention_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
  if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>((p.H + kHeadsPerBlock - 1) / kHeadsPerBlock));
  kernel<<<grid, kThreads, sizeof(Shared), stream>>>(p);
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
  (void)T;
  (void)B;
  (void)H;
  return 0;
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
