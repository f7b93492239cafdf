// Attention of every query row over the tokens selected for it, read from the
// attention cache through their slots.
//
// "DeepSeek V3.2 稀疏注意力 DSA 推理流程图解", data-flow items 2-3: the selection hands
// the main attention a list of cache slots per query row; all heads of the row
// attend to the same list and share the token's one latent (key: its 512 latent
// and 64 position dims, value: the latent).
#include <cuda_bf16.h>

#include <cmath>

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
};

constexpr int kTile = 32;
constexpr int kHeadGroup = 8;
constexpr int kKRow = kKvDim + 1;  // odd row length: a warp's 32 tokens fall into 32 banks

__global__ void __launch_bounds__(256) attention_simple_kernel(const AttnParams p) {
  extern __shared__ float sm[];
  float* ks = sm;                              // [kTile][kKRow]
  float* qs = ks + kTile * kKRow;              // [kHeadGroup][kKvDim]
  float* ps = qs + kHeadGroup * kKvDim;        // [kHeadGroup][kTile]
  float* corr = ps + kHeadGroup * kTile;       // [kHeadGroup]
  float* inv = corr + kHeadGroup;              // [kHeadGroup]
  const int t = blockIdx.x, h0 = blockIdx.y * kHeadGroup;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kHeadGroup * kKvDim; i += 256) {
    const int h = h0 + i / kKvDim;
    qs[i] = h < p.H ? __bfloat162float(p.q[t * p.ld_q + h * p.ld_qh + i % kKvDim]) : 0.f;
  }
  int n = p.k;
  if (p.n_sel) n = min(n, max(__ldg(p.n_sel + t), 0));
  float m = -INFINITY, l = 0.f;  // of head h0 + warp
  float acc[kHeadGroup][2] = {};
  for (int base = 0; base < n; base += kTile) {
    __syncthreads();
    for (int j = warp; j < kTile; j += 8) {
      int slot = base + j < n ? __ldg(p.slots + t * p.ld_slots + base + j) : -1;
      bool ok = slot >= 0;
      int blk = 0, off = 0;
      if (ok) {
        blk = slot / p.block_span;
        off = slot - blk * p.block_span;
        if (blk >= p.num_blocks || off >= p.block_size) {
          ok = false;
          if (lane == 0) atomicOr(&g_attention_error, 1u);
        }
      }
      if (lane == 0) ps[j] = ok ? 1.f : 0.f;
      const uint8_t* b = p.cache + blk * p.block_stride;
      uint32_t codes = ok ? __ldg(reinterpret_cast<const uint32_t*>(b + p.block_size * kKvScaleAt + 4 * off)) : 0u;
      for (int d = 4 * lane; d < kKvLatent; d += 128) {
        uint32_t w = ok ? __ldg(reinterpret_cast<const uint32_t*>(b + off * kKvLatent + d)) : 0u, lo, hi;
        kv_dequant4(w, kv_dequant_multiplier((codes >> (8 * (d / 128))) & 0xFFu), lo, hi);
        ks[j * kKRow + d] = __uint_as_float(lo << 16);
        ks[j * kKRow + d + 1] = __uint_as_float(lo & 0xFFFF0000u);
        ks[j * kKRow + d + 2] = __uint_as_float(hi << 16);
        ks[j * kKRow + d + 3] = __uint_as_float(hi & 0xFFFF0000u);
      }
      uint32_t w = ok ? __ldg(reinterpret_cast<const uint32_t*>(b + p.block_size * kKvRopeAt + off * 128 + 4 * lane)) : 0u;
      ks[j * kKRow + kKvLatent + 2 * lane] = __uint_as_float(w << 16);
      ks[j * kKRow + kKvLatent + 2 * lane + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
    __syncthreads();
    const bool ok = ps[lane] != 0.f;
    float s = 0.f;
    for (int d = 0; d < kKvDim; ++d) s = fmaf(qs[warp * kKvDim + d], ks[lane * kKRow + d], s);
    s = ok ? s * p.scale_log2 : -INFINITY;
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float m2 = fmaxf(m, top);
    const float e = ok ? exp2f(s - m2) : 0.f;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float c = m == -INFINITY ? 0.f : exp2f(m - m2);
    l = l * c + sum;
    m = m2;
    __syncthreads();
    ps[warp * kTile + lane] = e;
    if (lane == 0) corr[warp] = c;
    __syncthreads();
    for (int h = 0; h < kHeadGroup; ++h) {
      acc[h][0] *= corr[h];
      acc[h][1] *= corr[h];
      for (int j = 0; j < kTile; ++j) {
        const float w = ps[h * kTile + j];
        acc[h][0] = fmaf(w, ks[j * kKRow + 2 * tid], acc[h][0]);
        acc[h][1] = fmaf(w, ks[j * kKRow + 2 * tid + 1], acc[h][1]);
      }
    }
  }
  __syncthreads();
  if (lane == 0) {
    inv[warp] = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
    if (p.lse && h0 + warp < p.H) {
      p.lse[t * p.ld_lse + h0 + warp] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  for (int h = 0; h < kHeadGroup && h0 + h < p.H; ++h) {
    __nv_bfloat16* o = p.out + t * p.ld_out + (h0 + h) * p.ld_oh + 2 * tid;
    o[0] = __float2bfloat16_rn(acc[h][0] * inv[h]);
    o[1] = __float2bfloat16_rn(acc[h][1] * inv[h]);
  }
}

constexpr int kSimpleSmem = (kTile * kKRow + kHeadGroup * kKvDim + kHeadGroup * kTile + 2 * kHeadGroup) * 4;

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
  (void)T;
  (void)H;
  (void)k;
  return 0;
}

extern "C" idx_status_t idx_sparse_attention(const void* q, int64_t ld_q, int64_t ld_qh, const uint8_t* cache,
                                             int32_t num_blocks, int32_t block_size, int64_t block_stride_bytes,
                                             int32_t block_span, const int32_t* slots, int64_t ld_slots, int32_t k,
                                             const int32_t* n_sel, int32_t T, int32_t H, float softmax_scale,
                                             void* out, int64_t ld_out, int64_t ld_oh, float* lse, int64_t ld_lse,
                                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  const char* fn = "idx_sparse_attention";
  (void)ws;
  (void)ws_bytes;
  if (T < 0 || H < 0 || k < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H > IDX_ATTENTION_MAX_HEADS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d heads", fn, H);
  if (ld_slots < k || ld_q < kKvDim || ld_qh < kKvDim || ld_out < kKvLatent || ld_oh < kKvLatent || (lse && ld_lse < H)) {
    return fail(IDX_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  }
  if (!std::isfinite(softmax_scale)) return fail(IDX_ERR_INVALID_ARG, "%s: softmax_scale is not finite", fn);
  if (T == 0 || H == 0) return IDX_OK;
  if (!q || !cache || !out || (!slots && k > 0)) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  idx_status_t st = check_kv_cache(fn, cache, num_blocks, block_size, block_stride_bytes);
  if (st != IDX_OK) return st;
  if (block_span < block_size) return fail(IDX_ERR_UNSUPPORTED, "%s: block_span %d < block_size", fn, block_span);
  if (!aligned(q, 16) || ld_q % 8 != 0 || ld_qh % 8 != 0 || !aligned(out, 16) || ld_out % 8 != 0 || ld_oh % 8 != 0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: q and out rows must be 16-byte aligned", fn);
  }
  if (ws && !aligned(ws, 16)) return fail(IDX_ERR_UNSUPPORTED, "%s: the workspace is not 16-byte aligned", fn);
  AttnParams p{static_cast<const __nv_bfloat16*>(q), ld_q, ld_qh, cache, num_blocks, block_size, block_span,
               block_stride_bytes, slots, ld_slots, k, n_sel, T, H, softmax_scale * 1.4426950408889634f,
               static_cast<__nv_bfloat16*>(out), ld_out, ld_oh, lse, ld_lse};
  cudaError_t e = cudaFuncSetAttribute(attention_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSimpleSmem);
  if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  attention_simple_kernel<<<dim3(T, (H + kHeadGroup - 1) / kHeadGroup), 256, kSimpleSmem, stream>>>(p);
  return check_launch(fn);
}
