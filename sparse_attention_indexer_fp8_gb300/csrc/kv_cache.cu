// The cache writers that also normalise and rotate, and the read-back of the
// attention cache.
//
// "DeepSeek V3.2 稀疏注意力 DSA 推理流程图解", "Indexer 内部六步": the indexer's k is
// LayerNorm'ed (k_norm), rotated on its first 64 dims and quantised into the
// indexer cache (steps 2, 3 and 5); the main attention's latent of the same token
// goes through its own RMSNorm, rotation and insert. Each is one pass here: the
// projection is read once, the record written once, nothing in between is stored.
// All three kernels move a few hundred bytes per token and are bound by memory
// for a prefill chunk and by launch latency for a decode batch, so a token is
// one warp's work: reductions are shuffles, no block waits for another.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv_layout.cuh"

namespace idx {
namespace {

constexpr int kWarpsPerBlock = 8;

// Bit 0: a position outside the cos/sin table (the token is written as zeros).
// Bit 1: a page of the block table outside the cache (the row is written as zeros).
__device__ unsigned int g_kv_cache_error = 0;

struct RopeArgs {
  const int32_t* positions;
  const float* cos_sin;  // [max_pos, ld_cs]: cos of the 32 pair angles, then their sin
  int64_t ld_cs;
  int max_pos;
  int interleaved;
};

__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// kN consecutive elements at p: one or two 16-byte loads (8 bytes for four bf16)
// when `vec`, else element loads.
template <bool kBf16, int kN>
__device__ __forceinline__ void load_run(const void* base, int64_t off, bool vec, float (&x)[kN]) {
  if constexpr (kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    if (vec) {
      uint32_t w[kN / 2];
      if constexpr (kN == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        x[2 * i] = bf16_bits(w[i] & 0xFFFFu);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = bf16_bits(__ldg(p + i));
    }
  } else {
    const float* p = static_cast<const float*>(base) + off;
    if (vec) {
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = __ldg(p + i);
    }
  }
}

__device__ __forceinline__ float4 load4(const float* p, bool vec) {
  return vec ? __ldg(reinterpret_cast<const float4*>(p))
             : make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
}

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* base, int64_t off) {
  if constexpr (kBf16) return bf16_bits(__ldg(static_cast<const uint16_t*>(base) + off));
  return __ldg(static_cast<const float*>(base) + off);
}

// Row of the angle table for token `tok`, or null outside the table.
__device__ __forceinline__ const float* angles(const RopeArgs& r, int tok) {
  const int pos = __ldg(r.positions + tok);
  return pos >= 0 && pos < r.max_pos ? r.cos_sin + static_cast<int64_t>(pos) * r.ld_cs : nullptr;
}

// Indexer k: y = LayerNorm(x) * weight + bias, the first 64 dims rotated, e4m3 with
// one scale per token, insert. Lane l owns dims 4l..4l+3 (as the plain insert
// does), so the rotary dims are lanes 0-15: NeoX pairs (i, i + 32) meet by one
// shuffle with lane l ^ 8, interleaved pairs lie in one lane. The variance is
// taken of the centred values (a second sum over registers), in binary32. The
// only chain of loads is position, then angles, and both are asked for before
// anything is used: a token costs two memory latencies, not four. Measured on a
// GB300 (bf16 in): 128 tokens 4.2 us, 8192 tokens 6.4 us (0.8 us of bytes; at 39
// registers 48 warps fit an SM, so these are 1.12 waves of two latencies each).
template <bool kBf16>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
k_norm_rope_quant_kernel(const void* __restrict__ k, int64_t ld_k, int n_tok, bool vec,
                         const float* __restrict__ weight, const float* __restrict__ bias, float eps,
                         const RopeArgs rope, bool ue8m0, const int64_t* __restrict__ slot_mapping,
                         uint8_t* __restrict__ cache, int64_t n_slots, int block_size, int64_t block_stride) {
  const int tok = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (tok >= n_tok) return;
  float x[4], y[4];
  const float* cs = angles(rope, tok);
  load_run<kBf16, 4>(k, static_cast<int64_t>(tok) * ld_k + 4 * lane, vec, x);
  const int64_t slot = __ldg(slot_mapping + tok);
  float wt[4], bs[4], co[4] = {}, si[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wt[i] = __ldg(weight + 4 * lane + i);
    bs[i] = bias ? __ldg(bias + 4 * lane + i) : 0.f;
  }
  if (lane < 16 && cs) {  // the angle of this lane's dim i: pair 2 l + i / 2, or 4 (l % 8) + i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = rope.interleaved ? 2 * lane + i / 2 : 4 * (lane & 7) + i;
      co[i] = __ldg(cs + pair);
      si[i] = __ldg(cs + 32 + pair);
    }
  }
  if (slot < 0 || slot >= n_slots) return;
  if (!cs && lane == 0) atomicOr(&g_kv_cache_error, 1u);

  const float mean = warp_sum((x[0] + x[1]) + (x[2] + x[3])) * (1.0f / kDim);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] -= mean;
    sq = fmaf(x[i], x[i], sq);
  }
  const float rstd = 1.0f / sqrtf(warp_sum(sq) * (1.0f / kDim) + eps);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = fmaf(x[i] * rstd, wt[i], bs[i]);
  }

  float other[4];  // NeoX: the partner lane's dims
#pragma unroll
  for (int i = 0; i < 4; ++i) other[i] = __shfl_xor_sync(0xFFFFFFFFu, y[i], 8);
  if (lane < 16) {
    if (rope.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float a = y[i], b = y[i + 1];
        y[i] = a * co[i] - b * si[i];
        y[i + 1] = b * co[i] + a * si[i];
      }
    } else {
      const float sign = lane < 8 ? -1.f : 1.f;  // first member: a c - b s; second: b c + a s
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = y[i] * co[i] + sign * (other[i] * si[i]);
    }
  }
  if (!cs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = 0.f;
  }

  float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  float scale = __fdiv_rn(amax, 448.0f);
  if (ue8m0) scale = ue8m0_ceil(scale);
  uint32_t packed = 0;
  if (scale >= 0x1p-126f) {
    const float r = __frcp_rn(scale);
    packed = e4m3x2_of_quotients(y[0], y[1], scale, r) | (e4m3x2_of_quotients(y[2], y[3], scale, r) << 16);
  } else if (scale != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) packed |= e4m3_of_quotient_exact(y[i], scale) << (8 * i);
  }
  const int64_t blk = slot / block_size;
  const int off = static_cast<int>(slot - blk * block_size);
  uint8_t* base = cache + blk * block_stride;
  *reinterpret_cast<uint32_t*>(base + off * kDim + 4 * lane) = packed;
  if (lane == 0) *reinterpret_cast<float*>(base + block_size * kDim + 4 * off) = scale;
}

// E8M0 code of a 128-dim tile: the smallest power of two >= amax / 448, held to
// 2^-127 .. 2^7 (code 0 .. 134). The upper end makes one bf16 multiplication
// by 2^(code - 7) dequantise a value exactly (kv_layout.cuh); it saturates
// latents beyond 57344. `amax` is the bit pattern of the largest |value|: as whole numbers the patterns are
// ordered as the values are, infinity above them and NaN above infinity, so the maximum of a tile
// says whether all of it is finite (fmaxf would pass over a NaN).
__device__ __forceinline__ uint32_t kv_scale_code(uint32_t amax) {
  if (amax >= 0x7F800000u) return kKvNanScaleCode;
  const uint32_t b = __float_as_uint(ue8m0_ceil(__fdiv_rn(__uint_as_float(amax), 448.0f)));
  return min(b >> 23, static_cast<uint32_t>(kKvMaxScaleCode));
}

// Eight dims as e4m3 under a power-of-two scale: the product by 2^(127 - code) is
// exact (up to results far below e4m3's smallest step), so the code is the
// definition's round-to-nearest-even of y / scale. Zeros under the code for NaN.
__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8], uint32_t code) {
  if (code == kKvNanScaleCode) return make_uint2(0u, 0u);
  // 2^(127 - code), code <= 134: exponent field 254 - code, a normal float
  const float inv = __uint_as_float((254u - code) << 23);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv, y[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Attention latent: RMSNorm of 512 dims (weight optional), rotation of the 64
// position dims (optional), e4m3 with one E8M0 scale per 128 dims, insert. Lane l
// owns dims 8l..8l+7 and 256 + 8l..+7, so each of the two loads and stores of the
// warp is one contiguous run and a scale's tile is half a warp. Of the position
// dims it owns one pair. Measured on a GB300 (bf16 in): 128 tokens 4.2 us, 8192
// tokens 8.3 us (2.5 us of bytes; at 43 registers 40 warps fit an SM: 1.35 waves;
// with the angles asked for after the slot 11.3).
template <bool kBf16>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
kv_norm_rope_quant_kernel(const void* __restrict__ c, int64_t ld_c, const void* __restrict__ pe, int64_t ld_pe,
                          int n_tok, bool vec, const float* __restrict__ weight, bool vec_w, float eps,
                          const RopeArgs rope,
                          const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ cache,
                          int64_t n_slots, int block_size, int64_t block_stride) {
  const int tok = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (tok >= n_tok) return;
  float x[2][8];
  const float* cs = rope.positions ? angles(rope, tok) : nullptr;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_run<kBf16, 8>(c, static_cast<int64_t>(tok) * ld_c + 256 * h + 8 * lane, vec, x[h]);
  }
  const int ia = rope.interleaved ? 2 * lane : lane;
  const int ib = rope.interleaved ? 2 * lane + 1 : lane + 32;
  float a = load_one<kBf16>(pe, static_cast<int64_t>(tok) * ld_pe + ia);
  float b = load_one<kBf16>(pe, static_cast<int64_t>(tok) * ld_pe + ib);
  const int64_t slot = __ldg(slot_mapping + tok);
  float co = 1.f, si = 0.f;
  if (cs) {
    co = __ldg(cs + lane);
    si = __ldg(cs + 32 + lane);
  }
  if (slot < 0 || slot >= n_slots) return;
  const bool zero = rope.positions && !cs;
  if (zero && lane == 0) atomicOr(&g_kv_cache_error, 1u);
  if (cs) {
    const float u = a * co - b * si;
    b = b * co + a * si;
    a = u;
  }
  if (weight) {
    float sq = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(x[h][i], x[h][i], sq);
    }
    const float rstd = 1.0f / sqrtf(warp_sum(sq) * (1.0f / kKvLatent) + eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 wt = load4(weight + 256 * h + 8 * lane + i, vec_w);
        x[h][i] *= rstd * wt.x;
        x[h][i + 1] *= rstd * wt.y;
        x[h][i + 2] *= rstd * wt.z;
        x[h][i + 3] *= rstd * wt.w;
      }
    }
  }
  if (zero) {
    a = b = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[h][i] = 0.f;
    }
  }

  const int64_t blk = slot / block_size;
  const int off = static_cast<int>(slot - blk * block_size);
  uint8_t* base = cache + blk * block_stride;
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[h][i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    code[h] = kv_scale_code(amax);
    *reinterpret_cast<uint2*>(base + off * kKvLatent + 256 * h + 8 * lane) = e4m3x8(x[h], code[h]);
  }
  // the four codes as one word: tiles 0, 1 from lanes 0, 16 of the first half, 2, 3 of the second
  const uint32_t hi0 = __shfl_sync(0xFFFFFFFFu, code[0], 16), hi1 = __shfl_sync(0xFFFFFFFFu, code[1], 16);
  if (lane == 0) {
    *reinterpret_cast<uint32_t*>(base + block_size * kKvScaleAt + 4 * off) =
        code[0] | (hi0 << 8) | (code[1] << 16) | (hi1 << 24);
  }
  __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(base + block_size * kKvRopeAt + off * (2 * kKvRope));
  row[ia] = __float2bfloat16_rn(a);
  row[ib] = __float2bfloat16_rn(b);
}

// Read-back: row r of the packed output holds token starts[b] + (r - cu[b]) of the
// request b whose range [cu[b], cu[b + 1]) covers r. One warp takes kGatherRows
// consecutive rows: one search of the ranges, then all rows' loads before any
// store, which keeps enough bytes in flight. Lane l moves dims 8l..8l+7 and
// 256 + 8l..+7 (every load and store of the warp one contiguous run), lanes 0-7
// also 8 position dims each. Bound by HBM: 184 K tokens of eight requests take
// 57.4 us (5.75 TB/s of records read and rows written, 0.86 of the measured copy rate;
// two rows a warp 57.2, one 61.2).
constexpr int kGatherRows = 4;

template <bool kBf16>
__device__ __forceinline__ void store8(void* out, int64_t at, const uint32_t (&w)[4]) {
  if constexpr (kBf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      p[i] = make_float4(bf16_bits(w[2 * i] & 0xFFFFu), __uint_as_float(w[2 * i] & 0xFFFF0000u),
                         bf16_bits(w[2 * i + 1] & 0xFFFFu), __uint_as_float(w[2 * i + 1] & 0xFFFF0000u));
    }
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
gather_kv_kernel(const uint8_t* __restrict__ cache, int num_blocks, int block_size, int64_t block_stride,
                 const int32_t* __restrict__ block_table, int64_t ld_bt, int n_pages,
                 const int32_t* __restrict__ starts, const int32_t* __restrict__ cu, int B, void* __restrict__ out, int64_t ld_out, int n_out) {
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5)) * kGatherRows;
  const int lane = threadIdx.x & 31;
  if (r0 >= n_out) return;
  // the last b in [0, B) with cu[b] <= r0
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= r0) lo = mid; else hi = mid;
  }
  uint2 v[kGatherRows][2];
  uint4 pe[kGatherRows];
  uint32_t codes[kGatherRows];
  int state[kGatherRows];  // 0: not a row of any request, 1: a token, 2: a bad page
  int b = lo;
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    const int64_t r = r0 + i;
    state[i] = 0;
    v[i][0] = v[i][1] = make_uint2(0u, 0u);
    pe[i] = make_uint4(0u, 0u, 0u, 0u);
    codes[i] = 0;
    if (r >= n_out) continue;
    while (b + 1 < B && __ldg(cu + b + 1) <= r) ++b;
    const int first = __ldg(cu + b);
    if (r < first || r >= __ldg(cu + b + 1)) continue;
    const int64_t p = (r - first) + (starts ? __ldg(starts + b) : 0);
    const int64_t page = p / block_size;
    int blk = -1;
    if (p >= 0 && page < n_pages) blk = __ldg(block_table + b * ld_bt + page);
    if (blk < 0 || blk >= num_blocks) {
      state[i] = 2;
      continue;
    }
    state[i] = 1;
    const int off = static_cast<int>(p - page * block_size);
    const uint8_t* base = cache + blk * block_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[i][h] = __ldg(reinterpret_cast<const uint2*>(base + off * kKvLatent + 256 * h + 8 * lane));
    }
    codes[i] = __ldg(reinterpret_cast<const uint32_t*>(base + block_size * kKvScaleAt + 4 * off));
    if (lane < 8) {
      pe[i] = __ldg(reinterpret_cast<const uint4*>(base + block_size * kKvRopeAt + off * (2 * kKvRope) + 16 * lane));
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    if (state[i] == 0) continue;
    if (state[i] == 2 && lane == 0) atomicOr(&g_kv_cache_error, 2u);
    const int64_t row = (r0 + i) * ld_out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t mul = kv_dequant_multiplier((codes[i] >> (8 * (2 * h + (lane >> 4)))) & 0xFFu);
      uint32_t w[4];
      kv_dequant4(v[i][h].x, mul, w[0], w[1]);
      kv_dequant4(v[i][h].y, mul, w[2], w[3]);
      store8<kBf16>(out, row + 256 * h + 8 * lane, w);
    }
    if (lane < 8) {
      const uint32_t w[4] = {pe[i].x, pe[i].y, pe[i].z, pe[i].w};
      store8<kBf16>(out, row + kKvLatent + 8 * lane, w);
    }
  }
}

bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

idx_status_t check_rope(const char* fn, const int32_t* positions, const float* cos_sin, int64_t ld_cs,
                        int32_t max_pos, int32_t rope_style) {
  if (rope_style != IDX_ROPE_NEOX && rope_style != IDX_ROPE_INTERLEAVED) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: rope_style %d", fn, rope_style);
  }
  if (!positions != !cos_sin) {
    return fail(IDX_ERR_INVALID_ARG, "%s: positions and cos_sin go together", fn);
  }
  if (positions && (max_pos < 1 || ld_cs < 64)) {
    return fail(IDX_ERR_INVALID_ARG, "%s: max_pos < 1 or ld_cs < 64", fn);
  }
  return IDX_OK;
}

}  // namespace

idx_status_t check_kv_cache(const char* fn, const void* cache, int32_t num_blocks, int32_t block_size,
                            int64_t block_stride) {
  if (num_blocks < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative num_blocks", fn);
  if (!block_size_ok(block_size)) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: block_size %d is not one of 16, 32, 64, 128", fn, block_size);
  }
  if (block_stride < static_cast<int64_t>(block_size) * IDX_KV_TOKEN_BYTES) {
    return fail(IDX_ERR_INVALID_ARG, "%s: block_stride_bytes %lld < block_size * 644", fn,
                static_cast<long long>(block_stride));
  }
  if (block_stride % 16 != 0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: block_stride_bytes %lld is not a multiple of 16", fn,
                static_cast<long long>(block_stride));
  }
  if (!aligned(cache, 16)) return fail(IDX_ERR_UNSUPPORTED, "%s: cache is not 16-byte aligned", fn);
  return IDX_OK;
}

unsigned int kv_cache_read_and_clear_error(cudaStream_t stream, cudaError_t* err) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  *err = cudaStreamSynchronize(stream);
  if (*err != cudaSuccess) return 0;
  *err = cudaMemcpyFromSymbol(&v, g_kv_cache_error, sizeof(v));
  if (*err != cudaSuccess) return 0;
  if (v) *err = cudaMemcpyToSymbol(g_kv_cache_error, &zero, sizeof(zero));
  return v;
}

}  // namespace idx

using namespace idx;

extern "C" idx_status_t idx_k_norm_rope_quant_and_cache(
    const void* k, int k_dtype, int64_t ld_k, int32_t n_tok, const float* weight, const float* bias, float eps,
    const int32_t* positions, const float* cos_sin, int64_t ld_cs, int32_t max_pos, int32_t rope_style,
    const int64_t* slot_mapping, uint8_t* cache, int32_t num_blocks, int32_t block_size,
    int64_t block_stride_bytes, int scale_fmt, cudaStream_t stream) {
  const char* fn = "idx_k_norm_rope_quant_and_cache";
  if (n_tok < 0 || num_blocks < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (k_dtype != IDX_BF16 && k_dtype != IDX_F32) return fail(IDX_ERR_UNSUPPORTED, "%s: k_dtype %d", fn, k_dtype);
  if (scale_fmt != IDX_SCALE_FP32 && scale_fmt != IDX_SCALE_UE8M0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: scale_fmt %d", fn, scale_fmt);
  }
  if (ld_k < kDim) return fail(IDX_ERR_INVALID_ARG, "%s: ld_k %lld < 128", fn, static_cast<long long>(ld_k));
  if (!(eps >= 0.f)) return fail(IDX_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (n_tok == 0) return IDX_OK;
  if (!k || !weight || !positions || !cos_sin || !slot_mapping || !cache) {
    return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  }
  idx_status_t st = check_rope(fn, positions, cos_sin, ld_cs, max_pos, rope_style);
  if (st != IDX_OK) return st;
  if (!block_size_ok(block_size)) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: block_size %d is not one of 16, 32, 64, 128", fn, block_size);
  }
  if (block_stride_bytes < static_cast<int64_t>(block_size) * kTokenBytes) {
    return fail(IDX_ERR_INVALID_ARG, "%s: block_stride_bytes %lld < block_size * 132", fn,
                static_cast<long long>(block_stride_bytes));
  }
  if (block_stride_bytes % 16 != 0 || !aligned(cache, 16)) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: cache blocks must be 16-byte aligned", fn);
  }
  const bool bf16 = k_dtype == IDX_BF16;
  const size_t vec_bytes = bf16 ? 8 : 16;
  const bool vec = aligned(k, vec_bytes) && ld_k % 4 == 0;
  const int64_t n_slots = static_cast<int64_t>(num_blocks) * block_size;
  const RopeArgs rope{positions, cos_sin, ld_cs, max_pos, rope_style == IDX_ROPE_INTERLEAVED};
  const dim3 grid((static_cast<unsigned>(n_tok) + kWarpsPerBlock - 1) / kWarpsPerBlock);
  auto* kernel = bf16 ? k_norm_rope_quant_kernel<true> : k_norm_rope_quant_kernel<false>;
  kernel<<<grid, kWarpsPerBlock * 32, 0, stream>>>(k, ld_k, n_tok, vec, weight, bias, eps, rope,
                                                   scale_fmt == IDX_SCALE_UE8M0, slot_mapping, cache, n_slots,
                                                   block_size, block_stride_bytes);
  return check_launch(fn);
}

extern "C" idx_status_t idx_kv_norm_rope_quant_and_cache(
    const void* c, int64_t ld_c, const void* pe, int64_t ld_pe, int dtype, int32_t n_tok, const float* weight,
    float eps, const int32_t* positions, const float* cos_sin, int64_t ld_cs, int32_t max_pos,
    int32_t rope_style, const int64_t* slot_mapping, uint8_t* cache, int32_t num_blocks, int32_t block_size,
    int64_t block_stride_bytes, cudaStream_t stream) {
  const char* fn = "idx_kv_norm_rope_quant_and_cache";
  if (n_tok < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative n_tok", fn);
  if (dtype != IDX_BF16 && dtype != IDX_F32) return fail(IDX_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (ld_c < kKvLatent || ld_pe < kKvRope) {
    return fail(IDX_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  }
  if (!(eps >= 0.f)) return fail(IDX_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  idx_status_t st = check_rope(fn, positions, cos_sin, ld_cs, max_pos, rope_style);
  if (st != IDX_OK) return st;
  if (n_tok == 0) return IDX_OK;
  if (!c || !pe || !slot_mapping || !cache) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  st = check_kv_cache(fn, cache, num_blocks, block_size, block_stride_bytes);
  if (st != IDX_OK) return st;
  const bool bf16 = dtype == IDX_BF16;
  const bool vec = aligned(c, 16) && ld_c % (bf16 ? 8 : 4) == 0;
  const int64_t n_slots = static_cast<int64_t>(num_blocks) * block_size;
  const RopeArgs rope{positions, cos_sin, ld_cs, max_pos, rope_style == IDX_ROPE_INTERLEAVED};
  const dim3 grid((static_cast<unsigned>(n_tok) + kWarpsPerBlock - 1) / kWarpsPerBlock);
  auto* kernel = bf16 ? kv_norm_rope_quant_kernel<true> : kv_norm_rope_quant_kernel<false>;
  kernel<<<grid, kWarpsPerBlock * 32, 0, stream>>>(c, ld_c, pe, ld_pe, n_tok, vec, weight, aligned(weight, 16),
                                                   eps, rope, slot_mapping,
                                                   cache, n_slots, block_size, block_stride_bytes);
  return check_launch(fn);
}

extern "C" idx_status_t idx_gather_kv(const uint8_t* cache, int32_t num_blocks, int32_t block_size,
                                      int64_t block_stride_bytes, const int32_t* block_table, int64_t ld_bt,
                                      int32_t n_pages, const int32_t* starts, const int32_t* cu_lens, int32_t B,
                                      void* out, int out_dtype, int64_t ld_out, int32_t n_out, cudaStream_t stream) {
  const char* fn = "idx_gather_kv";
  if (B < 0 || n_out < 0 || n_pages < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (out_dtype != IDX_BF16 && out_dtype != IDX_F32) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: out_dtype %d", fn, out_dtype);
  }
  if (ld_out < kKvDim || ld_bt < n_pages) {
    return fail(IDX_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  }
  if (B == 0 || n_out == 0) return IDX_OK;
  if (!cache || !block_table || !cu_lens || !out) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  idx_status_t st = check_kv_cache(fn, cache, num_blocks, block_size, block_stride_bytes);
  if (st != IDX_OK) return st;
  const bool bf16 = out_dtype == IDX_BF16;
  if (!aligned(out, 16) || ld_out % (bf16 ? 8 : 4) != 0) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: out rows must be 16-byte aligned", fn);
  }
  const int per_block = kWarpsPerBlock * kGatherRows;
  const dim3 grid((static_cast<unsigned>(n_out) + per_block - 1) / per_block);
  auto* kernel = bf16 ? gather_kv_kernel<true> : gather_kv_kernel<false>;
  kernel<<<grid, kWarpsPerBlock * 32, 0, stream>>>(cache, num_blocks, block_size, block_stride_bytes, block_table,
                                                   ld_bt, n_pages, starts, cu_lens, B, out, ld_out, n_out);
  return check_launch(fn);
}
