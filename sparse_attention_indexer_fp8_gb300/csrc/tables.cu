// What a step's other calls index by, computed from lengths on the GPU: block
// tables, slots, positions and row ranges (idx_build_tables), and the ancestors of
// the drafted tokens of a tree (idx_tree_mask).
#include <algorithm>

#include "common.cuh"

namespace idx {
namespace {

// Bit 0: a length, a page count or free_start out of its range. Bit 1: free_blocks ran out. Bit 2: a context
// longer than the table. Bit 3: more rows than n_rows. Bit 4: a tree's parent, or a node without a bit.
__device__ unsigned int g_tables_error = 0;

struct TableParams {
  const int32_t* cached;
  const int32_t* add;
  const int32_t* held;
  int B;
  const int32_t* free_blocks;
  int n_free;
  const int32_t* free_start;
  int32_t* table;
  int64_t ld_bt;
  int n_pages;
  int shift;  // log2(block_size)
  int32_t* ctx_lens;
  int32_t* cu_rows;
  int32_t* cu_ctx;
  int32_t* held_out;
  int32_t* free_end;
  int32_t* positions;
  int64_t* slots;
  int32_t* row_to_req;
  int32_t* row_ke;
  int n_rows;
};

// ---------------------------------------------------------------------------
// Block tables and slot maps
//
// Three sums over the requests (new rows, context lengths, fresh blocks) give every offset, and everything
// else follows from a row's or a fresh page's request, found by bisection of the sums:
//   row i of request b       position cached[b] + i, slot table[b][position / bs] * bs + position % bs
//   fresh page j of b        block free_blocks[start + (fresh blocks of the requests before b) + j].
// Bytes are few (20 written a row), so launches and round trips decide: one launch, in which every block
// computes the sums of all requests by itself. Outputs may overwrite the lengths they come from, so no block
// writes before all have read: one block needs its own barrier for that, several are one cluster. A slot
// in a fresh page comes from free_blocks, not from the table, which another block writes.
//
// One block while every thread has one row and one request at most, 3.4 us for a decode step of 128 requests; a cluster of
// eight above. One block and a cluster take, for 900 rows of 16 requests 3.9 and 4.3 us, for 1152 4.7 and 4.5, for 2048
// 5.0 and 4.6; for 900 requests of a row 5.7 and 6.1 us, for 1152 8.3 and 7.9, for 2047 9.4 and 8.5; one request of 1152 to
// 1408 rows alone is better off in one block (4.1 and 4.2 us). 44216 rows of 256 requests take 39.2 and 9.6 us (1.3 MB
// written there; the bisections' shared-memory reads bound it).
// ---------------------------------------------------------------------------
constexpr int kClusterBlocks = 8;  // the portable cluster size
constexpr int kMaxTableThreads = 1024;
constexpr size_t kTableSmemUnasked = 47 * 1024;  // with warp_sums, 48 KB are a block's without asking for more

constexpr size_t table_smem_bytes(int requests) { return (5 * static_cast<size_t>(requests) + 2) * sizeof(int32_t); }

// The last b in [0, n) with first[b] <= i, for first[0] <= i.
__device__ __forceinline__ int last_at_most(const int32_t* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t to_int32(int64_t v) { return static_cast<int32_t>(min(v, static_cast<int64_t>(INT32_MAX))); }

template <bool kCluster>
__global__ void __launch_bounds__(kMaxTableThreads) build_tables_kernel(const TableParams p) {
  extern __shared__ int32_t table_smem[];
  int32_t* rows_at = table_smem;            // [B + 1] first row of each request
  int32_t* fresh_at = rows_at + p.B + 1;    // [B + 1] its first fresh block, counted from free_start
  int32_t* cached_s = fresh_at + p.B + 1;   // [B]
  int32_t* held_s = cached_s + p.B;         // [B]
  int32_t* ctx_s = held_s + p.B;            // [B] kept apart: the sums may be held to 2^31 - 1
  __shared__ int64_t warp_sums[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int rank = kCluster ? static_cast<int>(blockIdx.x) : 0;
  const int step = kCluster ? kClusterBlocks * static_cast<int>(blockDim.x) : static_cast<int>(blockDim.x);
  const int me = rank * static_cast<int>(blockDim.x) + tid;
  unsigned int bad = 0;

  int start = p.free_start ? *p.free_start : 0;
  if (start < 0) {
    start = 0;
    bad |= 1u;
  }
  int64_t carry[3] = {0, 0, 0};  // new rows, fresh blocks, context lengths of the requests before this pass's
  for (int base = 0; base < p.B; base += blockDim.x) {
    const int b = base + tid;
    int64_t v[3] = {0, 0, 0};
    int cached = 0, held = 0;
    if (b < p.B) {
      cached = p.cached[b];
      int add = p.add[b];
      if (cached < 0 || add < 0 || static_cast<int64_t>(cached) + add > INT32_MAX) {
        bad |= 1u;
        cached = add = 0;
      }
      const int64_t bs = int64_t{1} << p.shift;
      held = p.held ? p.held[b] : static_cast<int>(min((cached + bs - 1) >> p.shift, static_cast<int64_t>(p.n_pages)));
      if (held < 0 || held > p.n_pages) {
        bad |= 1u;
        held = min(max(held, 0), p.n_pages);
      }
      const int64_t ctx = static_cast<int64_t>(cached) + add;
      const int64_t pages = (ctx + bs - 1) >> p.shift;
      if (pages > p.n_pages) bad |= 4u;
      v[0] = add;
      v[1] = max(min(pages, static_cast<int64_t>(p.n_pages)) - held, int64_t{0});
      v[2] = ctx;
    }
    int64_t s[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      s[k] = v[k];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, s[k], d);
        if (lane >= d) s[k] += o;
      }
      if (lane == 31) warp_sums[k][warp] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int64_t w = lane < warps ? warp_sums[k][lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
        if (lane >= d) w += o;
      }
      const int64_t before = __shfl_sync(0xFFFFFFFFu, w, max(warp - 1, 0));
      s[k] += carry[k] + (warp > 0 ? before : 0);
      carry[k] += __shfl_sync(0xFFFFFFFFu, w, 31);
    }
    __syncthreads();  // warp_sums may be written again
    if (b < p.B) {
      rows_at[b] = to_int32(s[0] - v[0]);
      fresh_at[b] = to_int32(s[1] - v[1]);
      cached_s[b] = cached;
      held_s[b] = held;
      ctx_s[b] = static_cast<int>(v[2]);
    }
    // cu_ctx is none of the inputs, so it is written at once
    if (rank == 0 && p.cu_ctx && b < p.B) {
      p.cu_ctx[b + 1] = to_int32(s[2]);
      if (s[2] > INT32_MAX) bad |= 1u;
    }
  }
  if (tid == 0) {
    rows_at[p.B] = to_int32(carry[0]);
    fresh_at[p.B] = to_int32(carry[1]);
  }
  if (carry[0] > p.n_rows) bad |= 8u;
  if (carry[1] > static_cast<int64_t>(p.n_free) - start && carry[1] > 0) bad |= 2u;
  if (kCluster) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (rank == 0 && bad) atomicOr(&g_tables_error, bad);

  const int total_rows = rows_at[p.B], total_fresh = fresh_at[p.B];
  const int available = max(p.n_free - start, 0);
  for (int b = me; b <= p.B; b += step) {
    p.cu_rows[b] = rows_at[b];
    if (b == p.B) break;
    p.ctx_lens[b] = ctx_s[b];
    if (p.held_out) {
      const int need = fresh_at[b + 1] - fresh_at[b];
      p.held_out[b] = held_s[b] + min(need, max(available - fresh_at[b], 0));
    }
  }
  if (me == 0) {
    if (p.cu_ctx) p.cu_ctx[0] = 0;
    if (p.free_end) *p.free_end = start + min(total_fresh, available);
  }
  for (uint32_t i = me; i < static_cast<uint32_t>(total_fresh); i += step) {
    const int f = static_cast<int>(i), b = last_at_most(fresh_at, p.B, f);
    const int page = held_s[b] + (f - fresh_at[b]);
    p.table[b * p.ld_bt + page] = f < available ? __ldg(p.free_blocks + start + f) : -1;
  }
  const int mask = (1 << p.shift) - 1;
  for (uint32_t i = me; i < static_cast<uint32_t>(p.n_rows); i += step) {
    const int r = static_cast<int>(i);
    int pos = 0, req = 0, ke = 0;
    int64_t slot = -1;
    if (r < total_rows) {
      req = last_at_most(rows_at, p.B, r);
      pos = cached_s[req] + (r - rows_at[req]);  // each sum on the way fits too
      ke = pos + 1;
      const int page = pos >> p.shift;
      int block = -1;
      if (page < held_s[req]) {
        block = p.table[req * p.ld_bt + page];
      } else if (page < p.n_pages) {
        const int f = fresh_at[req] + (page - held_s[req]);
        if (f < available) block = __ldg(p.free_blocks + start + f);
      }
      if (block >= 0) slot = (static_cast<int64_t>(block) << p.shift) + (pos & mask);
    }
    p.positions[r] = pos;
    p.slots[r] = slot;
    if (p.row_to_req) p.row_to_req[r] = req;
    if (p.row_ke) p.row_ke[r] = ke;
  }
}

// ---------------------------------------------------------------------------
// Ancestors of the nodes of drafted trees
//
// One block per request, one thread per node: it climbs from the node to the root through the parents in shared
// memory. Ancestors have falling indices, so the words of a row are finished one after the other, from
// its own down to word 0, and each is written once.
// 1.8 us for 8 trees of 16 nodes, 2.7 us for 128 of 64: the launch, and the climb's dependent reads.
// ---------------------------------------------------------------------------
constexpr int kTreeThreads = 128;
constexpr int kTreeNodes = 32 * IDX_TREE_MAX_WORDS;

__global__ void __launch_bounds__(kTreeThreads)
tree_mask_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ cu_rows, int n_rows,
                 const int32_t* __restrict__ base_lens, int32_t* __restrict__ mask, int64_t ld_mask, int words,
                 int32_t* __restrict__ positions) {
  __shared__ int16_t up[kTreeNodes];
  const int b = blockIdx.x;
  const int first = min(max(__ldg(cu_rows + b), 0), n_rows), end = min(max(__ldg(cu_rows + b + 1), first), n_rows);
  const int n = end - first, known = min(n, 32 * words);
  const int base = base_lens ? __ldg(base_lens + b) : 0;
  bool bad = n > known;
  for (int i = threadIdx.x; i < known; i += kTreeThreads) {
    int parent = __ldg(parents + first + i);
    if (parent < -1 || parent >= i) {
      bad = true;
      parent = -1;
    }
    up[i] = static_cast<int16_t>(parent);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kTreeThreads) {
    int32_t* row = mask + (first + i) * ld_mask;
    int depth = 0, at = i < known ? i : -1;
    if (at < 0) depth = 1;  // a node without a bit sees nothing, and counts as a root
    for (int w = words - 1; w >= 0; --w) {
      uint32_t bits = 0;
      while (at >= 32 * w) {
        bits |= 1u << (at & 31);
        at = up[at];
        ++depth;
      }
      row[w] = static_cast<int32_t>(bits);
    }
    if (positions) positions[first + i] = base + depth - 1;
  }
  if (bad) atomicOr(&g_tables_error, 16u);
}

}  // namespace

unsigned int tables_read_and_clear_error(cudaStream_t stream, cudaError_t* err) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  *err = cudaStreamSynchronize(stream);
  if (*err != cudaSuccess) return 0;
  *err = cudaMemcpyFromSymbol(&v, g_tables_error, sizeof(v));
  if (*err != cudaSuccess) return 0;
  if (v) *err = cudaMemcpyToSymbol(g_tables_error, &zero, sizeof(zero));
  return v;
}

}  // namespace idx

using namespace idx;

extern "C" idx_status_t idx_build_tables(const int32_t* cached_lens, const int32_t* new_lens, const int32_t* held_pages,
                                         int32_t B, const int32_t* free_blocks, int32_t n_free,
                                         const int32_t* free_start, int32_t* block_table, int64_t ld_bt,
                                         int32_t n_pages, int32_t block_size, int32_t* ctx_lens, int32_t* cu_rows,
                                         int32_t* cu_ctx, int32_t* held_out, int32_t* free_end, int32_t* positions,
                                         int64_t* slot_mapping, int32_t* row_to_req, int32_t* row_ke, int32_t n_rows,
                                         cudaStream_t stream) {
  const char* fn = "idx_build_tables";
  if (B < 0 || n_free < 0 || n_pages < 0 || n_rows < 0) return fail(IDX_ERR_INVALID_ARG, "%s: negative size", fn);
  if (B > IDX_TABLES_MAX_REQUESTS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d requests", fn, B);
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) {
    return fail(IDX_ERR_UNSUPPORTED, "%s: block_size %d is not one of 16, 32, 64, 128", fn, block_size);
  }
  if (static_cast<int64_t>(B) * n_pages > INT32_MAX) {  // fresh blocks of all requests are numbered in 32 bits
    return fail(IDX_ERR_UNSUPPORTED, "%s: a table of %d x %d entries", fn, B, n_pages);
  }
  if (ld_bt < n_pages) return fail(IDX_ERR_INVALID_ARG, "%s: ld_bt is smaller than n_pages", fn);
  if (!cu_rows || (B > 0 && (!cached_lens || !new_lens || !ctx_lens)) || (B > 0 && n_pages > 0 && !block_table) ||
      (n_free > 0 && !free_blocks) || (n_rows > 0 && (!positions || !slot_mapping))) {
    return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  }
  TableParams p{};
  p.cached = cached_lens;
  p.add = new_lens;
  p.held = held_pages;
  p.B = B;
  p.free_blocks = free_blocks;
  p.n_free = n_free;
  p.free_start = free_start;
  p.table = block_table;
  p.ld_bt = ld_bt;
  p.n_pages = n_pages;
  p.shift = block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
  p.ctx_lens = ctx_lens;
  p.cu_rows = cu_rows;
  p.cu_ctx = cu_ctx;
  p.held_out = held_out;
  p.free_end = free_end;
  p.positions = positions;
  p.slots = slot_mapping;
  p.row_to_req = row_to_req;
  p.row_ke = row_ke;
  p.n_rows = n_rows;
  const int most = std::max(B, n_rows);
  const bool cluster = most > kMaxTableThreads;
  const int threads = (std::min(std::max(most, 64), kMaxTableThreads) + 31) / 32 * 32;
  const size_t smem = table_smem_bytes(B);
  auto* kernel = cluster ? build_tables_kernel<true> : build_tables_kernel<false>;
  if (smem > kTableSmemUnasked) {
    // of the most requests, whatever this call's: another thread's smaller call must not take back what this one needs
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(table_smem_bytes(IDX_TABLES_MAX_REQUESTS)));
    if (e != cudaSuccess) return fail(IDX_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster ? kClusterBlocks : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cluster ? kClusterBlocks : 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const TableParams>(p));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(IDX_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  }
  return check_launch(fn);
}

extern "C" idx_status_t idx_tree_mask(const int32_t* parents, const int32_t* cu_rows, int32_t B, int32_t n_rows,
                                      const int32_t* base_lens, int32_t* mask, int64_t ld_mask, int32_t words,
                                      int32_t* positions, cudaStream_t stream) {
  const char* fn = "idx_tree_mask";
  if (B < 0 || n_rows < 0 || words < 1) return fail(IDX_ERR_INVALID_ARG, "%s: negative size, or no words", fn);
  if (words > IDX_TREE_MAX_WORDS) return fail(IDX_ERR_UNSUPPORTED, "%s: %d words", fn, words);
  if (ld_mask < words) return fail(IDX_ERR_INVALID_ARG, "%s: ld_mask is smaller than words", fn);
  if (B == 0 || n_rows == 0) return IDX_OK;
  if (!parents || !cu_rows || !mask) return fail(IDX_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  tree_mask_kernel<<<static_cast<unsigned>(B), kTreeThreads, 0, stream>>>(parents, cu_rows, n_rows, base_lens, mask,
                                                                          ld_mask, words, positions);
  return check_launch(fn);
}
