// What the paged serving operators share: the cache as their kernels see it,
// each kernel's parameters and launcher.
#pragma once

#include "kernels.h"
#include "work_split.h"

namespace gqa {

// Device status code beside those of common.cuh (mirrors GQA_DEV_BAD_PAGE).
constexpr int DEV_BAD_PAGE = 3;

constexpr int PAGED_MAX_SEQS = 2048;  // sequences per launch (prefix sums live in shared memory)
constexpr int PAGED_MAX_REP = 16;     // query heads per KV head

// Launch with programmatic stream serialization: the grid may be set up while
// the previous kernel of the stream ends. Only for kernels that execute
// pdl_wait() before they touch memory.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                          const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A paged cache as the kernels see it (gqa_pages with the page size as a shift).
struct PagedCache {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  long long page_stride, row_stride, head_stride;  // elements
  const int* table;
  int num_pages, page_shift, table_stride, columns;
  __device__ __forceinline__ long long capacity() const { return static_cast<long long>(columns) << page_shift; }
};

// 16 bytes global -> shared, asynchronously; zeros when `bytes` is 0 (src is
// then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's committed groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// The sequence of packed token m by a 32-way search (one load per 32-fold
// range) of cu[0..B], by one whole warp: the number of j in 1..B with
// cu[j] <= m, so empty sequences are passed over. B: m is past the last one.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int m) {
  const int lane = threadIdx.x & 31;
  return search_sequence(B, [&](int lo, int size, int step) {
    return __popc(__ballot_sync(0xffffffffu, search_at_or_before(cu, lo, size, step, lane, m)));
  });
}

// RoPE of packed queries and keys, keys and values into the pages.
struct PagedAppendParams {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int N, n_heads, n_kv;                    // n_heads 0: no queries
  const int* cu;                           // [B + 1], or null: token b is sequence b's
  int B;
  const int* start;
  const float* rope;
  int rope_rows;
  PagedCache pages;
  __nv_bfloat16* q_out;
  int* status;
};
cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s);

// One new token per sequence over the pages.
struct PagedDecodeParams {
  const __nv_bfloat16* q;
  long long q_stride;
  int B, n_heads, n_kv;
  const int* start;
  PagedCache pages;
  float scale_log2;         // softmax scale * log2(e)
  __nv_bfloat16* out;       // [B][n_heads][128]
  float* part_o;            // [2 * ctas][n_rep][128]
  float* part_ml;           // [2 * ctas][n_rep][2] (running max in log2 units, sum)
  int* tickets;             // [ctas], zero-filled, left zero-filled
  int* status;
  int ctas;
};
cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s);

// Causal attention of packed tokens; keys and values packed (cu gives their
// rows too) or in the pages.
struct PackedPrefillParams {
  int N, B, n_heads, n_kv;
  const int* cu;
  const int* start;         // null: packed keys
  PagedCache pages;         // packed keys: k, v and their strides (row_stride, head_stride); no table
  long long v_row_stride;   // packed values: elements between rows (pages: row_stride for both)
  const __nv_bfloat16* q;
  long long q_stride;
  float scale_log2;
  __nv_bfloat16* out;       // [N][n_heads][128]
  // Parts of items that several CTAs share: [2 * ctas][32 column groups][256
  // rows at most][4], their (max in log2 units, sum); the items that the second
  // kernel joins (packed_prefill_join_bytes; null: there are none); two counts
  // per CTA (parts that arrived, parts written); the claims of whole items and
  // the count of CTAs that are done. Counts zero-filled, left so.
  float *part_o, *part_ml;
  void* joins;
  int *tickets, *claims;
  int* status;
  unsigned long long wait_ns;  // limit of the waits
  int ctas;
};
// q: (dim, head, token), boxes of 64 dims x n_rep heads x 128 / n_rep tokens.
// k, v: (dim, KV head, row, page), boxes of 64 dims x 1 head x
// prefill_box_rows(page) rows; packed keys are one page of N rows.
struct PackedPrefillMaps {
  CUtensorMap q, k, v;
};
constexpr int PACKED_TILE = 128;  // keys of a tile
__host__ __device__ constexpr int prefill_box_rows(int page_size) { return page_size < PACKED_TILE ? page_size : PACKED_TILE; }
cudaError_t launch_packed_prefill(const PackedPrefillMaps& maps, const PackedPrefillParams& p, cudaStream_t s);
// With p.joins set, the join follows.
cudaError_t launch_packed_prefill_join(const PackedPrefillParams& p, cudaStream_t s);
bool packed_prefill_may_join(int N, int n_rep, long long most_keys);
size_t packed_prefill_join_bytes(int ctas);

}  // namespace gqa
