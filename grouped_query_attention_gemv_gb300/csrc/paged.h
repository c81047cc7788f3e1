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

// A paged cache in 8 bits (gqa_fp8_pages): rows of 128 e4m3 values, a byte
// beside each row that holds its exponent + 127.
struct Fp8Cache {
  uint8_t *k, *v, *k_scale, *v_scale;
  long long page_stride, row_stride, head_stride;        // values
  long long scale_page, scale_row, scale_head;           // scales
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

// The same in any rotary layout: dims 0 .. rotary_dim - 1 of a head are turned,
// as pairs (2i, 2i + 1) or, with `halves`, (i, i + rotary_dim / 2); rope rows
// are rotary_dim / 2 pairs. Into `pages`, or with `fp8` set into `pages8`.
struct RotaryAppendParams {
  PagedAppendParams a;
  int rotary_dim, halves, fp8;
  Fp8Cache pages8;
};
cudaError_t launch_rotary_append(const RotaryAppendParams& p, cudaStream_t s);

// Rows 0 .. rows[b] - 1 of sequences from 8-bit pages into bf16 pages.
struct Fp8ReadParams {
  int B, n_kv;
  const int* rows;
  Fp8Cache from;
  PagedCache to;
  int* status;
  int ctas;
};
cudaError_t launch_fp8_read(const Fp8ReadParams& p, cudaStream_t s);

// The parts (paged_decode_shared.cu) of a sequence's KV head in a batch with
// shared rows: `prefixes` of those that it shares, 256 rows apart from row
// `prefix` on, `span` rows in each and its own from `at` on; `owns` of its own
// rows, n_rep rows apart from row `own` on.
struct SharedParts {
  int prefix, prefixes, span, at, own, owns, unused[2];
};
constexpr int SHARED_MAX_GROUPS = 1024;  // groups that are looked at
constexpr int SHARED_MAX_ROWS = 28672;   // query rows of a batch that shares (the workspace's room)
// Cache rows (of one KV head) that sharing has to save, or it is not done: those
// that are really not read. It takes 15 us at least, of which 4 to plan and 4 to
// join. Measured, plain and shared, own rows up to 50, 100,000 / 150,000 / 200,000
// rows saved: 8 KV heads of 4 query heads, 4 sequences 14.2 and 17.1 us / 18.9 and
// 18.4 / 22.1 and 20.3, 16 sequences 10.7 and 16.8 / 14.1 and 16.5 / 16.8 and 17.8,
// 32 sequences 12.5 and 16.5 / 15.0 and 17.0 / 17.3 and 16.7; 32 KV heads of 1, 16
// sequences 12.9 and 14.8 / 15.3 and 16.0 / 17.5 and 16.3; 4 KV heads of 16, 16
// sequences 18.2 and 20.3 / 21.5 and 20.7 / 24.5 and 22.6; one KV head of 16, 4
// sequences 31.9 and 25.9 / 37.2 and 30.7 / 40.8 and 34.1, 64 sequences 18.2 and
// 20.2 / 20.7 and 20.7 / 23.9 and 21.1. One number is within 2.5 us of the better
// way but for few sequences of 16 heads on one KV head (6).
constexpr unsigned long long SHARED_LEAST_ROWS = 150000;

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
  float *own_o, *own_ml;  // of rows that are part of a whole (SharedDecodeParams)
};
cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s);

// An attention with shared rows: prefixes and own rows. own: pages, queries and
// what streams the own rows; own_o, own_ml: their parts.
struct SharedDecodeParams {
  PagedDecodeParams own;
  int G;
  const int *cu, *prefix;
  float *part_o, *part_ml;  // rows of the prefixes' parts: O [32 column groups][span][4], (max in log2 units, sum)
  SharedParts* rows;        // [B][n_kv]
  unsigned long long wait_ns;
};
// Its join.
struct SharedJoinParams {
  int pairs, n_rep, sets;  // (sequence, KV head) pairs; sets: of rows in a pair
  const SharedParts* rows;
  const float *parts, *part_ml, *own_ml;  // parts: the prefixes' O, and own_at groups of 4 floats behind, the own rows'
  int part_rows, own_rows, own_at;
  __nv_bfloat16* out;
};

// The same over 8-bit pages. k, v: (dim, KV head, row, page), boxes of 128 dims
// x 1 head x fp8_decode_box_rows(page) rows.
struct Fp8DecodeParams {
  const __nv_bfloat16* q;
  long long q_stride;
  int B, n_heads, n_kv;
  const int* start;
  Fp8Cache pages;
  float scale_log2;
  __nv_bfloat16* out;
  float *part_o, *part_ml;  // as in PagedDecodeParams
  int* tickets;
  int* status;
  int ctas;
  unsigned long long wait_ns;  // limit of the waits
};
struct Fp8DecodeMaps {
  CUtensorMap k, v;
};
int fp8_decode_box_rows(int page_size);
cudaError_t launch_paged_decode_fp8(const Fp8DecodeMaps& maps, const Fp8DecodeParams& p, cudaStream_t s);

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
cudaError_t launch_shared_decode(const PackedPrefillMaps& maps, const SharedDecodeParams& p, cudaStream_t s);
cudaError_t launch_shared_join(const SharedJoinParams& p, cudaStream_t s);
long long shared_most_units(int B, int n_rep, int n_kv, long long keys);
bool packed_prefill_may_join(int N, int n_rep, long long most_keys);
size_t packed_prefill_join_bytes(int ctas);

}  // namespace gqa
