// RoPE and cache append of packed tokens: the epilogue of the block's Q|K|V
// projection ("Llama 3.1 8B · Grouped-query attention": apply_rotary_emb, then
// cache_k/v[b, start_pos + t] = k, v) for tokens projected elsewhere, into a
// paged cache.
//
// Every row is read once and written once and nothing is reused but a token's
// 512-byte table row, so the bound is memory. One warp takes 8 of a token's
// n_heads + 2 n_kv head rows, two at a time (16 lanes x 16 bytes each). The
// rows' loads are issued first: they need no position, while the chain
// sequence -> start position -> table entry -> RoPE row is three dependent
// loads. A lane's four pairs have the same place in every head, so the (cos,
// sin) of a token are loaded once for the warp's 8 rows.
#include "paged.h"

namespace gqa {

namespace {

constexpr int WARPS = 4;
constexpr int ROWS = 8;  // head rows per warp

__device__ __forceinline__ uint32_t rotate(uint32_t x, float c, float s) {
  const float a = bf16_lo(x), b = bf16_hi(x);
  return pack_bf16(a * c - b * s, a * s + b * c);
}

__global__ void __launch_bounds__(WARPS * 32) paged_append_kernel(PagedAppendParams p, int groups) {
  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, half = lane >> 4, piece = lane & 15;
  const long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int m = static_cast<int>(item / groups);
  if (m >= p.N) return;
  const int row0 = static_cast<int>(item - static_cast<long long>(m) * groups) * ROWS;
  const int rows = p.n_heads + 2 * p.n_kv;

  uint4 x[ROWS / 2];
#pragma unroll
  for (int i = 0; i < ROWS / 2; ++i) {
    const int r = row0 + 2 * i + half;
    if (r < rows) {
      const __nv_bfloat16* src = r < p.n_heads ? p.q + m * p.q_stride + r * HEAD_DIM
                                 : r < p.n_heads + p.n_kv
                                     ? p.k + m * p.k_stride + (r - p.n_heads) * HEAD_DIM
                                     : p.v + m * p.v_stride + (r - p.n_heads - p.n_kv) * HEAD_DIM;
      // q may be rotated in place: not the read-only path
      x[i] = *(reinterpret_cast<const uint4*>(src) + piece);
    }
  }

  int b = m, t = 0;
  if (p.cu) {
    b = sequence_of(p.cu, p.B, m);
    if (b >= p.B) return;
    t = m - p.cu[b];
    if (t < 0) return;
  }
  const int start = p.start[b];
  if (start == -1) return;  // unused slot
  const long long pos = static_cast<long long>(start) + t;
  if (start < 0 || pos >= p.rope_rows || pos >= p.pages.capacity()) {
    if (lane == 0) report(p.status, DEV_BAD_POSITION);
    return;
  }
  const int page = p.pages.table[static_cast<long long>(b) * p.pages.table_stride + (pos >> p.pages.page_shift)];
  if (page < 0 || page >= p.pages.num_pages) {
    if (lane == 0) report(p.status, DEV_BAD_PAGE);
    return;
  }
  const long long row = page * p.pages.page_stride +
                        (pos & ((1 << p.pages.page_shift) - 1)) * p.pages.row_stride + piece * 8;
  const float4* cs = reinterpret_cast<const float4*>(p.rope + pos * (2 * ROPE_PAIRS)) + piece * 2;
  const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);

#pragma unroll
  for (int i = 0; i < ROWS / 2; ++i) {
    const int r = row0 + 2 * i + half;
    if (r >= rows) continue;
    __nv_bfloat16* dst;
    if (r < p.n_heads)
      dst = p.q_out + (static_cast<long long>(m) * p.n_heads + r) * HEAD_DIM + piece * 8;
    else if (r < p.n_heads + p.n_kv)
      dst = p.pages.k + row + (r - p.n_heads) * p.pages.head_stride;
    else
      dst = p.pages.v + row + (r - p.n_heads - p.n_kv) * p.pages.head_stride;
    uint4 y = x[i];
    if (r < p.n_heads + p.n_kv)
      y = make_uint4(rotate(y.x, c0.x, c0.y), rotate(y.y, c0.z, c0.w), rotate(y.z, c1.x, c1.y),
                     rotate(y.w, c1.z, c1.w));
    *reinterpret_cast<uint4*>(dst) = y;
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  const int groups = (p.n_heads + 2 * p.n_kv + ROWS - 1) / ROWS;
  const long long blocks = (static_cast<long long>(p.N) * groups + WARPS - 1) / WARPS;
  if (blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_behind(paged_append_kernel, static_cast<unsigned>(blocks), WARPS * 32, 0, s, p, groups);
}

}  // namespace gqa
