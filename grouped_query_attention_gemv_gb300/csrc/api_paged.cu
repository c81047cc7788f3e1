// C ABI of the paged serving operators (declared in include/gqa.h): argument
// validation on the host, workspace layout, tensor maps and one launch each (the
// prefill attention's join is a second).
#include <math.h>

#include "api_internal.h"
#include "paged.h"

using namespace gqa;

namespace {

// Workspace: the status word and its 256 bytes (the prefill attention's claims
// among them), the tickets, the items that the prefill attention's second
// kernel joins, the partials (two per CTA) of the decode or prefill attention.
constexpr size_t CLAIMS_OFFSET = 64;
constexpr size_t TICKETS_OFFSET = 256;
constexpr size_t PREFILL_ROWS = 256;  // query rows of an item
constexpr size_t PREFILL_ML_BYTES = static_cast<size_t>(2) * REF_SMS * PREFILL_ROWS * 2 * 4;
constexpr size_t PREFILL_O_BYTES = static_cast<size_t>(2) * REF_SMS * PREFILL_ROWS * HEAD_DIM * 4;
constexpr size_t JOINS_OFFSET = TICKETS_OFFSET + 2048;
constexpr size_t JOINS_BYTES = 16384;
constexpr size_t PART_ML_OFFSET = JOINS_OFFSET + JOINS_BYTES;
static_assert(PART_ML_OFFSET + PREFILL_ML_BYTES + PREFILL_O_BYTES <= GQA_PAGED_WORKSPACE_BYTES, "workspace");
constexpr size_t PART_ML_BYTES = static_cast<size_t>(2) * REF_SMS * PAGED_MAX_REP * 2 * 4;
constexpr size_t PART_O_OFFSET = (PART_ML_OFFSET + PART_ML_BYTES + 255) / 256 * 256;
constexpr size_t PART_O_BYTES = static_cast<size_t>(2) * REF_SMS * PAGED_MAX_REP * HEAD_DIM * 4;
static_assert(REF_SMS * 2 * 4 <= JOINS_OFFSET - TICKETS_OFFSET, "tickets");
static_assert(PART_O_OFFSET + PART_O_BYTES <= GQA_PAGED_WORKSPACE_BYTES, "workspace");
static_assert(GQA_PAGED_MAX_SEQS == PAGED_MAX_SEQS && GQA_PAGED_MAX_REP == PAGED_MAX_REP, "limits");

constexpr long long MAX_POSITIONS = 1LL << 30;  // positions a block table row can address
constexpr int MAX_TOKENS = 1 << 24;
constexpr long long MAX_STRIDE = 1LL << 38;     // elements (tensor maps take strides below 2^40 bytes)

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_stride(int64_t s, int64_t least) { return s >= least && s < MAX_STRIDE && s % 8 == 0; }

int check_heads(int n_heads, int n_kv) {
  return n_kv >= 1 && n_heads >= n_kv && n_heads <= (1 << 16) && n_heads % n_kv == 0 && n_heads / n_kv <= PAGED_MAX_REP
             ? GQA_OK : GQA_EINVAL;
}

int check_pages(const gqa_pages* g, PagedCache* c) {
  if (!g || !g->k || !g->v || !g->block_table) return GQA_EINVAL;
  if (g->num_pages <= 0 || g->columns <= 0 || g->table_stride < g->columns || g->n_kv_heads <= 0) return GQA_EINVAL;
  if (g->page_size < 16 || g->page_size > 65536 || (g->page_size & (g->page_size - 1)) != 0) return GQA_EINVAL;
  if (static_cast<long long>(g->columns) * g->page_size > MAX_POSITIONS) return GQA_EINVAL;
  if (!valid_stride(g->page_stride, HEAD_DIM) || !valid_stride(g->row_stride, HEAD_DIM) ||
      !valid_stride(g->head_stride, HEAD_DIM))
    return GQA_EINVAL;
  if (!aligned16(g->k) || !aligned16(g->v) || !aligned4(g->block_table)) return GQA_EALIGN;
  c->k = reinterpret_cast<__nv_bfloat16*>(g->k);
  c->v = reinterpret_cast<__nv_bfloat16*>(g->v);
  c->page_stride = g->page_stride;
  c->row_stride = g->row_stride;
  c->head_stride = g->head_stride;
  c->table = g->block_table;
  c->num_pages = g->num_pages;
  c->page_shift = 0;
  while ((1 << c->page_shift) < g->page_size) ++c->page_shift;
  c->table_stride = g->table_stride;
  c->columns = g->columns;
  return GQA_OK;
}

int check_workspace(const void* ws, size_t bytes) {
  if (!ws) return GQA_EINVAL;
  if (!aligned16(ws)) return GQA_EALIGN;
  return bytes < GQA_PAGED_WORKSPACE_BYTES ? GQA_EWORKSPACE : GQA_OK;
}

// A tensor's memory, from its first byte to its last (counted in 128 bits:
// strides times counts of a faulty call may pass 64).
struct Span {
  __int128 first, end;
  Span(const void* p, __int128 bytes) : first(reinterpret_cast<uintptr_t>(p)), end(first + (p ? bytes : 0)) {}
  bool meets(const Span& o) const { return end > first && o.end > o.first && first < o.end && o.first < end; }
};
// n packed rows of `row` elements
Span span_of(const gqa_bf16* p, int n, int64_t stride, int64_t row) {
  return {p, n > 0 ? (static_cast<__int128>(n - 1) * stride + row) * 2 : 0};
}
Span span_of(const int32_t* p, __int128 n) { return {p, n * 4}; }
// rows of keys or values in pages
Span span_of(const __nv_bfloat16* p, const PagedCache& c, int pages, int rows, int n_kv, long long row_stride) {
  return {p, (static_cast<__int128>(pages - 1) * c.page_stride + static_cast<__int128>(n_kv - 1) * c.head_stride +
              HEAD_DIM + static_cast<__int128>(rows - 1) * row_stride) * 2};
}
Span span_of_table(const PagedCache& c, int B) {
  return span_of(c.table, static_cast<__int128>(B - 1) * c.table_stride + c.columns);
}

// Whether some row of 128 elements of the key pages and some of the value pages
// share memory. The two may interleave (both halves of one [pages, 2, ...]
// tensor, say), so spans do not tell: rows at x page_stride + y row_stride + z
// head_stride are `d` apart for some |x| < pages, |y| < rows, |z| < heads. Taken
// from the largest stride down, what is left must be within the smaller
// strides' reach, so each count is one of two.
bool pages_meet(const PagedCache& c, int pages, int rows, int n_kv) {
  struct Axis {
    long long stride, n;
  } axes[3] = {{c.page_stride, pages}, {c.row_stride, rows}, {c.head_stride, n_kv}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (axes[j].stride < axes[j + 1].stride) {
        const Axis x = axes[j];
        axes[j] = axes[j + 1];
        axes[j + 1] = x;
      }
  const long long between = (reinterpret_cast<intptr_t>(c.v) - reinterpret_cast<intptr_t>(c.k)) / 2;
  for (int pick = 0; pick < 8; ++pick) {
    long long d = between;
    for (int i = 0; i < 3; ++i) {
      const long long s = axes[i].stride, most = axes[i].n - 1;
      long long x = d / s - (d % s < 0) + (pick >> i & 1);
      x = x > most ? most : x < -most ? -most : x;
      d -= x * s;
    }
    if (d < HEAD_DIM && d > -HEAD_DIM) return true;
  }
  return false;
}

// Whether the output of an attention call shares memory with what it reads.
bool out_meets(const Span& out, const Span& q, const PagedCache& c, int pages, int rows, int n_kv, long long v_row_stride,
               int B, const int32_t* start, const int32_t* cu, const void* workspace) {
  const Span read[] = {q, span_of(c.k, c, pages, rows, n_kv, c.row_stride), span_of(c.v, c, pages, rows, n_kv, v_row_stride),
                       span_of(start, B), span_of(cu, static_cast<__int128>(B) + 1),
                       span_of_table(c, B), {workspace, GQA_PAGED_WORKSPACE_BYTES}};
  for (const Span& r : read)
    if (out.meets(r)) return true;
  return false;
}

int check_scale(float scale) { return scale > 0.f && scale < 1e30f ? GQA_OK : GQA_EINVAL; }

const __nv_bfloat16* bf(const gqa_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(gqa_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

// Keys or values as (dim, KV head, row, page) with boxes of 64 dims x 1 head x box_rows rows.
bool map_kv(CUtensorMap* m, const void* ptr, int n_kv, long long rows, int pages, long long head_stride,
            long long row_stride, long long page_stride, int box_rows) {
  const cuuint64_t dims[4] = {HEAD_DIM, static_cast<cuuint64_t>(n_kv), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2,
                                 static_cast<cuuint64_t>(page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
  return encode_bf16(m, 4, ptr, dims, strides, box);
}

}  // namespace

extern "C" {

int gqa_paged_append(const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride, const gqa_bf16* v,
                     int64_t v_stride, int N, int n_heads, const int32_t* cu_tokens, int B, const int32_t* start_pos,
                     const float* rope, int rope_rows, const gqa_pages* pages, gqa_bf16* q_out, void* workspace,
                     size_t workspace_bytes, void* stream) {
  PagedAppendParams p{};
  if (!k || !v || !start_pos || !rope || rope_rows <= 0 || !q != !q_out) return GQA_EINVAL;
  if (N < 0 || N > MAX_TOKENS || B <= 0 || (!cu_tokens && N != B)) return GQA_EINVAL;
  int r = check_pages(pages, &p.pages);
  if (r != GQA_OK) return r;
  p.n_kv = pages->n_kv_heads;
  if (q && (r = check_heads(n_heads, p.n_kv)) != GQA_OK) return r;
  const int64_t kv_row = static_cast<int64_t>(p.n_kv) * HEAD_DIM, q_row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  if (p.n_kv > (1 << 16) || !valid_stride(k_stride, kv_row) || !valid_stride(v_stride, kv_row) ||
      (q && !valid_stride(q_stride, q_row)) || (q && q == q_out && q_stride != q_row))
    return GQA_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(rope) || (q && (!aligned16(q) || !aligned16(q_out))) ||
      !aligned4(start_pos) || (cu_tokens && !aligned4(cu_tokens)))
    return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
  if (N > 0) {
    // what the call writes: the queries, the key and the value pages
    const Span written[3] = {
        span_of(q_out, N, q_row, q_row),
        span_of(p.pages.k, p.pages, pages->num_pages, pages->page_size, p.n_kv, p.pages.row_stride),
        span_of(p.pages.v, p.pages, pages->num_pages, pages->page_size, p.n_kv, p.pages.row_stride)};
    const Span read[] = {span_of(k, N, k_stride, kv_row), span_of(v, N, v_stride, kv_row), span_of(start_pos, B),
                         span_of(cu_tokens, static_cast<__int128>(B) + 1), span_of_table(p.pages, B),
                         {rope, static_cast<__int128>(rope_rows) * ROPE_PAIRS * 8},
                         {workspace, GQA_PAGED_WORKSPACE_BYTES}};
    for (const Span& w : written)
      for (const Span& r : read)
        if (w.meets(r)) return GQA_EINVAL;
    const Span queries = span_of(q, N, q_stride, q_row);
    if ((q != q_out && written[0].meets(queries)) || written[1].meets(queries) || written[2].meets(queries) ||
        written[0].meets(written[1]) || written[0].meets(written[2]) ||
        (written[1].meets(written[2]) && pages_meet(p.pages, pages->num_pages, pages->page_size, p.n_kv)))
      return GQA_EINVAL;
  }
  begin_call();
  if (N == 0) return GQA_OK;
  p.q = bf(q);
  p.k = bf(k);
  p.v = bf(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.N = N;
  p.n_heads = q ? n_heads : 0;
  p.cu = cu_tokens;
  p.B = B;
  p.start = start_pos;
  p.rope = rope;
  p.rope_rows = rope_rows;
  p.q_out = bf(q_out);
  p.status = static_cast<int*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_mark(0, s);
  r = launched(launch_paged_append(p, s));
  prof_mark(1, s);
  return r;
}

int gqa_paged_decode(const gqa_bf16* q, int64_t q_stride, int B, int n_heads, const int32_t* start_pos,
                     const gqa_pages* pages, float scale, gqa_bf16* out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  PagedDecodeParams p{};
  if (!q || !start_pos || !out || B <= 0 || B > PAGED_MAX_SEQS) return GQA_EINVAL;
  int r = check_pages(pages, &p.pages);
  if (r == GQA_OK) r = check_heads(n_heads, pages->n_kv_heads);
  if (r == GQA_OK) r = check_scale(scale);
  if (r != GQA_OK) return r;
  if (!valid_stride(q_stride, static_cast<int64_t>(n_heads) * HEAD_DIM)) return GQA_EINVAL;
  // the batch's chunks of 16 positions and one KV head are counted in 31 bits
  if (p.pages.columns * static_cast<long long>(pages->page_size) / 16 * B * pages->n_kv_heads > 0x7fffffffLL)
    return GQA_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned4(start_pos)) return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
  const int64_t row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  if (out_meets(span_of(out, B, row, row), span_of(q, B, q_stride, row), p.pages, pages->num_pages, pages->page_size,
                pages->n_kv_heads, p.pages.row_stride, B, start_pos, nullptr, workspace))
    return GQA_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = bf(q);
  p.q_stride = q_stride;
  p.B = B;
  p.n_heads = n_heads;
  p.n_kv = pages->n_kv_heads;
  p.start = start_pos;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = bf(out);
  p.tickets = reinterpret_cast<int*>(ws + TICKETS_OFFSET);
  p.part_ml = reinterpret_cast<float*>(ws + PART_ML_OFFSET);
  p.part_o = reinterpret_cast<float*>(ws + PART_O_OFFSET);
  p.status = reinterpret_cast<int*>(ws);
  p.ctas = launch_sms();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  begin_call();
  prof_mark(0, s);
  r = launched(launch_paged_decode(p, s));
  prof_mark(1, s);
  return r;
}

static int prefill_call(const gqa_bf16* q, int64_t q_stride, int N, int n_heads, int n_kv, const int32_t* cu_tokens,
                        int B, float scale, gqa_bf16* out, void* workspace, size_t workspace_bytes, void* stream,
                        PackedPrefillParams& p, int kv_rows, int kv_pages, int box_rows, long long most_keys) {
  if (!q || !cu_tokens || !out || N < 0 || N > MAX_TOKENS || B <= 0 || B > PAGED_MAX_SEQS) return GQA_EINVAL;
  int r = check_heads(n_heads, n_kv);
  if (r == GQA_OK) r = check_scale(scale);
  if (r != GQA_OK) return r;
  if (!valid_stride(q_stride, static_cast<int64_t>(n_heads) * HEAD_DIM)) return GQA_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned4(cu_tokens)) return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
  const int64_t row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  const PagedCache& c = p.pages;
  const long long v_row = p.v_row_stride ? p.v_row_stride : c.row_stride;
  if (N > 0 && out_meets(span_of(out, N, row, row), span_of(q, N, q_stride, row), c, kv_pages, kv_rows, n_kv, v_row, B,
                         p.start, cu_tokens, workspace))
    return GQA_EINVAL;
  begin_call();
  if (N == 0) return GQA_OK;
  p.N = N;
  p.B = B;
  p.n_heads = n_heads;
  p.n_kv = n_kv;
  p.cu = cu_tokens;
  p.q = bf(q);
  p.q_stride = q_stride;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = bf(out);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int*>(ws);
  p.claims = reinterpret_cast<int*>(ws + CLAIMS_OFFSET);
  p.tickets = reinterpret_cast<int*>(ws + TICKETS_OFFSET);
  p.part_ml = reinterpret_cast<float*>(ws + PART_ML_OFFSET);
  p.part_o = reinterpret_cast<float*>(ws + PART_ML_OFFSET + PREFILL_ML_BYTES);
  p.wait_ns = wait_limit_ns();
  p.ctas = launch_sms();
  const int n_rep = n_heads / n_kv;
  if (packed_prefill_may_join(N, n_rep, most_keys)) p.joins = ws + JOINS_OFFSET;
  if (packed_prefill_join_bytes(p.ctas) > JOINS_BYTES) return fail_cuda(cudaErrorInvalidConfiguration);
  PackedPrefillMaps maps;
  const cuuint64_t dims[3] = {HEAD_DIM, static_cast<cuuint64_t>(n_heads), static_cast<cuuint64_t>(N)};
  const cuuint64_t strides[2] = {HEAD_DIM * 2, static_cast<cuuint64_t>(q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(n_rep), static_cast<cuuint32_t>(128 / n_rep)};
  if (!encode_bf16(&maps.q, 3, q, dims, strides, box) ||
      !map_kv(&maps.k, c.k, n_kv, kv_rows, kv_pages, c.head_stride, c.row_stride, c.page_stride, box_rows) ||
      !map_kv(&maps.v, c.v, n_kv, kv_rows, kv_pages, c.head_stride, v_row, c.page_stride, box_rows))
    return fail_cuda(cudaErrorInvalidValue);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_mark(0, s);
  r = launched(launch_packed_prefill(maps, p, s));
  prof_mark(1, s);
  if (r == GQA_OK && p.joins) {
    r = launched(launch_packed_prefill_join(p, s));
    prof_mark(2, s);
  }
  return r;
}

int gqa_paged_prefill(const gqa_bf16* q, int64_t q_stride, int N, int n_heads, const int32_t* cu_tokens, int B,
                      const int32_t* start_pos, const gqa_pages* pages, float scale, gqa_bf16* out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  PackedPrefillParams p{};
  if (!start_pos) return GQA_EINVAL;
  const int r = check_pages(pages, &p.pages);
  if (r != GQA_OK) return r;
  if (!aligned4(start_pos)) return GQA_EALIGN;
  // the key tiles of the (at most 320) items that are cut into ranges, and two
  // units for each item, are counted in 31 bits over the KV heads
  if ((static_cast<long long>(pages->columns) * pages->page_size / PACKED_TILE + 3) * 320 * pages->n_kv_heads >
      0x7fffffffLL)
    return GQA_EINVAL;
  p.start = start_pos;
  return prefill_call(q, q_stride, N, n_heads, pages->n_kv_heads, cu_tokens, B, scale, out, workspace,
                      workspace_bytes, stream, p, pages->page_size, pages->num_pages,
                      prefill_box_rows(pages->page_size),
                      static_cast<long long>(pages->columns) * pages->page_size);
}

int gqa_packed_prefill(const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride, const gqa_bf16* v,
                       int64_t v_stride, int N, int n_heads, int n_kv_heads, const int32_t* cu_tokens, int B,
                       float scale, gqa_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  PackedPrefillParams p{};
  if (!k || !v) return GQA_EINVAL;
  const int64_t kv_row = static_cast<int64_t>(n_kv_heads) * HEAD_DIM;
  if (n_kv_heads <= 0 || !valid_stride(k_stride, kv_row) || !valid_stride(v_stride, kv_row)) return GQA_EINVAL;
  if (!aligned16(k) || !aligned16(v)) return GQA_EALIGN;
  // one page of N rows
  p.pages.k = const_cast<__nv_bfloat16*>(bf(k));
  p.pages.v = const_cast<__nv_bfloat16*>(bf(v));
  p.pages.head_stride = HEAD_DIM;
  p.pages.row_stride = k_stride;
  p.pages.page_stride = k_stride;
  p.v_row_stride = v_stride;
  return prefill_call(q, q_stride, N, n_heads, n_kv_heads, cu_tokens, B, scale, out, workspace, workspace_bytes,
                      stream, p, N, 1, PACKED_TILE, N);
}

}  // extern "C"
