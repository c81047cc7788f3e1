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
// of a decode attention with shared rows: its plan, the parts of own rows, the parts of prefixes
constexpr size_t SHARED_PARTS_OFFSET = (PART_O_OFFSET + PART_O_BYTES + 255) / 256 * 256;
constexpr size_t OWN_ML_OFFSET = SHARED_PARTS_OFFSET + SHARED_MAX_ROWS * sizeof(SharedParts);
// one part more per warp, and per CTA with prefixes, than there are (sequence, KV head) pairs
constexpr int OWN_ROWS = SHARED_MAX_ROWS + REF_SMS * 8 * PAGED_MAX_REP;
constexpr int PREFIX_ROWS = SHARED_MAX_ROWS + REF_SMS * 256;
constexpr size_t PREFIX_ML_OFFSET = OWN_ML_OFFSET + OWN_ROWS * static_cast<size_t>(8);
constexpr size_t PREFIX_O_OFFSET = PREFIX_ML_OFFSET + PREFIX_ROWS * static_cast<size_t>(8);
constexpr size_t OWN_O_OFFSET = PREFIX_O_OFFSET + PREFIX_ROWS * static_cast<size_t>(HEAD_DIM * 4);
static_assert(OWN_O_OFFSET + OWN_ROWS * static_cast<size_t>(HEAD_DIM * 4) <= GQA_PAGED_WORKSPACE_BYTES, "workspace");
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

bool valid_scale_stride(int64_t s) { return s >= 1 && s < MAX_STRIDE; }

int check_pages(const gqa_fp8_pages* g, Fp8Cache* c) {
  if (!g || !g->k || !g->v || !g->k_scale || !g->v_scale) return GQA_EINVAL;
  // bytes as elements of half the size: the same limits, and 16-byte steps
  gqa_pages b{};
  b.k = reinterpret_cast<gqa_bf16*>(g->k);
  b.v = reinterpret_cast<gqa_bf16*>(g->v);
  b.page_stride = g->page_stride;
  b.row_stride = g->row_stride;
  b.head_stride = g->head_stride;
  b.block_table = g->block_table;
  b.num_pages = g->num_pages;
  b.page_size = g->page_size;
  b.n_kv_heads = g->n_kv_heads;
  b.table_stride = g->table_stride;
  b.columns = g->columns;
  PagedCache p{};
  const int r = check_pages(&b, &p);
  if (r != GQA_OK) return r;
  if (g->page_stride % 16 || g->row_stride % 16 || g->head_stride % 16 || !valid_scale_stride(g->scale_page_stride) ||
      !valid_scale_stride(g->scale_row_stride) || !valid_scale_stride(g->scale_head_stride))
    return GQA_EINVAL;
  *c = {g->k, g->v, g->k_scale, g->v_scale, p.page_stride, p.row_stride, p.head_stride,
        g->scale_page_stride, g->scale_row_stride, g->scale_head_stride, p.table, p.num_pages, p.page_shift,
        p.table_stride, p.columns};
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
// rows of an 8-bit cache and their scales
Span span_of(const uint8_t* p, long long page_stride, long long row_stride, long long head_stride, int pages, int rows,
             int n_kv, int width) {
  return {p, static_cast<__int128>(pages - 1) * page_stride + static_cast<__int128>(rows - 1) * row_stride +
                 static_cast<__int128>(n_kv - 1) * head_stride + width};
}
template <class Cache>
Span span_of_table(const Cache& c, int B) {
  return span_of(c.table, static_cast<__int128>(B - 1) * c.table_stride + c.columns);
}

// Whether some row of `width` of the key pages and some of the value pages
// share memory. The two may interleave (both halves of one [pages, 2, ...]
// tensor, say), so spans do not tell: rows at x page_stride + y row_stride + z
// head_stride are `d` apart for some |x| < pages, |y| < rows, |z| < heads. Taken
// from the largest stride down, what is left must be within the smaller
// strides' reach, so each count is one of two.
bool rows_meet(long long between, int width, long long page_stride, int pages, long long row_stride, int rows,
               long long head_stride, int n_kv) {
  struct Axis {
    long long stride, n;
  } axes[3] = {{page_stride, pages}, {row_stride, rows}, {head_stride, n_kv}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (axes[j].stride < axes[j + 1].stride) {
        const Axis x = axes[j];
        axes[j] = axes[j + 1];
        axes[j + 1] = x;
      }
  for (int pick = 0; pick < 8; ++pick) {
    long long d = between;
    for (int i = 0; i < 3; ++i) {
      const long long s = axes[i].stride, most = axes[i].n - 1;
      long long x = d / s - (d % s < 0) + (pick >> i & 1);
      x = x > most ? most : x < -most ? -most : x;
      d -= x * s;
    }
    if (d < width && d > -width) return true;
  }
  return false;
}
long long apart(const void* k, const void* v) { return reinterpret_cast<intptr_t>(v) - reinterpret_cast<intptr_t>(k); }
bool pages_meet(const PagedCache& c, int pages, int rows, int n_kv) {
  return rows_meet(apart(c.k, c.v) / 2, HEAD_DIM, c.page_stride, pages, c.row_stride, rows, c.head_stride, n_kv);
}

// The four tensors of an 8-bit cache.
struct Fp8Spans {
  Span s[4];
  Fp8Spans(const Fp8Cache& c, const gqa_fp8_pages& g)
      : s{span_of(c.k, c.page_stride, c.row_stride, c.head_stride, g.num_pages, g.page_size, g.n_kv_heads, HEAD_DIM),
          span_of(c.v, c.page_stride, c.row_stride, c.head_stride, g.num_pages, g.page_size, g.n_kv_heads, HEAD_DIM),
          span_of(c.k_scale, c.scale_page, c.scale_row, c.scale_head, g.num_pages, g.page_size, g.n_kv_heads, 1),
          span_of(c.v_scale, c.scale_page, c.scale_row, c.scale_head, g.num_pages, g.page_size, g.n_kv_heads, 1)} {}
  bool meet(const Span& o) const { return s[0].meets(o) || s[1].meets(o) || s[2].meets(o) || s[3].meets(o); }
};
// Whether tensors of an 8-bit cache that is written share memory: values with
// values, scales with scales by their rows, values with scales by their spans.
bool pages_meet(const Fp8Cache& c, const gqa_fp8_pages& g, const Fp8Spans& x) {
  for (int i = 0; i < 2; ++i)
    if (x.s[i].meets(x.s[2]) || x.s[i].meets(x.s[3])) return true;
  return (x.s[0].meets(x.s[1]) && rows_meet(apart(c.k, c.v), HEAD_DIM, c.page_stride, g.num_pages, c.row_stride,
                                            g.page_size, c.head_stride, g.n_kv_heads)) ||
         (x.s[2].meets(x.s[3]) && rows_meet(apart(c.k_scale, c.v_scale), 1, c.scale_page, g.num_pages, c.scale_row,
                                            g.page_size, c.scale_head, g.n_kv_heads));
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

// What the appends check and share: everything but the pages that are written.
int append_args(PagedAppendParams& p, const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride,
                       const gqa_bf16* v, int64_t v_stride, int N, int n_heads, int n_kv, const int32_t* cu_tokens,
                       int B, const int32_t* start_pos, const float* rope, int rope_rows, gqa_bf16* q_out,
                       void* workspace, size_t workspace_bytes) {
  int r = GQA_OK;
  p.n_kv = n_kv;
  if (q && (r = check_heads(n_heads, p.n_kv)) != GQA_OK) return r;
  const int64_t kv_row = static_cast<int64_t>(p.n_kv) * HEAD_DIM, q_row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  if (p.n_kv > (1 << 16) || !valid_stride(k_stride, kv_row) || !valid_stride(v_stride, kv_row) ||
      (q && !valid_stride(q_stride, q_row)) || (q && q == q_out && q_stride != q_row))
    return GQA_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(rope) || (q && (!aligned16(q) || !aligned16(q_out))) ||
      !aligned4(start_pos) || (cu_tokens && !aligned4(cu_tokens)))
    return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
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
  return GQA_OK;
}
bool append_given(const gqa_bf16* q, const gqa_bf16* k, const gqa_bf16* v, int N, const int32_t* cu_tokens, int B,
                         const int32_t* start_pos, const float* rope, int rope_rows, const gqa_bf16* q_out) {
  if (!k || !v || !start_pos || !rope || rope_rows <= 0 || !q != !q_out) return false;
  return N >= 0 && N <= MAX_TOKENS && B > 0 && (cu_tokens || N == B);
}
// Whether something that an append writes (the queries, the spans of the pages)
// shares memory with what it reads, or the queries with the pages.
bool append_meets(const PagedAppendParams& p, int n_heads, int pairs, const Span* pages, int n_pages,
                         const Span& table, const void* workspace) {
  const int64_t kv_row = static_cast<int64_t>(p.n_kv) * HEAD_DIM, q_row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  const Span read[] = {{p.k, (static_cast<__int128>(p.N - 1) * p.k_stride + kv_row) * 2},
                       {p.v, (static_cast<__int128>(p.N - 1) * p.v_stride + kv_row) * 2},
                       span_of(p.start, p.B),
                       span_of(p.cu, static_cast<__int128>(p.B) + 1),
                       table,
                       {p.rope, static_cast<__int128>(p.rope_rows) * pairs * 8},
                       {workspace, GQA_PAGED_WORKSPACE_BYTES}};
  const Span queries{p.q, (static_cast<__int128>(p.N - 1) * p.q_stride + q_row) * 2};
  const Span q_out{p.q_out, static_cast<__int128>(p.N) * q_row * 2};
  for (const Span& r : read) {
    if (q_out.meets(r)) return true;
    for (int i = 0; i < n_pages; ++i)
      if (pages[i].meets(r)) return true;
  }
  if (p.q != p.q_out && q_out.meets(queries)) return true;
  for (int i = 0; i < n_pages; ++i)
    if (pages[i].meets(queries) || pages[i].meets(q_out)) return true;
  return false;
}
bool append_meets(const PagedAppendParams& p, int n_heads, int pairs, const gqa_pages& g, const void* workspace) {
  const Span pages[2] = {span_of(p.pages.k, p.pages, g.num_pages, g.page_size, p.n_kv, p.pages.row_stride),
                         span_of(p.pages.v, p.pages, g.num_pages, g.page_size, p.n_kv, p.pages.row_stride)};
  return append_meets(p, n_heads, pairs, pages, 2, span_of_table(p.pages, p.B), workspace) ||
         (pages[0].meets(pages[1]) && pages_meet(p.pages, g.num_pages, g.page_size, p.n_kv));
}
// A part of a head is whole 16-byte pieces in both layouts.
bool valid_rotary(int rotary_dim) { return rotary_dim >= 16 && rotary_dim <= HEAD_DIM && rotary_dim % 16 == 0; }
template <class Launch>
int one_launch(void* stream, Launch launch) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_mark(0, s);
  const int r = launched(launch(s));
  prof_mark(1, s);
  return r;
}

}  // namespace

extern "C" {

int gqa_paged_append(const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride, const gqa_bf16* v,
                     int64_t v_stride, int N, int n_heads, const int32_t* cu_tokens, int B, const int32_t* start_pos,
                     const float* rope, int rope_rows, const gqa_pages* pages, gqa_bf16* q_out, void* workspace,
                     size_t workspace_bytes, void* stream) {
  PagedAppendParams p{};
  if (!append_given(q, k, v, N, cu_tokens, B, start_pos, rope, rope_rows, q_out)) return GQA_EINVAL;
  int r = check_pages(pages, &p.pages);
  if (r == GQA_OK)
    r = append_args(p, q, q_stride, k, k_stride, v, v_stride, N, n_heads, pages->n_kv_heads, cu_tokens, B, start_pos,
                    rope, rope_rows, q_out, workspace, workspace_bytes);
  if (r != GQA_OK) return r;
  if (N > 0 && append_meets(p, n_heads, ROPE_PAIRS, *pages, workspace)) return GQA_EINVAL;
  begin_call();
  if (N == 0) return GQA_OK;
  return one_launch(stream, [&](cudaStream_t s) { return launch_paged_append(p, s); });
}

int gqa_paged_append_rotary(const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride, const gqa_bf16* v,
                            int64_t v_stride, int N, int n_heads, const int32_t* cu_tokens, int B,
                            const int32_t* start_pos, const float* rope, int rope_rows, int rotary_dim, int halves,
                            const gqa_pages* pages, gqa_bf16* q_out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  RotaryAppendParams p{};
  if (!append_given(q, k, v, N, cu_tokens, B, start_pos, rope, rope_rows, q_out) || !valid_rotary(rotary_dim))
    return GQA_EINVAL;
  int r = check_pages(pages, &p.a.pages);
  if (r == GQA_OK)
    r = append_args(p.a, q, q_stride, k, k_stride, v, v_stride, N, n_heads, pages->n_kv_heads, cu_tokens, B, start_pos,
                    rope, rope_rows, q_out, workspace, workspace_bytes);
  if (r != GQA_OK) return r;
  if (N > 0 && append_meets(p.a, n_heads, rotary_dim / 2, *pages, workspace)) return GQA_EINVAL;
  begin_call();
  if (N == 0) return GQA_OK;
  p.rotary_dim = rotary_dim;
  p.halves = halves != 0;
  return one_launch(stream, [&](cudaStream_t s) { return launch_rotary_append(p, s); });
}

int gqa_paged_append_fp8(const gqa_bf16* q, int64_t q_stride, const gqa_bf16* k, int64_t k_stride, const gqa_bf16* v,
                         int64_t v_stride, int N, int n_heads, const int32_t* cu_tokens, int B,
                         const int32_t* start_pos, const float* rope, int rope_rows, int rotary_dim, int halves,
                         const gqa_fp8_pages* pages, gqa_bf16* q_out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  RotaryAppendParams p{};
  if (!append_given(q, k, v, N, cu_tokens, B, start_pos, rope, rope_rows, q_out) || !valid_rotary(rotary_dim))
    return GQA_EINVAL;
  int r = check_pages(pages, &p.pages8);
  if (r == GQA_OK)
    r = append_args(p.a, q, q_stride, k, k_stride, v, v_stride, N, n_heads, pages->n_kv_heads, cu_tokens, B, start_pos,
                    rope, rope_rows, q_out, workspace, workspace_bytes);
  if (r != GQA_OK) return r;
  if (N > 0) {
    const Fp8Spans spans(p.pages8, *pages);
    if (append_meets(p.a, n_heads, rotary_dim / 2, spans.s, 4, span_of_table(p.pages8, B), workspace) ||
        pages_meet(p.pages8, *pages, spans))
      return GQA_EINVAL;
  }
  begin_call();
  if (N == 0) return GQA_OK;
  p.rotary_dim = rotary_dim;
  p.halves = halves != 0;
  p.fp8 = 1;
  return one_launch(stream, [&](cudaStream_t s) { return launch_rotary_append(p, s); });
}

int gqa_paged_read_fp8(const int32_t* rows, int B, const gqa_fp8_pages* from, const gqa_pages* to, void* workspace,
                       size_t workspace_bytes, void* stream) {
  Fp8ReadParams p{};
  if (!rows || B <= 0 || B > PAGED_MAX_SEQS) return GQA_EINVAL;
  int r = check_pages(from, &p.from);
  if (r == GQA_OK) r = check_pages(to, &p.to);
  if (r != GQA_OK) return r;
  if (from->n_kv_heads != to->n_kv_heads || from->n_kv_heads > (1 << 16)) return GQA_EINVAL;
  // units of 16 positions are counted in 31 bits
  const long long most = static_cast<long long>(from->columns) * from->page_size;
  const long long most_to = static_cast<long long>(to->columns) * to->page_size;
  if ((most < most_to ? most : most_to) / 16 * B > 0x7fffffffLL) return GQA_EINVAL;
  if (!aligned4(rows)) return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
  const Span written[2] = {span_of(p.to.k, p.to, to->num_pages, to->page_size, to->n_kv_heads, p.to.row_stride),
                           span_of(p.to.v, p.to, to->num_pages, to->page_size, to->n_kv_heads, p.to.row_stride)};
  const Fp8Spans spans(p.from, *from);
  const Span read[] = {span_of(rows, B), span_of_table(p.from, B), span_of_table(p.to, B),
                       {workspace, GQA_PAGED_WORKSPACE_BYTES}};
  for (const Span& w : written) {
    if (spans.meet(w)) return GQA_EINVAL;
    for (const Span& x : read)
      if (w.meets(x)) return GQA_EINVAL;
  }
  if (written[0].meets(written[1]) && pages_meet(p.to, to->num_pages, to->page_size, to->n_kv_heads)) return GQA_EINVAL;
  p.B = B;
  p.n_kv = from->n_kv_heads;
  p.rows = rows;
  p.status = static_cast<int*>(workspace);
  p.ctas = launch_sms();
  begin_call();
  return one_launch(stream, [&](cudaStream_t s) { return launch_fp8_read(p, s); });
}

int gqa_paged_decode_fp8(const gqa_bf16* q, int64_t q_stride, int B, int n_heads, const int32_t* start_pos,
                         const gqa_fp8_pages* pages, float scale, gqa_bf16* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  Fp8DecodeParams p{};
  if (!q || !start_pos || !out || B <= 0 || B > PAGED_MAX_SEQS) return GQA_EINVAL;
  int r = check_pages(pages, &p.pages);
  if (r == GQA_OK) r = check_heads(n_heads, pages->n_kv_heads);
  if (r == GQA_OK) r = check_scale(scale);
  if (r != GQA_OK) return r;
  if (!valid_stride(q_stride, static_cast<int64_t>(n_heads) * HEAD_DIM)) return GQA_EINVAL;
  // the batch's chunks of 32 positions and one KV head are counted in 31 bits
  if ((p.pages.columns * static_cast<long long>(pages->page_size) / 32 + 1) * B * pages->n_kv_heads > 0x7fffffffLL)
    return GQA_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned4(start_pos)) return GQA_EALIGN;
  if ((r = check_workspace(workspace, workspace_bytes)) != GQA_OK) return r;
  const int64_t row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  const Span o = span_of(out, B, row, row);
  if (o.meets(span_of(q, B, q_stride, row)) || Fp8Spans(p.pages, *pages).meet(o) || o.meets(span_of(start_pos, B)) ||
      o.meets(span_of_table(p.pages, B)) || o.meets({workspace, GQA_PAGED_WORKSPACE_BYTES}))
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
  p.wait_ns = wait_limit_ns();
  Fp8DecodeMaps maps;
  const cuuint64_t dims[4] = {HEAD_DIM, static_cast<cuuint64_t>(p.n_kv), static_cast<cuuint64_t>(pages->page_size),
                              static_cast<cuuint64_t>(pages->num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.pages.head_stride), static_cast<cuuint64_t>(p.pages.row_stride),
                                 static_cast<cuuint64_t>(p.pages.page_stride)};
  const cuuint32_t box[4] = {HEAD_DIM, 1, static_cast<cuuint32_t>(fp8_decode_box_rows(pages->page_size)), 1};
  if (!encode_bytes(&maps.k, 4, p.pages.k, dims, strides, box) || !encode_bytes(&maps.v, 4, p.pages.v, dims, strides, box))
    return fail_cuda(cudaErrorInvalidValue);
  begin_call();
  return one_launch(stream, [&](cudaStream_t s) { return launch_paged_decode_fp8(maps, p, s); });
}

// What the decode attentions over bf16 pages check and share.
static int decode_args(PagedDecodeParams& p, const gqa_bf16* q, int64_t q_stride, int B, int n_heads,
                       const int32_t* start_pos, const gqa_pages* pages, float scale, gqa_bf16* out, void* workspace,
                       size_t workspace_bytes) {
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
  return GQA_OK;
}

int gqa_paged_decode(const gqa_bf16* q, int64_t q_stride, int B, int n_heads, const int32_t* start_pos,
                     const gqa_pages* pages, float scale, gqa_bf16* out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  PagedDecodeParams p{};
  const int r = decode_args(p, q, q_stride, B, n_heads, start_pos, pages, scale, out, workspace, workspace_bytes);
  if (r != GQA_OK) return r;
  begin_call();
  return one_launch(stream, [&](cudaStream_t s) { return launch_paged_decode(p, s); });
}

// The maps of packed queries and of keys and values for the attentions on the
// tensor cores.
static bool attention_maps(PackedPrefillMaps& maps, const gqa_bf16* q, int64_t q_stride, int N, int n_heads, int n_kv,
                           const PagedCache& c, long long v_row, int kv_rows, int kv_pages, int box_rows) {
  const int n_rep = n_heads / n_kv;
  const cuuint64_t dims[3] = {HEAD_DIM, static_cast<cuuint64_t>(n_heads), static_cast<cuuint64_t>(N)};
  const cuuint64_t strides[2] = {HEAD_DIM * 2, static_cast<cuuint64_t>(q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(n_rep), static_cast<cuuint32_t>(128 / n_rep)};
  return encode_bf16(&maps.q, 3, q, dims, strides, box) &&
         map_kv(&maps.k, c.k, n_kv, kv_rows, kv_pages, c.head_stride, c.row_stride, c.page_stride, box_rows) &&
         map_kv(&maps.v, c.v, n_kv, kv_rows, kv_pages, c.head_stride, v_row, c.page_stride, box_rows);
}

int gqa_paged_decode_shared(const gqa_bf16* q, int64_t q_stride, int B, int n_heads, const int32_t* start_pos,
                            const int32_t* cu_groups, int G, const int32_t* prefix_rows, const gqa_pages* pages,
                            float scale, gqa_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  PagedDecodeParams p{};
  if (!cu_groups || !prefix_rows || G <= 0 || G > PAGED_MAX_SEQS) return GQA_EINVAL;
  const int r = decode_args(p, q, q_stride, B, n_heads, start_pos, pages, scale, out, workspace, workspace_bytes);
  if (r != GQA_OK) return r;
  if (!aligned4(cu_groups) || !aligned4(prefix_rows)) return GQA_EALIGN;
  const int64_t row = static_cast<int64_t>(n_heads) * HEAD_DIM;
  const Span o = span_of(out, B, row, row);
  if (o.meets(span_of(cu_groups, static_cast<__int128>(G) + 1)) || o.meets(span_of(prefix_rows, G))) return GQA_EINVAL;
  begin_call();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The same function without sharing: where the batch cannot save enough, and
  // where it passes what the plan and the workspace hold.
  const int n_rep = n_heads / p.n_kv;
  const long long keys = static_cast<long long>(pages->columns) * pages->page_size;
  if (static_cast<unsigned long long>(keys) * (B - 1) * p.n_kv < SHARED_LEAST_ROWS || G > SHARED_MAX_GROUPS ||
      B * n_heads > SHARED_MAX_ROWS || shared_most_units(B, n_rep, p.n_kv, keys) > 0x7fffffffLL)
    return one_launch(stream, [&](cudaStream_t) { return launch_paged_decode(p, s); });

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.own_o = reinterpret_cast<float*>(ws + OWN_O_OFFSET);
  p.own_ml = reinterpret_cast<float*>(ws + OWN_ML_OFFSET);
  SharedDecodeParams a{};
  a.own = p;
  a.G = G;
  a.cu = cu_groups;
  a.prefix = prefix_rows;
  a.part_o = reinterpret_cast<float*>(ws + PREFIX_O_OFFSET);
  a.part_ml = reinterpret_cast<float*>(ws + PREFIX_ML_OFFSET);
  a.rows = reinterpret_cast<SharedParts*>(ws + SHARED_PARTS_OFFSET);
  a.wait_ns = wait_limit_ns();
  SharedJoinParams j{};
  j.pairs = B * p.n_kv;
  j.n_rep = n_rep;
  j.rows = a.rows;
  j.parts = a.part_o;
  j.part_ml = a.part_ml;
  j.part_rows = PREFIX_ROWS;
  j.own_rows = OWN_ROWS;
  j.own_ml = p.own_ml;
  j.own_at = static_cast<int>((OWN_O_OFFSET - PREFIX_O_OFFSET) / 16);
  j.out = p.out;
  PackedPrefillMaps maps;
  if (!attention_maps(maps, q, q_stride, B, n_heads, p.n_kv, p.pages, p.pages.row_stride, pages->page_size,
                      pages->num_pages, prefill_box_rows(pages->page_size)))
    return fail_cuda(cudaErrorInvalidValue);
  prof_mark(0, s);
  int e = launched(launch_shared_decode(maps, a, s));
  prof_mark(1, s);
  if (e == GQA_OK) e = launched(launch_shared_join(j, s));
  prof_mark(2, s);
  return e;
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
  if (!attention_maps(maps, q, q_stride, N, n_heads, n_kv, c, v_row, kv_rows, kv_pages, box_rows))
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
