// Causal attention of packed tokens of different sequences on the
// 5th-generation tensor cores, keys and values in a paged cache or packed
// beside the queries ("Llama 3.1 8B · Grouped-query attention": query t sees
// keys 0..start_pos + t, softmax in fp32, output heads merged h * 128 + d).
//
// Bound by the tensor cores from a few hundred keys on (4 x 128 flops per
// visible (query, key) pair and head).
//
// Tiles. A work item is two 128-row Q tiles of one KV head and one sequence,
// each 128 / n_rep positions x n_rep query heads (row r: position r / n_rep,
// head r % n_rep; n_rep need not divide 128, the last rows then stay unused),
// and every 128-key K/V tile is staged once for both. S = Q K^T (M=128, N=128)
// goes to TMEM, P = 2^(S scale - max) over its first half as bf16, and
// O += P V takes P from TMEM and V as an MN-major operand. 512 TMEM columns:
// S and O of both Q tiles; S is not doubled. Tiles of 64 keys, which leave
// room for that (the dense prefill's scheme), measured 8% slower over long
// prompts: a product of N = 64 waits for its operands in shared memory (49
// cycles measured where the arithmetic takes 32; N = 128: 64 and 64). The last
// key tile of a Q tile is half as wide where its second half is all masked.
//
// Turns. The two Q tiles' issuers alternate step by step (P V of one key tile,
// S of the next), so that one tile's softmax (~1,400 cycles from S to all of
// P) runs beside the other's products (~1,430 a step). Left alone they fall
// into step, both softmaxes and then all products: 3,900 cycles a key tile
// against 3,150 (2,800 as it stands). One issuer for both took 3,700.
//
// Ragged sequences. Entries (pairs of Q tiles of a sequence) x KV heads are
// the items. Up to 320 entries are sorted longest first, and the CTAs claim
// whole items as they get free (the next one when the last copies of one have
// been issued). Whole items dealt out longest first may leave the fullest CTA
// far behind the mean (few or long items: a chunk after a long prefix). The key
// tiles of all items can be cut into one equal range per CTA instead, two ways,
// and the cheapest of the three by the costs below is taken:
//   - Ranges of half the longest item at least. An item then has three parts
//     at most, and the CTA that arrives last at its count adds the others to
//     its own in its epilogue, all in CTA order: it waits only for CTAs that
//     have arrived, which are running and about to write. 1,024 tokens after
//     7,168 (128 items on 152 SMs): 100 us, 112 with all parts left to a second
//     kernel.
//   - Shorter ranges, whose items' parts a second kernel joins, in CTA order:
//     22 us for 40 tokens after 8,000 (8 heads, 2 KV heads), where a join by
//     the last CTA took 47; 32 for 256 after 4,000 (32 and 8 heads) against 52.
//     Empty, that kernel takes 2 us, so it is not launched where no sequence
//     can have more than 2,048 keys (packed_prefill_may_join: what that costs).
// Above 320 entries nothing is sorted or cut, and a long sequence among them is
// walked by one CTA per KV head: 320 single tokens and one after 131,071 take
// 1,280 us, 319 and one 180.
// An item counts ITEM_UNITS key tiles more than it has, or a range of many
// short items ends last: 45 us against 59 for one prompt of 4,000 tokens (8 and
// 2 heads), 32 against 36 for 2,340.
//
// Masked and foreign values. Q boxes may reach into the next sequence (rows
// that are never stored), K and V boxes into the next sequence's rows, a
// page's unwritten rows, or past the end (zeros): scores there are masked, and
// the issuers clear those value rows in shared memory before the product,
// because 0 x NaN is NaN. A NaN among the values of an item's own later
// positions, which only its earlier rows mask, cannot be cleared for some rows
// of a tile and not for others: a row whose result is not finite, with such
// values behind it, is computed again by a warp from its visible keys alone.
//
//   warp 8        plans the items, TMA producer: a K/V tile is 128 / min(page,
//                 128) boxes, one lane each, so that the table look-ups of a
//                 tile are one load wide
//   warps 9, 10   MMA issuers, one per Q tile
//   warps 0-3/4-7 one softmax warpgroup per Q tile, one thread per row
// P is rounded to bf16 (the product takes no wider operand); sums are fp32 of
// the unrounded values. O is rescaled only when a row's max grows by more than
// 2^8 over the max its P values were taken against.
// Every wait is bounded (gqa_set_wait_limit_ns); one that gives up records
// DEV_WAIT_TIMEOUT, lets
// issued copies and products finish (bounded) and frees TMEM before the CTA
// exits.
// Measured: 382 us for nine prompts of up to 4,095 tokens in a short run (578
// GFLOP: 1,515 TFLOP/s of 1,962 measured), 420 under the power cap, 98 to 104
// for 1,024 tokens after 7,168, 34.2 for 2,048 tokens, 7.1 for 17. What bounds
// the long ones is the alternation: per key tile the tensor pipe works 2 x 1,024
// of about 2,800 cycles.
#include <math.h>

#include "paged.h"

namespace gqa {

namespace {

constexpr int ROWS = 128;                 // rows of a Q tile = MMA M
constexpr int NQ = 2;                     // Q tiles per CTA
constexpr int KT = PACKED_TILE;           // keys per tile
constexpr int HALF = KT / 2;
constexpr int STAGES = 2;                 // K tiles and V tiles in shared memory
constexpr int Q_HALF = ROWS * 128;        // 128 rows x 64 dims
constexpr int Q_TILE = 2 * Q_HALF;
constexpr int KV_HALF = KT * 128;         // 64 keys x 64 dims
constexpr int KV_TILE = 2 * KV_HALF;
constexpr int K_OFF = NQ * Q_TILE;
constexpr int V_OFF = K_OFF + STAGES * KV_TILE;
constexpr int BAR_OFF = V_OFF + STAGES * KV_TILE;
constexpr int MAX_SORT = 320;             // entries that are sorted, or cut into equal ranges
constexpr int BARS_BYTES = 5120;
constexpr int DIRECT = 2;                 // other parts of an item that are added in its epilogue at most
constexpr int PRE_OFF = BAR_OFF + BARS_BYTES;
constexpr int OUT_OFF = (PRE_OFF + (PAGED_MAX_SEQS + 1) * 4 + 127) / 128 * 128;
constexpr int OUT_WARP = 32 * 64;         // staging of 32 output rows x 32 columns, per softmax warp
constexpr int SMEM_BYTES = OUT_OFF + 8 * OUT_WARP + 1024;
constexpr int THREADS = 352;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9;  // MMA warps 9 (Q tile 0) and 10 (Q tile 1)
constexpr int SLOTS = 2;                  // items handed from the producer to the other warps
// What sharing items costs, in key tiles of one CTA (about 1.6 us), by the rows
// of an item: with up to 1 + DIRECT parts, of which the last CTA reads two; with
// more, for the second kernel, writing two parts and reading all. Measured: 18
// and 14 us for full items of 256 rows and 9 us per 40 MB that the second kernel
// reads, little for few rows (5 tokens after 2,100, 8 and 2 heads: 17 us by
// short ranges, 29 by halves).
constexpr float DIRECT_TILES = 2.f, DIRECT_ROW = 8.f / (NQ * ROWS);
constexpr float JOIN_TILES = 4.f, JOIN_ROW = 5.f / (NQ * ROWS), JOIN_PART_ROW = 1.4e-4f;
constexpr uint32_t TMEM_COLS = 512;
// TMEM columns: S (128, P over its first 64) of Q tiles 0 and 1, then O of both
constexpr uint32_t S_COLS = 128, O_COL = 256, O_COLS = 128;
constexpr float RESCALE_LOG2 = 8.f;

// What a CTA works on at a time: 2 Q tiles (NQ x qp query positions) of one
// KV head g of sequence b, and n of the key tiles they see, from tile j0 on.
struct Item {
  int g, b, q0, row0, T;
  int start, kv_end;  // cached rows before the sequence's tokens; keys behind kv_end are not the item's
  int j0, n;          // key tiles [j0, j0 + n); n = 0: the rows are zero
  int nt[NQ];         // of those, the tiles of each Q tile (0: none, or the tile is past T)
  int first, last;    // the CTAs with a part of the same Q tiles (first = last: all of it is here)
};

struct Bars {
  uint64_t q_full[NQ];
  uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
  uint64_t s_full[NQ], p_full[NQ][2];  // p_full: the first and the second half of the keys
  uint64_t turn[NQ];                   // the issuer of Q tile t has issued a step
  uint64_t o_done[NQ], mma_done[NQ];
  uint64_t item_full[SLOTS], item_empty[SLOTS], joint;
  uint32_t tmem_slot;
  int abort;
  unsigned long long wait_ns;  // limit of the waits
  unsigned alive;             // counts up while rows are computed again
  int q_issued[NQ], k_issued, v_issued;
  int warp_sum[THREADS / 32];
  int rows;                   // most query rows of an item
  int warps_here;             // softmax warps with their rows of a shared item
  int is_last;                // of an item's parts, this CTA's is the last
  int parts_there;            // the others are written
  Item item[SLOTS];           // g < 0: no more
  int cum[MAX_SORT + 1];      // key tiles before entry e, if there are at most MAX_SORT entries
  short order[MAX_SORT];      // entries, longest first
};
static_assert(sizeof(Bars) <= BARS_BYTES, "barrier block");
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool aborted(const Bars& bs) { return *reinterpret_cast<const volatile int*>(&bs.abort) != 0; }

// The packed rows of sequence b: those of cu[b] .. cu[b+1]-1 that exist.
struct Seq {
  int row0, T;
};
__device__ __forceinline__ Seq seq_at(const PackedPrefillParams& a, int b) {
  const int r = a.cu[b], e = min(a.cu[b + 1], a.N);
  return {r, r >= 0 && e > r ? e - r : 0};
}

// Entry e: the pairs of Q tiles of the sequences in order, the last pair of
// each sequence first.
__device__ __forceinline__ Item entry_at(int e, const int* pre, int qp, const PackedPrefillParams& a) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= e) lo = mid; else hi = mid;
  }
  Item it;
  it.g = 0;
  it.b = lo;
  const Seq s = seq_at(a, lo);
  it.row0 = s.row0;
  it.T = s.T;
  it.q0 = (pre[lo + 1] - 1 - e) * NQ * qp;
  it.start = a.start ? a.start[lo] : 0;
  const bool ok = it.start >= 0 && (!a.start || it.start + static_cast<long long>(s.T) <= a.pages.capacity());
  it.j0 = it.n = it.first = it.last = 0;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int qt = it.q0 + t * qp;
    it.nt[t] = ok && qt < s.T ? (it.start + min(qt + qp, s.T) + KT - 1) / KT : 0;
    it.n = max(it.n, it.nt[t]);
  }
  it.kv_end = it.start + min(it.q0 + NQ * qp, s.T);
  return it;
}

// Equal ranges: the item with unit u, from u on as far as the range that ends
// at `end` goes (n = 0: it has no tile there); u becomes the first unit behind
// that.
__device__ __forceinline__ Item ranged_item(int& u, int end, const Split& split, int E, const int* cum, const int* pre,
                                            int qp, const PackedPrefillParams& a) {
  const Piece p = piece_at(u, end, split, E, cum, a.n_kv);
  Item it = entry_at(p.entry, pre, qp, a);
  it.g = p.g;
  it.j0 = p.j0;
  it.first = p.first;
  it.last = p.last;
  it.n = max(0, p.j1 - p.j0);
  u = p.behind;
#pragma unroll
  for (int t = 0; t < NQ; ++t) it.nt[t] = max(0, min(it.nt[t], p.j1) - p.j0);
  return it;
}

// Wait of a whole warp for phase `parity` of a barrier; false when it gave up:
// after bs.wait_ns in which no row was computed again either (masked_row takes
// as long as the row's keys are many, and the others wait for its warp). All
// but the first try is out of line: inlined at the eleven waits the loop cost
// 3% (2,048 tokens 35.9 us against 34.3, nine prompts 439 against 424).
__device__ __noinline__ bool wait_longer(const Bars& bs, uint32_t bar, unsigned parity) {
  unsigned alive = 0;
  while (!__all_sync(0xffffffffu, mbar_wait(bar, parity, bs.wait_ns))) {
    const unsigned now = *const_cast<const volatile unsigned*>(&bs.alive);
    if (!__any_sync(0xffffffffu, now != alive)) return false;
    alive = now;
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(const Bars& bs, uint64_t& bar, unsigned parity) {
  const uint32_t at = smem_u32(&bar);
  return __all_sync(0xffffffffu, mbar_try_wait(at, parity)) || wait_longer(bs, at, parity);
}

// The items of this CTA in order, as the other warps take them from the
// producer's slots.
struct ItemWalk {
  int k = 0;
  bool ok = true;
  __device__ __forceinline__ bool next(Bars& bs, Item& it) {
    const int s = k % SLOTS;
    ok = wait_bar(bs, bs.item_full[s], (k / SLOTS) & 1);
    if (!ok) return false;
    it = bs.item[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bs.item_empty[s]));
    ++k;
    return it.g >= 0;
  }
};

// Element offset of key (value) row `key` of sequence b and KV head g
// (a table entry out of range, reported by the producer, reads page 0).
__device__ __forceinline__ long long key_row(const PackedPrefillParams& a, int b, int row0, int g, int key, bool value) {
  if (!a.start)
    return (static_cast<long long>(row0) + key) * (value ? a.v_row_stride : a.pages.row_stride) +
           g * a.pages.head_stride;
  const int page = a.pages.table[static_cast<long long>(b) * a.pages.table_stride + (key >> a.pages.page_shift)];
  return (page < 0 || page >= a.pages.num_pages ? 0 : page) * a.pages.page_stride +
         (key & ((1 << a.pages.page_shift) - 1)) * a.pages.row_stride + g * a.pages.head_stride;
}

// One output row from its visible keys 0..lim alone, by a whole warp, in
// fp32: 32 keys at a time, a key a lane for the scores, 4 dims a lane for the
// values. For rows whose result is not finite and that share tiles with later
// keys of their item (up to kv_end): nothing is done where those values are
// all finite, because the row's own keys then made it so. A row takes 0.37 us
// a key (48 ms after 131,072), so `alive`, if there is one, is counted up on
// the way: waits on this warp then go on.
__device__ __noinline__ void masked_row(const PackedPrefillParams& a, int b, int row0, int g, int start, int pos,
                                        int head, int kv_end, unsigned* alive) {
  const size_t row = static_cast<size_t>(row0) + pos;
  const __nv_bfloat16* q = a.q + static_cast<long long>(row) * a.q_stride + head * HEAD_DIM;
  __nv_bfloat16* dst = a.out + (row * a.n_heads + head) * HEAD_DIM;
  const int lim = start + pos;
  const int lane = threadIdx.x & 31;
  bool dirty = false;
  for (int j = lim + 1; j < kv_end && !dirty; j += 4) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j + k >= kv_end) continue;
      const uint2 v = *(reinterpret_cast<const uint2*>(a.pages.v + key_row(a, b, row0, g, j + k, true)) + lane);
      x += bf16_lo(v.x) * 0.f + bf16_hi(v.x) * 0.f + bf16_lo(v.y) * 0.f + bf16_hi(v.y) * 0.f;
    }
    dirty = __any_sync(0xffffffffu, x != x);
  }
  if (!dirty) return;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 <= lim; j0 += 32) {
    if (alive && lane == 0) atomicAdd(alive, 1u);
    float s = -INFINITY;
    if (j0 + lane <= lim) {
      const uint4* k4 = reinterpret_cast<const uint4*>(a.pages.k + key_row(a, b, row0, g, j0 + lane, false));
      const uint4* q4 = reinterpret_cast<const uint4*>(q);
      float x = 0.f;
#pragma unroll 2
      for (int i = 0; i < HEAD_DIM / 8; ++i) {
        const uint4 u = k4[i], w = q4[i];
        const uint32_t ku[4] = {u.x, u.y, u.z, u.w}, qu[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) x += bf16_lo(ku[e]) * bf16_lo(qu[e]) + bf16_hi(ku[e]) * bf16_hi(qu[e]);
      }
      s = x * a.scale_log2;
    }
    float mx = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    mx = fmaxf(mx, m);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float al = ex2_approx(m - ref), pr = ex2_approx(s - ref);
    float sum = pr;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * al + sum;
    m = mx;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= al;
    for (int j = j0; j <= min(lim, j0 + 31); ++j) {
      const float w = __shfl_sync(0xffffffffu, pr, j - j0);
      const uint2 v = *(reinterpret_cast<const uint2*>(a.pages.v + key_row(a, b, row0, g, j, true)) + lane);
      o[0] += w * bf16_lo(v.x);
      o[1] += w * bf16_hi(v.x);
      o[2] += w * bf16_lo(v.y);
      o[3] += w * bf16_hi(v.y);
    }
  }
  const float inv = 1.f / l;
  *(reinterpret_cast<uint2*>(dst) + lane) = make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
}

// Barrier of the softmax warps, the n-th of a CTA; false when it gave up.
__device__ __forceinline__ bool softmax_sync(Bars& bs, unsigned& n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bs.joint));
  return wait_bar(bs, bs.joint, n++ & 1);
}

// Parts of an item that several CTAs share: slot 2 c + 1 for the CTA with the
// item's first key tile (slot 2 c may hold its part of the item before), 2 c
// otherwise. A part is the fp32 O, [32 column groups][span rows][4] without
// gaps, and [256 rows] (max in log2 units, sum).
__device__ __forceinline__ size_t part_slot(int c, int first) { return 2 * static_cast<size_t>(c) + (c == first); }
__device__ __forceinline__ float2* part_ml(const PackedPrefillParams& a, size_t slot) {
  return reinterpret_cast<float2*>(a.part_ml) + slot * NQ * ROWS;
}
__device__ __forceinline__ float4* part_o(const PackedPrefillParams& a, size_t slot) {
  return reinterpret_cast<float4*>(a.part_o) + slot * NQ * ROWS * (HEAD_DIM / 4);
}

// The sum of three parts' terms, this CTA's and the others' in CTA order, so
// that it does not depend on whose it is: the first two, then the last.
__device__ __forceinline__ float in_order(bool behind, float own, float x, float y) {
  return behind ? __fadd_rn(__fadd_rn(x, y), own) : __fadd_rn(__fadd_rn(own, x), y);
}

// The real rows of an item's Q tiles, each tile's first ones, and the rows
// 0 .. span - 1 that hold them all (tile 1 from row 128 on).
struct Rows {
  int rows0, rows1, span;
  __device__ __forceinline__ Rows(const Item& it, int qp, int nrep)
      : rows0(min(qp, it.T - it.q0) * nrep), rows1(max(0, min(qp, it.T - it.q0 - qp)) * nrep),
        span(rows1 ? ROWS + rows1 : rows0) {}
};

// ---- the second kernel: joins the parts of items that more than 1 + DIRECT
// CTAs share, block x the item
// that CTA x of the first kernel began, if it is shared, block y a slice of its
// rows. One part per (CTA, item), in CTA order: the result does not depend on
// who was first.
// Short slices are faster (40 tokens after 8,000: 21.7 us with 16 rows, 25.3
// with 32), many blocks slower where there is nothing to join (16 a CTA 1.2 us
// more than 8): 16 rows where an item can have no more than 160.
constexpr int JOIN_THREADS = 256;
template <int SLICE>
__global__ void __launch_bounds__(JOIN_THREADS) packed_prefill_join_kernel(const __grid_constant__ PackedPrefillParams a) {
  constexpr int LANES = JOIN_THREADS / SLICE;  // of a row
  __shared__ float weight[MAX_PARTS][SLICE];
  __shared__ int off[SLICE], bad[SLICE];
  pdl_trigger();
  pdl_wait();
  const Item it = reinterpret_cast<const Item*>(a.joins)[blockIdx.x];
  const int np = it.last - it.first + 1;
  if (np <= 1 + DIRECT) return;
  // an item of another call (a workspace that two calls use at once, or that
  // was not zeroed): nothing of it is read or written
  const long long keys = a.start ? a.pages.capacity() : it.T;
  if (np > MAX_PARTS || it.first < 0 || it.last >= a.ctas || it.b < 0 || it.b >= a.B || it.g < 0 || it.g >= a.n_kv ||
      it.q0 < 0 || it.q0 >= it.T || it.row0 < 0 || it.T > a.N - it.row0 || it.start < 0 || it.kv_end > keys)
    return;
  const int nrep = a.n_heads / a.n_kv, qp = ROWS / nrep, tid = threadIdx.x, lane = tid & 31;
  const Rows n(it, qp, nrep);
  const int r0 = blockIdx.y * SLICE;
  if (r0 >= n.span) return;
  {
    // a row's lanes: its max over the parts, the parts' factors, the sum
    const int r = tid / LANES, row = r0 + r, t = row / ROWS, rr = row & (ROWS - 1), rp = rr / nrep;
    const bool real = row < n.span && rr < (t ? n.rows1 : n.rows0);
    float m = -INFINITY, l = 0.f;
    if (real)
      for (int c = tid % LANES; c < np; c += LANES) m = fmaxf(m, __ldcg(part_ml(a, part_slot(it.first + c, it.first)) + row).x);
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (m == -INFINITY) m = 0.f;
    if (real)
      for (int c = tid % LANES; c < np; c += LANES) {
        const float2 ml = __ldcg(part_ml(a, part_slot(it.first + c, it.first)) + row);
        const float w = ex2_approx(ml.x - m);
        l += w * ml.y;
        weight[c][r] = w;
      }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float inv = 1.f / l;
    if (real)
      for (int c = tid % LANES; c < np; c += LANES) weight[c][r] *= inv;
    if (tid % LANES == 0) {
      off[r] = real ? ((t * qp + rp) * a.n_heads + it.g * nrep + rr - rp * nrep) * HEAD_DIM : -1;
      bad[r] = 0;
    }
  }
  __syncthreads();
  // a warp: 8 rows x 4 column groups, so that whole sectors are read and stored
  __nv_bfloat16* out = a.out + (static_cast<size_t>(it.row0) + it.q0) * a.n_heads * HEAD_DIM;
  const int g = (tid >> 5) * 4 + (lane >> 3);
  constexpr int EACH = SLICE / 8;
  float4 o[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int c = 0; c < np; ++c) {
    const float4* x4 = part_o(a, part_slot(it.first + c, it.first)) + g * n.span + r0 + (lane & 7);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int r = 8 * i + (lane & 7);
      if (off[r] < 0) continue;
      const float4 x = __ldcg(x4 + 8 * i);
      const float w = weight[c][r];
      o[i].x += w * x.x;
      o[i].y += w * x.y;
      o[i].z += w * x.z;
      o[i].w += w * x.w;
    }
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int r = 8 * i + (lane & 7);
    if (off[r] < 0) continue;
    const float chk = o[i].x * 0.f + o[i].y * 0.f + o[i].z * 0.f + o[i].w * 0.f;
    if (chk != chk) bad[r] = 1;
    *(reinterpret_cast<uint2*>(out + off[r]) + g) = make_uint2(pack_bf16(o[i].x, o[i].y), pack_bf16(o[i].z, o[i].w));
  }
  __syncthreads();
  for (int r = tid >> 5; r < SLICE; r += JOIN_THREADS / 32) {
    const int row = r0 + r, t = row / ROWS, rr = row & (ROWS - 1), rp = rr / nrep, pos = it.q0 + t * qp + rp;
    if (bad[r] && it.start + pos < it.kv_end - 1)
      masked_row(a, it.b, it.row0, it.g, it.start, pos, it.g * nrep + rr - rp * nrep, it.kv_end, nullptr);
  }
}

__global__ void __launch_bounds__(THREADS, 1)
    packed_prefill_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ PackedPrefillParams a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bs = *reinterpret_cast<Bars*>(smem + BAR_OFF);
  int* pre = reinterpret_cast<int*>(smem + PRE_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrep = a.n_heads / a.n_kv;
  const int qp = ROWS / nrep;  // query positions per Q tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&bs.k_full[s]), 1);
      mbar_init(smem_u32(&bs.k_empty[s]), NQ);  // one arrival per MMA issuer
      mbar_init(smem_u32(&bs.v_full[s]), 1);
      mbar_init(smem_u32(&bs.v_empty[s]), NQ);
    }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(smem_u32(&bs.q_full[t]), 1);
      mbar_init(smem_u32(&bs.s_full[t]), 1);
      mbar_init(smem_u32(&bs.turn[t]), 1);
      for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&bs.p_full[t][h]), 4);
      mbar_init(smem_u32(&bs.o_done[t]), 1);
      mbar_init(smem_u32(&bs.mma_done[t]), 1);
    }
    mbar_init(smem_u32(&bs.joint), 8);
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&bs.item_full[s]), 1);
      mbar_init(smem_u32(&bs.item_empty[s]), 10);  // issuers, softmax warps
    }
    bs.abort = 0;
    bs.alive = 0;
    bs.warps_here = 0;
    bs.wait_ns = a.wait_ns;
    bs.rows = 0;
    bs.q_issued[0] = bs.q_issued[1] = 0;
    bs.k_issued = bs.v_issued = 0;
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&bs.tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  // nothing in global memory is read or written before the previous kernel of
  // the stream is done
  pdl_trigger();
  pdl_wait();
  // pairs of Q tiles per sequence, prefix-summed
  {
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, a.B), b1 = min(b0 + per, a.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = seq_at(a, b);
      if (a.start && blockIdx.x == 0 && s.T > 0) {
        const int st = a.start[b];
        // an unused slot (-1) holds any number of tokens
        if (st < -1 || (st >= 0 && st + static_cast<long long>(s.T) > a.pages.capacity()))
          report(a.status, DEV_BAD_POSITION);
      }
      const int n = (s.T + NQ * qp - 1) / (NQ * qp);
      pre[b + 1] = n;
      sum += n;
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) bs.warp_sum[warp] = run;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += bs.warp_sum[w];
    for (int b = b0; b < b1; ++b) {
      run += pre[b + 1];
      pre[b + 1] = run;
    }
  }
  __syncthreads();
  // ---- the plan. E entries x n_kv KV heads are the items. Few entries: their
  // key tiles are prefix-summed and sorted by length.
  const int E = pre[a.B], G = gridDim.x;
  const long long nitems = static_cast<long long>(E) * a.n_kv;
  bool equal = false;   // equal ranges of key tiles instead of whole items
  bool sorted = false;  // whole items in the order of bs.order
  int units = 0, parts = 1;
  int own_n = 0;
  if (E <= MAX_SORT && static_cast<int>(threadIdx.x) < E) {
    const Item own = entry_at(threadIdx.x, pre, qp, a);
    own_n = own.n;
    atomicMax(&bs.rows, min(own.T - own.q0, NQ * qp) * nrep);
  }
  // nothing to plan where every CTA has one short item at most
  if (E <= MAX_SORT && (__syncthreads_or(own_n > 2 * MIN_TILES) || nitems > G)) {
    const int e = threadIdx.x;
    const int own_w = own_n ? own_n + ITEM_UNITS : 0;
    if (e < E) bs.cum[e + 1] = own_w;
    if (e == 0) bs.cum[0] = 0;
    __syncthreads();
    int before = 0, rank = 0;
    if (e < E)
      for (int f = 0; f < E; ++f) {
        const int m = bs.cum[f + 1];
        before += f <= e ? m : 0;
        rank += m > own_w || (m == own_w && f < e);
      }
    __syncthreads();
    if (e < E) {
      bs.order[rank] = static_cast<short>(e);
      bs.cum[e + 1] = before;
    }
    __syncthreads();
    sorted = true;
    units = bs.cum[E] * a.n_kv;
    // The load of CTA `threadIdx.x` if whole items went round in turn, longest
    // first, against equal ranges (no shorter than pays for the joins) and the
    // joins they bring.
    int load = 0;
    if (static_cast<int>(threadIdx.x) < G)
#pragma unroll 1
      for (int k = 0; k * G < nitems; ++k) {
        const int i = k * G + ((k & 1) ? G - 1 - static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x));
        if (i < nitems) {
          const int o = bs.order[i / a.n_kv];
          load += bs.cum[o + 1] - bs.cum[o];
        }
      }
    const int o = bs.order[0], longest = bs.cum[o + 1] - bs.cum[o];
    const int mean = mean_range(units, G);
    const int few = few_parts_range(mean, longest);
    const float few_cost = few + DIRECT_TILES + DIRECT_ROW * bs.rows;
    const int many = many_parts_range(mean, longest);
    const float many_cost = a.joins ? many + JOIN_TILES + (JOIN_ROW + JOIN_PART_ROW * (units / many)) * bs.rows : INFINITY;
    equal = __syncthreads_or(static_cast<float>(load) > fminf(few_cost, many_cost));
    if (equal) parts = range_count(units, few_cost <= many_cost ? few : many, G);
  }
  const bool claim = !equal && nitems > G;  // items are claimed as CTAs get to them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bs.tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  ItemWalk walk;
  Item it;

  if (warp == PRODUCER_WARP) {
    // ---- which item comes next. Asked for when the last copies of the one
    // before have been issued: whole items go to the CTAs that are free first.
    const Split split(units, parts);
    const bool ranged = equal && static_cast<int>(blockIdx.x) < parts;
    int ru = ranged ? split.start(blockIdx.x) : 0;
    const int rend = ranged ? split.start(blockIdx.x + 1) : 0;
    int ze = 0, zg = -1;          // equal ranges: the next entry without keys
    long long wi = blockIdx.x;    // whole items: the next one
    bool asked = false;
    auto next_item = [&](Item& it) {
      if (!equal) {
        if (asked) {
          if (!claim) return false;
          int c = 0;
          if (lane == 0) c = atomicAdd(a.claims, 1);
          wi = static_cast<long long>(G) + static_cast<unsigned>(__shfl_sync(0xffffffffu, c, 0));
        }
        asked = true;
        if (wi >= nitems) return false;
        const int e = static_cast<int>(wi / a.n_kv);
        it = entry_at(sorted ? bs.order[e] : e, pre, qp, a);
        it.g = static_cast<int>(wi - static_cast<long long>(e) * a.n_kv);
        return true;
      }
      // units in (entry, KV head, key tile) order; this CTA's range of them
      while (ru < rend) {
        it = ranged_item(ru, rend, split, E, bs.cum, pre, qp, a);
        if (it.n > 0) return true;
      }
      // entries without keys (unused slots), whose rows are zero
      for (;;) {
        if (zg >= 0 && zg < a.n_kv) {
          it = entry_at(ze, pre, qp, a);
          it.g = zg;
          zg += G;
          return true;
        }
        if (zg >= 0) ++ze;
        while (ze < E && bs.cum[ze + 1] != bs.cum[ze]) ++ze;
        if (ze >= E) return false;
        zg = (static_cast<int>(blockIdx.x) + ze) % G;
      }
    };
    int puts = 0;
    auto put = [&](const Item& x) {
      const int s = puts % SLOTS;
      if (puts >= SLOTS && !wait_bar(bs, bs.item_empty[s], (puts / SLOTS - 1) & 1)) return false;
      if (lane == 0) {
        bs.item[s] = x;
        mbar_arrive(smem_u32(&bs.item_full[s]));
      }
      __syncwarp();
      ++puts;
      return true;
    };
    if (lane == 0) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
    // Lane x < boxes handles box x of every tile. u counts tiles over the
    // CTA's items, ring slot u % STAGES.
    const int box = a.start ? prefill_box_rows(1 << a.pages.page_shift) : KT;
    const int boxes = KT / box;
    const uint32_t q_bytes = static_cast<uint32_t>(qp * nrep) * 128;
    int u = 0, kn = 0, vn = 0, qn[NQ] = {};
    int cs[NQ] = {};  // score tiles of each Q tile so far (as its issuer counts them)
    bool ok = true, stop = false;
    auto go_on = [&](uint64_t& bar, int parity) {
      ok = wait_bar(bs, bar, parity);
      return ok && !__any_sync(0xffffffffu, aborted(bs));
    };
    auto copy = [&](const CUtensorMap* map, uint64_t& full, uint32_t dst, int held, int g, int row, int page) {
      const uint32_t fb = smem_u32(&full);
      if (lane == 0) mbar_expect_tx(fb, static_cast<uint32_t>(held * box) * 256);
      __syncwarp();
      if (lane < held) {
        const uint32_t at = dst + static_cast<uint32_t>(lane * box) * 128;
        tma_load_4d(at, map, fb, 0, g, row, page);
        tma_load_4d(at + KV_HALF, map, fb, 64, g, row, page);
      }
      __syncwarp();
    };
    while (!stop && next_item(it)) {
      if (!put(it)) {
        ok = false;
        break;
      }
      for (int j = 0; j < it.n && !stop; ++j, ++u) {
        const int s = u % STAGES;
        // boxes of the tile that hold keys of the item; this lane's
        const int held = min(boxes, (it.kv_end - (it.j0 + j) * KT + box - 1) / box);
        const int key = (it.j0 + j) * KT + lane * box;
        int row = it.row0 + key, page = 0;
        if (a.start) {
          row = key & ((1 << a.pages.page_shift) - 1);
          if (lane < held)
            page = a.pages.table[static_cast<long long>(it.b) * a.pages.table_stride + (key >> a.pages.page_shift)];
        }
        if (u >= STAGES && !go_on(bs.k_empty[s], (u / STAGES - 1) & 1)) {
          stop = true;
          break;
        }
        if (page < 0 || (a.start && page >= a.pages.num_pages)) {
          report(a.status, DEV_BAD_PAGE);
          page = 0;
        }
        copy(&mk, bs.k_full[s], sbase + K_OFF + s * KV_TILE, held, it.g, row, page);
        kn = u + 1;
        if (j == 0) {
          // Q tile t is free once the last score product of the previous item
          // that read it has completed (the next one on its S needs the new
          // Q, so that phase is the latest)
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            if (stop || !it.nt[t]) continue;
            if (cs[t] > 0 && !go_on(bs.s_full[t], (cs[t] - 1) & 1)) {
              stop = true;
              continue;
            }
            if (lane == 0) {
              const uint32_t qb = smem_u32(&bs.q_full[t]);
              mbar_expect_tx(qb, 2 * q_bytes);
              // boxes may reach into the next sequence, or past N (zeros): rows that are never stored
              tma_load_3d(sbase + t * Q_TILE, &mq, qb, 0, it.g * nrep, it.row0 + it.q0 + t * qp);
              tma_load_3d(sbase + t * Q_TILE + Q_HALF, &mq, qb, 64, it.g * nrep, it.row0 + it.q0 + t * qp);
            }
            __syncwarp();
            ++qn[t];
          }
          if (stop) break;
        }
        if (u >= STAGES && !go_on(bs.v_empty[s], (u / STAGES - 1) & 1)) {
          stop = true;
          break;
        }
        copy(&mv, bs.v_full[s], sbase + V_OFF + s * KV_TILE, held, it.g, row, page);
        vn = u + 1;
      }
#pragma unroll
      for (int t = 0; t < NQ; ++t) cs[t] += it.nt[t];
    }
    if (ok && !stop) {
      it.g = -1;
      ok = put(it);
    }
    if (lane == 0) {
      if (!ok) atomicExch(&bs.abort, 1);
      bs.q_issued[0] = qn[0];
      bs.q_issued[1] = qn[1];
      bs.k_issued = kn;
      bs.v_issued = vn;
    }
  } else if (warp == MMA_WARP || warp == MMA_WARP + 1) {
    // issuer of Q tile t (the whole warp runs the loop; one elected lane
    // issues). Step j: P_{j-1} V_{j-1}, then S_j into the columns P_{j-1} lay
    // in (products of one thread complete in order). The two issuers take
    // turns step by step: both tiles' products side by side would end
    // together, and both softmaxes run side by side after them; in turns, one
    // tile's softmax runs beside the other's products. They wait on every K
    // and V tile of the item, so that their arrivals on the empty barriers
    // stay in step; a tile past the causal range gets a plain arrival. cs
    // counts this Q tile's score tiles over the items, qi its items, step the
    // steps of all items.
    const int t = warp - MMA_WARP;
    const uint32_t idesc_s = umma_idesc_bf16(ROWS, KT), idesc_sh = umma_idesc_bf16(ROWS, HALF);
    const uint32_t idesc_o = umma_idesc_bf16(ROWS, HEAD_DIM) | (1u << 16);  // B (V) MN-major
    const uint32_t qt = sbase + t * Q_TILE;
    const uint32_t s_at = tmem + t * S_COLS, o_at = tmem + O_COL + t * O_COLS;
    unsigned u0 = 0, cs = 0, qi = 0, step = 0;
    bool ok = true;
    auto wait = [&](uint64_t& bar, unsigned parity) {
      return ok = wait_bar(bs, bar, parity);
    };
    // the stage is free once this issuer's products on it are done (a commit
    // covers every product the thread issued before it)
    auto release = [&](uint64_t& bar, bool used) {
      if (elect_one()) {
        if (used) umma_commit(smem_u32(&bar));
        else mbar_arrive(smem_u32(&bar));
      }
      __syncwarp();
    };
    while (ok && walk.next(bs, it)) {
      if (it.n == 0) continue;
      const int n_t = t ? it.nt[1] : it.nt[0];
      const int end_t = min(it.kv_end, it.start + it.q0 + (t + 1) * qp);  // keys of this Q tile
      for (int j = 0; j <= it.n; ++j, ++step) {
        // everything S_j needs but its turn, so that it follows P_{j-1} V_{j-1} at once
        const unsigned uk = u0 + j, sk = uk % STAGES;
        if (j < it.n && !wait(bs.k_full[sk], (uk / STAGES) & 1)) break;
        if (j == 0 && n_t > 0 && !wait(bs.q_full[t], qi & 1)) break;
        const uint32_t kt = sbase + K_OFF + sk * KV_TILE;
        const uint32_t idesc = end_t - (it.j0 + j) * KT > HALF ? idesc_s : idesc_sh;
        if (j >= 1) {
          const int i = j - 1, tile = it.j0 + i;
          const unsigned u = u0 + i, s = u % STAGES;
          if (!wait(bs.v_full[s], (u / STAGES) & 1)) break;
          const uint32_t vt = sbase + V_OFF + s * KV_TILE;
          const bool second = end_t - tile * KT > HALF;
          if (i < n_t) {
            const int left = it.kv_end - tile * KT, read = second ? KT : HALF;
            if (left < read) {
              // clear the value rows that are not the item's (both issuers
              // write the same zeros)
              for (int w = lane; w < (read - left) * 16; w += 32) {
                const int row = left + (w >> 4);
                st_shared_v4(vt + ((w >> 3) & 1) * KV_HALF + row * 128 + (w & 7) * 16, make_uint4(0, 0, 0, 0));
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            // P of the item's first key tile also tells that the softmax
            // warps have read the previous item's O (their epilogue comes
            // first), so that the first product may overwrite it
            if (!wait(bs.p_full[t][0], (cs + i) & 1)) break;
          }
          if (t == 0 ? step > 0 && !wait(bs.turn[1], (step - 1) & 1) : !wait(bs.turn[0], step & 1)) break;
          if (i < n_t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1 && !wait(bs.p_full[t][1], (cs + i) & 1)) break;
              tc_fence_after();
              if (h == 1 && !second) break;  // no visible keys in the second half
              if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < HALF / 16; ++ks)
                  umma_bf16_ts(o_at, s_at + h * (HALF / 2) + ks * 8,
                               umma_desc_sw128_mn(vt + (h * HALF + ks * 16) * 128, KV_HALF), idesc_o,
                               (i > 0 || h > 0 || ks > 0) ? 1u : 0u);
              }
              __syncwarp();
            }
            if (!ok) break;
          }
        } else if (t == 0 ? step > 0 && !wait(bs.turn[1], (step - 1) & 1) : !wait(bs.turn[0], step & 1)) {
          break;
        }
        if (j < n_t) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < HEAD_DIM / 16; ++ks) {
              const uint32_t off = (ks & 3) * 32;
              umma_bf16(s_at, umma_desc_sw128(qt + (ks >> 2) * Q_HALF + off),
                        umma_desc_sw128(kt + (ks >> 2) * KV_HALF + off), idesc, ks > 0 ? 1u : 0u);
            }
            umma_commit(smem_u32(&bs.s_full[t]));
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(smem_u32(&bs.turn[t]));
        if (j >= 1) {
          if (j == n_t) {
            if (elect_one()) umma_commit(smem_u32(&bs.o_done[t]));
            __syncwarp();
          }
          release(bs.v_empty[(u0 + j - 1) % STAGES], j <= n_t);
        }
        if (j < it.n) {
          release(bs.k_empty[sk], j < n_t);
        }
      }
      if (!ok) break;
      u0 += it.n;
      cs += n_t;
      qi += n_t > 0;
    }
    if ((!ok || !walk.ok) && lane == 0) atomicExch(&bs.abort, 1);
    if (elect_one()) umma_commit(smem_u32(&bs.mma_done[t]));
    __syncwarp();
    mbar_wait(smem_u32(&bs.mma_done[t]), 0);
  } else {
    // softmax / epilogue: warpgroup t, thread r owns row r = TMEM lane r of Q tile t
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int rp = r / nrep, hh = r - rp * nrep;
    const bool used = rp < qp;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + t * S_COLS + lanes, o_at = tmem + O_COL + t * O_COLS + lanes;
    const float scale = a.scale_log2;
    unsigned cs = 0;  // score tiles of this Q tile over the items (as the issuer counts them)
    unsigned syncs = 0, items = 0;  // items with keys of this Q tile
    bool ok = true;
    while (ok && walk.next(bs, it)) {
      const int n_t = t ? it.nt[1] : it.nt[0];
      const int pos = it.q0 + t * qp + rp;  // query index within the sequence
      const bool real = used && pos < it.T;
      const int end_t = min(it.kv_end, it.start + it.q0 + (t + 1) * qp);  // keys of this Q tile
      const int lim = used ? min(it.start + pos, it.kv_end - 1) : -1;  // last key this row sees
      // the item's first output row, and this thread's elements behind it (-1: no row)
      __nv_bfloat16* out = a.out + (static_cast<size_t>(it.row0) + it.q0) * a.n_heads * HEAD_DIM;
      const int dst_off = real ? ((pos - it.q0) * a.n_heads + it.g * nrep + hh) * HEAD_DIM : -1;
      if (it.n == 0 && real) {
#pragma unroll 1
        for (int e = 0; e < HEAD_DIM / 8; ++e) reinterpret_cast<uint4*>(out + dst_off)[e] = make_uint4(0, 0, 0, 0);
      }
      float m_ref = -INFINITY;  // max the current P values and O are taken against (raw score units)
      float l = 0.f;
      float m_limit = -INFINITY, neg = 0.f;  // max that P is still taken against m_ref with; -m_ref in log2 units
      for (int j = 0; j < n_t; ++j) {
        // S_j is there, and with it every product before it, P_{j-1} V_{j-1} among them
        if (!wait_bar(bs, bs.s_full[t], (cs + j) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int tile = it.j0 + j;
        const bool second = end_t - tile * KT > HALF;
        const int vis = lim - tile * KT;  // columns 0..vis are visible to this row
        // columns of half h, keys past the row's position at -inf; the second
        // half is read for the max first and again for its P (registers)
        uint32_t sr[HALF];
        auto load = [&](int h) {
          tmem_ld32(s_at + h * HALF, sr);
          tmem_ld32(s_at + h * HALF + 32, sr + 32);
          tmem_ld_wait();
          if (vis < h * HALF + HALF - 1) {
#pragma unroll
            for (int cc = 0; cc < HALF; ++cc)
              if (h * HALF + cc > vis) sr[cc] = __float_as_uint(-INFINITY);
          }
          __syncwarp();  // the TMEM accesses want the warp converged
        };
        float mx = -INFINITY, m1 = mx, m2 = mx, m3 = mx;
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          if (h == 1 && !second) continue;
          load(h);
#pragma unroll
          for (int cc = 0; cc < HALF; cc += 8) {
            mx = max3(mx, __uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1]));
            m1 = max3(m1, __uint_as_float(sr[cc + 2]), __uint_as_float(sr[cc + 3]));
            m2 = max3(m2, __uint_as_float(sr[cc + 4]), __uint_as_float(sr[cc + 5]));
            m3 = max3(m3, __uint_as_float(sr[cc + 6]), __uint_as_float(sr[cc + 7]));
          }
        }
        mx = fmaxf(max3(mx, m1, m2), m3);
        // the max outgrew the reference (always at a row's first keys)
        if (__any_sync(0xffffffffu, mx > m_limit)) {
          float alpha = 1.f;
          if (mx > m_limit) {
            alpha = m_ref == -INFINITY ? 0.f : ex2_approx((m_ref - mx) * scale);
            m_ref = mx;
            m_limit = mx + RESCALE_LOG2 / scale;
            neg = -mx * scale;
            l *= alpha;
          }
          if (j > 0) {
#pragma unroll 1
            for (int cc = 0; cc < HEAD_DIM; cc += 32) {
              uint32_t o[32];
              __syncwarp();
              tmem_ld32(o_at + cc, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_at + cc, o);
            }
          }
          __syncwarp();
        }
        // exponent arguments and the row sum two columns per instruction
        const float2 sc2 = make_float2(scale, scale), ng2 = make_float2(neg, neg);
        float2 sum2 = make_float2(0.f, 0.f), sum3 = sum2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0 || second) {
            if (h == 1) load(1);
            uint32_t pk[HALF / 2];
#pragma unroll
            for (int cc = 0; cc < HALF; cc += 4) {
              const float2 e = fma2(make_float2(__uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1])), sc2, ng2);
              const float2 f =
                  fma2(make_float2(__uint_as_float(sr[cc + 2]), __uint_as_float(sr[cc + 3])), sc2, ng2);
              const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              const float2 q = make_float2(ex2_approx(f.x), ex2_approx(f.y));
              sum2 = add2(sum2, p);
              sum3 = add2(sum3, q);
              pk[cc >> 1] = pack_bf16(p.x, p.y);
              pk[(cc >> 1) + 1] = pack_bf16(q.x, q.y);
            }
            tmem_st32(s_at + h * (HALF / 2), pk);
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bs.p_full[t][h]));
          __syncwarp();
        }
        sum2 = add2(sum2, sum3);
        l += sum2.x + sum2.y;
      }
      if (!ok) break;
      if (n_t > 0) {
        if (!wait_bar(bs, bs.o_done[t], items & 1)) {
          ok = false;
          break;
        }
        ++items;
        tc_fence_after();
      }
      bool whole = true;
      // of a shared item that is joined here: the factor of this CTA's O, the
      // other parts' slots and factors
      float w_own = 1.f, w_part[DIRECT] = {};
      size_t at_part[DIRECT] = {};
      int nparts = 0;
      bool behind = false;  // its part comes after the others
      if (it.first != it.last) {
        // Of few parts, the CTA that arrives last at the item's ticket adds the
        // others (they have arrived, so they are running and about to write
        // theirs) to its own, in CTA order all the same. More are left to the
        // second kernel. A CTA arrives with the last of its warps: one may still
        // be computing rows of the item before again, which takes any time.
        const int c = blockIdx.x, others = it.last - it.first;
        int* arrived = a.tickets + 2 * it.first;
        if (others <= DIRECT) {
          if (lane == 0 && atomicAdd(&bs.warps_here, 1) == 7) {
            bs.warps_here = 0;
            bs.is_last = atomicAdd(arrived, 1) == others;
          }
          if (!softmax_sync(bs, syncs)) {
            ok = false;
            break;
          }
          whole = bs.is_last;
        } else {
          whole = false;
        }
        const float m2 = l > 0.f || l != l ? m_ref * scale : -INFINITY;
        const int span = Rows(it, qp, nrep).span;
        if (!whole) {
          const size_t slot = part_slot(c, it.first);
          if (real) __stcg(part_ml(a, slot) + t * ROWS + r, make_float2(m2, l));
          __syncwarp();
#pragma unroll 1
          for (int cc = 0; cc < HEAD_DIM; cc += 32) {
            uint32_t o[32];
            if (n_t > 0) {
              tmem_ld32(o_at + cc, o);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            if (real) {
              float4* o4 = part_o(a, slot) + (cc / 4) * span + t * ROWS + r;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __stcg(o4 + e * span, make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                  __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
            }
            __syncwarp();
          }
        }
        if (others <= DIRECT) {
          if (whole && threadIdx.x == 0) {
            // the others' parts are written
            bs.parts_there = wait_counter(arrived + 1, others, a.wait_ns);
            arrived[0] = 0;
            arrived[1] = 0;
          }
          if (!softmax_sync(bs, syncs) || (whole && !bs.parts_there)) {
            ok = false;
            break;
          }
          if (!whole && threadIdx.x == 0) signal_counter(arrived + 1, 1);  // all warps' parts: the barrier is before it
        }
        if (whole) {
          static_assert(DIRECT == 2, "the two parts below");
          nparts = others;
          float2 ml[DIRECT];
#pragma unroll
          for (int d = 0; d < DIRECT; ++d) {
            const int o = it.first + d + (it.first + d >= c);  // the d-th other CTA
            at_part[d] = part_slot(o, it.first);
            ml[d] = d < others && real ? __ldcg(part_ml(a, at_part[d]) + t * ROWS + r) : make_float2(-INFINITY, 0.f);
          }
          float m = max3(m2, ml[0].x, ml[1].x);
          if (m == -INFINITY) m = 0.f;
          w_own = ex2_approx(m2 - m);
#pragma unroll
          for (int d = 0; d < DIRECT; ++d) w_part[d] = ex2_approx(ml[d].x - m);
          behind = c == it.last;
          l = in_order(behind, __fmul_rn(w_own, l), __fmul_rn(w_part[0], ml[0].y), __fmul_rn(w_part[1], ml[1].y));
        }
      }
      if (whole && (n_t > 0 || it.first != it.last)) {
        __syncwarp();
        const float inv = 1.f / l;
        uint8_t* turn_at = smem + OUT_OFF + warp * OUT_WARP;
        float chk = 0.f;  // NaN when any value of the row is not finite
#pragma unroll 1
        for (int cc = 0; cc < HEAD_DIM; cc += 32) {
          uint32_t o[32];
          if (n_t > 0) {
            tmem_ld32(o_at + cc, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (nparts > 0 && real) {
            const int span = Rows(it, qp, nrep).span, at = (cc / 4) * span + t * ROWS + r;
            const float4 *o0 = part_o(a, at_part[0]) + at, *o1 = part_o(a, at_part[1]) + at;
            float4 x[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] = __ldcg(o0 + e * span);
              y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (nparts > 1) y[e] = __ldcg(o1 + e * span);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float xe[4] = {x[e].x, x[e].y, x[e].z, x[e].w}, ye[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[4 * e + k] = __float_as_uint(in_order(behind, __fmul_rn(__uint_as_float(o[4 * e + k]), w_own),
                                                        __fmul_rn(xe[k], w_part[0]), __fmul_rn(ye[k], w_part[1])));
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) chk = fmaf(__uint_as_float(o[e]), 0.f, chk);
          // Rows are turned round in shared memory, so that four lanes store
          // 64 bytes of a row (a lane storing its own row's 16 bytes at a
          // time touches 32 lines an instruction: 1.8 us an item).
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(o[8 * e + 0]) * inv, __uint_as_float(o[8 * e + 1]) * inv);
            w.y = pack_bf16(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv);
            w.z = pack_bf16(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv);
            w.w = pack_bf16(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv);
            *reinterpret_cast<uint4*>(turn_at + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4)) = w;
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 8 * e + (lane >> 2), piece = lane & 3;
            const uint4 w = *reinterpret_cast<const uint4*>(turn_at + row * 64 + ((piece ^ (row >> 1 & 3)) << 4));
            const int off = __shfl_sync(0xffffffffu, dst_off, row);
            if (off >= 0)
              reinterpret_cast<uint4*>(out + off + cc)[piece] = w;
          }
          __syncwarp();
        }
        unsigned again = __ballot_sync(0xffffffffu, real && chk != chk && lim < it.kv_end - 1);
        for (; again; again &= again - 1) {
          const int src = __ffs(again) - 1;
          masked_row(a, it.b, it.row0, it.g, it.start, __shfl_sync(0xffffffffu, pos, src),
                     it.g * nrep + __shfl_sync(0xffffffffu, hh, src), it.kv_end, &bs.alive);
        }
      }
      cs += n_t;
    }
    if ((!ok || !walk.ok) && lane == 0) atomicExch(&bs.abort, 1);
  }

  tc_fence_before();
  __syncthreads();
  if (aborted(bs)) {
    if (threadIdx.x == 0) report(a.status, DEV_WAIT_TIMEOUT);
    if (warp == PRODUCER_WARP && lane == 0) {
      // the last copy into each buffer may still be in flight
      for (int t = 0; t < NQ; ++t)
        if (bs.q_issued[t] > 0) mbar_wait(smem_u32(&bs.q_full[t]), (bs.q_issued[t] - 1) & 1);
      for (int u = max(0, bs.k_issued - STAGES); u < bs.k_issued; ++u)
        mbar_wait(smem_u32(&bs.k_full[u % STAGES]), (u / STAGES) & 1);
      for (int u = max(0, bs.v_issued - STAGES); u < bs.v_issued; ++u)
        mbar_wait(smem_u32(&bs.v_full[u % STAGES]), (u / STAGES) & 1);
    }
    __syncthreads();
  }
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  // what the second kernel has to join: the item that this CTA's range begins
  // and does not end
  if (a.joins && threadIdx.x == 0) {
    Item it = {};
    if (equal && static_cast<int>(blockIdx.x) < parts) {
      const Split split(units, parts);
      const int end = split.start(blockIdx.x + 1);
      int u = end - 1;
      it = ranged_item(u, end, split, E, bs.cum, pre, qp, a);
      if (it.first != static_cast<int>(blockIdx.x)) it.last = it.first;
    }
    reinterpret_cast<Item*>(a.joins)[blockIdx.x] = it;
  }
  // the last CTA out clears the claims for the next call
  if (threadIdx.x == 0 && claim) {
    __threadfence();
    if (atomicAdd(a.claims + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      a.claims[0] = 0;
      a.claims[1] = 0;
    }
  }
}

}  // namespace

// Whether items can come to have parts for the second kernel: no more entries
// than are sorted, and more than 2,048 keys that a sequence may have. The host
// knows only that bound, so this weighs calls that share nothing, which pay for
// an empty kernel (17 tokens 7.1 us without and 9.0 with, 2,048 tokens 36.9 and
// 38.8), against those that would share more (without / with the second kernel,
// 8 and 2 heads: 5 tokens at 512 keys 11.3 / 12.5 us, 1,024 15.7 / 17.2, 1,500
// 18.3 / 15.0, 2,048 20.9 / 15.4; 256 tokens 12.9 / 15.4, 19.0 / 21.6, 24.5 /
// 20.2, 30.0 / 21.7; 32 and 8 heads: 5 tokens 11.4 / 12.7, 16.3 / 20.9, 18.9 /
// 16.5, 21.7 / 16.7; 256 tokens 13.1 / 15.5, 19.1 / 21.8, 24.6 / 27.3, 30.1 /
// 32.9). Few rows after 1,500 to 2,048 keys lose 2 to 8 us by it; whole prompts
// of that length, which it was set for, gain 2.
bool packed_prefill_may_join(int N, int n_rep, long long most_keys) {
  return N / (NQ * (ROWS / n_rep)) <= MAX_SORT && most_keys > 2048;
}
size_t packed_prefill_join_bytes(int ctas) { return ctas * sizeof(Item); }

cudaError_t launch_packed_prefill_join(const PackedPrefillParams& a, cudaStream_t s) {
  // the most rows that an item can span
  const int n_rep = a.n_heads / a.n_kv, qp = ROWS / n_rep;
  const int rows = a.N <= qp ? a.N * n_rep : ROWS + (a.N - qp < qp ? a.N - qp : qp) * n_rep;
  if (rows <= 160)
    return launch_behind(packed_prefill_join_kernel<16>, dim3(a.ctas, (rows + 15) / 16), JOIN_THREADS, 0, s, a);
  return launch_behind(packed_prefill_join_kernel<32>, dim3(a.ctas, (rows + 31) / 32), JOIN_THREADS, 0, s, a);
}

cudaError_t launch_packed_prefill(const PackedPrefillMaps& maps, const PackedPrefillParams& a, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(packed_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  if (a.B <= 0 || a.B > PAGED_MAX_SEQS || a.N <= 0 || a.ctas <= 0) return cudaErrorInvalidValue;
  // one CTA per SM (shared memory and TMEM admit no second), each walking its items
  const unsigned ctas = static_cast<unsigned>(a.ctas);
  return launch_behind(packed_prefill_kernel, ctas, THREADS, SMEM_BYTES, s, maps.q, maps.k, maps.v, a);
}

}  // namespace gqa
