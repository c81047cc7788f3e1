// Attention of one new token per sequence for groups of sequences that share
// their first rows ("Llama 3.1 8B · Grouped-query attention", mode decode): the
// shared rows are read once for a group instead of once for each of its
// sequences, the rows of its own are streamed for each, and the parts, each an
// O, a max and a sum, are joined by the log-sum-exp rule.
//
// The prefix part is matrix-shaped: members x n_rep query rows of a KV head
// against the prefix's keys, 4 x 128 flops a pair, so it runs on the
// 5th-generation tensor cores as the prefill attention does
// (packed_prefill.cu, whose tiles and turns these are), without a causal mask:
//   * An item is two 128-row Q tiles (128 / n_rep sequences x n_rep heads each)
//     of one KV head and the whole prefix. S = Q K^T goes to TMEM, P over it, O +=
//     P V; 128-key tiles, staged once for both Q tiles, whose issuers take turns
//     so that one's softmax runs beside the other's products.
//   * P enters the product as two bf16 terms, as in paged_decode.cu: the upper 16
//     bits and the rest, each over half of the columns of the scores that it
//     comes from, O += hi V + lo V. A sequence is then as exact in a batch that
//     shares as in one that does not, for a third product: with prefixes of
//     32,000 rows and more a tile takes 1.85 us for 1.54, with two Q tiles 2.25 for 1.76.
//   * The key tiles of all items, ITEM_UNITS more for each, are cut into one equal
//     range per CTA. A CTA's piece of an item leaves a part in the workspace,
//     at (rows of the items before) + 256 x CTA: from one piece to the next
//     either grows by what the last one took, so that no two meet.
//   * All rows of a Q tile see all keys, so only the last tile is masked, and
//     value rows behind the prefix are cleared in shared memory.
// The own rows are bound by memory and streamed as in paged_decode.cu
// (decode_stream.cuh). One kernel does both: some of its CTAs, one per SM, take
// the prefixes, the others the own rows, as many each as makes both end
// together by measured costs; every CTA plans alike. A second kernel joins.
// Which sequences share: the members of a group, those that see all of its
// prefix (start_pos + 1 >= prefix_rows). Its items reach from the first of them to
// the last, so the prefix is read once for each NQ Q tiles in between. It shares if
// that is less often than for each member by itself, and if the batch saves
// enough rows in all. The others are streamed from their row 0 on; where they lie
// between members, in rows of the Q tiles that nobody reads.
//
// Warps of a CTA with prefixes:
//   warp 8        TMA producer: 128 / min(page, 128) boxes a tile, one lane each
//   warps 9, 10   MMA issuers, one per Q tile
//   warps 0-3/4-7 one softmax warpgroup per Q tile, one thread per row
// Sums are fp32 of the probabilities before they are cut in two. Every wait is
// bounded (gqa_set_wait_limit_ns); one that gives up records DEV_WAIT_TIMEOUT, lets
// issued copies and products finish and frees TMEM before the CTA exits.
//
// Measured (GB300, 6.8 TB/s copied): 35.8 us for 64 sequences with up to 512
// rows of their own under a prefix of 8,000 (103 MB), 49.7 for 96 under
// three prefixes of up to 4,095 (210 MB), 22.8 for 32 under 8,000 with up to 8
// rows of their own; 64 sequences with 16 query heads per KV head 37.2 (4 KV heads,
// two prefixes of up to 6,000) and 25.9 (one, a prefix of 8,000), with one 95.6 (32
// KV heads, a prefix of 8,000, 408 MB). Of the first, when P was one term (33.7):
// 3.8 us to plan, then 3 to the first chunks and 4 to the first scores, 15 to 20 of
// streaming and products at 4 to 5 TB/s together, 1.2 for a part's way to memory, 6
// from the last CTA's end to that of the join. Three launches (prefixes, own rows,
// join) took 68.5; own rows joined in their CTAs 53. Slower were: one Q tile's key
// tiles shared out between the two issuers (70 us for 60: two stages do not hide
// the memory for both), and L2 asked for tiles ahead, once pages are looked up ahead
// (54 us for 48.5, a prefix of 32,000).
#include <math.h>

#include "decode_stream.cuh"

namespace gqa {

namespace {

constexpr int ROWS = 128;                 // rows of a Q tile = MMA M
constexpr int NQ = 2;                     // Q tiles per CTA
constexpr int KT = PACKED_TILE;           // keys per tile
constexpr int HALF = KT / 2;
constexpr int STAGES = 2;                 // K tiles and V tiles in shared memory
constexpr int Q_HALF = ROWS * 128;        // 128 rows x 64 dims
constexpr int Q_TILE = 2 * Q_HALF;
constexpr int KV_HALF = KT * 128;         // 128 keys x 64 dims
constexpr int KV_TILE = 2 * KV_HALF;
constexpr int K_OFF = NQ * Q_TILE;
constexpr int V_OFF = K_OFF + STAGES * KV_TILE;
constexpr int BAR_OFF = V_OFF + STAGES * KV_TILE;
constexpr int BARS_BYTES = 1024;
constexpr int PLAN_OFF = BAR_OFF + BARS_BYTES;
constexpr int PLAN_ARRAY = SHARED_MAX_GROUPS + 1;
constexpr int SMEM_BYTES = PLAN_OFF + 6 * PLAN_ARRAY * 4 + 1024;
constexpr int THREADS = 352;
// Shared memory of a CTA with own rows: four numbers of each sequence, then the
// warps' rings.
__host__ __device__ constexpr int own_ints(int B) { return ((4 * B + 1) * 4 + 127) / 128 * 128; }
static_assert(own_ints(PAGED_MAX_SEQS) <= K_OFF &&
              own_ints(PAGED_MAX_SEQS) + decode::WARPS * decode::RING_BYTES <= BAR_OFF, "the plan is not in the way");
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
// Costs in us, measured with CTAs of both kinds running: a key tile (or unit) of
// an item with one and with two Q tiles, a chunk of own rows by a CTA (with 8
// query heads per KV head at most, and with more) and by the whole memory, and
// what a CTA of either kind takes beside. A tenth more or less of them changes the
// time by 1 or 2%.
constexpr float ONE_TILE = 2.4f, TWO_TILES = 2.2f, CHUNK = 0.15f, WIDE_CHUNK = 0.2f, CHUNK_MEMORY = 1.f / 750,
                PREFIX_MORE = 8.f, OWN_MORE = 5.f;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9;  // MMA warps 9 (Q tile 0) and 10 (Q tile 1)
constexpr int SLOTS = 2;                        // items handed from the producer to the other warps
constexpr uint32_t TMEM_COLS = 512;
// TMEM columns: S (128; P over it, of each half of the keys its upper and its lower
// terms) of Q tiles 0 and 1, then O of both
constexpr uint32_t S_COLS = 128, O_COL = 256, O_COLS = 128;
constexpr float RESCALE_LOG2 = 8.f;
// The exponent of a score is s x scale - m in one rounding, m = m_ref x scale rounded:
// off by half a step of m for all alike, which cancels, but past 2^30 is no
// exponent any more. From here on m_ref is taken off the scores instead.
constexpr float FAR = 0x1p24f;

// A CTA's piece of an item: KV head g, sequences seq0 .. seq0 + nseq - 1, key
// tiles j0 .. j0 + n - 1 of the prefix's `end` keys, read by sequence lead's
// table; its part's first row in the workspace.
struct Item {
  int g, seq0, nseq, lead, end, j0, n;
  int base;
  // key tiles of Q tile t (qp: sequences per Q tile)
  __device__ __forceinline__ int tiles(int t, int qp) const { return nseq > t * qp ? n : 0; }
};

struct Bars {
  uint64_t q_full[NQ];
  uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
  uint64_t s_full[NQ], p_full[NQ][2];  // p_full: the first and the second half of the keys
  uint64_t turn[NQ];                   // the issuer of Q tile t has issued a step
  uint64_t o_done[NQ], mma_done[NQ];
  uint64_t item_full[SLOTS], item_empty[SLOTS];
  uint32_t tmem_slot;
  int abort;
  unsigned long long wait_ns;  // limit of the waits
  int q_issued[NQ], k_issued, v_issued;
  int warp_sum[THREADS / 32][2];
  unsigned long long saved;    // rows that sharing saves
  unsigned long long tiles[2]; // units of items with one and with two Q tiles
  unsigned long long best;     // least cost (float bits) << 32 | CTAs with prefixes
  Item item[SLOTS];            // g < 0: no more
};
static_assert(sizeof(Bars) <= BARS_BYTES, "barrier block");

__device__ __forceinline__ bool aborted(const Bars& bs) { return *reinterpret_cast<const volatile int*>(&bs.abort) != 0; }

// Wait of a whole warp for phase `parity` of a barrier; false when it gave up.
__device__ __noinline__ bool wait_longer(const Bars& bs, uint32_t bar, unsigned parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, bs.wait_ns));
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

// The groups in shared memory: sequences cu[g] .. cu[g+1]-1, the rows that they
// share; lead and size: the first of those that see them all, and how many
// sequences there are from it to the last (while members are counted: the last);
// prefix sums of the units of one KV head and of the query rows of one KV head (no
// step: does not share).
struct Groups {
  int *cu, *prefix, *lead, *size, *units, *rows;
};

// Two probabilities as bf16 pairs: their upper 16 bits, and the rest. The rest is
// above 0 where the probability is (a 2^-23 of it is added, far below its own
// rounding of 2^-15, and 2^-133, the least bf16), so that an infinite value gives
// an infinite sum and not a NaN.
__device__ __forceinline__ void two_terms(float2 p, uint32_t& hi, uint32_t& lo) {
  const uint32_t u0 = __float_as_uint(p.x), u1 = __float_as_uint(p.y);
  hi = __byte_perm(u0, u1, 0x7632);
  const float2 minus = make_float2(__uint_as_float((u0 & 0xffff0000u) ^ 0x80000000u),
                                   __uint_as_float((u1 & 0xffff0000u) ^ 0x80000000u));
  const float2 rest = add2(fma2(p, make_float2(1.f + 0x1p-23f, 1.f + 0x1p-23f), minus), make_float2(0x1p-133f, 0x1p-133f));
  lo = pack_bf16(rest.x, rest.y);
}

__device__ __forceinline__ int tiles_of(int prefix) { return ceil_div(prefix, KT); }

template <int NT>
__global__ void __launch_bounds__(THREADS, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const __grid_constant__ SharedDecodeParams sp) {
  const PagedDecodeParams& a = sp.own;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bs = *reinterpret_cast<Bars*>(smem + BAR_OFF);
  __shared__ decode::Shared sh;
  int* plan = reinterpret_cast<int*>(smem + PLAN_OFF);
  const Groups gs{plan, plan + PLAN_ARRAY, plan + 2 * PLAN_ARRAY, plan + 3 * PLAN_ARRAY, plan + 4 * PLAN_ARRAY,
                  plan + 5 * PLAN_ARRAY};
  // of each sequence: chunks of own rows before it, its last row, its first own
  // one, its group (-1: it does not share)
  int* pre = reinterpret_cast<int*>(smem);
  int *last = pre + a.B + 1, *begin = last + a.B, *group = begin + a.B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int nrep = a.n_heads / a.n_kv;
  const int qp = ROWS / nrep;  // sequences per Q tile

  if (tid == 0) {
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
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&bs.item_full[s]), 1);
      mbar_init(smem_u32(&bs.item_empty[s]), 10);  // issuers, softmax warps
    }
    bs.abort = 0;
    bs.wait_ns = sp.wait_ns;
    bs.q_issued[0] = bs.q_issued[1] = 0;
    bs.k_issued = bs.v_issued = 0;
    bs.saved = bs.tiles[0] = bs.tiles[1] = 0;
    bs.best = ~0ull;
    fence_barrier_init();
  }
  // nothing in global memory is read or written before the previous kernel of
  // the stream is done
  pdl_trigger();
  pdl_wait();

  // ---- the plan, from one look at what it takes. Members of each group
  // (counted where K tiles will lie), the first and the last of them.
  int* members = reinterpret_cast<int*>(smem + K_OFF);
#pragma unroll 1
  for (int b = tid; b < a.B; b += THREADS) last[b] = a.start[b];
  bool bad = false;
#pragma unroll 1
  for (int g = tid; g <= sp.G; g += THREADS) {
    const int c = sp.cu[g];
    gs.cu[g] = c;
    bad |= c < 0 || c > a.B || (g < sp.G && c > sp.cu[g + 1]);
    if (g < sp.G) {
      gs.prefix[g] = sp.prefix[g];
      members[g] = 0;
      gs.lead[g] = a.B;
      gs.size[g] = -1;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && tid == 0) report(a.status, DEV_BAD_POSITION);
  // the group of a sequence whose prefix it sees whole, or -1
#pragma unroll 1
  for (int b = tid; b < a.B; b += THREADS) {
    int g = -1;
    if (!bad && b >= gs.cu[0] && b < gs.cu[sp.G]) {
      int lo = 0, hi = sp.G;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (gs.cu[mid] <= b) lo = mid; else hi = mid;
      }
      const int p = gs.prefix[lo];
      if (p > 0 && last[b] >= p - 1 && last[b] < a.pages.capacity()) {
        g = lo;
        atomicAdd(&members[g], 1);
        atomicMin(&gs.lead[g], b);
        atomicMax(&gs.size[g], b);
      }
    }
    group[b] = g;
  }
  __syncthreads();
  {
    const int per = ceil_div(sp.G, THREADS);
    const int g0 = min(tid * per, sp.G), g1 = min(g0 + per, sp.G);
    unsigned long long saved = 0;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      gs.size[g] = members[g] ? gs.size[g] - gs.lead[g] + 1 : 0;
      // reads that there are fewer
      members[g] -= members[g] ? ceil_div(gs.size[g], NQ * qp) : 0;
      if (members[g] > 0) saved += static_cast<unsigned long long>(members[g]) * gs.prefix[g];
    }
    if (saved) atomicAdd(&bs.saved, saved);
    __syncthreads();
    const bool shares = bs.saved * a.n_kv >= SHARED_LEAST_ROWS;
    int sum[2] = {0, 0};
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      const int size = gs.size[g];
      const bool on = shares && members[g] > 0;
      const int units = on ? ceil_div(size, NQ * qp) * (tiles_of(gs.prefix[g]) + ITEM_UNITS) : 0;
      gs.units[g + 1] = units;
      gs.rows[g + 1] = on ? size * nrep : 0;
      sum[0] += units;
      sum[1] += gs.rows[g + 1];
      if (on) atomicAdd(&bs.tiles[size > qp], static_cast<unsigned long long>(units));
    }
    int run[2] = {sum[0], sum[1]};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, run[k], o);
        if (lane >= o) run[k] += x;
      }
      if (lane == 31) bs.warp_sum[warp][k] = run[k];
    }
    if (tid == 0) gs.units[0] = gs.rows[0] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) run[k] += __reduce_add_sync(0xffffffffu, lane < warp ? bs.warp_sum[lane][k] : 0) - sum[k];
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      run[0] += gs.units[g + 1];
      run[1] += gs.rows[g + 1];
      gs.units[g + 1] = run[0];
      gs.rows[g + 1] = run[1];
    }
  }
  __syncthreads();
  const int units = gs.units[sp.G] * a.n_kv;
  // the own rows' chunks
  const decode::Count count = decode::count_chunks<THREADS / 32>(sh, pre, a.B, [&](int b) {
    const int s = last[b], g = group[b];
    const bool ok = s >= 0 && s < a.pages.capacity();
    if (!ok && s != -1 && blockIdx.x == 0) report(a.status, DEV_BAD_POSITION);
    const bool shares = g >= 0 && gs.units[g + 1] > gs.units[g];
    const int first = shares ? gs.prefix[g] : 0;
    if (!shares) group[b] = -1;
    begin[b] = first;
    return ok && s >= first ? s / decode::KEYS - first / decode::KEYS + 1 : 0;
  });
  // rows of sequences without keys
#pragma unroll 1
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (pre[b + 1] == pre[b] && begin[b] == 0) decode::zero_rows(a.out, b, a.n_heads);
  // how many CTAs take prefixes: thread n looks at n of them
  const int chunks = count.total * a.n_kv, grid = gridDim.x;
  if (units > 0 && warp * 32 <= grid) {
    const float tile = static_cast<float>(bs.tiles[0]) * ONE_TILE + static_cast<float>(bs.tiles[1]) * TWO_TILES;
    float cost = INFINITY;
    if (tid > 0 && tid <= grid && (tid < grid || chunks == 0)) {
      const float chunk = (NT > 1 ? WIDE_CHUNK : CHUNK) / (grid - tid);
      const float own = chunks > 0 ? chunks * fmaxf(chunk, CHUNK_MEMORY) + OWN_MORE : 0.f;
      cost = fmaxf(tile * a.n_kv / tid + PREFIX_MORE, own);
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(cost));
    const unsigned who = __ballot_sync(0xffffffffu, __float_as_uint(cost) == least);
    if (lane == 0) atomicMin(&bs.best, static_cast<unsigned long long>(least) << 32 | (tid + __ffs(who) - 1));
  }
  fence_proxy_async_smem();  // tiles come where the counts lie
  __syncthreads();
  const int most = units ? static_cast<int>(bs.best & 0xffffffffu) : 0;
  const int parts = units ? range_count(units, mean_range(units, most), most) : 0;  // CTAs with prefixes
  const int own_ctas = chunks ? full_ctas(chunks, grid - parts, decode::WARPS) : 0;
  // where the parts of a sequence's KV head will lie, for the join
  auto tell = [&](int pair) {
    const int b = pair / a.n_kv, h = pair - b * a.n_kv, g = group[b];
    SharedParts r = {};
    if (g >= 0) {
      const int i = b - gs.lead[g], size = gs.size[g], e = i / (NQ * qp), w = tiles_of(gs.prefix[g]) + ITEM_UNITS;
      const int unit = gs.units[g] * a.n_kv + h * (gs.units[g + 1] - gs.units[g]) + e * w;
      const Split split(units, parts);
      const int c0 = split.holder(unit + ITEM_UNITS);
      r.prefixes = split.holder(unit + w - 1) - c0 + 1;
      r.prefix = gs.rows[g] * a.n_kv + (h * size + e * NQ * qp) * nrep + NQ * ROWS * c0;
      r.span = min(NQ * qp, size - e * NQ * qp) * nrep;
      r.at = (i - e * NQ * qp) * nrep;
    }
    const int n = pre[b + 1] - pre[b];
    if (n > 0) {
      const int first = pre[b] * a.n_kv + h * n;
      const WarpSpan w = warps_of(first, first + n, Split(chunks, own_ctas), least(decode::WARPS, chunks));
      r.own = (pair + w.first) * nrep;
      r.owns = w.last - w.first + 1;
    }
    sp.rows[pair] = r;
  };
  const int pairs = a.B * a.n_kv;
  if (static_cast<int>(blockIdx.x) >= parts) {
    // ---- own rows
    const int cta = blockIdx.x - parts;
    if (warp >= decode::WARPS) {
      // the warps that stream nothing
      constexpr int FREE = THREADS - decode::WARPS * 32;
#pragma unroll 1
      for (int p = cta * FREE + tid - decode::WARPS * 32; p < pairs; p += (grid - parts) * FREE) tell(p);
      return;
    }
    if (cta >= own_ctas) return;
    const Split split(chunks, own_ctas);
    decode::stream_chunks<NT, true>(a, sh, smem + own_ints(a.B), nullptr, pre, last, begin, split, cta, split.start(cta),
                                    split.start(cta + 1));
    return;
  }
  if (parts == grid) {
#pragma unroll 1
    for (int p = blockIdx.x * THREADS + tid; p < pairs; p += grid * THREADS) tell(p);
    // tiles come where the numbers lie
    fence_proxy_async_smem();
    __syncthreads();
  }
  // ---- prefixes
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&bs.tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bs.tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  ItemWalk walk;
  Item it = {};

  if (warp == PRODUCER_WARP) {
    const Split split(units, parts);
    int ru = split.start(blockIdx.x);
    const int rend = split.start(blockIdx.x + 1);
    // units in (group, KV head, pair of Q tiles, key tile) order; this CTA's range of them
    auto next_item = [&](Item& x) {
      while (ru < rend) {
        int lo = 0, hi = sp.G;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (gs.units[mid] * a.n_kv <= ru) lo = mid; else hi = mid;
        }
        const int size = gs.size[lo], w = tiles_of(gs.prefix[lo]) + ITEM_UNITS;
        const int pairs = ceil_div(size, NQ * qp), in_group = ru - gs.units[lo] * a.n_kv;
        const int item = in_group / w, in = in_group - item * w, base = ru - in, end = min(rend, base + w);
        const int e = item % pairs;
        x.g = item / pairs;
        x.seq0 = gs.lead[lo] + e * NQ * qp;
        x.nseq = min(NQ * qp, size - e * NQ * qp);
        x.lead = gs.lead[lo];
        x.end = gs.prefix[lo];
        x.j0 = max(0, in - ITEM_UNITS);
        x.n = max(0, end - base - ITEM_UNITS - x.j0);
        x.base = gs.rows[lo] * a.n_kv + (x.g * size + e * NQ * qp) * nrep + NQ * ROWS * static_cast<int>(blockIdx.x);
        ru = end;
        if (x.n > 0) return true;
      }
      return false;
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
    const int box = prefill_box_rows(1 << a.pages.page_shift);
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
      // Pages of a window of 32 / boxes tiles, a box a lane, and of the next one.
      const int window = 32 / boxes, my_tile = lane / boxes, my_box = lane - my_tile * boxes;
      const int in_page = (1 << a.pages.page_shift) - 1;
      const int* table = a.pages.table + static_cast<long long>(it.lead) * a.pages.table_stride;
      const int keys = min(it.end, (it.j0 + it.n) * KT);  // behind the item's
      auto first_key = [&](int j) { return (it.j0 + j) * KT + my_box * box; };
      auto look_up = [&](int j) {  // the window that begins with tile j
        const int key = first_key(j + my_tile);
        return key < keys ? table[key >> a.pages.page_shift] : -1;
      };
      int pages = 0, next_pages = look_up(0);
      for (int j = 0; j < it.n && !stop; ++j, ++u) {
        const int s = u % STAGES, in_window = j % window;
        if (in_window == 0) {
          pages = next_pages;
          next_pages = look_up(j + window);
        }
        // boxes of the tile that hold keys of the prefix; this lane's
        const int held = min(boxes, (it.end - (it.j0 + j) * KT + box - 1) / box);
        const int row = ((it.j0 + j) * KT + lane * box) & in_page;
        int page = __shfl_sync(0xffffffffu, pages, (in_window * boxes + lane) & 31);
        if (u >= STAGES && !go_on(bs.k_empty[s], (u / STAGES - 1) & 1)) {
          stop = true;
          break;
        }
        if (lane < held && (page < 0 || page >= a.pages.num_pages)) {
          report(a.status, DEV_BAD_PAGE);
          page = 0;
        }
        copy(&mk, bs.k_full[s], sbase + K_OFF + s * KV_TILE, held, it.g, row, page);
        kn = u + 1;
        if (j == 0) {
          // Q tile t is free once the last score product of the previous item
          // that read it has completed
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            if (stop || it.tiles(t, qp) == 0) continue;
            if (cs[t] > 0 && !go_on(bs.s_full[t], (cs[t] - 1) & 1)) {
              stop = true;
              continue;
            }
            if (lane == 0) {
              const uint32_t qb = smem_u32(&bs.q_full[t]);
              mbar_expect_tx(qb, 2 * q_bytes);
              // boxes may reach past the group, or past B (zeros): rows that are never stored
              tma_load_3d(sbase + t * Q_TILE, &mq, qb, 0, it.g * nrep, it.seq0 + t * qp);
              tma_load_3d(sbase + t * Q_TILE + Q_HALF, &mq, qb, 64, it.g * nrep, it.seq0 + t * qp);
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
      for (int t = 0; t < NQ; ++t) cs[t] += it.tiles(t, qp);
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
    // in (products of one thread complete in order); the two issuers take turns
    // step by step. They wait on every K and V tile of the item, so that their
    // arrivals on the empty barriers stay in step. cs counts this Q tile's score
    // tiles over the items, qi its items, step the steps of all items.
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
      const int n_t = it.tiles(t, qp);
      for (int j = 0; j <= it.n; ++j, ++step) {
        // everything S_j needs but its turn, so that it follows P_{j-1} V_{j-1} at once
        const unsigned uk = u0 + j, sk = uk % STAGES;
        if (j < it.n && !wait(bs.k_full[sk], (uk / STAGES) & 1)) break;
        if (j == 0 && n_t > 0 && !wait(bs.q_full[t], qi & 1)) break;
        const uint32_t kt = sbase + K_OFF + sk * KV_TILE;
        const uint32_t idesc = it.end - (it.j0 + j) * KT > HALF ? idesc_s : idesc_sh;
        const unsigned uv = u0 + j - 1, sv = uv % STAGES;
        const uint32_t vt = sbase + V_OFF + sv * KV_TILE;
        const int left = it.end - (it.j0 + j - 1) * KT, read = left > HALF ? KT : HALF;
        if (j >= 1) {
          if (!wait(bs.v_full[sv], (uv / STAGES) & 1)) break;
          if (n_t > 0) {
            if (left < read) {
              // clear the value rows behind the prefix (both issuers write the same zeros)
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
            if (!wait(bs.p_full[t][0], (cs + j - 1) & 1)) break;
          }
        }
        if (t == 0 ? step > 0 && !wait(bs.turn[1], (step - 1) & 1) : !wait(bs.turn[0], step & 1)) break;
        if (j >= 1 && n_t > 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !wait(bs.p_full[t][1], (cs + j - 1) & 1)) break;
            tc_fence_after();
            if (h == 1 && read == HALF) break;  // no keys in the second half
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < HALF / 16; ++ks) {
                const uint64_t v = umma_desc_sw128_mn(vt + (h * HALF + ks * 16) * 128, KV_HALF);
                umma_bf16_ts(o_at, s_at + h * HALF + ks * 8, v, idesc_o, (j > 1 || h > 0 || ks > 0) ? 1u : 0u);
                umma_bf16_ts(o_at, s_at + h * HALF + HALF / 2 + ks * 8, v, idesc_o, 1u);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
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
        if (j >= 1 && j == n_t) {
          if (elect_one()) umma_commit(smem_u32(&bs.o_done[t]));
          __syncwarp();
        }
        if (j >= 1) release(bs.v_empty[sv], n_t > 0);
        if (j < it.n) release(bs.k_empty[sk], n_t > 0);
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
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + t * S_COLS + lanes, o_at = tmem + O_COL + t * O_COLS + lanes;
    const float scale = a.scale_log2;
    unsigned cs = 0;     // score tiles of this Q tile over the items (as the issuer counts them)
    unsigned items = 0;  // items of this Q tile
    bool ok = true;
    while (ok && walk.next(bs, it)) {
      const int n_t = it.tiles(t, qp);
      const int rows = min(qp, it.nseq - t * qp) * nrep;  // of this Q tile
      const bool real = r < rows;
      const bool works = (warp & 3) * 32 < rows;          // some row of this warp is real
      float m_ref = -INFINITY;  // max the current P values and O are taken against (raw score units)
      float l = 0.f;
      float m_limit = -INFINITY, neg = 0.f;  // max that P is still taken against m_ref with; -m_ref in log2 units
      float far = 0.f;                       // m_ref, taken off beforehand, where `neg` would be past FAR (and is 0 then)
      for (int j = 0; j < n_t; ++j) {
        // S_j is there, and with it every product before it, P_{j-1} V_{j-1} among them
        if (!wait_bar(bs, bs.s_full[t], (cs + j) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int vis = it.end - 1 - (it.j0 + j) * KT;  // columns 0..vis are keys
        const bool second = vis >= HALF;
        // columns of half h, what is behind the prefix at -inf; the second
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
        if (works) {
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
              far = 0.f;
              if (!(fabsf(neg) <= FAR)) {
                far = mx;
                neg = 0.f;
              }
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
        }
        // exponent arguments and the row sum two columns per instruction
        const float2 sc2 = make_float2(scale, scale), ng2 = make_float2(neg, neg);
        float2 sum2 = make_float2(0.f, 0.f), sum3 = sum2;
        const bool any_far = __any_sync(0xffffffffu, far != 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (works && (h == 0 || second)) {
            if (h == 1) load(1);
            if (any_far) {
#pragma unroll
              for (int cc = 0; cc < HALF; ++cc) sr[cc] = __float_as_uint(__uint_as_float(sr[cc]) - far);
            }
            uint32_t hi[HALF / 2], lo[HALF / 2];
#pragma unroll
            for (int cc = 0; cc < HALF; cc += 4) {
              const float2 e = fma2(make_float2(__uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1])), sc2, ng2);
              const float2 f =
                  fma2(make_float2(__uint_as_float(sr[cc + 2]), __uint_as_float(sr[cc + 3])), sc2, ng2);
              const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              const float2 q = make_float2(ex2_approx(f.x), ex2_approx(f.y));
              sum2 = add2(sum2, p);
              sum3 = add2(sum3, q);
              two_terms(p, hi[cc >> 1], lo[cc >> 1]);
              two_terms(q, hi[(cc >> 1) + 1], lo[(cc >> 1) + 1]);
            }
            tmem_st32(s_at + h * HALF, hi);
            tmem_st32(s_at + h * HALF + HALF / 2, lo);
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
        // the part: [32 column groups][rows of the item][4] and (max in log2 units, sum)
        if (works) {
          const int span = it.nseq * nrep, row = t * qp * nrep + r;
          const float m2 = l > 0.f || l != l ? m_ref * scale : -INFINITY;
          if (real) __stcg(reinterpret_cast<float2*>(sp.part_ml) + it.base + row, make_float2(m2, l));
          float4* o4 = reinterpret_cast<float4*>(sp.part_o) + static_cast<size_t>(it.base) * (HEAD_DIM / 4) + row;
          __syncwarp();
#pragma unroll 1
          for (int cc = 0; cc < HEAD_DIM; cc += 32) {
            uint32_t o[32];
            tmem_ld32(o_at + cc, o);
            tmem_ld_wait();
            if (real) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __stcg(o4 + static_cast<size_t>(cc / 4 + e) * span,
                       make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
            }
            __syncwarp();
          }
        }
      }
      cs += n_t;
    }
    if ((!ok || !walk.ok) && lane == 0) atomicExch(&bs.abort, 1);
  }

  tc_fence_before();
  __syncthreads();
  if (aborted(bs)) {
    if (tid == 0) report(a.status, DEV_WAIT_TIMEOUT);
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
}

// ---- the join: WAYS warps for R query rows of one (sequence, KV head), which
// share their parts: those of the prefix, one per CTA that holds a piece of its
// item, then those of the own rows, one per warp. 32 / R parts at a time: a lane
// finds the max and sum of a row of one, then the warp adds the parts up in
// order, R float4 of a row a lane. The R rows lie side by side in a prefix's
// part, 16 bytes each. The kernel waits for its code more than for data, so that
// it is short: where parts lie was found out beside the streaming.
constexpr int JOIN_WARPS = 8, JOIN_CTAS = 2;  // CTAs per SM: with three, registers go to local memory, 3 us more
constexpr int MOST_PARTS = 152 * (1 + decode::WARPS);  // of a pair: one per CTA, one per warp
template <int R, int WAYS>
__global__ void __launch_bounds__(JOIN_WARPS * 32, JOIN_CTAS) shared_join_kernel(const __grid_constant__ SharedJoinParams a) {
  constexpr int PARTS = 32 / R, BATCH = 8 / R;
  __shared__ float4 others_o[JOIN_WARPS][R][32];
  __shared__ float2 others_ml[JOIN_WARPS][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rr = lane % R, cg = lane / R;
  const int set = (blockIdx.x * JOIN_WARPS + warp) / WAYS, way = warp % WAYS;  // of R rows
  const int pair = a.sets == 1 ? set : set / a.sets, h = a.sets == 1 ? rr : (set - pair * a.sets) * R + rr;
  const bool real = pair < a.pairs && h < a.n_rep;
  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  SharedParts s = {};
  if (real) s = a.rows[pair];
  const int all = __shfl_sync(0xffffffffu, min(s.prefixes + s.owns, MOST_PARTS), 0);
  float m = -INFINITY, l = 0.f;  // of row rr, the same in its lanes
  float4 o[R];                   // of row rr, dims 4 (cg + PARTS i) ..
#pragma unroll
  for (int i = 0; i < R; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = way; k0 < all; k0 += PARTS * WAYS) {
    // row rr of part k0 + WAYS cg: where its 4-dim groups lie, and how far apart.
    // One of another call (a workspace that two calls use at once) is not read.
    const int k = k0 + cg * WAYS;
    int at = -1, apart = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    const bool own = k >= s.prefixes;
    const int part = own ? s.own + (k - s.prefixes) * a.n_rep : s.prefix + k * (NQ * ROWS);
    if (real && k < all && part >= 0 &&
        (own ? part < a.own_rows - h
             : s.at >= 0 && s.at <= a.part_rows && s.at + h < s.span && s.span <= a.part_rows - part)) {
      ml = reinterpret_cast<const float2*>(own ? a.own_ml : a.part_ml)[part + (own ? 0 : s.at) + h];
      at = own ? a.own_at + (part + h) * (HEAD_DIM / 4) : part * (HEAD_DIM / 4) + s.at + h;
      apart = own ? 1 : s.span;
    }
    const int n = min(PARTS, ceil_div(all - k0, WAYS));
    float4 x[BATCH][R];
    auto load = [&](int i, float4 (&y)[R]) {
      const int from = __shfl_sync(0xffffffffu, at, (i * R + rr) & 31), step = __shfl_sync(0xffffffffu, apart, (i * R + rr) & 31);
#pragma unroll
      for (int e = 0; e < R; ++e)
        y[e] = i < n && from != -1 ? reinterpret_cast<const float4*>(a.parts)[from + (cg + PARTS * e) * step]
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    // the first ones come beside the maxima
#pragma unroll
    for (int i = 0; i < BATCH; ++i) load(i, x[i]);
    float mx = ml.x;
#pragma unroll
    for (int d = R; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    mx = fmaxf(mx, m);
    const float ref = mx == -INFINITY ? 0.f : mx, f = ex2_approx(m - ref), weight = ex2_approx(ml.x - ref);
    float sum = weight * ml.y;
#pragma unroll
    for (int d = R; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    m = mx;
    l = l * f + sum;
#pragma unroll
    for (int e = 0; e < R; ++e) o[e] = make_float4(o[e].x * f, o[e].y * f, o[e].z * f, o[e].w * f);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += BATCH) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (i0 > 0) load(i0 + i, x[i]);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float w = __shfl_sync(0xffffffffu, weight, ((i0 + i) * R + rr) & 31);
#pragma unroll
        for (int e = 0; e < R; ++e) {
          o[e].x += w * x[i][e].x;
          o[e].y += w * x[i][e].y;
          o[e].z += w * x[i][e].z;
          o[e].w += w * x[i][e].w;
        }
      }
    }
  }
  if (WAYS > 1) {
    if (way) {
#pragma unroll
      for (int e = 0; e < R; ++e) others_o[warp][e][lane] = o[e];
      if (cg == 0) others_ml[warp][rr] = make_float2(m, l);
    }
    __syncthreads();
    if (way) return;
#pragma unroll 1
    for (int w = warp + 1; w < warp + WAYS; ++w) {
      const float2 ml = others_ml[w][rr];
      const float mx = fmaxf(m, ml.x), ref = mx == -INFINITY ? 0.f : mx;
      const float f = ex2_approx(m - ref), y = ex2_approx(ml.x - ref);
      m = mx;
      l = l * f + y * ml.y;
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const float4 x = others_o[w][e][lane];
        o[e].x = o[e].x * f + y * x.x;
        o[e].y = o[e].y * f + y * x.y;
        o[e].z = o[e].z * f + y * x.z;
        o[e].w = o[e].w * f + y * x.w;
      }
    }
  }
  // a sequence without keys has its zeros
  if (!real || all == 0) return;
  const float inv = 1.f / l;
  uint2* out = reinterpret_cast<uint2*>(a.out + (static_cast<long long>(pair) * a.n_rep + h) * HEAD_DIM) + cg;
#pragma unroll
  for (int e = 0; e < R; ++e)
    out[PARTS * e] = make_uint2(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv));
}

}  // namespace

cudaError_t launch_shared_decode(const PackedPrefillMaps& maps, const SharedDecodeParams& a, cudaStream_t s) {
  const PagedDecodeParams& p = a.own;
  const int n_rep = p.n_heads / p.n_kv;
  if (p.B <= 0 || p.B > PAGED_MAX_SEQS || a.G <= 0 || a.G > SHARED_MAX_GROUPS || p.ctas < 2 || p.ctas >= THREADS ||
      n_rep < 1 || n_rep > PAGED_MAX_REP)
    return cudaErrorInvalidValue;
  const auto kernel = n_rep <= 8 ? shared_decode_kernel<1> : shared_decode_kernel<2>;
  static bool attr_set[64][2] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev][n_rep <= 8]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev][n_rep <= 8] = true;
  }
  // one CTA per SM (shared memory admits no second)
  return launch_behind(kernel, static_cast<unsigned>(p.ctas), THREADS, SMEM_BYTES, s, maps.q, maps.k, maps.v, a);
}

// R: 4 rows where a KV head has as many. Warps for them: as many as still run
// at once. 64 sequences under 8,000 rows: 34.0 us with as many as here, 35.8
// with half, 35.4 with twice as many.
template <int R>
static cudaError_t launch_join(SharedJoinParams a, cudaStream_t s) {
  a.sets = (a.n_rep + R - 1) / R;
  const int sets = a.pairs * a.sets;
  constexpr int WARPS_AT_ONCE = 152 * JOIN_CTAS * JOIN_WARPS;
  const int most = WARPS_AT_ONCE / sets, ways = most >= 8 ? 8 : most >= 4 ? 4 : most >= 2 ? 2 : 1, each = JOIN_WARPS / ways;
  const auto kernel = ways == 8 ? shared_join_kernel<R, 8> : ways == 4 ? shared_join_kernel<R, 4>
                                                         : ways == 2 ? shared_join_kernel<R, 2> : shared_join_kernel<R, 1>;
  return launch_behind(kernel, static_cast<unsigned>((sets + each - 1) / each), JOIN_WARPS * 32, 0, s, a);
}
cudaError_t launch_shared_join(const SharedJoinParams& a, cudaStream_t s) {
  return a.n_rep >= 3 ? launch_join<4>(a, s) : a.n_rep == 2 ? launch_join<2>(a, s) : launch_join<1>(a, s);
}

// Units of a batch at most: of groups of two sequences at least, with `keys` in
// common, and their pairs of Q tiles.
long long shared_most_units(int B, int n_rep, int n_kv, long long keys) {
  const int qp = ROWS / n_rep;
  return (B / 2 + B / (NQ * qp) + 1) * ((keys + KT - 1) / KT + ITEM_UNITS) * n_kv;
}

}  // namespace gqa
