// Attention of one new token per sequence over a paged cache, split over the
// length and joined ("Llama 3.1 8B · Grouped-query attention", mode decode:
// o_h = softmax(scale q_h K_g^T) V_g over cache rows 0..start_pos, KV head
// g = h / n_rep; each K/V row is loaded once for its n_rep query heads).
//
// n_rep flops a byte: the bound is memory, so the design is about keeping
// every SM streaming the same number of bytes whatever the lengths.
//   * A chunk is 16 positions of one KV head (8 KB of K and V). All chunks, in
//     (sequence, KV head, position) order, are cut into equal contiguous
//     ranges, one per CTA, and each CTA's range into one per warp. KV heads
//     come before positions so that few ranges meet in one output: a long
//     sequence is joined from ctas / n_kv partials per KV head.
//   * Each warp streams its range through its own ring of STAGES chunks with
//     cp.async, its page ids looked up one chunk ahead; nothing but the end
//     of the CTA synchronises warps. Rows past the sequence are filled with
//     zeros instead of being read (they may hold anything). 64 to 128 KB are
//     in flight per SM. More is worse: four groups of about ten SMs get 10 to
//     15% less of a saturated memory than the others, the more so the deeper
//     the queues, and the ranges are equal (3 stages: 182.6 us where 2 take
//     174.7, 64 sequences of up to 8,192 rows). Fewer warps are too: the work
//     on a chunk then shows (6: 178.7, 4: 190).
//   * S^T = K Q^T and O^T += V^T P^T by mma.sync m16n8k16 (the 16 keys, then
//     the dims, on the M side, query heads padded to 8 or 16 on the N side).
//     The probabilities enter the product as two bf16 terms (P = hi + lo), so
//     that the output's own rounding is the only 8-bit one; the tensor pipe
//     has the time.
//   * A (sequence, KV head) wholly inside a warp's range is finished in
//     registers. The other parts are joined by the log-sum-exp rule, first in
//     shared memory among the CTA's warps, then, where several CTAs hold
//     parts, by the CTA that arrives last at a ticket, in CTA order: the
//     result does not depend on the order of arrival, and no CTA waits.
//   * Joining across CTAs (ticket, read back) takes 2.5 to 4 us. Where one CTA
//     per (sequence, KV head) is no more than 2.5 us behind the equal ranges,
//     the ranges are those. Both measured, own / equal: 16 sequences of 2,001
//     rows and 8 KV heads 25.7 / 29.7 us, of 8,192 rows 83.3 / 86.8, of 301
//     7.4 / 10.2, 12 of 4,001 37.3 / 38.5, 8 of 2,001 20.4 / 20.0, 4 of 1,001
//     11.9 / 9.7, of 401 8.2 / 8.6, one of 2,001 18.6 / 9.3. The longest
//     sequence's time alone on a CTA, or the batch's at the memory's rate,
//     tells them apart.
//   * Code that runs once a CTA, and the join that runs in a few CTAs, wait
//     for instructions more than for data: their loops are not unrolled.
// Measured (GB300, 6.8 TB/s copied): 171.8 us for 1.108 GB (64 sequences of
// up to 8,192 rows), 87.0 for 537 MB (one of 131,072), 48.5 for 263 MB (16 of
// 1,001, 32 KV heads), 16.2 for 66 MB (8 KV heads), 3.4 for one sequence of
// 16 rows. Head-major pages ([page, KV head,
// row]) are 2 to 4% faster than [page, row, KV head]: longer runs per CTA.
#include <math.h>

#include "paged.h"

namespace gqa {

namespace {

constexpr int KEYS = 16;                          // positions of a chunk
constexpr int ROW_BYTES = HEAD_DIM * 2;
constexpr int TILE_BYTES = KEYS * ROW_BYTES;      // K or V of a chunk
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int STAGES = 2;
constexpr int WARPS = 8;
// In 1/800 us, what a chunk takes at the whole memory's rate: a chunk of a CTA
// by itself (it streams 9 or 10 a us, 64 to 128 KB in flight), and joining
// across CTAs (2.5 us).
constexpr float ALONE = 85.f, JOIN_COST = 2000.f;
constexpr int BATCH = 5;                          // partials a warp has in flight when it joins
constexpr int PART = HEAD_DIM + 2;                // floats of a partial row: o, max, sum

// Row r, 16-byte piece c of a 256-byte-row tile: eight rows of one piece fall
// into eight different 16-byte columns.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return static_cast<uint32_t>(r * ROW_BYTES + ((c ^ (r & 7)) << 4));
}

// A place in the chunk order.
struct Cursor {
  int b, h, j;  // sequence, KV head, chunk of it
  int n;        // chunks of the sequence (for each KV head)
};

// pre[b]: chunks per KV head of the sequences before b.
__device__ __forceinline__ Cursor locate(int u, const int* pre, int B, int n_kv) {
  const int x = u / n_kv;  // pre[b] <= x < pre[b + 1] exactly when u lies in sequence b
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  Cursor c;
  c.b = lo;
  c.n = pre[lo + 1] - pre[lo];
  const int r = u - pre[lo] * n_kv;
  c.h = r / c.n;
  c.j = r - c.h * c.n;
  return c;
}
__device__ __forceinline__ void advance(Cursor& c, const int* pre, int B, int n_kv) {
  if (++c.j < c.n) return;
  c.j = 0;
  if (++c.h < n_kv) return;
  c.h = 0;
  do {
    if (++c.b >= B) return;
    c.n = pre[c.b + 1] - pre[c.b];
  } while (c.n == 0);
}

// A part of a (sequence, KV head), left for joining: its chunks
// [first, end) identify it, `row` is its first row of the output.
struct Part {
  int first, end, row;
};

// This lane's 4 dims of an output row.
__device__ __forceinline__ void store_row(__nv_bfloat16* out, int row, float4 o, float inv) {
  *(reinterpret_cast<uint2*>(out + static_cast<long long>(row) * HEAD_DIM) + (threadIdx.x & 31)) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

// Counts this CTA at a ticket: behind the barrier before it, it publishes all
// the CTA's stores, and to the barrier behind it those of the CTAs before.
__device__ __forceinline__ int arrive(int* ticket) {
  int n;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(ticket) : "memory");
  return n;
}

// A running (max, sum, output) taken to the max mx.
__device__ __forceinline__ void rescale(float& m, float mx, float& l, float4& o) {
  const float s = ex2_approx(m - (mx == -INFINITY ? 0.f : mx));
  m = mx;
  l *= s;
  o = make_float4(o.x * s, o.y * s, o.z * s, o.w * s);
}

// NT: 8-wide tiles of query heads (1: n_rep <= 8, 2: n_rep <= 16).
template <int NT>
__global__ void __launch_bounds__(WARPS * 32, 1) paged_decode_kernel(PagedDecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int W = WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rep = p.n_heads / p.n_kv;
  uint8_t* ring = smem + warp * (STAGES * STAGE_BYTES);
  // per warp: the partial of the part that began before its range; the one
  // that goes on behind it is put into the ring when the warp is done
  float* stash = reinterpret_cast<float*>(smem + W * (STAGES * STAGE_BYTES));
  int* pre = reinterpret_cast<int*>(stash + W * n_rep * PART);
  int* last = pre + p.B + 1;  // last row of each sequence
  __shared__ Part parts[2 * WARPS];  // each warp's two, first = -1: none
  __shared__ int warp_sum[WARPS], warp_max[WARPS];
  __shared__ int is_last[2];
  __shared__ Part joint[2];  // of the shared segments: first and last CTA, first output row

  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  // chunks per sequence, prefix-summed; unused slots and bad positions have none
  int total, longest;
  {
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0, most = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int s = p.start[b];
      const bool ok = s >= 0 && s < p.pages.capacity();
      if (!ok && s != -1 && blockIdx.x == 0) report(p.status, DEV_BAD_POSITION);
      const int n = ok ? s / KEYS + 1 : 0;
      pre[b + 1] = n;
      last[b] = s;
      sum += n;
      most = max(most, n);
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (lane == 31) warp_sum[warp] = run;
    if (lane == 0) warp_max[warp] = most;
    if (threadIdx.x < 2 * WARPS) parts[threadIdx.x].first = -1;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
    run -= sum;
    total = longest = 0;
    for (int w = 0; w < W; ++w) {
      if (w == warp) run += total;
      total += warp_sum[w];
      longest = max(longest, warp_max[w]);
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      run += pre[b + 1];
      pre[b + 1] = run;
    }
    __syncthreads();
  }
  // rows of sequences without keys
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (pre[b + 1] == pre[b])
#pragma unroll 1
      for (int i = threadIdx.x; i < p.n_heads * (HEAD_DIM / 8); i += blockDim.x)
        reinterpret_cast<uint4*>(p.out + static_cast<long long>(b) * p.n_heads * HEAD_DIM)[i] = make_uint4(0, 0, 0, 0);

  total *= p.n_kv;
  if (total == 0) return;
  const int ctas = decode_ctas(total, gridDim.x, W);
  const Split split(total, ctas);
  // One CTA per (sequence, KV head) instead of equal ranges where that costs
  // less than joining parts across CTAs.
  const float memory = static_cast<float>(total);
  const bool own = p.B * p.n_kv <= static_cast<int>(gridDim.x) &&
                   fmaxf(static_cast<float>(longest) * ALONE, memory) <=
                       fmaxf(static_cast<float>(split.each) * ALONE, memory) + JOIN_COST;
  int c0, c1;
  if (own) {
    if (static_cast<int>(blockIdx.x) >= p.B * p.n_kv) return;
    const int b = blockIdx.x / p.n_kv, h = blockIdx.x - b * p.n_kv, n = pre[b + 1] - pre[b];
    c0 = pre[b] * p.n_kv + h * n;
    c1 = c0 + n;
  } else {
    if (static_cast<int>(blockIdx.x) >= ctas) return;
    c0 = split.start(blockIdx.x);
    c1 = split.start(blockIdx.x + 1);
  }
  const int a0 = warp_start(c0, c1, warp, W), a1 = warp_start(c0, c1, warp + 1, W);
  const int n = a1 - a0;

  const int gr = lane >> 2, t = lane & 3;
  const int half = lane >> 4, piece = lane & 15;

  if (n > 0) {
    Cursor iss = locate(a0, pre, p.B, p.n_kv), cur = iss;
    // element offset of row lane % 16 of the chunk at `iss`, -1 for a row past the sequence
    auto row_offset = [&]() -> long long {
      const int pos = iss.j * KEYS + piece;
      if (pos > last[iss.b]) return -1;
      const int page = p.pages.table[static_cast<long long>(iss.b) * p.pages.table_stride + (pos >> p.pages.page_shift)];
      if (page < 0 || page >= p.pages.num_pages) {
        report(p.status, DEV_BAD_PAGE);
        return -1;
      }
      return page * p.pages.page_stride + (pos & ((1 << p.pages.page_shift) - 1)) * p.pages.row_stride +
             iss.h * p.pages.head_stride;
    };
    int issued = 0;
    long long next = row_offset();
    const uint32_t ring32 = smem_u32(ring);
    auto issue = [&]() {
      if (issued < n) {
        const uint32_t dst = ring32 + (issued % STAGES) * STAGE_BYTES;
        const long long off = next;
        ++issued;
        if (issued < n) {
          advance(iss, pre, p.B, p.n_kv);
          next = row_offset();
        }
#pragma unroll
        for (int i = 0; i < KEYS / 2; ++i) {
          const int r = 2 * i + half;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const long long e = (o < 0 ? 0 : o) + piece * 8;
          const uint32_t bytes = o < 0 ? 0u : 16u;
          cp_async16(dst + tile_at(r, piece), p.pages.k + e, bytes);
          cp_async16(dst + TILE_BYTES + tile_at(r, piece), p.pages.v + e, bytes);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    uint32_t qb[NT][8][2];  // Q^T as B fragments: dims 16s + 2t (+1) | +8, query head 8 nt + gr
    float m_run[NT][2], l_run[NT][2], oacc[NT][8][4];  // heads 8 nt + 2t (+1); O^T tile d: dims 16d + gr (+8)
    for (int i = 0; i < n; ++i) {
      issue();
      if (i == 0 || cur.j == 0) {
        const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q + cur.b * p.q_stride + cur.h * n_rep * HEAD_DIM);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int h = nt * 8 + gr;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            qb[nt][s][0] = h < n_rep ? __ldg(q32 + h * (HEAD_DIM / 2) + s * 8 + t) : 0u;
            qb[nt][s][1] = h < n_rep ? __ldg(q32 + h * (HEAD_DIM / 2) + s * 8 + 4 + t) : 0u;
          }
          m_run[nt][0] = m_run[nt][1] = -INFINITY;
          l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
          for (int d = 0; d < 8; ++d) oacc[nt][d][0] = oacc[nt][d][1] = oacc[nt][d][2] = oacc[nt][d][3] = 0.f;
        }
      }
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint32_t kt = ring32 + (i % STAGES) * STAGE_BYTES, vt = kt + TILE_BYTES;

      float sc[NT][4], sd[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = sd[nt][0] = sd[nt][1] = sd[nt][2] = sd[nt][3] = 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t k0, k1, k2, k3;
        ldsm_x4(kt + tile_at(lane & 15, 2 * s + half), k0, k1, k2, k3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816((s & 1) ? sd[nt] : sc[nt], k0, k1, k2, k3, qb[nt][s][0], qb[nt][s][1]);
      }
      // rows gr and gr + 8 of the chunk
      const int left = last[cur.b] - cur.j * KEYS;
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float(&x)[4] = sc[nt];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += sd[nt][e];
        x[0] = gr <= left ? x[0] * p.scale_log2 : -INFINITY;
        x[1] = gr <= left ? x[1] * p.scale_log2 : -INFINITY;
        x[2] = gr + 8 <= left ? x[2] * p.scale_log2 : -INFINITY;
        x[3] = gr + 8 <= left ? x[3] * p.scale_log2 : -INFINITY;
        float pr[4], al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[e], x[e + 2]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(mx, m_run[nt][e]);
          // scores that are all -inf leave the maximum there: no term, not a NaN
          const float ref = mx == -INFINITY ? 0.f : mx;
          al[e] = ex2_approx(m_run[nt][e] - ref);
          pr[e] = ex2_approx(x[e] - ref);
          pr[e + 2] = ex2_approx(x[e + 2] - ref);
          m_run[nt][e] = mx;
          l_run[nt][e] = l_run[nt][e] * al[e] + (pr[e] + pr[e + 2]);  // this lane's rows; summed over lanes at the end
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          oacc[nt][d][0] *= al[0];
          oacc[nt][d][1] *= al[1];
          oacc[nt][d][2] *= al[0];
          oacc[nt][d][3] *= al[1];
        }
        // P^T as B fragments, (head gr, keys 2t, 2t + 1) and 8 keys further
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // hi: the upper 16 bits; lo: the rest, kept above 0 where P is (P is
          // 0 or 2^-126 and more; 2^-133 is the least bf16 above 0), so that an
          // infinite value row gives an infinite sum and not a NaN
          const float x0 = pr[2 * e], x1 = pr[2 * e + 1];
          const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
          hi[nt][e] = movmatrix_t(__byte_perm(u0, u1, 0x7632));
          const float y0 = x0 - __uint_as_float(u0 & 0xffff0000u), y1 = x1 - __uint_as_float(u1 & 0xffff0000u);
          lo[nt][e] = movmatrix_t(pack_bf16(fmaxf(y0, fminf(x0, 0x1p-133f)), fmaxf(y1, fminf(x1, 0x1p-133f))));
        }
      }
      const int vr = (lane & 7) + (half << 3);  // key row of this lane's ldmatrix address
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t v0, v1, v2, v3;
        ldsm_x4_t(vt + tile_at(vr, 2 * d + ((lane >> 3) & 1)), v0, v1, v2, v3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(oacc[nt][d], v0, v1, v2, v3, hi[nt][0], hi[nt][1]);
          mma16816(oacc[nt][d], v0, v1, v2, v3, lo[nt][0], lo[nt][1]);
        }
      }
      __syncwarp();  // the chunk's rows are read before its slot is filled again

      const Cursor here = cur;
      advance(cur, pre, p.B, p.n_kv);
      if (i + 1 < n && cur.j != 0) continue;

      // end of this warp's part of (here.b, here.h)
      const int first = pre[here.b] * p.n_kv + here.h * here.n;
      const Part seg{first, first + here.n, here.b * p.n_heads + here.h * n_rep};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], o);
      if (seg.first >= a0 && seg.end <= a1) {
        __nv_bfloat16* out = p.out + static_cast<long long>(seg.row) * HEAD_DIM;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float i0 = 1.f / l_run[nt][0], i1 = 1.f / l_run[nt][1];
          const int h = nt * 8 + gr;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            // (dim gr, heads 2t, 2t + 1) -> (head gr, dims 2t, 2t + 1)
            const uint32_t w0 = movmatrix_t(pack_bf16(oacc[nt][d][0] * i0, oacc[nt][d][1] * i1));
            const uint32_t w1 = movmatrix_t(pack_bf16(oacc[nt][d][2] * i0, oacc[nt][d][3] * i1));
            if (h < n_rep) {
              uint32_t* o32 = reinterpret_cast<uint32_t*>(out + h * HEAD_DIM + 16 * d) + t;
              o32[0] = w0;
              o32[4] = w1;
            }
          }
        }
      } else {
        const int slot = seg.first < a0 ? 0 : 1;
        float* part = slot == 0 ? stash + warp * n_rep * PART : reinterpret_cast<float*>(ring);
        if (slot == 1) {
          // the last part of the range: every copy into the ring has landed and been read
          cp_async_wait<0>();
          __syncwarp();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = nt * 8 + 2 * t + e;
            if (h >= n_rep) continue;
            float* row = part + h * PART;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              row[16 * d + gr] = oacc[nt][d][e];
              row[16 * d + gr + 8] = oacc[nt][d][e + 2];
            }
            if (gr == 0) {
              row[HEAD_DIM] = m_run[nt][e];
              row[HEAD_DIM + 1] = l_run[nt][e];
            }
          }
        if (lane == 0) parts[2 * warp + slot] = seg;
      }
    }
  }
  __syncthreads();

  // ---- join this CTA's parts: lane e < 2W looks at entry e; those of one
  // (sequence, KV head) follow each other. (part, query head) pairs are dealt
  // to the warps.
  auto part_at = [&](int e) -> const float* {
    return (e & 1) ? reinterpret_cast<const float*>(smem + (e >> 1) * (STAGES * STAGE_BYTES))
                   : stash + (e >> 1) * n_rep * PART;
  };
  Part cross[2] = {{-1, 0, 0}, {-1, 0, 0}};  // with parts in other CTAs too: begun before this one, going on behind it
  {
    Part mine{-1, 0, 0};
    if (lane < 2 * W) mine = parts[lane];
    const unsigned peers = __match_any_sync(0xffffffffu, mine.first);
    unsigned heads = __ballot_sync(0xffffffffu, mine.first >= 0 && __ffs(peers) - 1 == lane);
#pragma unroll 1
    for (int k = 0; heads; heads &= heads - 1) {
      const int e = __ffs(heads) - 1;
      const unsigned members = __shfl_sync(0xffffffffu, peers, e);
      const Part seg{__shfl_sync(0xffffffffu, mine.first, e), __shfl_sync(0xffffffffu, mine.end, e),
                     __shfl_sync(0xffffffffu, mine.row, e)};
      const int side = seg.first < c0 ? 0 : seg.end > c1 ? 1 : 2;  // 2: all of it is here
      if (side == 0) cross[0] = seg;
      if (side == 1) cross[1] = seg;
#pragma unroll 1
      for (int r = 0; r < n_rep; ++r, ++k) {
        if (k % W != warp) continue;
        float m_e = -INFINITY, l_e = 0.f;
        if (members >> lane & 1) {
          const float2 ml = *reinterpret_cast<const float2*>(part_at(lane) + r * PART + HEAD_DIM);
          m_e = ml.x;
          l_e = ml.y;
        }
        float m = m_e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float w_e = ex2_approx(m_e - (m == -INFINITY ? 0.f : m));
        float l = w_e * l_e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (unsigned g = members; g; g &= g - 1) {
          const int f = __ffs(g) - 1;
          const float w = __shfl_sync(0xffffffffu, w_e, f);
          const float* row = part_at(f) + r * PART + 4 * lane;
          const float2 x = *reinterpret_cast<const float2*>(row), y = *reinterpret_cast<const float2*>(row + 2);
          o.x += w * x.x;
          o.y += w * x.y;
          o.z += w * y.x;
          o.w += w * y.y;
        }
        if (side == 2) {
          store_row(p.out, seg.row + r, o, 1.f / l);
        } else {
          const long long at = (2LL * blockIdx.x + side) * n_rep + r;
          __stcg(reinterpret_cast<float4*>(p.part_o + at * HEAD_DIM) + lane, o);
          if (lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml) + at, make_float2(m, l));
        }
      }
    }
  }
  if (cross[0].first < 0 && cross[1].first < 0) return;

  // ---- across CTAs: the ticket is that of the CTA with the first chunk
  __syncthreads();
  if (threadIdx.x < 2) {
    const Part seg = threadIdx.x ? cross[1] : cross[0];
    int last = 0;
    if (seg.first >= 0) {
      const int a = split.holder(seg.first), z = split.holder(seg.end - 1);
      last = arrive(p.tickets + a) == z - a;
      if (last) p.tickets[a] = 0;
      joint[threadIdx.x] = {a, z, seg.row};
    }
    is_last[threadIdx.x] = last;
  }
  __syncthreads();
  // Per query head `ways` warps share the partials, each with a running max,
  // then the first of them adds up. Few CTAs come here and their instruction
  // caches are cold: the loops are kept short (one sequence of 1,001 rows: 8.8
  // us with batches of 5, 9.2 with 8 or 4; 9.35 with a pass for the max before).
  const int ways = max(1, W / n_rep);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    if (!is_last[side]) continue;
    const int a = joint[side].first, z = joint[side].end;
#pragma unroll 1
    for (int r0 = 0; r0 < n_rep; r0 += W / ways) {
      const int r = r0 + warp / ways, way = warp % ways;
      const bool on = warp / ways < W / ways && r < n_rep;
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) {
        // the part of its first CTA goes on behind that CTA (slot 1), the others began before theirs (slot 0)
        auto at = [&](int c) { return (2 * c + (c == a)) * n_rep + r; };
        const float2* mls = reinterpret_cast<const float2*>(p.part_ml);
        const float4* os = reinterpret_cast<const float4*>(p.part_o) + lane;
#pragma unroll 1
        for (int c0 = a + way; c0 <= z; c0 += BATCH * ways) {
          float2 ml[BATCH];
          float4 x[BATCH];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int c = c0 + k * ways;
            ml[k] = make_float2(-INFINITY, 0.f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c <= z) {
              ml[k] = __ldcg(mls + at(c));
              x[k] = __ldcg(os + at(c) * (HEAD_DIM / 4));
            }
          }
          float mx = m;
#pragma unroll
          for (int k = 0; k < BATCH; ++k) mx = fmaxf(mx, ml[k].x);
          rescale(m, mx, l, o);
          const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const float w = ex2_approx(ml[k].x - ref);
            l += w * ml[k].y;
            o.x += w * x[k].x;
            o.y += w * x[k].y;
            o.z += w * x[k].z;
            o.w += w * x[k].w;
          }
        }
      }
      if (ways > 1) {
        float* mine = reinterpret_cast<float*>(smem) + warp * PART;
        __syncthreads();
        if (on && way) {
          *reinterpret_cast<float2*>(mine + 4 * lane) = make_float2(o.x, o.y);
          *reinterpret_cast<float2*>(mine + 4 * lane + 2) = make_float2(o.z, o.w);
          if (lane == 0) *reinterpret_cast<float2*>(mine + HEAD_DIM) = make_float2(m, l);
        }
        __syncthreads();
        if (on && !way)
#pragma unroll 1
          for (int g = 1; g < ways; ++g) {
            const float* row = mine + g * PART;
            const float2 ml = *reinterpret_cast<const float2*>(row + HEAD_DIM);
            const float2 x = *reinterpret_cast<const float2*>(row + 4 * lane);
            const float2 y = *reinterpret_cast<const float2*>(row + 4 * lane + 2);
            rescale(m, fmaxf(m, ml.x), l, o);
            const float w = ex2_approx(ml.x - (m == -INFINITY ? 0.f : m));
            l += w * ml.y;
            o.x += w * x.x;
            o.y += w * x.y;
            o.z += w * y.x;
            o.w += w * y.y;
          }
      }
      if (on && !way) store_row(p.out, joint[side].row + r, o, 1.f / l);
    }
  }
}

template <int NT>
cudaError_t launch_nt(const PagedDecodeParams& p, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int n_rep = p.n_heads / p.n_kv;
  const size_t smem = static_cast<size_t>(WARPS) * (STAGES * STAGE_BYTES + n_rep * PART * 4) + (2 * p.B + 1) * 4;
  return launch_behind(paged_decode_kernel<NT>, static_cast<unsigned>(p.ctas), WARPS * 32, smem, s, p);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s) {
  if (p.B <= 0 || p.B > PAGED_MAX_SEQS || p.ctas <= 0) return cudaErrorInvalidValue;
  const int n_rep = p.n_heads / p.n_kv;
  if (n_rep < 1 || n_rep > PAGED_MAX_REP) return cudaErrorInvalidValue;
  return n_rep <= 8 ? launch_nt<1>(p, s) : launch_nt<2>(p, s);
}

}  // namespace gqa
