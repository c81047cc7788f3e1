// What the paged decode attentions share beside their inner loops: the batch's
// chunks cut into ranges, one per CTA and one per warp of it, and the parts of
// (sequence, KV head) pairs joined by the log-sum-exp rule, first in shared
// memory among a CTA's warps, then, where several CTAs hold parts, by the CTA
// that arrives last at a ticket, in CTA order: the result does not depend on
// the order of arrival, and no CTA waits.
#pragma once

#include <math.h>

#include "paged.h"

namespace gqa {
namespace decode {

constexpr int WARPS = 8;
// In 1/800 us, what a chunk (8 KB) takes at the whole memory's rate: a chunk of
// a CTA by itself (it streams 9 or 10 a us, 64 to 128 KB in flight), and joining
// across CTAs (2.5 us).
constexpr float ALONE = 85.f, JOIN_COST = 2000.f;
constexpr int BATCH = 5;             // partials a warp has in flight when it joins
constexpr int TOGETHER = 2;          // parts of a CTA's warps that are read together (1: 1 us more, 4: 0.1, 8: 0.2 to 1)
constexpr int PART = HEAD_DIM + 2;   // floats of a partial row: o, max, sum

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

// The largest of a warp's values (NaN only where all are).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Zeros for all heads of sequence b, by the whole CTA.
__device__ __forceinline__ void zero_rows(__nv_bfloat16* out, int b, int n_heads) {
#pragma unroll 1
  for (int i = threadIdx.x; i < n_heads * (HEAD_DIM / 8); i += blockDim.x)
    reinterpret_cast<uint4*>(out + static_cast<long long>(b) * n_heads * HEAD_DIM)[i] = make_uint4(0, 0, 0, 0);
}

// Static shared memory of a CTA.
constexpr int MAX_WARPS = 11;
struct Shared {
  Part parts[2 * WARPS];  // each warp's two, first = -1: none
  int warp_sum[MAX_WARPS], warp_max[MAX_WARPS];
  int is_last[2];
  Part joint[2];  // of the shared segments: first and last CTA, first output row
};

// Chunks of the batch per KV head, and of its longest sequence; pre[0..B] gets
// their prefix sums. chunks(b): those of sequence b. By a CTA of W warps.
struct Count {
  int total, longest;
};
template <int W, class Chunks>
__device__ __forceinline__ Count count_chunks(Shared& sh, int* pre, int B, Chunks chunks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, B), b1 = min(b0 + per, B);
  int sum = 0, most = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int n = chunks(b);
    pre[b + 1] = n;
    sum += n;
    most = max(most, n);
  }
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += x;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) sh.warp_sum[warp] = run;
  if (lane == 0) sh.warp_max[warp] = most;
  if (threadIdx.x < 2 * WARPS) sh.parts[threadIdx.x].first = -1;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  // a lane for each warp: short code, as it is fetched anew by every launch
  static_assert(W <= 32, "a lane for each warp");
  const int of_warp = lane < W ? sh.warp_sum[lane] : 0;
  Count c;
  c.total = __reduce_add_sync(0xffffffffu, of_warp);
  c.longest = __reduce_max_sync(0xffffffffu, lane < W ? sh.warp_max[lane] : 0);
  run += __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0) - sum;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    run += pre[b + 1];
    pre[b + 1] = run;
  }
  __syncthreads();
  return c;
}

// Chunks [c0, c1) of CTA `cta` of `grid` (total: of the batch, KV heads
// included; ctas: with a range, of equal ones); false: it has none. One CTA per (sequence, KV head) instead of equal ranges where
// that costs less than joining parts across CTAs.
__device__ __forceinline__ bool cta_range(int total, int longest, const Split& split, int ctas, int cta, int grid,
                                          const int* pre, int B, int n_kv, int& c0, int& c1) {
  const float memory = static_cast<float>(total);
  const bool own = B * n_kv <= grid &&
                   fmaxf(static_cast<float>(longest) * ALONE, memory) <=
                       fmaxf(static_cast<float>(split.each) * ALONE, memory) + JOIN_COST;
  if (own) {
    if (cta >= B * n_kv) return false;
    const int b = cta / n_kv, h = cta - b * n_kv, n = pre[b + 1] - pre[b];
    c0 = pre[b] * n_kv + h * n;
    c1 = c0 + n;
  } else {
    if (cta >= ctas) return false;
    c0 = split.start(cta);
    c1 = split.start(cta + 1);
  }
  return true;
}

// Joins the parts that the CTA's warps left (a barrier is before it): lane
// e < 2 WARPS looks at entry e; those of one (sequence, KV head) follow each
// other. (part, query head) pairs are dealt to the warps. Then the segments
// with parts in other CTAs too. part_at(e): entry e's rows [n_rep][PART] in
// shared memory; work: the CTA's shared memory from its begin, WARPS * PART
// floats of it are used once the parts are read; finish(row, o, m, l): takes a
// finished row's 4 dims of each lane, by a whole warp.
template <class PartAt, class Finish>
__device__ __forceinline__ void join_parts(Shared& sh, float* work, const Split& split, int cta, int c0, int c1, int n_rep,
                                           float* part_o, float* part_ml, int* tickets, PartAt part_at, Finish finish) {
  constexpr int W = WARPS;
  static_assert((W & (W - 1)) == 0, "rows are dealt by a mask");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Part cross[2] = {{-1, 0, 0}, {-1, 0, 0}};  // with parts in other CTAs too: begun before this one, going on behind it
  {
    Part mine{-1, 0, 0};
    if (lane < 2 * W) mine = sh.parts[lane];
    const unsigned peers = __match_any_sync(0xffffffffu, mine.first);
    unsigned heads = __ballot_sync(0xffffffffu, mine.first >= 0 && __ffs(peers) - 1 == lane);
#pragma unroll 1
    for (int k = 0; heads; heads &= heads - 1, k += n_rep) {
      const int e = __ffs(heads) - 1;
      const unsigned members = __shfl_sync(0xffffffffu, peers, e);
      const Part seg{__shfl_sync(0xffffffffu, mine.first, e), __shfl_sync(0xffffffffu, mine.end, e),
                     __shfl_sync(0xffffffffu, mine.row, e)};
      const int side = seg.first < c0 ? 0 : seg.end > c1 ? 1 : 2;  // 2: all of it is here
      if (side == 0) cross[0] = seg;
      if (side == 1) cross[1] = seg;
#pragma unroll 1
      for (int r = (warp - k) & (W - 1); r < n_rep; r += W) {
        float m_e = -INFINITY, l_e = 0.f;
        if (members >> lane & 1) {
          const float2 ml = *reinterpret_cast<const float2*>(part_at(lane) + r * PART + HEAD_DIM);
          m_e = ml.x;
          l_e = ml.y;
        }
        const float m = warp_max(m_e);
        const float w_e = ex2_approx(m_e - (m == -INFINITY ? 0.f : m));
        float l = w_e * l_e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (unsigned g = members; g;) {
          float w[TOGETHER];
          float2 x[TOGETHER], y[TOGETHER];
#pragma unroll
          for (int i = 0; i < TOGETHER; ++i) {
            const int f = (__ffs(g) - 1) & 31;
            w[i] = __shfl_sync(0xffffffffu, w_e, f);
            x[i] = y[i] = make_float2(0.f, 0.f);
            if (g) {
              const float* row = part_at(f) + r * PART + 4 * lane;
              x[i] = *reinterpret_cast<const float2*>(row);
              y[i] = *reinterpret_cast<const float2*>(row + 2);
            } else {
              w[i] = 0.f;
            }
            g &= g - 1;
          }
#pragma unroll
          for (int i = 0; i < TOGETHER; ++i) {
            o.x += w[i] * x[i].x;
            o.y += w[i] * x[i].y;
            o.z += w[i] * y[i].x;
            o.w += w[i] * y[i].y;
          }
        }
        if (side == 2) {
          finish(seg.row + r, o, m, l);
        } else {
          const long long at = (2LL * cta + side) * n_rep + r;
          __stcg(reinterpret_cast<float4*>(part_o + at * HEAD_DIM) + lane, o);
          if (lane == 0) __stcg(reinterpret_cast<float2*>(part_ml) + at, make_float2(m, l));
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
      last = arrive(tickets + a) == z - a;
      if (last) tickets[a] = 0;
      sh.joint[threadIdx.x] = {a, z, seg.row};
    }
    sh.is_last[threadIdx.x] = last;
  }
  __syncthreads();
  // Per query head `ways` warps share the partials, each with a running max,
  // then the first of them adds up. Few CTAs come here and their instruction
  // caches are cold: the loops are kept short (one sequence of 1,001 rows: 8.8
  // us with batches of 5, 9.2 with 8 or 4; 9.35 with a pass for the max before).
  // Two parts, the common case, need no second warp, and the rows of both
  // segments are dealt together (0.5 us less).
  const bool few = (!sh.is_last[0] || sh.joint[0].end - sh.joint[0].first == 1) &&
                   (!sh.is_last[1] || sh.joint[1].end - sh.joint[1].first == 1);
  const int ways = few ? 1 : max(1, W / n_rep);
  const bool back = few && W / n_rep > 1;  // added up as two warps would: the second part first
#pragma unroll 1
  for (int t0 = 0; t0 < 2 * n_rep; t0 += W / ways) {
    const int task = t0 + warp / ways, side = task >= n_rep, r = task - side * n_rep, way = warp % ways;
    const bool on = warp / ways < W / ways && r < n_rep && sh.is_last[side];
    const int a = sh.joint[side].first, z = sh.joint[side].end;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      // the part of its first CTA goes on behind that CTA (slot 1), the others began before theirs (slot 0)
      auto at = [&](int c) { return (2 * c + (c == a)) * n_rep + r; };
      const float2* mls = reinterpret_cast<const float2*>(part_ml);
      const float4* os = reinterpret_cast<const float4*>(part_o) + lane;
#pragma unroll 1
      for (int c0 = a + way; c0 <= z; c0 += BATCH * ways) {
        float2 ml[BATCH];
        float4 x[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int c = back ? z - k : c0 + k * ways;
          ml[k] = make_float2(-INFINITY, 0.f);
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c >= a && c <= z) {
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
      float* mine = work + warp * PART;
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
    if (on && !way) finish(sh.joint[side].row + r, o, m, l);
  }
}

}  // namespace decode
}  // namespace gqa
