// Rows of an 8-bit cache back into bf16 pages (exact, fp8.cuh), for what reads
// a bf16 cache: the prefill attention of a chunk after a quantised prefix, or a
// cache that moves.
//
// 129 bytes read and 256 written a row: the bound is memory. A task is 16
// positions (one page of both sides each) of one KV head, K and V; a warp takes
// every so-manieth, so that neighbours read neighbouring heads at the same time.
// Its 32 rows' loads are issued together, 16 lanes x 8 values a row, and the
// next task's place is looked up meanwhile. 3 CTAs per SM: 1.23 GB 202 us with 2,
// 3 or 4, 232 with 5; one prompt of 7,168 rows 10.9, 9.1 and 9.9.
// Measured (GB300, 6.8 TB/s copied): 202 us for 1.23 GB (48 sequences of up to
// 8,191 rows), 9.1 for 44 MB (7,168 rows).
#include "fp8.cuh"
#include "paged.h"

namespace gqa {

namespace {

constexpr int WARPS = 8, CTAS_PER_SM = 3;
constexpr int UNIT = 16;  // positions

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 to_bf16(uint2 x, float s) {
  uint32_t h[4];
  e4m3x4_to_f16(x.x, h[0], h[1]);
  e4m3x4_to_f16(x.y, h[2], h[3]);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    r[i] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__global__ void __launch_bounds__(WARPS * 32, CTAS_PER_SM) fp8_read_kernel(const __grid_constant__ Fp8ReadParams p) {
  extern __shared__ int pre[];  // units before each sequence, then its rows
  int* count = pre + p.B + 1;
  __shared__ int warp_sum[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  const long long capacity = min(p.from.capacity(), p.to.capacity());
  int total = 0;
  {
    const int per = (p.B + WARPS * 32 - 1) / (WARPS * 32);
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int n = p.rows[b];
      const bool ok = n >= 0 && n <= capacity;
      if (!ok && n != -1 && blockIdx.x == 0) report(p.status, DEV_BAD_POSITION);
      const int u = ok && n > 0 ? ceil_div(n, UNIT) : 0;
      pre[b + 1] = u;
      count[b] = n;
      sum += u;
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) warp_sum[warp] = run;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < WARPS; ++w) {
      if (w == warp) run += total;
      total += warp_sum[w];
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      run += pre[b + 1];
      pre[b + 1] = run;
    }
    __syncthreads();
  }
  struct Task {
    int b, h, first, n, src, dst;  // n: rows that it has
  };
  const long long tasks = static_cast<long long>(total) * p.n_kv, all_warps = static_cast<long long>(gridDim.x) * WARPS;
  auto find = [&](long long t) {
    Task x{0, 0, 0, 0, -1, -1};
    if (t >= tasks) return x;
    const int u = static_cast<int>(t / p.n_kv);
    x.h = static_cast<int>(t - static_cast<long long>(u) * p.n_kv);
    int lo = 0, hi = p.B;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u) lo = mid; else hi = mid;
    }
    x.b = lo;
    x.first = (u - pre[lo]) * UNIT;
    x.n = min(UNIT, count[lo] - x.first);
    x.src = p.from.table[static_cast<long long>(lo) * p.from.table_stride + (x.first >> p.from.page_shift)];
    x.dst = p.to.table[static_cast<long long>(lo) * p.to.table_stride + (x.first >> p.to.page_shift)];
    return x;
  };
  const int half = lane >> 4, piece = lane & 15;
  long long t = static_cast<long long>(blockIdx.x) * WARPS + warp;
  Task x = find(t);
#pragma unroll 1
  for (; t < tasks; t += all_warps) {
    const Task here = x;
    const bool good = here.src >= 0 && here.src < p.from.num_pages && here.dst >= 0 && here.dst < p.to.num_pages;
    if (!good) {
      if (lane == 0) report(p.status, DEV_BAD_PAGE);
      x = find(t + all_warps);
      continue;
    }
    const int from_row = here.first & ((1 << p.from.page_shift) - 1), to_row = here.first & ((1 << p.to.page_shift) - 1);
    const long long at = here.src * p.from.page_stride + (from_row + half) * p.from.row_stride + here.h * p.from.head_stride + 8 * piece;
    uint2 k[UNIT / 2], v[UNIT / 2];
#pragma unroll
    for (int i = 0; i < UNIT / 2; ++i) {
      k[i] = v[i] = make_uint2(0, 0);
      if (2 * i + half < here.n) {
        k[i] = ld_stream8(p.from.k + at + 2 * i * p.from.row_stride);
        v[i] = ld_stream8(p.from.v + at + 2 * i * p.from.row_stride);
      }
    }
    // the key's scale of row `lane`, the value's of row lane - 16
    uint32_t scale = 0;
    if (piece < here.n)
      scale = (half ? p.from.v_scale : p.from.k_scale)[here.src * p.from.scale_page + (from_row + piece) * p.from.scale_row +
                                                       here.h * p.from.scale_head];
    x = find(t + all_warps);
    const long long to = here.dst * p.to.page_stride + (to_row + half) * p.to.row_stride + here.h * p.to.head_stride + 8 * piece;
#pragma unroll
    for (int i = 0; i < UNIT / 2; ++i) {
      const float ks = scale_value(__shfl_sync(0xffffffffu, scale, 2 * i + half));
      const float vs = scale_value(__shfl_sync(0xffffffffu, scale, 16 + 2 * i + half));
      if (2 * i + half < here.n) {
        *reinterpret_cast<uint4*>(p.to.k + to + 2 * i * p.to.row_stride) = to_bf16(k[i], ks);
        *reinterpret_cast<uint4*>(p.to.v + to + 2 * i * p.to.row_stride) = to_bf16(v[i], vs);
      }
    }
  }
}

}  // namespace

cudaError_t launch_fp8_read(const Fp8ReadParams& p, cudaStream_t s) {
  if (p.B <= 0 || p.B > PAGED_MAX_SEQS || p.ctas <= 0) return cudaErrorInvalidValue;
  // no more CTAs than the tables have tasks for: a CTA finds out first how many rows there are
  const long long rows = static_cast<long long>(p.from.columns) << p.from.page_shift;
  const long long to = static_cast<long long>(p.to.columns) << p.to.page_shift;
  const long long tasks = (rows < to ? rows : to) / UNIT * p.B * p.n_kv;
  const long long most = static_cast<long long>(p.ctas) * CTAS_PER_SM, need = (tasks + WARPS - 1) / WARPS;
  return launch_behind(fp8_read_kernel, dim3(static_cast<unsigned>(need < most ? need : most)), WARPS * 32,
                       static_cast<size_t>(2 * p.B + 1) * 4, s, p);
}

}  // namespace gqa
