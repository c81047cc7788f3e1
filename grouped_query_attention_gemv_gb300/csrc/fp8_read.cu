// Rows of an 8-bit cache back into bf16 pages (exact, fp8.cuh), for what reads
// a bf16 cache: the prefill attention of a chunk after a quantised prefix, or a
// cache that moves.
//
// 129 bytes read and 256 written a row: the bound is memory. The batch's rows
// are cut into units of 16 positions (one page of both sides each), shared out
// evenly over the grid; a warp takes 4 rows of K and of V at a time, 8 lanes x
// 16 values each.
#include "fp8.cuh"
#include "paged.h"

namespace gqa {

namespace {

constexpr int WARPS = 8, CTAS_PER_SM = 4;
constexpr int UNIT = 16;  // positions

__device__ __forceinline__ uint4 to_bf16(uint32_t x, uint32_t y, float s) {
  uint32_t h[4];
  e4m3x4_to_f16(x, h[0], h[1]);
  e4m3x4_to_f16(y, h[2], h[3]);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    r[i] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__global__ void __launch_bounds__(WARPS * 32, CTAS_PER_SM) fp8_read_kernel(const __grid_constant__ Fp8ReadParams p) {
  extern __shared__ int pre[];  // units before each sequence
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
  const Split split(total, gridDim.x);
  const int u0 = split.start(blockIdx.x), u1 = split.start(blockIdx.x + 1);
  const int sub = lane >> 3, piece = lane & 7;
  int b = 0;
#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    if (u == u0) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= u) lo = mid; else hi = mid;
      }
      b = lo;
    }
    while (pre[b + 1] <= u) ++b;
    const int pos0 = (u - pre[b]) * UNIT, n = min(UNIT, p.rows[b] - pos0) * p.n_kv;
    const int src = p.from.table[static_cast<long long>(b) * p.from.table_stride + (pos0 >> p.from.page_shift)];
    const int dst = p.to.table[static_cast<long long>(b) * p.to.table_stride + (pos0 >> p.to.page_shift)];
    if (src < 0 || src >= p.from.num_pages || dst < 0 || dst >= p.to.num_pages) {
      if (threadIdx.x == 0) report(p.status, DEV_BAD_PAGE);
      continue;
    }
    const long long at = src * p.from.page_stride + (pos0 & ((1 << p.from.page_shift) - 1)) * p.from.row_stride;
    const long long sc = src * p.from.scale_page + (pos0 & ((1 << p.from.page_shift) - 1)) * p.from.scale_row;
    const long long to = dst * p.to.page_stride + (pos0 & ((1 << p.to.page_shift) - 1)) * p.to.row_stride;
#pragma unroll 2
    for (int r = 4 * warp + sub; r < n; r += 4 * WARPS) {
      const int x = r / p.n_kv, h = r - x * p.n_kv;
      const long long from = at + x * p.from.row_stride + h * p.from.head_stride;
      const uint4 k = ld_stream(p.from.k + from + 16 * piece), v = ld_stream(p.from.v + from + 16 * piece);
      const long long s = sc + x * p.from.scale_row + h * p.from.scale_head;
      const float ks = scale_value(p.from.k_scale[s]), vs = scale_value(p.from.v_scale[s]);
      const long long out = to + x * p.to.row_stride + h * p.to.head_stride + 16 * piece;
      uint4* ko = reinterpret_cast<uint4*>(p.to.k + out);
      uint4* vo = reinterpret_cast<uint4*>(p.to.v + out);
      ko[0] = to_bf16(k.x, k.y, ks);
      ko[1] = to_bf16(k.z, k.w, ks);
      vo[0] = to_bf16(v.x, v.y, vs);
      vo[1] = to_bf16(v.z, v.w, vs);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_read(const Fp8ReadParams& p, cudaStream_t s) {
  if (p.B <= 0 || p.B > PAGED_MAX_SEQS || p.ctas <= 0) return cudaErrorInvalidValue;
  return launch_behind(fp8_read_kernel, dim3(static_cast<unsigned>(p.ctas) * CTAS_PER_SM), WARPS * 32,
                       static_cast<size_t>(p.B + 1) * 4, s, p);
}

}  // namespace gqa
