// RoPE in any layout and cache append of packed tokens, into bf16 pages or,
// quantised, into 8-bit pages ("Llama 3.1 8B · Grouped-query attention":
// apply_rotary_emb, then cache_k/v[b, start_pos + t] = k, v; other models turn
// dims i and i + R/2 as a pair, or the first R of the 128 dims alone).
//
// Turned values are products and sums of fp32, each rounded (not contracted:
// a value near the border of two e4m3 steps is then on the same side as in the
// formula's own arithmetic), rounded once to what is stored. Scales and e4m3:
// fp8.cuh. Values that are not finite take no part in a row's scale and are
// held as e4m3's NaN.
//
// Every row is read once and written once, so the bound is memory. As in
// paged_append.cu one warp takes 8 of a token's n_heads + 2 n_kv head rows, two
// at a time (16 lanes x 8 dims each), the rows' loads first, and the (cos, sin)
// of a token once for its 8 rows. A pair of halves lies in two lanes: they
// swap their dims. The largest |x| of a row is four exchanges of its 16 lanes.
#include "fp8.cuh"
#include "paged.h"

namespace gqa {

namespace {

constexpr int WARPS = 4;
constexpr int ROWS = 8;  // head rows per warp

__device__ __forceinline__ void unpack(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
// a c - b s and a s + b c
__device__ __forceinline__ float turned_first(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turned_second(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
}

template <bool HALVES, bool FP8>
__global__ void __launch_bounds__(WARPS * 32) rotary_append_kernel(const __grid_constant__ RotaryAppendParams rp, int groups) {
  const PagedAppendParams& p = rp.a;
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
    x[i] = make_uint4(0, 0, 0, 0);
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
  if (start < 0 || pos >= p.rope_rows || pos >= (FP8 ? rp.pages8.capacity() : p.pages.capacity())) {
    if (lane == 0) report(p.status, DEV_BAD_POSITION);
    return;
  }
  const int shift = FP8 ? rp.pages8.page_shift : p.pages.page_shift;
  const int* table = FP8 ? rp.pages8.table : p.pages.table;
  const int page = table[static_cast<long long>(b) * (FP8 ? rp.pages8.table_stride : p.pages.table_stride) + (pos >> shift)];
  if (page < 0 || page >= (FP8 ? rp.pages8.num_pages : p.pages.num_pages)) {
    if (lane == 0) report(p.status, DEV_BAD_PAGE);
    return;
  }
  const long long in_page = pos & ((1 << shift) - 1);

  // the (cos, sin) of this lane's 8 dims: 4 adjacent pairs, or 8 pairs that it
  // has one dim of; lanes past the turned dims have none
  const int pieces = rp.rotary_dim / 8, across = pieces / 2;
  const bool turns = piece < pieces, second = HALVES && piece >= across;
  constexpr int CS = HALVES ? 8 : 4;
  float2 cs[CS];
  {
    const float4* src = reinterpret_cast<const float4*>(p.rope + pos * rp.rotary_dim) +
                        (HALVES ? (second ? piece - across : piece) * 4 : piece * 2);
#pragma unroll
    for (int i = 0; i < CS / 2; ++i) {
      float4 c = make_float4(1.f, 0.f, 1.f, 0.f);
      if (turns) c = __ldg(src + i);
      cs[2 * i] = make_float2(c.x, c.y);
      cs[2 * i + 1] = make_float2(c.z, c.w);
    }
  }
  const int other = (lane & 16) | (turns ? (second ? piece - across : piece + across) : piece);

#pragma unroll
  for (int i = 0; i < ROWS / 2; ++i) {
    const int r = row0 + 2 * i + half;
    const bool is_kv = r >= p.n_heads, is_v = r >= p.n_heads + p.n_kv;
    float f[8];
    unpack(x[i], f);
    if (HALVES) {
      uint4 y;
      y.x = __shfl_sync(0xffffffffu, x[i].x, other);
      y.y = __shfl_sync(0xffffffffu, x[i].y, other);
      y.z = __shfl_sync(0xffffffffu, x[i].z, other);
      y.w = __shfl_sync(0xffffffffu, x[i].w, other);
      float g[8];
      unpack(y, g);
      if (!is_v && turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = second ? turned_second(g[e], f[e], cs[e % CS]) : turned_first(f[e], g[e], cs[e % CS]);
      }
    } else if (!is_v && turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = f[2 * e], c = f[2 * e + 1];
        f[2 * e] = turned_first(a, c, cs[e]);
        f[2 * e + 1] = turned_second(a, c, cs[e]);
      }
    }
    if (!FP8 || !is_kv) {
      const uint4 y = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
      if (r < rows) {
        __nv_bfloat16* dst;
        if (!is_kv) {
          dst = p.q_out + (static_cast<long long>(m) * p.n_heads + r) * HEAD_DIM;
        } else {
          const long long at = page * p.pages.page_stride + in_page * p.pages.row_stride;
          dst = is_v ? p.pages.v + at + (r - p.n_heads - p.n_kv) * p.pages.head_stride
                     : p.pages.k + at + (r - p.n_heads) * p.pages.head_stride;
        }
        // what is not turned is stored as it came, a NaN's bits among it
        *(reinterpret_cast<uint4*>(dst) + piece) = is_v || !turns ? x[i] : y;
      }
    }
    if (FP8) {
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(f[e]) & 0x7fffffffu;
        if (u < 0x7f800000u) most = max(most, u);
        else f[e] = __uint_as_float(0x7fffffffu);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      const int e = row_exponent(most);
      const float s = power_of_two(-e);
      if (r < rows && is_kv) {
        const int h = r - p.n_heads - (is_v ? p.n_kv : 0);
        const Fp8Cache& c = rp.pages8;
        uint8_t* dst = (is_v ? c.v : c.k) + page * c.page_stride + in_page * c.row_stride + h * c.head_stride;
        const uint2 y = make_uint2(to_e4m3x2(f[0] * s, f[1] * s) | to_e4m3x2(f[2] * s, f[3] * s) << 16,
                                   to_e4m3x2(f[4] * s, f[5] * s) | to_e4m3x2(f[6] * s, f[7] * s) << 16);
        *(reinterpret_cast<uint2*>(dst) + piece) = y;
        if (piece == 0)
          (is_v ? c.v_scale : c.k_scale)[page * c.scale_page + in_page * c.scale_row + h * c.scale_head] =
              static_cast<uint8_t>(e + 127);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryAppendParams& p, cudaStream_t s) {
  const int groups = (p.a.n_heads + 2 * p.a.n_kv + ROWS - 1) / ROWS;
  const long long blocks = (static_cast<long long>(p.a.N) * groups + WARPS - 1) / WARPS;
  if (blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const auto kernel = p.halves ? (p.fp8 ? rotary_append_kernel<true, true> : rotary_append_kernel<true, false>)
                               : (p.fp8 ? rotary_append_kernel<false, true> : rotary_append_kernel<false, false>);
  return launch_behind(kernel, static_cast<unsigned>(blocks), WARPS * 32, 0, s, p, groups);
}

}  // namespace gqa
