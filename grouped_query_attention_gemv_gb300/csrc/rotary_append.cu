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
// Every row is read once and written once, so the bound is memory, and as near
// to it the instructions a value: 40 bytes a lane and row pass some 90 of them.
// As in paged_append.cu a warp takes 8 of a token's n_heads + 2 n_kv head rows,
// two at a time (16 lanes x 8 dims each), the rows' loads first, and the (cos,
// sin) of a token once. A batch of 8 is of queries, keys or values alone, so
// that addresses and what is done with it are found once (7 prompts, 356 MB:
// 80 us row by row, 69 so). A pair of halves lies in two lanes: they swap their
// dims. The largest |x| of a row is four exchanges of its 16 lanes. With many
// tokens a warp takes several batches, so that the chain to the token's place
// is walked less often.
// Measured (GB300, 6.8 TB/s copied), 32 and 8 heads: 59.6 us for 7 prompts into
// 8 bits (356 MB), 38.7 for 5 prompts into bf16, 64 dims turned (244 MB), 2.8
// for one token, 2.9 for 64.
#include <math.h>

#include "fp8.cuh"
#include "paged.h"

namespace gqa {

namespace {

constexpr int WARPS = 4;
constexpr int ROWS = 8;  // head rows of a warp at a time

__device__ __forceinline__ void unpack(uint4 x, float2 (&f)[4]) {
  f[0] = make_float2(bf16_lo(x.x), bf16_hi(x.x));
  f[1] = make_float2(bf16_lo(x.y), bf16_hi(x.y));
  f[2] = make_float2(bf16_lo(x.z), bf16_hi(x.z));
  f[3] = make_float2(bf16_lo(x.w), bf16_hi(x.w));
}
// own c + other s: dims of a pair (a, b) turned, a c - b s with s negated, b c + a s
__device__ __forceinline__ float2 turned(float2 own, float2 other, float2 c, float2 s) {
  return make_float2(__fadd_rn(__fmul_rn(own.x, c.x), __fmul_rn(other.x, s.x)),
                     __fadd_rn(__fmul_rn(own.y, c.y), __fmul_rn(other.y, s.y)));
}

template <bool HALVES, bool FP8>
__global__ void __launch_bounds__(WARPS * 32) rotary_append_kernel(const __grid_constant__ RotaryAppendParams rp, int shares, int each) {
  const PagedAppendParams& p = rp.a;
  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, half = lane >> 4, piece = lane & 15;
  // the warps of a token follow each other
  const unsigned long long item = static_cast<unsigned long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int m = static_cast<int>(item >> 32 ? item / shares : static_cast<unsigned>(item) / static_cast<unsigned>(shares));
  if (m >= p.N) return;
  int row0 = static_cast<int>(item - static_cast<unsigned long long>(m) * shares) * each * ROWS;
  const int row_end = min(p.n_heads + 2 * p.n_kv, row0 + each * ROWS);
  // A batch is rows row0 .. row0 + n - 1 of the queries, the keys or the values:
  // addresses are found once a batch, and a batch does one thing.
  int n = 0;
  enum { QUERY, KEY, VALUE } kind = QUERY;
  uint4 x[ROWS / 2];
  auto load = [&]() {
    kind = row0 < p.n_heads ? QUERY : row0 < p.n_heads + p.n_kv ? KEY : VALUE;
    const int first = kind == QUERY ? 0 : kind == KEY ? p.n_heads : p.n_heads + p.n_kv;
    n = min(ROWS, min(row_end, first + (kind == QUERY ? p.n_heads : p.n_kv)) - row0);
    const __nv_bfloat16* src = (kind == QUERY ? p.q + m * p.q_stride : kind == KEY ? p.k + m * p.k_stride : p.v + m * p.v_stride) +
                               (row0 - first + half) * HEAD_DIM + piece * 8;
#pragma unroll
    for (int i = 0; i < ROWS / 2; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      // q may be rotated in place: not the read-only path
      if (2 * i + half < n) x[i] = *reinterpret_cast<const uint4*>(src + 2 * i * HEAD_DIM);
    }
  };
  load();

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
  float2 cos2[4], sin2[4];  // of this lane's dims, two each; -sin for the first dim of a pair
  {
    const float4* src = reinterpret_cast<const float4*>(p.rope + pos * rp.rotary_dim) +
                        (HALVES ? (second ? piece - across : piece) * 4 : piece * 2);
    const float sign = second ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < (HALVES ? 4 : 2); ++i) {
      float4 c = make_float4(1.f, 0.f, 1.f, 0.f);
      if (turns) c = __ldg(src + i);
      if (HALVES) {
        cos2[i] = make_float2(c.x, c.z);
        sin2[i] = make_float2(c.y * sign, c.w * sign);
      } else {
        cos2[2 * i] = make_float2(c.x, c.x);
        sin2[2 * i] = make_float2(-c.y, c.y);
        cos2[2 * i + 1] = make_float2(c.z, c.z);
        sin2[2 * i + 1] = make_float2(-c.w, c.w);
      }
    }
  }
  const int other = (lane & 16) | (turns ? (second ? piece - across : piece + across) : piece);

  // a lane's dims of its row of the i-th two, turned
  auto turn = [&](int i, float2(&f)[4]) {
    unpack(x[i], f);
    if (HALVES) {
      uint4 y;
      y.x = __shfl_sync(0xffffffffu, x[i].x, other);
      y.y = __shfl_sync(0xffffffffu, x[i].y, other);
      y.z = __shfl_sync(0xffffffffu, x[i].z, other);
      y.w = __shfl_sync(0xffffffffu, x[i].w, other);
      float2 g[4];
      unpack(y, g);
      if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = turned(f[e], g[e], cos2[e], sin2[e]);
      }
    } else if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = turned(f[e], make_float2(f[e].y, f[e].x), cos2[e], sin2[e]);
    }
  };
  // the row in bf16; what is not turned as it came, a NaN's bits among it
  auto in_bf16 = [&](int i, const float2(&f)[4]) {
    return turns ? make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                              pack_bf16(f[3].x, f[3].y))
                 : x[i];
  };
  // a row's values to 8 bits; its exponent
  auto in_fp8 = [&](float2(&f)[4], int& e) {
    // fmaxf passes over NaN, which stays one; infinities are rare
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) most = max3(most, fabsf(f[k].x), fabsf(f[k].y));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (__any_sync(0xffffffffu, most == INFINITY)) {
      most = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (fabsf(f[k].x) == INFINITY) f[k].x = __uint_as_float(0x7fffffffu);
        if (fabsf(f[k].y) == INFINITY) f[k].y = __uint_as_float(0x7fffffffu);
        most = max3(most, fabsf(f[k].x), fabsf(f[k].y));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    e = row_exponent(__float_as_uint(most));
    const float2 s = make_float2(power_of_two(-e), power_of_two(-e));
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = mul2(f[k], s);
    if (e == MOST_E) {
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = make_float2(within_reach(f[k].x), within_reach(f[k].y));
    }
    return make_uint2(to_e4m3x2(f[0].x, f[0].y) | to_e4m3x2(f[1].x, f[1].y) << 16,
                      to_e4m3x2(f[2].x, f[2].y) | to_e4m3x2(f[3].x, f[3].y) << 16);
  };

#pragma unroll 1
  for (;;) {
    if (kind == QUERY) {
      __nv_bfloat16* dst = p.q_out + (static_cast<long long>(m) * p.n_heads + row0 + half) * HEAD_DIM + piece * 8;
#pragma unroll
      for (int i = 0; i < ROWS / 2; ++i) {
        float2 f[4];
        turn(i, f);
        if (2 * i + half < n) *reinterpret_cast<uint4*>(dst + 2 * i * HEAD_DIM) = in_bf16(i, f);
      }
    } else {
      const bool key = kind == KEY;
      const int h = row0 + half - p.n_heads - (key ? 0 : p.n_kv);
      if (FP8) {
        const Fp8Cache& c = rp.pages8;
        uint8_t* dst = (key ? c.k : c.v) + page * c.page_stride + in_page * c.row_stride + h * c.head_stride + piece * 8;
        uint8_t* scale = (key ? c.k_scale : c.v_scale) + page * c.scale_page + in_page * c.scale_row + h * c.scale_head;
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i) {
          float2 f[4];
          if (key) turn(i, f);
          else unpack(x[i], f);
          int e;
          const uint2 y = in_fp8(f, e);
          if (2 * i + half < n) {
            *reinterpret_cast<uint2*>(dst) = y;
            if (piece == 0) *scale = static_cast<uint8_t>(e + 127);
          }
          dst += 2 * c.head_stride;
          scale += 2 * c.scale_head;
        }
      } else {
        __nv_bfloat16* dst = (key ? p.pages.k : p.pages.v) + page * p.pages.page_stride + in_page * p.pages.row_stride +
                             h * p.pages.head_stride + piece * 8;
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i) {
          uint4 y = x[i];
          if (key) {
            float2 f[4];
            turn(i, f);
            y = in_bf16(i, f);
          }
          if (2 * i + half < n) *reinterpret_cast<uint4*>(dst) = y;
          dst += 2 * p.pages.head_stride;
        }
      }
    }
    row0 += n;
    if (row0 >= row_end) break;
    load();
  }
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryAppendParams& p, cudaStream_t s) {
  // Batches of a warp. Measured, 1 / 2 / all 6 of a token, halves, us: into 8
  // bits 1,024 tokens 7.0 / 6.8 / 10.4, 2,048 13.1 / 13.5 / 14.3, 4,096 21.4 /
  // 20.7 / 18.7, 8,192 37.7 / 35.4 / 32.7; into bf16 1,024 6.5 / 6.2 / 9.4, 2,048
  // 12.6 / 12.2 / 12.9, 4,096 20.7 / 19.1 / 18.9, 8,192 36.6 / 33.7 / 34.0.
  const int groups = (p.a.n_heads + 2 * p.a.n_kv + ROWS - 1) / ROWS;
  const int each = p.fp8 ? (p.a.N >= 4096 ? groups : 1) : p.a.N >= 2048 ? 2 : 1, shares = (groups + each - 1) / each;
  const long long blocks = (static_cast<long long>(p.a.N) * shares + WARPS - 1) / WARPS;
  if (blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const auto kernel = p.halves ? (p.fp8 ? rotary_append_kernel<true, true> : rotary_append_kernel<true, false>)
                               : (p.fp8 ? rotary_append_kernel<false, true> : rotary_append_kernel<false, false>);
  return launch_behind(kernel, static_cast<unsigned>(blocks), WARPS * 32, 0, s, p, shares, each);
}

}  // namespace gqa
