// Attention of one new token per sequence over an 8-bit paged cache ("Llama 3.1
// 8B · Grouped-query attention", mode decode; rows as in fp8.cuh): split over
// the length and joined as in paged_decode.cu, whose ranges and joins it uses.
//
// The bound is memory as there, with half the bytes a position: the arithmetic
// on a byte must cost half as much.
//   * A chunk is 32 positions of one KV head (8 KB of K and V), fetched by TMA:
//     one or two boxes of K and of V, 128-byte rows, swizzled. Its scale bytes
//     and page ids come one chunk ahead through registers, a position a lane.
//   * e4m3 goes to f16 (exact, one instruction for two values) between
//     ldmatrix and mma.sync m16n8k16, which then takes f16: to bf16 it would be
//     nine instructions for four values instead of two. Which dims share a
//     fragment is free as long as both operands agree: a lane's 4 bytes of K are
//     4 adjacent dims, and so are its dims of Q; V is transposed by pairs of
//     dims, the two tiles of a pair being its even and its odd dims.
//   * Queries enter as f16 times a power of two per head that takes their
//     largest dim to [2^14, 2^15): 11 bits for the 8 of bf16, exact down to
//     2^-28 of the largest dim, 2^-39 of it off below.
//   * A score is the product times the key's scale, in fp32. Values' scales go
//     into the probabilities, as exponents: 2^(s - m + e - M + 15) with m the
//     running max of s, M that of s - m + e, so that the largest term has all bits
//     whatever the scales, and 11 bits (f16) are left of each down to 2^-29 of it.
//     e is added to what is left of s once m is taken off: to a score in the
//     thousands it would be added with a rounding that shows in the result.
//   * The waits on the copies are bounded (gqa_set_wait_limit_ns). One that gives up
//     records DEV_WAIT_TIMEOUT; its CTA lets issued copies land and joins nothing.
// Measured (GB300, 6.8 TB/s copied): 93 to 102 us for 559 MB (64 sequences of
// up to 8,192 rows), 49 to 53 for 271 MB (one of 131,072), 29.9 for 133 MB
// (16 of 1,001, 32 KV heads), 11.5 for 33 MB (8 KV heads), 4.2 for one sequence
// of 16 rows. What bounds the long ones is the memory at 128-byte rows 1 KB
// apart: head-major pages ([page, KV head, row]) take 93.5 us where [page, row,
// KV head] took 104. More in flight changes nothing (3 stages: 99.7 for 99.9) or
// is worse (10 or 11 warps: 109 for 102), fewer warps are (6: 103); an L2 hint
// to evict first costs 5, 256-byte L2 promotion 20%. Eight KV heads side by side,
// a warp each, so that neighbouring rows are read together, took 101 us where 96
// (more parts to join, and the warps drift apart). With more than 8 query heads
// per KV head the joins are longer and the two tiles of heads bound it: 30.7 us
// for 88 MB.
#include "decode_parts.cuh"
#include "fp8.cuh"

namespace gqa {

namespace {

using namespace decode;

constexpr int KEYS = 32;                       // positions of a chunk
constexpr int TILE_BYTES = KEYS * HEAD_DIM;    // K or V of a chunk
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int STAGES = 2;
constexpr float P_EXP = 15.f;                  // probabilities enter the product times 2^15

// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// NT: 8-wide tiles of query heads (1: n_rep <= 8, 2: n_rep <= 16).
template <int NT>
__global__ void __launch_bounds__(WARPS * 32, 1)
    paged_decode_fp8_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                            const __grid_constant__ Fp8DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int W = WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rep = p.n_heads / p.n_kv;
  uint8_t* ring = smem + warp * (STAGES * STAGE_BYTES);
  // per warp: the partial of the part that began before its range; the one
  // that goes on behind it is put into the ring when the warp is done
  float* stash = reinterpret_cast<float*>(smem + W * (STAGES * STAGE_BYTES));
  int* pre = reinterpret_cast<int*>(stash + W * n_rep * PART);
  int* last = pre + p.B + 1;  // last row of each sequence
  __shared__ Shared sh;
  __shared__ uint64_t full[WARPS][STAGES];
  __shared__ int gave_up;  // a wait did
  if (threadIdx.x == 0) gave_up = 0;

  if (lane < STAGES) mbar_init(smem_u32(&full[warp][lane]), 1);
  fence_barrier_init();
  // nothing is read or written before the previous kernel of the stream is done
  pdl_trigger();
  pdl_wait();
  // chunks per sequence, prefix-summed; unused slots and bad positions have none
  const Count count = count_chunks<WARPS>(sh, pre, p.B, [&](int b) {
    const int s = p.start[b];
    const bool ok = s >= 0 && s < p.pages.capacity();
    if (!ok && s != -1 && blockIdx.x == 0) report(p.status, DEV_BAD_POSITION);
    last[b] = s;
    return ok ? s / KEYS + 1 : 0;
  });
  // rows of sequences without keys
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (pre[b + 1] == pre[b]) zero_rows(p.out, b, p.n_heads);

  const int total = count.total * p.n_kv;
  if (total == 0) return;
  const int ctas = decode_ctas(total, gridDim.x, W);
  const Split split(total, ctas);
  int c0, c1;
  if (!cta_range(total, count.longest, split, ctas, blockIdx.x, gridDim.x, pre, p.B, p.n_kv, c0, c1)) return;
  const int a0 = warp_start(c0, c1, warp, W), a1 = warp_start(c0, c1, warp + 1, W);
  const int n = a1 - a0;

  const int gr = lane >> 2, t = lane & 3;
  const int half = lane >> 4;

  bool ok = true;  // false: a wait gave up
  if (n > 0) {
    Cursor iss = locate(a0, pre, p.B, p.n_kv), cur = iss;
    const int in_page = (1 << p.pages.page_shift) - 1;
    const int box = min(KEYS, in_page + 1), boxes = KEYS / box;
    // The page of this lane's position of the chunk at `iss`, -1 past the
    // sequence. What is loaded ahead (pages, scales) is not looked at before it
    // is used: a look waits for it, 0.3 us each a chunk.
    constexpr int NONE = -1;
    bool in_seq;  // of `next`
    auto page_of = [&]() -> int {
      const int pos = iss.j * KEYS + lane;
      in_seq = pos <= last[iss.b];
      return in_seq ? p.pages.table[static_cast<long long>(iss.b) * p.pages.table_stride + (pos >> p.pages.page_shift)] : NONE;
    };
    int issued = 0;
    int next = page_of();
    const uint32_t ring32 = smem_u32(ring);
    // copies the chunk at `iss`; its scale bytes of this lane's position
    struct Scales {
      uint32_t k, v;
    };
    auto issue = [&]() -> Scales {
      Scales scales{127, 127};
      if (issued < n) {
        const uint32_t dst = ring32 + (issued % STAGES) * STAGE_BYTES, bar = smem_u32(&full[warp][issued % STAGES]);
        const int row = (iss.j * KEYS + lane) & in_page, h = iss.h;
        const bool good = next >= 0 && next < p.pages.num_pages;
        if (in_seq && !good) report(p.status, DEV_BAD_PAGE);
        const int page = good ? next : NONE;
        if (good) {
          const long long at = page * p.pages.scale_page + row * p.pages.scale_row + h * p.pages.scale_head;
          scales = {p.pages.k_scale[at], p.pages.v_scale[at]};
        }
        // lane x < boxes: box x of K, the next ones of V
        const int x = lane % boxes;
        const int first_page = __shfl_sync(0xffffffffu, page, x * box);
        const int first_row = __shfl_sync(0xffffffffu, row, x * box);
        const bool copies = lane < 2 * boxes && first_page >= 0;
        const unsigned held = __popc(__ballot_sync(0xffffffffu, copies));
        if (lane == 0) mbar_expect_tx(bar, held * box * HEAD_DIM);
        __syncwarp();
        if (copies)
          tma_load_4d(dst + (lane >= boxes ? TILE_BYTES : 0) + x * box * HEAD_DIM, lane >= boxes ? &mv : &mk, bar,
                             0, h, first_row, first_page);
        ++issued;
        if (issued < n) {
          advance(iss, pre, p.B, p.n_kv);
          next = page_of();
        }
      }
      return scales;
    };
    static_assert(STAGES == 2, "one chunk's scales in hand");
    Scales ahead = issue();

    uint32_t qb[NT][8][2];  // Q^T as B fragments: dims 16s + 4t (+1) | +2 (+3), query head 8 nt + gr
    float q_scale[NT][2];   // what takes the products of heads 8 nt + 2t (+1) to scores in log2 units
    float m_run[NT][2], l_run[NT][2], v_run[NT][2], oacc[NT][8][4];  // heads 8 nt + 2t (+1); O^T tile d: dims 16d + 2 gr (+1)
    for (int i = 0; i < n; ++i) {
      const Scales scales = ahead;
      ahead = issue();
      if (i == 0 || cur.j == 0) {
        const __nv_bfloat16* q = p.q + cur.b * p.q_stride + cur.h * n_rep * HEAD_DIM + 4 * t;
        uint2 all[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            all[nt][s] = make_uint2(0, 0);
            if (nt * 8 + gr < n_rep) all[nt][s] = __ldg(reinterpret_cast<const uint2*>(q + (nt * 8 + gr) * HEAD_DIM + 16 * s));
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2(&x)[8] = all[nt];
          uint32_t most = 0;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            most = max(most, max(max(finite_bits(bf16_lo(x[s].x)), finite_bits(bf16_hi(x[s].x))),
                                 max(finite_bits(bf16_lo(x[s].y)), finite_bits(bf16_hi(x[s].y)))));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int e = min(14 + 127 - static_cast<int>(most >> 23), 120);
          const float up = power_of_two(e);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            qb[nt][s][0] = pack_f16(bf16_lo(x[s].x) * up, bf16_hi(x[s].x) * up);
            qb[nt][s][1] = pack_f16(bf16_lo(x[s].y) * up, bf16_hi(x[s].y) * up);
          }
          const float down = p.scale_log2 * power_of_two(-e);
          q_scale[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
          q_scale[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
          m_run[nt][0] = m_run[nt][1] = v_run[nt][0] = v_run[nt][1] = -INFINITY;
          l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
          for (int d = 0; d < 8; ++d) oacc[nt][d][0] = oacc[nt][d][1] = oacc[nt][d][2] = oacc[nt][d][3] = 0.f;
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait_within(smem_u32(&full[warp][i % STAGES]), (i / STAGES) & 1, p.wait_ns));
      if (!ok) break;
      const uint32_t kt = ring32 + (i % STAGES) * STAGE_BYTES, vt = kt + TILE_BYTES;
      const int left = last[cur.b] - cur.j * KEYS;
      if (left < KEYS - 1) {
        // value rows past the sequence may hold anything: 0 x NaN is NaN
        for (int w = lane; w < (KEYS - 1 - left) * 8; w += 32)
          st_shared_v4(vt + (left + 1 + (w >> 3)) * HEAD_DIM + (w & 7) * 16, make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();
        __syncwarp();
      }

      float sc[NT][2][4], sd[NT][2][4];  // keys 16 m + gr (+8), heads 2t (+1): two sums, added up below
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][m][e] = sd[nt][m][e] = 0.f;
      uint32_t kr[4][2][4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          ldsm_x4(kt + m * 16 * HEAD_DIM + sw128(lane & 15, 2 * s + half), kr[s][m][0], kr[s][m][1], kr[s][m][2], kr[s][m][3]);
#pragma unroll
      for (int s = 0; s < 8; s += 2)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t lo[4], hi[4];
          const uint32_t(&r)[4] = kr[s / 2][m];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_f16(r[e], lo[e], hi[e]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(sc[nt][m], lo[0], lo[1], hi[0], hi[1], qb[nt][s][0], qb[nt][s][1]);
            mma_f16(sd[nt][m], lo[2], lo[3], hi[2], hi[3], qb[nt][s + 1][0], qb[nt][s + 1][1]);
          }
        }
      // One tile of heads: the values are converted here, beside the softmax's long
      // chain of dependent steps, two while it leaves no registers for that.
      uint32_t even[4][2][4], odd[4][2][4];
      auto values = [&](int d, int m) {
        uint32_t r[4];
        ldsm_x4_t(vt + m * 16 * HEAD_DIM + sw128(lane & 15, 2 * d + half), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) e4m3x4_to_f16(__byte_perm(r[e], 0, 0x3120), even[d][m][e], odd[d][m][e]);
      };
      if (NT == 1) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int m = 0; m < 2; ++m) values(d, m);
      }
      // the scales of keys gr, gr + 8, gr + 16, gr + 24
      float ks[4], ve[4];
      const uint32_t both = scales.k | scales.v << 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = __shfl_sync(0xffffffffu, both, gr + 8 * e);
        ks[e] = scale_value(x & 0xffu);
        ve[e] = static_cast<float>(static_cast<int>(x >> 8) - 127);
      }
      uint32_t pb[NT][2][2];  // P^T as B fragments: keys 16 m + 2t (+1) | +8, head gr
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pw[2][4], al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x[4], y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = gr + 8 * k <= left ? (sc[nt][k >> 1][(k & 1) * 2 + e] + sd[nt][k >> 1][(k & 1) * 2 + e]) * (ks[k] * q_scale[nt][e])
                                      : -INFINITY;
          float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(mx, m_run[nt][e]);
          // scores that are all -inf leave the maximum there: no term, not a NaN
          const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] -= ref;
            y[k] = x[k] + ve[k];
          }
          float my = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, o));
          const float before = v_run[nt][e] + (m_run[nt][e] - ref);
          my = fmaxf(my, before);
          const float vref = my == -INFINITY ? 0.f : my;
          al[e] = ex2_approx(before - vref);
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum += ex2_approx(x[k]);
            pw[k >> 1][(k & 1) * 2 + e] = ex2_approx(y[k] - vref + P_EXP);
          }
          l_run[nt][e] = l_run[nt][e] * ex2_approx(m_run[nt][e] - ref) + sum;  // this lane's rows; summed over lanes at the end
          m_run[nt][e] = mx;
          v_run[nt][e] = my;
        }
        // the maxima settle after a few chunks
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            oacc[nt][d][0] *= al[0];
            oacc[nt][d][1] *= al[1];
            oacc[nt][d][2] *= al[0];
            oacc[nt][d][3] *= al[1];
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          pb[nt][m][0] = movmatrix_t(pack_f16(pw[m][0], pw[m][1]));
          pb[nt][m][1] = movmatrix_t(pack_f16(pw[m][2], pw[m][3]));
        }
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (NT > 1) values(d, m);
          const uint32_t(&x)[4] = even[d][m], (&y)[4] = odd[d][m];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(oacc[nt][2 * d], x[0], y[0], x[1], y[1], pb[nt][m][0], pb[nt][m][1]);
            mma_f16(oacc[nt][2 * d + 1], x[2], y[2], x[3], y[3], pb[nt][m][0], pb[nt][m][1]);
          }
        }
      __syncwarp();  // the chunk's rows are read before its slot is filled again

      const Cursor here = cur;
      advance(cur, pre, p.B, p.n_kv);
      if (i + 1 < n && cur.j != 0) continue;

      // end of this warp's part of (here.b, here.h)
      const int first = pre[here.b] * p.n_kv + here.h * here.n;
      const Part seg{first, first + here.n, here.b * p.n_heads + here.h * n_rep};
      float to_m[NT][2];  // what takes O from its own reference to the sum's
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], o);
          to_m[nt][e] = v_run[nt][e] == -INFINITY ? 0.f : ex2_approx(v_run[nt][e] - P_EXP);
        }
      if (seg.first >= a0 && seg.end <= a1) {
        __nv_bfloat16* out = p.out + static_cast<long long>(seg.row) * HEAD_DIM;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float i0 = 1.f / l_run[nt][0], i1 = 1.f / l_run[nt][1];
          const int h = nt * 8 + gr;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            // (dims 2 gr, 2 gr + 1, heads 2t, 2t + 1) -> (head gr, dims 4t .. 4t + 3)
            const uint32_t w0 = movmatrix_t(pack_bf16(oacc[nt][d][0] * i0 * to_m[nt][0], oacc[nt][d][1] * i1 * to_m[nt][1]));
            const uint32_t w1 = movmatrix_t(pack_bf16(oacc[nt][d][2] * i0 * to_m[nt][0], oacc[nt][d][3] * i1 * to_m[nt][1]));
            if (h < n_rep)
              *(reinterpret_cast<uint2*>(out + h * HEAD_DIM + 16 * d) + t) =
                  make_uint2(__byte_perm(w0, w1, 0x5410), __byte_perm(w0, w1, 0x7632));
          }
        }
      } else {
        const int slot = seg.first < a0 ? 0 : 1;
        // the last part of the range goes into the ring: every copy into it has landed and been read
        float* part = slot == 0 ? stash + warp * n_rep * PART : reinterpret_cast<float*>(ring);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = nt * 8 + 2 * t + e;
            if (h >= n_rep) continue;
            float* row = part + h * PART;
#pragma unroll
            for (int d = 0; d < 8; ++d)
              *reinterpret_cast<float2*>(row + 16 * d + 2 * gr) =
                  make_float2(oacc[nt][d][e] * to_m[nt][e], oacc[nt][d][e + 2] * to_m[nt][e]);
            if (gr == 0) {
              row[HEAD_DIM] = m_run[nt][e];
              row[HEAD_DIM + 1] = l_run[nt][e];
            }
          }
        if (lane == 0) sh.parts[2 * warp + slot] = seg;
      }
    }
    if (!ok) {
      // the copies in flight land in the ring: nothing else is done with it before
      if (lane == 0) report(p.status, DEV_WAIT_TIMEOUT);
      for (int u = max(0, issued - STAGES); u < issued; ++u) mbar_wait(smem_u32(&full[warp][u % STAGES]), (u / STAGES) & 1);
    }
  }
  // A CTA that gave up joins nothing, and counts at no ticket.
  if (!ok) gave_up = 1;
  __syncthreads();
  if (gave_up) return;
  join_parts(
      sh, reinterpret_cast<float*>(smem), split, blockIdx.x, c0, c1, n_rep, p.part_o, p.part_ml, p.tickets,
      [&](int e) -> const float* {
        return (e & 1) ? reinterpret_cast<const float*>(smem + (e >> 1) * (STAGES * STAGE_BYTES))
                       : stash + (e >> 1) * n_rep * PART;
      },
      [&](int row, float4 o, float m, float l) { store_row(p.out, row, o, 1.f / l); });
}

template <int NT>
cudaError_t launch_nt(const Fp8DecodeMaps& maps, const Fp8DecodeParams& p, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_decode_fp8_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int n_rep = p.n_heads / p.n_kv;
  const size_t smem = static_cast<size_t>(WARPS) * (STAGES * STAGE_BYTES + n_rep * PART * 4) + (2 * p.B + 1) * 4 + 1024;
  return launch_behind(paged_decode_fp8_kernel<NT>, static_cast<unsigned>(p.ctas), WARPS * 32, smem, s, maps.k, maps.v, p);
}

}  // namespace

int fp8_decode_box_rows(int page_size) { return page_size < KEYS ? page_size : KEYS; }

cudaError_t launch_paged_decode_fp8(const Fp8DecodeMaps& maps, const Fp8DecodeParams& p, cudaStream_t s) {
  if (p.B <= 0 || p.B > PAGED_MAX_SEQS || p.ctas <= 0) return cudaErrorInvalidValue;
  const int n_rep = p.n_heads / p.n_kv;
  if (n_rep < 1 || n_rep > PAGED_MAX_REP) return cudaErrorInvalidValue;
  return n_rep <= 8 ? launch_nt<1>(maps, p, s) : launch_nt<2>(maps, p, s);
}

}  // namespace gqa
