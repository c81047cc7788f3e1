// The inner loop of the decode attentions over bf16 pages: a CTA's chunks
// streamed by its warps and joined (paged_decode.cu says how and why).
#pragma once

#include "decode_parts.cuh"

namespace gqa {
namespace decode {

constexpr int KEYS = 16;                          // positions of a chunk
constexpr int ROW_BYTES = HEAD_DIM * 2;
constexpr int TILE_BYTES = KEYS * ROW_BYTES;      // K or V of a chunk
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int STAGES = 2;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;  // of a warp

// Row r, 16-byte piece c of a 256-byte-row tile: eight rows of one piece fall
// into eight different 16-byte columns.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return static_cast<uint32_t>(r * ROW_BYTES + ((c ^ (r & 7)) << 4));
}

// Chunks [c0, c1) of the batch, by CTA `cta` of those that share its chunks
// out, the first WARPS warps of it. rings: WARPS * RING_BYTES of shared memory,
// stash: WARPS * n_rep * PART floats. pre, last: chunks before each sequence, its
// last row. NT: 8-wide tiles of query heads (1: n_rep <= 8, 2: n_rep <= 16).
// SHARED: begin is a sequence's first row that is read, and nothing is joined
// (no stash): each warp's part of a (sequence, KV head) goes to p.own_o and
// p.own_ml, n_rep rows at place (sequence x n_kv + KV head) + (cta x WARPS +
// warp), of which every step from part to part takes one at least further.
// Joining in the CTA and across CTAs took 8 us at its end, 14 in the last, where
// a join follows anyway.
template <int NT, bool SHARED>
__device__ __forceinline__ void stream_chunks(const PagedDecodeParams& p, Shared& sh, uint8_t* rings, float* stash,
                                              const int* pre, const int* last, const int* begin, const Split& split,
                                              int cta, int c0, int c1) {
  constexpr int W = WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rep = p.n_heads / p.n_kv;
  // per warp: a ring, and the partial of the part that began before its range;
  // the one that goes on behind it is put into the ring when the warp is done
  uint8_t* ring = rings + warp * RING_BYTES;
  const int with = SHARED ? least(W, c1 - c0) : W;  // warps that share the chunks
  const int a0 = warp_start(c0, c1, warp, with), a1 = warp < with ? warp_start(c0, c1, warp + 1, with) : a0;
  const int n = a1 - a0;

  const int gr = lane >> 2, t = lane & 3;
  const int half = lane >> 4, piece = lane & 15;

  if (n > 0) {
    Cursor iss = locate(a0, pre, p.B, p.n_kv), cur = iss;
    // The page of row lane % 16 of the chunk at `iss`, if it is one that is read.
    // It is loaded a chunk ahead and not looked at before its use: a look waits.
    int row = 0;          // within the page
    bool reads = false;
    auto page_of = [&]() -> int {
      const int f = SHARED ? begin[iss.b] : 0;
      const int pos = (iss.j + f / KEYS) * KEYS + piece;
      reads = pos <= last[iss.b] && (!SHARED || pos >= f);
      row = pos & ((1 << p.pages.page_shift) - 1);
      return reads ? p.pages.table[static_cast<long long>(iss.b) * p.pages.table_stride + (pos >> p.pages.page_shift)] : 0;
    };
    int issued = 0;
    int page = page_of();
    const uint32_t ring32 = smem_u32(ring);
    auto issue = [&]() {
      if (issued < n) {
        const uint32_t dst = ring32 + (issued % STAGES) * STAGE_BYTES;
        // element offset of the row, -1: zeros instead
        long long off = -1;
        if (reads) {
          if (page < 0 || page >= p.pages.num_pages)
            report(p.status, DEV_BAD_PAGE);
          else
            off = page * p.pages.page_stride + row * p.pages.row_stride + iss.h * p.pages.head_stride;
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
        ++issued;
        if (issued < n) {
          advance(iss, pre, p.B, p.n_kv);
          page = page_of();
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
      const int from = SHARED ? begin[cur.b] : 0;
      const int left = last[cur.b] - (cur.j + from / KEYS) * KEYS;
      const int before = SHARED ? cur.j ? 0 : from % KEYS : 0;  // rows of the chunk that are shared
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float(&x)[4] = sc[nt];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += sd[nt][e];
        const bool sees0 = gr <= left && (!SHARED || gr >= before), sees1 = gr + 8 <= left && (!SHARED || gr + 8 >= before);
        x[0] = sees0 ? x[0] * p.scale_log2 : -INFINITY;
        x[1] = sees0 ? x[1] * p.scale_log2 : -INFINITY;
        x[2] = sees1 ? x[2] * p.scale_log2 : -INFINITY;
        x[3] = sees1 ? x[3] * p.scale_log2 : -INFINITY;
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
      if (SHARED) {
        const long long at = (here.b * p.n_kv + here.h + cta * W + warp) * static_cast<long long>(n_rep);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = nt * 8 + 2 * t + e;
            if (h >= n_rep) continue;
            float* row = p.own_o + (at + h) * HEAD_DIM;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              __stcg(row + 16 * d + gr, oacc[nt][d][e]);
              __stcg(row + 16 * d + gr + 8, oacc[nt][d][e + 2]);
            }
            if (gr == 0) __stcg(reinterpret_cast<float2*>(p.own_ml) + at + h, make_float2(m_run[nt][e], l_run[nt][e]));
          }
      } else if (seg.first >= a0 && seg.end <= a1) {
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
        if (lane == 0) sh.parts[2 * warp + slot] = seg;
      }
    }
  }
  if (SHARED) return;
  __syncthreads();
  join_parts(
      sh, reinterpret_cast<float*>(rings), split, cta, c0, c1, n_rep, p.part_o, p.part_ml, p.tickets,
      [&](int e) -> const float* {
        return (e & 1) ? reinterpret_cast<const float*>(rings + (e >> 1) * RING_BYTES) : stash + (e >> 1) * n_rep * PART;
      },
      [&](int row, float4 o, float m, float l) { store_row(p.out, row, o, 1.f / l); });
}

}  // namespace decode
}  // namespace gqa
