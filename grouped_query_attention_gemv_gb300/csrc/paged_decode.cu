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
// Measured (GB300, 6.8 TB/s copied): 170.1 us for 1.108 GB (64 sequences of
// up to 8,192 rows), 86.6 for 537 MB (one of 131,072), 46.5 for 263 MB (16 of
// 1,001, 32 KV heads), 16.1 for 66 MB (8 KV heads), 3.4 for one sequence of
// 16 rows. Head-major pages ([page, KV head,
// row]) are 2 to 4% faster than [page, row, KV head]: longer runs per CTA.
#include "decode_stream.cuh"

namespace gqa {

namespace {

using namespace decode;

template <int NT>
__global__ void __launch_bounds__(WARPS * 32, 1) paged_decode_kernel(PagedDecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int n_rep = p.n_heads / p.n_kv;
  float* stash = reinterpret_cast<float*>(smem + WARPS * RING_BYTES);
  int* pre = reinterpret_cast<int*>(stash + WARPS * n_rep * PART);
  int* last = pre + p.B + 1;  // last row of each sequence
  __shared__ Shared sh;

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
  const int ctas = decode_ctas(total, gridDim.x, WARPS);
  const Split split(total, ctas);
  int c0, c1;
  if (!cta_range(total, count.longest, split, ctas, blockIdx.x, gridDim.x, pre, p.B, p.n_kv, c0, c1)) return;
  stream_chunks<NT, false>(p, sh, smem, stash, pre, last, nullptr, split, blockIdx.x, c0, c1);
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
  const size_t smem = static_cast<size_t>(WARPS) * (RING_BYTES + n_rep * PART * 4) + (2 * p.B + 1) * 4;
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
