// Rotary positions of queries and keys (forward, and backward with the angle's sign
// turned): y = mscale R(theta) x, one read and one write of every element.
//
// HBM bound: 2 x size bytes and 3 FLOP an element.  A CTA takes a few tokens with all their
// heads (queries, then keys).  Its threads first ask for their elements, then compute the
// tokens' cos and sin into shared memory while those are on the way.  One chunk pair a thread
// and six CTAs an SM (40 registers) measured best: 10800 tokens of 80 heads, 442 MB in bf16, in
// 72 us (0.94 of the copy rate), with four pairs a thread at two CTAs 92, with two at four 77; cos
// and sin computed by each thread for a share of the heads, without shared memory, 81.
#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace hsa {
namespace {

constexpr int kRopeThreads = 256;
// On an SM: that many threads' loads hide the latency, one unit each.  In the 40 registers that leaves, 8 of the 12
// instances spill (fp32 20 or 44 bytes, the interleaved layout in 16 bits 8 or 12).
constexpr int kRopeCtas = 6;
constexpr int kRopeRounds = 5;
constexpr int kRopeMaxRows = 32;  // tokens of a CTA (16 KB of cos and sin at d = 128)

template <typename T, int J, int ROPE>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeArgs r, int tokens, int rows_per_cta,
                                                                       int slab, const RowsArgs qi, const RowsArgs qo,
                                                                       const RowsArgs ki, const RowsArgs ko) {
  extern __shared__ float4 table[];
  const int tid = threadIdx.x, j = tid % J;
  const long long t0 = (long long)blockIdx.x * rows_per_cta;
  const int rows = (int)min((long long)rows_per_cta, tokens - t0);
  const int h0 = blockIdx.y * slab;
  const int heads = min(slab, qi.H + ki.H - h0);
  const ChunkPair c = chunk_pair<J, ROPE>(r, j);
  constexpr int kUnits = kRopeThreads / J;  // (token, head) units of a round, J threads each
  int row = tid / J / heads, head = tid / J % heads;
  bool first = true;
  while (first || row < rows) {
    Chunk<T> lo, hi;
    T* dst = nullptr;
    if (row < rows) {
      const int h = h0 + head;
      const bool is_q = h < qi.H;
      const RowsArgs& in = is_q ? qi : ki;
      const RowsArgs& out = is_q ? qo : ko;
      const int hh = is_q ? h : h - qi.H;
      const T* src = static_cast<const T*>(in.data) + (t0 + row) * in.token_stride + hh * in.head_stride;
      dst = static_cast<T*>(out.data) + (t0 + row) * out.token_stride + hh * out.head_stride;
      lo.load(src + c.lo * 8);
      hi.load(src + c.hi * 8);
    }
    if (first) {  // every thread comes here once
      rope_table<J, ROPE>(r, t0, rows, table, tid, kRopeThreads);
      __syncthreads();
      first = false;
    }
    if (row < rows) {
      if (c.rot_lo || c.rot_hi) {
        float a[8], b[8];
        lo.get(a);
        hi.get(b);
        rotate_chunks<J, ROPE>(c, table + row * 4 * J, j, a, b);
        if (c.rot_lo) lo.set(a);
        if (c.rot_hi) hi.set(b);
      }
      lo.store(dst + c.lo * 8);
      hi.store(dst + c.hi * 8);
    }
    for (head += kUnits; head >= heads; head -= heads) ++row;
  }
}

template <typename T, int J, int ROPE>
cudaError_t launch(const RopeArgs& r, int tokens, const RowsArgs& qi, const RowsArgs& qo, const RowsArgs& ki,
                   const RowsArgs& ko, cudaStream_t s) {
  const int heads = qi.H + ki.H;
  // Tokens of a CTA: where there are CTAs enough for every SM, of those that its threads get
  // through in kRopeRounds rounds the number that leaves the fewest of them idle in the last
  // one.  Its heads are shared out as well while that leaves SMs idle.  Whole waves of CTAs are not looked at: 4099 fp32
  // tokens of 15 heads of 64 make 1025 CTAs for 888 places (9.7 us, 4.8 for the bytes), 4680 tokens of 24 heads 1170
  // (10.7 us, 8.8 for the bytes).
  int rows = 1, best = 0;
  const int most = tokens / (148 * kRopeCtas);
  for (int n = 1; n == 1 || (n <= kRopeMaxRows && n <= most); ++n) {
    const int rounds = (n * heads + kRopeThreads / J - 1) / (kRopeThreads / J);
    const int used = n * heads * 100 / (rounds * (kRopeThreads / J));
    if (n > 1 && rounds > kRopeRounds) break;
    if (used > best) rows = n, best = used;
  }
  const long long ctas = ((long long)tokens + rows - 1) / rows;
  int slab = heads;
  while (slab > kRopeThreads / J && ctas * ((heads + slab - 1) / slab) < 148) slab = (slab + 1) / 2;
  rope_kernel<T, J, ROPE><<<dim3((unsigned)ctas, (heads + slab - 1) / slab), kRopeThreads,
                            (size_t)rows * 8 * J * sizeof(float2), s>>>(r, tokens, rows, slab, qi, qo, ki, ko);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeArgs& r, int tokens, int d, const RowsArgs& qi, const RowsArgs& qo, const RowsArgs& ki,
                        const RowsArgs& ko, cudaStream_t s) {
  if (d == 128)
    return r.half_layout ? launch<T, 8, kRopeHalf>(r, tokens, qi, qo, ki, ko, s)
                         : launch<T, 8, kRopeInterleaved>(r, tokens, qi, qo, ki, ko, s);
  return r.half_layout ? launch<T, 4, kRopeHalf>(r, tokens, qi, qo, ki, ko, s)
                       : launch<T, 4, kRopeInterleaved>(r, tokens, qi, qo, ki, ko, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& r, int tokens, int d, int dtype, const RowsArgs& qi, const RowsArgs& qo,
                        const RowsArgs& ki, const RowsArgs& ko, cudaStream_t s) {
  switch (dtype) {
    case HSA_DTYPE_BF16: return launch_type<__nv_bfloat16>(r, tokens, d, qi, qo, ki, ko, s);
    case HSA_DTYPE_FP16: return launch_type<__half>(r, tokens, d, qi, qo, ki, ko, s);
    default: return launch_type<float>(r, tokens, d, qi, qo, ki, ko, s);
  }
}

}  // namespace hsa
