// Rotary positions of queries and keys (forward, and backward with the angle's sign
// turned): y = mscale R(theta) x, one read and one write of every element.
//
// HBM bound: 2 x size bytes and 3 FLOP an element.  A thread keeps the cos and sin of its
// eight pairs in registers and walks over a share of the token's heads (queries, then
// keys), so an angle is computed once per share and not once per head, and nothing is
// written to or read from a table.
#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace hsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;  // heads in flight a thread

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs r, long long tokens, int J, int groups,
                                                            const RowsArgs qi, const RowsArgs qo, const RowsArgs ki,
                                                            const RowsArgs ko) {
  const long long item = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int j = (int)(item % J);
  const long long rest = item / J;
  const int g = (int)(rest % groups);
  const long long t = rest / groups;
  if (t >= tokens) return;
  const ChunkPair c = chunk_pair(r, j, J);
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    cs[i] = (i < 4 ? c.rot_lo : c.rot_hi) ? rope_cos_sin(r, t, slot_pair(r, c, i)) : make_float2(1.f, 0.f);
  const int heads = qi.H + ki.H;
  const T* qsrc = static_cast<const T*>(qi.data) + t * qi.token_stride;
  const T* ksrc = static_cast<const T*>(ki.data) + t * ki.token_stride;
  T* qdst = static_cast<T*>(qo.data) + t * qo.token_stride;
  T* kdst = static_cast<T*>(ko.data) + t * ko.token_stride;
  for (int h0 = g; h0 < heads; h0 += groups * kRopeUnroll) {
    Chunk<T> lo[kRopeUnroll], hi[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * groups;
      if (h < heads) {
        const T* src = h < qi.H ? qsrc + h * qi.head_stride : ksrc + (h - qi.H) * ki.head_stride;
        lo[u].load(src + c.lo * 8);
        hi[u].load(src + c.hi * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * groups;
      if (h < heads) {
        T* dst = h < qi.H ? qdst + h * qo.head_stride : kdst + (h - qi.H) * ko.head_stride;
        if (c.rot_lo || c.rot_hi) {
          float a[8], b[8];
          lo[u].get(a);
          hi[u].get(b);
          rotate_chunks(r, c, cs, a, b);
          if (c.rot_lo) lo[u].set(a);
          if (c.rot_hi) hi[u].set(b);
        }
        lo[u].store(dst + c.lo * 8);
        hi[u].store(dst + c.hi * 8);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RopeArgs& r, int tokens, int d, const RowsArgs& qi, const RowsArgs& qo, const RowsArgs& ki,
                   const RowsArgs& ko, cudaStream_t s) {
  const int J = d / 16, heads = qi.H + ki.H;
  const int groups = rope_head_groups(tokens, J, heads);
  const long long items = (long long)tokens * groups * J;
  rope_kernel<T><<<(unsigned)((items + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0, s>>>(r, tokens, J, groups, qi,
                                                                                             qo, ki, ko);
  return cudaGetLastError();
}

}  // namespace

// Shares that a token's heads are cut into: as many as it takes to have about 2048 threads
// on each SM, at most one a head.  Fewer shares compute fewer angles, more shares keep more
// loads in flight.
int rope_head_groups(long long tokens, int J, int heads) {
  const long long want = (148LL * 2048 + tokens * J - 1) / (tokens * J);
  return (int)(want < 1 ? 1 : (want > heads ? heads : want));
}

cudaError_t launch_rope(const RopeArgs& r, int tokens, int d, int dtype, const RowsArgs& qi, const RowsArgs& qo,
                        const RowsArgs& ki, const RowsArgs& ko, cudaStream_t s) {
  switch (dtype) {
    case HSA_DTYPE_BF16: return launch<__nv_bfloat16>(r, tokens, d, qi, qo, ki, ko, s);
    case HSA_DTYPE_FP16: return launch<__half>(r, tokens, d, qi, qo, ki, ko, s);
    default: return launch<float>(r, tokens, d, qi, qo, ki, ko, s);
  }
}

}  // namespace hsa
