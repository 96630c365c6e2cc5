// Rows quantised as they are written into the history pages, with the keys rotated on the way
// where they are stored at absolute positions.
//
// HBM bound: an element is read (2 or 4 bytes) and its code written (1 or 1/2), both once.
// Threads share a head as in rope.cuh: d / 16 of them, two 8-column chunks each, so that a
// group's largest magnitude is a few warp shuffles and a rotation needs none.  12480 rows of 40
// heads, bf16 to e4m3 with the keys rotated, 387 MB, take 60 us (0.98 of the copy rate).
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "rope.cuh"

namespace hsa {
namespace {

// A CTA takes a few tokens' K or V and a slab of heads: thread (head, j, phase) owns two
// chunks of the tokens phase, phase + phases, ...  Its elements of the next two rounds are
// always on their way to a ring in shared memory that it alone reads (74 us with one round
// ahead in registers, 97 with K and V of a head in one thread and nothing ahead); the tokens'
// places and their cos and sin are computed while the first ones are.
constexpr int kRowsThreads = 320;
constexpr int kRowsCtas = 4;   // on an SM (48 registers: 29 of the 135 instances spill, up to 28 bytes)
constexpr int kRowsRing = 3;
constexpr int kRowsRounds = 8;
constexpr int kRowsMaxRows = 64;  // tokens of a CTA (32 KB of cos and sin at d = 128)

// The largest magnitude of 8 columns; NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float chunk_amax(const float* f) {
  const float m = max3_nan(fabsf(f[0]), fabsf(f[1]), fabsf(f[2]));
  const float n = max3_nan(fabsf(f[3]), fabsf(f[4]), fabsf(f[5]));
  return max3_nan(max_nan(fabsf(f[6]), fabsf(f[7])), m, n);
}

// Largest magnitudes of the groups that a thread's two chunks lie in.  The chunks are j and
// j + J, so a group is `per` neighbouring lanes of one half, or the whole head; in the partly
// rotated half layout (STRAIGHT false) the chunks' groups are matched one by one.
template <int J, int GROUP, int ROPE, bool STRAIGHT>
__device__ __forceinline__ void group_amax(const RopeArgs& r, const ChunkPair& c, int j, float& lo, float& hi) {
  constexpr int per = GROUP / 8;  // chunks of a group
  constexpr bool whole = per == 2 * J;
  if constexpr (whole) {
    lo = max_nan(lo, hi);
#pragma unroll
    for (int o = J / 2; o > 0; o >>= 1) lo = max_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = lo;
  } else if constexpr (STRAIGHT) {
#pragma unroll
    for (int o = per / 2; o > 0; o >>= 1) {
      lo = max_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  } else {
    const float own_lo = lo, own_hi = hi;
#pragma unroll
    for (int o = 1; o < J; ++o) {
      const float a = __shfl_xor_sync(0xffffffffu, own_lo, o), b = __shfl_xor_sync(0xffffffffu, own_hi, o);
      const ChunkPair q = chunk_pair<J, ROPE>(r, j ^ o);
      if (q.lo / per == c.lo / per) lo = max_nan(lo, a);
      if (q.hi / per == c.lo / per) lo = max_nan(lo, b);
      if (q.lo / per == c.hi / per) hi = max_nan(hi, a);
      if (q.hi / per == c.hi / per) hi = max_nan(hi, b);
    }
    if (c.lo / per == c.hi / per) {
      lo = max_nan(own_lo, lo);
      lo = hi = max_nan(lo, max_nan(own_hi, hi));
    }
  }
}

// What a group is multiplied with (0 where it is stored as zeros, or is not finite) and its scale (NaN where it is not
// finite).
template <int FMT>
__device__ __forceinline__ void group_scale(float amax, float& inv, float& scale) {
  const bool kept = amax >= kQuantTiny && amax < INFINITY;
  inv = kept ? __fmul_rn(__frcp_rn(amax), qmax_of<FMT>()) : 0.f;
  scale = kept ? __fmul_rn(amax, 1.f / qmax_of<FMT>()) : (amax < kQuantTiny ? 0.f : __uint_as_float(0x7fc00000u));
}

struct RowsLaunch {
  QuantArgs q;
  RopeArgs r;
  RowsArgs K, V;
  int tokens;
  void* const* page_k;
  void* const* page_v;
  int NP;
  long long first_row;
  const long long* first_row_dev;
  int* status;
  int rows_per_cta, slab, phases, ring_offset;
};

// Where a token's row goes: its codes and scales (NULL for nowhere).
struct RowPlace {
  char* codes;
  float* scales;
};

template <typename T, int FMT, int J, int GROUP, int ROPE>
__device__ __forceinline__ void write_rows(const RowsLaunch& w, const RowsArgs& x, void* const* __restrict__ pages,
                                           void* const* __restrict__ twins, RowPlace* place, float4* table) {
  constexpr int D = 16 * J, BITS = code_bits<FMT>(), per = GROUP / 8;
  const QuantArgs& q = w.q;
  const int tid = threadIdx.x, j = tid % J;
  const long long t0 = (long long)blockIdx.x * w.rows_per_cta;
  const int rows = (int)min((long long)w.rows_per_cta, w.tokens - t0);
  const int h0 = blockIdx.y * w.slab;
  const int phase = tid / (w.slab * J), h = h0 + (tid - phase * (w.slab * J)) / J;
  const bool active = phase < w.phases && h < q.H;
  const ChunkPair c = chunk_pair<J, ROPE>(w.r, j);
  const bool straight = ROPE != kRopeHalf || w.r.pairs == 8 * J;
  const T* src = static_cast<const T*>(x.data) + (t0 + phase) * x.token_stride + h * x.head_stride;
  const long long step = w.phases * x.token_stride;
  // A thread's own ring in shared memory (as the read's): its elements of the next
  // kRowsRing - 1 rounds are on their way while it works on one.
  constexpr int kVecs = sizeof(T) / 2;  // 16-byte vectors of a chunk
  const int threads = blockDim.x;
  char* ring = reinterpret_cast<char*>(table) + w.ring_offset + tid * 16;
  const uint32_t dst = smem_u32(ring);
  int ask_row = phase;
  auto ask = [&](int slot) {
    if (active && ask_row < rows) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        cp_async<16>(dst + ((slot * 2 * kVecs + k) * threads) * 16, src + c.lo * 8 + k * 4);
        cp_async<16>(dst + ((slot * 2 * kVecs + kVecs + k) * threads) * 16, src + c.hi * 8 + k * 4);
      }
    }
    ask_row += w.phases;
    src += step;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kRowsRing - 1; ++s) ask(s);
  const long long more = w.first_row_dev ? *w.first_row_dev : 0;
  for (int i = tid; i < rows; i += threads) {
    const long long g = more >= -kQuantMaxRow && more <= kQuantMaxRow ? w.first_row + more + t0 + i : -1;
    RowPlace p = {nullptr, nullptr};
    if (g >= 0 && g < (long long)w.NP * q.P_tok) {
      const long long page = g / q.P_tok;
      char* base = static_cast<char*>(pages[page]);
      const char* twin = static_cast<char*>(twins[page]);  // a row is written with its K and its V, or not at all
      if (base && twin && ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(twin)) & 15u) == 0) {
        p.codes = base + (g - page * q.P_tok) * q.H * (D * BITS / 8);
        p.scales = reinterpret_cast<float*>(base + q.scale_offset) + (g - page * q.P_tok) * q.H * (D / GROUP);
      }
    }
    if (!p.codes) set_status(w.status, HSA_ERR_DEVICE);
    place[i] = p;
  }
  if constexpr (ROPE != kRopeNone) rope_table<J, ROPE>(w.r, t0, rows, table, tid, blockDim.x);
  __syncthreads();
  const int code_lo = h * (D * BITS / 8) + c.lo * BITS, code_hi = h * (D * BITS / 8) + c.hi * BITS;
  const int scale_lo = h * (D / GROUP) + c.lo / per, scale_hi = h * (D / GROUP) + c.hi / per;
  const bool tell_lo = c.lo % per == 0, tell_hi = c.hi % per == 0;
  // the same number of rounds for every thread (warp shuffles)
  int slot = 0;
  for (int i0 = 0; i0 < rows; i0 += w.phases) {
    const int i = i0 + phase;
    ask(slot == 0 ? kRowsRing - 1 : slot - 1);
    cp_async_wait<kRowsRing - 1>();
    float a[8], b[8];
    const bool on = active && i < rows;
    Chunk<T> lo, hi;
    lo.load_split(ring + slot * 2 * kVecs * threads * 16, threads * 16);
    hi.load_split(ring + (slot * 2 * kVecs + kVecs) * threads * 16, threads * 16);
    lo.get(a);
    hi.get(b);
    if (ROPE != kRopeNone && on) rotate_chunks<J, ROPE>(c, table + i * 4 * J, j, a, b);
    float ma = chunk_amax(a), mb = chunk_amax(b);
    if (ROPE == kRopeHalf && !straight) group_amax<J, GROUP, ROPE, false>(w.r, c, j, ma, mb);
    else group_amax<J, GROUP, ROPE, true>(w.r, c, j, ma, mb);
    float inv, scale;
    group_scale<FMT>(ma, inv, scale);
    const RowPlace p = place[min(i, rows - 1)];
    if (on && p.codes) {
      store_codes<FMT>(p.codes + code_lo, encode8<FMT>(a, inv, ma < INFINITY));
      if (tell_lo) p.scales[scale_lo] = scale;
      if constexpr (GROUP != D) group_scale<FMT>(mb, inv, scale);
      store_codes<FMT>(p.codes + code_hi, encode8<FMT>(b, inv, mb < INFINITY));
      if (tell_hi) p.scales[scale_hi] = scale;
    }
    slot = slot == kRowsRing - 1 ? 0 : slot + 1;
  }
  cp_async_wait<0>();
}

template <typename T, int FMT, int J, int GROUP, int ROPE>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtas) quant_rows_kernel(const RowsLaunch w) {
  extern __shared__ float4 table[];
  __shared__ RowPlace place[kRowsMaxRows];
  if (blockIdx.z == 0) write_rows<T, FMT, J, GROUP, ROPE>(w, w.K, w.page_k, w.page_v, place, table);
  else write_rows<T, FMT, J, GROUP, kRopeNone>(w, w.V, w.page_v, w.page_k, place, table);
}

template <typename T, int FMT, int J, int GROUP, int ROPE>
cudaError_t launch_rows(RowsLaunch& w, cudaStream_t s) {
  const int H = w.q.H;
  int slabs = (H * J + kRowsThreads - 1) / kRowsThreads;
  w.slab = (H + slabs - 1) / slabs;
  slabs = (H + w.slab - 1) / w.slab;
  w.phases = kRowsThreads / (w.slab * J);
  if (w.phases > w.tokens) w.phases = w.tokens;
  if (w.phases > kRowsMaxRows) w.phases = kRowsMaxRows;
  // rounds of a CTA: up to kRowsRounds while that leaves eight CTAs to an SM
  int rounds = 1;
  while (rounds < kRowsRounds && w.phases * rounds * 2 <= kRowsMaxRows &&
         2LL * slabs * w.tokens >= 148LL * 8 * w.phases * rounds * 2)
    rounds *= 2;
  w.rows_per_cta = w.phases * rounds;
  const int need = (w.slab * J * w.phases + 31) / 32 * 32;
  const int threads = need > 8 * J ? need : 8 * J;  // 8 J: the cos and sin of a row
  size_t smem = ROPE != kRopeNone ? (size_t)w.rows_per_cta * 8 * J * sizeof(float2) : 0;
  w.ring_offset = (int)smem;
  smem += (size_t)kRowsRing * 16 * sizeof(T) * threads;
  if (smem > kDefaultSmemOptIn) {
    const cudaError_t e = cudaFuncSetAttribute(quant_rows_kernel<T, FMT, J, GROUP, ROPE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const unsigned ctas = (unsigned)(((long long)w.tokens + w.rows_per_cta - 1) / w.rows_per_cta);
  quant_rows_kernel<T, FMT, J, GROUP, ROPE><<<dim3(ctas, slabs, 2), threads, smem, s>>>(w);
  return cudaGetLastError();
}

template <typename T, int FMT, int J, int GROUP>
cudaError_t launch_rows_rope(RowsLaunch& a, cudaStream_t s) {
  if (!a.r.on) return launch_rows<T, FMT, J, GROUP, kRopeNone>(a, s);
  return a.r.half_layout ? launch_rows<T, FMT, J, GROUP, kRopeHalf>(a, s) : launch_rows<T, FMT, J, GROUP, kRopeInterleaved>(a, s);
}

template <typename T, int FMT>
cudaError_t launch_rows_group(RowsLaunch& a, cudaStream_t s) {
  if (a.q.d == 128) {
    if (a.q.group == 128) return launch_rows_rope<T, FMT, 8, 128>(a, s);
    if (a.q.group == 64) return launch_rows_rope<T, FMT, 8, 64>(a, s);
    return launch_rows_rope<T, FMT, 8, 32>(a, s);
  }
  return a.q.group == 64 ? launch_rows_rope<T, FMT, 4, 64>(a, s) : launch_rows_rope<T, FMT, 4, 32>(a, s);
}

template <typename T>
cudaError_t launch_rows_type(RowsLaunch& a, cudaStream_t s) {
  switch (a.q.format) {
    case HKV_QUANT_E4M3: return launch_rows_group<T, HKV_QUANT_E4M3>(a, s);
    case HKV_QUANT_INT8: return launch_rows_group<T, HKV_QUANT_INT8>(a, s);
    default: return launch_rows_group<T, HKV_QUANT_INT4>(a, s);
  }
}

}  // namespace

cudaError_t launch_quant_rows(const QuantArgs& q, const RopeArgs& r, const RowsArgs& K, const RowsArgs& V, int tokens,
                              int dtype, void* const* page_k, void* const* page_v, int NP, long long first_row,
                              const long long* first_row_dev, int* status, cudaStream_t s) {
  RowsLaunch a{q, r, K, V, tokens, page_k, page_v, NP, first_row, first_row_dev, status, 0, 0, 0, 0};
  switch (dtype) {
    case HSA_DTYPE_BF16: return launch_rows_type<__nv_bfloat16>(a, s);
    case HSA_DTYPE_FP16: return launch_rows_type<__half>(a, s);
    default: return launch_rows_type<float>(a, s);
  }
}

}  // namespace hsa
