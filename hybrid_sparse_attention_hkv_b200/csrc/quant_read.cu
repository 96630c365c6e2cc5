// Selected quantised pages read back into the contiguous bf16 active cache, with the keys
// rotated to their places there and their 128-row block means taken in the same pass.
//
// HBM bound, two thirds and more of it writes: 1 or 1/2 byte read and 2 written an element.
// What counts beside enough loads in flight is that the CTAs which run at one time write
// neighbouring memory: 16-row CTAs (a window of some 70 MB, all of it written from end to
// end) reach 99% of the copy rate without a rotation, where CTAs of 128 rows, each on a
// stretch of its own, stayed at 85%.  After that it is the instructions: with addresses that
// are a pointer and a constant, a rotated cache with its means takes 250 us instead of 272.
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "rope.cuh"

namespace hsa {
namespace {

// A CTA takes 16 rows of V, or of K, and a slab of heads: thread (item, phase) owns the two
// chunks `item` of every row phase, phase + phases, ...  With the block means it takes 128
// rows of K instead (a cluster of eight 16-row CTAs that added up their sums took 35%
// longer, and smaller slabs compute more cos and sin: 20 heads to a slab 7% longer than
// 40).  The cos and sin of 32 rows at a time are computed
// into shared memory (all heads of the slab use them).  The block means are summed a thread's
// rows first, then phase by phase in order (deterministic).
constexpr int kReadCtas = 3;  // on an SM (8 of the 36 instances spill, up to 16 bytes)
constexpr int kReadRing = 4;
constexpr int kReadThreads = 320;
constexpr int kReadRows = 16;   // of a CTA, or more:
constexpr int kReadRounds = 8;
constexpr int kReadBatch = 32;  // rows whose cos and sin are held at once

struct ReadArgs {
  QuantArgs q;
  RopeArgs r;
  const void* const* page_k;
  const void* const* page_v;
  int NP;
  const int32_t* sel;
  int Lc;
  struct Part {        // how K's, or V's, rows are shared out to CTAs
    int slab, slabs;   // heads of a CTA, and how many such slabs there are (the fastest index)
    int phases, rows;  // rows of a CTA, and those that it works on at once
    unsigned ctas;
  } k, v;
  int ring_offset;
  uint16_t* Kc;
  uint16_t* Vc;
  float* kbar128;
  int* status;
};

// A thread's way through its rows phase, phase + phases, ... of a CTA: where the codes of its
// chunk `lo` of the next one are, and their scale.
template <int FMT, int J>
struct ReadCursor {
  const char* codes;
  const float* scales;
  long long code_step, scale_step;
  int row;         // next row
  int left;        // rows from there to its page's end
  int phases;

  __device__ __forceinline__ void seek(const ReadArgs& a, const void* const* table, int r0, int h, const ChunkPair& c) {
    constexpr int D = 16 * J;
    const int slot = (unsigned)(r0 + row) / (unsigned)a.q.P_tok;
    const int t = r0 + row - slot * a.q.P_tok;
    left = a.q.P_tok - t;
    const int p = a.sel[slot];
    const char* base = (p >= 0 && p < a.NP) ? static_cast<const char*>(table[p]) : nullptr;
    codes = nullptr;
    if (base == nullptr || (reinterpret_cast<uintptr_t>(base) & 15u) != 0) {
      set_status(a.status, HSA_ERR_DEVICE);
    } else {
      const long long head_row = (long long)t * a.q.H + h;
      codes = base + head_row * (D * code_bits<FMT>() / 8) + c.lo * code_bits<FMT>();
      scales = reinterpret_cast<const float*>(base + a.q.scale_offset) + head_row * (D / a.q.group) + c.lo * 8 / a.q.group;
    }
  }
  // The step to the next row; false at the CTA's end.
  __device__ __forceinline__ bool next(const ReadArgs& a, const void* const* table, int r0, int h, const ChunkPair& c,
                                       int rows) {
    row += phases;
    if (row >= rows) return false;
    left -= phases;
    if (left > 0) {
      if (codes) {
        codes += code_step;
        scales += scale_step;
      }
    } else {
      seek(a, table, r0, h, c);
    }
    return true;
  }
};

// A thread's own ring in shared memory: its codes and scales of the next kReadRing - 1
// rounds are on their way while it works on one, at no cost in registers.  A slot is filled
// again one round after it was read.
template <int FMT>
struct ReadSlot {
  static constexpr int kCodeBytes = code_bits<FMT>();               // of 8 columns
  static constexpr int kHi = kReadThreads * kCodeBytes;             // lo chunks of all threads, their hi chunks,
  static constexpr int kScales = 2 * kHi;                           // ... the two scales
  static constexpr int kBytes = kScales + 8 * kReadThreads;
};

template <int FMT, int J, int ROPE, bool POOL>
__device__ __forceinline__ void read_rows(const ReadArgs& a, const ReadArgs::Part& part, unsigned cta,
                                          const void* const* table, uint16_t* dst, float* smem) {
  constexpr int D = 16 * J, BITS = code_bits<FMT>();
  const QuantArgs& q = a.q;
  const int blk = cta / (unsigned)part.slabs, r0 = blk * part.rows;
  const int rows = min(part.rows, a.Lc - r0);
  const int h0 = (int)(cta - blk * part.slabs) * part.slab;
  const int items = min(part.slab, q.H - h0) * J, phases = part.phases;
  const int tid = threadIdx.x;
  const int phase = tid / (part.slab * J), item = tid - phase * (part.slab * J);
  const int j = item % J, h = h0 + item / J;
  const bool active = phase < phases && item < items;
  const ChunkPair c = chunk_pair<J, ROPE>(a.r, j);
  const int next_group = c.hi * 8 / q.group - c.lo * 8 / q.group;  // from lo's scale to hi's
  const int next_chunk = (ROPE == kRopeHalf ? c.hi - c.lo : J) * BITS;
  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  ReadCursor<FMT, J> at;
  at.phases = phases;
  at.code_step = (long long)phases * q.H * (D * BITS / 8);
  at.scale_step = (long long)phases * q.H * (D / q.group);
  at.row = phase;
  bool more = active && phase < rows;
  if (more) at.seek(a, table, r0, h, c);
  // the ring lies behind the cos and sin
  using Slot = ReadSlot<FMT>;
  constexpr int CB = Slot::kCodeBytes;
  const int threads = blockDim.x;
  char* codes = reinterpret_cast<char*>(smem) + a.ring_offset + tid * CB;
  char* scales = reinterpret_cast<char*>(smem) + a.ring_offset + Slot::kScales + tid * 8;
  const uint32_t to_codes = smem_u32(codes), to_scales = smem_u32(scales);
  uint32_t there = 0;  // whether the rows asked for are, the last one in bit 0
  auto ask = [&](int slot) {  // slot: its offset in the ring
    there <<= 1;
    if (more) {
      if (at.codes) {
        there |= 1u;
        cp_async<CB>(to_codes + slot, at.codes);
        cp_async<CB>(to_codes + slot + Slot::kHi, at.codes + next_chunk);
        cp_async<4>(to_scales + slot, at.scales);
        if (next_group != 0) cp_async<4>(to_scales + slot + 4, at.scales + next_group);
      }
      more = at.next(a, table, r0, h, c, rows);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kReadRing - 1; ++s) ask(s * Slot::kBytes);
  uint16_t* out = dst + ((long long)(r0 + phase) * q.H + h) * D + c.lo * 8;
  const long long out_step = (long long)phases * q.H * D;
  const int out_hi = next_chunk / BITS * 8;
  int slot = 0, last = (kReadRing - 1) * Slot::kBytes, i = phase;
  for (int b0 = 0; b0 < rows; b0 += kReadBatch) {
    if constexpr (ROPE != kRopeNone) {
      if (b0) __syncthreads();  // the last rows' cos and sin have been read
      rope_table<J, ROPE>(a.r, r0 + b0, min(kReadBatch, rows - b0), reinterpret_cast<float4*>(smem), tid, threads);
      __syncthreads();
    }
    const float4* turn = reinterpret_cast<const float4*>(smem) + (i - b0) * 4 * J;
    const int end = active ? min(rows, b0 + kReadBatch) : 0;
    for (; i < end; i += phases) {
      ask(last);
      cp_async_wait<kReadRing - 1>();
      if (there >> (kReadRing - 1) & 1) {
        Codes8<FMT> lo, hi;
        if constexpr (FMT == HKV_QUANT_INT4) {
          lo.w[0] = *reinterpret_cast<const uint32_t*>(codes + slot);
          hi.w[0] = *reinterpret_cast<const uint32_t*>(codes + slot + Slot::kHi);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(codes + slot);
          const uint2 v = *reinterpret_cast<const uint2*>(codes + slot + Slot::kHi);
          lo.w[0] = u.x; lo.w[1] = u.y;
          hi.w[0] = v.x; hi.w[1] = v.y;
        }
        const float2 s = *reinterpret_cast<const float2*>(scales + slot);
        float x[8], y[8];
        decode8<FMT>(lo, s.x, x);
        decode8<FMT>(hi, next_group != 0 ? s.y : s.x, y);
        rotate_chunks<J, ROPE>(c, turn, j, x, y);
        if constexpr (POOL) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            acc[k] += x[k];
            acc[8 + k] += y[k];
          }
        }
        Chunk<__nv_bfloat16> w;
        w.set(x);
        w.store(out);
        w.set(y);
        w.store(out + out_hi);
      }
      out += out_step;
      turn += phases * 4 * J;
      last = slot;
      slot = slot == (kReadRing - 1) * Slot::kBytes ? 0 : slot + Slot::kBytes;
    }
  }
  cp_async_wait<0>();
  if constexpr (POOL) {
    __syncthreads();  // the last cos and sin have been read
#pragma unroll
    for (int k = 0; k < 16; ++k) smem[k * threads + tid] = acc[k];
    __syncthreads();
    const float inv = 1.f / (float)rows;
    float* mean = a.kbar128 + ((long long)blk * q.H + h0) * D;
    for (int v = tid; v < items * 16; v += threads) {
      const int k = v / items, it = v - k * items;
      const ChunkPair cc = chunk_pair<J, ROPE>(a.r, it % J);
      float sum = smem[k * threads + it];
      for (int p = 1; p < phases; ++p) sum += smem[k * threads + p * (part.slab * J) + it];
      mean[it / J * D + (k < 8 ? cc.lo * 8 + k : cc.hi * 8 + k - 8)] = sum * inv;
    }
  }
}

// (Both members of eight pairs and their sums at once are too much for 64 registers: with two
// CTAs an SM and no spills the half layout's block means take 265 us where three took 300.)
template <int FMT, int J, int ROPE, bool POOL>
__global__ void __launch_bounds__(kReadThreads, ROPE == kRopeHalf && POOL ? 2 : kReadCtas) gather_quant_kernel(const ReadArgs a) {
  extern __shared__ __align__(16) float smem[];
  if (blockIdx.x < a.k.ctas)
    read_rows<FMT, J, ROPE, POOL>(a, a.k, blockIdx.x, a.page_k, a.Kc, smem);
  else
    read_rows<FMT, J, kRopeNone, false>(a, a.v, blockIdx.x - a.k.ctas, a.page_v, a.Vc, smem);
}

// The shares of CTAs of 128 rows (for the block means), or of about 16, in eight rounds or more,
// fewer where a short cache leaves SMs idle.  Slabs are as wide as they can be, or narrower (and
// so more rows at once) where a short cache leaves SMs idle all the same.  Whole waves are not looked
// at: 4689 rows of 12 heads make 626 CTAs for 444 places, a second wave that is mostly empty, which is
// part of why they take 12 us where their bytes take 6.
template <int J>
ReadArgs::Part read_part(const ReadArgs& a, bool pool) {
  ReadArgs::Part p;
  p.slabs = (a.q.H * J + kReadThreads - 1) / kReadThreads;
  p.slab = (a.q.H + p.slabs - 1) / p.slabs;
  p.phases = kReadThreads / (p.slab * J);
  int rounds = p.phases < kReadRows / kReadRounds ? kReadRows / p.phases : kReadRounds;
  while (rounds > 1 && 1LL * a.Lc / (p.phases * rounds) * p.slabs < 2 * 148) --rounds;
  p.rows = pool ? 128 : p.phases * rounds;
  while (p.slabs < a.q.H && ((a.Lc - 1) / p.rows + 1LL) * p.slabs < 148) p.slabs = min(2 * p.slabs, a.q.H);
  p.slab = (a.q.H + p.slabs - 1) / p.slabs;
  p.slabs = (a.q.H + p.slab - 1) / p.slab;
  p.phases = kReadThreads / (p.slab * J);
  if (p.phases > p.rows) p.phases = p.rows;
  p.ctas = (unsigned)((a.Lc - 1) / p.rows + 1) * p.slabs;
  return p;
}

template <int FMT, int J, int ROPE, bool POOL>
cudaError_t launch_read(ReadArgs& a, cudaStream_t s) {
  a.k = read_part<J>(a, POOL);
  a.v = read_part<J>(a, false);
  const int need = max(a.k.slab * a.k.phases, a.v.slab * a.v.phases) * J;
  const int threads = max(8 * J, (need + 31) / 32 * 32);  // 8 J: the cos and sin of a row
  size_t smem = ROPE != kRopeNone ? (size_t)kReadBatch * 8 * J * sizeof(float2) : 0;
  if (POOL) smem = max(smem, (size_t)threads * 16 * sizeof(float));
  a.ring_offset = (int)smem;
  smem += (size_t)kReadRing * ReadSlot<FMT>::kBytes;
  if (smem > kDefaultSmemOptIn) {
    const cudaError_t e = cudaFuncSetAttribute(gather_quant_kernel<FMT, J, ROPE, POOL>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  gather_quant_kernel<FMT, J, ROPE, POOL><<<a.k.ctas + a.v.ctas, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int FMT, int J>
cudaError_t launch_read_rope(ReadArgs& a, cudaStream_t s) {
  if (!a.r.on) return a.kbar128 ? launch_read<FMT, J, kRopeNone, true>(a, s) : launch_read<FMT, J, kRopeNone, false>(a, s);
  if (a.r.half_layout)
    return a.kbar128 ? launch_read<FMT, J, kRopeHalf, true>(a, s) : launch_read<FMT, J, kRopeHalf, false>(a, s);
  return a.kbar128 ? launch_read<FMT, J, kRopeInterleaved, true>(a, s) : launch_read<FMT, J, kRopeInterleaved, false>(a, s);
}

template <int FMT>
cudaError_t launch_read_head(ReadArgs& a, cudaStream_t s) {
  return a.q.d == 128 ? launch_read_rope<FMT, 8>(a, s) : launch_read_rope<FMT, 4>(a, s);
}

}  // namespace

cudaError_t launch_gather_quant(const QuantArgs& q, const RopeArgs& r, const void* const* page_k,
                                const void* const* page_v, int NP, const int32_t* sel, int Kp, uint16_t* Kc,
                                uint16_t* Vc, float* kbar128, int* status, cudaStream_t s) {
  ReadArgs a{q, r, page_k, page_v, NP, sel, Kp * q.P_tok, {}, {}, 0, Kc, Vc, kbar128, status};
  switch (q.format) {
    case HKV_QUANT_E4M3: return launch_read_head<HKV_QUANT_E4M3>(a, s);
    case HKV_QUANT_INT8: return launch_read_head<HKV_QUANT_INT8>(a, s);
    default: return launch_read_head<HKV_QUANT_INT4>(a, s);
  }
}

}  // namespace hsa
