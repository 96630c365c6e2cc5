// The quantised history pages: rows quantised as they are written (with the keys rotated
// on the way where they are stored at absolute positions), and the selected pages read
// back into the contiguous bf16 active cache (with the keys rotated to their places there,
// and their 128-row block means taken in the same pass).
//
// Both are HBM bound.  Threads share a head as in rope.cuh: d / 16 of them, two 8-column
// chunks each, so that a group's largest magnitude is a few warp shuffles and a rotation
// needs none.
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "rope.cuh"

namespace hsa {
namespace {

// ------------------------------------------------------------------ write
constexpr int kRowsThreads = 128;

__device__ __forceinline__ uint32_t chunk_amax(const float* f) {
  uint32_t m = 0;  // magnitudes compare as integers, infinities and NaN above all others
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// Largest magnitudes of the groups that a thread's two chunks lie in.  straight: the chunks
// are j and j + J, so a group is `group / 8` neighbouring lanes of one half, or the whole
// head; else (partly rotated half layout) the chunks' groups are matched one by one.
__device__ __forceinline__ void group_amax(bool straight, const RopeArgs& r, const ChunkPair& c, int j, int J, int group,
                                           uint32_t& lo, uint32_t& hi) {
  const int per = group / 8;  // chunks of a group
  if (straight) {
    const bool whole = per == 2 * J;
    if (whole) lo = hi = max(lo, hi);
    for (int o = (whole ? J : per) / 2; o > 0; o >>= 1) {
      lo = max(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    return;
  }
  const uint32_t own_lo = lo, own_hi = hi;
  for (int o = 1; o < J; ++o) {
    const uint32_t a = __shfl_xor_sync(0xffffffffu, own_lo, o), b = __shfl_xor_sync(0xffffffffu, own_hi, o);
    const ChunkPair q = chunk_pair(r, j ^ o, J);
    if (q.lo / per == c.lo / per) lo = max(lo, a);
    if (q.hi / per == c.lo / per) lo = max(lo, b);
    if (q.lo / per == c.hi / per) hi = max(hi, a);
    if (q.hi / per == c.hi / per) hi = max(hi, b);
  }
  if (c.lo / per == c.hi / per) lo = hi = max(lo, hi);
}

template <int FMT>
__device__ __forceinline__ void write_chunk(const QuantArgs& q, char* page, long long head_row, int chunk, const float* f,
                                            uint32_t amax) {
  const bool finite = amax < 0x7f800000u;
  const float a = __uint_as_float(amax);
  const bool kept = finite && a >= kQuantTiny;
  const float inv = kept ? __fmul_rn(__frcp_rn(a), qmax_of<FMT>()) : 0.f;
  store_codes<FMT>(page + (head_row * q.d + chunk * 8) * code_bits<FMT>() / 8, encode8<FMT>(f, inv, finite));
  if (chunk * 8 % q.group == 0) {
    const float scale = kept ? __fmul_rn(a, 1.f / qmax_of<FMT>()) : (finite ? 0.f : __uint_as_float(0x7fc00000u));
    reinterpret_cast<float*>(page + q.scale_offset)[head_row * (q.d / q.group) + chunk * 8 / q.group] = scale;
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kRowsThreads) quant_rows_kernel(const QuantArgs q, const RopeArgs r, const RowsArgs K,
                                                                  const RowsArgs V, long long tokens, int groups,
                                                                  void* const* __restrict__ page_k,
                                                                  void* const* __restrict__ page_v, int NP,
                                                                  long long first_row,
                                                                  const long long* __restrict__ first_row_dev,
                                                                  int* status) {
  const int J = q.d / 16;
  const long long item = (long long)blockIdx.x * kRowsThreads + threadIdx.x;
  const int j = (int)(item % J);
  const long long rest = item / J;
  const int g = (int)(rest % groups);
  const long long t = rest / groups;
  // every thread stays for the warp shuffles; one without a row (or a page) loads and stores nothing
  const bool inside = t < tokens;
  char *pk = nullptr, *pv = nullptr;
  long long row = 0;
  if (inside) {
    const long long more = first_row_dev ? *first_row_dev : 0;
    const long long at = more >= -kQuantMaxRow && more <= kQuantMaxRow ? first_row + t + more : -1;
    if (at >= 0 && at < (long long)NP * q.P_tok) {
      row = at % q.P_tok;
      pk = static_cast<char*>(page_k[at / q.P_tok]);
      pv = static_cast<char*>(page_v[at / q.P_tok]);
    }
    if (!pk || !pv || ((reinterpret_cast<uintptr_t>(pk) | reinterpret_cast<uintptr_t>(pv)) & 15u)) {
      pk = nullptr;
      set_status(status, HSA_ERR_DEVICE);
    }
  }
  const bool live = inside && pk;
  const ChunkPair c = chunk_pair(r, j, J);
  const bool straight = !(r.on && r.half_layout && r.pairs != q.d / 2);
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    cs[i] = live && (i < 4 ? c.rot_lo : c.rot_hi) ? rope_cos_sin(r, t, slot_pair(r, c, i)) : make_float2(1.f, 0.f);
  const T* src_k = static_cast<const T*>(K.data) + (live ? t : 0) * K.token_stride;
  const T* src_v = static_cast<const T*>(V.data) + (live ? t : 0) * V.token_stride;
  for (int h0 = 0; h0 < q.H; h0 += groups) {
    const int h = h0 + g;
    const bool on = live && h < q.H;
    Chunk<T> klo, khi, vlo, vhi;
    float a[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) {
      klo.load(src_k + h * K.head_stride + c.lo * 8);
      khi.load(src_k + h * K.head_stride + c.hi * 8);
      vlo.load(src_v + h * V.head_stride + c.lo * 8);
      vhi.load(src_v + h * V.head_stride + c.hi * 8);
      klo.get(a);
      khi.get(b);
      vlo.get(x);
      vhi.get(y);
      rotate_chunks(r, c, cs, a, b);
    }
    uint32_t ka = chunk_amax(a), kb = chunk_amax(b), va = chunk_amax(x), vb = chunk_amax(y);
    group_amax(straight, r, c, j, J, q.group, ka, kb);
    group_amax(straight, r, c, j, J, q.group, va, vb);
    if (on) {
      const long long head_row = row * q.H + h;
      write_chunk<FMT>(q, pk, head_row, c.lo, a, ka);
      write_chunk<FMT>(q, pk, head_row, c.hi, b, kb);
      write_chunk<FMT>(q, pv, head_row, c.lo, x, va);
      write_chunk<FMT>(q, pv, head_row, c.hi, y, vb);
    }
  }
}

template <typename T>
cudaError_t launch_rows(const QuantArgs& q, const RopeArgs& r, const RowsArgs& K, const RowsArgs& V, int tokens,
                        void* const* page_k, void* const* page_v, int NP, long long first_row,
                        const long long* first_row_dev, int* status, cudaStream_t s) {
  const int J = q.d / 16;
  const int groups = rope_head_groups(tokens, J, q.H);
  const long long items = (long long)tokens * groups * J;
  const unsigned blocks = (unsigned)((items + kRowsThreads - 1) / kRowsThreads);
  auto go = [&](auto kernel) {
    kernel<<<blocks, kRowsThreads, 0, s>>>(q, r, K, V, tokens, groups, page_k, page_v, NP, first_row, first_row_dev,
                                           status);
    return cudaGetLastError();
  };
  switch (q.format) {
    case HKV_QUANT_E4M3: return go(quant_rows_kernel<T, HKV_QUANT_E4M3>);
    case HKV_QUANT_INT8: return go(quant_rows_kernel<T, HKV_QUANT_INT8>);
    default: return go(quant_rows_kernel<T, HKV_QUANT_INT4>);
  }
}

// ------------------------------------------------------------------ read
// A CTA takes `rows_per_cta` rows of K or of V and a slab of heads: thread (item, phase)
// owns the two chunks `item` of every row phase, phase + phases, ...  The rows' cos and sin
// are computed once into shared memory (all heads of the slab use them), laid out so that
// the threads of a head read 16-byte vectors without bank conflicts.  The block means are
// summed a thread's rows first, then phase by phase in order (deterministic).
constexpr int kReadThreads = 512;
constexpr int kReadUnroll = 4;

template <int FMT>
__global__ void __launch_bounds__(kReadThreads) gather_quant_kernel(
    const QuantArgs q, const RopeArgs rope, const void* const* __restrict__ page_k, const void* const* __restrict__ page_v,
    int NP, const int32_t* __restrict__ sel, long long Lc, int rows_per_cta, int slab, int phases,
    uint16_t* __restrict__ Kc, uint16_t* __restrict__ Vc, float* __restrict__ kbar128, int* status) {
  extern __shared__ __align__(16) float smem[];
  const int J = q.d / 16;
  const long long nblk = (Lc + rows_per_cta - 1) / rows_per_cta;
  const long long blk = blockIdx.x % nblk;
  const bool is_v = blockIdx.x >= nblk;
  const long long r0 = blk * rows_per_cta;
  const int rows = (int)min((long long)rows_per_cta, Lc - r0);
  const int h0 = blockIdx.y * slab;
  const int heads = min(slab, q.H - h0);
  const int items = heads * J;
  const int tid = threadIdx.x;
  const int item = tid % (slab * J), phase = tid / (slab * J);
  const int j = item % J, h = h0 + item / J;
  RopeArgs r = rope;
  r.on = rope.on && !is_v;
  const ChunkPair c = chunk_pair(r, j, J);
  if (r.on) {
    for (int k = tid; k < rows * 8 * J; k += blockDim.x) {
      const int row = k / (8 * J), slot = k % (8 * J);
      const int jj = slot % J, i = slot / J;
      const ChunkPair cc = chunk_pair(r, jj, J);
      const float2 v = (i < 4 ? cc.rot_lo : cc.rot_hi) ? rope_cos_sin(r, r0 + row, slot_pair(r, cc, i)) : make_float2(1.f, 0.f);
      reinterpret_cast<float2*>(smem)[row * 8 * J + ((i >> 1) * J + jj) * 2 + (i & 1)] = v;
    }
    __syncthreads();
  }
  const void* const* table = is_v ? page_v : page_k;
  uint16_t* dst = is_v ? Vc : Kc;
  const bool pool = !is_v && kbar128 != nullptr;
  const bool active = phase < phases && item < items;
  const int G = q.d / q.group;
  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  if (active) {
    int slot = (int)((r0 + phase) / q.P_tok), known = -1;
    long long t = r0 + phase - (long long)slot * q.P_tok;
    const char* base = nullptr;
    for (int i0 = phase; i0 < rows; i0 += phases * kReadUnroll) {
      Codes8<FMT> lo[kReadUnroll], hi[kReadUnroll];
      float slo[kReadUnroll], shi[kReadUnroll];
      bool ok[kReadUnroll];
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        const int i = i0 + u * phases;
        ok[u] = false;
        if (i < rows) {
          while (t >= q.P_tok) {
            t -= q.P_tok;
            ++slot;
          }
          if (slot != known) {
            known = slot;
            const int p = sel[slot];
            base = (p >= 0 && p < NP) ? static_cast<const char*>(table[p]) : nullptr;
            if (base == nullptr || (reinterpret_cast<uintptr_t>(base) & 15u) != 0) {
              base = nullptr;
              set_status(status, HSA_ERR_DEVICE);
            }
          }
          if (base != nullptr) {
            ok[u] = true;
            const long long head_row = t * q.H + h;
            const char* codes = base + head_row * q.d * code_bits<FMT>() / 8;
            const float* scales = reinterpret_cast<const float*>(base + q.scale_offset) + head_row * G;
            lo[u] = load_codes<FMT>(codes + c.lo * code_bits<FMT>());
            hi[u] = load_codes<FMT>(codes + c.hi * code_bits<FMT>());
            slo[u] = __ldg(scales + c.lo * 8 / q.group);
            shi[u] = __ldg(scales + c.hi * 8 / q.group);
          }
          t += phases;
        }
      }
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        const int i = i0 + u * phases;
        if (ok[u]) {
          float a[8], b[8];
          decode8<FMT>(lo[u], slo[u], a);
          decode8<FMT>(hi[u], shi[u], b);
          if (r.on) {
            float2 cs[8];
            const float4* src = reinterpret_cast<const float4*>(smem) + (i * 4) * J + j;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 v = src[k * J];
              cs[2 * k] = make_float2(v.x, v.y);
              cs[2 * k + 1] = make_float2(v.z, v.w);
            }
            rotate_chunks(r, c, cs, a, b);
          }
          if (pool) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              acc[k] += a[k];
              acc[8 + k] += b[k];
            }
          }
          uint16_t* out = dst + ((r0 + i) * q.H + h) * q.d;
          Chunk<__nv_bfloat16> w;
          w.set(a);
          w.store(out + c.lo * 8);
          w.set(b);
          w.store(out + c.hi * 8);
        }
      }
    }
  }
  if (pool) {  // rows_per_cta is 128 here
    __syncthreads();  // the last cos and sin have been read
    for (int p = 0; p < phases; ++p) {
      if (active && phase == p) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float& s = smem[k * slab * J + item];
          s = p == 0 ? acc[k] : s + acc[k];
        }
      }
      __syncthreads();
    }
    if (active && phase == 0) {
      const float inv = 1.f / (float)rows;
      float* out = kbar128 + (blk * q.H + h) * q.d;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        out[c.lo * 8 + k] = smem[k * slab * J + item] * inv;
        out[c.hi * 8 + k] = smem[(8 + k) * slab * J + item] * inv;
      }
    }
  }
}

}  // namespace

cudaError_t launch_quant_rows(const QuantArgs& q, const RopeArgs& r, const RowsArgs& K, const RowsArgs& V, int tokens,
                              int dtype, void* const* page_k, void* const* page_v, int NP, long long first_row,
                              const long long* first_row_dev, int* status, cudaStream_t s) {
  switch (dtype) {
    case HSA_DTYPE_BF16:
      return launch_rows<__nv_bfloat16>(q, r, K, V, tokens, page_k, page_v, NP, first_row, first_row_dev, status, s);
    case HSA_DTYPE_FP16:
      return launch_rows<__half>(q, r, K, V, tokens, page_k, page_v, NP, first_row, first_row_dev, status, s);
    default:
      return launch_rows<float>(q, r, K, V, tokens, page_k, page_v, NP, first_row, first_row_dev, status, s);
  }
}

cudaError_t launch_gather_quant(const QuantArgs& q, const RopeArgs& r, const void* const* page_k,
                                const void* const* page_v, int NP, const int32_t* sel, int Kp, uint16_t* Kc,
                                uint16_t* Vc, float* kbar128, int* status, cudaStream_t s) {
  const long long Lc = (long long)Kp * q.P_tok;
  const int J = q.d / 16;
  const int slab = q.H < kReadThreads / J ? q.H : kReadThreads / J;
  const int slabs = (q.H + slab - 1) / slab;
  // The block means want 128 rows to a CTA; without them short caches are cut finer, until
  // there are two CTAs an SM.
  int rows = 128;
  while (!kbar128 && rows > 16 && 2 * ((Lc + rows - 1) / rows) * slabs < 2 * 148) rows /= 2;
  int phases = kReadThreads / (slab * J);
  if (phases > rows) phases = rows;
  const int threads = (slab * J * phases + 31) / 32 * 32;
  size_t smem = r.on ? (size_t)rows * 8 * J * sizeof(float2) : 0;
  const size_t pool = kbar128 ? (size_t)slab * J * 16 * sizeof(float) : 0;
  if (pool > smem) smem = pool;
  const long long nblk = (Lc + rows - 1) / rows;
  auto go = [&](auto kernel) {
    if (smem > kDefaultSmemOptIn) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<dim3((unsigned)(2 * nblk), slabs), threads, smem, s>>>(q, r, page_k, page_v, NP, sel, Lc, rows, slab, phases,
                                                                    Kc, Vc, kbar128, status);
    return cudaGetLastError();
  };
  switch (q.format) {
    case HKV_QUANT_E4M3: return go(gather_quant_kernel<HKV_QUANT_E4M3>);
    case HKV_QUANT_INT8: return go(gather_quant_kernel<HKV_QUANT_INT8>);
    default: return go(gather_quant_kernel<HKV_QUANT_INT4>);
  }
}

}  // namespace hsa
