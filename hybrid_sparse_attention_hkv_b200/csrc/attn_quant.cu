// Attention of a few query tokens straight over quantised history pages.
//
// The codes are read once, as stored: 1 or 1/2 byte an element against the 5 bytes an
// element (1 read, 2 written, 2 read back) of assembling a bf16 cache first.  HBM bound, as
// long as turning codes into matrix operands stays cheap.
//
// Every code is exact as a half (fp16): e4m3 has 3 mantissa bits within half's exponents,
// the integers are below 2^7.  So the products run on mma.sync m16n8k16 with the codes as
// the 16-row operand (16 keys, or 16 columns of V) and the queries, up to 8 to a tile, as
// the 8-column one -- a query more costs nothing, where the instruction's other orientation
// would pad one query to 16.  (tcgen05 would want the decoded codes written back to shared
// memory first; at 1-16 queries the tensor rate is not what bounds.)  The scales are
// applied in fp32, outside the products:
//   S[key][query]  = (q . code) per group, x the key's scale, summed over the groups
//   O[col][query] += code x w,  w = p x the value scale of (key, the column's group)
// What enters a product in 16 bits beside the codes keeps fp32-like accuracy:
//   q    bf16 has 8 significant bits; scaled per query by a power of two to magnitudes
//        below 2 it is exact in fp16 down to 2^-24 of the query's largest element (less
//        is rounded at 2^-25 of it);
//   w    is split into two halves, w = hi + lo, with an error of 2^-22 of w, or 2^-25 of
//        the largest weight for small ones.  To stay within fp16's range, value scales
//        are taken relative to a running power of two per group (`vref`), which only rises;
//        the accumulators are rescaled when it does, as when the running maximum rises.
//
// Work: a warp takes 16-key tiles of one page and head; a CTA is 4 warps on one
// (split of the rows, head, query tile); the splits are joined by a second kernel in order
// (deterministic).  A tile never straddles pages; keys behind a page's or the cache's end
// are read from the tile's last valid row and get no weight.
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace hsa {
namespace {

constexpr int kAqWarps = 4;
constexpr int kAqThreads = kAqWarps * 32;

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {  // transpose of an 8x8 matrix of 16-bit elements
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t hsub2_u(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// N bytes of codes a thread loads at once, as words (N = 2: the low half of one).
template <int N>
struct Raw {
  uint32_t w[(N + 3) / 4];
};
template <int N>
__device__ __forceinline__ Raw<N> load_raw(const void* p) {
  Raw<N> r;
  if constexpr (N >= 16) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 v = ld_nc_v4(static_cast<const char*>(p) + 16 * i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 8) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p));
  } else if constexpr (N == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
  } else {
    static_assert(N == 2, "2, 4, 8 or a multiple of 16 bytes");
    uint16_t h;
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
    r.w[0] = h;
  }
  return r;
}

// Four codes of a thread's run starting at code 4 s (for 4 bits: codes 0, 4, 1, 5 of its
// eight when s is even, 2, 6, 3, 7 when odd) as two operand registers.
template <int FMT>
__device__ __forceinline__ void four_codes(const uint32_t* w, int s, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == HKV_QUANT_E4M3) {
    p0 = e4m3x2_to_half2(w[s]);
    p1 = e4m3x2_to_half2(w[s] >> 16);
  } else if constexpr (FMT == HKV_QUANT_INT8) {
    const uint32_t u = w[s] ^ 0x80808080u;
    p0 = hsub2_u(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);  // 1024 + u - 1152
    p1 = hsub2_u(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    const uint32_t u = (w[s >> 1] ^ 0x88888888u) >> (s & 1 ? 8 : 0);
    p0 = hsub2_u((u & 0x000f000fu) | 0x64006400u, 0x64086408u);  // 1024 + u - 1032
    p1 = hsub2_u(((u >> 4) & 0x000f000fu) | 0x64006400u, 0x64086408u);
  }
}
// Where code i (0..3) of step s sits in the thread's run of codes.
template <int FMT>
__device__ __forceinline__ constexpr int code_at(int s, int i) {
  if (FMT != HKV_QUANT_INT4) return 4 * s + i;
  return 8 * (s >> 1) + 2 * (s & 1) + (i >> 1) + 4 * (i & 1);
}

// Codes 2m and 2m + 1 of two keys' runs, a and b: (a's, b's) pairs.
template <int FMT>
__device__ __forceinline__ void two_keys(const uint32_t* a, const uint32_t* b, int m, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == HKV_QUANT_INT4) {
    const uint32_t u = __byte_perm(a[m >> 2], b[m >> 2], m & 2 ? 0x7632 : 0x5410) ^ 0x88888888u;
    const int sh = m & 1 ? 8 : 0;
    p0 = hsub2_u(((u >> sh) & 0x000f000fu) | 0x64006400u, 0x64086408u);
    p1 = hsub2_u(((u >> (sh + 4)) & 0x000f000fu) | 0x64006400u, 0x64086408u);
  } else {
    const uint32_t u = __byte_perm(a[m >> 1], b[m >> 1], m & 1 ? 0x7362 : 0x5140);  // a0 b0 a1 b1
    if constexpr (FMT == HKV_QUANT_E4M3) {
      p0 = e4m3x2_to_half2(u);
      p1 = e4m3x2_to_half2(u >> 16);
    } else {
      const uint32_t x = u ^ 0x80808080u;
      p0 = hsub2_u(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
      p1 = hsub2_u(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
    }
  }
}

__device__ __forceinline__ float pow2_below(float x) {  // the power of two at or below x, within [2^-126, 2^126]
  const uint32_t e = min(max(__float_as_uint(x) >> 23, 1u), 253u);
  return __uint_as_float(e << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

template <int FMT, int D, int GROUP, int NT>
__global__ void __launch_bounds__(kAqThreads) attn_quant_kernel(const AttnQuantArgs a) {
  constexpr int G = D / GROUP;               // groups of a head
  constexpr int KS = GROUP / 16;             // product steps of a group (S), and 16-column tiles of a group (O)
  constexpr int BITS = code_bits<FMT>();
  constexpr int KB = GROUP / 4 * BITS / 8;   // bytes of a group a thread loads of a key row
  constexpr int VB = GROUP / 8 * BITS / 8;   // ... of a value row
  constexpr int COLS = 8 * NT;               // queries of a tile
  __shared__ float s_o[COLS][D];
  __shared__ float s_m[kAqWarps][COLS], s_l[kAqWarps][COLS];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t = lane % 4;
  const int h = blockIdx.x % a.q.H, split = blockIdx.x / a.q.H;
  const int share = a.Hq / a.q.H;            // query heads of this key head
  const int cols = a.T * share, col0 = blockIdx.y * COLS;
  const int P = a.q.P_tok;

  // The queries of this tile as product operands: column g of each 8-query tile.
  uint32_t qf[NT][G * KS][2];
  float qs[NT][2];  // what S of columns 2t and 2t + 1 is multiplied with
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = col0 + n * 8 + g;
    const bool on = col < cols;
    const uint16_t* src = a.Q + ((long long)(on ? col / share : 0) * a.Hq + h * share + (on ? col % share : 0)) * D;
    float v[G * KS * 4];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < G * KS; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = (k / KS) * GROUP + t * (GROUP / 4) + code_at<FMT>(k % KS, i);
        const float x = on ? __uint_as_float((uint32_t)__ldg(src + d) << 16) : 0.f;
        v[4 * k + i] = x;
        top = fmaxf(top, fabsf(x));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float unit = pow2_below(top), inv = pow2_inverse(unit);
#pragma unroll
    for (int k = 0; k < G * KS; ++k) {
      qf[n][k][0] = pack_half2(v[4 * k] * inv, v[4 * k + 1] * inv);
      qf[n][k][1] = pack_half2(v[4 * k + 2] * inv, v[4 * k + 3] * inv);
    }
    qs[n][0] = __shfl_sync(0xffffffffu, unit, 8 * t) * a.scale_log2e;
    qs[n][1] = __shfl_sync(0xffffffffu, unit, 8 * t + 4) * a.scale_log2e;
  }

  // Tiles of the first n rows: tiles_per_page of each whole page, then those of the last one.
  const long long all = (long long)a.Kp * P;
  long long n_rows = a.n_rows ? (long long)*a.n_rows : all;
  n_rows = n_rows < 0 ? 0 : (n_rows > all ? all : n_rows);
  const int tiles_page = (P + 15) / 16;
  const long long tiles = n_rows / P * tiles_page + (n_rows % P + 15) / 16;
  const long long per = (tiles + a.splits - 1) / a.splits;
  const long long tile_end = min(tiles, (split + 1) * per);

  float o[NT][G * KS][4];
  float m[NT][2], l[NT][2];
  float vref[G];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int k = 0; k < G * KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < G; ++i) vref[i] = pow2_below(0.f);

  int known = -1;
  const char *kbase = nullptr, *vbase = nullptr;
  const long long row_bytes = (long long)D * BITS / 8;
  for (long long tile = split * per + warp; tile < tile_end; tile += kAqWarps) {
    const int slot = (int)(tile / tiles_page);
    const int row0 = (int)(tile - (long long)slot * tiles_page) * 16;
    if (slot != known) {
      known = slot;
      const int p = a.sel[slot];
      const bool in = p >= 0 && p < a.NP;
      kbase = in ? static_cast<const char*>(a.page_k[p]) : nullptr;
      vbase = in ? static_cast<const char*>(a.page_v[p]) : nullptr;
      if (!kbase || !vbase || ((reinterpret_cast<uintptr_t>(kbase) | reinterpret_cast<uintptr_t>(vbase)) & 15u)) {
        kbase = nullptr;
        set_status(a.status, HSA_ERR_DEVICE);
      }
    }
    if (!kbase) continue;
    const int valid = (int)min(min((long long)P, n_rows - (long long)slot * P) - row0, 16LL);  // >= 1
    // loads: keys g and g + 8; values 2t, 2t + 1, 2t + 8, 2t + 9
    Raw<KB> kw[2][G];
    Raw<VB> vw[4][G];
    float ks[2][G], vs[2][G];  // scales of rows g and g + 8
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long head_row = (long long)(row0 + min(g + 8 * i, valid - 1)) * a.q.H + h;
#pragma unroll
      for (int k = 0; k < G; ++k) {
        kw[i][k] = load_raw<KB>(kbase + head_row * row_bytes + (k * GROUP + t * (GROUP / 4)) * BITS / 8);
        ks[i][k] = __ldg(reinterpret_cast<const float*>(kbase + a.q.scale_offset) + head_row * G + k);
        vs[i][k] = __ldg(reinterpret_cast<const float*>(vbase + a.q.scale_offset) + head_row * G + k);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long head_row = (long long)(row0 + min(2 * t + (i & 1) + 4 * (i & 2), valid - 1)) * a.q.H + h;
#pragma unroll
      for (int k = 0; k < G; ++k)
        vw[i][k] = load_raw<VB>(vbase + head_row * row_bytes + (k * GROUP + g * (GROUP / 8)) * BITS / 8);
    }
    // S = K q
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      float part[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
#pragma unroll
      for (int st = 0; st < KS; ++st) {
        uint32_t f[4];
        four_codes<FMT>(kw[0][k].w, st, f[0], f[2]);
        four_codes<FMT>(kw[1][k].w, st, f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(part[n], f, qf[n][k * KS + st][0], qf[n][k * KS + st][1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][0] = fmaf(part[n][0], ks[0][k], s[n][0]);
        s[n][1] = fmaf(part[n][1], ks[0][k], s[n][1]);
        s[n][2] = fmaf(part[n][2], ks[1][k], s[n][2]);
        s[n][3] = fmaf(part[n][3], ks[1][k], s[n][3]);
      }
    }
    // softmax weights of this tile; p of rows g and g + 8, columns 2t and 2t + 1
    const bool in0 = g < valid, in1 = g + 8 < valid;
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = in0 ? s[n][e] * qs[n][e] : -INFINITY;
        float y = in1 ? s[n][2 + e] * qs[n][e] : -INFINITY;
        float top = fmaxf(x, y);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float next = fmaxf(m[n][e], top);
        const float ref = next == -INFINITY ? 0.f : next;
        alpha[n][e] = exp2f(m[n][e] - ref);
        moved |= next != m[n][e];
        m[n][e] = next;
        x = exp2f(x - ref);
        y = exp2f(y - ref);
        l[n][e] = l[n][e] * alpha[n][e] + (x + y);
        s[n][e] = x;
        s[n][2 + e] = y;
      }
    }
    // O += V w, group by group
    const bool rescale = __any_sync(0xffffffffu, moved);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const float v0 = in0 ? vs[0][k] : 0.f, v1 = in1 ? vs[1][k] : 0.f;
      float top = fmaxf(fabsf(v0), fabsf(v1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float next = fmaxf(vref[k], pow2_below(top));
      if (rescale || next != vref[k]) {
        const float beta = vref[k] * pow2_inverse(next);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][k * KS + mt][e] *= alpha[n][e & 1] * beta;
        vref[k] = next;
      }
      const float inv = pow2_inverse(next);
      const float r0 = v0 * inv, r1 = v1 * inv;
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float w0 = s[n][2 * i] * (i ? r1 : r0), w1 = s[n][2 * i + 1] * (i ? r1 : r0);
          const uint32_t hh = pack_half2(w0, w1);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hh));
          hi[n][i] = movmatrix(hh);
          lo[n][i] = movmatrix(pack_half2(w0 - back.x, w1 - back.y));
        }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        uint32_t f[4];
        two_keys<FMT>(vw[0][k].w, vw[1][k].w, mt, f[0], f[1]);
        two_keys<FMT>(vw[2][k].w, vw[3][k].w, mt, f[2], f[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(o[n][k * KS + mt], f, hi[n][0], hi[n][1]);
          mma16816(o[n][k * KS + mt], f, lo[n][0], lo[n][1]);
        }
      }
    }
  }

  // Join the warps in order.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[n][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (g == 0) {
        s_m[warp][n * 8 + 2 * t + e] = m[n][e];
        s_l[warp][n * 8 + 2 * t + e] = sum;
      }
    }
  __syncthreads();
  float share_of[NT][2];  // 2^(this warp's maximum - the CTA's)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = -INFINITY;
      for (int w = 0; w < kAqWarps; ++w) top = fmaxf(top, s_m[w][n * 8 + 2 * t + e]);
      share_of[n][e] = top == -INFINITY ? 0.f : exp2f(m[n][e] - top);
    }
  for (int w = 0; w < kAqWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < G * KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = (k / KS) * GROUP + g * (GROUP / 8) + 2 * (k % KS) + (e >> 1);
            float& dst = s_o[n * 8 + 2 * t + (e & 1)][d];
            // a warp without rows has nothing to add (its maximum is -inf)
            const float add = o[n][k][e] * vref[k / KS] * share_of[n][e & 1];
            dst = w == 0 ? add : dst + add;
          }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < COLS * D; i += kAqThreads) {
    const int c = i / D, d = i % D, col = col0 + c;
    if (col >= cols) break;
    float top = -INFINITY;
    for (int w = 0; w < kAqWarps; ++w) top = fmaxf(top, s_m[w][c]);
    float sum = 0.f;
    for (int w = 0; w < kAqWarps; ++w) sum += top == -INFINITY ? s_l[w][c] : s_l[w][c] * exp2f(s_m[w][c] - top);
    const float v = s_o[c][d];
    const long long row = (long long)(col / share) * a.Hq + h * share + col % share;
    if (a.splits > 1) {
      const long long at = (long long)split * a.T * a.Hq + row;
      a.part_o[at * D + d] = v;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
    } else {
      const float r = sum == 0.f ? 0.f : v / sum;
      if (a.out_f32) a.out_f32[row * D + d] = r;
      else a.out_bf16[row * D + d] = (uint16_t)pack_bf16x2(r, 0.f);
      if (d == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * 0.69314718055994531f + logf(sum);
    }
  }
}

// out = sum over the splits of 2^(m_i - m) O_i / sum of 2^(m_i - m) l_i, in split order.
__global__ void attn_quant_join_kernel(const AttnQuantArgs a, int D) {
  const long long rows = (long long)a.T * a.Hq;
  const long long row = (long long)blockIdx.x * (blockDim.x / D) + threadIdx.x / D;
  const int d = threadIdx.x % D;
  if (row >= rows) return;
  float top = -INFINITY;
  for (int i = 0; i < a.splits; ++i) top = fmaxf(top, a.part_ml[i * rows + row].x);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, v = 0.f;
  for (int i = 0; i < a.splits; ++i) {
    const float2 ml = a.part_ml[i * rows + row];
    const float w = exp2f(ml.x - ref);
    // a NaN score leaves the maximum as it was: its sum counts whatever the maximum says
    sum += ml.x == -INFINITY ? ml.y : ml.y * w;
    v += a.part_o[(i * rows + row) * D + d] * w;
  }
  const float r = sum == 0.f ? 0.f : v / sum;
  if (a.out_f32) a.out_f32[row * D + d] = r;
  else a.out_bf16[row * D + d] = (uint16_t)pack_bf16x2(r, 0.f);
  if (d == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : ref * 0.69314718055994531f + logf(sum);
}

constexpr int kAqCtasPerSM = 4;

template <int FMT, int D, int GROUP>
cudaError_t launch(const AttnQuantArgs& a, cudaStream_t s) {
  const int cols = a.T * (a.Hq / a.q.H);
  const unsigned x = (unsigned)(a.q.H * a.splits);
  if (cols <= 8) attn_quant_kernel<FMT, D, GROUP, 1><<<dim3(x, 1), kAqThreads, 0, s>>>(a);
  else attn_quant_kernel<FMT, D, GROUP, 2><<<dim3(x, (cols + 15) / 16), kAqThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  const int per = 256 / D;
  const long long rows = (long long)a.T * a.Hq;
  attn_quant_join_kernel<<<(unsigned)((rows + per - 1) / per), 256, 0, s>>>(a, D);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_fmt(const AttnQuantArgs& a, cudaStream_t s) {
  if (a.q.d == 128) {
    if (a.q.group == 128) return launch<FMT, 128, 128>(a, s);
    if (a.q.group == 64) return launch<FMT, 128, 64>(a, s);
    return launch<FMT, 128, 32>(a, s);
  }
  if (a.q.group == 64) return launch<FMT, 64, 64>(a, s);
  return launch<FMT, 64, 32>(a, s);
}

}  // namespace

// Splits of the rows: about kAqCtasPerSM CTAs on each SM in one wave, at least 4 tiles (one a
// warp) to a split.
int attn_quant_splits(int T, int Hq, int H, int d, int Kp, int P_tok) {
  (void)d;
  const int cols = T * (Hq / H);
  const long long tiles = (long long)Kp * ((P_tok + 15) / 16);
  const long long units = (long long)H * (cols <= 8 ? 1 : (cols + 15) / 16);
  long long n = 148LL * kAqCtasPerSM / units;
  const long long most = (tiles + kAqWarps - 1) / kAqWarps;
  if (n > most) n = most;
  return (int)(n < 1 ? 1 : n);
}

cudaError_t launch_attn_quant(const AttnQuantArgs& a, cudaStream_t s) {
  switch (a.q.format) {
    case HKV_QUANT_E4M3: return launch_fmt<HKV_QUANT_E4M3>(a, s);
    case HKV_QUANT_INT8: return launch_fmt<HKV_QUANT_INT8>(a, s);
    default: return launch_fmt<HKV_QUANT_INT4>(a, s);
  }
}

}  // namespace hsa
