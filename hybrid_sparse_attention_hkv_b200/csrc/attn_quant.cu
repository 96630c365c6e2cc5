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
#ifndef AQ_S
#define AQ_S 3
#define AQ_C 3
#endif
constexpr int kAqStages = AQ_S;  // tiles of a warp's ring
constexpr int kAqCtas = AQ_C;    // on an SM
constexpr int kAqCtasWide = 2;   // ... with 16 queries to a tile

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

// N bytes of codes a thread reads at once, as words (N = 2: the low half of one).
template <int N>
struct Raw {
  uint32_t w[(N + 3) / 4];
};
template <int N>
__device__ __forceinline__ Raw<N> read_raw(const char* p) {
  Raw<N> r;
  if constexpr (N >= 16) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x; r.w[1] = v.y;
  } else if constexpr (N == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    static_assert(N == 2, "2, 4, 8 or a multiple of 16 bytes");
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
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

// A warp's ring of 16-key tiles in shared memory: codes of K and of V, rows padded by 16 bytes
// (the operand reads below are then free of bank conflicts at 128-byte rows), and scales.
template <int FMT, int D, int GROUP>
struct Stage {
  static constexpr int kRow = D * code_bits<FMT>() / 8, kPitch = kRow + 16;
  static constexpr int kScales = 16 * (D / GROUP) * 4;  // bytes of a tile's
  static constexpr int kV = 16 * kPitch, kKs = 2 * kV, kVs = kKs + kScales, kBytes = kVs + kScales;
};

template <int FMT, int D, int GROUP, int NT>
__global__ void __launch_bounds__(kAqThreads, NT == 1 ? kAqCtas : kAqCtasWide) attn_quant_kernel(const AttnQuantArgs a) {
  constexpr int G = D / GROUP;               // groups of a head
  constexpr int KS = GROUP / 16;             // product steps of a group (S), and 16-column tiles of a group (O)
  constexpr int BITS = code_bits<FMT>();
  constexpr int KB = GROUP / 4 * BITS / 8;   // bytes of a group a thread reads of a key row
  constexpr int VB = GROUP / 8 * BITS / 8;   // ... of a value row
  constexpr int COLS = 8 * NT;               // queries of a tile
  using St = Stage<FMT, D, GROUP>;
  extern __shared__ __align__(16) char ring_all[];
  __shared__ float s_m[kAqWarps][COLS], s_l[kAqWarps][COLS];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t = lane % 4;
  const int h = blockIdx.x % a.q.H, split = blockIdx.x / a.q.H;
  const int share = a.Hq / a.q.H;            // query heads of this key head
  const int cols = a.T * share, col0 = blockIdx.y * COLS;
  const int P = a.q.P_tok;

  // Tiles of the first n rows: tiles_page of each whole page, then those of the last one.
  const long long all = (long long)a.Kp * P;
  long long n_rows = a.n_rows ? (long long)*a.n_rows : all;
  n_rows = n_rows < 0 ? 0 : (n_rows > all ? all : n_rows);
  const int tiles_page = (P + 15) / 16;
  const int whole = (int)(n_rows / P), rest = (int)(n_rows - (long long)whole * P);
  const int tiles = whole * tiles_page + (rest + 15) / 16;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int tile_end = (int)min((long long)tiles, (long long)(split + 1) * per);

  // asking for tiles: this warp's are warp, warp + kAqWarps, ... of the split's
  char* ring = ring_all + warp * kAqStages * St::kBytes;
  const uint32_t ring_s = smem_u32(ring);
  constexpr int CH = St::kRow / 16;          // 16-byte vectors of a row
  constexpr int PER = 16 * CH / 32;          // ... of a tile that a lane copies
  const int my_row = lane / CH, my_vec = lane % CH;
  const long long row_step = (long long)a.q.H * St::kRow;
  long long tile_l = (long long)split * per + warp;
  int tile = tile_l < tile_end ? (int)tile_l : tile_end;
  int slot = tile / tiles_page, in_page = tile - slot * tiles_page, known = -1;
  const char *kbase = nullptr, *vbase = nullptr;
  unsigned long long valid_of = 0;  // rows of the tiles asked for, a byte each, the next to be worked on first
  int asked = 0;
  auto ask = [&](int stage) {
    int valid = 0;
    if (tile < tile_end) {
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
      if (kbase) {
        const int row0 = in_page * 16;
        valid = min((slot < whole ? P : rest) - row0, 16);
        const uint32_t dst = ring_s + stage * St::kBytes;
        const long long from = ((long long)row0 * a.q.H + h) * St::kRow + my_vec * 16;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int row = my_row + i * (32 / CH);
          const long long src = from + (row < valid ? row * row_step : 0);
          cp_async_zero<16>(dst + row * St::kPitch + my_vec * 16, kbase + src, row < valid);
          cp_async_zero<16>(dst + St::kV + row * St::kPitch + my_vec * 16, vbase + src, row < valid);
        }
        const int row = lane & 15;
        const long long head_row = (long long)(row0 + (row < valid ? row : 0)) * a.q.H + h;
        cp_async_zero<4 * G>(dst + (lane < 16 ? St::kKs : St::kVs) + row * 4 * G,
                             (lane < 16 ? kbase : vbase) + a.q.scale_offset + head_row * 4 * G, row < valid);
      }
      tile += kAqWarps;
      for (in_page += kAqWarps; in_page >= tiles_page; in_page -= tiles_page) ++slot;
    }
    cp_async_commit();
    valid_of |= (unsigned long long)valid << (8 * asked);
    ++asked;
  };
  const int rounds = tile < tile_end ? (tile_end - tile + kAqWarps - 1) / kAqWarps : 0;
#pragma unroll
  for (int s = 0; s < kAqStages - 1; ++s) ask(s);

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

  for (int i = 0, stage = 0; i < rounds; ++i, stage = stage == kAqStages - 1 ? 0 : stage + 1) {
    cp_async_wait<kAqStages - 2>();
    __syncwarp();  // all lanes' copies are there, and all are done with the stage before
    const int valid = (int)(valid_of & 255u);
    valid_of >>= 8;
    --asked;
    ask(stage == 0 ? kAqStages - 1 : stage - 1);
    if (valid == 0) continue;
    // keys g and g + 8; values 2t, 2t + 1, 2t + 8, 2t + 9
    const char* st = ring + stage * St::kBytes;
    Raw<KB> kw[2][G];
    Raw<VB> vw[4][G];
    float ks[2][G], vs[2][G];  // scales of rows g and g + 8
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        kw[r][k] = read_raw<KB>(st + (g + 8 * r) * St::kPitch + k * GROUP * BITS / 8 + t * KB);
        ks[r][k] = *reinterpret_cast<const float*>(st + St::kKs + ((g + 8 * r) * G + k) * 4);
        vs[r][k] = *reinterpret_cast<const float*>(st + St::kVs + ((g + 8 * r) * G + k) * 4);
      }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int k = 0; k < G; ++k)
        vw[r][k] = read_raw<VB>(st + St::kV + (2 * t + (r & 1) + 4 * (r & 2)) * St::kPitch + k * GROUP * BITS / 8 + g * VB);
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

  cp_async_wait<0>();
  float(*s_o)[D] = reinterpret_cast<float(*)[D]>(ring_all);  // after the barrier below the ring is free
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

template <int FMT, int D, int GROUP>
cudaError_t launch(const AttnQuantArgs& a, cudaStream_t s) {
  const int cols = a.T * (a.Hq / a.q.H);
  const unsigned x = (unsigned)(a.q.H * a.splits);
  const size_t ring = (size_t)kAqWarps * kAqStages * Stage<FMT, D, GROUP>::kBytes;
  auto go = [&](auto kernel, int nt) {
    const size_t join = (size_t)8 * nt * D * sizeof(float), smem = ring > join ? ring : join;
    if (smem > kDefaultSmemOptIn) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<dim3(x, (cols + 8 * nt - 1) / (8 * nt)), kAqThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
  cudaError_t e = cols <= 8 ? go(attn_quant_kernel<FMT, D, GROUP, 1>, 1) : go(attn_quant_kernel<FMT, D, GROUP, 2>, 2);
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

// Splits of the rows: about kAqCtas CTAs on each SM in one wave, at least 4 tiles (one a
// warp) to a split.
int attn_quant_splits(int T, int Hq, int H, int d, int Kp, int P_tok) {
  (void)d;
  const int cols = T * (Hq / H);
  const long long tiles = (long long)Kp * ((P_tok + 15) / 16);
  const long long units = (long long)H * (cols <= 8 ? 1 : (cols + 15) / 16);
  long long n = 148LL * (cols <= 8 ? kAqCtas : kAqCtasWide) / units;
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
