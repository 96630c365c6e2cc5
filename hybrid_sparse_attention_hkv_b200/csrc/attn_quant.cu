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
//   w    enters as two halves: what a half holds of it, and what that leaves, 2^12 times as
//        large, in a product of its own.  For each 32 keys, query and group, w is scaled by the
//        power of two that brings the largest to [2^14, 2^15): every w down to 2^-28 of it enters
//        with an error below 2^-23 of its own, smaller ones with one below 2^-51 of the largest.
//        A large value scale on a key with little weight, or a key with all the weight and a
//        value of zero, costs the others nothing.
// The products of 16 or 32 keys go to accumulators of their own and are added to O by fp32 FMAs:
// the tensor core's adder cuts off what a long sum does not hold (one token over 49920 rows: off by
// 2e-7 of the output; 8e-7 with one accumulator for all rows).
// Weights in three parts of bf16, which need no scaling, measured 39 us for one token over 49920
// rows of 12 heads against 37 (codes cost three times as much to turn into bf16), without the
// FMAs.  One running power of two for a group's value scales took 36, but left small weights
// beside a large scale, or behind a large weight, without their bits.
//
// Work: a CTA takes tiles of a split of the rows, four warps with 32 keys of a head each: of
// four neighbouring heads where there are so many, so that a row's codes are fetched in runs of
// 256 to 512 bytes and its scales in 16-byte vectors (with a head to a CTA the scales, 4 bytes
// from each 32-byte sector, were half of all requests: 124 us instead of 96 for one token over
// 49920 rows of 40 heads).  Tiles are on their way to a ring in shared memory while one is
// worked on; small CTAs, three to an SM, drift apart and keep the loads going where one of 8 or
// 12 warps stops at its barrier (before the weights took their present form 329 us for 199680 rows
// of 40 heads against 395 to 425; 334 with it, 0.96 of the copy rate).  The splits are joined by a
// second kernel in order (deterministic).  A tile never straddles pages; what lies behind a page's
// or the cache's end is fetched as zeros and gets no weight.
//
// Short caches are bound by their latency: two launches, the way from the row count to the page
// table to the rows, and the join cost 9 us together.  4-bit codes, and groups of 32 columns, are
// bound by instructions: turning codes into operands, and scaling and splitting the weights for each
// group (49920 rows of 12 heads of 128 columns in 8 bits, 4 bits, 8 bits in groups of 32: 37, 36 and 50 us).
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace hsa {
namespace {

constexpr int kAqWarps = 4;
constexpr int kAqThreads = kAqWarps * 32;
constexpr int kAqRows = 32;    // keys of a warp's unit
constexpr int kAqStages = 2;   // tiles of the ring
constexpr int kAqMostCtas = 4;

// CTAs on an SM, with up to 8 (NT = 1) or 16 queries to a tile: as many as registers and the ring allow (56 of the 90
// instances spill, up to 80 bytes).
template <int FMT, int D, int GROUP, int NT>
constexpr int ctas_per_sm() {
  if (NT == 2) return D == 64 ? 3 : 2;
  if (D == 64) return 4;
  return code_bits<FMT>() == 8 && GROUP == 32 ? 2 : 3;
}

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

// Integers become halves through the mantissa of 1024, a published conversion (Kim, Henry, Fahim and Awadalla, "Who Says
// Elephants Can't Run", 2022, for unsigned ones), which costs a mask or a byte permute and a subtraction for two.
// The low two nibbles of each half of w as halves: p0 the lowest of both, p1 the next.  Flipping
// a nibble's sign bit gives n + 8, which becomes the low bits of 1024 + (n + 8), or, left where
// it is, of 1024 + 16 (n + 8).
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t& p0, uint32_t& p1) {
  p0 = hsub2_u((w & 0x000f000fu) ^ 0x64086408u, 0x64086408u);  // - 1032
  const uint32_t x = (w & 0x00f000f0u) ^ 0x64806480u, sixteenth = 0x2c002c00u, minus72 = 0xd480d480u;
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&sixteenth),
                            *reinterpret_cast<const __half2*>(&minus72));
  p1 = *reinterpret_cast<const uint32_t*>(&y);
}

// The upper halves, or the lower ones, of two words: a's below b's.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ uint32_t lower_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }

// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 w, x, y, z;\n\tmov.b64 w, {%2, %3};\n\tmov.b64 x, {%4, %5};\n\tmov.b64 y, {%6, %7};\n\t"
      "fma.rn.f32x2 z, w, x, y;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

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

// Neighbouring heads of a CTA: their codes and scales of a row are fetched in one piece.
inline int attn_quant_heads(int H) { return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1; }

// Splits of the rows: one wave of CTAs, at least a tile to each.
inline int attn_quant_splits_of(int ctas_per_sm, int T, int Hq, int H, int Kp, int P_tok) {
  const int cols = T * (Hq / H), heads = attn_quant_heads(H), tile = kAqRows * kAqWarps / heads;
  const long long tiles = (long long)Kp * ((P_tok - 1) / tile + 1);
  const long long units = (long long)(H / heads) * (cols <= 8 ? 1 : (cols + 15) / 16);
  long long n = 148LL * ctas_per_sm / units;
  if (n > tiles) n = tiles;
  return (int)(n < 1 ? 1 : n);
}

// Four codes of a thread's run starting at code 4 s (for 4 bits: codes 0, 4, 1, 5 of its
// eight when s is even, 2, 6, 3, 7 when odd) as two operand registers.
template <int FMT>
__device__ __forceinline__ void four_codes(const uint32_t* w, int s, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == HKV_QUANT_E4M3) {
    e4m3x4_to_half2(w[s], p0, p1);
  } else if constexpr (FMT == HKV_QUANT_INT8) {
    const uint32_t u = w[s] ^ 0x80808080u;
    p0 = hsub2_u(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);  // 1024 + u - 1152
    p1 = hsub2_u(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    nibbles(w[s >> 1] >> (s & 1 ? 8 : 0), p0, p1);
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
    nibbles(__byte_perm(a[m >> 1 >> 1], b[m >> 1 >> 1], m & 2 ? 0x7632 : 0x5410) >> (m & 1 ? 8 : 0), p0, p1);
  } else {
    const uint32_t u = __byte_perm(a[m >> 1], b[m >> 1], m & 1 ? 0x7362 : 0x5140);  // a0 b0 a1 b1
    if constexpr (FMT == HKV_QUANT_E4M3) {
      e4m3x4_to_half2(u, p0, p1);
    } else {
      const uint32_t x = u ^ 0x80808080u;
      p0 = hsub2_u(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
      p1 = hsub2_u(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
    }
  }
}

// 2^x within 2 ulp; results below 2^-126 are zero.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float pow2_below(float x) {  // the power of two at or below x, within [2^-126, 2^126]
  const uint32_t e = min(max(__float_as_uint(x) >> 23, 1u), 253u);
  return __uint_as_float(e << 23);
}
// The power of two that brings weights of at most x to below 2^15: within [2^-126, 2^114].
__device__ __forceinline__ float weight_unit(float x) {
  return __uint_as_float((uint32_t)max((int)(__float_as_uint(x) >> 23) - 14, 1) << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// The CTA's ring of tiles in shared memory.  A tile is some rows of a few neighbouring heads,
// cut into a unit of kAqRows rows of one head for each warp: codes of K and of V, rows padded
// by 16 bytes (the operand reads below are then free of bank conflicts at 128-byte rows), and
// behind the units the rows' scales, as they lie in the page.
template <int FMT, int D, int GROUP>
struct Stage {
  static constexpr int kRow = D * code_bits<FMT>() / 8, kPitch = kRow + 16;
  static constexpr int kV = kAqRows * kPitch, kUnit = 2 * kV;
  static constexpr int kScales = kAqWarps * kAqRows * (D / GROUP) * 4;  // bytes of K's, or V's, scales of a tile
  static constexpr int kKs = kAqWarps * kUnit, kVs = kKs + kScales, kBytes = kVs + kScales;
};

// Column d of a row: v / sum, the weights taken relative to 2^top (-inf: to 1).
__device__ __forceinline__ void write_out(const AttnQuantArgs& a, long long row, int D, int d, float v, float top,
                                          float sum) {
  const float r = sum == 0.f ? 0.f : v / sum;
  if (a.out_f32) a.out_f32[row * D + d] = r;
  else a.out_bf16[row * D + d] = (uint16_t)pack_bf16x2(r, 0.f);
  if (d == 0 && a.lse)
    a.lse[row] = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * 0.69314718055994531f + logf(sum);
}

template <int FMT, int D, int GROUP, int NT, int HEADS>
__global__ void __launch_bounds__(kAqThreads, (ctas_per_sm<FMT, D, GROUP, NT>())) attn_quant_kernel(const AttnQuantArgs a) {
  constexpr int G = D / GROUP;               // groups of a head
  constexpr int KS = GROUP / 16;             // product steps of a group (S), and 16-column tiles of a group (O)
  constexpr int BITS = code_bits<FMT>();
  constexpr int KB = GROUP / 4 * BITS / 8;   // bytes of a group a thread reads of a key row
  constexpr int VB = GROUP / 8 * BITS / 8;   // ... of a value row
  constexpr int COLS = 8 * NT;               // queries of a tile
  using St = Stage<FMT, D, GROUP>;
  constexpr int M = kAqRows / 16;              // 16-key products of a unit
  extern __shared__ __align__(16) char ring[];
  __shared__ float s_m[kAqWarps][COLS], s_l[kAqWarps][COLS];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, t = lane % 4;
  // the CTA's warps: HEADS neighbouring heads, kAqWarps / HEADS units of rows of each
  const int split = blockIdx.x / (a.q.H / HEADS), h0 = (blockIdx.x - split * (a.q.H / HEADS)) * HEADS;
  const int own_head = warp % HEADS, own_rows = warp / HEADS * kAqRows, h = h0 + own_head;
  const int share = a.Hq / a.q.H;            // query heads of a key head
  const int cols = a.T * share, col0 = blockIdx.y * COLS;
  const int P = a.q.P_tok;

  // Tiles of the first n rows: tiles_page of each whole page, then those of the last one.
  constexpr int TILE = kAqRows * kAqWarps / HEADS;
  const long long all = (long long)a.Kp * P;
  long long n_rows = a.n_rows ? (long long)*a.n_rows : all;
  n_rows = n_rows < 0 ? 0 : (n_rows > all ? all : n_rows);
  const int tiles_page = (P - 1) / TILE + 1;
  const int whole = (int)(n_rows / P), rest = (int)(n_rows - (long long)whole * P);
  const int tiles = whole * tiles_page + rest / TILE + (rest % TILE != 0);
  const int per = tiles / a.splits + (tiles % a.splits != 0);
  const int first = (int)min((long long)tiles, (long long)split * per), rounds = min(per, tiles - first);

  // asking for tiles: a row's codes are HEADS * kRow bytes next to each other, its scales
  // HEADS * G floats
  const uint32_t ring_s = smem_u32(ring);
  constexpr int CH = HEADS * St::kRow / 16;          // 16-byte vectors of a row
  constexpr int ROWS_AT_ONCE = kAqThreads / CH;      // rows that the CTA copies at once
  constexpr int PER = TILE / ROWS_AT_ONCE;
  const int my_row = tid / CH, my_vec = tid % CH;
  const int my_head = my_vec / (CH / HEADS), my_col = my_vec % (CH / HEADS) * 16;
  // where a row's vector goes in a tile: my_row's place, and from there each ROWS_AT_ONCE-th row's
  const int my_place = (my_row / kAqRows * HEADS + my_head) * St::kUnit + my_row % kAqRows * St::kPitch + my_col;
  auto place_of = [](int i) {
    return i * ROWS_AT_ONCE / kAqRows * HEADS * St::kUnit + i * ROWS_AT_ONCE % kAqRows * St::kPitch;
  };
  static_assert(kAqRows % ROWS_AT_ONCE == 0 || ROWS_AT_ONCE % kAqRows == 0, "rows keep their unit");
  constexpr int SF = HEADS * G;                      // scales of a row
  const long long row_step = (long long)a.q.H * St::kRow, scale_step = (long long)a.q.H * 4 * G;
  // ... in 16-byte vectors where they come in fours (H is a multiple of HEADS, so every row of them is aligned then)
  constexpr int PIECE = SF % 4 == 0 ? 4 : 1, PIECES = SF / PIECE;
  int asked_tile = 0, slot = first / tiles_page, in_page = first - slot * tiles_page, known = -1;
  const char *kbase = nullptr, *vbase = nullptr;
  unsigned long long valid_of = 0;  // rows of the tiles asked for, 16 bits each, the next to be worked on first
  int asked = 0;
  auto ask = [&](int stage) {
    int valid = 0;
    if (asked_tile < rounds) {
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
        const int row0 = in_page * TILE;
        valid = min((slot < whole ? P : rest) - row0, TILE);
        const uint32_t dst = ring_s + stage * St::kBytes, to = dst + my_place;
        const long long from = ((long long)row0 + my_row) * row_step + h0 * St::kRow + my_vec * 16;
        const char *k = kbase + from, *v = vbase + from;
        if (valid == TILE) {
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            cp_async<16>(to + place_of(i), k);
            cp_async<16>(to + place_of(i) + St::kV, v);
            k += ROWS_AT_ONCE * row_step;
            v += ROWS_AT_ONCE * row_step;
          }
        } else {  // zeros behind the last row
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const bool on = my_row + i * ROWS_AT_ONCE < valid;
            cp_async_zero<16>(to + place_of(i), on ? k : kbase, on);
            cp_async_zero<16>(to + place_of(i) + St::kV, on ? v : vbase, on);
            k += ROWS_AT_ONCE * row_step;
            v += ROWS_AT_ONCE * row_step;
          }
        }
#pragma unroll
        for (int i0 = 0; i0 < TILE * PIECES; i0 += kAqThreads) {
          const int i = i0 + tid, row = i / PIECES, at = i % PIECES * PIECE;
          if (i < TILE * PIECES) {
            const bool on = row < valid;
            const long long src = a.q.scale_offset + (on ? (row0 + row) * scale_step + (h0 * G + at) * 4 : 0);
            const uint32_t to = dst + St::kKs + (row * SF + at) * 4;
            cp_async_zero<4 * PIECE>(to, kbase + src, on);
            cp_async_zero<4 * PIECE>(to + St::kScales, vbase + src, on);
          }
        }
      }
      ++asked_tile;
      if (++in_page == tiles_page) {
        in_page = 0;
        ++slot;
      }
    }
    cp_async_commit();
    valid_of |= (unsigned long long)valid << (16 * asked);
    ++asked;
  };
  static_assert(kAqStages <= 4 && TILE % ROWS_AT_ONCE == 0 && kAqWarps % HEADS == 0, "four tiles asked for at most");
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
    float v[G * KS * 4];  // a group's codes of thread t are a run of GROUP / 4 columns
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      uint32_t w[GROUP / 8];
#pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) {
        const uint4 x = on ? __ldg(reinterpret_cast<const uint4*>(src + k * GROUP + t * (GROUP / 4)) + i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < KS * 4; ++i) {
        const int c = code_at<FMT>(i / 4, i % 4);
        const float x = c & 1 ? bf16_hi(w[c / 2]) : bf16_lo(w[c / 2]);
        v[k * KS * 4 + i] = x;
        top = fmaxf(top, fabsf(x));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float unit = pow2_below(top), inv = pow2_inverse(unit);
#pragma unroll
    for (int k = 0; k < G * KS; ++k) {
      qf[n][k][0] = pack_half2(v[4 * k] * inv, v[4 * k + 1] * inv);
      qf[n][k][1] = pack_half2(v[4 * k + 2] * inv, v[4 * k + 3] * inv);
    }
    // (kept above 0: -inf times it is to be -inf; what 2^-149 makes of a score of any size is below 2^-21)
    qs[n][0] = fmaxf(__shfl_sync(0xffffffffu, unit, 8 * t) * a.scale_log2e, __uint_as_float(1u));
    qs[n][1] = fmaxf(__shfl_sync(0xffffffffu, unit, 8 * t + 4) * a.scale_log2e, __uint_as_float(1u));
  }

  float o[NT][G * KS][4];
  // the references that products are taken relative to (before qs, so that the largest differs
  // from itself by nothing): raised when something in a tile is more than 2^6 above them
  float m[NT][2], ref[NT][2], high_at[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int k = 0; k < G * KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
    m[n][0] = m[n][1] = -INFINITY;
    ref[n][0] = ref[n][1] = 0.f;  // m, or 0 while that is -inf
    high_at[n][0] = high_at[n][1] = -INFINITY;  // m + 6 / qs: what a product has to be above
    l[n][0] = l[n][1] = 0.f;
  }

  for (int i = 0, stage = 0; i < rounds; ++i, stage = stage == kAqStages - 1 ? 0 : stage + 1) {
    cp_async_wait<kAqStages - 2>();
    __syncthreads();  // all copies are there, and all warps are done with the stage before
    const int valid = (int)(valid_of & 0xffffu) - own_rows;
    valid_of >>= 16;
    --asked;
    ask(stage == 0 ? kAqStages - 1 : stage - 1);
    if (valid <= 0) continue;
    const char* st = ring + stage * St::kBytes + warp * St::kUnit;
    const float* k_scale = reinterpret_cast<const float*>(ring + stage * St::kBytes + St::kKs) + own_rows * SF + own_head * G;
    const float* v_scale = k_scale + St::kScales / 4;
    // S = K q, keys g and g + 8 of each 16
    float s[M][NT][4];
#pragma unroll
    for (int mi = 0; mi < M; ++mi) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const char* row = st + (16 * mi + g) * St::kPitch + k * GROUP * BITS / 8 + t * KB;
        const Raw<KB> k0 = read_raw<KB>(row), k1 = read_raw<KB>(row + 8 * St::kPitch);
        const float ks0 = k_scale[(16 * mi + g) * SF + k], ks1 = k_scale[(16 * mi + g + 8) * SF + k];
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
#pragma unroll
        for (int q = 0; q < KS; ++q) {
          uint32_t f[4];
          four_codes<FMT>(k0.w, q, f[0], f[2]);
          four_codes<FMT>(k1.w, q, f[1], f[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(part[n], f, qf[n][k * KS + q][0], qf[n][k * KS + q][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[mi][n][0] = k == 0 ? part[n][0] * ks0 : fmaf(part[n][0], ks0, s[mi][n][0]);
          s[mi][n][1] = k == 0 ? part[n][1] * ks0 : fmaf(part[n][1], ks0, s[mi][n][1]);
          s[mi][n][2] = k == 0 ? part[n][2] * ks1 : fmaf(part[n][2], ks1, s[mi][n][2]);
          s[mi][n][3] = k == 0 ? part[n][3] * ks1 : fmaf(part[n][3], ks1, s[mi][n][3]);
        }
      }
    }
    if (valid < kAqRows) {
#pragma unroll
      for (int mi = 0; mi < M; ++mi)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * mi + g + 8 * (e >> 1) >= valid) s[mi][n][e] = -INFINITY;
    }
    bool high = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
        for (int mi = 1; mi < M; ++mi) top = fmaxf(top, fmaxf(s[mi][n][e], s[mi][n][2 + e]));
        high |= top > high_at[n][e];
      }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = m[n][e];
#pragma unroll
          for (int mi = 0; mi < M; ++mi) top = fmaxf(top, fmaxf(s[mi][n][e], s[mi][n][2 + e]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          ref[n][e] = top == -INFINITY ? 0.f : top;
          alpha[e] = exp2f((m[n][e] - ref[n][e]) * qs[n][e]);
          m[n][e] = top;
          high_at[n][e] = top + 6.f / qs[n][e];
          l[n][e] *= alpha[e];
        }
#pragma unroll
        for (int k = 0; k < G * KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][k][e] *= alpha[e & 1];
      }
    }
    // The weights' transposes, in upper and lower halves: keys 2t, 2t + 1 (+ 8 r) of column g.
    float2 p[M][NT][2];
#pragma unroll
    for (int mi = 0; mi < M; ++mi)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mi][n][e] = exp2_approx((s[mi][n][e] - ref[n][e & 1]) * qs[n][e & 1]);
          l[n][e & 1] += s[mi][n][e];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t x = __float_as_uint(s[mi][n][2 * r]), y = __float_as_uint(s[mi][n][2 * r + 1]);
          const uint32_t up = movmatrix(upper_halves(x, y)), low = movmatrix(lower_halves(x, y));
          p[mi][n][r] = make_float2(__uint_as_float(lower_halves(low, up)), __uint_as_float(upper_halves(low, up)));
        }
      }
    // O += V w, group by group; keys 2t, 2t + 1, 2t + 8, 2t + 9 of each 16
#pragma unroll
    for (int k = 0; k < G; ++k) {
      auto key = [&](int mi, int r) { return 16 * mi + 2 * t + (r & 1) + 4 * (r & 2); };
      float2 w[NT][M][2];
      uint32_t tops = 0;  // the largest weight of column g; of both query tiles, the upper halves side by side
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top = 0.f;
#pragma unroll
        for (int mi = 0; mi < M; ++mi)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            w[n][mi][r] = mul2(p[mi][n][r], make_float2(v_scale[key(mi, 2 * r) * SF + k], v_scale[key(mi, 2 * r + 1) * SF + k]));
            top = fmaxf(fmaxf(top, fabsf(w[n][mi][r].x)), fabsf(w[n][mi][r].y));
          }
        tops = NT == 2 ? upper_halves(tops, __float_as_uint(top)) : __float_as_uint(top);
      }
#pragma unroll
      for (int i = 1; i < 4; i *= 2) {
        const uint32_t x = __shfl_xor_sync(0xffffffffu, tops, i);
        tops = NT == 2 ? __vmaxu2(tops, x) : __float_as_uint(fmaxf(__uint_as_float(tops), __uint_as_float(x)));
      }
      if constexpr (NT == 1) tops = __float_as_uint(weight_unit(__uint_as_float(tops)));
      const uint32_t tops0 = __shfl_sync(0xffffffffu, tops, 8 * t), tops1 = __shfl_sync(0xffffffffu, tops, 8 * t + 4);
      uint32_t hi[NT][M][2], lo[NT][M][2];
      float2 unit[NT];  // of columns 2t and 2t + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        auto unit_of = [&](uint32_t x) {
          return NT == 1 ? __uint_as_float(x) : weight_unit(__uint_as_float(n == 0 ? x << 16 : x));
        };
        unit[n] = make_float2(unit_of(tops0), unit_of(tops1));
        const float2 inv = both(pow2_inverse(unit_of(tops)));
#pragma unroll
        for (int mi = 0; mi < M; ++mi)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 x = mul2(w[n][mi][r], inv);
            const __half2 h = __floats2half2_rn(x.x, x.y);
            const float2 rest = mul2(fma2(__half22float2(h), both(-1.f), x), both(4096.f));
            hi[n][mi][r] = *reinterpret_cast<const uint32_t*>(&h);
            lo[n][mi][r] = pack_half2(rest.x, rest.y);
          }
      }
      // 16-key products between two updates of O: both of the unit, or one where a run is 16 bytes and registers are
      // short (one token over 49920 rows 37 us; with both 38 to 53, as the registers fall)
      constexpr int KEYS = VB == 16 && NT == 1 ? 1 : M;
#pragma unroll
      for (int m0 = 0; m0 < M; m0 += KEYS) {
        Raw<VB> vw[KEYS][4];
#pragma unroll
        for (int mi = 0; mi < KEYS; ++mi)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            vw[mi][r] = read_raw<VB>(st + St::kV + key(m0 + mi, r) * St::kPitch + k * GROUP * BITS / 8 + g * VB);
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          float a0[NT][4], a1[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) a0[n][e] = a1[n][e] = 0.f;
#pragma unroll
          for (int mi = 0; mi < KEYS; ++mi) {
            uint32_t f[4];
            two_keys<FMT>(vw[mi][0].w, vw[mi][1].w, mt, f[0], f[1]);
            two_keys<FMT>(vw[mi][2].w, vw[mi][3].w, mt, f[2], f[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(a0[n], f, hi[n][m0 + mi][0], hi[n][m0 + mi][1]);
              mma16816(a1[n], f, lo[n][m0 + mi][0], lo[n][m0 + mi][1]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float* y = o[n][k * KS + mt];
            const float2 small = mul2(unit[n], both(1.f / 4096.f));
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float2 z = fma2(make_float2(a0[n][e], a0[n][e + 1]), unit[n],
                                           fma2(make_float2(a1[n][e], a1[n][e + 1]), small, make_float2(y[e], y[e + 1])));
              y[e] = z.x;
              y[e + 1] = z.y;
            }
          }
        }
      }
    }
  }

  // Join the warps, in order.  The ring is free once all of them are done with it.
  cp_async_wait<0>();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[n][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      m[n][e] = m[n][e] == -INFINITY ? -INFINITY : m[n][e] * qs[n][e];  // in log2 units from here on
      if (g == 0) {
        s_m[warp][n * 8 + 2 * t + e] = m[n][e];
        s_l[warp][n * 8 + 2 * t + e] = sum;
      }
    }
  __syncthreads();
  float* s_o = reinterpret_cast<float*>(ring);  // [warp][column][kOPitch]
  constexpr int kOPitch = D + 4;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAqWarps; w += HEADS) top = fmaxf(top, s_m[w + own_head][n * 8 + 2 * t + e]);
      const float part = top == -INFINITY ? 0.f : exp2f(m[n][e] - top);  // a warp without rows has m = -inf and o = 0
      float* dst = s_o + (warp * COLS + n * 8 + 2 * t + e) * kOPitch;
#pragma unroll
      for (int k = 0; k < G * KS; ++k) {
        const int d = (k / KS) * GROUP + g * (GROUP / 8) + 2 * (k % KS);
        *reinterpret_cast<float2*>(dst + d) = make_float2(o[n][k][e] * part, o[n][k][2 + e] * part);
      }
    }
  __syncthreads();
  for (int i = tid; i < HEADS * COLS * (D / 4); i += kAqThreads) {
    const int hw = i / (COLS * (D / 4)), c = i / (D / 4) % COLS, d = i % (D / 4) * 4, col = col0 + c;
    if (col >= cols) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAqWarps; w += HEADS) top = fmaxf(top, s_m[w + hw][c]);
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kAqWarps; w += HEADS) {
      sum += top == -INFINITY ? s_l[w + hw][c] : s_l[w + hw][c] * exp2f(s_m[w + hw][c] - top);
      const float4 x = *reinterpret_cast<const float4*>(s_o + ((w + hw) * COLS + c) * kOPitch + d);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    const int token = col / share;
    const long long row = (long long)token * a.Hq + (h0 + hw) * share + col - token * share;
    if (a.splits > 1) {
      const long long at = row * a.splits + split;
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
    } else {
      write_out(a, row, D, d, v.x, top, sum);
      write_out(a, row, D, d + 1, v.y, top, sum);
      write_out(a, row, D, d + 2, v.z, top, sum);
      write_out(a, row, D, d + 3, v.w, top, sum);
    }
  }
}

// out = sum over the splits of 2^(m_i - m) O_i / sum of 2^(m_i - m) l_i.  A CTA a row; a warp
// takes every kJoinWarps-th split and adds up its own in order, then the warps are added in
// order; a lane holds D / 32 columns.  The O_i are asked for before the weights are known.
constexpr int kJoinWarps = 8;
constexpr int kJoinAhead = 10;
constexpr int kJoinSplits = 148 * kAqMostCtas;  // most splits

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_quant_join_kernel(const AttnQuantArgs a) {
  constexpr int C = D / 32;
  __shared__ float s_w[kJoinSplits], s_top[kJoinWarps], s_sum[kJoinWarps], s_v[kJoinWarps][D];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const long long row = blockIdx.x;
  const float* o = a.part_o + row * a.splits * D + lane * C;
  float y[kJoinAhead][C];
  auto ask = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      const int i = i0 + k * kJoinWarps;
      if (i < a.splits) {
        if constexpr (C == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o + (long long)i * D);
          y[k][0] = x.x; y[k][1] = x.y; y[k][2] = x.z; y[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o + (long long)i * D);
          y[k][0] = x.x; y[k][1] = x.y;
        }
      }
    }
  };
  ask(warp);
  constexpr int kOwn = (kJoinSplits + kJoinWarps * 32 - 1) / (kJoinWarps * 32);
  float2 ml[kOwn];
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int i = tid + k * kJoinWarps * 32;
    ml[k] = i < a.splits ? a.part_ml[row * a.splits + i] : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, ml[k].x);
  }
  top = warp_max(top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int i = tid + k * kJoinWarps * 32;
    const float weight = exp2f(ml[k].x - (top == -INFINITY ? 0.f : top));
    if (i < a.splits) s_w[i] = weight;
    // a NaN score leaves the maximum as it was: its sum counts all the same
    sum += ml[k].x == -INFINITY ? ml[k].y : ml[k].y * weight;
  }
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  float v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = 0.f;
  for (int i0 = warp; i0 < a.splits; i0 += kJoinWarps * kJoinAhead) {
    if (i0 != warp) ask(i0);
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      const int i = i0 + k * kJoinWarps;
      if (i < a.splits) {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] += y[k][c] * s_w[i];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_v[warp][lane * C + c] = v[c];
  __syncthreads();
  if (tid < D) {
    float all = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      all += s_sum[w];
      x += s_v[w][tid];
    }
    write_out(a, row, D, tid, x, top, all);
  }
}

template <int FMT, int D, int GROUP, int NT, int HEADS>
cudaError_t launch(AttnQuantArgs a, cudaStream_t s) {
  a.splits = attn_quant_splits_of(ctas_per_sm<FMT, D, GROUP, NT>(), a.T, a.Hq, a.q.H, a.Kp, a.q.P_tok);
  const int cols = a.T * (a.Hq / a.q.H);
  const size_t ring = (size_t)kAqStages * Stage<FMT, D, GROUP>::kBytes;
  const size_t join = (size_t)kAqWarps * 8 * NT * (D + 4) * sizeof(float), smem = ring > join ? ring : join;
  if (smem > kDefaultSmemOptIn) {
    const cudaError_t e = cudaFuncSetAttribute(attn_quant_kernel<FMT, D, GROUP, NT, HEADS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)(a.q.H / HEADS * a.splits), (cols + 8 * NT - 1) / (8 * NT));
  attn_quant_kernel<FMT, D, GROUP, NT, HEADS><<<grid, kAqThreads, smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  attn_quant_join_kernel<D><<<(unsigned)(a.T * a.Hq), kJoinWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

template <int FMT, int D, int GROUP>
cudaError_t launch_heads(const AttnQuantArgs& a, cudaStream_t s) {
  const int heads = attn_quant_heads(a.q.H);
  if (a.T * (a.Hq / a.q.H) <= 8) {
    if (heads == 4) return launch<FMT, D, GROUP, 1, 4>(a, s);
    return heads == 2 ? launch<FMT, D, GROUP, 1, 2>(a, s) : launch<FMT, D, GROUP, 1, 1>(a, s);
  }
  if (heads == 4) return launch<FMT, D, GROUP, 2, 4>(a, s);
  return heads == 2 ? launch<FMT, D, GROUP, 2, 2>(a, s) : launch<FMT, D, GROUP, 2, 1>(a, s);
}

template <int FMT>
cudaError_t launch_fmt(const AttnQuantArgs& a, cudaStream_t s) {
  if (a.q.d == 128) {
    if (a.q.group == 128) return launch_heads<FMT, 128, 128>(a, s);
    if (a.q.group == 64) return launch_heads<FMT, 128, 64>(a, s);
    return launch_heads<FMT, 128, 32>(a, s);
  }
  if (a.q.group == 64) return launch_heads<FMT, 64, 64>(a, s);
  return launch_heads<FMT, 64, 32>(a, s);
}

}  // namespace

int attn_quant_most_splits(int T, int Hq, int H, int Kp, int P_tok) {
  return attn_quant_splits_of(kAqMostCtas, T, Hq, H, Kp, P_tok);
}

cudaError_t launch_attn_quant(const AttnQuantArgs& a, cudaStream_t s) {
  switch (a.q.format) {
    case HKV_QUANT_E4M3: return launch_fmt<HKV_QUANT_E4M3>(a, s);
    case HKV_QUANT_INT8: return launch_fmt<HKV_QUANT_INT8>(a, s);
    default: return launch_fmt<HKV_QUANT_INT4>(a, s);
  }
}

}  // namespace hsa
