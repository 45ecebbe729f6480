// llm_w4.hip -- linear layer on 4-bit weights with group scales, for few rows, on matrix instructions; compiled once per type
// of x (-DCBS_W4_X=n: int8, float16, bfloat16, float32).
//
//   y[m][n] = x_scale[m] * sum_g scales[g][n] * sum_{k in g} x[m][k] * (code[n][k] - zero[g][n])
//
// The inner sums are exact products of x and whole numbers: float16 and bfloat16 hold code - zero (-255 to 15) exactly, a
// float32 x goes as the three bfloat16 terms whose sum it is, int8 sums are whole numbers.  Sums are 32 bits wide; scales
// meet them once a group, in float32.
//
// A wave has 16 rows of x as the rows of a 16x16 instruction and 16 output features as its columns; lane l holds feature
// l % 16 and of a block of 128 input features the 32 of its group l / 16, one 16-byte load; a step takes a word of it, and x
// lies accordingly.  Where a block has more than one scale, words are first exchanged between the four groups, so that step s
// has its input features 32 s to 32 s + 31, all of one scale; group g holds 8 g to 8 g + 7 of them.
#include <type_traits>

#include "llm_w4.h"

namespace cbs {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef f16_t f16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));

enum { X_I8, X_F16, X_BF16, X_F32 };
constexpr int X = CBS_W4_X;
constexpr int TERMS = X == X_F32 ? 3 : 1;
constexpr int RAW = X == X_I8 ? 8 : X == X_F32 ? 32 : 16;  // bytes of eight elements

struct Piece {
  uint32_t w[RAW / 4];
};

__device__ __forceinline__ int fdiv(int n, FastDiv f) { return (int)((__umulhi((unsigned)n, f.magic) + (unsigned)n) >> f.shift); }

// words[s] of group g <- words[g] of group s
__device__ __forceinline__ void exchange(u32x4 &w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false), b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false), d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = u32x4{c[0], c[1], d[0], d[1]};
}

// The same for x that lies in its own order, int8: words 2 s and 2 s + 1 of group g <- the two of input features 64 s + 16 g on.
[[maybe_unused]] __device__ __forceinline__ void exchange_pairs(u32x4 &w) {
  const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[2], false, false), b = __builtin_amdgcn_permlane16_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], a[1], false, false), d = __builtin_amdgcn_permlane32_swap(b[0], b[1], false, false);
  w = u32x4{c[0], d[0], c[1], d[1]};
}
// Bytes of even and of odd input features, eight in all, to their own order.
__device__ __forceinline__ void mix(uint32_t &even, uint32_t &odd) {
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  even = lo, odd = hi;
}

// Eight codes as 16-bit floats, even input features then odd ones (the order in which x lies, too; OWN: in their own).  A code is, as it stands in
// a byte, the 8-bit float of 1/512 of it: two conversions a byte pair cost one instruction.
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
template <bool OWN>
[[maybe_unused]] __device__ __forceinline__ u32x4 codes16(uint32_t w) {
  uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  if constexpr (OWN) mix(even, odd);
  u32x4 r;
  if constexpr (X == X_F16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true));
  }
  return r;
}
// The same less the zero point; bfloat16: 16 times that.
template <bool ZEROS, bool OWN>
[[maybe_unused]] __device__ __forceinline__ u32x4 weights(uint32_t w, uint32_t zero) {
  u32x4 r;
  if constexpr (X == X_F16) {
    const f16_t z = (f16_t)(float)zero;
    r = codes16<OWN>(w);
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (uint32_t)r[i]) - f16x2{z, z});
  } else {  // no instruction subtracts two bfloat16
    const uint32_t u = w ^ 0x88888888u;
    uint32_t even = (u << 4) & 0xf0f0f0f0u, odd = u & 0xf0f0f0f0u;  // bytes 16 (code - 8)
    if constexpr (OWN) mix(even, odd);
    asm("" : "+v"(even), "+v"(odd));                                // a byte's conversion is one instruction
    const float away = (float)(16 * ((int)zero - 8));
#pragma unroll
    for (int i = 0; i < 4; i++) {  // 16 times whole numbers below 2^8: the upper half of a float32 holds them
      const uint32_t two = (i < 2 ? even : odd) >> (16 * (i & 1));
      float lo = (float)(int8_t)two, hi = (float)(int8_t)(two >> 8);
      if constexpr (ZEROS) lo -= away, hi -= away;
      r[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
  }
  return r;
}
// int8: 16 (code - 8).
template <bool OWN>
[[maybe_unused]] __device__ __forceinline__ u32x2 weights_i8(uint32_t w) {
  const uint32_t u = w ^ 0x88888888u;
  uint32_t even = (u << 4) & 0xf0f0f0f0u, odd = u & 0xf0f0f0f0u;
  if constexpr (OWN) mix(even, odd);
  return u32x2{even, odd};
}

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (X == X_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// x in LDS: pieces of eight elements, as the instructions' lanes read them.  A block of 128 input features has STEPS fragments
// of RB * 16 rows, or of R < 16; a row's place in a fragment turns with the piece, so that neither writes nor reads of
// neighbours meet in a bank.
constexpr int XB = kW4Bytes[X];
__device__ __forceinline__ void read_tail(Piece &v, const char *at, int left) {  // the first `left` of a piece, zeros behind them
  constexpr int EB = RAW / 8;
#pragma unroll
  for (int j = 0; j < RAW / 4; j++) v.w[j] = 0;
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (j < left) {
      uint32_t e;
      if constexpr (EB == 1) e = (uint32_t)((const uint8_t *)at)[j] << (8 * (j % 4));
      else if constexpr (EB == 2) e = (uint32_t)((const uint16_t *)at)[j] << (16 * (j % 2));
      else e = ((const uint32_t *)at)[j];
      v.w[j * EB / 4] |= e;
    }
}
// The place of row mr of group g in fragment s, term t, of a block of r rows (a power of two, 16 at most); rb fragments a step.
__device__ __forceinline__ int frag_at(int rb, int s, int t, int g, int mr, int r) {
  return ((s * rb * TERMS + t) * 4 + g) * r * 16 + ((mr ^ (4 * s + g)) & (r - 1)) * 16;
}
// Piece q (of 16) of row mr into such a block.
template <int GS>
__device__ __forceinline__ void write_piece(const Piece &x, unsigned char *block, int q, int mr, int r, int rb) {
  const int s = GS == 4 ? q & 3 : q >> 2, g = GS == 4 ? q >> 2 : q & 3;
  if constexpr (X == X_I8) {  // an instruction takes two steps: 16 bytes of a row
    const u32x2 v = {__builtin_amdgcn_perm(x.w[1], x.w[0], 0x06040200u), __builtin_amdgcn_perm(x.w[1], x.w[0], 0x07050301u)};
    *(u32x2 *)(block + frag_at(rb, s >> 1, 0, g, mr, r) + (s & 1) * 8) = v;
  } else if constexpr (X == X_F32) {
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; j++) rest[j] = __uint_as_float(x.w[j]);
#pragma unroll
    for (int t = 0; t < TERMS; t++) {  // an infinity or NaN stays whole in the first
      bf16x8 v;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const bf16_t part = (bf16_t)rest[j];
        v[j / 2 + 4 * (j & 1)] = part;
        rest[j] = __builtin_isfinite((float)part) ? rest[j] - (float)part : 0.0f;
      }
      *(bf16x8 *)(block + frag_at(rb, s, t, g, mr, r)) = v;
    }
  } else {
    const u32x4 v = {__builtin_amdgcn_perm(x.w[1], x.w[0], 0x05040100u), __builtin_amdgcn_perm(x.w[3], x.w[2], 0x05040100u),
                     __builtin_amdgcn_perm(x.w[1], x.w[0], 0x07060302u), __builtin_amdgcn_perm(x.w[3], x.w[2], 0x07060302u)};
    *(u32x4 *)(block + frag_at(rb, s, 0, g, mr, r)) = v;
  }
}

// A wave's output features are n0 + 16 b + mr, b < NB.  GS: steps of 32 input features that share a scale (1, 2, or 4: 128 and
// more).  WIDE: float32 scales.
template <int NB, int GS, bool WIDE>
struct Weights {
  static constexpr int GPB = 4 / GS;  // scales of a block
  const W4Params &p;
  const char *codes0;
  uint32_t row[NB], sc_at[NB], zp_at[NB];  // byte offsets; a tile's codes are 2^31 bytes at most
  int last_piece, g;
  bool has_zeros;

  struct Block {
    u32x4 codes[NB];
    uint32_t sc[NB][GPB], zp[NB][GPB];
  };

  __device__ __forceinline__ Weights(const W4Params &params, int first, int n0, int lane) : p(params), g(lane >> 4) {
    const int first_row = min(first, p.n - 1);
    codes0 = (const char *)p.a.codes + (int64_t)first_row * p.code_stride;
    last_piece = p.code_stride / 16 - 1;
    has_zeros = p.a.zeros != nullptr;
#pragma unroll
    for (int b = 0; b < NB; b++) {
      const int feature = min(n0 + 16 * b + (lane & 15), p.n - 1);
      row[b] = (uint32_t)(feature - first_row) * (uint32_t)p.code_stride;
      sc_at[b] = (uint32_t)feature * (WIDE ? 4 : 2);
      zp_at[b] = has_zeros ? (uint32_t)feature : 0;
    }
  }
  // Never under a condition: the count of loads in flight is what the waits go by.  A block past the last is the last again.
  __device__ __forceinline__ void load(Block &w, int block) const {
    block = min(block, p.blocks - 1);
    const uint32_t piece = (uint32_t)min(block * 4 + g, last_piece) * 16;
#pragma unroll
    for (int b = 0; b < NB; b++) w.codes[b] = *(const u32x4 *)(codes0 + (row[b] + piece));
#pragma unroll
    for (int q = 0; q < GPB; q++) {
      const int64_t first = (int64_t)min(GS == 4 ? fdiv(block, p.by_wide) : block * GPB + q, p.groups - 1) * p.n;
      const char *sc0 = (const char *)p.a.scales + first * (WIDE ? 4 : 2), *zp0 = (const char *)(has_zeros ? p.a.zeros + first : p.a.codes);
#pragma unroll
      for (int b = 0; b < NB; b++) {
        if constexpr (WIDE) w.sc[b][q] = *(const uint32_t *)(sc0 + sc_at[b]);
        else w.sc[b][q] = *(const uint16_t *)(sc0 + sc_at[b]);
        w.zp[b][q] = *(const uint8_t *)(zp0 + zp_at[b]);  // without zero points a byte is read for nothing
      }
    }
  }
  __device__ __forceinline__ float scale_of(uint32_t bits) const {
    return WIDE ? __uint_as_float(bits) : p.scale_dtype == CBS_F16 ? (float)__builtin_bit_cast(f16_t, (uint16_t)bits) : __uint_as_float(bits << 16);
  }
};

// A block's products with RB blocks of 16 rows; x_at(s, m, t): fragment s (int8: of two steps) of row block m, term t.
// SUMS: codes as they are, less the zero point times the rows' own sums -- 7 instructions for eight codes rather than 11
// (float16) or 16 (bfloat16), for one more product a fragment and a step's end that is twice as long, so for one block of rows
// only.  Errors are those of sum |x| (code + zero) in place of sum |x| |code - zero|, in 32 bits.  Not for what wild_of() finds.
// OWN: x lies in its own order (int8: 16 bytes of a lane are neighbours, so that a group of 32 is two of the lanes' groups).
template <bool ZEROS, bool SUMS, bool OWN, int RB, int NB, int GS, bool WIDE, typename XAt>
__device__ __forceinline__ void multiply(const Weights<NB, GS, WIDE> &ws, typename Weights<NB, GS, WIDE>::Block &w, const XAt &x_at, f32x4 (&total)[NB][RB]) {
  if constexpr (GS < 4 || OWN) {
#pragma unroll
    for (int b = 0; b < NB; b++) {
      if constexpr (X == X_I8 && OWN) exchange_pairs(w.codes[b]);
      else exchange(w.codes[b]);
    }
  }
  if constexpr (X == X_I8) {
    i32x4 sum[NB][RB], ones[RB];
    u32x4 xs[2][RB];  // one block of rows: all at once, to wait for LDS once
#pragma unroll
    for (int s2 = 0; s2 < 2; s2++) {
      // the next step's rows on their way while this one is computed; all at once would not fit the registers
#pragma unroll
      for (int i = s2 == 0 ? 0 : 2; i < 2; i++)
#pragma unroll
        for (int m = 0; m < RB; m++) xs[i][m] = *(const u32x4 *)x_at(i, m, 0);
      if (RB > 1) __builtin_amdgcn_sched_barrier(0);
      u32x4(&xf)[RB] = xs[s2];
#pragma unroll
      for (int h = 0; h < (GS == 1 ? 2 : 1); h++) {
        const bool start = GS < 4 || s2 == 0, end = GS < 4 || s2 == 1;
        const int q = GS == 1 ? 2 * s2 + h : GS == 2 ? s2 : 0;
        const auto product = [&](u32x4 x, u32x4 y, i32x4 c) {
          if constexpr (GS == 1 && OWN) {
            const uint32_t in = (ws.g >> 1) == h ? ~0u : 0u;
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, y & u32x4{in, in, in, in}), c, 0, 0, 0);
          } else if constexpr (GS == 1) {
            const u32x2 yh = {y[2 * h], y[2 * h + 1]}, xh = {x[2 * h], x[2 * h + 1]};
            return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, xh), __builtin_bit_cast(long, yh), c, 0, 0, 0);
          } else {
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, y), c, 0, 0, 0);
          }
        };
#pragma unroll
        for (int b = 0; b < NB; b++) {
          const u32x2 w0 = weights_i8<OWN>(w.codes[b][2 * s2]), w1 = weights_i8<OWN>(w.codes[b][2 * s2 + 1]);
          const u32x4 wf = {w0[0], w0[1], w1[0], w1[1]};
#pragma unroll
          for (int m = 0; m < RB; m++) sum[b][m] = product(xf[m], wf, start ? i32x4{0, 0, 0, 0} : sum[b][m]);
        }
        if constexpr (ZEROS) {  // the rows' own sums, for zero points other than 8
          const u32x4 one = {0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u};
#pragma unroll
          for (int m = 0; m < RB; m++) ones[m] = product(xf[m], one, start ? i32x4{0, 0, 0, 0} : ones[m]);
        }
        if (end) {
#pragma unroll
          for (int b = 0; b < NB; b++) {
            const float scale = ws.scale_of(w.sc[b][q]) * 0.0625f;
            const int z = ws.has_zeros ? 16 * ((int)w.zp[b][q] - 8) : 0;
#pragma unroll
            for (int m = 0; m < RB; m++) {
              if constexpr (ZEROS) {
#pragma unroll
                for (int i = 0; i < 4; i++) sum[b][m][i] -= __mul24(z, ones[m][i]);
              }
#pragma unroll
              for (int i = 0; i < 4; i++) total[b][m][i] = __builtin_fmaf(scale, (float)sum[b][m][i], total[b][m][i]);
            }
          }
        }
      }
    }
  } else {
    f32x4 sum[NB][RB], ones[RB];
    u32x4 xs[4][RB][TERMS];  // one block of rows: all at once, to wait for LDS once
#pragma unroll
    for (int s = 0; s < 4; s++) {
      const bool start = s % GS == 0, end = s % GS == GS - 1;
      constexpr bool ALL = RB * TERMS == 1;
#pragma unroll
      for (int i = s == 0 ? 0 : ALL ? 4 : s + 1; i < (ALL ? 4 : min(s + 2, 4)); i++)  // the next step's on their way while this one is computed
#pragma unroll
        for (int m = 0; m < RB; m++)
#pragma unroll
          for (int t = 0; t < TERMS; t++) xs[i][m][t] = *(const u32x4 *)x_at(i, m, t);
      if (RB > 1) __builtin_amdgcn_sched_barrier(0);  // and not more: all at once would not fit the registers
      u32x4(&xf)[RB][TERMS] = xs[s];
      u32x4 wf[NB];
#pragma unroll
      for (int b = 0; b < NB; b++) wf[b] = SUMS ? codes16<OWN>(w.codes[b][s]) : weights<ZEROS, OWN>(w.codes[b][s], ZEROS && ws.has_zeros ? w.zp[b][s / GS] : 8);
      // OWN: products before what other waves have to issue, 37 -> 35 us (64 rows 8192 -> 16384, bfloat16)
      if (OWN) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int m = 0; m < RB; m++)
#pragma unroll
          for (int t = TERMS - 1; t >= 0; t--) sum[b][m] = mma(xf[m][t], wf[b], start && t == TERMS - 1 ? f32x4{0, 0, 0, 0} : sum[b][m]);
      if (OWN) __builtin_amdgcn_s_setprio(0);
      if constexpr (SUMS) {
        const uint32_t one = X == X_F16 ? 0x3c003c00u : 0x3f803f80u;
#pragma unroll
        for (int m = 0; m < RB; m++) ones[m] = mma(xf[m][0], u32x4{one, one, one, one}, start ? f32x4{0, 0, 0, 0} : ones[m]);
      }
      if (end) {
#pragma unroll
        for (int b = 0; b < NB; b++) {
          const float scale = ws.scale_of(w.sc[b][s / GS]) * (X != X_F16 && !SUMS ? 0.0625f : 1.0f), zero = ws.has_zeros ? (float)w.zp[b][s / GS] : 8.0f;
#pragma unroll
          for (int m = 0; m < RB; m++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
              if constexpr (SUMS) sum[b][m][i] = __builtin_fmaf(-zero, ones[m][i], sum[b][m][i]);
              total[b][m][i] = __builtin_fmaf(scale, sum[b][m][i], total[b][m][i]);
            }
        }
      }
    }
  }
}

// Sums of the waves that shared the input features, through LDS ([wave][r rows][tile_n + 4]), scaled and written.
// TAIL, not 0: the sums are without the last k % TAIL input features.
template <int RB, int NB, int TAIL>
__device__ __forceinline__ void join(const W4Params &p, f32x4 (&total)[NB][RB], float *joined, int r, int rows, int64_t m0, int tile, int wk, int wks, int wn, int tile_n, int lane) {
  const int g = lane >> 4, mr = lane & 15, pitch = tile_n + 4, fours = tile_n / 4;
#pragma unroll
  for (int b = 0; b < NB; b++)
#pragma unroll
    for (int m = 0; m < RB; m++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (m * 16 + 4 * g + i < r) joined[(wk * r + m * 16 + 4 * g + i) * pitch + (wn * NB + b) * 16 + mr] = total[b][m][i];
  __syncthreads();
  for (int e = threadIdx.x; e < rows * fours; e += blockDim.x) {
    const int m = e / fours, c = e - m * fours;
    f32x4 sum = {0, 0, 0, 0};
    for (int w = 0; w < wks; w++) sum += *(const f32x4 *)(joined + (w * r + m) * pitch + 4 * c);
    const int n = tile * tile_n + 4 * c;
    if (TAIL > 0 && p.k % max(TAIL, 1)) {
      for (int k = p.k / max(TAIL, 1) * TAIL; k < p.k; k++) {
        const float x = X == X_I8 ? (float)((const int8_t *)p.a.x)[(m0 + m) * p.a.x_stride + k] : load_as_f32(p.a.x, (m0 + m) * p.a.x_stride + k, X == X_F16 ? CBS_F16 : X == X_BF16 ? CBS_BF16 : CBS_F32);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int f = min(n + i, p.n - 1);
          const int64_t at = (int64_t)(k / p.group) * p.n + f;
          const int code = (p.a.codes[(int64_t)f * p.code_stride + k / 2] >> (4 * (k & 1)) & 15) - (p.a.zeros ? p.a.zeros[at] : 8);
          sum[i] = __builtin_fmaf(x * (float)code, load_as_f32(p.a.scales, at, p.scale_dtype), sum[i]);
        }
      }
    }
    if constexpr (X == X_I8) sum *= p.a.x_scale[m0 + m];
    const int64_t at = (m0 + m) * p.a.out_stride + n;
    if (n + 4 <= p.n) {
      if (p.out_dtype == CBS_F32) {
        store_vec<float, 4>((float *)p.a.out + at, Vec<float, 4>{sum[0], sum[1], sum[2], sum[3]});
      } else if (p.out_dtype == CBS_F16) {
        store_vec<f16_t, 4>((f16_t *)p.a.out + at, Vec<f16_t, 4>{(f16_t)sum[0], (f16_t)sum[1], (f16_t)sum[2], (f16_t)sum[3]});
      } else {
        store_vec<bf16_t, 4>((bf16_t *)p.a.out + at, Vec<bf16_t, 4>{(bf16_t)sum[0], (bf16_t)sum[1], (bf16_t)sum[2], (bf16_t)sum[3]});
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < p.n) store_f32_as(p.a.out, at + i, sum[i], p.out_dtype);
    }
  }
}

// Of two 16-bit floats, one is infinite or NaN, or as a bfloat16 2^97 and more: the sums of 2^16 such times codes and zero points
// would leave 32 bits where those of their differences need not.
[[maybe_unused]] __device__ __forceinline__ bool wild_of(uint32_t two) {
  constexpr uint32_t E = X == X_F16 ? 0x7c00u : 0x7000u;
  return (two & E) == E || (two & E << 16) == E << 16;
}

// neighbouring tiles to one XCD: they share cache lines of scales
__device__ __forceinline__ int tile_of(const W4Params &p) {
  const int per = p.tiles >> 3, extra = p.tiles & 7, xcd = blockIdx.x & 7;
  return xcd * per + min(xcd, extra) + (blockIdx.x >> 3);
}

// Up to 16 rows, all of x in LDS: brought there once, then each wave goes through its blocks on its own, DEPTH of them on
// their way to registers.  What it costs is reading the codes: 8 rows 8192 -> 28672 of int8 27 us, 4.5 TB/s; one row
// 4096 -> 4096 5.6 us, of which 2 for the codes: the rest is a launch, x's way to LDS and the join, one after the other.
template <int GS, bool WIDE>
__global__ __launch_bounds__(kW4Waves * 64) void w4_few_kernel(const W4Params p) {
  constexpr int DEPTH = 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, mr = lane & 15;
  const int wns = p.waves_n, wks = p.waves_k, wk = fdiv(wave, p.by_waves_n), wn = wave - wk * wns;
  const int tile_n = wns * 16, tile = tile_of(p);
  const int rows = (int)p.a.rows, r = p.few_rows, stage = r * kW4Block * XB;
  const Weights<1, GS, WIDE> ws(p, tile * tile_n, tile * tile_n + wn * 16, lane);
  // a wave's blocks wk, wk + wks, ..., from one on that differs between tiles: rows of codes often lie a power of two apart, and
  // all of them read at the same place would meet in a few memory channels
  const int count = p.count - (wk + (p.count - 1) * wks >= p.blocks), from = tile & p.from_mask;
  const auto block_at = [&](int j) {
    const int i = j + from;
    return wk + (i < count ? i : i - count) * wks;
  };
  typename Weights<1, GS, WIDE>::Block w[DEPTH];
  constexpr bool SUMS = X == X_F16 || X == X_BF16;
  constexpr int BATCH = X == X_F32 ? 2 : X == X_I8 ? 8 : 4;
  __shared__ int s_wild[kW4Waves];
  bool wild = false;  // see wild_of()
  const int whole = p.k / 8, rest = p.blocks * 16 - whole;  // pieces of a row
  const auto put = [&](const Piece &v, int m, int q) {
    if constexpr (SUMS) {
#pragma unroll
      for (int j = 0; j < 4; j++) wild |= wild_of(v.w[j]);
    }
    write_piece<GS>(v, lds + (q >> 4) * stage, q & 15, m, r, 1);
  };
  Piece v[BATCH];
  int m[BATCH], q[BATCH];
  const auto get = [&](int e0) {
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
      if (e0 - lane + i * threads >= rows * whole) break;
      const int e = min(e0 + i * threads, rows * whole - 1);  // the last one more than once
      m[i] = fdiv(e, p.by_whole), q[i] = e - m[i] * whole;
      __builtin_memcpy(&v[i], (const char *)p.a.x + m[i] * p.a.x_stride * (RAW / 8) + (int64_t)q[i] * RAW, RAW);
    }
  };
  get(tid);  // the first of x ahead of the codes: loads return in order
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < DEPTH; d++) ws.load(w[d], block_at(min(d, count - 1)));
  __builtin_amdgcn_sched_barrier(0);
  for (int e0 = tid; e0 < rows * whole; e0 += BATCH * threads) {
    if (e0 != tid) get(e0);
#pragma unroll
    for (int i = 0; i < BATCH; i++)
      if (e0 - lane + i * threads < rows * whole) put(v[i], m[i], q[i]);
  }
  for (int e = tid; e < rest * r; e += threads) {
    const int m = e / rest, q = whole + e - m * rest;
    Piece t;
    read_tail(t, (const char *)p.a.x + m * p.a.x_stride * (RAW / 8) + (int64_t)q * RAW, m < rows ? p.k - q * 8 : 0);
    put(t, m, q);
  }
  if (SUMS) s_wild[wave] = __any(wild);
  __syncthreads();

  f32x4 total[1][1] = {{f32x4{0, 0, 0, 0}}};
  const auto step = [&](int d, int j) {
    if (j >= count) return;
    const unsigned char *x = lds + block_at(j) * stage;
    const auto x_at = [&](int s, int, int t) { return x + frag_at(1, s, t, g, mr, r); };
    multiply<!SUMS, SUMS, false, 1>(ws, w[d], x_at, total);
  };
  int j = 0;
  for (; j + DEPTH < count; j += DEPTH) {  // no way out between its parts: it would cost the waits' counts
#pragma unroll
    for (int d = 0; d < DEPTH; d++) {
      step(d, j + d);
      ws.load(w[d], block_at(min(j + DEPTH + d, count - 1)));
    }
  }
#pragma unroll
  for (int d = 0; d < DEPTH; d++) step(d, j + d);
  __syncthreads();
  join<1, 1, 0>(p, total, (float *)lds, r, rows, 0, tile, wk, wks, wn, tile_n, lane);
  if constexpr (!SUMS) return;
  int any = 0;
  for (int i = 0; i < threads / 64; i++) any |= s_wild[i];
  if (any) {  // rare: a wave an output, as the formula has it, times 2^-8: no product of x and a whole number leaves 32 bits
    __syncthreads();
    for (int e = wave; e < rows * tile_n; e += threads / 64) {
      const int m = e / tile_n, n = tile * tile_n + e % tile_n;
      if (n >= p.n) continue;
      const uint8_t *codes = p.a.codes + (int64_t)n * p.code_stride;
      float sum = 0.0f;
      for (int k = lane; k < p.k; k += 64) {
        const int64_t at = (int64_t)(k / p.group) * p.n + n;
        const int c = (codes[k / 2] >> (4 * (k & 1)) & 15) - (ws.has_zeros ? p.a.zeros[at] : 8);
        const float x = load_as_f32(p.a.x, m * p.a.x_stride + k, X == X_F16 ? CBS_F16 : CBS_BF16) * 0x1p-8f;
        sum = __builtin_fmaf(x * (float)c, load_as_f32(p.a.scales, at, p.scale_dtype), sum);
      }
      sum = wave_sum(sum) * 0x1p8f;
      if (lane == 0) store_f32_as(p.a.out, m * p.a.out_stride + n, sum, p.out_dtype);
    }
  }
}

// More rows, RB blocks of 16 of them; of float32, which is split into its terms on the way to LDS, or from other than 16-byte
// boundaries.  A round is a block of input features for each of the waves that share them.  While one
// is computed, the next one's codes and x are on their way to registers; x then goes to the other of two buffers in LDS.  It
// waits for x: each tile reads all of it from the L2, in lines' halves.  us (k, n, rows): 5120, 13824, 61 of float16 30;
// 4096, 11008, 64 of float32 40, of which three products for each take 16.
template <int RB, int NB, int GS, bool WIDE>
__global__ __launch_bounds__(512, 2) void w4_kernel(const W4Params p) {
  constexpr int PIECES = kW4Most[X][RB / 2], STAGE = RB * 16 * kW4Block * XB;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, mr = lane & 15;
  const int wks = 1 << p.wk_log, wk = wave & (wks - 1), wn = wave >> p.wk_log;
  const int tile_n = (kW4Waves >> p.wk_log) * NB * 16, tile = tile_of(p);
  const int64_t m0 = (int64_t)blockIdx.y * (RB * 16);
  const int rows = (int)min((int64_t)(RB * 16), p.a.rows - m0);
  const int rounds = (p.blocks + wks - 1) >> p.wk_log, buffer = STAGE << p.wk_log;

  // x: a row's pieces along the threads
  const int row_log = p.wk_log + 4, row_mask = (1 << row_log) - 1, xq = tid & row_mask;
  Piece xr[PIECES];
  const char *x_row[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; i++) {
    const int m = ((tid + i * 512) >> row_log) & (RB * 16 - 1);
    // a piece that is not whole, or of a row beyond the last, reads what is there, for nothing
    x_row[i] = p.k >= 8 ? (const char *)p.a.x + (m0 + (m < rows ? m : 0)) * p.a.x_stride * (RAW / 8) : (const char *)p.a.codes;
  }
  const int x_half = p.k >= 8 ? 16 : 0;
  const auto fetch = [&](int round) {
    const int k = round * (kW4Block << p.wk_log) + xq * 8;  // below 2^24 + 2^12
    const uint32_t at = (k + 8 <= p.k ? (uint32_t)k : 0u) * (RAW / 8);
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      __builtin_memcpy(&xr[i], x_row[i] + at, RAW < 16 ? RAW : 16);
      if constexpr (RAW > 16) __builtin_memcpy(&xr[i].w[4], x_row[i] + at + x_half, 16);
    }
  };
  const auto keep = [&](int round, unsigned char *to) {  // no loads here, and no lane that does not write: see Weights::load
    if ((round + 1) * (kW4Block << p.wk_log) > p.k) {
      const uint32_t is = round * (kW4Block << p.wk_log) + xq * 8 + 8 <= p.k ? ~0u : 0u;
#pragma unroll
      for (int i = 0; i < PIECES; i++)
#pragma unroll
        for (int j = 0; j < RAW / 4; j++) xr[i].w[j] &= is;
    }
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const int m = ((tid + i * 512) >> row_log) & (RB * 16 - 1);  // more pieces than there are: some twice
      write_piece<GS>(xr[i], to + (xq >> 4) * STAGE + (m >> 4) * TERMS * 1024, xq & 15, m & 15, 16, RB);
    }
  };

  const Weights<NB, GS, WIDE> ws(p, tile * tile_n, tile * tile_n + wn * NB * 16, lane);
  typename Weights<NB, GS, WIDE>::Block w[2];
  f32x4 total[NB][RB];  // of rows 4 g to 4 g + 3 of a block of rows
#pragma unroll
  for (int b = 0; b < NB; b++)
#pragma unroll
    for (int m = 0; m < RB; m++) total[b][m] = f32x4{0, 0, 0, 0};
  fetch(0);
  ws.load(w[0], wk);
  keep(0, lds);
  fetch(1);
  ws.load(w[1], wks + wk);
  __syncthreads();
  for (int r0 = 0; r0 < rounds; r0 += 2) {  // always both
#pragma unroll
    for (int d = 0; d < 2; d++) {
      const int round = r0 + d, block = (round << p.wk_log) + wk;
      if (block < p.blocks) {
        const unsigned char *x = lds + d * buffer + wk * STAGE;
        const auto x_at = [&](int s, int m, int t) { return x + m * TERMS * 1024 + frag_at(RB, s, t, g, mr, 16); };
        if (X == X_F16 || ws.has_zeros) multiply<true, false, false, RB>(ws, w[d], x_at, total);
        else multiply<false, false, false, RB>(ws, w[d], x_at, total);
      }
      keep(round + 1, lds + (d ^ 1) * buffer);
      fetch(round + 2);
      ws.load(w[d], block + (2 << p.wk_log));
      __syncthreads();
    }
  }
  join<RB, NB, 8>(p, total, (float *)lds, RB * 16, rows, m0, tile, wk, wks, wn, tile_n, lane);
}

// The same for rows of 16-bit or int8 elements that begin at 16 bytes: x goes straight to LDS as it lies, a round ahead, codes
// two rounds ahead to registers; a step's codes are put in x's order instead.  x alone, all of it for each tile, comes from the
// L2 in 8 us where the codes take 7 (whole lines; in halves, 21); what bounds it is the vector instructions, 13 for eight codes, 4
// for a group's sums of 16 products, 290 in all for 32 products, which the two waves of a SIMD issue nearly in turn with those.
// us, here and through registers: 61 rows 5120 -> 13824 float16 24.0 and 30.4; 64 rows 8192 -> 16384 bfloat16 35 and 42;
// 64 rows 8192 -> 8192 int8 17.7 and 22.6; 32 rows 4096 -> 4096, groups of 32, 9.4 and 12.2.  The next step's weights made between
// this step's products, by scheduling barriers, spilled for half of the types.
template <int RB, int NB, int GS, bool WIDE>
__global__ __launch_bounds__(512, 2) void w4_ring_kernel(const W4Params p) {
  constexpr int WK = kW4Shared[RB / 2], STEPS = X == X_I8 ? 2 : 4, PF = 16 / XB, BUFFER = WK * STEPS * RB * 1024, LOADS = BUFFER / 1024 / kW4Waves;
  constexpr int OURS = NB * (1 + 2 * (4 / GS));  // loads of a block of codes
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, mr = lane & 15;
  const int wk = wave % WK, wn = wave / WK;
  constexpr int tile_n = kW4Waves / WK * NB * 16;
  const int tile = tile_of(p);
  const int64_t m0 = (int64_t)blockIdx.y * (RB * 16);
  const int rows = (int)min((int64_t)(RB * 16), p.a.rows - m0), rounds = (p.blocks + WK - 1) / WK;
  // from a round on that differs between tiles: rows of x often lie a power of two apart, and all tiles at the same place of all
  // rows would meet in a few channels of the L2
  const int from = tile % rounds;
  const auto turned = [&](int round) {
    const int i = round + from;
    return i < rounds ? i : i - rounds;
  };
  // A load brings 128 bytes of 8 rows, whole lines; which lane has which of a row's pieces turns with the row, so that a
  // fragment's 16 rows lie in different banks.
  constexpr int R8 = 2 * RB, ALONG = 8 * PF;
  const int r8 = wave % R8, mine = ((lane & 7) ^ (lane >> 3) ^ (r8 & 1)) * PF + wave / R8 * ALONG;
  const char *x_lane = (const char *)p.a.x + (m0 + min(r8 * 8 + (lane >> 3), rows - 1)) * p.a.x_stride * XB;
  const auto bring = [&](int round, unsigned char *to) {
    const int first = round * (WK * kW4Block);
    if (first + WK * kW4Block <= p.k) {
      const char *from = x_lane + (uint32_t)(first + mine) * XB;
#pragma unroll
      for (int i = 0; i < LOADS; i++) to_lds<16>(to + (wave + kW4Waves * i) * 1024, from + i * (kW4Waves / R8 * 128));
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; i++) {
        const int k = first + mine + i * (kW4Waves / R8 * ALONG);
        to_lds<16>(to + (wave + kW4Waves * i) * 1024, x_lane + (k + PF <= p.k ? (uint32_t)k * XB : 0u));
      }
    }
  };
  const int x_at0 = (mr >> 3) * 1024 + (mr & 7) * 128 + (g ^ (mr & 7) ^ (mr >> 3)) * 16;
  const Weights<NB, GS, WIDE> ws(p, tile * tile_n, tile * tile_n + wn * NB * 16, lane);
  typename Weights<NB, GS, WIDE>::Block w[2];
  f32x4 total[NB][RB];  // of rows 4 g to 4 g + 3 of a block of rows
#pragma unroll
  for (int b = 0; b < NB; b++)
#pragma unroll
    for (int m = 0; m < RB; m++) total[b][m] = f32x4{0, 0, 0, 0};
  bring(turned(0), lds);
  __builtin_amdgcn_sched_barrier(0);
  ws.load(w[0], turned(0) * WK + wk);
  __builtin_amdgcn_sched_barrier(0);
  ws.load(w[1], turned(1) * WK + wk);
  for (int r0 = 0; r0 < rounds; r0 += 2) {  // always both
#pragma unroll
    for (int d = 0; d < 2; d++) {
      const int round = turned(r0 + d), block = round * WK + wk;
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<OURS>();
      lds_barrier();
      if ((round + 1) * (WK * kW4Block) > p.k) {  // the last: zeros where a row has no whole piece
#pragma unroll
        for (int i = 0; i < LOADS; i++)
          if (round * (WK * kW4Block) + mine + i * (kW4Waves / R8 * ALONG) + PF > p.k) *(u32x4 *)(lds + d * BUFFER + (wave + kW4Waves * i) * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
        wait_vm<0>();
        lds_barrier();
      }
      bring(turned(r0 + d + 1), lds + (d ^ 1) * BUFFER);
      if (r0 + d < rounds && block < p.blocks) {
        const unsigned char *x = lds + d * BUFFER + wk * (STEPS * RB * 1024);
        const auto x_at = [&](int s, int m, int) { return x + (s >> 1) * (R8 * 1024) + m * 2048 + (x_at0 ^ (s & 1) * 64); };
        if (X == X_F16 || ws.has_zeros) multiply<true, false, true, RB>(ws, w[d], x_at, total);
        else multiply<false, false, true, RB>(ws, w[d], x_at, total);
      }
      __builtin_amdgcn_sched_barrier(0);
      ws.load(w[d], turned(r0 + d + 2) * WK + wk);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();  // also the round past the last
  lds_barrier();
  join<RB, NB, PF>(p, total, (float *)lds, RB * 16, rows, m0, tile, wk, WK, wn, tile_n, lane);
}

template <int GS, bool WIDE>
void run(const W4Params &p, int rb, int nb, dim3 grid, unsigned lds, hipStream_t stream) {
  if (p.few_rows) {
    hipLaunchKernelGGL((w4_few_kernel<GS, WIDE>), grid, dim3(p.waves_n * p.waves_k * 64), lds, stream, p);
  } else if (p.ring) {
    if constexpr (X != X_F32) {
#define CBS_W4_GO(r, n) hipLaunchKernelGGL((w4_ring_kernel<r, n, GS, WIDE>), grid, dim3(512), lds, stream, p)
      if (rb == 4 && nb == 1) CBS_W4_GO(4, 1);
      else if (rb == 4) CBS_W4_GO(4, 2);
      else if (rb == 2 && nb == 1) CBS_W4_GO(2, 1);
      else if (rb == 2 && nb == 2) CBS_W4_GO(2, 2);
      else if (nb == 1) CBS_W4_GO(1, 1);
      else if (nb == 2) CBS_W4_GO(1, 2);
      else if constexpr (GS > 1) {  // not with four scales a block: more registers than there are
        if (rb == 2) CBS_W4_GO(2, 4);
        else CBS_W4_GO(1, 4);
      }
#undef CBS_W4_GO
    }
  } else {
#define CBS_W4_GO(r, n) hipLaunchKernelGGL((w4_kernel<r, n, GS, WIDE>), grid, dim3(512), lds, stream, p)
    if (rb == 1 && nb == 1) CBS_W4_GO(1, 1);
    else if (rb == 1) CBS_W4_GO(1, 2);
    else if (rb == 2 && nb == 1) CBS_W4_GO(2, 1);
    else if (rb == 2) CBS_W4_GO(2, 2);
    else if constexpr (X != X_F32) {
      if (nb == 1) CBS_W4_GO(4, 1);
      else CBS_W4_GO(4, 2);
    }
#undef CBS_W4_GO
  }
}

template <int GS>
void pick(const W4Params &p, int rb, int nb, dim3 grid, unsigned lds, hipStream_t stream) {
  if (p.scale_dtype == CBS_F32) run<GS, true>(p, rb, nb, grid, lds, stream);
  else run<GS, false>(p, rb, nb, grid, lds, stream);
}

}  // namespace

#if CBS_W4_X == 0
hipError_t launch_w4_i8
#elif CBS_W4_X == 1
hipError_t launch_w4_f16
#elif CBS_W4_X == 2
hipError_t launch_w4_bf16
#else
hipError_t launch_w4_f32
#endif
    (const W4Params &p, int rb, int nb, dim3 grid, unsigned lds, hipStream_t stream) {
  if (p.group == 32) pick<1>(p, rb, nb, grid, lds, stream);
  else if (p.group == 64) pick<2>(p, rb, nb, grid, lds, stream);
  else pick<4>(p, rb, nb, grid, lds, stream);
  return hipGetLastError();
}

}  // namespace cbs
