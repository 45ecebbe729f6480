// llm_attn.hip -- attention of new tokens over a paged cache, on matrix instructions; compiled once per pair of query and
// cache type (-DCBS_ATTN_PAIR=n).
//
// With rows r (queries) and keys j, one pass over the keys holds a running maximum m_r, the sum l_r of 2^(s_rj - m_r) and
// the output's sum O_r of 2^(s_rj - m_r) v_j;  s_rj = (scale log2 e) q_r . k_j.  When a step of keys raises the maximum, l
// and O shrink by 2^(old - new).  Ranges of keys done apart are joined the same way.
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane holds one row's scores after the first
// and feeds them, as they lie, to the second: lane l has row l % 16, and of a step's keys those of its group g = l / 16.  The
// instruction gives group g the rows 4 g to 4 g + 3 of the 16 keys that it was fed; the keys are therefore fed in the order
// that makes the scores of a group belong to GK consecutive keys, the ones whose values the group's lanes read as one
// 16-byte piece of V^T.  No score crosses a lane; only the maximum is taken over the four lanes of a row.
//
// Weights that meet float16 values are float16, whose smallest is 2^-24: many keys of small weight would be lost to O and not to
// l.  They are taken times a power of two, which O / l does not have, so that the largest is 2^15: weights down to 2^-39 of the
// largest (long chunks, whose maximum may lag by 2^8: 2^-31) count.
#include <type_traits>

#include "llm_attn.h"

namespace cbs {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));
typedef f16_t f16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kPairQ[5] = {CBS_BF16, CBS_BF16, CBS_F16, CBS_F16, CBS_F32};
constexpr int kPairC[5] = {CBS_BF16, CBS_I8, CBS_F16, CBS_I8, CBS_I8};

__device__ __forceinline__ int fdiv(int n, FastDiv f) { return (int)((__umulhi((unsigned)n, f.magic) + (unsigned)n) >> f.shift); }

template <bool F16>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight floats as N terms of 16 bits whose sum they are: one rounded term, or (bfloat16) two or three that keep 16 or all
// 24 bits.  An infinity or NaN stays whole in the first.
template <bool F16, int N>
__device__ __forceinline__ void split8(const float *x, u32x4 *terms) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; i++) rest[i] = x[i];
#pragma unroll
  for (int n = 0; n < N; n++) {
    if constexpr (F16) {
      f16x8 t;
#pragma unroll
      for (int i = 0; i < 8; i++) t[i] = (f16_t)rest[i];
      terms[n] = __builtin_bit_cast(u32x4, t);
    } else {
      bf16x8 t;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        t[i] = (bf16_t)rest[i];
        if (n + 1 < N) rest[i] = __builtin_isfinite((float)t[i]) ? rest[i] - (float)t[i] : 0.0f;
      }
      terms[n] = __builtin_bit_cast(u32x4, t);
    }
  }
}

// Eight int8 codes as 16-bit floats (exact).  float16: code + 128 in the low bits of 1024, less 1152.
template <bool F16>
__device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi) {
  u32x4 r;
  if constexpr (F16) {
    const f16x2 off = {(f16_t)1152.0f, (f16_t)1152.0f};
    const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t two = __builtin_amdgcn_perm(0x64646464u, w[i / 2], i % 2 ? 0x04030402u : 0x04010400u);
      r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, two) - off);
    }
  } else {
    asm("" : "+v"(lo), "+v"(hi));  // widened here, not where they were loaded: four times the registers
    bf16x8 t;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      t[i] = (bf16_t)(float)(int8_t)(lo >> (8 * i));
      t[4 + i] = (bf16_t)(float)(int8_t)(hi >> (8 * i));
    }
    r = __builtin_bit_cast(u32x4, t);
  }
  return r;
}

__device__ __forceinline__ u32x4 load16(const void *p) {
  u32x4 v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, 16), 16);
  return v;
}

// Where piece c of a key's row lies in LDS, and the piece that lies at a place: turned by the key, which a read's 16 lanes have
// as 8 (mr / 4) + mr % 4.
template <int DS>
__device__ __forceinline__ int turn(int key, int c) {
  if constexpr (DS == 3) {  // rows of 12 pieces differ in their banks by themselves, but for every eighth
    const int at = c + ((key >> 3) & 3);
    return at >= 12 ? at - 12 : at;
  } else {
    return c ^ (((key & 3) | ((key >> 3) & 3) << 2) & (4 * DS - 1));
  }
}
template <int DS>
__device__ __forceinline__ int unturn(int key, int at) {
  if constexpr (DS == 3) {
    const int c = at - ((key >> 3) & 3);
    return c < 0 ? c + 12 : c;
  } else {
    return turn<DS>(key, at);
  }
}

// Partial results pass between workgroups of different XCDs: written through to memory and read past the caches.
__device__ __forceinline__ void put(float *p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float get(const float *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t get2(const float *p) { return __hip_atomic_load((const uint64_t *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// A sequence's new tokens and keys, and what a block of rows sees of them.
struct Seq {
  int start, count, length, rows;
};
__device__ __forceinline__ Seq seq_of(const AttnParams &p, int b) {
  Seq s;
  const int tokens = (int)p.a.tokens;
  s.start = min(max(p.a.q_start[b], 0), tokens);
  s.count = min(max(p.a.q_start[b + 1], s.start), tokens) - s.start;
  const int64_t room = p.a.pages > 0 ? min((int64_t)p.a.columns * p.page, (int64_t)0x7fffff00) : 0;
  s.length = (int)min((int64_t)max(p.a.kv_len[b], 0), room);
  s.rows = s.count * p.group;
  return s;
}
// First and last key that new token i sees.
__device__ __forceinline__ int first_key(const AttnParams &p, const Seq &s, int i) {
  return p.window > 0 ? max(0, max(0, s.length - s.count + i) - p.window + 1) : 0;  // a place before the first key sees what that place does: no sum leaves 31 bits
}
__device__ __forceinline__ int last_key(const AttnParams &p, const Seq &s, int i) {
  return p.causal ? min(s.length - s.count + i, s.length - 1) : s.length - 1;
}
// The page that holds key j of sequence b, -1 if there is none.
__device__ __forceinline__ int page_of(const AttnParams &p, const Seq &s, int b, int j) {
  if (j < 0 || j >= s.length) return -1;
  const int pg = p.a.table[b * p.a.table_stride + fdiv(j, p.by_page)];
  return pg < p.a.pages ? pg : -1;
}

// A unit of few rows.  Four waves take steps of 64 (int8) or 32 keys in turn, keys and values straight to registers: with
// few rows the cost is to read the cache, once, and what each wave holds in flight (the next step's keys during a step, its
// values during the scores) covers the memory's latency; nothing of it is shared between waves.  32 sequences, a token each of 32
// heads over 8 of int8 and 8192 tokens: 94 us, 4.6 TB/s; one sequence over 1000 tokens: 12.6 us, of which the data is 1: lengths,
// pages, keys, values, and the join of the splits, one after the other.
template <int QK, int CK, int DS, bool PAD>
__global__ __launch_bounds__(kAttnThreads, QK == CBS_F32 || DS > 4 ? 1 : 2) void attn_rows_kernel(const AttnParams p) {
  constexpr bool I8 = CK == CBS_I8, SF16 = QK == CBS_F16, PF16 = CK == CBS_F16;
  // float32 queries and weights as three bfloat16 terms, all 24 bits; float16 rows on int8 values: weight times the value's
  // step leaves float16's range, so two bfloat16 terms; else the weights are rounded once to the 16-bit type
  constexpr int NQ = QK == CBS_F32 ? 3 : 1, NP = QK == CBS_F32 ? 3 : I8 && QK == CBS_F16 ? 2 : 1;
  constexpr int TILE = I8 ? 64 : 32, GK = TILE / 4, NB = TILE / 16;  // keys of a step, of a group; blocks of 16 keys
  constexpr int DB = 2 * DS, BYTES = I8 ? 1 : 2;
  constexpr int KP = I8 ? DS / 2 : DS;                               // 16-byte pieces of a key; an odd int8 step has 8 more
  constexpr bool ODD = I8 && DS % 2 == 1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, mr = lane & 15;
  const int dim = PAD ? p.dim : DS * 32;

  const int split = p.splits > 1 ? (int)blockIdx.x - fdiv(blockIdx.x, p.by_splits) * p.splits : 0;
  const int unit = p.splits > 1 ? fdiv(blockIdx.x, p.by_splits) : (int)blockIdx.x;
  const int sh = fdiv(unit, p.by_row_blocks), block = unit - sh * p.row_blocks;
  const int b = fdiv(sh, p.by_kv_heads), kvh = sh - b * p.kv_heads;
  const Seq s = seq_of(p, b);

  __shared__ float s_o[4][kAttnRows][132];
  __shared__ float s_m[4][kAttnRows], s_l[4][kAttnRows], s_w[kAttnMaxSplits][kAttnRows], s_sum[kAttnMaxSplits][kAttnRows], s_total[kAttnRows];
  __shared__ int s_last;

  // blocks of rows beyond those that the grid was made for: the first split takes all their keys
  for (int rb = block; rb < units_of(s.rows, kAttnRows); rb += p.row_blocks) {
    const int splits = rb == block ? p.splits : 1;
    if (split >= splits) break;
    const int r0 = rb * kAttnRows, rows = min(kAttnRows, s.rows - r0);
    const int token0 = fdiv(r0, p.by_group), token1 = fdiv(r0 + rows - 1, p.by_group);
    const int row = min(r0 + mr, s.rows - 1), token = fdiv(row, p.by_group), head = kvh * p.group + row - token * p.group;
    const int lo = first_key(p, s, token0), hi = last_key(p, s, token1);  // of all the block's rows
    const int row_lo = first_key(p, s, token), row_hi = last_key(p, s, token);
    const int all_lo = first_key(p, s, token1), all_hi = last_key(p, s, token0);

    // queries: group g's features of step d, in the order in which the keys' pieces hold them
    u32x4 qf[NQ][DS];
    {
      const int64_t at = (int64_t)(s.start + token) * p.a.q_token_stride + (int64_t)head * p.a.q_head_stride;
#pragma unroll
      for (int d = 0; d < DS; d++) {
        const int f = I8 && d < (DS & ~1) ? 64 * (d / 2) + 16 * g + 8 * (d % 2) : 32 * d + 8 * g;
        float x[8];
        if (!PAD || f < dim) {
          if constexpr (QK == CBS_F32) {
            const Vec<float, 8> v = load_vec<float, 8>((const float *)p.a.q + at + f);
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = v.v[i];
            u32x4 t[NQ];
            split8<false, NQ>(x, t);
#pragma unroll
            for (int n = 0; n < NQ; n++) qf[n][d] = t[n];
          } else {
            __builtin_memcpy(&qf[0][d], (const uint16_t *)p.a.q + at + f, 16);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NQ; n++) qf[n][d] = u32x4{0, 0, 0, 0};
        }
      }
    }

    f32x4 o[DB];
#pragma unroll
    for (int d = 0; d < DB; d++) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    int t0 = 0, t1 = 0;
    if (hi >= lo) {
      const int first = lo / TILE, n = hi / TILE - first + 1;
      t0 = first + (int)((int64_t)n * split / splits);
      t1 = first + (int)((int64_t)n * (split + 1) / splits);
    }

    u32x4 kr[NB][KP > 0 ? KP : 1];
    u32x2 ko[NB];
    // key block kb's row mr, in the order explained above
    const auto fetch = [&](int t, int page) {
      const int j = t * TILE + GK * (mr >> 2);
      const int64_t key = ((int64_t)max(page, 0) * p.kv_heads + kvh) * p.page + (j - fdiv(j, p.by_page) * p.page) + (mr & 3);
      const char *at = (const char *)p.a.k_cache + key * dim * BYTES;
#pragma unroll
      for (int kb = 0; kb < NB; kb++) {
        const char *row_at = at + (8 * (kb / 2) + 4 * (kb % 2)) * dim * BYTES;
#pragma unroll
        for (int c = 0; c < KP; c++) {
          const int f = (I8 ? 64 : 32) * c + (I8 ? 16 : 8) * g;
          if (PAD) {
            kr[kb][c] = load16(row_at + (f < dim ? f * BYTES : 0));
            if (!I8 && f >= dim) kr[kb][c] = u32x4{0, 0, 0, 0};  // int8: the query's zero is enough
          } else {
            kr[kb][c] = load16(row_at + f * BYTES);
          }
        }
        if constexpr (ODD) {
          const int f = 32 * (DS - 1) + 8 * g;
          __builtin_memcpy(&ko[kb], row_at + (!PAD || f < dim ? f : 0), 8);
        }
      }
    };

    int t = t0 + wave;
    int kpage = t < t1 ? page_of(p, s, b, t * TILE + GK * (mr >> 2)) : -1, vpage = t < t1 ? page_of(p, s, b, t * TILE + GK * g) : -1;
    if (t < t1) fetch(t, kpage);
    for (; t < t1; t += 4) {
      // this step's values, the next one's pages
      const int base = t * TILE, j0 = base + GK * g;
      const int place = j0 - fdiv(j0, p.by_page) * p.page;
      const int64_t vunit = (int64_t)max(vpage, 0) * p.kv_heads + kvh;
      const char *vat = (const char *)p.a.v_cache + ((vunit * dim + mr) * p.page + place) * BYTES;
      u32x4 vr[DB];
#pragma unroll
      for (int d = 0; d < DB; d++)
        if (!PAD || 16 * d < dim) vr[d] = load16(vat + (int64_t)(16 * d) * p.page * BYTES);
      Vec<float, GK> ks, vs;
      if constexpr (I8) {
        ks = load_vec<float, GK>(p.a.k_scale + vunit * p.page + place);
        vs = load_vec<float, GK>(p.a.v_scale + vunit * p.page + place);
      }
      const bool ok = vpage >= 0;
      const bool full = base >= all_lo && base + TILE - 1 <= all_hi && __all(ok);
      int kpage2 = -1, vpage2 = -1;
      if (t + 4 < t1) {
        kpage2 = page_of(p, s, b, base + 4 * TILE + GK * (mr >> 2));
        vpage2 = page_of(p, s, b, base + 4 * TILE + GK * g);
      }

      __builtin_amdgcn_sched_barrier(0);  // loads first; and no product's operands before its turn, which would not fit the registers
      // scores: element 4 kb + i is key j0 + 8 (kb / 2) + 4 (kb % 2) + i = j0 + 4 kb + i
      float sc[GK];
#pragma unroll
      for (int kb = 0; kb < NB; kb++) {
        f32x4 acc = {0, 0, 0, 0};
        if (I8 && kb > 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < DS; d++) {
          u32x4 kf;
          if constexpr (!I8)
            kf = kr[kb][d];
          else if (ODD && d == DS - 1)
            kf = widen8<SF16>(ko[kb][0], ko[kb][1]);
          else
            kf = d % 2 ? widen8<SF16>(kr[kb][d / 2][2], kr[kb][d / 2][3]) : widen8<SF16>(kr[kb][d / 2][0], kr[kb][d / 2][1]);
#pragma unroll
          for (int n = NQ - 1; n >= 0; n--) acc = mma<SF16>(kf, qf[n][d], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) sc[4 * kb + i] = acc[i] * (I8 ? ks.v[4 * kb + i] * p.scale : p.scale);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (t + 4 < t1) fetch(t + 4, kpage2);
      __builtin_amdgcn_sched_barrier(0);

      if (!full) {
#pragma unroll
        for (int i = 0; i < GK; i++)
          if (!(ok && j0 + i >= row_lo && j0 + i <= row_hi)) sc[i] = -INFINITY;
      }
      float top = sc[0];
#pragma unroll
      for (int i = 1; i < GK; i++) top = fmaxf(top, sc[i]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > m)) {
        const float up = fmaxf(m, top), keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - up);
        m = up;
        l *= keep;
#pragma unroll
        for (int d = 0; d < DB; d++) o[d] *= keep;
      }
      const float from = m == -INFINITY ? 0.0f : m - (PF16 ? 15.0f : 0.0f);  // weights up to 2^15
#pragma unroll
      for (int i = 0; i < GK; i++) {
        sc[i] = __builtin_amdgcn_exp2f(sc[i] - from);
        l += sc[i];
        if constexpr (I8) sc[i] = full || sc[i] != 0.0f ? sc[i] * vs.v[i] : 0.0f;  // a hidden key's step may be anything
      }
      u32x4 pf[NB / 2][NP];
#pragma unroll
      for (int u = 0; u < NB / 2; u++) split8<PF16, NP>(sc + 8 * u, pf[u]);

      // values that are infinite or NaN: hidden ones must not meet a weight of zero
      bool wild = false;
      if constexpr (!I8) {
        if (!full) {
          constexpr uint32_t EXP = PF16 ? 0x7c00u : 0x7f80u;
          u32x4 keep;
#pragma unroll
          for (int i = 0; i < 4; i++)
            keep[i] = (ok && j0 + 2 * i >= lo && j0 + 2 * i <= hi ? 0xffffu : 0u) | (ok && j0 + 2 * i + 1 >= lo && j0 + 2 * i + 1 <= hi ? 0xffff0000u : 0u);
#pragma unroll
          for (int d = 0; d < DB; d++)
            if (!PAD || 16 * d < dim)
#pragma unroll
              for (int i = 0; i < 4; i++) {
                uint32_t v = vr[d][i] & keep[i];
                if ((v & EXP) == EXP) v &= 0xffff0000u, wild = true;
                if ((v & (EXP << 16)) == EXP << 16) v &= 0xffffu, wild = true;
                vr[d][i] = v;
              }
        }
      }
#pragma unroll
      for (int d = 0; d < DB; d++) {
        if (PAD && 16 * d >= dim) continue;
        if (I8 && d % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < NB / 2; u++) {
          u32x4 vf;
          if constexpr (I8)
            vf = widen8<PF16>(vr[d][2 * u], vr[d][2 * u + 1]);
          else
            vf = vr[d];
#pragma unroll
          for (int n = NP - 1; n >= 0; n--) o[d] = mma<PF16>(vf, pf[u][n], o[d]);
        }
      }
      if constexpr (!I8) {
        if (__any(wild)) {  // rare: add them where they are seen, one key at a time
#pragma unroll 1
          for (int j = max(base, lo); j <= min(base + TILE - 1, hi); j++) {
            const int pg = page_of(p, s, b, j);
            if (pg < 0) continue;
            const uint16_t *at = (const uint16_t *)p.a.v_cache + (((int64_t)pg * p.kv_heads + kvh) * dim + 4 * g) * p.page + (j - fdiv(j, p.by_page) * p.page);
            const bool seen = j >= row_lo && j <= row_hi;
#pragma unroll
            for (int d = 0; d < DB; d++)
              if (!PAD || 16 * d < dim)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                  const uint16_t bits = at[(int64_t)(16 * d + i) * p.page];
                  const float v = PF16 ? (float)__builtin_bit_cast(f16_t, bits) : (float)__builtin_bit_cast(bf16_t, bits);
                  if (seen && !__builtin_isfinite(v)) o[d][i] += v;
                }
          }
        }
      }
      kpage = kpage2;
      vpage = vpage2;
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();  // of a former block of rows
    if (g == 0) s_m[wave][mr] = m, s_l[wave][mr] = l;
    float *part = p.part + ((int64_t)unit * p.splits + split) * part_floats(dim);
    for (int d0 = 0; d0 < dim; d0 += 128) {
      if (d0 > 0) __syncthreads();
#pragma unroll
      for (int d = 0; d < DB; d++)
        if (16 * d >= d0 && 16 * d < d0 + 128) *(f32x4 *)&s_o[wave][mr][16 * d - d0 + 4 * g] = o[d];
      __syncthreads();
      const int width = min(128, dim - d0);
      for (int e = threadIdx.x; e < rows * 128; e += 256) {
        const int r = e >> 7, d = e & 127;
        if (d >= width) continue;
        const float top = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        float sum = 0.0f, total = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const float k = s_m[w][r] == -INFINITY ? (s_l[w][r] == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(s_m[w][r] - top);
          if (k != 0.0f) sum = __builtin_fmaf(s_o[w][r][d], k, sum), total = __builtin_fmaf(s_l[w][r], k, total);
        }
        if (splits == 1) {
          const int out_row = r0 + r, tok = fdiv(out_row, p.by_group), hd = kvh * p.group + out_row - tok * p.group;
          store_f32_as(p.a.out, (int64_t)(s.start + tok) * p.a.out_token_stride + (int64_t)hd * p.a.out_head_stride + d0 + d,
                       total == 0.0f ? 0.0f : sum / total, QK);
        } else {
          put(part + 2 * kAttnRows + r * dim + d0 + d, sum);
          if (d0 + d == 0) put(part + r, top), put(part + kAttnRows + r, total);
        }
      }
    }
    if (splits == 1) continue;

    // join the splits
    __builtin_amdgcn_s_waitcnt(0);  // this wave's part is in memory
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = __hip_atomic_fetch_add(p.tickets + unit, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(splits - 1);
    __syncthreads();
    if (!s_last) continue;
    const float *parts = p.part + (int64_t)unit * splits * part_floats(dim);
    const int stride = part_floats(dim);
    // loads of several parts at a time: each goes to memory
    constexpr int BATCH = 8, PAIRS = 4;
    for (int e = threadIdx.x; e < splits * kAttnRows; e += 256) {
      const int k = e / kAttnRows, r = e % kAttnRows;
      if (r < rows) s_w[k][r] = get(parts + k * stride + r), s_sum[k][r] = get(parts + k * stride + kAttnRows + r);
    }
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += 256) {
      float top = -INFINITY, total = 0.0f;
      for (int k = 0; k < splits; k++) top = fmaxf(top, s_w[k][r]);
      for (int k = 0; k < splits; k++) {
        const float sum = s_sum[k][r];
        const float w = s_w[k][r] == -INFINITY ? (sum == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(s_w[k][r] - top);
        s_w[k][r] = w;
        if (w != 0.0f) total = __builtin_fmaf(sum, w, total);
      }
      s_total[r] = total;
    }
    __syncthreads();
    const int pairs = rows * dim / 2;  // of features
    for (int e0 = threadIdx.x; e0 < pairs; e0 += 256 * PAIRS) {
      int r[PAIRS], at[PAIRS];
      float sum[PAIRS][2];
#pragma unroll
      for (int i = 0; i < PAIRS; i++) {
        const int e = min(e0 + 256 * i, pairs - 1) * 2;
        r[i] = e / dim, at[i] = 2 * kAttnRows + e, sum[i][0] = sum[i][1] = 0.0f;
      }
      for (int k0 = 0; k0 < splits; k0 += BATCH) {
        uint64_t v[PAIRS][BATCH];
#pragma unroll
        for (int i = 0; i < PAIRS; i++)
#pragma unroll
          for (int k = 0; k < BATCH; k++) v[i][k] = get2(parts + min(k0 + k, splits - 1) * stride + at[i]);
#pragma unroll
        for (int i = 0; i < PAIRS; i++)
#pragma unroll
          for (int k = 0; k < BATCH; k++) {
            const float w = k0 + k < splits ? s_w[k0 + k][r[i]] : 0.0f;
            sum[i][0] = w != 0.0f ? __builtin_fmaf(__uint_as_float((uint32_t)v[i][k]), w, sum[i][0]) : sum[i][0];
            sum[i][1] = w != 0.0f ? __builtin_fmaf(__uint_as_float((uint32_t)(v[i][k] >> 32)), w, sum[i][1]) : sum[i][1];
          }
      }
#pragma unroll
      for (int i = 0; i < PAIRS; i++) {
        if (e0 + 256 * i >= pairs) break;
        const int out_row = r0 + r[i], d = at[i] - 2 * kAttnRows - r[i] * dim, tok = fdiv(out_row, p.by_group), hd = kvh * p.group + out_row - tok * p.group;
        const int64_t to = (int64_t)(s.start + tok) * p.a.out_token_stride + (int64_t)hd * p.a.out_head_stride + d;
        const float total = s_total[r[i]];
        store_f32_as(p.a.out, to, total == 0.0f ? 0.0f : sum[i][0] / total, QK);
        store_f32_as(p.a.out, to + 1, total == 0.0f ? 0.0f : sum[i][1] / total, QK);
      }
    }
    if (threadIdx.x == 0) __hip_atomic_store(p.tickets + unit, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// LDS of a unit of many rows, in bytes.
template <bool I8, int DS>
struct ChunkLds {
  static constexpr int BYTES = I8 ? 1 : 2;
  static constexpr int PIECES = 4 * DS;  // 16-byte pieces of a key as 16-bit floats
  static constexpr int HALF = (32 * PIECES + kAttnChunkThreads - 1) / kAttnChunkThreads * kAttnChunkThreads * 16;  // keys of a slot, values behind them
  static constexpr int SLOT = 2 * HALF;
  static constexpr int LOADS = I8 ? (4 * 32 * DS + kAttnChunkThreads - 1) / kAttnChunkThreads : HALF / 16 / kAttnChunkThreads;  // of a thread a tile; 16-bit: each of keys, values
  static constexpr bool LATE = DS <= 4;  // a tile's values meet its weights a tile later, for which LDS has to have room
  static constexpr int SLOTS = I8 ? LATE ? 4 : 3 : LATE ? 7 : 4;
  static constexpr int AHEAD = I8 ? LATE ? 4 : 3 : LATE ? SLOTS - 2 : SLOTS - 1;  // tiles on their way; int8: slots of their codes
  static constexpr int RAW = SLOTS * SLOT, RAW_STEPS = LOADS * kAttnChunkThreads * 16;
  static constexpr int RAW_SLOT = RAW_STEPS + 256 * (kAttnChunkThreads / 64);
  static constexpr int ZEROS = RAW + (I8 ? AHEAD * RAW_SLOT : 0);  // values that are none
  static constexpr int TOTAL = ZEROS + (LATE ? 2 * DS * 1024 : 0);
  static_assert(TOTAL <= 156 * 1024, "LDS");
};

// A unit of many rows: eight waves of RB blocks of 16 rows each go through the same keys, tiles of 32 in a ring of LDS slots, the
// next tiles on their way there.  Rows of a key lie whole in LDS, 16-byte pieces turned by the key so that the lanes of a read
// meet in no bank; values as in the cache, 32 keys of a feature.  A running maximum is raised only where a score is 2^8 above
// it: weights are then at most 256.  16-bit caches go straight to their slots; int8 codes come to a ring of their own and are
// widened from there, once for all waves.
//
// Tile t + 1's scores are taken and tile t - 1's values added on the matrix cores while tile t's scores become weights, a few
// instructions of each in turn.  Two sequences of 512 new tokens, 32 heads over 8 of bfloat16 and 8192 tokens: 160 us with the
// join, 760 TFLOP/s, where a large matrix product reaches 1109; the vector instructions of the weights bound it.
template <int QK, int CK, int DS, int RB>
__global__ __launch_bounds__(kAttnChunkThreads, 2) void attn_chunk_kernel(const AttnParams p) {
  constexpr bool I8 = CK == CBS_I8, SF16 = QK == CBS_F16, PF16 = CK == CBS_F16;
  constexpr int NP = I8 && QK == CBS_F16 ? 2 : 1;
  constexpr int DIM = DS * 32, DB = 2 * DS, THREADS = kAttnChunkThreads, WAVES = THREADS / 64, WROWS = RB * 16, ROWS = WROWS * WAVES;
  typedef ChunkLds<I8, DS> L;
  constexpr int CH = L::PIECES, LOADS = L::LOADS, AHEAD = L::AHEAD;
  constexpr int PAGES = 256;  // halves of tiles whose places are at hand
  constexpr bool LATE = L::LATE;
  constexpr int KD = 2, VD = 2;  // pieces read ahead of their products
  constexpr int OPS = I8 ? LOADS + 1 : 2 * LOADS;  // a tile's loads
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  // of a half of a tile: bytes from the cache's begin to its keys, its values, and (int8) their steps; whether its page is one
  __shared__ int64_t s_keys[PAGES], s_values[PAGES], s_steps[I8 ? PAGES : 1];
  __shared__ int s_ok[PAGES], s_wild[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, mr = lane & 15;

  // neighbouring units read the same keys: to one XCD, whose cache then has them
  const int per = gridDim.x >> 3, extra = gridDim.x & 7, xcd = blockIdx.x & 7, index = xcd * per + min(xcd, extra) + ((int)blockIdx.x >> 3);
  const int shs = fdiv(index, p.by_row_blocks), block = index - shs * p.row_blocks;
  const int sh = fdiv(shs, p.by_splits), split = shs - sh * p.splits;
  const int unit = sh * p.row_blocks + block;
  const int b = fdiv(sh, p.by_kv_heads), kvh = sh - b * p.kv_heads;
  const Seq s = seq_of(p, b);

  // where a thread's pieces of a tile come from: bytes from the first place of their half of it
  int off[I8 ? 1 : 2][LOADS];
  bool second[I8 ? 1 : 2][LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; i++) {
    const int e = i * THREADS + tid;
    if constexpr (I8) {  // keys, then values, 16 codes a piece
      const int key = min(e / DS / 2, 31), f = min(max(e - 64 * DS, 0) / 2, DIM - 1);
      const bool value = e >= 64 * DS;
      second[0][i] = value ? e & 1 : key >= 16;
      off[0][i] = value ? f * p.page : (key & 15) * DIM + e % (2 * DS) * 16;
    } else {
      const int key = min(e / CH, 31), c = unturn<DS>(key, e % CH);
      second[0][i] = key >= 16;
      off[0][i] = (key & 15) * DIM * 2 + c * 16;
      const int f = min(e / 4, DIM - 1), vc = (e & 3) ^ ((f >> 2) & 3);
      second[1][i] = vc >= 2;
      off[1][i] = (f * p.page + (vc & 1) * 8) * 2;
    }
  }
  // where a lane reads
  int k_at[DS];
#pragma unroll
  for (int d = 0; d < DS; d++) {
    const int key = 8 * (mr >> 2) + (mr & 3);
    k_at[d] = (key * CH + turn<DS>(key, 4 * d + g)) * 16;  // 4 keys on: as much on, for the turn is the same
  }
  const int v_at = L::HALF + (mr * 4 + (g ^ (mr >> 2))) * 16;
  // scores are taken times a positive scale: a negative one goes into the queries' sign, and zero queries stand for one of zero
  const float scale = p.scale == 0.0f ? 1.0f : __builtin_fabsf(p.scale);
  const uint32_t sign = p.scale < 0.0f ? 0x80008000u : 0u, whole = p.scale == 0.0f ? 0u : ~0u;

  for (int rb = block; rb < units_of(s.rows, ROWS); rb += p.row_blocks) {  // blocks of rows beyond those that the grid was made for: the first split takes all their keys
    const int splits = rb == block ? p.splits : 1;
    if (split >= splits) break;
    const int r0 = rb * ROWS, rows = min(ROWS, s.rows - r0), w0 = r0 + wave * WROWS;
    int t0 = 0, t1 = 0, all_lo, all_hi;  // tiles; keys that all rows see
    {
      const int token0 = fdiv(r0, p.by_group), token1 = fdiv(r0 + rows - 1, p.by_group);
      const int lo = first_key(p, s, token0), hi = last_key(p, s, token1);
      all_lo = first_key(p, s, token1), all_hi = last_key(p, s, token0);
      if (hi >= lo) {
        const int first = lo / 32, n = hi / 32 - first + 1;
        t0 = first + (int)((int64_t)n * split / splits);
        t1 = first + (int)((int64_t)n * (split + 1) / splits);
      }
    }
    u32x4 qf[RB][DS];
#pragma unroll
    for (int m = 0; m < RB; m++) {
      const int row = min(w0 + 16 * m + mr, s.rows - 1), token = fdiv(row, p.by_group), head = kvh * p.group + row - token * p.group;
      const uint16_t *at = (const uint16_t *)p.a.q + (int64_t)(s.start + token) * p.a.q_token_stride + (int64_t)head * p.a.q_head_stride + 8 * g;
#pragma unroll
      for (int d = 0; d < DS; d++) {
        __builtin_memcpy(&qf[m][d], at + 32 * d, 16);
        qf[m][d] = (qf[m][d] ^ sign) & whole;
      }
    }
    f32x4 o[RB][DB];
    constexpr float UP = PF16 ? 7.0f : 0.0f;  // weights up to 2^8, float16 2^15
    float top[RB], l[RB];                     // the maximum, less UP
#pragma unroll
    for (int m = 0; m < RB; m++) {
      top[m] = -INFINITY, l[m] = 0.0f;
#pragma unroll
      for (int d = 0; d < DB; d++) o[m][d] = f32x4{0, 0, 0, 0};
    }

    int page_t = t0;  // places of tiles from here on
    const auto bring_places = [&](int t) {
      page_t = t;
      for (int e = tid; e < PAGES; e += THREADS) {
        const int j = t * 32 + 16 * e, place = j - fdiv(j, p.by_page) * p.page, pg = page_of(p, s, b, j);
        const int64_t first = ((int64_t)max(pg, 0) * p.kv_heads + kvh) * p.page;
        s_keys[e] = (first + place) * DIM * L::BYTES;
        s_values[e] = (first * DIM + place) * L::BYTES;
        if constexpr (I8) s_steps[e] = (first + place) * 4;
        s_ok[e] = pg >= 0;
      }
    };
    const auto issue = [&](int t, int slot) {  // tile t on its way; past the last, the last again, so that each tile has its count
      const int e = (min(t, t1 - 1) - page_t) * 2;
      if constexpr (I8) {
        unsigned char *to = lds + L::RAW + slot * L::RAW_SLOT;
#pragma unroll
        for (int i = 0; i < LOADS; i++) {
          const bool value = i * THREADS + tid >= 64 * DS;
          const char *from = value ? (const char *)p.a.v_cache + s_values[e + second[0][i]] : (const char *)p.a.k_cache + s_keys[e + second[0][i]];
          to_lds<16>(to + (i * THREADS + wave * 64) * 16, from + off[0][i]);
        }
        // the steps of 32 keys and 32 values, for each wave its own
        const char *from = (const char *)(lane < 32 ? p.a.k_scale : p.a.v_scale) + s_steps[e + ((lane >> 4) & 1)];
        to_lds<4>(to + L::RAW_STEPS + wave * 256, from + (lane & 15) * 4);
      } else {
        unsigned char *to = lds + slot * L::SLOT + wave * 1024;
#pragma unroll
        for (int i = 0; i < LOADS; i++) to_lds<16>(to + i * THREADS * 16, (const char *)p.a.k_cache + s_keys[e + second[0][i]] + off[0][i]);
#pragma unroll
        for (int i = 0; i < LOADS; i++) to_lds<16>(to + L::HALF + i * THREADS * 16, (const char *)p.a.v_cache + s_values[e + second[1][i]] + off[1][i]);
      }
    };
    // int8: a thread's codes of a tile from the ring `raw` to their slot, as 16-bit floats
    const auto widen = [&](int raw, int slot) {
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < LOADS; i++) {
          const int e = i * THREADS + tid;
          const u32x4 c = *(const u32x4 *)(lds + L::RAW + raw * L::RAW_SLOT + e * 16);
          unsigned char *to = lds + slot * L::SLOT;
          if (e < 64 * DS) {
            const int key = e / DS / 2, at = e % (2 * DS) * 2;
            *(u32x4 *)(to + (key * CH + turn<DS>(key, at)) * 16) = widen8<SF16>(c[0], c[1]);
            *(u32x4 *)(to + (key * CH + turn<DS>(key, at + 1)) * 16) = widen8<SF16>(c[2], c[3]);
          } else if (e < 128 * DS) {
            const int f = (e - 64 * DS) / 2, at = (e & 1) * 2, by = (f >> 2) & 3;
            *(u32x4 *)(to + L::HALF + (f * 4 + (at ^ by)) * 16) = widen8<PF16>(c[0], c[1]);
            *(u32x4 *)(to + L::HALF + (f * 4 + ((at + 1) ^ by)) * 16) = widen8<PF16>(c[2], c[3]);
          }
        }
      }
    };

    // element [m][kb][i] is key 8 g + 4 kb + i of the tile
    const auto key_piece = [&](int slot, int n) -> u32x4 { return *(const u32x4 *)(lds + slot * L::SLOT + k_at[n % DS] + n / DS * 4 * CH * 16); };
    const auto scores_step = [&](int slot, int n, u32x4 (&kf)[KD], f32x4 (&sc)[RB][2]) {  // step n: kb = n / DS, d = n % DS
      const u32x4 now = kf[n % KD];
      if (n + KD < 2 * DS) kf[n % KD] = key_piece(slot, n + KD);
#pragma unroll
      for (int m = 0; m < RB; m++) sc[m][n / DS] = mma<SF16>(now, qf[m][n % DS], n % DS == 0 ? f32x4{0, 0, 0, 0} : sc[m][n / DS]);
    };
    const auto most_of = [&](const f32x4 (&sc)[2]) {
      const float a = fmaxf(fmaxf(sc[0][0], sc[0][1]), sc[0][2]), c = fmaxf(fmaxf(sc[0][3], sc[1][0]), sc[1][1]);
      return fmaxf(fmaxf(a, c), fmaxf(sc[1][2], sc[1][3]));
    };

    __syncthreads();  // of a former block of rows
    if constexpr (L::LATE) {
      for (int e = tid; e < 2 * DS * 64; e += THREADS) *(u32x4 *)(lds + L::ZEROS + e * 16) = u32x4{0, 0, 0, 0};
    }
    bring_places(t0);
    __syncthreads();
    if (t0 < t1) {
      f32x4 sc[RB][2];
#pragma unroll
      for (int i = 0; i < AHEAD; i++) issue(t0 + i, i);
      if constexpr (I8) {
        wait_vm<OPS *(AHEAD - 1)>();
        widen(0, 0);
        wait_vm<OPS *(AHEAD - 2)>();
        widen(1, 1);
        wait_vm<OPS *(AHEAD - 2)>();
        lds_barrier();
      } else {
        wait_vm<OPS *(AHEAD - 1)>();
        lds_barrier();
      }
      {
        u32x4 kf[KD];
#pragma unroll
        for (int n = 0; n < KD; n++) kf[n] = key_piece(0, n);
#pragma unroll
        for (int n = 0; n < 2 * DS; n++) scores_step(0, n, kf, sc);
      }
      int slot = 0, raw = 0;  // of tile t
      u32x4 pf[RB][NP];       // weights
      if constexpr (LATE) {
#pragma unroll
        for (int m = 0; m < RB; m++)
#pragma unroll
          for (int k = 0; k < NP; k++) pf[m][k] = u32x4{0, 0, 0, 0};
      }
      // values' pieces of a slot, from a multiple of 16 features on
      const auto value_piece = [&](int from, int d) -> u32x4 { return *(const u32x4 *)(lds + from + v_at + d * 1024); };
      const auto add_step = [&](u32x4 v, int d) {
#pragma unroll
        for (int m = 0; m < RB; m++)
#pragma unroll
          for (int k = NP - 1; k >= 0; k--) o[m][d] = mma<PF16>(v, pf[m][k], o[m][d]);
      };
#pragma unroll 1
      for (int t = t0; t < t1; t++) {
        if ((t + AHEAD - page_t) * 2 + 2 > PAGES && t + AHEAD < t1) {  // every 120 tiles or so
          __syncthreads();
          bring_places(t);
          __syncthreads();
        }
        const int next = slot + 1 == L::SLOTS ? 0 : slot + 1, last = slot == 0 ? L::SLOTS - 1 : slot - 1;
        const int spare = !LATE ? last : last == 0 ? L::SLOTS - 1 : last - 1;  // the slot that no tile needs any more
        f32x4 step_k[2], step_v[2];  // int8: of the lane's keys
        [[maybe_unused]] float step_one = 0.0f;  // of the tile's values, a lane's own
        if constexpr (I8) {
          // tile t + 1 is in its slot once all waves are here; t + 2's codes go to the spare one, and t + AHEAD's to where t's were
          const unsigned char *steps = lds + L::RAW + raw * L::RAW_SLOT + L::RAW_STEPS + wave * 256 + 32 * g;
          step_k[0] = *(const f32x4 *)steps, step_k[1] = *(const f32x4 *)(steps + 16);
          step_v[0] = *(const f32x4 *)(steps + 128), step_v[1] = *(const f32x4 *)(steps + 144);
          if (NP > 1) step_one = *(const float *)(lds + L::RAW + raw * L::RAW_SLOT + L::RAW_STEPS + wave * 256 + 128 + (lane & 31) * 4);
          wait_vm<OPS *(AHEAD - 3)>();
          lds_barrier();
          const int raw2 = raw + 2 >= AHEAD ? raw + 2 - AHEAD : raw + 2;
          widen(raw2, spare);
        } else {
          wait_vm<OPS *(AHEAD - 2)>();  // tile t + 1 is there
          lds_barrier();
        }
        const int ok0 = __builtin_amdgcn_readfirstlane(s_ok[(t - page_t) * 2]), ok1 = __builtin_amdgcn_readfirstlane(s_ok[(t - page_t) * 2 + 1]), base = t * 32;
        issue(t + AHEAD, I8 ? raw : spare);
        if constexpr (I8) raw = raw + 1 == AHEAD ? 0 : raw + 1;

        float by = scale;
        if constexpr (I8) {
          by = 1.0f;
#pragma unroll
          for (int m = 0; m < RB; m++)
#pragma unroll
            for (int kb = 0; kb < 2; kb++) sc[m][kb] *= step_k[kb] * scale;
        }
        bool wild = false;
        const bool edge = !(base >= all_lo && base + 31 <= all_hi && ok0 && ok1);
        if (edge) {  // not all rows see all of it
          const bool ok = (g < 2 ? ok0 : ok1) != 0;
          int w1 = w0;
          asm volatile("" : "+s"(w1));  // what is seldom needed is not kept in registers
#pragma unroll
          for (int m = 0; m < RB; m++) {
            const int token = fdiv(min(w1 + 16 * m + mr, s.rows - 1), p.by_group), lo = first_key(p, s, token), hi = last_key(p, s, token);
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const int j = base + 8 * g + i;
              sc[m][i / 4][i % 4] = (ok & (j >= lo) & (j <= hi)) ? sc[m][i / 4][i % 4] : -INFINITY;
            }
          }
          if constexpr (!I8) {  // values that are infinite or NaN: hidden ones must not meet a weight of zero
            bool any = false;
#pragma unroll
            for (int i = 0; i < LOADS; i++) {
              u32x4 *at = (u32x4 *)(lds + slot * L::SLOT + L::HALF + (i * THREADS + tid) * 16), v = *at;
              constexpr uint32_t EXP = PF16 ? 0x7c00u : 0x7f80u;
              bool here = false;
#pragma unroll
              for (int j = 0; j < 4; j++) {
                uint32_t two = v[j];
                if ((two & EXP) == EXP) two &= 0xffff0000u, here = true;
                if ((two & (EXP << 16)) == EXP << 16) two &= 0xffffu, here = true;
                v[j] = two;
              }
              if (here) *at = v;
              any |= here;
            }
            if (lane == 0) s_wild[wave] = 0;
            if (any) s_wild[wave] = 1;
            wait_vm<63>();
            lds_barrier();
            int sum = 0;
#pragma unroll
            for (int w = 0; w < WAVES; w++) sum |= s_wild[w];
            wild = __builtin_amdgcn_readfirstlane(sum);
          }
        }
        if constexpr (I8) {
          // Values' steps that are infinite or NaN: hidden ones must not meet a weight of zero, and none can be taken apart in two terms.
          if (edge || (NP > 1 && __any(!__builtin_isfinite(step_one)))) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < 8; i++)
              if (!__builtin_isfinite(step_v[i / 4][i % 4])) step_v[i / 4][i % 4] = 0.0f, any = true;
            wild = __any(any);
          }
        }
        float most[RB];
        bool rise = false, none = t == t0;  // none: no weights are due
#pragma unroll
        for (int m = 0; m < RB; m++) most[m] = most_of(sc[m]) * by, rise |= most[m] > top[m] + (8.0f + UP);
        if (__any(rise)) {
          if constexpr (LATE) {  // what is due, at the old maxima
            if (!none) {
#pragma unroll
              for (int d = 0; d < DB; d++) add_step(value_piece(last * L::SLOT, d), d);
            }
            none = true;
          }
#pragma unroll
          for (int m = 0; m < RB; m++) {
            most[m] = fmaxf(most[m], __shfl_xor(most[m], 16));
            most[m] = fmaxf(most[m], __shfl_xor(most[m], 32));
            const float up = fmaxf(top[m], most[m] - UP), less = top[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top[m] - up);
            top[m] = up;
            l[m] *= less;
#pragma unroll
            for (int d = 0; d < DB; d++) o[m][d] *= less;
          }
        }
        if (wild) {  // rare: infinities and NaNs where they are seen, one key at a time
          const int end = min(base + 31, s.length - 1);
          int w1 = w0, g1 = g;
          asm volatile("" : "+s"(w1), "+v"(g1));
#pragma unroll 1
          for (int j = base; j <= end; j++) {
            const int pg = page_of(p, s, b, j);
            if (pg < 0) continue;
            const int64_t head = (int64_t)pg * p.kv_heads + kvh;
            const int place = j - fdiv(j, p.by_page) * p.page;
            const float step = I8 ? p.a.v_scale[head * p.page + place] : 1.0f;
            bool seen[RB];
#pragma unroll
            for (int m = 0; m < RB; m++) {
              const int token = fdiv(min(w1 + 16 * m + mr, s.rows - 1), p.by_group);
              seen[m] = j >= first_key(p, s, token) && j <= last_key(p, s, token);
            }
            int64_t at = (head * DIM + 4 * g1) * p.page + place;
#pragma unroll
            for (int d = 0; d < DB; d++) {
#pragma unroll
              for (int i = 0; i < 4; i++) {
                float v;
                if constexpr (I8) v = (float)((const int8_t *)p.a.v_cache)[at + i * p.page] * step;
                else v = load_as_f32(p.a.v_cache, at + i * p.page, CK);
                const float more = __builtin_isfinite(v) ? 0.0f : v;
#pragma unroll
                for (int m = 0; m < RB; m++) o[m][d][i] = seen[m] ? o[m][d][i] + more : o[m][d][i];
              }
              at += 16 * p.page;
              asm volatile("" : "+v"(at));  // one after the other: few registers
            }
          }
          __builtin_amdgcn_s_waitcnt(7 << 4 | 15 << 8);  // its loads: none in flight where the ways meet again
        }
        float from[RB];
#pragma unroll
        for (int m = 0; m < RB; m++) from[m] = top[m] == -INFINITY ? 0.0f : -top[m];

        // pair i of the tile's weights: two keys of a row
        f32x4 sc2[RB][2];
        u32x4 pf2[RB][NP];
        const auto pair = [&](int n) {
          const int m = n / 4, i = n % 4;
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float x = sc[m][i / 2][i % 2 * 2 + e];
            w[e] = __builtin_amdgcn_exp2f(I8 ? x + from[m] : __builtin_fmaf(x, by, from[m]));
          }
          l[m] += w[0] + w[1];
          if constexpr (I8) w[0] *= step_v[i / 2][i % 2 * 2], w[1] *= step_v[i / 2][i % 2 * 2 + 1];
#pragma unroll
          for (int k = 0; k < NP; k++) {
            if constexpr (PF16) {
              pf2[m][k][i] = __builtin_bit_cast(uint32_t, f16x2{(f16_t)w[0], (f16_t)w[1]});
            } else {
              const bf16x2 two = {(bf16_t)w[0], (bf16_t)w[1]};
              pf2[m][k][i] = __builtin_bit_cast(uint32_t, two);
              if (k + 1 < NP) w[0] -= (float)two[0], w[1] -= (float)two[1];
            }
            asm volatile("" : "+v"(pf2[m][k][i]));  // here, not where they are needed
          }
          asm volatile("" : "+v"(l[m]));
        };
        __builtin_amdgcn_sched_barrier(0);
        u32x4 kf[KD], vf[VD];
        const int values = !LATE ? slot * L::SLOT : none ? L::ZEROS - L::HALF : last * L::SLOT;
#pragma unroll
        for (int n = 0; n < KD; n++) kf[n] = key_piece(next, n);
        if constexpr (LATE) {
#pragma unroll
          for (int d = 0; d < VD; d++) vf[d] = value_piece(values, d);
        }
#pragma unroll
        for (int n = 0; n < 2 * DS; n++) {  // DB is 2 DS
          scores_step(next, n, kf, sc2);
          if constexpr (LATE) {
            const u32x4 now = vf[n % VD];
            if (n + VD < DB) vf[n % VD] = value_piece(values, n + VD);
            add_step(now, n);
          } else {
            if (n >= 2 * DS - VD) vf[n - (2 * DS - VD)] = value_piece(values, n - (2 * DS - VD));
          }
#pragma unroll
          for (int i = n * (4 * RB) / (2 * DS); i < (n + 1) * (4 * RB) / (2 * DS); i++) pair(i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int m = 0; m < RB; m++)
#pragma unroll
          for (int k = 0; k < NP; k++) pf[m][k] = pf2[m][k];
        if constexpr (!LATE) {
#pragma unroll
          for (int d = 0; d < DB; d++) {
            const u32x4 now = vf[d % VD];
            if (d + VD < DB) vf[d % VD] = value_piece(values, d + VD);
            add_step(now, d);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int m = 0; m < RB; m++) sc[m][0] = sc2[m][0], sc[m][1] = sc2[m][1];
        slot = next;
      }
      if constexpr (LATE) {
        const int last = slot == 0 ? L::SLOTS - 1 : slot - 1;
#pragma unroll
        for (int d = 0; d < DB; d++) add_step(value_piece(last * L::SLOT, d), d);
      }
      wait_vm<0>();
      lds_barrier();
    }

    // ---- out, or this split's part of it
#pragma unroll
    for (int m = 0; m < RB; m++) {
      l[m] += __shfl_xor(l[m], 16);
      l[m] += __shfl_xor(l[m], 32);
      const int row = w0 + 16 * m + mr;
      if (row >= r0 + rows) continue;
      if (splits == 1) {
        const int token = fdiv(row, p.by_group), head = kvh * p.group + row - token * p.group;
        const float by = l[m] == 0.0f ? 0.0f : 1.0f / l[m];
        typedef typename std::conditional<SF16, f16_t, bf16_t>::type T;
        T *out = (T *)p.a.out + (int64_t)(s.start + token) * p.a.out_token_stride + (int64_t)head * p.a.out_head_stride + 4 * g;
#pragma unroll
        for (int d = 0; d < DB; d++) {
          Vec<T, 4> v;
#pragma unroll
          for (int i = 0; i < 4; i++) v.v[i] = (T)(l[m] == 0.0f ? 0.0f : o[m][d][i] * by);
          store_vec<T, 4>(out + 16 * d, v);
        }
      } else {
        float *part = p.part + ((int64_t)unit * splits + split) * chunk_floats(ROWS, DIM);
        const int r = row - r0;
        if (g == 0) part[r] = top[m], part[ROWS + r] = l[m];
#pragma unroll
        for (int d = 0; d < DB; d++) *(f32x4 *)(part + 2 * ROWS + r * DIM + 16 * d + 4 * g) = o[m][d];
      }
    }
  }
}

// Parts of a unit's rows, joined: a thread has four features of a row.  10 us for the two sequences above: the parts, through
// memory.
template <int QK, int DS, int ROWS>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnParams p) {
  constexpr int DIM = DS * 32, FOURS = DIM / 4, PER = 256 / FOURS;  // rows of a workgroup
  const int unit = fdiv(blockIdx.x, p.by_join), r = ((int)blockIdx.x - unit * p.join_blocks) * PER + (int)threadIdx.x / FOURS, c = threadIdx.x % FOURS;
  const int sh = fdiv(unit, p.by_row_blocks), block = unit - sh * p.row_blocks;
  const int b = fdiv(sh, p.by_kv_heads), kvh = sh - b * p.kv_heads;
  const Seq s = seq_of(p, b);
  const int row = block * ROWS + r;
  if ((int)threadIdx.x >= PER * FOURS || r >= ROWS || row >= s.rows) return;
  const float *parts = p.part + (int64_t)unit * p.splits * chunk_floats(ROWS, DIM);
  float top = -INFINITY, total = 0.0f;
  for (int k = 0; k < p.splits; k++) top = fmaxf(top, parts[(int64_t)k * chunk_floats(ROWS, DIM) + r]);
  f32x4 sum = {0, 0, 0, 0};
  for (int k = 0; k < p.splits; k++) {
    const float *part = parts + (int64_t)k * chunk_floats(ROWS, DIM);
    const float l = part[ROWS + r], w = part[r] == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(part[r] - top);
    if (w != 0.0f) {
      total = __builtin_fmaf(l, w, total);
      sum += *(const f32x4 *)(part + 2 * ROWS + r * DIM + 4 * c) * w;
    }
  }
  const int token = fdiv(row, p.by_group), head = kvh * p.group + row - token * p.group;
  typedef typename std::conditional<QK == CBS_F16, f16_t, bf16_t>::type T;
  Vec<T, 4> v;
#pragma unroll
  for (int i = 0; i < 4; i++) v.v[i] = (T)(total == 0.0f ? 0.0f : sum[i] / total);
  store_vec<T, 4>((T *)p.a.out + (int64_t)(s.start + token) * p.a.out_token_stride + (int64_t)head * p.a.out_head_stride + 4 * c, v);
}

template <int DS>
hipError_t run_chunk(const AttnParams &p, unsigned grid, hipStream_t stream) {
  constexpr int Q = kPairQ[CBS_ATTN_PAIR], C = kPairC[CBS_ATTN_PAIR];
  if constexpr (Q != CBS_F32) {
    constexpr int RB = DS == 8 ? 1 : 2, ROWS = RB * 16 * (kAttnChunkThreads / 64);
    static_assert(ROWS == chunk_rows(DS * 32), "the host cuts the rows");
    hipLaunchKernelGGL((attn_chunk_kernel<Q, C, DS, RB>), dim3(grid), dim3(kAttnChunkThreads), (ChunkLds<C == CBS_I8, DS>::TOTAL), stream, p);
    if (p.splits > 1) {
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((attn_join_kernel<Q, DS, ROWS>), dim3(grid / p.splits * p.join_blocks), dim3(256), 0, stream, p);
    }
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

template <int DS, bool PAD>
hipError_t run_rows(const AttnParams &p, unsigned grid, hipStream_t stream) {
  hipLaunchKernelGGL((attn_rows_kernel<kPairQ[CBS_ATTN_PAIR], kPairC[CBS_ATTN_PAIR], DS, PAD>), dim3(grid), dim3(kAttnThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

#define CBS_ATTN_NAME2(n) launch_attn_pair_##n
#define CBS_ATTN_NAME(n) CBS_ATTN_NAME2(n)
hipError_t CBS_ATTN_NAME(CBS_ATTN_PAIR)(const AttnParams &p, unsigned grid, hipStream_t stream) {
  if (p.chunk) {
    switch (p.dim) {
      case 64: return run_chunk<2>(p, grid, stream);
      case 96: return run_chunk<3>(p, grid, stream);
      case 128: return run_chunk<4>(p, grid, stream);
      default: return run_chunk<8>(p, grid, stream);
    }
  }
  switch (p.dim) {
    case 64: return run_rows<2, false>(p, grid, stream);
    case 96: return run_rows<3, false>(p, grid, stream);
    case 128: return run_rows<4, false>(p, grid, stream);
    case 256: return run_rows<8, false>(p, grid, stream);
    default: return p.dim < 128 ? run_rows<4, true>(p, grid, stream) : run_rows<8, true>(p, grid, stream);
  }
}

}  // namespace cbs
