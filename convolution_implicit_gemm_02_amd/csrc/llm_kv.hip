// llm_kv.hip -- new keys and values into a paged cache (int8 codes with a step per token and head, or as they are), and back.
#include "cbs_internal.h"
#include "llm_internal.h"

namespace cbs {
namespace {

struct KvParams {
  cbs_kv_desc d;
  cbs_kv_args a;
  FastDiv by_heads, by_page;
  bool far;  // slots past 31 bits
};
__device__ __forceinline__ int fdiv(int n, FastDiv f) { return (int)((__umulhi((unsigned)n, f.magic) + (unsigned)n) >> f.shift); }

// ---- few tokens: one wave per vector of one token and head; blockIdx.y 0: keys, 1: values.  What it costs is a round trip for
// the slot, one for the vector and its reduction.
template <bool WRITE>
__global__ __launch_bounds__(256) void kv_kernel(const KvParams p) {
  const int lane = threadIdx.x % 64;
  const int64_t u = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int heads = p.d.heads, dim = p.d.head_dim, page = p.d.page_size;
  if (u >= p.a.tokens * heads) return;
  const bool val = blockIdx.y;
  const int64_t t = u / heads;
  const int h = (int)(u - t * heads);
  const int64_t slot = p.a.slots[t];
  const bool ok = slot >= 0 && slot < p.a.pages * page;
  const int64_t unit = (ok ? slot / page : 0) * heads + h;  // the page's part for this head
  const int place = ok ? (int)(slot % page) : 0;
  void *vec = val ? p.a.v : p.a.k, *cache = val ? p.a.v_cache : p.a.k_cache;
  float *scale = val ? p.a.v_scale : p.a.k_scale;
  const int64_t at = val ? t * p.a.v_token_stride + h * p.a.v_head_stride : t * p.a.k_token_stride + h * p.a.k_head_stride;
  const int64_t first = unit * page * dim + (val ? place : (int64_t)place * dim), step = val ? page : 1;
  float v[4];
  if constexpr (WRITE) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (lane + 64 * i < dim) {
        v[i] = load_as_f32(vec, at + lane + 64 * i, p.d.dtype);
        top = max(top, abs_bits(v[i]));
      }
    if (!ok) return;
    if (p.d.cache_dtype == CBS_I8) {
      const float s = code_step(__uint_as_float(wave_max_bits(top)));
      if (lane == 0) scale[unit * page + place] = s;
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (lane + 64 * i < dim) ((int8_t *)cache)[first + (lane + 64 * i) * step] = (int8_t)code_of(v[i], s);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (lane + 64 * i < dim) store_f32_as(cache, first + (lane + 64 * i) * step, v[i], p.d.cache_dtype);
    }
  } else {
    const float s = ok && p.d.cache_dtype == CBS_I8 ? scale[unit * page + place] : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (lane + 64 * i < dim) {
        const int64_t c = first + (lane + 64 * i) * step;
        float r = 0.0f;
        if (ok) r = p.d.cache_dtype == CBS_I8 ? (float)((int8_t *)cache)[c] * s : load_as_f32(cache, c, p.d.cache_dtype);
        store_f32_as(vec, at + lane + 64 * i, r, p.d.read_dtype);
      }
  }
}

// ---- many tokens: one wave per 16 tokens of one head.  A token's vector lies on four lanes, lane l's being token l / 4: pieces
// of 16 features, 4 n + l % 4 for n = 0, 1, ...  The value cache has a feature's tokens side by side: vectors turn in LDS, so
// that 16 tokens (or four) whose slots follow one another in a page are one access a feature.
// The cost is the vectors' and the cache's bytes: 8191 tokens of 8 heads of 128 bfloat16 features into int8, in runs, 23 us to
// write and 20 to read back, 2.3 TB/s (a wave per vector: 54 and 43, single bytes to the value cache).
// Vectors (tokens times heads) from which tiles are taken, a wave a vector below; us of tiles | vectors, 8 heads:
//   write, 4096 vectors: 128 bf16 to i8 in runs of 500 5.9 | 6.5, scattered 11.0 | 8.8; 256 bf16 9.0 | 10.8, 17.8 | 17.6
//          8192:         6.6 | 10.0, 13.3 | 13.7;  7.9 | 18.4, 30 | 32
//   read,  4096:         6.1 | 5.1, 10.5 | 5.2;    9.0 | 7.1, 20.9 | 13.7
//          8192:         6.2 | 7.5, 13.5 | 9.6;    6.3 | 12.1, 25 | 27;  16384: 6.8 | 12.1, 16.7 | 18.0;  10.6 | 21.5, 45 | 53
// The host does not see the slots: scattered ones are read at a loss from here to nearly 16384 vectors.
constexpr int kTile = 16;
constexpr int64_t kManyVectors = 8192;
constexpr int64_t kMostVectors = 1 << 29;  // of a launch: a wave has 16, 2^31 threads in all

// A tile's slots, the same in all waves of its heads.
struct Slots {
  int page, place;     // of token lane % 16; page -1 where it has none
  bool whole;          // the 16 follow one another in a page
  uint32_t quads;      // bit j: tokens 4 j to 4 j + 3 do
};
__device__ __forceinline__ Slots slots_of(const KvParams &p, int64_t tile, int lane) {
  Slots s;
  const int t = lane & 15, size = p.d.page_size;
  const int64_t token = tile * kTile + t, slot = p.a.slots[min(token, p.a.tokens - 1)];
  const bool ok = token < p.a.tokens && slot >= 0 && slot < p.a.pages * size;
  const int64_t page = !ok ? 0 : p.far ? slot / size : fdiv((int)slot, p.by_page);  // 64-bit divisions: 24.9 -> 24.4 us of the write above, 19.4 -> 18.5 of the read
  s.page = ok ? (int)page : -1;
  s.place = ok ? (int)(slot - page * size) : 0;
  const int from = (lane & 48) | ((t + 15) & 15);
  const int page1 = __shfl(s.page, from), place1 = __shfl(s.place, from);
  const uint32_t chain = (uint32_t)__ballot(ok && page1 == s.page && place1 + 1 == s.place) & 0xffffu;  // bit t: token t lies right behind t - 1
  s.whole = (chain | 1) == 0xffffu;
  s.quads = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) s.quads |= (((chain >> (4 * j)) & 14) == 14) << j;
  return s;
}
// Byte of the first feature of token t's values in the cache, wave-uniform; -1 where it has none.  Only where all lanes are on: one
// that is off need not hold anything.
template <int B>
__device__ __forceinline__ int64_t values_at(const KvParams &p, const Slots &s, int t, int h) {
  const int page = __builtin_amdgcn_readlane(s.page, t), place = __builtin_amdgcn_readlane(s.place, t);
  return page < 0 ? -1 : (((int64_t)page * p.d.heads + h) * p.d.head_dim * p.d.page_size + place) * B;
}

// Four words of four bytes each, turned: byte i of word j <- byte j of word i.
__device__ __forceinline__ void turn4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(b, a, 0x05040100u), w[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, c, 0x05040100u), w[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// 16 tokens' words of a feature group (E = 4 features of a byte, or 2 of two bytes) as words of four (two) tokens of a feature,
// and back: out[feature][.].
template <int E>
__device__ __forceinline__ void to_features(const uint32_t (&in)[kTile], uint32_t (&out)[E][kTile / E]) {
#pragma unroll
  for (int j = 0; j < kTile / E; j++) {
    if constexpr (E == 4) {
      uint32_t w[4] = {in[4 * j], in[4 * j + 1], in[4 * j + 2], in[4 * j + 3]};
      turn4(w);
#pragma unroll
      for (int i = 0; i < 4; i++) out[i][j] = w[i];
    } else {
      out[0][j] = __builtin_amdgcn_perm(in[2 * j + 1], in[2 * j], 0x05040100u);
      out[1][j] = __builtin_amdgcn_perm(in[2 * j + 1], in[2 * j], 0x07060302u);
    }
  }
}
template <int E>
__device__ __forceinline__ void to_tokens(const uint32_t (&in)[E][kTile / E], uint32_t (&out)[kTile]) {
#pragma unroll
  for (int j = 0; j < kTile / E; j++) {
    if constexpr (E == 4) {
      uint32_t w[4] = {in[0][j], in[1][j], in[2][j], in[3][j]};
      turn4(w);
#pragma unroll
      for (int i = 0; i < 4; i++) out[4 * j + i] = w[i];
    } else {
      out[2 * j] = __builtin_amdgcn_perm(in[1][j], in[0][j], 0x05040100u);
      out[2 * j + 1] = __builtin_amdgcn_perm(in[1][j], in[0][j], 0x07060302u);
    }
  }
}

// 16 features of a token as they lie in the cache: BYTES each.
template <int BYTES>
struct Kept {
  uint32_t w[4 * BYTES];
};

template <bool I8>
__device__ __forceinline__ int pitch_of(int dim) { return dim * (I8 ? 1 : 2) + 16; }  // bytes of a token in LDS

// Features of the values in LDS ([token][pitch]) to the cache.
template <bool I8>
__device__ __forceinline__ void values_out(const KvParams &p, const Slots &s, const unsigned char *lds, int h, int lane) {
  constexpr int E = I8 ? 4 : 2, B = I8 ? 1 : 2, PER = kTile / E;
  const int dim = p.d.head_dim, pitch = pitch_of<I8>(dim);
  const uint32_t step = (uint32_t)p.d.page_size * B;  // from a feature to the next; a page's head is below 2^20 bytes
  char *cache = (char *)p.a.v_cache;
  for (int first = 0; first < dim; first += 64 * E) {
    const bool mine = first + lane * E < dim;  // a lane without features has the last ones, for nothing
    const int f0 = min(first + lane * E, dim - E);
    uint32_t in[kTile], out[E][PER];
#pragma unroll
    for (int t = 0; t < kTile; t++) in[t] = *(const uint32_t *)(lds + t * pitch + f0 * B);
    to_features<E>(in, out);
    const uint32_t off = (uint32_t)f0 * step;
    if (s.whole) {
      char *to = cache + values_at<B>(p, s, 0, h);
      if (mine) {
#pragma unroll
        for (int i = 0; i < E; i++) __builtin_memcpy(to + (off + i * step), out[i], kTile * B);
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (s.quads >> j & 1) {
        char *to = cache + values_at<B>(p, s, 4 * j, h);
        if (mine) {
#pragma unroll
          for (int i = 0; i < E; i++) __builtin_memcpy(to + (off + i * step), &out[i][j * B], 4 * B);
        }
        continue;
      }
#pragma unroll
      for (int t = 4 * j; t < 4 * j + 4; t++) {
        const int64_t at = values_at<B>(p, s, t, h);
        if (at < 0) continue;
        char *to = cache + at;
        if (mine) {
#pragma unroll
          for (int i = 0; i < E; i++) {
            const uint32_t v = out[i][t * B / 4] >> (8 * B * (t % E));
            if constexpr (I8) *(uint8_t *)(to + (off + i * step)) = (uint8_t)v;
            else *(uint16_t *)(to + (off + i * step)) = (uint16_t)v;
          }
        }
      }
    }
  }
}
// And back; zeros where a token has no slot.
template <bool I8>
__device__ __forceinline__ void values_in(const KvParams &p, const Slots &s, unsigned char *lds, int h, int lane) {
  constexpr int E = I8 ? 4 : 2, B = I8 ? 1 : 2, PER = kTile / E;
  const int dim = p.d.head_dim, pitch = pitch_of<I8>(dim);
  const uint32_t step = (uint32_t)p.d.page_size * B;
  const char *cache = (const char *)p.a.v_cache;
  for (int first = 0; first < dim; first += 64 * E) {
    const bool mine = first + lane * E < dim;  // as above
    const int f0 = min(first + lane * E, dim - E);
    uint32_t in[E][PER], out[kTile];
    const uint32_t off = (uint32_t)f0 * step;
    if (s.whole) {
      const char *from = cache + values_at<B>(p, s, 0, h);
      if (mine) {
#pragma unroll
        for (int i = 0; i < E; i++) __builtin_memcpy(in[i], from + (off + i * step), kTile * B);
        to_tokens<E>(in, out);
#pragma unroll
        for (int t = 0; t < kTile; t++) *(uint32_t *)(lds + t * pitch + f0 * B) = out[t];
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (s.quads >> j & 1) {
        const char *from = cache + values_at<B>(p, s, 4 * j, h);
#pragma unroll
        for (int i = 0; i < E; i++) __builtin_memcpy(&in[i][j * B], from + (off + i * step), 4 * B);
        continue;
      }
      uint32_t one[4][E];  // all read, of the cache's first page where a token has none: one wait
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int64_t at = values_at<B>(p, s, 4 * j + k, h);
        const char *from = cache + max(at, (int64_t)0);
#pragma unroll
        for (int i = 0; i < E; i++) {
          if (p.a.pages == 0) one[k][i] = 0;
          else if constexpr (I8) one[k][i] = *(const uint8_t *)(from + (off + i * step));
          else one[k][i] = *(const uint16_t *)(from + (off + i * step));
          if (at < 0) one[k][i] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < E; i++) {
        if constexpr (I8) in[i][j] = one[0][i] | one[1][i] << 8 | one[2][i] << 16 | one[3][i] << 24;
        else in[i][2 * j] = one[0][i] | one[1][i] << 16, in[i][2 * j + 1] = one[2][i] | one[3][i] << 16;
      }
    }
    to_tokens<E>(in, out);
#pragma unroll
    for (int t = 0; t < kTile; t++) *(uint32_t *)(lds + t * pitch + f0 * B) = out[t];
  }
}

// Neighbouring tiles to one XCD: they write to the same lines of the value cache.
__device__ __forceinline__ unsigned near_block() {
  const unsigned per = gridDim.x >> 3, extra = gridDim.x & 7, xcd = blockIdx.x & 7;
  return xcd * per + min(xcd, extra) + (blockIdx.x >> 3);
}

// NP: pieces of 16 features of a lane, 1 (64 features a head) to 4.
template <typename T, bool I8, int NP>
__global__ __launch_bounds__(256) void kv_write_tile_kernel(const KvParams p) {
  constexpr int B = I8 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) unsigned char lds_all[4][kTile * (64 * NP * B + 16)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, heads = p.d.heads, dim = p.d.head_dim, page = p.d.page_size;
  const int u = (int)near_block() * 4 + wave;  // below 2^31
  const int64_t tile = fdiv(u, p.by_heads);
  const int h = u - (int)tile * heads, q = lane & 3;
  if (tile * kTile >= p.a.tokens) return;
  const bool val = blockIdx.y;
  const int64_t token = tile * kTile + lane / 4, row = min(token, p.a.tokens - 1);
  const T *vec = (const T *)(val ? p.a.v : p.a.k) + (val ? row * p.a.v_token_stride + h * p.a.v_head_stride : row * p.a.k_token_stride + h * p.a.k_head_stride);
  Vec<T, 16> x[NP];
#pragma unroll
  for (int n = 0; n < NP; n++) x[n] = load_vec<T, 16>(vec + min((4 * n + q) * 16, dim - 16));
  const Slots s = slots_of(p, tile, lane);
  const int page_no = __shfl(s.page, lane / 4), place = __shfl(s.place, lane / 4);
  const bool ok = page_no >= 0;
  const int64_t unit = (int64_t)max(page_no, 0) * heads + h;

  Kept<B> kept[NP];
  if constexpr (I8) {
    uint32_t top = 0;
    float y[NP][16];
    if constexpr (sizeof(T) == 2) {  // magnitudes of 16 bits, two at a time
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 most = {0, 0};
#pragma unroll
      for (int n = 0; n < NP; n++) {
        uint32_t two[8];
        __builtin_memcpy(two, &x[n], 32);
#pragma unroll
        for (int i = 0; i < 8; i++) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, two[i] & 0x7fff7fffu));
      }
      const uint16_t bits = most[0] > most[1] ? most[0] : most[1];
      top = abs_bits((float)__builtin_bit_cast(T, bits));
    } else {
#pragma unroll
      for (int n = 0; n < NP; n++)
#pragma unroll
        for (int i = 0; i < 16; i++) top = max(top, abs_bits((float)x[n].v[i]));
    }
#pragma unroll
    for (int n = 0; n < NP; n++)
#pragma unroll
      for (int i = 0; i < 16; i++) y[n][i] = (float)x[n].v[i];
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const float step = code_step(__uint_as_float(top));
    if (q == 0 && ok) (val ? p.a.v_scale : p.a.k_scale)[unit * page + place] = step;
#pragma unroll
    for (int n = 0; n < NP; n++) {
      const Vec<int8_t, 16> c = codes_of<16>(y[n], step);
      __builtin_memcpy(&kept[n], &c, 16);
    }
  } else {
#pragma unroll
    for (int n = 0; n < NP; n++) __builtin_memcpy(&kept[n], &x[n], 32);
  }
  if (!val) {
    char *to = (char *)p.a.k_cache + (unit * page + place) * dim * B;
#pragma unroll
    for (int n = 0; n < NP; n++)
      if (ok && (4 * n + q) * 16 < dim) __builtin_memcpy(to + (4 * n + q) * 16 * B, &kept[n], 16 * B);
  } else {
    unsigned char *lds = lds_all[wave];
    const int pitch = pitch_of<I8>(dim);
#pragma unroll
    for (int n = 0; n < NP; n++)
      if ((4 * n + q) * 16 < dim) {
#pragma unroll
        for (int i = 0; i < B; i++) *(u32x4 *)(lds + lane / 4 * pitch + (4 * n + q) * 16 * B + 16 * i) = u32x4{kept[n].w[4 * i], kept[n].w[4 * i + 1], kept[n].w[4 * i + 2], kept[n].w[4 * i + 3]};
      }
    asm volatile("" ::: "memory");  // the wave's own part of LDS: its operations there are in order
    values_out<I8>(p, s, lds, h, lane);
  }
}

template <typename T, bool I8, int NP>
__global__ __launch_bounds__(256) void kv_read_tile_kernel(const KvParams p) {
  constexpr int B = I8 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) unsigned char lds_all[4][kTile * (64 * NP * B + 16)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, heads = p.d.heads, dim = p.d.head_dim, page = p.d.page_size;
  const int u = (int)near_block() * 4 + wave;  // below 2^31
  const int64_t tile = fdiv(u, p.by_heads);
  const int h = u - (int)tile * heads, q = lane & 3;
  if (tile * kTile >= p.a.tokens) return;
  const bool val = blockIdx.y;
  const int64_t token = tile * kTile + lane / 4;
  const Slots s = slots_of(p, tile, lane);
  const int page_no = __shfl(s.page, lane / 4), place = __shfl(s.place, lane / 4);
  const bool ok = page_no >= 0;
  const int64_t unit = (int64_t)max(page_no, 0) * heads + h;
  float step = 1.0f;
  if constexpr (I8)
    if (ok) step = (val ? p.a.v_scale : p.a.k_scale)[unit * page + place];
  Kept<B> kept[NP];
#pragma unroll
  for (int n = 0; n < NP; n++)
#pragma unroll
    for (int i = 0; i < 4 * B; i++) kept[n].w[i] = 0;
  if (!val) {
    const char *from = (const char *)p.a.k_cache + (unit * page + place) * dim * B;
    if (ok) {
#pragma unroll
      for (int n = 0; n < NP; n++) __builtin_memcpy(&kept[n], from + min((4 * n + q) * 16, dim - 16) * B, 16 * B);
    }
  } else {
    unsigned char *lds = lds_all[wave];
    const int pitch = pitch_of<I8>(dim);
    values_in<I8>(p, s, lds, h, lane);
    asm volatile("" ::: "memory");  // the wave's own part of LDS: its operations there are in order
#pragma unroll
    for (int n = 0; n < NP; n++) {
      const int at = min((4 * n + q) * 16, dim - 16) * B;
#pragma unroll
      for (int i = 0; i < B; i++) {
        const u32x4 w = *(const u32x4 *)(lds + lane / 4 * pitch + at + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; j++) kept[n].w[4 * i + j] = w[j];
      }
    }
  }
  if (token >= p.a.tokens) return;
  T *vec = (T *)(val ? p.a.v : p.a.k) + (val ? token * p.a.v_token_stride + h * p.a.v_head_stride : token * p.a.k_token_stride + h * p.a.k_head_stride);
#pragma unroll
  for (int n = 0; n < NP; n++) {
    if ((4 * n + q) * 16 >= dim) continue;
    constexpr int VE = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16; i += VE) {
      Vec<T, VE> y;
      if constexpr (I8) {
#pragma unroll
        for (int j = 0; j < VE; j++) y.v[j] = (T)((float)(int8_t)(kept[n].w[(i + j) / 4] >> (8 * ((i + j) % 4))) * step);
      } else {
        __builtin_memcpy(&y, &kept[n].w[i / 2], 16);
      }
      store_past(vec + (4 * n + q) * 16 + i, y);
    }
  }
}

template <bool WRITE, typename T, bool I8>
hipError_t run_tile(const KvParams &p, hipStream_t stream) {
  const int64_t units = (p.a.tokens + kTile - 1) / kTile * p.d.heads;
  const dim3 grid((unsigned)((units + 3) / 4), 2);
  const int np = (p.d.head_dim + 63) / 64;
#define CBS_KV_GO(n)                                                                                  \
  if constexpr (WRITE) hipLaunchKernelGGL((kv_write_tile_kernel<T, I8, n>), grid, dim3(256), 0, stream, p); \
  else hipLaunchKernelGGL((kv_read_tile_kernel<T, I8, n>), grid, dim3(256), 0, stream, p)
  if (np == 1) { CBS_KV_GO(1); }
  else if (np == 2) { CBS_KV_GO(2); }
  else { CBS_KV_GO(4); }
#undef CBS_KV_GO
  return hipGetLastError();
}

template <bool WRITE>
hipError_t run(const cbs_kv_desc &d, const cbs_kv_args &a, hipStream_t stream) {
  KvParams p = {d, a, make_fastdiv(d.heads), make_fastdiv(d.page_size), a.pages >= ((int64_t)1 << 31) / d.page_size};
  const int kind = WRITE ? d.dtype : d.read_dtype, size = kind == CBS_F32 ? 4 : 2;
  if (a.tokens * d.heads < kManyVectors) {
    hipLaunchKernelGGL(kv_kernel<WRITE>, dim3((unsigned)((a.tokens * d.heads + 3) / 4), 2), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  const int64_t most = kMostVectors / d.heads / kTile * kTile;  // whole tiles: 65535 heads have some
  for (int64_t token = 0; token < a.tokens; token += most) {
    p.a.tokens = a.tokens - token < most ? a.tokens - token : most;
    p.a.slots = a.slots + token;
    p.a.k = (char *)a.k + token * a.k_token_stride * size;
    p.a.v = (char *)a.v + token * a.v_token_stride * size;
    hipError_t e;
    if (d.cache_dtype != CBS_I8) e = kind == CBS_F16 ? run_tile<WRITE, f16_t, false>(p, stream) : run_tile<WRITE, bf16_t, false>(p, stream);
    else if (kind == CBS_F16) e = run_tile<WRITE, f16_t, true>(p, stream);
    else if (kind == CBS_BF16) e = run_tile<WRITE, bf16_t, true>(p, stream);
    else e = run_tile<WRITE, float, true>(p, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_write(const cbs_kv_desc &d, const cbs_kv_args &a, hipStream_t stream) { return run<true>(d, a, stream); }
hipError_t launch_kv_read(const cbs_kv_desc &d, const cbs_kv_args &a, hipStream_t stream) { return run<false>(d, a, stream); }

}  // namespace cbs
