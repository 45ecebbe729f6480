// llm_host.cpp -- host side of the decoder-step operators: checks of descriptors and arguments, and launches.  The public
// contract is include/cbs_llm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/cbs_llm.h"
#include "cbs_scratch.h"
#include "llm_attn.h"
#include "llm_internal.h"
#include "llm_w4.h"

using namespace cbs;

struct cbs_attn {
  cbs_attn_desc d;
  int device;
  float *part;        // partial results of split units
  unsigned *tickets;  // of their workgroups' arrival, zero between runs
};

namespace {

constexpr int64_t kMaxRows = 0x7fffffff;  // of one call; more than a launch takes go in several
constexpr int64_t kMaxSpan = (int64_t)1 << 46;  // elements from a tensor's first to its last, so that byte offsets fit 64 bits

cbs_status refuse(cbs_status st, const char *where, const char *fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(st, where, buf);
}

bool is_float(int t) { return t == CBS_F32 || t == CBS_F16 || t == CBS_BF16; }
bool is_half(int t) { return t == CBS_F16 || t == CBS_BF16; }
bool aligned(const void *p, uintptr_t by) { return ((uintptr_t)p & (by - 1)) == 0; }

cbs_status launched(hipError_t e, const char *where) {
  return e == hipSuccess ? CBS_OK : refuse(CBS_ELAUNCH, where, "launch: %s", hipGetErrorString(e));
}

// Rows `stride` elements apart: none overlap where `out`.
cbs_status check_rows(const char *where, const char *what, int64_t rows, int64_t stride, int64_t width, bool out) {
  if (stride < 0 || (out && rows > 1 && stride < width))
    return refuse(CBS_EINVAL, where, "%s: a stride of %lld for rows of %lld", what, (long long)stride, (long long)width);
  if (rows > 1 && stride > kMaxSpan / rows) return refuse(CBS_EUNSUPPORTED, where, "%s: the tensor is too long", what);
  return CBS_OK;
}

// Of rows that are read and rows that are written, bytes apart: where they begin in one place, row lies on row.
cbs_status check_same_rows(const char *where, const char *what, int64_t rows, const void *in, int64_t in_pitch, const void *out, int64_t out_pitch) {
  if (!in || in != out || rows < 2 || in_pitch == out_pitch) return CBS_OK;
  return refuse(CBS_EINVAL, where, "%s begins at an input whose rows are %lld bytes apart, its own %lld", what, (long long)in_pitch, (long long)out_pitch);
}

// Vectors of `heads` heads of `tokens` tokens.
cbs_status check_heads(const char *where, const char *what, int64_t tokens, int64_t token_stride, int heads, int64_t head_stride,
                       int dim, bool out) {
  if (head_stride < 0 || token_stride < 0) return refuse(CBS_EINVAL, where, "%s: negative stride", what);
  if ((heads > 1 && head_stride > kMaxSpan / heads) || (tokens > 1 && token_stride > kMaxSpan / tokens))
    return refuse(CBS_EUNSUPPORTED, where, "%s: the tensor is too long", what);
  if (!out || tokens == 0) return CBS_OK;
  // of the two axes, the one with the shorter stride lies within one step of the other
  const bool by_token = tokens == 1 || (heads > 1 && token_stride >= head_stride);
  const int64_t inner = by_token ? (heads - 1) * head_stride : (tokens - 1) * token_stride;
  const bool inner_ok = by_token ? heads == 1 || head_stride >= dim : tokens == 1 || token_stride >= dim;
  const bool outer_ok = by_token ? tokens == 1 || token_stride >= inner + dim : heads == 1 || head_stride >= inner + dim;
  if (!inner_ok || !outer_ok) return refuse(CBS_EINVAL, where, "%s: its vectors overlap", what);
  return CBS_OK;
}

cbs_status check_cache_shape(const char *where, int heads, int head_dim, int page_size) {
  if (heads < 1) return refuse(CBS_EINVAL, where, "%d heads", heads);
  if (head_dim < 1 || page_size < 1) return refuse(CBS_EINVAL, where, "head_dim %d, page_size %d", head_dim, page_size);
  if (head_dim % 16 != 0 || head_dim > 256) return refuse(CBS_EUNSUPPORTED, where, "head_dim %d: multiples of 16 up to 256", head_dim);
  if (page_size % 16 != 0 || page_size > 1024) return refuse(CBS_EUNSUPPORTED, where, "page_size %d: multiples of 16 up to 1024", page_size);
  if (heads > 65535) return refuse(CBS_EUNSUPPORTED, where, "%d heads", heads);
  return CBS_OK;
}

cbs_status check_cache(const char *where, const void *k, const void *v, const float *ks, const float *vs, int cache_dtype,
                       int64_t pages, int64_t page_elems) {
  if (pages < 0) return refuse(CBS_EINVAL, where, "negative pages");
  if (pages == 0) return CBS_OK;  // its pointers, which may be null, are not looked at
  if (!k || !v) return refuse(CBS_EINVAL, where, "null cache");
  if (!aligned(k, 16) || !aligned(v, 16)) return refuse(CBS_EINVAL, where, "the cache does not begin at a 16-byte boundary");
  if ((cache_dtype == CBS_I8) != (ks != nullptr) || (cache_dtype == CBS_I8) != (vs != nullptr))
    return refuse(CBS_EINVAL, where, "an int8 cache has scales, and no other has");
  if (pages > kMaxRows || pages > kMaxSpan / page_elems) return refuse(CBS_EUNSUPPORTED, where, "too many pages");
  return CBS_OK;
}

cbs_status check_kv(const char *where, const cbs_kv_desc *d, const cbs_kv_args *a, bool write) {
  if (!d || !a) return refuse(CBS_EINVAL, where, "null descriptor or arguments");
  cbs_status st = check_cache_shape(where, d->heads, d->head_dim, d->page_size);
  if (st != CBS_OK) return st;
  if (!is_float(d->dtype) || !is_float(d->read_dtype)) return refuse(CBS_EINVAL, where, "dtype %d, read_dtype %d", d->dtype, d->read_dtype);
  if (d->cache_dtype != CBS_I8 && (!is_half(d->cache_dtype) || d->cache_dtype != d->dtype || d->read_dtype != d->cache_dtype))
    return refuse(CBS_EUNSUPPORTED, where, "cache_dtype %d: int8, or the 16-bit type that is written and read", d->cache_dtype);
  if (a->tokens < 0) return refuse(CBS_EINVAL, where, "negative tokens");
  if (a->tokens > kMaxRows / d->heads) return refuse(CBS_EUNSUPPORTED, where, "too many tokens");
  if (a->tokens > 0 && (!a->k || !a->v || !a->slots)) return refuse(CBS_EINVAL, where, "null vectors or slots");
  st = check_cache(where, a->k_cache, a->v_cache, a->k_scale, a->v_scale, d->cache_dtype, a->pages, (int64_t)d->heads * d->head_dim * d->page_size);
  if (st != CBS_OK) return st;
  st = check_heads(where, "keys", a->tokens, a->k_token_stride, d->heads, a->k_head_stride, d->head_dim, !write);
  if (st != CBS_OK) return st;
  return check_heads(where, "values", a->tokens, a->v_token_stride, d->heads, a->v_head_stride, d->head_dim, !write);
}

// How a run is cut.  Two kernels: of units of 16 rows, which each read their keys, and of 256 (128) rows, which share them
// but take longer to begin and to join.  The latter where rows fill two fifths of such a unit and there is work for it, counted
// in keys read by blocks of 16 rows of 128 16-bit features.  us, of 16 and of 256: 2x40 (160 rows a head) over 4096 69 and 38,
// 1x512 (2048) over 16 39 and 33, 4x20 (80) over 4096 of int8 32 and 42, 2x200 (800) over 300 of int8 13 and 32.
// It is the longest sequence's choice for all: 31 single tokens beside a chunk of 512 over 8192 of int8 take 1700, apart 90 and 108.
void cut(const cbs_attn_desc &d, const cbs_attn_args &a, AttnParams *p) {
  const int64_t rows = std::min<int64_t>(a.max_new, a.tokens) * p->group, seqs_heads = (int64_t)a.seqs * d.kv_heads;
  int64_t keys = std::min<int64_t>(a.max_kv, (int64_t)a.columns * d.page_size);
  if (d.window > 0 && d.causal) keys = std::min<int64_t>(keys, (int64_t)d.window + a.max_new);
  const int64_t blocks = (rows + kAttnRows - 1) / kAttnRows;
  const double work = (double)(seqs_heads * blocks) * std::max<double>(0, keys - (d.causal ? a.max_new / 2 : 0)) * d.head_dim / 128 * (d.cache_dtype == CBS_I8 ? 0.6 : 1.0);
  const bool dims = d.head_dim == 64 || d.head_dim == 96 || d.head_dim == 128 || d.head_dim == 256;
  p->chunk = dims && d.dtype != CBS_F32 && rows * 5 >= chunk_rows(d.head_dim) * 2 && work >= 150e3;
  // what a launch takes; a workgroup goes on to the blocks of rows behind them
  const int64_t most_blocks = kMaxThreads / (p->chunk ? kAttnChunkThreads : kAttnThreads) / seqs_heads;
  if (p->chunk) {
    p->row_blocks = (int)std::max<int64_t>(1, std::min((rows + chunk_rows(d.head_dim) - 1) / chunk_rows(d.head_dim), most_blocks));
    const int64_t units = seqs_heads * p->row_blocks;
    // one workgroup on each compute unit; a split's eight tiles pay for its part
    p->splits = units >= kAttnMaxChunkParts ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(kAttnMaxChunkParts / units, keys / 32 / 8));
    const int join_rows = 256 / (d.head_dim / 4);
    p->join_blocks = (chunk_rows(d.head_dim) + join_rows - 1) / join_rows;
    p->by_join = make_fastdiv(p->join_blocks);
    return;
  }
  p->row_blocks = (int)std::max<int64_t>(1, std::min(blocks, most_blocks));
  const int64_t units = seqs_heads * p->row_blocks;
  const int64_t steps = keys / (d.cache_dtype == CBS_I8 ? 64 : 32);
  // As many workgroups as run at a time, with eight steps at least, two for each wave, or four where few splits are to be
  // joined.  us at one, two (chosen) and four times as many: 32x1 over 8192 of int8 125, 96, 108; 4x1 over 4096 20, 21, 42.
  const int resident = d.dtype == CBS_F32 || d.head_dim > 128 ? 256 : 512;
  p->splits = units >= resident ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({(resident + units - 1) / units, std::max(std::min<int64_t>(steps / 4, 8), steps / 8), kAttnMaxSplits}));
}

hipError_t launch_attn(const AttnParams &p, const cbs_attn_desc &d, hipStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)p.a.seqs * d.kv_heads * p.row_blocks * p.splits);
  if (d.dtype == CBS_BF16) return d.cache_dtype == CBS_I8 ? launch_attn_pair_1(p, grid, stream) : launch_attn_pair_0(p, grid, stream);
  if (d.dtype == CBS_F16) return d.cache_dtype == CBS_I8 ? launch_attn_pair_3(p, grid, stream) : launch_attn_pair_2(p, grid, stream);
  return launch_attn_pair_4(p, grid, stream);
}

int log2_up(int64_t n) {
  int l = 0;
  while (((int64_t)1 << l) < n) l++;
  return l;
}

hipError_t launch_w4(const cbs_w4_desc &d, const cbs_w4_args &a, hipStream_t stream) {
  const int x = d.dtype == CBS_I8 ? 0 : d.dtype == CBS_F16 ? 1 : d.dtype == CBS_BF16 ? 2 : 3;
  const int size = kW4Bytes[x];
  // A group that is longer than k is one group all the same: cut to k's blocks, no sum or product of it leaves 31 bits.
  const int group = std::min(d.group, std::max(kW4Block, (d.k + kW4Block - 1) / kW4Block * kW4Block));
  W4Params p = {};
  p.ring = x != 3 && d.k >= kW4Block && (uintptr_t)a.x % 16 == 0 && a.x_stride * size % 16 == 0;
  // Blocks of 16 rows of a workgroup: as many as there are, where its output tiles then fill the card; fewer where not, for more
  // workgroups.  us with 1 | 2 | 4: 64 rows 8192 -> 1024 bfloat16 8.7 | 10.3 | 19.6, 4096 21.1 | 16.2 | 23.0, 8192 39 | 25.9 | 23.7;
  // 32 rows 8192 -> 2048 9.6 | 12.5; float32, 64 rows 4096 -> 4096 19.7 | 29.6, 11008 63 | 40, 32 rows 4096 -> 11008 33.8 | 39.9.
  const int64_t tiles16 = (int64_t)((d.n + 15) / 16) * ((a.rows + 15) / 16);
  const int most_rb = tiles16 <= (x == 3 ? 2048 : 256) ? 1 : tiles16 <= 1024 || x == 3 ? 2 : 4;
  const int rb = std::min(most_rb, a.rows <= 16 ? 1 : a.rows <= 32 ? 2 : 4), stage = rb * 16 * kW4Block * size;
  p.a = a;
  p.k = d.k, p.n = d.n, p.group = group, p.out_dtype = d.out_dtype, p.scale_dtype = d.scale_dtype;
  p.code_stride = (d.k + 31) / 32 * 16;
  p.blocks = (d.k + kW4Block - 1) / kW4Block;
  p.groups = (d.k + group - 1) / group;
  p.by_wide = make_fastdiv(std::max(1, group / kW4Block));
  p.by_whole = make_fastdiv(std::max(1, d.k / 8));
  // All of x in LDS: room for two workgroups on a compute unit, or where x cannot go there straight, one.  us with room for one
  // and without: float32 1 row 4096 -> 4096 7.2 and 15.1, 4 rows 4096 -> 11008 16.7 and 19.1; x that can, 16 rows 4096 -> 4096 of
  // float16 10.6 and 6.5, 8 rows 8192 -> 8192 of bfloat16 15.9 and 13.7.
  const int few = a.rows > 16 ? 0 : 1 << log2_up(a.rows);
  const int64_t few_lds = (int64_t)p.blocks * few * kW4Block * kW4Bytes[x];
  p.few_rows = few_lds <= (p.ring ? kW4Lds / 2 : kW4Lds) ? few : 0;
  int nb = 1, tile_n;
  unsigned lds;
  if (p.few_rows) {
    // Two workgroups for each compute unit; where bringing x is more than an eighth of a workgroup's reading, one.  Waves go
    // along the output features first.  us (1 row, 8192 -> 16384, bfloat16; 8 rows, 8192 -> 28672, int8): two 16.7 and 32.8,
    // one 19.7 and 30.4.
    const int out_blocks = (d.n + 15) / 16;
    const auto share = [&](int groups) {
      const int turns = (out_blocks + groups * kW4Waves - 1) / (groups * kW4Waves);
      return (out_blocks + groups * turns - 1) / (groups * turns);
    };
    p.waves_n = share(512);
    if (a.rows * (x == 0 ? 1 : x == 3 ? 4 : 2) > p.waves_n) p.waves_n = share(256);
    p.waves_k = std::min(kW4Waves / p.waves_n, p.blocks);
    p.by_waves_n = make_fastdiv(p.waves_n);
    p.count = (p.blocks + p.waves_k - 1) / p.waves_k;
    p.from_mask = 0;
    while (2 * p.from_mask + 1 < p.blocks / p.waves_k) p.from_mask = 2 * p.from_mask + 1;
    tile_n = p.waves_n * 16;
    lds = std::max((unsigned)few_lds, 4u * p.few_rows * (tile_n + 4) * p.waves_k);
  } else {
    // A workgroup for each compute unit: tiles of 16 to 256 output features (64 where x goes straight to LDS, a wave's 4 blocks).
    // us there with 1 | 2 | 4 blocks a wave, first the chosen: 32 rows 4096 -> 4096 8.5 | 10.5 | 15.5, 64 rows 8192 -> 8192 17.5 |
    // 23.8; 32 rows 8192 -> 8192 2: 17.6, 1: 25.2, 4: 27.0; 64 rows 8192 -> 16384 2: 36, 1: 48; 32 rows 8192 -> 28672 4: 39.2, 2: 42.1.
    const int64_t wanted = d.n * ((a.rows + rb * 16 - 1) / (rb * 16)) / 256;
    if (p.ring) {
      const int shared = kW4Shared[rb / 2], least = kW4Waves / shared * 16, most = rb == 4 || group == 32 ? 2 : 4;
      while (nb < most && least * nb < wanted) nb *= 2;
      tile_n = least * nb;
      lds = std::max(2u * stage * shared, (unsigned)(4 * rb * 16 * (tile_n + 4)) * shared);
    } else {
      const int room = std::min(kW4Lds / (2 * stage), kW4Most[x][rb / 2] * 2 / rb);  // blocks of x of a round
      int room_log = 0;
      while ((2 << room_log) <= room) room_log++;
      // Two blocks of output features a wave from 64 on, where the fewer reads of x from LDS count more than the waves.
      const int tile_log = std::min(std::max(log2_up(wanted), 4), 8);
      nb = tile_log >= 6 ? 2 : 1;
      p.wk_log = std::min({room_log, log2_up(p.blocks), 7 + nb - 1 - tile_log});
      tile_n = (kW4Waves >> p.wk_log) * nb * 16;
      lds = std::max(2u * stage, (unsigned)(4 * rb * 16 * (tile_n + 4))) << p.wk_log;
    }
  }
  p.tiles = (d.n + tile_n - 1) / tile_n;
  const int64_t row_tiles = (a.rows + rb * 16 - 1) / (rb * 16);
  for (int64_t t = 0; t < row_tiles; t += 65535) {  // a grid's second axis
    W4Params q = p;
    const int64_t m = t * rb * 16;
    q.a.x = (const char *)a.x + m * a.x_stride * (x == 0 ? 1 : x == 3 ? 4 : 2);
    q.a.out = (char *)a.out + m * a.out_stride * (d.out_dtype == CBS_F32 ? 4 : 2);
    if (a.x_scale) q.a.x_scale = a.x_scale + m;
    q.a.rows = a.rows - m;
    const dim3 grid((unsigned)p.tiles, (unsigned)std::min<int64_t>(row_tiles - t, 65535));
    const auto launch = x == 0 ? launch_w4_i8 : x == 1 ? launch_w4_f16 : x == 2 ? launch_w4_bf16 : launch_w4_f32;
    const hipError_t e = launch(q, rb, nb, grid, lds, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

extern "C" {

cbs_status cbs_rms_norm(const cbs_rms_desc *d, const cbs_rms_args *a, void *stream) {
  const char *where = "rms_norm";
  if (!d || !a) return refuse(CBS_EINVAL, where, "null descriptor or arguments");
  if (d->dim < 1) return refuse(CBS_EINVAL, where, "dim %d", d->dim);
  if (d->dim > CBS_RMS_MAX_DIM) return refuse(CBS_EUNSUPPORTED, where, "dim %d: %d at most", d->dim, CBS_RMS_MAX_DIM);
  if (!is_float(d->dtype) || !is_float(d->weight_dtype)) return refuse(CBS_EINVAL, where, "dtype %d, weight_dtype %d", d->dtype, d->weight_dtype);
  if (d->out_dtype != d->dtype && d->out_dtype != CBS_I8) return refuse(CBS_EUNSUPPORTED, where, "out_dtype %d: dtype or int8", d->out_dtype);
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return refuse(CBS_EINVAL, where, "eps %g", d->eps);
  if (a->rows < 0) return refuse(CBS_EINVAL, where, "negative rows");
  if (a->rows > kMaxRows) return refuse(CBS_EUNSUPPORTED, where, "too many rows");
  if (a->rows > 0 && (!a->x || !a->weight || !a->out)) return refuse(CBS_EINVAL, where, "null buffer");
  if (a->residual_out && !a->residual) return refuse(CBS_EINVAL, where, "residual_out without residual");
  if (a->rows > 0 && (d->out_dtype == CBS_I8) != (a->out_scale != nullptr)) return refuse(CBS_EINVAL, where, "int8 output has a scale, and no other has");
  cbs_status st = check_rows(where, "x", a->rows, a->x_stride, d->dim, false);
  if (st == CBS_OK && a->residual) st = check_rows(where, "residual", a->rows, a->residual_stride, d->dim, false);
  if (st == CBS_OK) st = check_rows(where, "out", a->rows, a->out_stride, d->dim, true);
  if (st == CBS_OK && a->residual_out) st = check_rows(where, "residual_out", a->rows, a->residual_out_stride, d->dim, true);
  const int64_t size = d->dtype == CBS_F32 ? 4 : 2, out_pitch = a->out_stride * (d->out_dtype == CBS_I8 ? 1 : size);
  if (st == CBS_OK && a->rows > 0 && a->out == a->residual_out) st = refuse(CBS_EINVAL, where, "out is residual_out");
  if (st == CBS_OK) st = check_same_rows(where, "out", a->rows, a->x, a->x_stride * size, a->out, out_pitch);
  if (st == CBS_OK) st = check_same_rows(where, "out", a->rows, a->residual, a->residual_stride * size, a->out, out_pitch);
  if (st == CBS_OK) st = check_same_rows(where, "residual_out", a->rows, a->x, a->x_stride * size, a->residual_out, a->residual_out_stride * size);
  if (st == CBS_OK) st = check_same_rows(where, "residual_out", a->rows, a->residual, a->residual_stride * size, a->residual_out, a->residual_out_stride * size);
  if (st != CBS_OK || a->rows == 0) return st;
  return launched(launch_rms_norm(*d, *a, (hipStream_t)stream), where);
}

cbs_status cbs_w4_linear(const cbs_w4_desc *d, const cbs_w4_args *a, void *stream) {
  const char *where = "w4_linear";
  if (!d || !a) return refuse(CBS_EINVAL, where, "null descriptor or arguments");
  if (d->k < 1 || d->n < 1) return refuse(CBS_EINVAL, where, "k %d, n %d", d->k, d->n);
  if (d->k > (1 << 24) || d->n > (1 << 24)) return refuse(CBS_EUNSUPPORTED, where, "k %d, n %d: 2^24 at most", d->k, d->n);
  if (d->group < 1) return refuse(CBS_EINVAL, where, "group %d", d->group);
  if (d->group != 32 && d->group != 64 && d->group % 128 != 0) return refuse(CBS_EUNSUPPORTED, where, "group %d: 32, 64 or a multiple of 128", d->group);
  if (!is_float(d->dtype) && d->dtype != CBS_I8) return refuse(CBS_EINVAL, where, "dtype %d", d->dtype);
  if (!is_float(d->out_dtype) || !is_float(d->scale_dtype)) return refuse(CBS_EINVAL, where, "out_dtype %d, scale_dtype %d", d->out_dtype, d->scale_dtype);
  if (a->rows < 0) return refuse(CBS_EINVAL, where, "negative rows");
  if (a->rows > kMaxRows) return refuse(CBS_EUNSUPPORTED, where, "too many rows");
  if (!a->codes || !a->scales) return refuse(CBS_EINVAL, where, "null weights");
  if (!aligned(a->codes, 16)) return refuse(CBS_EINVAL, where, "the codes do not begin at a 16-byte boundary");
  if (a->rows > 0 && (!a->x || !a->out)) return refuse(CBS_EINVAL, where, "null buffer");
  if (a->rows > 0 && (d->dtype == CBS_I8) != (a->x_scale != nullptr)) return refuse(CBS_EINVAL, where, "int8 rows have scales, and no other has");
  cbs_status st = check_rows(where, "x", a->rows, a->x_stride, d->k, false);
  if (st == CBS_OK) st = check_rows(where, "out", a->rows, a->out_stride, d->n, true);
  if (st != CBS_OK || a->rows == 0) return st;
  return launched(launch_w4(*d, *a, (hipStream_t)stream), where);
}

cbs_status cbs_kv_write(const cbs_kv_desc *d, const cbs_kv_args *a, void *stream) {
  const cbs_status st = check_kv("kv_write", d, a, true);
  if (st != CBS_OK || a->tokens == 0) return st;
  return launched(launch_kv_write(*d, *a, (hipStream_t)stream), "kv_write");
}

cbs_status cbs_kv_read(const cbs_kv_desc *d, const cbs_kv_args *a, void *stream) {
  const cbs_status st = check_kv("kv_read", d, a, false);
  if (st != CBS_OK || a->tokens == 0) return st;
  return launched(launch_kv_read(*d, *a, (hipStream_t)stream), "kv_read");
}

cbs_status cbs_attn_create(const cbs_attn_desc *d, cbs_attn **out) {
  const char *where = "attn_create";
  if (!out) return refuse(CBS_EINVAL, where, "out is NULL");
  *out = nullptr;
  if (!d) return refuse(CBS_EINVAL, where, "null descriptor");
  cbs_status st = check_cache_shape(where, d->kv_heads, d->head_dim, d->page_size);
  if (st != CBS_OK) return st;
  if (d->heads < 1 || d->heads % d->kv_heads != 0) return refuse(CBS_EINVAL, where, "%d heads on %d of the cache", d->heads, d->kv_heads);
  if (d->heads > 65535) return refuse(CBS_EUNSUPPORTED, where, "%d heads", d->heads);
  if (!is_float(d->dtype)) return refuse(CBS_EINVAL, where, "dtype %d", d->dtype);
  if (d->cache_dtype != CBS_I8 && (!is_half(d->cache_dtype) || d->cache_dtype != d->dtype))
    return refuse(CBS_EUNSUPPORTED, where, "cache_dtype %d: int8, or the 16-bit dtype", d->cache_dtype);
  if (d->causal != 0 && d->causal != 1) return refuse(CBS_EINVAL, where, "causal %d", d->causal);
  if (d->window < 0) return refuse(CBS_EINVAL, where, "window %d", d->window);
  if (!std::isfinite(d->scale)) return refuse(CBS_EINVAL, where, "scale %g", d->scale);
  if (d->max_seqs < 1 || d->max_seqs > 65535) return refuse(CBS_EINVAL, where, "max_seqs %d: 1 to 65535", d->max_seqs);
  int device = -1;
  if (hipGetDevice(&device) != hipSuccess || device < 0) return refuse(CBS_EDEVICE, where, "no current HIP device");
  cbs_attn *h = new (std::nothrow) cbs_attn;
  if (!h) return refuse(CBS_ENOMEM, where, "out of host memory");
  *h = cbs_attn{*d, device, nullptr, nullptr};
  if (hipMalloc((void **)&h->part, std::max<size_t>(kAttnMaxParts * (size_t)part_floats(d->head_dim), kAttnMaxChunkParts * chunk_floats(chunk_rows(d->head_dim), d->head_dim)) * sizeof(float)) != hipSuccess ||
      hipMalloc((void **)&h->tickets, kAttnMaxParts * sizeof(unsigned)) != hipSuccess) {
    cbs_attn_destroy(h);
    return refuse(CBS_ENOMEM, where, "out of device memory");
  }
  if (hipMemset(h->tickets, 0, kAttnMaxParts * sizeof(unsigned)) != hipSuccess || hipStreamSynchronize(nullptr) != hipSuccess) {
    cbs_attn_destroy(h);
    return refuse(CBS_EDEVICE, where, "clearing the tickets failed");
  }
  *out = h;
  return CBS_OK;
}

cbs_status cbs_attn_run(const cbs_attn *attn, const cbs_attn_args *a, void *stream) {
  const char *where = "attn_run";
  if (!attn || !a) return refuse(CBS_EINVAL, where, "null handle or arguments");
  const cbs_attn_desc &d = attn->d;
  if (a->seqs < 0 || a->seqs > d.max_seqs) return refuse(CBS_EINVAL, where, "%d sequences: the handle takes %d", a->seqs, d.max_seqs);
  if (a->tokens < 0 || a->columns < 0) return refuse(CBS_EINVAL, where, "negative tokens or columns");
  if (a->tokens > kMaxRows / d.heads) return refuse(CBS_EUNSUPPORTED, where, "too many tokens");
  if (a->max_new < 0 || a->max_kv < 0) return refuse(CBS_EINVAL, where, "max_new %d, max_kv %d", a->max_new, a->max_kv);
  if (a->seqs > 0 && (!a->q_start || !a->kv_len || (!a->table && a->columns > 0))) return refuse(CBS_EINVAL, where, "null lengths or table");
  if (a->seqs > 1 && a->table_stride < a->columns) return refuse(CBS_EINVAL, where, "a table stride of %lld for %d columns", (long long)a->table_stride, a->columns);
  if (a->tokens > 0 && (!a->q || !a->out)) return refuse(CBS_EINVAL, where, "null q or out");
  cbs_status st = check_cache(where, a->k_cache, a->v_cache, a->k_scale, a->v_scale, d.cache_dtype, a->pages, (int64_t)d.kv_heads * d.head_dim * d.page_size);
  if (st == CBS_OK) st = check_heads(where, "q", a->tokens, a->q_token_stride, d.heads, a->q_head_stride, d.head_dim, false);
  if (st == CBS_OK) st = check_heads(where, "out", a->tokens, a->out_token_stride, d.heads, a->out_head_stride, d.head_dim, true);
  if (st != CBS_OK || a->tokens == 0 || a->seqs == 0) return st;
  int device = -1;
  if (hipGetDevice(&device) != hipSuccess || device != attn->device) return refuse(CBS_EINVAL, where, "the handle belongs to device %d", attn->device);
  AttnParams p = {};
  p.dim = d.head_dim;
  p.page = d.page_size;
  p.kv_heads = d.kv_heads;
  p.group = d.heads / d.kv_heads;
  p.causal = d.causal;
  p.window = d.window;
  p.scale = d.scale * 1.44269504088896340736f;
  p.by_page = make_fastdiv(p.page);
  p.by_group = make_fastdiv(p.group);
  p.by_kv_heads = make_fastdiv(p.kv_heads);
  p.part = attn->part;
  p.tickets = attn->tickets;
  const int most = (int)(kMaxThreads / kAttnChunkThreads / d.kv_heads);  // sequences of a launch
  for (int b = 0; b < a->seqs; b += most) {
    p.a = *a;
    p.a.seqs = std::min(a->seqs - b, most);
    p.a.q_start += b, p.a.kv_len += b, p.a.table += b * a->table_stride;
    cut(d, p.a, &p);
    p.by_splits = make_fastdiv(p.splits);
    p.by_row_blocks = make_fastdiv(p.row_blocks);
    st = launched(launch_attn(p, d, (hipStream_t)stream), where);
    if (st != CBS_OK) return st;
  }
  return CBS_OK;
}

void cbs_attn_destroy(cbs_attn *attn) {
  if (!attn) return;
  (void)hipFree(attn->part);
  (void)hipFree(attn->tickets);
  delete attn;
}

}  // extern "C"
