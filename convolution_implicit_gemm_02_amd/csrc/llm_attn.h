// llm_attn.h -- between the host side of paged attention (llm_host.cpp) and its kernels (llm_attn.hip, one translation unit
// per pair of query and cache type).
#pragma once
#include "cbs_internal.h"
#include "llm_internal.h"

namespace cbs {

// Work is cut in units -- a sequence, a head of the cache and a block of rows, a row being a new token's query of one of the
// heads that share the cache's -- and each unit's keys in `splits` ranges, one per workgroup, joined by the last to arrive.
constexpr int kAttnRows = 16;         // rows of a unit: the columns of one matrix instruction
constexpr int kAttnMaxSplits = 32;
constexpr int kAttnMaxParts = 1024;   // workgroups of a call whose units are split: as many partial results are kept
constexpr int kAttnMaxChunkParts = 256;
constexpr int kAttnThreads = 256, kAttnChunkThreads = 512;  // of a workgroup: units of 16 rows, of many

struct AttnParams {
  cbs_attn_args a;
  int dim, page, kv_heads, group;  // group: heads that share one of the cache
  int causal, window;
  float scale;                     // of q . k, times log2(e): exponentials are powers of two
  int row_blocks, splits;
  int chunk;                       // units of chunk_rows() rows
  int join_blocks;                 // workgroups that join such a unit's parts
  FastDiv by_join;
  FastDiv by_page, by_group, by_splits, by_row_blocks, by_kv_heads;
  float *part;                     // [unit][split]: a row's maxima, sums, then its output, see part_floats()
  unsigned *tickets;               // [unit], zero between launches
};

// Floats of one split's partial result: maxima and sums of the rows, then their unnormalised outputs.
inline __host__ __device__ int part_floats(int dim) { return kAttnRows * (dim + 2); }

// Units of n rows, n a power of two; not by a sum or a unit's last row, which may leave 31 bits.
inline __host__ __device__ constexpr int units_of(int rows, int n) { return rows / n + (rows % n != 0); }

// Rows of a unit where there are many, and the same of such a unit.
inline __host__ __device__ constexpr int chunk_rows(int dim) { return dim > 128 ? 128 : 256; }
inline __host__ __device__ constexpr int64_t chunk_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// By (dtype, cache_dtype): bf16 on bf16, bf16 on int8, f16 on f16, f16 on int8, f32 on int8.
hipError_t launch_attn_pair_0(const AttnParams &p, unsigned grid, hipStream_t stream);
hipError_t launch_attn_pair_1(const AttnParams &p, unsigned grid, hipStream_t stream);
hipError_t launch_attn_pair_2(const AttnParams &p, unsigned grid, hipStream_t stream);
hipError_t launch_attn_pair_3(const AttnParams &p, unsigned grid, hipStream_t stream);
hipError_t launch_attn_pair_4(const AttnParams &p, unsigned grid, hipStream_t stream);

}  // namespace cbs
