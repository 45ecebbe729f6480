// llm_norm.hip -- RMS norm with the residual's addition, output in the input's type or as int8 codes with a step per row.
#include "llm_internal.h"

namespace cbs {
namespace {

struct NormParams {
  cbs_rms_args a;
  int dim, weight_dtype;
  float eps;
  int waves;  // that share a row; one: a workgroup has four rows
};

constexpr int kNormWaves = 16;

// A row is held in registers from its one read to its one write: chunk c of thread t is the VE = 16 / sizeof(T) elements from
// (c * threads + t) * VE on.  A row costs what it reads and writes, or for few rows two memory round trips and the reductions
// between them.  Loads are never under a condition: a chunk that the row ends in begins early enough to lie in it whole, and its
// elements before its own place count as zeros.  Nothing is written before all of the row has been read, for outputs may be
// inputs.  4096 rows of 5120 bfloat16 with a residual into int8: 26.3 us, 5.6 TB/s (part of it from the caches); one row of 4096:
// 3.5 us.  WB: bytes of a weight; weights are read with the row, but for the longest rows, whose registers they would not fit.
template <typename T, bool I8, int WB, int CH>
__global__ __launch_bounds__(CH > 4 ? 1024 : 512) void rms_norm_kernel(const NormParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr bool EARLY = CH < 8;
  __shared__ float s_sum[kNormWaves];
  __shared__ uint32_t s_top[kNormWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), dim = p.dim, waves = p.waves;
  const int64_t row = waves == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int t = waves == 1 ? lane : threadIdx.x, threads = waves * 64;
  if (row >= p.a.rows) return;  // one wave a row: no barrier below
  const T *x = (const T *)p.a.x + row * p.a.x_stride;
  const bool adds = p.a.residual != nullptr;
  const T *res = adds ? (const T *)p.a.residual + row * p.a.residual_stride : x;  // without one, read for nothing

  Vec<T, VE> v[CH], r[CH];
  uint32_t w[CH][VE * WB / 4];
  const auto weights = [&](int c, int at) { __builtin_memcpy(w[c], (const char *)p.a.weight + at * WB, VE * WB); };
  int place[CH];  // of the first element that the chunk holds
  if (dim >= VE) {
#pragma unroll
    for (int c = 0; c < CH; c++) {
      place[c] = min((c * threads + t) * VE, dim - VE);
      v[c] = load_vec<T, VE>(x + place[c]);
      r[c] = load_vec<T, VE>(res + place[c]);
      if (!EARLY && adds) {  // few registers: added as they come
#pragma unroll
        for (int i = 0; i < VE; i++) v[c].v[i] = (T)((float)v[c].v[i] + (float)r[c].v[i]);
        if (c % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
      if (EARLY) weights(c, place[c]);
    }
  } else {  // less than a chunk: thread 0's first, and never the longest rows' form
#pragma unroll
    for (int c = 0; c < CH; c++) {
      place[c] = 0;
#pragma unroll
      for (int i = 0; i < VE; i++) {
        const int e = min(i, dim - 1);
        v[c].v[i] = x[e], r[c].v[i] = res[e];
        if constexpr (WB == 4) w[c][i] = ((const uint32_t *)p.a.weight)[e];
        else w[c][i / 2] = i % 2 ? w[c][i / 2] | (uint32_t)((const uint16_t *)p.a.weight)[e] << 16 : ((const uint16_t *)p.a.weight)[e];
      }
    }
  }

  // an element is its chunk's own where it lies neither before it nor behind the row
  const auto own = [&](int c, int i) { return place[c] + i >= (c * threads + t) * VE && place[c] + i < dim; };
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int i = 0; i < VE; i++) {
      if (EARLY && adds) v[c].v[i] = (T)((float)v[c].v[i] + (float)r[c].v[i]);
      const float h = own(c, i) ? (float)v[c].v[i] : 0.0f;
      ss = __builtin_fmaf(h, h, ss);
    }
  ss = wave_sum(ss);
  if (waves > 1) {
    if (lane == 0) s_sum[wave] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int k = 0; k < waves; k++) ss += s_sum[k];
  }
  const float rs = rsqrtf(ss / (float)dim + p.eps);

  const auto store = [&](auto *out, int c, const auto &vec) {
    if ((c * threads + t) * VE + VE <= dim) {
      store_past(out + place[c], vec);
    } else {
#pragma unroll
      for (int i = 0; i < VE; i++)
        if (own(c, i)) out[place[c] + i] = vec.v[i];
    }
  };
  if (p.a.residual_out) {
    T *sum = (T *)p.a.residual_out + row * p.a.residual_out_stride;
#pragma unroll
    for (int c = 0; c < CH; c++) store(sum, c, v[c]);
  }
  const auto normed = [&](int c, float (&y)[VE]) {
    if (!EARLY) {  // rows of these have more than a chunk
      weights(c, place[c]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < VE; i++) {
      float weight;
      if constexpr (WB == 4) weight = __uint_as_float(w[c][i]);
      else if (p.weight_dtype == CBS_F16) weight = (float)__builtin_bit_cast(f16_t, (uint16_t)(w[c][i / 2] >> (16 * (i % 2))));
      else weight = __uint_as_float(i % 2 ? w[c][i / 2] & 0xffff0000u : w[c][i / 2] << 16);
      y[i] = (float)v[c].v[i] * rs * weight;
    }
  };
  float y[EARLY ? CH : 1][VE];
  if constexpr (!I8) {
    T *out = (T *)p.a.out + row * p.a.out_stride;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      normed(c, y[0]);
      Vec<T, VE> rounded;
#pragma unroll
      for (int i = 0; i < VE; i++) rounded.v[i] = (T)y[0][i];
      store(out, c, rounded);
    }
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      normed(c, y[EARLY ? c : 0]);
#pragma unroll
      for (int i = 0; i < VE; i++)
        if (own(c, i)) top = max(top, abs_bits(y[EARLY ? c : 0][i]));
    }
    top = wave_max_bits(top);
    if (waves > 1) {
      if (lane == 0) s_top[wave] = top;
      __syncthreads();
      for (int k = 0; k < waves; k++) top = max(top, s_top[k]);
    }
    const float step = code_step(__uint_as_float(top));
    if (t == 0) p.a.out_scale[row] = step;
    int8_t *out = (int8_t *)p.a.out + row * p.a.out_stride;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      if (!EARLY) normed(c, y[0]);
      store(out, c, codes_of<VE>(y[EARLY ? c : 0], step));
    }
  }
}

template <typename T, bool I8, int WB, int CH>
hipError_t run(NormParams &p, int chunks, hipStream_t stream) {
  p.waves = (chunks + 64 * CH - 1) / (64 * CH);
  const int threads = p.waves == 1 ? 256 : p.waves * 64, rows = p.waves == 1 ? 4 : 1;  // of a workgroup
  const cbs_rms_args &a = p.a;
  const int64_t most = kMaxThreads / threads * rows;
  for (int64_t row = 0; row < a.rows; row += most) {
    NormParams q = p;
    q.a.rows = a.rows - row < most ? a.rows - row : most;
    q.a.x = (const T *)a.x + row * a.x_stride;
    if (a.residual) q.a.residual = (const T *)a.residual + row * a.residual_stride;
    if (a.residual_out) q.a.residual_out = (T *)a.residual_out + row * a.residual_out_stride;
    q.a.out = (char *)a.out + row * a.out_stride * (I8 ? 1 : (int)sizeof(T));
    if (I8) q.a.out_scale = a.out_scale + row;
    hipLaunchKernelGGL((rms_norm_kernel<T, I8, WB, CH>), dim3((unsigned)((q.a.rows + rows - 1) / rows)), dim3(threads), 0, stream, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Chunks of a thread: one where few rows leave the compute units idle, so that a row is read in one step; else two, so that
// more of it is on its way.  Longer rows take as many as 8 (16) waves hold.
template <typename T, bool I8, int WB>
hipError_t pick(NormParams &p, hipStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  const int chunks = (p.dim + VE - 1) / VE;
  if (chunks <= 64 || (chunks <= 512 && p.a.rows <= 1024)) return run<T, I8, WB, 1>(p, chunks, stream);
  if (chunks <= 1024) return run<T, I8, WB, 2>(p, chunks, stream);
  if (chunks <= 2048) return run<T, I8, WB, 4>(p, chunks, stream);
  if (chunks <= 8192) return run<T, I8, WB, 8>(p, chunks, stream);
  return run<T, I8, WB, CBS_RMS_MAX_DIM / 1024 / VE>(p, chunks, stream);
}

template <typename T>
hipError_t pick(NormParams &p, bool i8, hipStream_t stream) {
  if (p.weight_dtype == CBS_F32) return i8 ? pick<T, true, 4>(p, stream) : pick<T, false, 4>(p, stream);
  return i8 ? pick<T, true, 2>(p, stream) : pick<T, false, 2>(p, stream);
}

}  // namespace

hipError_t launch_rms_norm(const cbs_rms_desc &d, const cbs_rms_args &a, hipStream_t stream) {
  NormParams p = {a, d.dim, d.weight_dtype, d.eps, 0};
  const bool i8 = d.out_dtype == CBS_I8;
  switch (d.dtype) {
    case CBS_F16: return pick<f16_t>(p, i8, stream);
    case CBS_BF16: return pick<bf16_t>(p, i8, stream);
    default: return pick<float>(p, i8, stream);
  }
}

}  // namespace cbs
