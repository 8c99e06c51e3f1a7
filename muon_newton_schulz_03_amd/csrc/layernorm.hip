// gfx950 (CDNA4) layer norm, forward and backward.
//
// Per row: mean = sum x / n, var = sum (x - mean)^2 / n, rstd = 1 / sqrt(var + eps),
// xh = (x - mean) rstd, y = xh w + b.  Backward, with g = dy w:
//   dx = rstd (g - sum g / n - xh sum(g xh) / n),  dw = sum_rows dy xh,  db = sum_rows dy.
// All arithmetic is fp32; the variance is the mean square of the centred
// values, taken from registers, so a large common offset cancels nothing.
#include "block_internal.h"
#include "device_common.h"

namespace muon {
namespace {

// --------------------------------------------------------------- elements --
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = (float)*gv<T>(p);
  } else if constexpr (sizeof(T) == 2) {
    unpack8_bf16(*gv<u32x4>(p), v);
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const f32x4 r = *gv<f32x4>(p + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = r[e];
    }
  }
}
template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (VEC == 1) {
    *gv<T>(p) = (T)v[0];
  } else if constexpr (sizeof(T) == 2) {
    *gv<u32x4>(p) = pack8_bf16(v);
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) *gv<f32x4>(p + 4 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  }
}
// A row in vectors of VEC elements: 16 bytes, or one element where a row may
// start off a 16-byte boundary.
template <class T>
constexpr int vec_of(bool vec) {
  return vec ? 16 / (int)sizeof(T) : 1;
}

// Parameters are bf16 or fp32 independently of the activations; the vector
// path reads VEC of them at a time in either type.
template <class P, int VEC>
__device__ __forceinline__ void load_param(const void* p, int64_t at, float* v, float none) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = none;
    return;
  }
  const P* q = (const P*)p + at;
  if constexpr (VEC == 4 && sizeof(P) == 2) {
    unpack4_bf16(*gv<u32x2>(q), v);
  } else {
    load_vec<P, VEC>(q, v);
  }
}

// Sum over the TPR threads of a row, the same in all of them.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*lds)[N], int tid) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] += __shfl_xor(s[n], o);
  if constexpr (TPR > 64) {
    __syncthreads();  // the previous sum has been read
    if ((tid & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) lds[tid >> 6][n] = s[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      s[n] = 0.f;
#pragma unroll
      for (int w = 0; w < TPR / 64; ++w) s[n] += lds[w][n];
    }
  }
}

// ---------------------------------------------------------------- forward --
// TPR threads hold a row of at most TPR * VEC * NV elements in registers and
// stride over the rows, so the parameters are loaded once.
template <class T, class P, int VEC, int TPR, int NV>
__global__ __launch_bounds__(kThreads) void norm_forward_kernel(NormArgs a) {
  __shared__ float red[kThreads / 64][1];
  const int tid = threadIdx.x, t = tid % TPR;
  float w[NV][VEC], b[NV][VEC];
  bool on[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    on[i] = c < a.cols;
    if (on[i]) {
      load_param<P, VEC>(a.weight, c, w[i], 1.f);
      load_param<P, VEC>(a.bias, c, b[i], 0.f);
    }
  }
  const float inv = 1.f / (float)a.cols;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / TPR);
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + tid / TPR; row < a.rows; row += stride) {
    const T* x = (const T*)a.x + row * a.ld_x;
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      if (on[i]) load_vec<T, VEC>(x + (i * TPR + t) * VEC, v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[i][e];
    }
    row_sum<TPR, 1>(s, red, tid);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = on[i] ? v[i][e] - mean : 0.f;
        s[0] = __builtin_fmaf(v[i][e], v[i][e], s[0]);
      }
    row_sum<TPR, 1>(s, red, tid);
    const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
    T* y = (T*)a.out + row * a.ld_out;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on[i]) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = __builtin_fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
      store_vec<T, VEC>(y + (i * TPR + t) * VEC, v[i]);
    }
    if (t == 0) a.mean[row] = mean, a.rstd[row] = rstd;
  }
}

// Rows of any length: a block a row, which is read three times (from L2 after the first).
template <class T, class P, int VEC>
__global__ __launch_bounds__(kThreads) void norm_forward_long_kernel(NormArgs a) {
  __shared__ float red[kThreads / 64][1];
  const int tid = threadIdx.x;
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ld_x;
    T* y = (T*)a.out + row * a.ld_out;
    float s[1] = {0.f}, v[VEC], w[VEC], b[VEC];
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      load_vec<T, VEC>(x + c, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[e];
    }
    row_sum<kThreads, 1>(s, red, tid);
    const float mean = s[0] * inv;
    s[0] = 0.f;
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      load_vec<T, VEC>(x + c, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] = __builtin_fmaf(v[e] - mean, v[e] - mean, s[0]);
    }
    row_sum<kThreads, 1>(s, red, tid);
    const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      load_vec<T, VEC>(x + c, v);
      load_param<P, VEC>(a.weight, c, w, 1.f);
      load_param<P, VEC>(a.bias, c, b, 0.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = __builtin_fmaf((v[e] - mean) * rstd, w[e], b[e]);
      store_vec<T, VEC>(y + c, v);
    }
    if (tid == 0) a.mean[row] = mean, a.rstd[row] = rstd;
  }
}

// --------------------------------------------------------------- backward --
// As the forward pass; every thread also sums its columns of dw and db over
// its rows, the rows of a block are added through LDS, and the block's sums
// go to part[block] (fixed order: the result does not depend on timing).
template <class T, class P, int VEC, int TPR, int NV>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(NormArgs a) {
  constexpr int RPB = kThreads / TPR;
  __shared__ float red[kThreads / 64][2];
  __shared__ __align__(16) float cross[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * VEC : 1];
  const int tid = threadIdx.x, t = tid % TPR;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
  bool on[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    on[i] = c < a.cols;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    if (on[i]) load_param<P, VEC>(a.weight, c, w[i], 1.f);
  }
  const float inv = 1.f / (float)a.cols;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  for (int64_t row = (int64_t)blockIdx.x * RPB + tid / TPR; row < a.rows; row += stride) {
    const T* x = (const T*)a.x + row * a.ld_x;
    const T* dy = (const T*)a.dy + row * a.ld_dy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xh[NV][VEC], g[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) xh[i][e] = g[i][e] = 0.f;
      if (on[i]) {
        load_vec<T, VEC>(x + (i * TPR + t) * VEC, xh[i]);
        load_vec<T, VEC>(dy + (i * TPR + t) * VEC, g[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[i][e] = (xh[i][e] - mean) * rstd;
          dw[i][e] = __builtin_fmaf(g[i][e], xh[i][e], dw[i][e]);
          db[i][e] += g[i][e];
          g[i][e] *= w[i][e];
          s[0] += g[i][e];
          s[1] = __builtin_fmaf(g[i][e], xh[i][e], s[1]);
        }
      }
    }
    if (!a.out) continue;
    row_sum<TPR, 2>(s, red, tid);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    T* dx = (T*)a.out + row * a.ld_out;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on[i]) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[i][e] = rstd * (g[i][e] - __builtin_fmaf(xh[i][e], c2, c1));
      store_vec<T, VEC>(dx + (i * TPR + t) * VEC, g[i]);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float* v = k ? db[i] : dw[i];
      if constexpr (RPB > 1) {
        const int r = tid / TPR;
        __syncthreads();
        if (r > 0) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) cross[r - 1][t * VEC + e] = v[e];
        }
        __syncthreads();
        if (r > 0) continue;
#pragma unroll
        for (int q = 0; q < RPB - 1; ++q)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] += cross[q][t * VEC + e];
      }
      if (on[i]) store_vec<float, VEC>(part + (int64_t)k * a.cols + (i * TPR + t) * VEC, v);
    }
}

// Rows of any length: a block takes rows in turn and adds their terms to its
// own sums in memory (only this block and, for each column, only one thread
// touches them).
template <class T, class P, int VEC>
__global__ __launch_bounds__(kThreads) void norm_backward_long_kernel(NormArgs a) {
  __shared__ float red[kThreads / 64][2];
  const int tid = threadIdx.x;
  const float inv = 1.f / (float)a.cols;
  float* pw = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.cols : nullptr;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ld_x;
    const T* dy = (const T*)a.dy + row * a.ld_dy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f}, v[VEC], g[VEC], w[VEC];
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      load_vec<T, VEC>(x + c, v);
      load_vec<T, VEC>(dy + c, g);
      load_param<P, VEC>(a.weight, c, w, 1.f);
      float sw[VEC], sb[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) sw[e] = sb[e] = 0.f;
      if (pw && !first) {
        load_vec<float, VEC>(pw + c, sw);
        load_vec<float, VEC>(pw + a.cols + c, sb);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (v[e] - mean) * rstd;
        sw[e] = __builtin_fmaf(g[e], xh, sw[e]);
        sb[e] += g[e];
        s[0] = __builtin_fmaf(g[e], w[e], s[0]);
        s[1] = __builtin_fmaf(g[e] * w[e], xh, s[1]);
      }
      if (pw) {
        store_vec<float, VEC>(pw + c, sw);
        store_vec<float, VEC>(pw + a.cols + c, sb);
      }
    }
    first = false;
    if (!a.out) continue;
    row_sum<kThreads, 2>(s, red, tid);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    T* dx = (T*)a.out + row * a.ld_out;
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      load_vec<T, VEC>(x + c, v);
      load_vec<T, VEC>(dy + c, g);
      load_param<P, VEC>(a.weight, c, w, 1.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (v[e] - mean) * rstd;
        v[e] = rstd * (g[e] * w[e] - __builtin_fmaf(xh, c2, c1));
      }
      store_vec<T, VEC>(dx + c, v);
    }
  }
}

// Column sums of the blocks' partial sums: 64 columns a block, its 16 waves
// take every 16th row.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(NormSumArgs a) {
  __shared__ float red[kSumThreads / 64][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = 2 * a.cols;
  const int c = (int)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < n)
#pragma unroll 8
    for (int r = w; r < a.blocks; r += kSumThreads / 64) s += a.part[(int64_t)r * n + c];
  red[w][lane] = s;
  __syncthreads();
  if (w > 0 || c >= n) return;
  s = 0.f;
#pragma unroll
  for (int r = 0; r < kSumThreads / 64; ++r) s += red[r][lane];
  float* out = c < a.cols ? a.dweight : a.dbias;
  if (out) out[c < a.cols ? c : c - a.cols] = s;
}

// ----------------------------------------------------------------- launch --
// Rows a block holds at a time, by the row's length: a wave holds a row of up
// to 2048 elements, a block one of up to 8192 (4096 where rows are not
// aligned), and longer rows are read again instead of held.
constexpr int kWaveCols = 2048, kBlockCols = 8192, kScalarWaveCols = 512, kScalarBlockCols = 4096;
constexpr int kForwardBlocks = 2048;   // 8 a CU
constexpr int kBackwardBlocks = 1024;  // 4 a CU

template <class T, class P, int VEC, int TPR, int NV>
hipError_t run_norm(const NormArgs& a, bool backward, hipStream_t s) {
  if (backward) return launch_kernel(norm_backward_kernel<T, P, VEC, TPR, NV>, a.blocks, kThreads, a, s);
  const int64_t need = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
  return launch_kernel(norm_forward_kernel<T, P, VEC, TPR, NV>, need < kForwardBlocks ? need : kForwardBlocks, kThreads,
                       a, s);
}

template <class T, class P, int VEC, int TPR, int NV, int MAX>
hipError_t pick_nv(const NormArgs& a, bool backward, hipStream_t s) {
  if constexpr (NV >= MAX) {
    return run_norm<T, P, VEC, TPR, MAX>(a, backward, s);
  } else {
    if (a.cols <= TPR * VEC * NV) return run_norm<T, P, VEC, TPR, NV>(a, backward, s);
    return pick_nv<T, P, VEC, TPR, NV * 2, MAX>(a, backward, s);
  }
}

template <class T, class P, bool V>
hipError_t launch_norm_as(const NormArgs& a, bool backward, hipStream_t s) {
  constexpr int VEC = vec_of<T>(V);
  constexpr int wave_cols = V ? kWaveCols : kScalarWaveCols, block_cols = V ? kBlockCols : kScalarBlockCols;
  constexpr int wave_nv = wave_cols / 64 / VEC, block_first = 2 * wave_cols / kThreads / VEC,
                block_nv = block_cols / kThreads / VEC;
  if (a.cols <= wave_cols) return pick_nv<T, P, VEC, 64, 1, wave_nv>(a, backward, s);
  if (a.cols <= block_cols) return pick_nv<T, P, VEC, kThreads, block_first, block_nv>(a, backward, s);
  if (backward) return launch_kernel(norm_backward_long_kernel<T, P, VEC>, a.blocks, kThreads, a, s);
  return launch_kernel(norm_forward_long_kernel<T, P, VEC>, a.rows < kForwardBlocks ? a.rows : kForwardBlocks, kThreads,
                       a, s);
}

hipError_t launch_norm(const NormArgs& a, bool x_bf16, bool p_bf16, bool vec, bool backward, hipStream_t s) {
  if (x_bf16) {
    if (p_bf16) return vec ? launch_norm_as<__bf16, __bf16, true>(a, backward, s)
                           : launch_norm_as<__bf16, __bf16, false>(a, backward, s);
    return vec ? launch_norm_as<__bf16, float, true>(a, backward, s)
               : launch_norm_as<__bf16, float, false>(a, backward, s);
  }
  if (p_bf16) return vec ? launch_norm_as<float, __bf16, true>(a, backward, s)
                         : launch_norm_as<float, __bf16, false>(a, backward, s);
  return vec ? launch_norm_as<float, float, true>(a, backward, s)
             : launch_norm_as<float, float, false>(a, backward, s);
}

}  // namespace

// Blocks of the backward pass, each writing one row of partial sums: as many
// as hold a row each, at most 4 a CU.
int norm_backward_blocks(int64_t rows, int64_t cols, bool vec) {
  const int64_t rpb = cols <= (vec ? kWaveCols : kScalarWaveCols) ? kThreads / 64 : 1;
  const int64_t need = (rows + rpb - 1) / rpb;
  return (int)(need < kBackwardBlocks ? need : kBackwardBlocks);
}

hipError_t launch_norm_forward(const NormArgs& a, bool x_bf16, bool p_bf16, bool vec, hipStream_t stream) {
  return launch_norm(a, x_bf16, p_bf16, vec, false, stream);
}
hipError_t launch_norm_backward(const NormArgs& a, bool x_bf16, bool p_bf16, bool vec, hipStream_t stream) {
  return launch_norm(a, x_bf16, p_bf16, vec, true, stream);
}
hipError_t launch_norm_sum(const NormSumArgs& a, hipStream_t stream) {
  return launch_kernel(norm_sum_kernel, (2 * a.cols + 63) / 64, kSumThreads, a, stream);
}

}  // namespace muon
