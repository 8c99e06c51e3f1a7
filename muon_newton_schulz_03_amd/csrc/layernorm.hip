// gfx950 (CDNA4) layer norm, forward and backward.
//
// Per row: mean = sum x / n, var = sum (x - mean)^2 / n, rstd = 1 / sqrt(var + eps),
// xh = (x - mean) rstd, y = xh w + b.  Backward, with g = dy w:
//   dx = rstd (g - sum g / n - xh sum(g xh) / n),  dw = sum_rows dy xh,  db = sum_rows dy.
// All arithmetic is fp32; the variance is the mean square of the centred
// values, taken from registers, so a large common offset cancels nothing.
//
// Bound by memory: each operand moves once.  65536 x 768 in bf16 with inputs
// that no cache holds: forward 44 us (201 MB, 4.6 TB/s), both directions 101 us
// (504 MB, 5.0 TB/s), where a plain copy of 2 GiB reaches 5.0 TB/s.  Where the
// Infinity Cache holds the inputs (a copy of 100 MB: 7.1 TB/s): forward 36 us,
// backward 54 us, and 5 us for the parameter gradients' second stage.
#include "block_internal.h"
#include "device_common.h"
#include "row_vectors.h"

namespace muon {
namespace {

// Whether a row's loads are started while the row before is summed.  bf16 rows
// of whole vectors, forward / backward without it and with it: 65536 x 768
// 47 / 61 and 40 / 59 us, 8192 x 8192 72 / 119 and 65 / 100, 16384 x 2048
// 31 / 58 and 28 / 46; 16384 x 1536 19 / 46 and 21 / 37.  With rows of fp32 or
// of odd lengths the held row takes registers or branches that cost more than
// the wait: backward 44 and 59 us for 16384 x 1024 in fp32, 94 and 154 for
// 65536 x 770 in bf16.
template <class T, bool PART>
constexpr bool kAhead = sizeof(T) == 2 && !PART;

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
// stride over the rows, so the parameters are loaded once.  A wave a row up to
// 2048 elements: no barrier, and several rows in flight a SIMD.  Blocks: 1024
// instead of 2048 take the same 40 us for 65536 x 768 and 80 instead of 65 for
// 8192 x 8192.
template <class T, class P, int TPR, int NV, bool PART>
__global__ __launch_bounds__(kThreads) void norm_forward_kernel(NormArgs a) {
  constexpr int VEC = kVec<T>;
  constexpr bool AHEAD = kAhead<T, PART>;
  __shared__ float red[kThreads / 64][1];
  const int tid = threadIdx.x, t = tid % TPR;
  float w[NV][VEC], b[NV][VEC];
  int on[NV];  // elements of each vector inside the row
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    on[i] = min(max(a.cols - c, 0), VEC);
    if (on[i]) {
      load_param<P, VEC, PART>(a.weight, c, on[i], w[i], 1.f);
      load_param<P, VEC, PART>(a.bias, c, on[i], b[i], 0.f);
    }
  }
  const float inv = 1.f / (float)a.cols;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / TPR);
  const int64_t first = (int64_t)blockIdx.x * (kThreads / TPR) + tid / TPR;
  u32x4 next[NV];  // AHEAD: the row after this one, as it was loaded
  auto fetch = [&](int64_t row) {
    const T* x = (const T*)a.x + row * a.ld_x;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (on[i] && row < a.rows) next[i] = *gv<u32x4_any>(x + (i * TPR + t) * VEC);
  };
  if constexpr (AHEAD) fetch(first);
  for (int64_t row = first; row < a.rows; row += stride) {
    const T* x = (const T*)a.x + row * a.ld_x;
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      if (!on[i]) continue;
      if constexpr (AHEAD) unpack8_bf16(next[i], v[i]);
      else load_part<T, VEC, PART>(x + (i * TPR + t) * VEC, on[i], v[i]);
    }
    if constexpr (AHEAD) fetch(row + stride);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[i][e];
    row_sum<TPR, 1>(s, red, tid);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = (PART ? e < on[i] : on[i] > 0) ? v[i][e] - mean : 0.f;
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
      store_part<T, VEC, PART>(y + (i * TPR + t) * VEC, on[i], v[i]);
    }
    if (t == 0) a.mean[row] = mean, a.rstd[row] = rstd;
  }
}

// Rows of any length: a block a row, which is read three times (from L2 after the first).
template <class T, class P, bool PART>
__global__ __launch_bounds__(kThreads) void norm_forward_long_kernel(NormArgs a) {
  constexpr int VEC = kVec<T>;
  __shared__ float red[kThreads / 64][1];
  const int tid = threadIdx.x;
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ld_x;
    T* y = (T*)a.out + row * a.ld_out;
    float s[1] = {0.f}, v[VEC], w[VEC], b[VEC];
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      const int n = min(a.cols - c, VEC);
      load_part<T, VEC, PART>(x + c, n, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[e];
    }
    row_sum<kThreads, 1>(s, red, tid);
    const float mean = s[0] * inv;
    s[0] = 0.f;
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      const int n = min(a.cols - c, VEC);
      load_part<T, VEC, PART>(x + c, n, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] = !PART || e < n ? __builtin_fmaf(v[e] - mean, v[e] - mean, s[0]) : s[0];
    }
    row_sum<kThreads, 1>(s, red, tid);
    const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      const int n = min(a.cols - c, VEC);
      load_part<T, VEC, PART>(x + c, n, v);
      load_param<P, VEC, PART>(a.weight, c, n, w, 1.f);
      load_param<P, VEC, PART>(a.bias, c, n, b, 0.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = __builtin_fmaf((v[e] - mean) * rstd, w[e], b[e]);
      store_part<T, VEC, PART>(y + c, n, v);
    }
    if (tid == 0) a.mean[row] = mean, a.rstd[row] = rstd;
  }
}

// --------------------------------------------------------------- backward --
// As the forward pass; every thread also sums its columns of dw and db over
// its rows, the rows of a block are added through LDS, and the block's sums
// go to part[block] (fixed order: the result does not depend on timing).  Under
// the bound of four waves a SIMD, rows of 256 threads and two vectors spill 12
// registers with fp32 parameters, 2 with bf16.
template <class T, class P, int TPR, int NV, bool PART>
__global__ __launch_bounds__(kThreads, (kAhead<T, PART> && NV <= 2 ? 4 : 1)) void norm_backward_kernel(NormArgs a) {
  constexpr int VEC = kVec<T>;
  constexpr int RPB = kThreads / TPR;
  constexpr bool AHEAD = kAhead<T, PART>;
  __shared__ float red[kThreads / 64][2];
  __shared__ __align__(16) float cross[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * VEC : 1];
  const int tid = threadIdx.x, t = tid % TPR;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
  int on[NV];  // elements of each vector inside the row
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    on[i] = min(max(a.cols - c, 0), VEC);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    if (on[i]) load_param<P, VEC, PART>(a.weight, c, on[i], w[i], 1.f);
  }
  const float inv = 1.f / (float)a.cols;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  const int64_t first = (int64_t)blockIdx.x * RPB + tid / TPR;
  u32x4 nx[NV], ny[NV];  // AHEAD: the row after this one, as it was loaded
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t row) {
    if (row >= a.rows) return;
    const T* x = (const T*)a.x + row * a.ld_x;
    const T* dy = (const T*)a.dy + row * a.ld_dy;
    nmean = a.mean[row], nrstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (on[i]) {
        nx[i] = *gv<u32x4_any>(x + (i * TPR + t) * VEC);
        ny[i] = *gv<u32x4_any>(dy + (i * TPR + t) * VEC);
      }
  };
  if constexpr (AHEAD) fetch(first);
  for (int64_t row = first; row < a.rows; row += stride) {
    const T* x = (const T*)a.x + row * a.ld_x;
    const T* dy = (const T*)a.dy + row * a.ld_dy;
    const float mean = AHEAD ? nmean : a.mean[row], rstd = AHEAD ? nrstd : a.rstd[row];
    float xh[NV][VEC], g[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) xh[i][e] = g[i][e] = 0.f;
      if (!on[i]) continue;
      if constexpr (AHEAD) {
        unpack8_bf16(nx[i], xh[i]);
        unpack8_bf16(ny[i], g[i]);
      } else {
        load_part<T, VEC, PART>(x + (i * TPR + t) * VEC, on[i], xh[i]);
        load_part<T, VEC, PART>(dy + (i * TPR + t) * VEC, on[i], g[i]);  // 0 past the row: nothing there counts
      }
    }
    if constexpr (AHEAD) fetch(row + stride);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on[i]) continue;
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
    if (!a.out) continue;
    row_sum<TPR, 2>(s, red, tid);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    T* dx = (T*)a.out + row * a.ld_out;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on[i]) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[i][e] = rstd * (g[i][e] - __builtin_fmaf(xh[i][e], c2, c1));
      store_part<T, VEC, PART>(dx + (i * TPR + t) * VEC, on[i], g[i]);
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
      if (on[i]) store_part<float, VEC, PART>(part + (int64_t)k * a.cols + (i * TPR + t) * VEC, on[i], v);
    }
}

// Rows of any length: a block takes rows in turn and adds their terms to its
// own sums in memory (only this block and, for each column, only one thread
// touches them).
template <class T, class P, bool PART>
__global__ __launch_bounds__(kThreads) void norm_backward_long_kernel(NormArgs a) {
  constexpr int VEC = kVec<T>;
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
      const int n = min(a.cols - c, VEC);
      load_part<T, VEC, PART>(x + c, n, v);
      load_part<T, VEC, PART>(dy + c, n, g);
      load_param<P, VEC, PART>(a.weight, c, n, w, 1.f);
      float sw[VEC], sb[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) sw[e] = sb[e] = 0.f;
      if (pw && !first) {
        load_part<float, VEC, PART>(pw + c, n, sw);
        load_part<float, VEC, PART>(pw + a.cols + c, n, sb);
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
        store_part<float, VEC, PART>(pw + c, n, sw);
        store_part<float, VEC, PART>(pw + a.cols + c, n, sb);
      }
    }
    first = false;
    if (!a.out) continue;
    row_sum<kThreads, 2>(s, red, tid);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    T* dx = (T*)a.out + row * a.ld_out;
    for (int c = tid * VEC; c < a.cols; c += kThreads * VEC) {
      const int n = min(a.cols - c, VEC);
      load_part<T, VEC, PART>(x + c, n, v);
      load_part<T, VEC, PART>(dy + c, n, g);
      load_param<P, VEC, PART>(a.weight, c, n, w, 1.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (v[e] - mean) * rstd;
        v[e] = rstd * (g[e] * w[e] - __builtin_fmaf(xh, c2, c1));
      }
      store_part<T, VEC, PART>(dx + c, n, v);
    }
  }
}

// Column sums of the blocks' partial sums: 32 columns a block, whose 32 groups
// of 32 threads each take every 32nd row.  A few round trips to memory bound
// this launch: 64 columns a block with 8 rows in flight took 5.3 us for 1024
// rows of 2 x 768, this takes 4.1.
constexpr int kSumThreads = 1024, kSumCols = 32;
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(NormSumArgs a) {
  constexpr int kGroups = kSumThreads / kSumCols;
  __shared__ float red[kGroups][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols, n = 2 * a.cols;
  const int c = (int)blockIdx.x * kSumCols + col;
  float s = 0.f;
  if (c < n)
#pragma unroll 16
    for (int r = g; r < a.blocks; r += kGroups) s += a.part[(int64_t)r * n + c];
  red[g][col] = s;
  __syncthreads();
  if (g > 0 || c >= n) return;
  s = 0.f;
#pragma unroll
  for (int r = 0; r < kGroups; ++r) s += red[r][col];
  float* out = c < a.cols ? a.dweight : a.dbias;
  if (out) out[c < a.cols ? c : c - a.cols] = s;
}

// ----------------------------------------------------------------- launch --
// Rows a block holds at a time, by the row's length: a wave holds a row of up
// to 2048 elements, a block one of up to 8192, and longer rows are read again
// instead of held.
constexpr int kWaveCols = 2048, kBlockCols = 8192;
constexpr int kForwardBlocks = 2048;   // 8 a CU
constexpr int kBackwardBlocks = 1024;  // 4 a CU

template <class T, class P, bool PART, int TPR, int NV>
hipError_t run_norm(const NormArgs& a, bool backward, hipStream_t s) {
  if (backward) return launch_kernel(norm_backward_kernel<T, P, TPR, NV, PART>, a.blocks, kThreads, a, s);
  const int64_t need = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
  return launch_kernel(norm_forward_kernel<T, P, TPR, NV, PART>, need < kForwardBlocks ? need : kForwardBlocks,
                       kThreads, a, s);
}

// The smallest power of two of vectors a thread, from NV to MAX, that holds a row.
template <class T, class P, bool PART, int TPR, int NV, int MAX>
hipError_t pick_nv(const NormArgs& a, bool backward, hipStream_t s) {
  if constexpr (NV >= MAX) {
    return run_norm<T, P, PART, TPR, MAX>(a, backward, s);
  } else {
    if (a.cols <= TPR * kVec<T> * NV) return run_norm<T, P, PART, TPR, NV>(a, backward, s);
    return pick_nv<T, P, PART, TPR, NV * 2, MAX>(a, backward, s);
  }
}

template <class T, class P, bool PART>
hipError_t launch_norm_as(const NormArgs& a, bool backward, hipStream_t s) {
  constexpr int V = kVec<T>, wave_nv = kWaveCols / 64 / V, block_first = 2 * kWaveCols / kThreads / V,
                block_nv = kBlockCols / kThreads / V;
  if (a.cols <= kWaveCols) return pick_nv<T, P, PART, 64, 1, wave_nv>(a, backward, s);
  if (a.cols <= kBlockCols) return pick_nv<T, P, PART, kThreads, block_first, block_nv>(a, backward, s);
  if (backward) return launch_kernel(norm_backward_long_kernel<T, P, PART>, a.blocks, kThreads, a, s);
  return launch_kernel(norm_forward_long_kernel<T, P, PART>, a.rows < kForwardBlocks ? a.rows : kForwardBlocks,
                       kThreads, a, s);
}

template <class T, class P>
hipError_t launch_norm_types(const NormArgs& a, bool backward, hipStream_t s) {
  return a.cols % kVec<T> ? launch_norm_as<T, P, true>(a, backward, s) : launch_norm_as<T, P, false>(a, backward, s);
}

hipError_t launch_norm(const NormArgs& a, bool x_bf16, bool p_bf16, bool backward, hipStream_t s) {
  if (x_bf16)
    return p_bf16 ? launch_norm_types<__bf16, __bf16>(a, backward, s)
                  : launch_norm_types<__bf16, float>(a, backward, s);
  return p_bf16 ? launch_norm_types<float, __bf16>(a, backward, s) : launch_norm_types<float, float>(a, backward, s);
}

}  // namespace

// Blocks of the backward pass, each writing one row of partial sums: as many
// as hold a row each, at most 4 a CU.
int norm_backward_blocks(int64_t rows, int64_t cols) {
  const int64_t rpb = cols <= kWaveCols ? kThreads / 64 : 1;
  const int64_t need = (rows + rpb - 1) / rpb;
  return (int)(need < kBackwardBlocks ? need : kBackwardBlocks);
}

hipError_t launch_norm_forward(const NormArgs& a, bool x_bf16, bool p_bf16, hipStream_t stream) {
  return launch_norm(a, x_bf16, p_bf16, false, stream);
}
hipError_t launch_norm_backward(const NormArgs& a, bool x_bf16, bool p_bf16, hipStream_t stream) {
  return launch_norm(a, x_bf16, p_bf16, true, stream);
}
hipError_t launch_norm_sum(const NormSumArgs& a, hipStream_t stream) {
  return launch_kernel(norm_sum_kernel, (2 * a.cols + kSumCols - 1) / kSumCols, kSumThreads, a, stream);
}

}  // namespace muon
