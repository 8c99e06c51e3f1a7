// gfx950 (CDNA4) norm of queries and keys for each head with the position
// rotation in the same pass, forward and backward.
//
// Per token and head, x of D elements: r = 1 / sqrt(sum x^2 / D + eps),
// z = x r w, and y = R z, where R turns each pair (a, b) of the first elements
// by its angle: y_a = z_a cos - z_b sin, y_b = z_b cos + z_a sin.  Backward, with
// dz = R^T dy and g = dz w:
//   dx = r (g - x r^2 sum(g x) / D),  dw = sum over tokens and heads of dz x r.
// Nothing is kept from the forward pass: the backward pass reads x anyway, and
// r is one more sum over it.  All arithmetic is fp32.
//
// Angles are counted in turns, as 64-bit fractions: position times turn modulo
// 2^64 is exact, so up to position 2^32 only the fraction's own rounding, 2^-65,
// counts, and the eighth of a turn that is left for sine and cosine is exact to
// 2^-31 turns.
#include "block_internal.h"
#include "device_common.h"

namespace muon {
namespace {

// Sum over groups of N neighbouring lanes (4, 8 or 16), the same in all of
// them: lanes exchanged within quads, then quads and halves mirrored.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xB1>(v);                         // quad_perm 1 0 3 2
  v = dpp_add<0x4E>(v);                         // quad_perm 2 3 0 1
  if constexpr (N > 4) v = dpp_add<0x141>(v);   // row_half_mirror
  if constexpr (N > 8) v = dpp_add<0x140>(v);   // row_mirror
  return v;
}

// cos and sin of a phase in 2^-32 turns.  The phase is brought to an eighth of
// a turn around the nearest quarter, where the Taylor series to x^10 and x^9
// are off by less than 2^-28.
__device__ __forceinline__ void turn_sincos(uint32_t phase, float& s, float& c) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(phase - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float q = x * x;
  float p = __builtin_fmaf(q, 1.f / 362880.f, -1.f / 5040.f);
  p = __builtin_fmaf(q, p, 1.f / 120.f);
  p = __builtin_fmaf(q, p, -1.f / 6.f);
  const float sine = __builtin_fmaf(x * q, p, x);
  p = __builtin_fmaf(q, -1.f / 3628800.f, 1.f / 40320.f);
  p = __builtin_fmaf(q, p, -1.f / 720.f);
  p = __builtin_fmaf(q, p, 1.f / 24.f);
  p = __builtin_fmaf(q, p, -0.5f);
  const float cosine = __builtin_fmaf(q, p, 1.f);
  const bool odd = quarter & 1;
  s = odd ? cosine : sine;
  c = odd ? sine : cosine;
  s = quarter & 2 ? -s : s;
  c = (quarter + 1) & 2 ? -c : c;
}

template <class T, int N>
struct Raw;
template <>
struct Raw<__bf16, 8> { typedef u32x4 type; };
template <>
struct Raw<__bf16, 4> { typedef u32x2 type; };
template <>
struct Raw<float, 4> { typedef f32x4 type; };
__device__ __forceinline__ void unpack(u32x4 r, float* v) { unpack8_bf16(r, v); }
__device__ __forceinline__ void unpack(u32x2 r, float* v) { unpack4_bf16(r, v); }
__device__ __forceinline__ void unpack(f32x4 r, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = r[e];
}
__device__ __forceinline__ void pack(const float* v, u32x4& r) { r = pack8_bf16(v); }
__device__ __forceinline__ void pack(const float* v, u32x2& r) { r = pack4_bf16(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pack(const float* v, f32x4& r) { r = f32x4{v[0], v[1], v[2], v[3]}; }

// The two members of N pairs from a thread's two vectors, and back.
template <int N, bool NEIGH>
__device__ __forceinline__ void to_pairs(const float* v, float* a, float* b) {
#pragma unroll
  for (int e = 0; e < N; ++e) a[e] = v[NEIGH ? 2 * e : e], b[e] = v[NEIGH ? 2 * e + 1 : N + e];
}
template <int N, bool NEIGH>
__device__ __forceinline__ void from_pairs(const float* a, const float* b, float* v) {
#pragma unroll
  for (int e = 0; e < N; ++e) v[NEIGH ? 2 * e : e] = a[e], v[NEIGH ? 2 * e + 1 : N + e] = b[e];
}

__device__ __forceinline__ float param(const void* p, bool bf16, int at) {
  return !p ? 1.f : bf16 ? (float)*gv<__bf16>((const __bf16*)p + at) : *gv<float>((const float*)p + at);
}

// The start of the token's sequence: the last offset at or before it.
__device__ __forceinline__ int64_t sequence_start(const int32_t* cu, int seqs, int64_t token) {
  int lo = 0, hi = seqs;  // cu[lo] <= token < cu[hi]
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (*gv<int32_t>(cu + mid) <= token) lo = mid;
    else hi = mid;
  }
  return *gv<int32_t>(cu + lo);
}

// A group of LPH lanes holds one token's head, a lane two vectors of VEC
// elements that form VEC pairs; the lanes keep their place in the head, their
// weights and their token's angles while they go through a chunk of its heads.
template <class T, int VEC, int LPH, bool NEIGH, bool BACK>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkArgs a) {
  constexpr int TOKENS = kThreads / LPH;  // of a block
  typedef typename Raw<T, VEC>::type raw_t;
  const bool second = (int)blockIdx.x >= a.side[0].blocks;
  const QkSide& s = second ? a.side[1] : a.side[0];
  const int block = (int)blockIdx.x - (second ? a.side[0].blocks : 0);
  const int u = threadIdx.x % LPH, slot = threadIdx.x / LPH;

  const int turning = a.rotated / (2 * VEC);  // lanes with pairs that turn
  const bool turns = u < turning;
  const int lo = turns && !NEIGH ? u * VEC : turns ? u * 2 * VEC : a.rotated + (u - turning) * 2 * VEC;
  const int hi = turns && !NEIGH ? lo + a.rotated / 2 : lo + VEC;
  const bool on_lo = lo < a.dim, on_hi = hi < a.dim;
  float wa[VEC], wb[VEC], da[VEC], db[VEC];
  uint64_t turn[VEC];
  {
    float w[2 * VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[e] = on_lo ? param(s.weight, a.p_bf16, lo + e) : 0.f;
      w[VEC + e] = on_hi ? param(s.weight, a.p_bf16, hi + e) : 0.f;
      turn[e] = turns ? a.turns[u * VEC + e] : 0;
      da[e] = db[e] = 0.f;
    }
    to_pairs<VEC, NEIGH>(w, wa, wb);
  }
  const int64_t last = a.cu ? min(max((int64_t)*gv<int32_t>(a.cu + a.seqs), (int64_t)0), a.tokens) : a.tokens;
  const float inv = 1.f / (float)a.dim;
  const int chunks = (s.heads + s.chunk - 1) / s.chunk;
  const int64_t items = (a.tokens + TOKENS - 1) / TOKENS * chunks;
  for (int64_t item = block; item < items; item += s.blocks) {
    const int64_t token = item / chunks * TOKENS + slot;
    const int h0 = (int)(item % chunks) * s.chunk, h1 = min(h0 + s.chunk, s.heads);
    if (token >= last) {
      if (token < a.tokens && s.zero_tail)
        for (int h = h0; h < h1; ++h) {
          T* y = (T*)s.out.data + token * s.out.token + h * s.out.head;
          if (on_lo) *gv<raw_t>(y + lo) = raw_t{};
          if (on_hi) *gv<raw_t>(y + hi) = raw_t{};
        }
      continue;
    }
    float cs[VEC], sn[VEC];
    if (turns) {
      int64_t p = token;
      if (a.positions)
        p = a.pos64 ? *gv<int64_t>((const int64_t*)a.positions + token) : *gv<int32_t>((const int32_t*)a.positions + token);
      else if (a.cu)
        p = token - sequence_start(a.cu, a.seqs, token);
#pragma unroll
      for (int e = 0; e < VEC; ++e) turn_sincos((uint32_t)(((uint64_t)p * turn[e]) >> 32), sn[e], cs[e]);
    }
    for (int h = h0; h < h1; ++h) {
      const T* x = (const T*)s.x.data + token * s.x.token + h * s.x.head;
      float v[2 * VEC], xa[VEC], xb[VEC];
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) v[e] = 0.f;
      if (on_lo) unpack(*gv<raw_t>(x + lo), v);
      if (on_hi) unpack(*gv<raw_t>(x + hi), v + VEC);
      to_pairs<VEC, NEIGH>(v, xa, xb);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum = __builtin_fmaf(xa[e], xa[e], __builtin_fmaf(xb[e], xb[e], sum));
      const float r = 1.f / sqrtf(__builtin_fmaf(lanes_sum<LPH>(sum), inv, a.eps));
      float ya[VEC], yb[VEC];
      if constexpr (BACK) {
        const T* dy = (const T*)s.dy.data + token * s.dy.token + h * s.dy.head;
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) v[e] = 0.f;
        if (on_lo) unpack(*gv<raw_t>(dy + lo), v);
        if (on_hi) unpack(*gv<raw_t>(dy + hi), v + VEC);
        to_pairs<VEC, NEIGH>(v, ya, yb);
        float gx = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (turns) {
            const float t = __builtin_fmaf(ya[e], cs[e], yb[e] * sn[e]);
            yb[e] = __builtin_fmaf(yb[e], cs[e], -(ya[e] * sn[e]));
            ya[e] = t;
          }
          da[e] = __builtin_fmaf(ya[e] * r, xa[e], da[e]);
          db[e] = __builtin_fmaf(yb[e] * r, xb[e], db[e]);
          ya[e] *= wa[e];
          yb[e] *= wb[e];
          gx = __builtin_fmaf(ya[e], xa[e], __builtin_fmaf(yb[e], xb[e], gx));
        }
        const float c = lanes_sum<LPH>(gx) * inv * r * r;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ya[e] = r * __builtin_fmaf(-xa[e], c, ya[e]);
          yb[e] = r * __builtin_fmaf(-xb[e], c, yb[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ya[e] = xa[e] * r * wa[e];
          yb[e] = xb[e] * r * wb[e];
          if (turns) {
            const float t = __builtin_fmaf(ya[e], cs[e], -(yb[e] * sn[e]));
            yb[e] = __builtin_fmaf(yb[e], cs[e], ya[e] * sn[e]);
            ya[e] = t;
          }
        }
      }
      from_pairs<VEC, NEIGH>(ya, yb, v);
      T* y = (T*)s.out.data + token * s.out.token + h * s.out.head;
      raw_t o;
      pack(v, o);
      if (on_lo) *gv<raw_t>(y + lo) = o;
      pack(v + VEC, o);
      if (on_hi) *gv<raw_t>(y + hi) = o;
    }
  }
  if constexpr (BACK) {
    if (!a.part) return;
    // the block's sums: over the tokens of a wave, then over its waves, in a fixed order
    __shared__ float red[kThreads / 64][LPH * 2 * VEC];
#pragma unroll
    for (int o = LPH; o < 64; o *= 2)
#pragma unroll
      for (int e = 0; e < VEC; ++e) da[e] += __shfl_xor(da[e], o), db[e] += __shfl_xor(db[e], o);
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 < LPH) {
      float v[2 * VEC];
      from_pairs<VEC, NEIGH>(da, db, v);
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) red[wave][u * 2 * VEC + e] = v[e];
    }
    __syncthreads();
    if (threadIdx.x >= LPH) return;
    float* part = a.part + (int64_t)blockIdx.x * a.dim;
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) v += red[w][u * 2 * VEC + e];
      const int at = e < VEC ? lo + e : hi + e - VEC;
      if (e < VEC ? on_lo : on_hi) part[at] = v;
    }
  }
}

// Sums of the blocks' weight gradients: a block for 32 elements of one side.
constexpr int kSumThreads = 1024, kSumCols = 32;
__global__ __launch_bounds__(kSumThreads) void qk_sum_kernel(QkSumArgs a) {
  constexpr int kGroups = kSumThreads / kSumCols;
  __shared__ float red[kGroups][kSumCols + 1];
  const int tiles = (a.dim + kSumCols - 1) / kSumCols;
  const int side = (int)blockIdx.x / tiles, col = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int c = (int)blockIdx.x % tiles * kSumCols + col;
  const float* part = a.part + (side ? (int64_t)a.blocks[0] * a.dim : 0);
  float s = 0.f;
  if (c < a.dim)
#pragma unroll 16
    for (int r = g; r < a.blocks[side]; r += kGroups) s += part[(int64_t)r * a.dim + c];
  red[g][col] = s;
  __syncthreads();
  if (g > 0 || c >= a.dim || !a.dweight[side]) return;
  s = 0.f;
#pragma unroll
  for (int r = 0; r < kGroups; ++r) s += red[r][col];
  a.dweight[side][c] = s;
}

// ----------------------------------------------------------------- launch --
int vec_of(const QkArgs& a, bool bf16) { return bf16 && a.rotated % 16 == 0 ? 8 : 4; }
int lanes_of(const QkArgs& a, int vec) {
  const int units = (a.dim + 2 * vec - 1) / (2 * vec);
  return vec == 8 ? (units <= 4 ? 4 : 8) : units <= 8 ? 8 : 16;
}

template <class T, int VEC, int LPH, bool NEIGH>
hipError_t run_qk(const QkArgs& a, bool backward, hipStream_t s) {
  const int64_t grid = a.side[0].blocks + a.side[1].blocks;
  return backward ? launch_kernel(qk_norm_kernel<T, VEC, LPH, NEIGH, true>, grid, kThreads, a, s)
                  : launch_kernel(qk_norm_kernel<T, VEC, LPH, NEIGH, false>, grid, kThreads, a, s);
}
template <class T, int VEC, bool NEIGH>
hipError_t pick_lanes(const QkArgs& a, bool backward, hipStream_t s) {
  constexpr int FEW = 32 / VEC;  // 4 lanes of 2 x 8 elements, or 8 of 2 x 4
  return lanes_of(a, VEC) == FEW ? run_qk<T, VEC, FEW, NEIGH>(a, backward, s)
                                 : run_qk<T, VEC, 2 * FEW, NEIGH>(a, backward, s);
}
template <bool NEIGH>
hipError_t pick_type(const QkArgs& a, bool bf16, bool backward, hipStream_t s) {
  if (!bf16) return pick_lanes<float, 4, NEIGH>(a, backward, s);
  return vec_of(a, bf16) == 8 ? pick_lanes<__bf16, 8, NEIGH>(a, backward, s)
                              : pick_lanes<__bf16, 4, NEIGH>(a, backward, s);
}

}  // namespace

void plan_qk(QkArgs& a, bool bf16, bool backward) {
  (void)backward;
  const int tokens = kThreads / lanes_of(a, vec_of(a, bf16));
  for (QkSide& s : a.side) {
    s.chunk = s.heads < 8 ? s.heads : 8;
    if (s.chunk < 1) s.chunk = 1;  // no tokens: no side is filled in
    const int64_t items = (a.tokens + tokens - 1) / tokens * ((s.heads + s.chunk - 1) / s.chunk);
    s.blocks = (int)(items < kQkBlocks ? items : kQkBlocks);
  }
}

hipError_t launch_qk(const QkArgs& a, bool bf16, int pairs, bool backward, hipStream_t s) {
  return pairs == kPairNeighbours ? pick_type<true>(a, bf16, backward, s) : pick_type<false>(a, bf16, backward, s);
}
hipError_t launch_qk_sum(const QkSumArgs& a, hipStream_t stream) {
  return launch_kernel(qk_sum_kernel, 2 * ((a.dim + kSumCols - 1) / kSumCols), kSumThreads, a, stream);
}

}  // namespace muon
