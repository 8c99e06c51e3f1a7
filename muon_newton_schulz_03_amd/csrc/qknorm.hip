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
// 2^64 is exact, so up to position 2^32 the phase, cut to 2^-32 turns, is off by
// that and the fraction's own rounding, 2^-65 a position: 2^-31 turns together.
// Sine and cosine of it are fp32 (see turn_sincos).
//
// Bound by memory: each operand moves once a call.  65536 tokens of 24 heads of
// 64 in bf16 forward 83 us (403 MB, 4.8 TB/s, where a copy of 1 GiB reaches 5.1
// and vector operations take 42% of the time); 16384 tokens of 40 heads of 128
// forward 62 us and backward 108 (335 and 503 MB, 5.4 and 4.7 TB/s), and 5 us for
// the weight gradients' second stage.
#include "block_internal.h"
#include "device_common.h"
#include "wave.h"

namespace muon {
namespace {

// Sum over groups of N neighbouring lanes (8, 16 or 32), the same in all of
// them: lanes exchanged within quads, then quads and halves mirrored, then rows
// of 16 exchanged.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xB1>(v);                         // quad_perm 1 0 3 2
  v = dpp_add<0x4E>(v);                         // quad_perm 2 3 0 1
  v = dpp_add<0x141>(v);                        // row_half_mirror
  if constexpr (N > 8) v = dpp_add<0x140>(v);   // row_mirror
  if constexpr (N > 16) v += __shfl_xor(v, 16);
  return v;
}

// cos and sin of a phase in 2^-32 turns.  The phase is brought to an eighth of
// a turn around the nearest quarter, where the Taylor series to x^10 and x^9
// are off by less than 2^-28.  In radians it is rounded to fp32 twice (by up to
// 2^-28 turns on the way), the series' last steps once or twice: over all 2^32
// phases both are off by at most 1.71 2^-24.
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

// The same vector of another lane.
template <class R>
__device__ __forceinline__ R from_lane(R v, int lane) {
  constexpr int N = sizeof(R) / 4;
  typedef int words __attribute__((ext_vector_type(N)));
  words w = __builtin_bit_cast(words, v);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = __builtin_amdgcn_ds_bpermute(4 * lane, w[i]);
  return __builtin_bit_cast(R, w);
}

template <int N>
__device__ __forceinline__ void read_angles(const float* p, float* v) {
  if constexpr (N == 2) {
    const f32x2 r = *(const f32x2*)p;
    v[0] = r[0], v[1] = r[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) unpack(*(const f32x4*)(p + i), v + i);
  }
}

// A span of tokens of one sequence: [start, end).
struct Span {
  int64_t start, end;
};
// The one that holds the token, which is the same in all lanes: the offsets come through scalar loads.
__device__ __forceinline__ Span span_of(const int32_t* cu, int seqs, int64_t token) {
  const MUON_CONST int32_t* c = (const MUON_CONST int32_t*)(const void*)cu;
  int lo = 0, hi = seqs;  // cu[lo] <= token < cu[hi]
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (c[mid] <= token) lo = mid;
    else hi = mid;
  }
  return Span{c[lo], c[hi]};
}
__device__ __forceinline__ int64_t start_of(const int32_t* cu, int seqs, int64_t token) {
  int lo = 0, hi = seqs;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (*gv<int32_t>(cu + mid) <= token) lo = mid;
    else hi = mid;
  }
  return *gv<int32_t>(cu + lo);
}

// A wave takes a group of tokens at a time and goes through their queries and
// then their keys in steps: LPH lanes a head, a vector of VEC elements a lane,
// `wide` heads of each token a step.  So a step's loads are whole heads next to
// each other, and a lane's place in them never changes.  The other members of a
// vector's pairs are the vector of another lane (halves) or its own neighbours.
// The lanes first compute the group's cosines and sines, each once, and share
// them through LDS.
// The next steps' loads run while these are computed: three steps forward, one
// backward, which leave room for four waves a SIMD.  65536 tokens of 24 heads of
// 64 forward / 16384 tokens of 40 heads of 128 backward: 84 / 109 us; with two
// steps forward 92, four 93 (three waves); with two backward 121 (three waves) or
// 152 (registers spill).  A wave with both sides of a token reads the projection's
// row as it lies: with queries and keys in blocks of their own 94 / 110 us.
template <class T, int VEC, int LPH, bool NEIGH, bool BACK, bool W>
__global__ __launch_bounds__(kThreads, 4) void qk_norm_kernel(QkArgs a) {
  constexpr int AHEAD = BACK ? 1 : 3, WAVES = kThreads / 64;
  constexpr int ANGLES = NEIGH ? VEC / 2 : VEC;       // of a lane
  constexpr int TABLE = LPH * VEC * (64 / LPH) / 2;   // of a wave's tokens, at most
  typedef typename Raw<T, VEC>::type raw_t;
  __shared__ __align__(16) float table[WAVES][3][TABLE];  // cosines, sines and negative sines
  __shared__ __align__(16) float weights[2][W ? LPH * VEC : 4];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int u = lane % LPH, lo = u * VEC;
  const int my_head = lane / LPH & (a.wide - 1), my_token = lane / LPH >> a.wide_log;
  const int tokens = (64 / LPH) >> a.wide_log;  // of a group
  const bool on = lo < a.dim, turns = lo < a.rotated;
  const int half = a.rotated / 2 / VEC;  // lanes of a half
  const bool upper = !NEIGH && u >= half;
  const int across = NEIGH || !turns ? 0 : upper ? -half : half;  // lanes to the partner
  // where a lane's cosines and sines start, the latter with the sign that its vector takes them with
  const int pairs = a.rotated / 2;
  float* angles = table[wave][0];
  const float* cosines = angles + my_token * pairs + (NEIGH ? u * ANGLES : (upper ? u - half : u) * ANGLES);
  const float* sines = cosines + (upper != BACK ? TABLE : 2 * TABLE);

  if constexpr (W) {
    for (int i = threadIdx.x; i < 2 * LPH * VEC; i += kThreads) {
      const void* p = a.side[i / (LPH * VEC)].weight;
      const int at = i % (LPH * VEC);
      weights[i / (LPH * VEC)][at] = at >= a.dim ? 0.f : !p ? 1.f : a.p_bf16 ? (float)*gv<__bf16>((const __bf16*)p + at)
                                                                             : *gv<float>((const float*)p + at);
    }
    __syncthreads();
  }
  float w[VEC], wo[VEC], dw[2][VEC];  // own weights, and the partner's
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = wo[e] = dw[0][e] = dw[1][e] = 0.f;
  // a lane computes the angles of one pair, of one token or several
  const int pair = lane & ((1 << a.pair_lanes) - 1), pair_token = lane >> a.pair_lanes;
  const uint64_t turn = pair < pairs ? a.turns[pair] : 0;
  int64_t last = a.tokens;  // tokens that count
  if (a.cu) last = min(max((int64_t)((const MUON_CONST int32_t*)(const void*)a.cu)[a.seqs], (int64_t)0), last);
  const float inv = 1.f / (float)a.dim;

  const T* x[2];
  const T* dy[2];
  T* out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const QkSide& s = a.side[i];
    x[i] = (const T*)s.x.data + my_token * s.x.token + my_head * s.x.head + lo;
    dy[i] = (const T*)s.dy.data + my_token * s.dy.token + my_head * s.dy.head + lo;
    out[i] = (T*)s.out.data + my_token * s.out.token + my_head * s.out.head + lo;
  }
  raw_t nx[AHEAD] = {}, ny[AHEAD] = {};  // the next steps as they were loaded
  auto fetch = [&](auto side, int64_t first, int head) {
    constexpr int S = decltype(side)::value;
    const QkSide& s = a.side[S];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      if (on && head + q * a.wide + my_head < s.heads && first + my_token < last) {
        nx[q] = *gv<raw_t>(x[S] + (first * s.x.token + (head + q * a.wide) * s.x.head));
        if constexpr (BACK) ny[q] = *gv<raw_t>(dy[S] + (first * s.dy.token + (head + q * a.wide) * s.dy.head));
      }
  };
  typedef std::integral_constant<int, 0> queries;
  typedef std::integral_constant<int, 1> keys;
  // a block takes both sides, or where blocks are few one
  const bool do_q = !a.apart || blockIdx.x % 2 == 0, do_k = !a.apart || blockIdx.x % 2 == 1;
  const int64_t stride = (int64_t)(gridDim.x >> a.apart) * WAVES * tokens;
  int64_t first = ((int64_t)(blockIdx.x >> a.apart) * WAVES + wave) * tokens;
  Span span{0, 0};
  if (do_q) fetch(queries{}, first, 0);
  else fetch(keys{}, first, 0);
  for (; first < a.tokens; first += stride) {
    if (pairs) {
      wave_fence();  // the angles before have been read
      if (a.cu && !a.positions && first < last && (first < span.start || first >= span.end))
        span = span_of(a.cu, a.seqs, first);
      for (int t = pair_token; t < tokens && first + t < last; t += 64 >> a.pair_lanes) {
        int64_t p = first + t;
        if (a.positions)
          p = a.pos64 ? *gv<int64_t>((const int64_t*)a.positions + p) : *gv<int32_t>((const int32_t*)a.positions + p);
        else if (a.cu)
          p -= p < span.end ? span.start : start_of(a.cu, a.seqs, p);
        float sine, cosine;
        turn_sincos((uint32_t)(((uint64_t)p * turn) >> 32), sine, cosine);
        if (pair < pairs) {
          float* c = angles + t * pairs + pair;
          c[0] = cosine, c[TABLE] = sine, c[2 * TABLE] = -sine;
        }
      }
      wave_fence();
    }
    float cs[ANGLES], sn[ANGLES];
    if (turns) read_angles<ANGLES>(cosines, cs), read_angles<ANGLES>(sines, sn);
    const bool counts = on && first + my_token < last;
    auto heads_of = [&](auto side) {
      constexpr int S = decltype(side)::value;
      const QkSide& s = a.side[S];
      if constexpr (W) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          unpack(*(const f32x4*)(weights[S] + lo + e), w + e);
          if constexpr (!NEIGH && !BACK) unpack(*(const f32x4*)(weights[S] + lo + across * VEC + e), wo + e);
        }
      }
      for (int head = 0; head < s.heads; head += AHEAD * a.wide) {
        raw_t rx[AHEAD], ry[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) rx[q] = nx[q], ry[q] = ny[q];
        if (head + AHEAD * a.wide < s.heads) fetch(side, first, head + AHEAD * a.wide);
        else if (S == 0 && do_k) fetch(keys{}, first, 0);
        else if (S == 0 || do_q) fetch(queries{}, first + stride, 0);
        else fetch(keys{}, first + stride, 0);
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
          if (head + q * a.wide >= s.heads) break;
          float v[VEC], y[VEC], o[VEC];
          unpack(rx[q], v);
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
          const float mean = __builtin_fmaf(lanes_sum<LPH>(sum), inv, a.eps);
          const float r = sizeof(T) == 2 ? __builtin_amdgcn_rsqf(mean) : 1.f / sqrtf(mean);  // the former: off by 1 ulp
          if constexpr (!NEIGH) unpack(from_lane(BACK ? ry[q] : rx[q], lane + across), o);
          if constexpr (BACK) unpack(ry[q], y);
          else if constexpr (W) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              y[e] = v[e] * w[e];
              if constexpr (!NEIGH) o[e] *= wo[e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = v[e];
          }
          // y_a = z_a cos - z_b sin and y_b = z_b cos + z_a sin, or back with the sines' sign changed
          if (turns) {
            if constexpr (NEIGH) {
#pragma unroll
              for (int e = 0; e < ANGLES; ++e) {
                const float t = y[2 * e];
                y[2 * e] = __builtin_fmaf(t, cs[e], y[2 * e + 1] * sn[e]);
                y[2 * e + 1] = __builtin_fmaf(y[2 * e + 1], cs[e], -(t * sn[e]));
              }
            } else {
#pragma unroll
              for (int e = 0; e < VEC; ++e) y[e] = __builtin_fmaf(y[e], cs[e], o[e] * sn[e]);
            }
          }
          const bool live = counts && head + q * a.wide + my_head < s.heads;
          if constexpr (BACK) {
            if (W && a.part && live) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) dw[S][e] = __builtin_fmaf(y[e] * r, v[e], dw[S][e]);
            }
            if constexpr (W) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) y[e] *= w[e];
            }
            float gx = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) gx = __builtin_fmaf(y[e], v[e], gx);
            const float c = lanes_sum<LPH>(gx) * inv * r * r;
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = r * __builtin_fmaf(-v[e], c, y[e]);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] *= r;
          }
          T* to = out[S] + (first * s.out.token + (head + q * a.wide) * s.out.head);
          raw_t ro;
          pack(y, ro);
          if (live) *gv<raw_t>(to) = ro;
          else if (s.zero_tail && on && first + my_token < a.tokens && head + q * a.wide + my_head < s.heads)
            *gv<raw_t>(to) = raw_t{};
        }
      }
    };
    if (do_q) heads_of(queries{});
    if (do_k) heads_of(keys{});
  }
  if constexpr (BACK && W) {
    if (!a.part) return;
    // the block's sums: over the heads of a wave, then over its waves, in a fixed order
    __shared__ float red[WAVES][2][LPH * VEC];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = LPH; o < 64; o *= 2)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] += __shfl_xor(dw[i][e], o);
      if (lane < LPH) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) red[wave][i][lo + e] = dw[i][e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += kThreads) {
      const int i = c >= a.dim, at = c - i * a.dim;
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < WAVES; ++j) v += red[j][i][at];
      a.part[(int64_t)blockIdx.x * 2 * a.dim + c] = v;
    }
  }
}

// Sums of the blocks' weight gradients, 2 * dim columns: a block for 32 of them.
constexpr int kSumThreads = 1024, kSumCols = 32;
__global__ __launch_bounds__(kSumThreads) void qk_sum_kernel(QkSumArgs a) {
  constexpr int kGroups = kSumThreads / kSumCols;
  __shared__ float red[kGroups][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols, n = 2 * a.dim;
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
  float* out = c < a.dim ? a.dweight[0] : a.dweight[1];
  if (out) out[c < a.dim ? c : c - a.dim] = s;
}

// ----------------------------------------------------------------- launch --
// Halves have to be whole vectors.
int vec_of(const QkArgs& a, bool bf16, int pairs) {
  return bf16 && (pairs == kPairNeighbours || a.rotated % 16 == 0) ? 8 : 4;
}
int lanes_of(const QkArgs& a, int vec) { return a.dim <= 64 ? 64 / vec : 128 / vec; }

template <class T, int VEC, bool NEIGH, int LPH, bool BACK>
hipError_t run_qk(const QkArgs& a, hipStream_t s) {
  return a.side[0].weight || a.side[1].weight || a.part
             ? launch_kernel(qk_norm_kernel<T, VEC, LPH, NEIGH, BACK, true>, a.blocks, kThreads, a, s)
             : launch_kernel(qk_norm_kernel<T, VEC, LPH, NEIGH, BACK, false>, a.blocks, kThreads, a, s);
}
template <class T, int VEC, bool NEIGH>
hipError_t pick_lanes(const QkArgs& a, bool backward, hipStream_t s) {
  if (a.dim <= 64)
    return backward ? run_qk<T, VEC, NEIGH, 64 / VEC, true>(a, s) : run_qk<T, VEC, NEIGH, 64 / VEC, false>(a, s);
  return backward ? run_qk<T, VEC, NEIGH, 128 / VEC, true>(a, s) : run_qk<T, VEC, NEIGH, 128 / VEC, false>(a, s);
}

}  // namespace

void plan_qk(QkArgs& a, bool bf16, int pairs) {
  const int at_once = 64 / lanes_of(a, vec_of(a, bf16, pairs));  // heads that a wave holds
  a.pair_lanes = 0;
  while (1 << a.pair_lanes < a.rotated / 2) ++a.pair_lanes;
  // as many heads of a token at once as leave no more than an eighth of the steps' places empty
  a.wide_log = 0;
  while (2 << a.wide_log <= at_once) ++a.wide_log;
  auto places = [&] {
    int64_t n = 0;
    for (const QkSide& s : a.side) n += (int64_t)((s.heads + (1 << a.wide_log) - 1) >> a.wide_log) << a.wide_log;
    return n;
  };
  while (a.wide_log > 0 && places() * 8 > (int64_t)(a.side[0].heads + a.side[1].heads) * 9) --a.wide_log;
  a.wide = 1 << a.wide_log;
  const int64_t tokens = (int64_t)(at_once >> a.wide_log) * (kThreads / 64);
  const int64_t need = (a.tokens + tokens - 1) / tokens;
  // few blocks: half the work each (2048 tokens of 24 heads of 64 in fp32: 8.7 us forward instead of 10.3); where
  // the GPU's 1024 places are full, both sides in one block (see the kernel)
  a.apart = 2 * need <= kQkBlocks;
  a.blocks = (int)(a.apart ? 2 * need : need < kQkBlocks ? need : kQkBlocks);
}

hipError_t launch_qk(const QkArgs& a, bool bf16, int pairs, bool backward, hipStream_t s) {
  const bool wide = vec_of(a, bf16, pairs) == 8;
  if (pairs == kPairNeighbours)
    return bf16 ? pick_lanes<__bf16, 8, true>(a, backward, s) : pick_lanes<float, 4, true>(a, backward, s);
  if (!bf16) return pick_lanes<float, 4, false>(a, backward, s);
  return wide ? pick_lanes<__bf16, 8, false>(a, backward, s) : pick_lanes<__bf16, 4, false>(a, backward, s);
}
hipError_t launch_qk_sum(const QkSumArgs& a, hipStream_t stream) {
  return launch_kernel(qk_sum_kernel, (2 * a.dim + kSumCols - 1) / kSumCols, kSumThreads, a, stream);
}

}  // namespace muon
