// gfx950 (CDNA4) embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: y[t] = scale * table[id_t]; an id outside the table gives a row of zeros.
// Backward: dtable[v] = scale * sum of dout[t] over the tokens t with id_t = v, in
// fp32 and in an order that only the ids decide: the tokens are sorted by id
// (stable radix sort, so in token order within an id), each wave sums a chunk
// of the sorted list, and ids that reach over a chunk's end are joined in order.
#include "block_internal.h"
#include "device_common.h"
#include "row_vectors.h"

namespace muon {
namespace {

// The id of a token as the table's row, or `vocab` outside it.
__device__ __forceinline__ uint32_t id_at(const void* ids, bool id64, int64_t t, int64_t vocab) {
  const int64_t id = id64 ? *gv<int64_t>((const int64_t*)ids + t) : *gv<int32_t>((const int32_t*)ids + t);
  return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}

// ---------------------------------------------------------------- forward --
// A block takes a.rows tokens, whose ids it holds in LDS, and its threads the
// vectors of those rows in turn.
constexpr int kMaxRows = 256;
template <class T, class O, bool PART>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(EmbedArgs a) {
  constexpr int VEC = sizeof(T) == 4 && sizeof(O) == 4 ? 4 : 8;
  __shared__ uint32_t id[kMaxRows];
  const uint32_t vectors = (uint32_t)(a.cols + VEC - 1) / VEC;
  for (int64_t first = (int64_t)blockIdx.x * a.rows; first < a.tokens; first += (int64_t)gridDim.x * a.rows) {
    const int rows = (int)min((int64_t)a.rows, a.tokens - first);
    __syncthreads();  // the ids before have been read
    for (int i = threadIdx.x; i < rows; i += kThreads) id[i] = id_at(a.ids, a.id64, first + i, a.vocab);
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < rows * vectors; j += kThreads) {
      const uint32_t r = a.rows == 1 ? 0 : vectors == 1 ? j : __umulhi(j, a.magic);
      const int c = (int)(j - r * vectors) * VEC, n = PART ? min(a.cols - c, VEC) : VEC;
      float v[VEC];
      if (id[r] < (uint32_t)a.vocab) {
        load_part<T, VEC, PART>((const T*)a.table + id[r] * a.ld_table + c, n, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= a.scale;
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = 0.f;
      }
      store_part<O, VEC, PART>((O*)a.out + (first + r) * a.ld_out + c, n, v);
    }
  }
}

// ------------------------------------------------------------------- sort --
// One pass sorts by `digit` bits of the id: every block counts its segment's
// digits, then every block finds its places from all blocks' counts and moves
// its entries there.  The last pass's output is sorted; the tokens' order is
// kept among equals.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ EmbedEntry entry_at(const EmbedGradArgs& a, int64_t i) {
  if (a.pass == 0) return EmbedEntry{id_at(a.ids, a.id64, i, a.vocab), (uint32_t)i};
  return a.entry[(a.pass + 1) & 1][i];
}

__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedGradArgs a) {
  __shared__ uint32_t count[1 << kMaxDigit];
  const int bins = 1 << a.digit;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) count[i] = 0;
  if (a.pass == 0)
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < a.vocab; i += (int64_t)a.blocks * kSortThreads)
      a.present[i] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.segment, last = min(first + a.segment, a.tokens);
  for (int64_t i = first + threadIdx.x; i < last; i += kSortThreads)
    atomicAdd(&count[entry_at(a, i).id >> (a.pass * a.digit) & (bins - 1)], 1u);
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) a.hist[(int64_t)blockIdx.x * bins + i] = count[i];
}

__global__ __launch_bounds__(kSortThreads) void embed_move_kernel(EmbedGradArgs a) {
  __shared__ uint32_t base[1 << kMaxDigit];                // where the digit's next entry goes
  __shared__ uint16_t place[kSortWaves][1 << kMaxDigit];   // a wave's count of a digit, then its place after base
  __shared__ uint32_t wave_sum[kSortWaves];
  const int bins = 1 << a.digit, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  {
    // a thread a digit (at most 1024): entries of lower digits, and of this digit in earlier blocks
    uint32_t before = 0, total = 0;
    if ((int)threadIdx.x < bins)
      for (int b = 0; b < a.blocks; ++b) {
        const uint32_t n = a.hist[(int64_t)b * bins + threadIdx.x];
        before += b < (int)blockIdx.x ? n : 0;
        total += n;
      }
    uint32_t scan = total;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const uint32_t n = __shfl_up(scan, o);
      if (lane >= o) scan += n;
    }
    if (lane == 63) wave_sum[wave] = scan;
    __syncthreads();
    uint32_t lower = scan - total;
    for (int w = 0; w < wave; ++w) lower += wave_sum[w];
    if ((int)threadIdx.x < bins) base[threadIdx.x] = lower + before;
  }
  const int64_t first = (int64_t)blockIdx.x * a.segment, last = min(first + a.segment, a.tokens);
  for (int64_t at = first; at < last; at += kSortThreads) {
    __syncthreads();  // base is written; the previous round's places are read
    for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) place[i / bins][i % bins] = 0;
    __syncthreads();
    const int64_t i = at + threadIdx.x;
    const bool on = i < last;
    const EmbedEntry e = on ? entry_at(a, i) : EmbedEntry{};
    const uint32_t d = e.id >> (a.pass * a.digit) & (bins - 1);
    uint64_t same = __ballot(on);
    for (int b = 0; b < a.digit; ++b) {
      const uint64_t set = __ballot(d >> b & 1);
      same &= d >> b & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (on && rank == 0) place[wave][d] = (uint16_t)__popcll(same);
    __syncthreads();
    uint32_t sum = 0;
    if ((int)threadIdx.x < bins)
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t n = place[w][threadIdx.x];
        place[w][threadIdx.x] = (uint16_t)sum;
        sum += n;
      }
    __syncthreads();
    if (on) {
      a.entry[a.pass & 1][base[d] + place[wave][d] + rank] = e;
      if (a.pass == 0 && e.id < (uint32_t)a.vocab) a.present[e.id] = 1;
    }
    __syncthreads();
    if ((int)threadIdx.x < bins) base[threadIdx.x] += sum;
  }
}

// -------------------------------------------------------------------- sums --
template <class T, int VEC, bool PART>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, uint32_t id, int c, int n, float* v) {
  T* p = (T*)a.dtable + id * a.ld_dtable + c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= a.scale;
  if (a.accumulate) {
    float old[VEC];
    load_part<T, VEC, PART>(p, n, old);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] += old[e];
  }
  store_part<T, VEC, PART>(p, n, v);
}

// A wave sums a chunk of the sorted list over 64 vectors of columns.  An id's
// run goes to its row of the table if it lies within the chunk; otherwise to
// part[chunk][0] if it came in from the chunk before, to [1] if it starts here.
template <class T, class O, bool PART>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<O>, AHEAD = 8;
  const int lane = threadIdx.x % 64;
  const int slices = (a.cols + 64 * VEC - 1) / (64 * VEC);
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
  const int64_t chunk = unit / slices, first = chunk * kEmbedChunk;
  if (first >= a.tokens) return;
  const int c = ((int)(unit % slices) * 64 + lane) * VEC, n = min(a.cols - c, VEC);
  const int count = (int)min((int64_t)kEmbedChunk, a.tokens - first);
  const EmbedEntry* list = a.entry[(a.passes - 1) & 1];
  const uint32_t none = 0xFFFFFFFFu;
  EmbedEntry mine{none, 0};
  const int64_t i = first - 1 + lane;  // one before the chunk, and one behind
  if (lane < count + 2 && i >= 0 && i < a.tokens) mine = list[i];
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  uint32_t id = __builtin_amdgcn_readlane(mine.id, 1);
  bool began = __builtin_amdgcn_readlane(mine.id, 0) == id;  // in the chunk before
  for (int k = 0; k < count; k += AHEAD) {
    float v[AHEAD][VEC];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (k + q >= count) break;
      const uint32_t token = __builtin_amdgcn_readlane(mine.token, k + q + 1);
      if (n > 0) load_part<O, VEC, PART>((const O*)a.dout + token * a.ld_dout + c, n, v[q]);
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (k + q >= count) break;
      if (id == (uint32_t)a.vocab) return;  // sorted last: nothing more counts
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[q][e];
      const uint32_t next = __builtin_amdgcn_readlane(mine.id, k + q + 2);
      const bool end = k + q + 1 == count;
      if (next == id && !end) continue;
      if (n > 0) {
        if (began || next == id)
          store_part<float, VEC, PART>(a.part + (chunk * 2 + (began ? 0 : 1)) * a.cols + c, n, acc);
        else
          write_row<T, VEC, PART>(a, id, c, n, acc);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      id = next;
      began = false;
    }
  }
}

// Adds the parts of the ids that reach over chunks: the wave of the chunk where an id's run starts.
template <class T, class O, bool PART>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<O>;
  const int lane = threadIdx.x % 64;
  const int slices = (a.cols + 64 * VEC - 1) / (64 * VEC);
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
  const int64_t chunk = unit / slices, first = chunk * kEmbedChunk, end = first + kEmbedChunk;
  if (end >= a.tokens) return;
  const EmbedEntry* list = a.entry[(a.passes - 1) & 1];
  const uint32_t id = list[end - 1].id;
  if (id == (uint32_t)a.vocab || list[end].id != id) return;                   // ends here
  if (list[first].id == id && first > 0 && list[first - 1].id == id) return;  // came in from before
  const int c = ((int)(unit % slices) * 64 + lane) * VEC, n = min(a.cols - c, VEC);
  float acc[VEC], v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  if (n > 0) load_part<float, VEC, PART>(a.part + (chunk * 2 + 1) * a.cols + c, n, acc);
  for (int64_t at = chunk + 1;; at += 64) {
    const int64_t i = (at + lane) * kEmbedChunk;
    const uint64_t on = __ballot(i < a.tokens && list[i].id == id);
    const int more = __builtin_ctzll(~on | 1ull << 63);
    const int parts = on == ~0ull ? 64 : more;
    if (n > 0)
      for (int k = 0; k < parts; ++k) {
        load_part<float, VEC, PART>(a.part + (at + k) * 2 * a.cols + c, n, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      }
    if (parts < 64) break;
  }
  if (n > 0) write_row<T, VEC, PART>(a, id, c, n, acc);
}

// Zeros in the rows that no token has: a wave a row.
template <class T>
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<T>;
  const int lane = threadIdx.x % 64;
  const float zero[VEC] = {};
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; row < a.vocab;
       row += (int64_t)gridDim.x * (kThreads / 64)) {
    if (a.tokens && a.present[row]) continue;
    T* p = (T*)a.dtable + row * a.ld_dtable;
    for (int c = lane * VEC; c < a.cols; c += 64 * VEC) store_part<T, VEC, true>(p + c, min(a.cols - c, VEC), zero);
  }
}

// ----------------------------------------------------------------- launch --
constexpr int64_t kForwardBlocks = 1 << 20;  // what is left is taken in turn: a launch holds fewer than 2^32 threads
template <class T, class O>
hipError_t run_forward(const EmbedArgs& args, hipStream_t s) {
  constexpr int VEC = sizeof(T) == 4 && sizeof(O) == 4 ? 4 : 8;
  EmbedArgs a = args;
  const int vectors = (a.cols + VEC - 1) / VEC;
  // about four vectors a thread; a block's vectors, below 2048, are divided exactly by the multiplication
  a.rows = vectors >= 4 * kThreads ? 1 : (4 * kThreads + vectors - 1) / vectors;
  if (a.rows > kMaxRows) a.rows = kMaxRows;
  a.magic = (uint32_t)(((1ull << 32) + vectors - 1) / vectors);
  const int64_t blocks = (a.tokens + a.rows - 1) / a.rows;
  const int64_t grid = blocks < kForwardBlocks ? blocks : kForwardBlocks;
  return a.cols % VEC ? launch_kernel(embed_forward_kernel<T, O, true>, grid, kThreads, a, s)
                      : launch_kernel(embed_forward_kernel<T, O, false>, grid, kThreads, a, s);
}

template <class T, class O, bool PART>
hipError_t run_backward(EmbedGradArgs a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.tokens) {
    for (a.pass = 0; a.pass < a.passes && e == hipSuccess; ++a.pass) {
      e = launch_kernel(embed_count_kernel, a.blocks, kSortThreads, a, s);
      if (e == hipSuccess) e = launch_kernel(embed_move_kernel, a.blocks, kSortThreads, a, s);
    }
    const int64_t chunks = (a.tokens + kEmbedChunk - 1) / kEmbedChunk;
    const int64_t slices = (a.cols + 64 * kVec<O> - 1) / (64 * kVec<O>);
    const int64_t grid = (chunks * slices + kThreads / 64 - 1) / (kThreads / 64);
    if (e == hipSuccess) e = launch_kernel(embed_sum_kernel<T, O, PART>, grid, kThreads, a, s);
    if (e == hipSuccess) e = launch_kernel(embed_join_kernel<T, O, PART>, grid, kThreads, a, s);
  }
  if (e == hipSuccess && !a.accumulate) {
    const int64_t need = (a.vocab + kThreads / 64 - 1) / (kThreads / 64);
    e = launch_kernel(embed_zero_kernel<T>, need < 4096 ? need : 4096, kThreads, a, s);
  }
  return e;
}
template <class T, class O>
hipError_t pick_part(const EmbedGradArgs& a, hipStream_t s) {
  return a.cols % kVec<O> ? run_backward<T, O, true>(a, s) : run_backward<T, O, false>(a, s);
}

}  // namespace

void plan_embed(EmbedGradArgs& a) {
  const int64_t want = (a.tokens + kSortThreads - 1) / kSortThreads;
  const int64_t blocks = want < 1 ? 1 : want < 256 ? want : 256;
  const int64_t each = (a.tokens + blocks - 1) / blocks;
  a.segment = (int32_t)((each + kSortThreads - 1) / kSortThreads * kSortThreads);
  a.blocks = (int32_t)blocks;
  int bits = 1;
  while (bits < 31 && a.vocab >> bits) ++bits;  // ids 0 .. vocab
  a.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  a.digit = (bits + a.passes - 1) / a.passes;
}

hipError_t launch_embed_forward(const EmbedArgs& a, bool table_bf16, bool out_bf16, hipStream_t s) {
  if (table_bf16) return out_bf16 ? run_forward<__bf16, __bf16>(a, s) : run_forward<__bf16, float>(a, s);
  return out_bf16 ? run_forward<float, __bf16>(a, s) : run_forward<float, float>(a, s);
}
hipError_t launch_embed_backward(const EmbedGradArgs& a, bool table_bf16, bool out_bf16, hipStream_t s) {
  if (table_bf16) return out_bf16 ? pick_part<__bf16, __bf16>(a, s) : pick_part<__bf16, float>(a, s);
  return out_bf16 ? pick_part<float, __bf16>(a, s) : pick_part<float, float>(a, s);
}

}  // namespace muon
