// experts.hip -- HIP kernels and C ABI of the mixture-of-experts operators for AMD
// Instinct MI355X (gfx950, CDNA4, wave64):
//   dp_expert_route         a token's experts and their weights from its logits
//   dp_expert_route_grad    the gradient of the weights, to the logits
//   dp_expert_sort          places of the tokens' slots sorted by expert
//   dp_expert_dispatch      tokens' rows to those places
//   dp_expert_combine       rows back, summed with the weights (and the gradient
//                           of the dispatch)
//   dp_expert_combine_grad  gradient of that sum: to the rows and to the weights
//
// All are bound by HBM or, where small, by their launches: at most three flops
// per byte (the router apart, which its instructions bound).  Integer atomics in LDS
// only, so every result bit is the same from run to run.  Times below are of one
// MI355X, on three sets of inputs in turn unless a comment says one set (whose rows the
// caches then hold): of a kernel in a trace or a replayed graph of its calls, which agree
// within 0.6 us, or of a call from Python among others, where it says call.

#include <hip/hip_runtime.h>

#include <algorithm>

#include <limits.h>
#include <stdint.h>

#include "grz.h"
#include "rows.h"

namespace {

constexpr int64_t kSlots = int64_t{1} << 28;       // n * k of one call
constexpr int64_t kCols = int64_t{65535} * 64;     // columns of one call
constexpr int64_t kTokenBatch = int64_t{1} << 20;  // tokens of one launch
constexpr int64_t kUnitBatch = int64_t{1} << 23;   // their runs of columns, a wave each
constexpr float kLog2e = 1.44269504088896340736f;

// ---------------------------------------------------------------------------
// Vectors of a row that begin anywhere: gfx950 reads and writes 8 and 16 bytes at
// any element's address, so rows need no alignment of their own (8000 x 1601 bf16 to
// 4 experts, every row off the lines: 36 us for 128 MB, sort included, and back 25;
// 8000 x 1600 27 and 22).  Vectors shifted onto each row's own lines were slower.

// N consecutive elements as they lie in memory (8 or 16 bytes), widened one by one
// where they are used: many loads wait in few registers.
template <typename T, int N> struct Cols {
  static constexpr int kWords = N * sizeof(T) / 4;
  static_assert(kWords == 2 || kWords == 4, "accesses of 8 or 16 bytes");
  uint32_t w[kWords];
  template <bool STREAM = false> __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const u32x4e* q = reinterpret_cast<const u32x4e*>(p);
      u32x4 u;
      if constexpr (STREAM) u = __builtin_nontemporal_load(q);
      else u = *q;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = u[i];
    } else {
      const u32x2e* q = reinterpret_cast<const u32x2e*>(p);
      u32x2 u;
      if constexpr (STREAM) u = __builtin_nontemporal_load(q);
      else u = *q;
      w[0] = u[0];
      w[1] = u[1];
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

template <bool STREAM> __device__ __forceinline__ void store_words(void* p, u32x4 v) {
  u32x4e* q = static_cast<u32x4e*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}
template <bool STREAM> __device__ __forceinline__ void store_words(void* p, u32x2 v) {
  u32x2e* q = static_cast<u32x2e*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}

template <typename T, int N, bool STREAM = true>
__device__ __forceinline__ void store_cols(T* p, const float (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      u[i] = bf16_bits(x[2 * i]) | (bf16_bits(x[2 * i + 1]) << 16);
    if constexpr (N == 8) store_words<STREAM>(p, u32x4{u[0], u[1], u[2], u[3]});
    else store_words<STREAM>(p, u32x2{u[0], u[1]});
  } else {
    store_words<STREAM>(p, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]),
                                 __float_as_uint(x[2]), __float_as_uint(x[3])});
  }
}

// Columns of a lane's vector: 16 bytes, of fp32 if one of the types is.
template <typename A, typename B> constexpr int cols_of() {
  return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4;
}

__device__ __forceinline__ int wave_index() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// A wave's token and run of columns: the runs of a token's row are neighbours, so
// that a row is read or written at one time (runs a launch's length apart: 16384 x
// 4096 bf16 dispatched to 6 experts 205 instead of 177 us, combined 185 instead of 162).
struct Unit {
  int64_t token;
  int part;
};
template <int WAVES> __device__ __forceinline__ Unit unit_of(int64_t row0, int parts) {
  const uint32_t unit = blockIdx.x * WAVES + wave_index();
  const uint32_t token = unit / static_cast<uint32_t>(parts);
  return {row0 + token, static_cast<int>(unit - token * parts)};
}

// ---------------------------------------------------------------------------
// The router.  A row of up to 1024 logits stays in the registers of G lanes (16,
// four rows to a wave, or 64), V in each, so that every maximum and sum is V
// operations and four (or six) lane exchanges.  The k largest come one at a time: the
// row's largest key, the lowest element that has it, which is then taken out.  Bound by
// those rounds' instructions (V a round, so k V): normalized, k = 8, 16384 x 128 bf16 5.8
// us for 5 MB, fp32 6.8; 16384 x 256 7.8 and 10.8; 0.3 to 0.7 more not normalized.

// Keys ordered as the logits are: larger for larger, NaN above all, -0 as 0, and 0
// for an element that is not there or taken out.
constexpr uint32_t kClosed = 0x007fffffu;  // the key of -inf
constexpr uint32_t kNanKey = 0xffffffffu;

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
  return x != x ? kNanKey : key;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
// A bf16 value's key is its upper half (the lower half is 0, or 0xffff below zero, and
// is restored from its sign), which leaves room for the element's number, lower ones
// first: one maximum then finds both (16384 x 256 bf16, k = 8, one set: 9.2 us without,
// 7.7 with).
__device__ __forceinline__ uint32_t numbered(uint32_t key, int number) {
  return (key & 0xffff0000u) | (0xffffu - static_cast<uint32_t>(number));
}
__device__ __forceinline__ uint32_t unnumbered(uint32_t key) {
  return key & 0x80000000u ? key & 0xffff0000u : key | 0xffffu;
}

template <int CTRL> __device__ __forceinline__ uint32_t lane_swap_bits(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

template <int G, typename F> __device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, lane_swap_bits<kSwap1>(v));
  v = f(v, lane_swap_bits<kSwap2>(v));
  v = f(v, lane_swap_bits<kHalfMirror>(v));
  v = f(v, lane_swap_bits<kMirror>(v));
  if constexpr (G == 64) {
    auto row = [&](int lane) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(v, lane)); };
    v = f(f(row(0), row(16)), f(row(32), row(48)));
  }
  return v;
}
template <int G> __device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G> __device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int G> __device__ __forceinline__ float group_max(float v) {
  if constexpr (G == 64) return wave_max(v);
  v = fmaxf(v, lane_swap<kSwap1>(v));
  v = fmaxf(v, lane_swap<kSwap2>(v));
  v = fmaxf(v, lane_swap<kHalfMirror>(v));
  return fmaxf(v, lane_swap<kMirror>(v));
}
template <int G> __device__ __forceinline__ float group_sum(float v) {
  if constexpr (G == 64) return wave_sum(v);
  v += lane_swap<kSwap1>(v);
  v += lane_swap<kSwap2>(v);
  v += lane_swap<kHalfMirror>(v);
  return v + lane_swap<kMirror>(v);
}
// The lanes of the thread's group for which `yes` holds, the group's first at bit 0.
template <int G> __device__ __forceinline__ uint64_t group_ballot(bool yes) {
  const uint64_t b = __ballot(yes);
  if constexpr (G == 64) return b;
  return (b >> (threadIdx.x & 48)) & 0xffffu;
}

// e^(x - m) of an open expert, 0 of a closed one; one rounding each of the
// difference and its product.
__device__ __forceinline__ float weight_of(float x, float m) {
  return x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((x - m) * kLog2e);
}

// Which of the row's elements a lane of the group holds: runs of `kRun` (one access),
// the group's runs side by side, so that each access of a wave is one run of memory a
// row (with V consecutive elements a lane the gradient of 16384 x 256, one set, took 7.6
// us bf16 and 14.9 fp32, instead of 6.1 and 6.4).
template <typename T, int G, int V> struct Share {
  static constexpr int kRun = V == 1 ? 1 : sizeof(T) == 2 && V >= 8 ? 8 : 4;
  int g;
  __device__ __forceinline__ int first(int h) const { return (h * G + g) * kRun; }
  __device__ __forceinline__ int at(int i) const { return first(i / kRun) + i % kRun; }

  // The elements, -inf behind the last.
  __device__ __forceinline__ void load(const T* row, int experts, bool live,
                                       float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = -INFINITY;
    if (!live) return;
#pragma unroll
    for (int h = 0; h < V / kRun; ++h) {
      const int c = first(h);
      bool vector = false;
      if constexpr (kRun > 1) {
        vector = c + kRun <= experts;
        if (vector) {
          Cols<T, kRun> y;
          y.load(row + c);
#pragma unroll
          for (int i = 0; i < kRun; ++i) x[h * kRun + i] = y[i];
        }
      }
      if (!vector) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (c + i < experts) x[h * kRun + i] = widen(row[c + i]);
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int experts, const float (&x)[V]) const {
#pragma unroll
    for (int h = 0; h < V / kRun; ++h) {
      const int c = first(h);
      bool vector = false;
      if constexpr (kRun > 1) {
        vector = c + kRun <= experts;
        if (vector) {
          float y[kRun];
#pragma unroll
          for (int i = 0; i < kRun; ++i) y[i] = x[h * kRun + i];
          store_cols<T, kRun, false>(row + c, y);
        }
      }
      if (!vector) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (c + i < experts) put(row + c + i, x[h * kRun + i]);
      }
    }
  }
};

template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_kernel(const T* __restrict__ logits, int64_t stride,
                                                    int64_t row0, int64_t n, int experts, int k,
                                                    bool normalize, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const Share<T, G, V> share{static_cast<int>(threadIdx.x & (G - 1))};
  const int g = share.g;
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G;
  const bool live = row < n;
  float x[V];
  share.load(logits + (live ? row : 0) * stride, experts, live, x);
  constexpr bool kNumbered = sizeof(T) == 2;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int number = share.at(i);
    key[i] = key_of(x[i]);
    if constexpr (kNumbered) key[i] = numbered(key[i], number);
    if (!live || number >= experts) key[i] = 0;
  }
  // The row's largest key; its element's number and, in `top`, its value's key.
  auto next = [&](uint32_t& top) {
    uint32_t best = 0, at = UINT32_MAX;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    best = group_max<G>(best);
    if constexpr (kNumbered) {
      at = 0xffffu - (best & 0xffffu);
      top = unnumbered(best);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] == best ? 0u : key[i];
    } else {
      top = best;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == best) at = share.at(i);
      at = group_min<G>(at);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (share.at(i) == static_cast<int>(at)) key[i] = 0;
    }
    return static_cast<int>(at);
  };
  uint32_t top;
  int at = next(top);
  const float m = value_of(top);
  float total = 0.0f;
  if (!normalize) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += weight_of(x[i], m);
    total = group_sum<G>(total);
  }
  int id = -1;
  float e = 0.0f;  // of the slot that the thread stores
  for (int j = 0; j < k; ++j) {
    if (j > 0) at = next(top);
    const float p = top > kClosed ? weight_of(value_of(top), m) : 0.0f;
    if (normalize) total += p;
    if (g == j) {
      id = top > kClosed ? at : -1;
      e = p;
    }
  }
  if (live && g < k) {
    ids[row * k + g] = id;
    weights[row * k + g] = id >= 0 ? e / total : 0.0f;
  }
}

// Lane j of a row's group takes slot j.  The slots' shares meet the row through
// LDS, where each lane finds those of its elements; a token that lists an expert
// twice has both slots add theirs up first, in the slots' order.  Normalized weights
// depend on the listed logits alone, so only those are read.  16384 x 256 bf16, k = 8:
// 6.8 us, 8.4 not normalized (17 MB); fp32 7.3 and 10.9.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_grad_kernel(
    const T* logits, int64_t stride, int64_t row0, int64_t n, int experts, int k, bool normalize,
    const int32_t* __restrict__ ids, const float* __restrict__ dweights, T* dlogits,
    int64_t dstride) {
  __shared__ float shares[256 / G][G * V];
  const Share<T, G, V> share_of{static_cast<int>(threadIdx.x & (G - 1))};
  const int g = share_of.g;
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G;
  const bool live = row < n;
  const T* src = logits + (live ? row : 0) * stride;
  float* mine = shares[threadIdx.x / G];
  int id = -1;
  float dw = 0.0f, xj = -INFINITY;
  if (live && g < k) {
    id = ids[row * k + g];
    if (id < 0 || id >= experts) id = -1;
    if (id >= 0) {
      dw = dweights[row * k + g];
      xj = widen(src[id]);
    }
  }
  float x[V] = {}, m, total = 0.0f, ej;
  if (normalize) {
    m = group_max<G>(xj);
    ej = weight_of(xj, m);
    total = group_sum<G>(ej);
  } else {
    share_of.load(src, experts, live, x);
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = group_max<G>(m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = weight_of(x[i], m);
      total += x[i];
    }
    total = group_sum<G>(total);
    ej = weight_of(xj, m);
  }
  const float w = total == 0.0f ? 0.0f : ej / total;
  const float both = group_sum<G>(id >= 0 ? dw * w : 0.0f);
  const float share = id < 0 ? 0.0f : w * (normalize ? dw - both : dw);
  const bool some = group_ballot<G>(id >= 0 && dw != 0.0f) != 0;
#pragma unroll
  for (int i = 0; i < V; ++i) mine[share_of.at(i)] = 0.0f;
  float sum = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int other = __shfl(id, j, G);
    const float s = __shfl(share, j, G);
    if (other == id) sum += s;
  }
  wave_fence();
  if (id >= 0) mine[id] = sum;  // equal ids store the same sum
  wave_fence();
  if (!live) return;
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    d[i] = mine[share_of.at(i)];
    if (!normalize) d[i] -= total == 0.0f ? 0.0f : both * (x[i] / total);
    if (!some) d[i] = 0.0f;
  }
  share_of.store(dlogits + row * dstride, experts, d);
}

// ---------------------------------------------------------------------------
// The sort of the slots by expert: stable, so a place is the number of slots of
// lower experts, plus the slots of the same expert before it.  A workgroup places
// a tile of slots, 1024 at a time: the ballots of the id's bits give a slot's
// place among the equal ones of its wave, counts in LDS those of the waves before
// it, and `before` those of the tiles before its own.
//
//  - up to kDirectSlots one launch: each workgroup counts all slots itself, those
//    before its tile and all, with integer atomics in LDS;
//  - beyond that the tiles are counted by a first launch and each workgroup adds all
//    tiles' counts up (98304 slots of 64 experts 8.7 us: 2.4 and 6.4 in a trace, 4.8 and
//    6.0 where the ids come from HBM).  At most kMaxTiles tiles, and at most kTileCounts
//    counts, since everyone reads them (524288 slots of 1024 experts: 24.6 us, 28.2 with
//    256 tiles, 30.7 with 64).
//
// One launch and two, us, ids spread evenly:
//   slots    of 2          8          64         1024 experts   all of one of 64
//   4096     7.6  7.5   5.8  6.9   5.4  7.1   6.5  9.3      10.4  7.5
//   8192    11.5  7.5   7.5  7.0   6.2  7.2   7.3  9.0      17.3  7.7
//   16384   19.5  7.6  10.9  7.0   7.8  7.4   9.0  9.5      30.9  7.8
// The lanes of a wave add to one count one after the other, so few experts, or ids that
// are much alike, make the one launch slow.  The limit takes the slots alone: at
// 8192 of them it loses 0.5 us with 8 experts and saves 1.0 with 64, and how alike the
// ids are is known on the device only.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int64_t kDirectSlots = 8192;
constexpr int64_t kMaxTiles = 256, kTileCounts = 131072;

struct SortArgs {
  const void* ids;
  int id_bits;
  int64_t slots;
  int experts;
  int bits;       // of `experts`
  int64_t tile;   // slots of a tile, a multiple of kSortThreads
  int tiles;
  uint32_t* counts;  // [tiles][experts]
  int32_t* offsets;
  int32_t* places;
};

// The slot's expert, `experts` for none.
__device__ __forceinline__ int expert_at(const SortArgs& a, int64_t i) {
  const int64_t id = id_at(a.ids, a.id_bits, i);
  return id >= 0 && id < a.experts ? static_cast<int>(id) : a.experts;
}

__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortArgs a) {
  __shared__ uint32_t count[GRZ_MAX_EXPERTS];
  if (threadIdx.x < a.experts) count[threadIdx.x] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * a.tile;
  const int64_t to = from + a.tile < a.slots ? from + a.tile : a.slots;
  for (int64_t i = from + threadIdx.x; i < to; i += kSortThreads) {
    const int e = expert_at(a, i);
    if (e < a.experts) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  if (threadIdx.x < a.experts)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + threadIdx.x] = count[threadIdx.x];
}

template <bool DIRECT>
__global__ __launch_bounds__(kSortThreads) void expert_place_kernel(SortArgs a) {
  __shared__ uint32_t before[GRZ_MAX_EXPERTS], total[GRZ_MAX_EXPERTS];
  __shared__ uint32_t sums[kSortWaves];
  extern __shared__ uint16_t in_wave[];  // [kSortWaves][experts]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, experts = a.experts;
  const int64_t from = blockIdx.x * a.tile;
  const int64_t to = from + a.tile < a.slots ? from + a.tile : a.slots;
  if (tid < experts) before[tid] = total[tid] = 0;
  __syncthreads();
  if constexpr (DIRECT) {
#pragma unroll 4
    for (int64_t i = tid; i < a.slots; i += kSortThreads) {
      const int e = expert_at(a, i);
      if (e < experts) {
        atomicAdd(&total[e], 1u);
        if (i < from) atomicAdd(&before[e], 1u);
      }
    }
  } else {
    const int parts = kSortThreads / experts, e = tid % experts, part = tid / experts;
    if (part < parts) {
      uint32_t b = 0, t = 0;
#pragma unroll 8
      for (int k = part; k < a.tiles; k += parts) {
        const uint32_t c = a.counts[static_cast<int64_t>(k) * experts + e];
        t += c;
        b += k < static_cast<int>(blockIdx.x) ? c : 0u;
      }
      atomicAdd(&before[e], b);
      atomicAdd(&total[e], t);
    }
  }
  __syncthreads();
  // The experts' first rows: an exclusive scan of their totals.
  const uint32_t own = tid < experts ? total[tid] : 0u;
  uint32_t scan = own;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint32_t v = __shfl_up(scan, s, 64);
    if (lane >= s) scan += v;
  }
  if (lane == 63) sums[wave] = scan;
  __syncthreads();
  for (int w = 0; w < wave; ++w) scan += sums[w];
  if (tid < experts) {
    before[tid] += scan - own;
    if (blockIdx.x == 0) {
      a.offsets[tid] = static_cast<int32_t>(scan - own);
      if (tid == experts - 1) a.offsets[experts] = static_cast<int32_t>(scan);
    }
  }
  for (int64_t base = from; base < to; base += kSortThreads) {
    const int64_t i = base + tid;
    const int e = i < to ? expert_at(a, i) : experts;
    uint16_t* counts = in_wave + wave * experts;
    for (int c = lane; c < experts; c += 64) counts[c] = 0;
    uint64_t same = ~0ull;
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t v = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? v : ~v;
    }
    const uint32_t rank = static_cast<uint32_t>(__popcll(same & ((1ull << lane) - 1)));
    wave_fence();
    if (e < experts && rank == 0) counts[e] = static_cast<uint16_t>(__popcll(same));
    __syncthreads();
    uint32_t run = 0;
    if (tid < experts) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = in_wave[w * experts + tid];
        in_wave[w * experts + tid] = static_cast<uint16_t>(run);
        run += c;
      }
    }
    __syncthreads();
    if (i < to)
      a.places[i] = e < experts ? static_cast<int32_t>(before[e] + counts[e] + rank) : -1;
    __syncthreads();
    if (tid < experts) before[tid] += run;
  }
}

// ---------------------------------------------------------------------------
// Rows to their places and back: a wave takes a token and a run of its columns,
// its lanes 16-byte vectors along them; a token's places are the wave's, so they
// sit in scalar registers.  The columns behind the last whole vector are taken one
// by one by the waves of the last run.

// out[places[i][j]] = (weights[i][j]) x[i]: the row is read once and stored k times.
// Bound by HBM, and by what 64 experts' rows written side by side cost it: 16384 x
// 4096 bf16 to 6 experts of 64 147-160 us, 5.9-6.4 TB/s (places in the tokens' order
// 8 % less).  Small workgroups free their slots one by one: 174 us a call with two waves,
// 175 with four, 186 with eight; two or four vectors a lane 192 and 195.  Where rows lie
// off the lines, neighbouring waves write halves of one, which have to meet in one L2, so
// in one workgroup: 16384 x 2056 fp32 to 3 bf16 rows 91 us with two waves, 80 with four,
// 75 with eight; 4000 x 4097 bf16 to 8 83, 76 and 74.
template <typename TI, typename TO, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void dispatch_kernel(
    const TI* __restrict__ x, int64_t xstride, const int32_t* __restrict__ places,
    const float* __restrict__ weights, int64_t row0, int64_t n, int k, int64_t dim, int parts,
    int64_t rows, TO* __restrict__ out, int64_t ostride) {
  constexpr int VEC = cols_of<TI, TO>();
  const int lane = threadIdx.x & 63;
  const auto [token, run] = unit_of<WAVES>(row0, parts);
  if (token >= n) return;
  const TI* src = x + token * xstride;
  const int64_t whole = dim - dim % VEC;
  const int64_t c = static_cast<int64_t>(run) * (64 * VEC) + lane * VEC;
  const bool in = c < whole, tail = run == parts - 1 && lane < dim - whole;
  Cols<TI, VEC> v = {};
  float last = 0.0f;
  if (in) v.load(src + c);
  if (tail) last = widen(src[whole + lane]);
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[token * k + j];
    if (p < 0 || p >= rows) continue;
    const float w = weights != nullptr ? weights[token * k + j] : 1.0f;
    TO* dst = out + p * ostride;
    if (in) {
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = v[i] * w;
      store_cols<TO, VEC>(dst + c, y);
    }
    if (tail) put(dst + whole + lane, last * w);
  }
}

// out[i] = sum over j of (weights[i][j]) y[places[i][j]], added to out[i] with ACC:
// KB rows' vectors on their way at once, summed in the slots' order.  Bound by HBM:
// 16384 x 4096 bf16 from 6 rows 155 us, 6.0 TB/s; 8011 x 1600 fp32 from 2, added, 31.6
// us, 6.4 TB/s.
constexpr int kCombineWaves = 4;

template <typename TI, typename TO, int U, int KB, bool ACC, bool STREAM>
__global__ __launch_bounds__(kCombineWaves * 64) void combine_kernel(
    const TI* __restrict__ y, int64_t ystride, int64_t rows, const int32_t* __restrict__ places,
    const float* __restrict__ weights, int64_t row0, int64_t n, int k, int64_t dim, int parts,
    TO* __restrict__ out, int64_t ostride) {
  constexpr int VEC = cols_of<TI, TO>();
  const int lane = threadIdx.x & 63;
  const auto [token, run] = unit_of<kCombineWaves>(row0, parts);
  if (token >= n) return;
  TO* dst = out + token * ostride;
  const int64_t whole = dim - dim % VEC;
  const int64_t c0 = static_cast<int64_t>(run) * (64 * VEC * U) + lane * VEC;
  const bool tail = run == parts - 1 && lane < dim - whole;
  float acc[U][VEC], last = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[u][i] = 0.0f;
    const int64_t c = c0 + u * 64 * VEC;
    if (ACC && c < whole) {
      Cols<TO, VEC> old;
      old.load(dst + c);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[u][i] = old[i];
    }
  }
  if (ACC && tail) last = widen(dst[whole + lane]);
  for (int j0 = 0; j0 < k; j0 += KB) {
    Cols<TI, VEC> v[KB][U] = {};
    float w[KB];
    int64_t p[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      p[b] = j0 + b < k ? places[token * k + j0 + b] : -1;
      if (p[b] >= rows) p[b] = -1;
      w[b] = weights != nullptr && p[b] >= 0 ? weights[token * k + j0 + b] : 1.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * 64 * VEC;
        if (p[b] >= 0 && c < whole) v[b][u].template load<STREAM>(y + p[b] * ystride + c);
      }
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if (p[b] < 0) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[u][i] = fmaf(v[b][u][i], w[b], acc[u][i]);
      if (tail) last = fmaf(widen(y[p[b] * ystride + whole + lane]), w[b], last);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + u * 64 * VEC;
    if (c < whole) store_cols<TO, VEC>(dst + c, acc[u]);
  }
  if (tail) put(dst + whole + lane, last);
}

// dy[places[i][j]] = weights[i][j] dout[i] and dweights[i][j] = <dout[i],
// y[places[i][j]]>: a wave to a slot, so that it streams one row of y and one of dy;
// the token's other slots are its neighbours and find dout[i] in the caches.  U
// vectors of each row on their way at once.  dy may be y: a lane stores where it has
// read.  Bound by HBM, reads and writes mixed: 16384 x 4096 bf16 to 6 rows 324 us, 5.3
// TB/s (places in the tokens' order 287; a wave a token with all its slots 363, four
// waves 333); 8192 x 768 to 2 rows 12.5 us.
constexpr int kGradWaves = 8;

template <typename TD, typename TY, int U, bool STREAM>
__global__ __launch_bounds__(kGradWaves * 64) void combine_grad_kernel(
    const TD* __restrict__ dout, int64_t dstride, const TY* y, int64_t ystride, int64_t rows,
    const int32_t* __restrict__ places, const float* __restrict__ weights, int64_t row0,
    int64_t n, int k, int64_t dim, TY* dy, int64_t dystride, float* __restrict__ dweights) {
  constexpr int VEC = cols_of<TD, TY>();
  const int lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * kGradWaves + wave_index();
  const int64_t token = row0 + unit / static_cast<uint32_t>(k);
  if (token >= n) return;
  const int64_t slot = row0 * k + unit;
  const int64_t p = places[slot];
  if (p < 0 || p >= rows) {
    if (dweights != nullptr && lane == 0) dweights[slot] = 0.0f;
    return;
  }
  const float w = weights != nullptr ? weights[slot] : 1.0f;
  const TD* src = dout + token * dstride;
  const TY* in = y + p * ystride;
  TY* dst = dy + p * dystride;
  const int64_t whole = dim - dim % VEC;
  float dot = 0.0f;
  for (int64_t c0 = lane * VEC; c0 < whole; c0 += 64 * VEC * U) {
    Cols<TD, VEC> d[U] = {};
    Cols<TY, VEC> v[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 64 * VEC;
      if (c >= whole) continue;
      d[u].load(src + c);
      if (dweights != nullptr) v[u].template load<STREAM>(in + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 64 * VEC;
      if (c >= whole) continue;
#pragma unroll
      for (int i = 0; i < VEC; ++i) dot = fmaf(d[u][i], v[u][i], dot);
      if (dy == nullptr) continue;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = d[u][i] * w;
      store_cols<TY, VEC>(dst + c, o);
    }
  }
  if (lane < dim - whole) {
    const float d = widen(src[whole + lane]);
    if (dweights != nullptr) dot = fmaf(d, widen(in[whole + lane]), dot);
    if (dy != nullptr) put(dst + whole + lane, d * w);
  }
  if (dweights == nullptr) return;
  dot = wave_sum(dot);
  if (lane == 0) dweights[slot] = dot;
}

// ---------------------------------------------------------------------------
// Host side.

// n x k arrays of 4-byte values.
int check_slots(const void* p, int64_t n, int k, bool may_be_null = false) {
  if (n == 0) return GRZ_OK;
  if (p == nullptr) return may_be_null ? GRZ_OK : GRZ_EINVAL;
  return aligned(p, 4) ? GRZ_OK : GRZ_EALIGN;
}
int check_counts(int64_t n, int k) {
  if (n < 0 || k < 1 || k > GRZ_MAX_SLOTS) return GRZ_EINVAL;
  return n > kSlots / k ? GRZ_ERANGE : GRZ_OK;
}

struct Span {
  const void* at;
  size_t bytes;
};
Span slot_span(const void* p, int64_t n, int k) {
  return {p, p != nullptr ? static_cast<size_t>(n) * k * 4 : 0};
}
Span matrix_span(const void* p, int dtype, int64_t rows, int64_t cols, int64_t stride) {
  return {p, p != nullptr ? span_of(dtype, rows, cols, stride) : 0};
}
// Whether an output lies over one of the other arrays.
template <int N> bool clash(const Span& out, const Span (&others)[N]) {
  for (const Span& s : others)
    if (overlap(out.at, out.bytes, s.at, s.bytes)) return true;
  return false;
}

// f(rows of the batch, first row) over at most `batch` tokens at a time.
template <typename F> int in_batches(int64_t n, int64_t batch, F f) {
  for (int64_t r = 0; r < n; r += batch) {
    const int st = f(n - r < batch ? n - r : batch, r);
    if (st != GRZ_OK) return st;
  }
  return GRZ_OK;
}

// Lanes to a row and logits to a lane.  Sixteen lanes up to 256 experts and 16
// slots: four rows share a wave's instructions (16384 x 512 bf16, which do not, take
// 15.1 us where 256 take 7.6).
#define GRZ_ROUTE_SHAPES(CALL)               \
  if (k <= 16 && experts <= 16) CALL(16, 1)  \
  if (k <= 16 && experts <= 64) CALL(16, 4)  \
  if (k <= 16 && experts <= 128) CALL(16, 8) \
  if (k <= 16 && experts <= 256) CALL(16, 16) \
  if (experts <= 256) CALL(64, 4)            \
  if (experts <= 512) CALL(64, 8)            \
  CALL(64, 16)

template <typename T>
int route_run(const void* logits, int64_t n, int experts, int64_t stride, int k, bool normalize,
              int32_t* ids, float* weights, hipStream_t stream) {
#define GRZ_CALL(G, V)                                                                       \
  return in_batches(n, kTokenBatch, [&](int64_t rows, int64_t r) {                           \
    return launch(route_kernel<T, G, V>,                                                     \
                  dim3(static_cast<unsigned>(ceil_div(rows, 256 / G))), dim3(256), stream,   \
                  static_cast<const T*>(logits), stride, r, n, experts, k, normalize, ids,   \
                  weights);                                                                  \
  });
  GRZ_ROUTE_SHAPES(GRZ_CALL)
#undef GRZ_CALL
}

template <typename T>
int route_grad_run(const void* logits, int64_t n, int experts, int64_t stride, int k,
                   bool normalize, const int32_t* ids, const float* dweights, void* dlogits,
                   int64_t dstride, hipStream_t stream) {
#define GRZ_CALL(G, V)                                                                       \
  return in_batches(n, kTokenBatch, [&](int64_t rows, int64_t r) {                           \
    return launch(route_grad_kernel<T, G, V>,                                                \
                  dim3(static_cast<unsigned>(ceil_div(rows, 256 / G))), dim3(256), stream,   \
                  static_cast<const T*>(logits), stride, r, n, experts, k, normalize, ids,   \
                  dweights, static_cast<T*>(dlogits), dstride);                              \
  });
  GRZ_ROUTE_SHAPES(GRZ_CALL)
#undef GRZ_CALL
}

int check_route(const void* logits, int dtype, int64_t n, int64_t experts, int64_t stride, int k,
                int flags) {
  if (flags & ~GRZ_NORMALIZE) return GRZ_EINVAL;
  if (experts < 1 || k > experts) return GRZ_EINVAL;
  if (experts > GRZ_MAX_EXPERTS) return GRZ_ERANGE;
  const int st = check_counts(n, k);
  return st != GRZ_OK ? st : check_matrix(logits, dtype, n, experts, stride);
}

int64_t tile_of(int64_t slots, int64_t experts) {
  if (slots <= kDirectSlots) return kSortThreads;
  const int64_t tiles = std::min(kMaxTiles, kTileCounts / experts);
  return ceil_div(slots, tiles * kSortThreads) * kSortThreads;
}
int bits_of(int v) {
  int b = 1;
  while (v >> b) ++b;
  return b;
}
// Bytes of the tiles' counts.
size_t sort_bytes(int64_t slots, int64_t experts) {
  if (slots <= kDirectSlots) return 0;
  return static_cast<size_t>(ceil_div(slots, tile_of(slots, experts))) * experts * sizeof(uint32_t);
}

// Rows' bytes from which they are read past the caches, since larger ones leave nothing
// there that would be found again (102 MB combined: 32 us against 37.6, their gradient
// 41 against 49; 25 MB: 9.9 against 9.1, 15.8 against 13.1).
constexpr int64_t kStreamBytes = int64_t{64} << 20;

template <typename TI, typename TO>
int dispatch_run(const void* x, int64_t xstride, const int32_t* places, const float* weights,
                 int64_t n, int k, int64_t dim, int64_t rows, void* out, int64_t ostride,
                 hipStream_t stream) {
  const int parts = static_cast<int>(ceil_div(dim, 64 * cols_of<TI, TO>()));
  const bool on_lines = aligned(out, 128) && ostride * static_cast<int64_t>(sizeof(TO)) % 128 == 0;
  const int waves = on_lines ? 2 : 8;
  return in_batches(n, ceil_div(kUnitBatch, parts), [&](int64_t tokens, int64_t r) {
    return launch(on_lines ? dispatch_kernel<TI, TO, 2> : dispatch_kernel<TI, TO, 8>,
                  dim3(static_cast<unsigned>(ceil_div(tokens * parts, waves))), dim3(64 * waves),
                  stream, static_cast<const TI*>(x), xstride, places, weights, r,
                  std::min(n, r + tokens), k, dim, parts, rows, static_cast<TO*>(out), ostride);
  });
}

template <typename TI, typename TO, bool ACC>
int combine_run(const void* y, int64_t ystride, int64_t rows, const int32_t* places,
                const float* weights, int64_t n, int k, int64_t dim, void* out, int64_t ostride,
                hipStream_t stream) {
  constexpr int VEC = cols_of<TI, TO>();
  auto go = [&](auto kernel, int u) {
    const int parts = static_cast<int>(ceil_div(dim, 64 * VEC * u));
    return in_batches(n, ceil_div(kUnitBatch, parts), [&](int64_t tokens, int64_t r) {
      return launch(kernel, dim3(static_cast<unsigned>(ceil_div(tokens * parts, kCombineWaves))),
                    dim3(kCombineWaves * 64),
                    stream, static_cast<const TI*>(y), ystride, rows, places, weights, r,
                    std::min(n, r + tokens), k, dim, parts, static_cast<TO*>(out), ostride);
    });
  };
  // Vectors a lane: one while that gives the chip few waves, up to 2048, and up to 8192
  // where more than four rows are on their way in each.  us with one, two and four, bf16,
  // waves with one in brackets: 256 x 4096 from 4 (2048) 4.0, 4.3, 4.9; 512 x 4096 from 4
  // (4096) 5.9, 6.0, 6.4; 4096 x 768 from 4 (8192) 7.2, 7.2, 7.8; 1024 x 4096 from 8
  // (8192) 13.4, 14.2, 15.2; 8192 x 768 from 8 (16384) 21.6, 20.6, 23.8; 2048 x 4096 from
  // 8 (16384) 28.8, 26.9, 27.4.
  // Then two, or four from rows of eight on, where the two are close: 8000 rows from 4,
  // 2048 columns 30.9, 28.4, 28.7; 3584 51.6, 47.7, 49.1; 4096 58.5, 54.6, 55.6; 6144
  // 86.7, 81.2, 81.2; 8192 116, 111, 107; fp32 1600 columns 45.9, 42.3, 43.0; 2048 58.3,
  // 53.8, 54.0; 4096 115, 109, 106.  16384 x 4096 bf16 from 6: 171, 161, 157.  (Worst for
  // four: 8000 x 2560 fp32 from 2, 40.3 with two, 42.2.)
  const int64_t units = n * ceil_div(dim, 64 * VEC);
  const bool past = n * k * dim * static_cast<int64_t>(sizeof(TI)) >= kStreamBytes;
  const bool wide = dim >= 8 * 64 * VEC;
#define GRZ_CALL(KB, FEW)                                                                 \
  if (units <= FEW) return go(combine_kernel<TI, TO, 1, KB, ACC, false>, 1);              \
  if (wide) return past ? go(combine_kernel<TI, TO, 4, KB, ACC, true>, 4)                 \
                        : go(combine_kernel<TI, TO, 4, KB, ACC, false>, 4);               \
  return past ? go(combine_kernel<TI, TO, 2, KB, ACC, true>, 2)                           \
              : go(combine_kernel<TI, TO, 2, KB, ACC, false>, 2);
  if (k <= 2) { GRZ_CALL(2, 2048) }
  if (k <= 4) { GRZ_CALL(4, 2048) }
  GRZ_CALL(8, 8192)
#undef GRZ_CALL
}

template <typename TD, typename TY>
int combine_grad_run(const void* dout, int64_t dstride, const void* y, int64_t ystride,
                     int64_t rows, const int32_t* places, const float* weights, int64_t n, int k,
                     int64_t dim, void* dy, int64_t dystride, float* dweights,
                     hipStream_t stream) {
  auto go = [&](auto kernel) {
    return in_batches(n, kTokenBatch, [&](int64_t tokens, int64_t r) {
      return launch(kernel, dim3(static_cast<unsigned>(ceil_div(tokens * k, kGradWaves))),
                    dim3(kGradWaves * 64), stream, static_cast<const TD*>(dout), dstride,
                    static_cast<const TY*>(y), ystride, rows, places, weights, r,
                    std::min(n, r + tokens), k, dim, static_cast<TY*>(dy), dystride, dweights);
    });
  };
  // Eight vectors a lane for rows that four do not hold, which so read them in one
  // pass; a row that four hold leaves half of eight idle.  us with four and eight, 8000
  // rows from 4, bf16: 1601 columns 49 and 57, 2048 49.5 and 51.3; 2056 58.5 and 57.0,
  // 2304 56.6 and 57.7, 2560 62.8 and 62.3, 3080 84.7 and 80.4, 4096 100.0 and 98.2, 8192
  // 225 and 221; fp32: 1024 50.0 and 50.8; 1032 59.2 and 57.2, 1280 62.8 and 62.3, 1601
  // 91.0 and 85.7, 2048 99.3 and 97.0.
  const bool wide = dim > 4 * 64 * cols_of<TD, TY>();
  if (n * k * dim * static_cast<int64_t>(sizeof(TY)) >= kStreamBytes)
    return wide ? go(combine_grad_kernel<TD, TY, 8, true>)
                : go(combine_grad_kernel<TD, TY, 4, true>);
  return wide ? go(combine_grad_kernel<TD, TY, 8, false>)
              : go(combine_grad_kernel<TD, TY, 4, false>);
}

}  // namespace

// ---------------------------------------------------------------------------
// C ABI

extern "C" {

int dp_expert_route(const void* logits, int dtype, int64_t n, int64_t experts, int64_t stride,
                    int k, int flags, int32_t* ids, float* weights, hipStream_t stream) {
  int st = check_route(logits, dtype, n, experts, stride, k, flags);
  if (st != GRZ_OK) return st;
  if ((st = check_slots(ids, n, k)) != GRZ_OK) return st;
  if ((st = check_slots(weights, n, k)) != GRZ_OK) return st;
  if (n == 0) return GRZ_OK;
  const Span in = matrix_span(logits, dtype, n, experts, stride);
  const Span i = slot_span(ids, n, k), w = slot_span(weights, n, k);
  if (clash(i, {in, w}) || clash(w, {in})) return GRZ_EINVAL;
  const bool norm = flags & GRZ_NORMALIZE;
  const int e = static_cast<int>(experts);
  return dtype == GRZ_BF16
             ? route_run<uint16_t>(logits, n, e, stride, k, norm, ids, weights, stream)
             : route_run<float>(logits, n, e, stride, k, norm, ids, weights, stream);
}

int dp_expert_route_grad(const void* logits, int dtype, int64_t n, int64_t experts,
                         int64_t stride, int k, int flags, const int32_t* ids,
                         const float* dweights, void* dlogits, int64_t dlogits_stride,
                         hipStream_t stream) {
  int st = check_route(logits, dtype, n, experts, stride, k, flags);
  if (st != GRZ_OK) return st;
  if ((st = check_slots(ids, n, k)) != GRZ_OK) return st;
  if ((st = check_slots(dweights, n, k)) != GRZ_OK) return st;
  if ((st = check_matrix(dlogits, dtype, n, experts, dlogits_stride)) != GRZ_OK) return st;
  if (n == 0) return GRZ_OK;
  const Span out = matrix_span(dlogits, dtype, n, experts, dlogits_stride);
  if (clash(out, {slot_span(ids, n, k), slot_span(dweights, n, k)})) return GRZ_EINVAL;
  if (!(logits == dlogits && stride == dlogits_stride) &&
      clash(out, {matrix_span(logits, dtype, n, experts, stride)}))
    return GRZ_EINVAL;
  const bool norm = flags & GRZ_NORMALIZE;
  const int e = static_cast<int>(experts);
  return dtype == GRZ_BF16
             ? route_grad_run<uint16_t>(logits, n, e, stride, k, norm, ids, dweights, dlogits,
                                        dlogits_stride, stream)
             : route_grad_run<float>(logits, n, e, stride, k, norm, ids, dweights, dlogits,
                                     dlogits_stride, stream);
}

size_t dp_expert_sort_workspace(int64_t n, int k, int64_t experts) {
  if (check_counts(n, k) != GRZ_OK || experts < 1 || experts > GRZ_MAX_EXPERTS) return 0;
  return sort_bytes(n * k, experts);
}

int dp_expert_sort(const void* ids, int id_bits, int64_t n, int k, int64_t experts,
                   void* workspace, int32_t* offsets, int32_t* places, hipStream_t stream) {
  int st = check_counts(n, k);
  if (st != GRZ_OK) return st;
  if (experts < 1) return GRZ_EINVAL;
  if (experts > GRZ_MAX_EXPERTS) return GRZ_ERANGE;
  if ((st = check_ids(ids, id_bits, n * k)) != GRZ_OK) return st;
  if (offsets == nullptr) return GRZ_EINVAL;
  if (!aligned(offsets, 4)) return GRZ_EALIGN;
  if ((st = check_slots(places, n, k)) != GRZ_OK) return st;
  const size_t need = sort_bytes(n * k, experts);
  if (need > 0) {
    if (workspace == nullptr) return GRZ_EINVAL;
    if (!aligned(workspace, 4)) return GRZ_EALIGN;
  }
  const int64_t slots = n * k;
  const Span in{ids, static_cast<size_t>(slots) * (id_bits / 8)}, ws{workspace, need};
  const Span off{offsets, static_cast<size_t>(experts + 1) * 4}, pl = slot_span(places, n, k);
  if (clash(off, {in, ws, pl}) || clash(pl, {in, ws}) || clash(ws, {in})) return GRZ_EINVAL;
  SortArgs a;
  a.ids = ids;
  a.id_bits = id_bits;
  a.slots = slots;
  a.experts = static_cast<int>(experts);
  a.bits = bits_of(a.experts);
  a.tile = tile_of(slots, experts);
  a.tiles = static_cast<int>(slots > 0 ? ceil_div(slots, a.tile) : 1);
  a.counts = static_cast<uint32_t*>(workspace);
  a.offsets = offsets;
  a.places = places;
  const bool direct = slots <= kDirectSlots;
  if (!direct) {
    st = launch(expert_count_kernel, dim3(a.tiles), dim3(kSortThreads), stream, a);
    if (st != GRZ_OK) return st;
  }
  return launch_lds(direct ? expert_place_kernel<true> : expert_place_kernel<false>,
                    static_cast<size_t>(kSortWaves) * a.experts * sizeof(uint16_t), dim3(a.tiles),
                    dim3(kSortThreads), stream, a);
}

int dp_expert_dispatch(const void* x, int x_dtype, int64_t x_stride, const int32_t* places,
                       const float* weights, int64_t n, int k, int64_t dim, int64_t rows,
                       void* out, int out_dtype, int64_t out_stride, hipStream_t stream) {
  int st = check_counts(n, k);
  if (st != GRZ_OK) return st;
  if (dim > kCols) return GRZ_ERANGE;
  if ((st = check_matrix(x, x_dtype, n, dim, x_stride)) != GRZ_OK) return st;
  if ((st = check_matrix(out, out_dtype, rows, dim, out_stride)) != GRZ_OK) return st;
  if ((st = check_slots(places, n, k)) != GRZ_OK) return st;
  if ((st = check_slots(weights, n, k, true)) != GRZ_OK) return st;
  if (n == 0 || dim == 0 || rows == 0) return GRZ_OK;
  if (clash(matrix_span(out, out_dtype, rows, dim, out_stride),
            {matrix_span(x, x_dtype, n, dim, x_stride), slot_span(places, n, k),
             slot_span(weights, n, k)}))
    return GRZ_EINVAL;
#define GRZ_CALL(TI, TO)                                                                        \
  dispatch_run<TI, TO>(x, x_stride, places, weights, n, k, dim, rows, out, out_stride, stream)
  if (x_dtype == GRZ_BF16)
    return out_dtype == GRZ_BF16 ? GRZ_CALL(uint16_t, uint16_t) : GRZ_CALL(uint16_t, float);
  return out_dtype == GRZ_BF16 ? GRZ_CALL(float, uint16_t) : GRZ_CALL(float, float);
#undef GRZ_CALL
}

int dp_expert_combine(const void* y, int y_dtype, int64_t y_stride, int64_t rows,
                      const int32_t* places, const float* weights, int64_t n, int k, int64_t dim,
                      int flags, void* out, int out_dtype, int64_t out_stride,
                      hipStream_t stream) {
  if (flags & ~GRZ_ACCUMULATE) return GRZ_EINVAL;
  int st = check_counts(n, k);
  if (st != GRZ_OK) return st;
  if (dim > kCols) return GRZ_ERANGE;
  if ((st = check_matrix(y, y_dtype, rows, dim, y_stride)) != GRZ_OK) return st;
  if ((st = check_matrix(out, out_dtype, n, dim, out_stride)) != GRZ_OK) return st;
  if ((st = check_slots(places, n, k)) != GRZ_OK) return st;
  if ((st = check_slots(weights, n, k, true)) != GRZ_OK) return st;
  if (n == 0 || dim == 0) return GRZ_OK;
  if (clash(matrix_span(out, out_dtype, n, dim, out_stride),
            {matrix_span(y, y_dtype, rows, dim, y_stride), slot_span(places, n, k),
             slot_span(weights, n, k)}))
    return GRZ_EINVAL;
  const bool acc = flags & GRZ_ACCUMULATE;
#define GRZ_CALL(TI, TO)                                                                         \
  (acc ? combine_run<TI, TO, true>(y, y_stride, rows, places, weights, n, k, dim, out,           \
                                   out_stride, stream)                                           \
       : combine_run<TI, TO, false>(y, y_stride, rows, places, weights, n, k, dim, out,          \
                                    out_stride, stream))
  if (y_dtype == GRZ_BF16)
    return out_dtype == GRZ_BF16 ? GRZ_CALL(uint16_t, uint16_t) : GRZ_CALL(uint16_t, float);
  return out_dtype == GRZ_BF16 ? GRZ_CALL(float, uint16_t) : GRZ_CALL(float, float);
#undef GRZ_CALL
}

int dp_expert_combine_grad(const void* dout, int dout_dtype, int64_t dout_stride, const void* y,
                           int y_dtype, int64_t y_stride, int64_t rows, const int32_t* places,
                           const float* weights, int64_t n, int k, int64_t dim, void* dy,
                           int64_t dy_stride, float* dweights, hipStream_t stream) {
  int st = check_counts(n, k);
  if (st != GRZ_OK) return st;
  if (dim > kCols) return GRZ_ERANGE;
  if ((st = check_matrix(dout, dout_dtype, n, dim, dout_stride)) != GRZ_OK) return st;
  // y is read for the weights' gradient alone.
  st = dweights != nullptr ? check_matrix(y, y_dtype, rows, dim, y_stride)
                           : check_matrix(nullptr, y_dtype, rows, 0, 0);
  if (st != GRZ_OK) return st;
  if (dy == nullptr && dweights == nullptr)
    return n == 0 || rows == 0 || dim == 0 ? GRZ_OK : GRZ_EINVAL;
  if (dy != nullptr && (st = check_matrix(dy, y_dtype, rows, dim, dy_stride)) != GRZ_OK)
    return st;
  if ((st = check_slots(places, n, k)) != GRZ_OK) return st;
  if ((st = check_slots(weights, n, k, true)) != GRZ_OK) return st;
  if ((st = check_slots(dweights, n, k, true)) != GRZ_OK) return st;
  if (n == 0) return GRZ_OK;
  const Span d = matrix_span(dout, dout_dtype, n, dim, dout_stride);
  const Span in = dweights != nullptr ? matrix_span(y, y_dtype, rows, dim, y_stride) : Span{};
  const Span out = matrix_span(dy, y_dtype, rows, dim, dy_stride);
  const Span pl = slot_span(places, n, k), w = slot_span(weights, n, k);
  const Span dw = slot_span(dweights, n, k);
  if (clash(out, {d, pl, w, dw}) || clash(dw, {d, in, pl, w})) return GRZ_EINVAL;
  if (!(dy == y && dy_stride == y_stride) && clash(out, {in})) return GRZ_EINVAL;
#define GRZ_CALL(TD, TY)                                                                        \
  combine_grad_run<TD, TY>(dout, dout_stride, y, y_stride, rows, places, weights, n, k, dim, dy, \
                           dy_stride, dweights, stream)
  if (dout_dtype == GRZ_BF16)
    return y_dtype == GRZ_BF16 ? GRZ_CALL(uint16_t, uint16_t) : GRZ_CALL(uint16_t, float);
  return y_dtype == GRZ_BF16 ? GRZ_CALL(float, uint16_t) : GRZ_CALL(float, float);
#undef GRZ_CALL
}

}  // extern "C"
