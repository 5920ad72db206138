// tokens.hip -- HIP kernels and C ABI of the operators addressed by token ids
// (the two ends of a language model's arena) for AMD Instinct MI355X (gfx950,
// CDNA4, wave64):
//   dp_embed_lookup         rows of the embedding table, scaled
//   dp_embed_grad           its gradient: a stable sort of the token ids, then
//                           a segmented sum over the sorted rows
//   dp_token_logprobs       log probability of given tokens, entropy, top list
//   dp_token_logprobs_grad  its gradient
//   dp_distill_loss         loss against a teacher's top logits
//   dp_distill_grad         its gradient (and the loss with it)
//
// All are bound by HBM: at most some 15 flops per byte.  No float atomics, so
// every result bit is the same from run to run.

#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include "grz.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int64_t kMaxRows = INT32_MAX;  // rows and columns of one call
// dp_embed_grad: ids, table rows and columns whose launches stay below 2^32
// threads and 2^16 column blocks.
constexpr int64_t kGradIds = int64_t{1} << 28, kGradRows = int64_t{1} << 26;
constexpr int64_t kGradCols = int64_t{65535} * 64;
constexpr int64_t kRowBatch = int64_t{1} << 21;  // rows of one launch of the row kernels
constexpr float kMinTemperature = 1e-18f, kMaxTemperature = 1e18f;

template <typename T> struct NoDeduce { using type = T; };

// Returns the status of this launch alone (hipLaunchKernel's return value).  A
// dispatch counts its threads in 32 bits; the entry points' limits and kRowBatch
// keep below that.
template <typename... A>
int launch_lds(void (*kernel)(A...), size_t lds, dim3 grid, dim3 block, hipStream_t stream,
               typename NoDeduce<A>::type... a) {
  if (static_cast<uint64_t>(grid.x) * block.x > UINT32_MAX) return GRZ_ERANGE;
  void* params[] = {static_cast<void*>(&a)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, params, lds,
                         stream) == hipSuccess ? GRZ_OK : GRZ_EHIP;
}
template <typename... A>
int launch(void (*kernel)(A...), dim3 grid, dim3 block, hipStream_t stream,
           typename NoDeduce<A>::type... a) {
  return launch_lds(kernel, 0, grid, block, stream, a...);
}

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool float_type(int dtype) { return dtype == GRZ_F32 || dtype == GRZ_BF16; }
size_t elem_size(int dtype) { return dtype == GRZ_F32 ? 4 : 2; }

// A row matrix as the entry points take it: `rows` x `cols` values of `dtype`,
// row r at data + r * stride elements.
int check_matrix(const void* data, int dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (!float_type(dtype) || rows < 0 || cols < 0) return GRZ_EINVAL;
  if (rows > kMaxRows || cols > kMaxRows) return GRZ_ERANGE;
  if (stride < cols) return GRZ_EINVAL;
  if (stride > (INT64_MAX >> 4) / (rows > 0 ? rows : 1)) return GRZ_ERANGE;
  if (rows == 0 || cols == 0) return GRZ_OK;
  if (data == nullptr) return GRZ_EINVAL;
  return aligned(data, elem_size(dtype)) ? GRZ_OK : GRZ_EALIGN;
}

// Bytes from the first element of a row matrix to behind its last one.
size_t span_of(int dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (rows == 0 || cols == 0) return 0;
  return elem_size(dtype) * static_cast<size_t>((rows - 1) * stride + cols);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

int check_ids(const void* ids, int id_bits, int64_t n) {
  if ((id_bits != 32 && id_bits != 64) || n < 0) return GRZ_EINVAL;
  if (n > kMaxRows) return GRZ_ERANGE;
  if (n == 0) return GRZ_OK;
  if (ids == nullptr) return GRZ_EINVAL;
  return aligned(ids, id_bits / 8) ? GRZ_OK : GRZ_EALIGN;
}

// ---------------------------------------------------------------------------
// Elements.  bf16 values are uint16 patterns; widening is exact, narrowing is
// round-to-nearest-even with a quiet NaN.

__device__ __forceinline__ float widen(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ float widen(float v) { return v; }

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ void put(uint16_t* p, float f) {
  *p = static_cast<uint16_t>(bf16_bits(f));
}
__device__ __forceinline__ void put(float* p, float f) { *p = f; }

// N consecutive elements in one access (8 or 16 bytes; the address is aligned
// for it), as fp32.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = widen(*p);
  } else if constexpr (sizeof(T) == 2) {
    if constexpr (N == 8) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      static_assert(N == 4, "bf16 vectors hold 4 or 8 elements");
      const u32x2 u = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      const u32x4 u = reinterpret_cast<const u32x4*>(p)[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = __uint_as_float(u[i]);
    }
  }
}

// Output streams that nothing here reads again are stored non-temporally (a
// 16384 x 4096 bf16 lookup: 32 us against 46 us with plain stores; the gradient
// of 4096 x 50257 logits 154 against 163 us).
template <bool STREAM, typename V> __device__ __forceinline__ void store_as(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

template <typename T, int N, bool STREAM = false>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[N]) {
  if constexpr (N == 1) {
    put(p, x[0]);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      u[i] = bf16_bits(x[2 * i]) | (bf16_bits(x[2 * i + 1]) << 16);
    if constexpr (N == 8) {
      store_as<STREAM>(reinterpret_cast<u32x4*>(p), u32x4{u[0], u[1], u[2], u[3]});
    } else {
      static_assert(N == 4, "bf16 vectors hold 4 or 8 elements");
      store_as<STREAM>(reinterpret_cast<u32x2*>(p), u32x2{u[0], u[1]});
    }
  } else {
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      u32x4 u;
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(x[4 * h + i]);
      store_as<STREAM>(reinterpret_cast<u32x4*>(p) + h, u);
    }
  }
}

__device__ __forceinline__ int64_t id_at(const void* ids, int id_bits, int64_t i) {
  return id_bits == 64 ? static_cast<const int64_t*>(ids)[i]
                       : static_cast<int64_t>(static_cast<const int32_t*>(ids)[i]);
}

// What waves read of each other's LDS writes without a barrier is their own.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// Lookup: one wave per row, its lanes along the columns, four 16-byte accesses
// of each on their way.  Bound by HBM: 16384 rows of 4096 bf16 out of 32000 in
// 32 us, 6.6 TB/s of 77 MB read (frequent rows once per XCD's L2) and 134 MB
// written; with two accesses on their way and plain stores 46 us.

template <typename TI, typename TO, int VEC>
__global__ __launch_bounds__(256) void lookup_kernel(const TI* __restrict__ table, int64_t tstride,
                                                     int64_t vocab, int64_t dim,
                                                     const void* __restrict__ ids, int id_bits,
                                                     int64_t row0, int64_t n, float scale,
                                                     TO* __restrict__ out, int64_t ostride) {
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= n) return;
  const int64_t id = id_at(ids, id_bits, row);
  const bool ok = id >= 0 && id < vocab;
  const TI* src = table + (ok ? id : 0) * tstride;
  TO* dst = out + row * ostride;
  constexpr int U = 4;  // accesses on their way at once
  for (int64_t c0 = (threadIdx.x & 63) * VEC; c0 < dim; c0 += 64 * VEC * U) {
    float x[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 64 * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[u][i] = 0.0f;
      if (ok && c < dim) load_vec<TI, VEC>(src + c, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 64 * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[u][i] = ok ? x[u][i] * scale : 0.0f;
      if (c < dim) store_vec<TO, VEC, true>(dst + c, x[u]);
    }
  }
}

// ---------------------------------------------------------------------------
// The sort of the token ids: stable, so that equal ids end up in the order of
// their positions.  Ids outside [0, vocab) get the key `vocab` and sort behind
// every row.  What a sort costs here is its launches' latency, so few of them:
//
//  - up to kRankIds ids one launch: an id's place is the number of ids before
//    it in the sorted order, counted by comparing it with all of them (2048
//    ids: 4.3 us; the arithmetic grows with n^2: the gradient of 4000 ids takes
//    16.4 us against 19.0 with the next one, that of 16384 51-56 against 38 when
//    both were first built);
//  - up to kMergeIds two: tiles of kMergeTile ids are sorted by that count,
//    then an id's place is the sum of its places in all tiles, each found by a
//    binary search in LDS (8011 ids: 5 + 5 us, against 22 us for the radix
//    sort's four launches);
//  - beyond that a radix sort, least significant digit first, of a count and a
//    scatter per pass; a workgroup of NT threads takes a tile of NT *
//    kSortItems pairs: 1024 up to kSmallSort ids, so that they still spread
//    over many CUs, 4096 beyond (1 M ids: 5 + 5 + 13 us a pass).
//
// The sort leaves HBM idle, so the launches that place pairs carry workgroups
// behind their own that write the table's zeros (16384 ids, 77 MB of zeros: 16 us
// for both, of which the zeros alone take 11).

constexpr int kRankIds = 4096;
constexpr int kRankWaves = 16;
constexpr int kRankLanes = 16;  // ids of a workgroup
constexpr int kMergeIds = 32768;
constexpr int kMergeTile = 256;
constexpr int kSortItems = 4;
constexpr int kMaxDigitBits = 9;
constexpr int kDigits = 1 << kMaxDigitBits;
constexpr int kBigSort = 1024, kLittleSort = 256;  // threads
constexpr int64_t kSmallSort = 65536;
constexpr int tile_of(int threads) { return threads * kSortItems; }
// Behind the last id: larger than any key (vocab <= 2^26).
constexpr uint32_t kNoKey = 0x7fffffffu;

struct SortSrc {
  const void* ids;  // first pass: the tokens; later passes: null
  int id_bits;
  const u32x2* pairs;  // later passes: (key, position)
  uint32_t vocab;
};

__device__ __forceinline__ u32x2 sort_pair(const SortSrc& s, int64_t i) {
  if (s.ids == nullptr) return s.pairs[i];
  const int64_t id = id_at(s.ids, s.id_bits, i);
  const uint32_t key = id >= 0 && id < static_cast<int64_t>(s.vocab) ? static_cast<uint32_t>(id)
                                                                     : s.vocab;
  return u32x2{key, static_cast<uint32_t>(i)};
}

// Rows [row0, row1) of the table to be zeroed, as bytes; `unit` is the widest
// access that the rows' places and lengths allow (16, 8, 4 or 2 bytes).
struct ZeroRows {
  char* data;
  int64_t stride, bytes;  // of a row
  int64_t row0, row1;
  int unit;
  bool stream;  // non-temporal stores
};

template <typename U>
__device__ __forceinline__ void zero_units(const ZeroRows& z, int64_t first, int64_t step) {
  const int64_t units = z.bytes / static_cast<int64_t>(sizeof(U));
  const U zero = {};
  for (int64_t r = z.row0 + first; r < z.row1; r += step) {
    U* row = reinterpret_cast<U*>(z.data + r * z.stride);
    if (z.stream) {
      for (int64_t c = threadIdx.x & 63; c < units; c += 64) store_as<true>(row + c, zero);
    } else {
      for (int64_t c = threadIdx.x & 63; c < units; c += 64) row[c] = zero;
    }
  }
}

// One wave per row; `block` of `blocks` workgroups.
__device__ __forceinline__ void zero_rows(const ZeroRows& z, int64_t block, int64_t blocks) {
  const int waves = blockDim.x >> 6;
  const int64_t first = block * waves + (threadIdx.x >> 6), step = blocks * waves;
  if (z.unit == 16) zero_units<u32x4>(z, first, step);
  else if (z.unit == 8) zero_units<u32x2>(z, first, step);
  else if (z.unit == 4) zero_units<uint32_t>(z, first, step);
  else zero_units<uint16_t>(z, first, step);
}

__global__ __launch_bounds__(256) void zero_rows_kernel(ZeroRows z) {
  zero_rows(z, blockIdx.x, gridDim.x);
}

// counts[tile][digit] of one tile per workgroup.
template <int NT>
__global__ __launch_bounds__(NT) void sort_count_kernel(SortSrc src, int64_t n, int shift,
                                                        int bits, uint32_t* __restrict__ counts) {
  __shared__ uint32_t hist[kDigits];
  const int digits = 1 << bits;
  for (int d = threadIdx.x; d < digits; d += NT) hist[d] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * tile_of(NT);
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int64_t i = base + j * NT + threadIdx.x;
    if (i < n) atomicAdd(&hist[(sort_pair(src, i)[0] >> shift) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += NT)
    counts[static_cast<int64_t>(blockIdx.x) * digits + d] = hist[d];
}

// For many tiles: counts[tile][digit] becomes the pairs of the digit in earlier
// tiles, totals[digit] their number in all.  A workgroup takes 64 digits, each
// of its waves a run of tiles.
constexpr int kScanWaves = 16;

__global__ __launch_bounds__(kScanWaves * 64) void sort_scan_kernel(uint32_t* __restrict__ counts,
                                                                    uint32_t* __restrict__ totals,
                                                                    int64_t tiles, int digits) {
  __shared__ uint32_t sums[kScanWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int d = blockIdx.x * 64 + lane;
  const int64_t share = ceil_div(tiles, kScanWaves);
  const int64_t from = wave * share, to = from + share < tiles ? from + share : tiles;
  uint32_t sum = 0;
  if (d < digits) {
#pragma unroll 8
    for (int64_t t = from; t < to; ++t) sum += counts[t * digits + d];
  }
  sums[wave][lane] = sum;
  __syncthreads();
  uint32_t before = 0, total = 0;
  for (int w = 0; w < kScanWaves; ++w) {
    before += w < wave ? sums[w][lane] : 0u;
    total += sums[w][lane];
  }
  if (d >= digits) return;
  if (wave == 0) totals[d] = total;
#pragma unroll 8
  for (int64_t t = from; t < to; ++t) {
    const uint32_t c = counts[t * digits + d];
    counts[t * digits + d] = before;
    before += c;
  }
}

// Digits of a workgroup's thread: D consecutive ones.
template <int NT> constexpr int digits_each() { return kDigits > NT ? kDigits / NT : 1; }

template <int NT> struct RankLds {
  uint32_t wave_sum[NT / 64];
  uint32_t first[kDigits];            // where the tile's run of a digit begins
  uint16_t before[NT / 64][kDigits];  // the wave's first place in that run
};

// Places of the tile's pairs among its pairs of the same digit: lds.before of
// the wave plus rank[j].  Wave w holds the kSortItems * 64 consecutive pairs
// from w * kSortItems * 64 on, 64 at a time; a pair's rank among the equal
// digits before it in its wave comes from the lanes' ballots of each digit bit.
// total: the tile's number of pairs of each of the thread's digits.  Ends
// without a barrier.
template <int NT>
__device__ __forceinline__ void tile_ranks(const u32x2 (&pair)[kSortItems], int64_t left,
                                           int shift, int bits, RankLds<NT>& lds,
                                           uint32_t (&rank)[kSortItems],
                                           uint32_t (&total)[digits_each<NT>()]) {
  constexpr int D = digits_each<NT>();
  const int digits = 1 << bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int d = lane; d < digits; d += 64) lds.before[wave][d] = 0;
  wave_fence();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const bool in = (wave * kSortItems + j) * 64 + lane < left;
    const uint32_t d = in ? (pair[j][0] >> shift) & (digits - 1) : 0u;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t v = __ballot((d >> b) & 1u);
      same &= ((d >> b) & 1u) ? v : ~v;
    }
    const uint32_t earlier = static_cast<uint32_t>(__popcll(same & ((1ull << lane) - 1)));
    uint32_t r = 0;
    if (in) r = lds.before[wave][d];
    wave_fence();
    if (in && earlier == 0)
      lds.before[wave][d] = static_cast<uint16_t>(r + static_cast<uint32_t>(__popcll(same)));
    rank[j] = r + earlier;
    wave_fence();
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < D; ++k) {
    const int d = tid * D + k;
    uint32_t sum = 0;
    if (d < digits) {
      uint16_t c[NT / 64];
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) c[w] = lds.before[w][d];
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) {
        lds.before[w][d] = static_cast<uint16_t>(sum);
        sum += c[w];
      }
    }
    total[k] = sum;
  }
}

// lds.first[d] = pairs of smaller digits + `before`, from each thread's own
// digits' totals.  Begins and ends with a barrier.
template <int NT, int D>
__device__ __forceinline__ void digit_starts(const uint32_t (&total)[D],
                                             const uint32_t (&before)[D], int digits,
                                             RankLds<NT>& lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t own = 0;
#pragma unroll
  for (int k = 0; k < D; ++k) own += total[k];
  uint32_t scan = own;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint32_t o = __shfl_up(scan, s, 64);
    scan += lane >= s ? o : 0u;
  }
  if (lane == 63) lds.wave_sum[wave] = scan;
  __syncthreads();
  uint32_t start = scan - own;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) start += w < wave ? lds.wave_sum[w] : 0u;
#pragma unroll
  for (int k = 0; k < D; ++k) {
    const int d = static_cast<int>(threadIdx.x) * D + k;
    if (d < digits) lds.first[d] = start + before[k];
    start += total[k];
  }
  __syncthreads();
}

// How many of the four keys are below `below`.  A difference's sign is shifted
// into a word whose ones are counted: no lane masks, which a vector instruction
// may only read some cycles after they are written.
__device__ __forceinline__ uint32_t count_below(u32x4 k, uint32_t below) {
  uint32_t signs = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) signs = __builtin_amdgcn_alignbit(signs, k[q] - below, 31);
  return static_cast<uint32_t>(__popc(signs));
}

// keys[0 .. padded) = key(j), kNoKey behind the n-th, by a workgroup of kRankWaves
// waves.  U loads of a thread are on their way at once (behind the last key it is
// read again): one after the other they cost the merge of 16384 ids 3 us of 12.
template <int U, typename F>
__device__ __forceinline__ void load_keys(uint32_t* keys, int padded, int n, F key) {
  constexpr int step = kRankWaves * 64;
  for (int j0 = threadIdx.x; j0 < padded; j0 += U * step) {
    uint32_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u] = key(j0 + u * step < n ? j0 + u * step : n - 1);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u * step < padded) keys[j0 + u * step] = j0 + u * step < n ? k[u] : kNoKey;
  }
}

// The places of kRankLanes ids per workgroup among all n <= kRankIds.  The keys
// lie in LDS; each wave compares its share of them with the ids, its lanes in
// groups that take every G-th run of four keys.
__global__ __launch_bounds__(kRankWaves * 64) void rank_kernel(SortSrc src, int n,
                                                               u32x2* __restrict__ out,
                                                               ZeroRows zero) {
  constexpr int I = kRankLanes, G = 64 / I, kPart = kRankWaves * G * 4;
  __shared__ u32x4 keys4[kRankIds / 4];
  __shared__ uint32_t part[kRankWaves][64];
  uint32_t* keys = reinterpret_cast<uint32_t*>(keys4);
  const int blocks = (n + I - 1) / I;
  if (static_cast<int>(blockIdx.x) >= blocks) {
    zero_rows(zero, blockIdx.x - blocks, gridDim.x - blocks);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int padded = (n + kPart - 1) / kPart * kPart;
  load_keys<kRankIds / (kRankWaves * 64)>(keys, padded, n,
                                          [&](int j) { return sort_pair(src, j)[0]; });
  __syncthreads();
  const int first = blockIdx.x * I;          // a multiple of G * 4
  const int i = first + lane % I, group = lane / I;
  const uint32_t key = i < n ? keys[i] : 0u;
  // Runs of G * 4 keys: in those before the workgroup's own ids an equal key counts.
  const int runs = padded / (G * 4), own = first / (G * 4), share = runs / kRankWaves;
  const int from = wave * share, to = from + share;
  const int turn = own < from ? from : own < to ? own : to;
  uint32_t count = 0;
#pragma unroll 4
  for (int r = from; r < turn; ++r) count += count_below(keys4[r * G + group], key + 1);
#pragma unroll 4
  for (int r = turn; r < to; ++r) count += count_below(keys4[r * G + group], key);
  part[wave][lane] = count;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < I && i < n) {
    uint32_t place = 0;
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) {
#pragma unroll
      for (int g = 0; g < G; ++g) place += part[w][g * I + lane];
    }
    for (int m = 0; m < lane; ++m) place += keys[first + m] == key ? 1u : 0u;
    out[place] = u32x2{key, static_cast<uint32_t>(i)};
  }
}

// Sorts each tile of kMergeTile ids, one workgroup each, one id per thread.
__global__ __launch_bounds__(kMergeTile) void sort_tiles_kernel(SortSrc src, int n,
                                                                u32x2* __restrict__ out,
                                                                ZeroRows zero) {
  __shared__ u32x4 keys4[kMergeTile / 4];
  uint32_t* keys = reinterpret_cast<uint32_t*>(keys4);
  const int tiles = (n + kMergeTile - 1) / kMergeTile;
  if (static_cast<int>(blockIdx.x) >= tiles) {
    zero_rows(zero, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  const int tid = threadIdx.x, i = blockIdx.x * kMergeTile + tid;
  const uint32_t key = i < n ? sort_pair(src, i)[0] : kNoKey;
  keys[tid] = key;
  __syncthreads();
  // Runs of four keys before the wave's own 64 ids, its own, and behind them.
  const int own = __builtin_amdgcn_readfirstlane(tid >> 6) * 16;
  uint32_t place = 0;
#pragma unroll 8
  for (int r = 0; r < own; ++r) place += count_below(keys4[r], key + 1);
#pragma unroll 4
  for (int r = own; r < own + 16; ++r) {
    const u32x4 k = keys4[r];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      place += k[q] < key + (r * 4 + q < tid ? 1u : 0u) ? 1u : 0u;
  }
#pragma unroll 8
  for (int r = own + 16; r < kMergeTile / 4; ++r) place += count_below(keys4[r], key);
  if (i < n) out[blockIdx.x * kMergeTile + place] = u32x2{key, static_cast<uint32_t>(i)};
}

// Places the pairs of the sorted tiles among all n <= kMergeIds: 64 pairs of one
// tile per workgroup, one per lane, each wave searching every 16th tile.
__global__ __launch_bounds__(kRankWaves * 64) void merge_tiles_kernel(
    const u32x2* __restrict__ pairs, int n, u32x2* __restrict__ out, ZeroRows zero) {
  extern __shared__ uint32_t keys[];  // n, rounded up to whole tiles
  __shared__ uint32_t part[kRankWaves][64];
  const int blocks = (n + 63) / 64;
  if (static_cast<int>(blockIdx.x) >= blocks) {
    zero_rows(zero, blockIdx.x - blocks, gridDim.x - blocks);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (n + kMergeTile - 1) / kMergeTile;
  load_keys<8>(keys, tiles * kMergeTile, n, [&](int j) { return pairs[j][0]; });
  const int i = blockIdx.x * 64 + lane, own = blockIdx.x * 64 / kMergeTile;
  u32x2 pair = {0, 0};
  if (i < n) pair = pairs[i];
  __syncthreads();
  // Keys of tile t below the bound (an equal key of an earlier tile comes before).
  uint32_t count = 0;
#pragma unroll 4
  for (int t = wave; t < tiles; t += kRankWaves) {
    const uint32_t* tile = keys + t * kMergeTile;
    const uint32_t below = pair[0] + (t < own ? 1u : 0u);
    uint32_t at = 0;
#pragma unroll
    for (int s = kMergeTile / 2; s > 0; s /= 2) at += tile[at + s - 1] < below ? s : 0;
    at += tile[at] < below ? 1u : 0u;
    count += t == own ? static_cast<uint32_t>(i - own * kMergeTile) : at;
  }
  part[wave][lane] = count;
  __syncthreads();
  if (wave == 0 && i < n) {
    uint32_t place = 0;
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) place += part[w][lane];
    out[place] = pair;
  }
}

// One pass over several tiles, one workgroup each.  The number of each digit's
// pairs in all and in the tiles before comes, with few tiles, straight from
// counts[tile][digit], and with more from sort_scan_kernel's results.
constexpr int kDirectTiles = 64;
static_assert(kSmallSort <= int64_t{kDirectTiles} * tile_of(kLittleSort), "little tiles");

template <int NT, bool SCANNED>
__global__ __launch_bounds__(NT) void sort_scatter_kernel(
    SortSrc src, int64_t n, int shift, int bits, const uint32_t* __restrict__ counts,
    const uint32_t* __restrict__ totals, u32x2* __restrict__ out, ZeroRows zero) {
  constexpr int D = digits_each<NT>();
  __shared__ RankLds<NT> lds;
  const int64_t tiles = ceil_div(n, tile_of(NT)), tile = blockIdx.x;
  if (tile >= tiles) {
    zero_rows(zero, tile - tiles, gridDim.x - tiles);
    return;
  }
  const int digits = 1 << bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t base = tile * tile_of(NT);
  u32x2 pair[kSortItems] = {};
  uint32_t rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int64_t i = base + (wave * kSortItems + j) * 64 + lane;
    if (i < n) pair[j] = sort_pair(src, i);
  }
  uint32_t before[D] = {}, total[D] = {}, mine[D];
  if (tid * D < digits) {
    if constexpr (SCANNED) {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        if (tid * D + k >= digits) break;
        before[k] = counts[tile * digits + tid * D + k];
        total[k] = totals[tid * D + k];
      }
    } else {
#pragma unroll 16
      for (int64_t t = 0; t < tiles; ++t) {
#pragma unroll
        for (int k = 0; k < D; ++k) {
          const uint32_t c = tid * D + k < digits ? counts[t * digits + tid * D + k] : 0u;
          before[k] += t < tile ? c : 0u;
          total[k] += c;
        }
      }
    }
  }
  tile_ranks<NT>(pair, n - base, shift, bits, lds, rank, mine);
  digit_starts<NT>(total, before, digits, lds);
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (base + (wave * kSortItems + j) * 64 + lane < n) {
      const uint32_t d = (pair[j][0] >> shift) & (digits - 1);
      out[lds.first[d] + lds.before[wave][d] + rank[j]] = pair[j];
    }
  }
}

// ---------------------------------------------------------------------------
// The gradient over the sorted pairs.  The pairs are cut into chunks of equal
// size; a wave sums one chunk's rows over its columns, run of equal keys by
// run.  A run inside the chunk is written to its row; one that began in an
// earlier chunk or goes on in the next leaves its sum in `partial`
// (chunk, 0: began earlier; 1: begins here and goes on), which join_kernel
// adds up in chunk order.
//
// A wave's columns are P pieces of 64 * VEC, so that what it does per row (its
// address, where runs end) is shared by up to 2 KB of it; the next kBatch rows
// are on their way while the last ones are added.  Bound by HBM for many rows (1 M
// of 768 bf16: 1.6 GB in 300 us), by the chain pairs - rows - stores for few
// (16384: 25 MB in 10 us).
//
// Rows are loaded and written, and zeros written, non-temporally, except where
// the table's rows are added to (its loads then measured 6 % slower) and beside
// the one-launch sort (10 % slower): 16384 x 768 into 50257 rows 34 us against
// 38 us with plain accesses, 1 M ids 371 against 428 us.

constexpr int kBatch = 4;

template <typename T, int VEC> struct RawVec;  // a lane's part of a row as loaded
template <> struct RawVec<uint16_t, 1> { uint16_t v; };
template <> struct RawVec<float, 1> { float v; };
template <> struct RawVec<uint16_t, 4> { u32x2 v; };
template <> struct RawVec<float, 4> { u32x4 v; };

template <bool ONCE, typename T, int VEC>
__device__ __forceinline__ RawVec<T, VEC> load_raw(const T* p) {
  const RawVec<T, VEC>* at = reinterpret_cast<const RawVec<T, VEC>*>(p);
  RawVec<T, VEC> r;
  r.v = ONCE ? __builtin_nontemporal_load(&at->v) : at->v;
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void widen_vec(const RawVec<T, VEC>& r, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = widen(r.v);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = __uint_as_float(r.v[i] << 16);
      x[2 * i + 1] = __uint_as_float(r.v[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r.v[i]);
  }
}

// scale * acc, added to `old` (what the row holds) with ACC.
template <bool ACC, typename TO, int VEC>
__device__ __forceinline__ void finish_row(TO* dst, const float (&acc)[VEC], float scale,
                                           const RawVec<TO, VEC>& old) {
  float y[VEC];
  if constexpr (ACC) {
    widen_vec<TO, VEC>(old, y);
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = acc[i] * scale + y[i];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = acc[i] * scale;
  }
  store_vec<TO, VEC, !ACC>(dst, y);
}

__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), lane);
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

template <typename TI, typename TO, int VEC, int P, bool ACC>
__global__ __launch_bounds__(64) void embed_grad_kernel(
    const TI* __restrict__ dout, int64_t istride, const u32x2* __restrict__ pairs, int64_t n,
    int size, uint32_t vocab, int64_t dim, float scale, float* __restrict__ partial,
    TO* __restrict__ dtable, int64_t ostride) {
  const int lane = threadIdx.x;
  const int64_t chunk = blockIdx.x;
  const int64_t base = chunk * size;
  const int cnt = static_cast<int>(n - base < size ? n - base : size);
  const int64_t col0 = static_cast<int64_t>(blockIdx.y) * (64 * VEC * P) + lane * VEC;
  bool on[P];
  int64_t load_col[P];  // a lane behind the last column reads the first one
#pragma unroll
  for (int k = 0; k < P; ++k) {
    on[k] = col0 + k * 64 * VEC < dim;
    load_col[k] = on[k] ? col0 + k * 64 * VEC : 0;
  }
  uint32_t before = base > 0 ? pairs[base - 1][0] : vocab;
  float acc[P][VEC] = {};
  int slot = 0;       // where an unfinished run's sum goes: 0 while it began earlier
  bool open = false;  // rows have been added since the last run's end
  for (int part = 0; part < cnt; part += 64) {
    const int here = cnt - part < 64 ? cnt - part : 64;
    u32x2 mine = {vocab, 0};
    if (lane < here) mine = pairs[base + part + lane];
    const uint32_t after = base + part + here < n ? pairs[base + part + here][0] : vocab;
    uint32_t right = __shfl_down(mine[0], 1, 64);
    if (lane == here - 1) right = after;
    const int rows = __popcll(__ballot(mine[0] != vocab));  // the ids of no row come last
    const uint64_t ends = __ballot(mine[0] != right && mine[0] != vocab);
    if (part == 0) slot = rows > 0 && __builtin_amdgcn_readlane(mine[0], 0) == before ? 0 : 1;
    const int64_t in_at = static_cast<int64_t>(mine[1]) * istride;
    const int64_t out_at = static_cast<int64_t>(mine[0]) * ostride;
    if (rows == 0) break;
    struct Rows {
      RawVec<TI, VEC> x[kBatch][P];
      RawVec<TO, VEC> old[ACC ? kBatch : 1][P];  // what the table's rows hold
    } buf[2];
    // No branches: the loads of a batch stay in flight while the last one is
    // added.  Behind the last row it is read again, as is, with ACC, a table
    // row for every row of its run; both from the caches.
    auto fetch = [&](int from, Rows& to) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = from + b < rows ? from + b : rows - 1;
        const TI* src = dout + lane_of(in_at, e);
#pragma unroll
        for (int k = 0; k < P; ++k)
          to.x[b][k] = load_raw<!ACC, TI, VEC>(src + load_col[k]);
        if constexpr (ACC) {
          const TO* dst = dtable + lane_of(out_at, e);
#pragma unroll
          for (int k = 0; k < P; ++k)
            to.old[b][k] = *reinterpret_cast<const RawVec<TO, VEC>*>(dst + load_col[k]);
        }
      }
    };
    auto add = [&](int from, const Rows& in) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = from + b;
        if (e >= rows) break;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float x[VEC];
          widen_vec<TI, VEC>(in.x[b][k], x);
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[k][i] += x[i];
        }
        open = true;
        if (!((ends >> e) & 1)) continue;
        if (slot == 0) {
          float* dst = partial + chunk * 2 * dim + col0;
#pragma unroll
          for (int k = 0; k < P; ++k)
            if (on[k]) store_vec<float, VEC>(dst + k * 64 * VEC, acc[k]);
        } else {
          TO* dst = dtable + lane_of(out_at, e) + col0;
#pragma unroll
          for (int k = 0; k < P; ++k)
            if (on[k])
              finish_row<ACC, TO, VEC>(dst + k * 64 * VEC, acc[k], scale, in.old[ACC ? b : 0][k]);
        }
        slot = 1;
        open = false;
#pragma unroll
        for (int k = 0; k < P; ++k) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[k][i] = 0.0f;
        }
      }
    };
    fetch(0, buf[0]);
    for (int from = 0; from < rows; from += 2 * kBatch) {
      fetch(from + kBatch, buf[1]);
      add(from, buf[0]);
      fetch(from + 2 * kBatch, buf[0]);
      add(from + kBatch, buf[1]);
    }
  }
  if (open) {
    float* dst = partial + (chunk * 2 + slot) * dim + col0;
#pragma unroll
    for (int k = 0; k < P; ++k)
      if (on[k]) store_vec<float, VEC>(dst + k * 64 * VEC, acc[k]);
  }
}

// One workgroup per (chunk border, column block); the border where a run first
// crosses adds the whole run: its waves take equal parts of the run's partial
// sums, in order, then the waves' sums in order.  Most borders have nothing to add
// and leave after one read, so more waves cost more than they gain: 16384 ids 6 us;
// with 16 waves the fp32 gradient of 8011 x 1600 takes 39 us instead of 33.
constexpr int kJoinWaves = 4;

template <typename TO, int VEC, bool ACC>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(
    const u32x2* __restrict__ pairs, int64_t n, int size, uint32_t vocab, int64_t dim, float scale,
    const float* __restrict__ partial, TO* __restrict__ dtable, int64_t ostride) {
  __shared__ float part[kJoinWaves][64 * VEC];
  const int64_t c = static_cast<int64_t>(blockIdx.x) + 1;  // border between chunks c - 1 and c
  const uint32_t key = pairs[c * size][0];
  const uint32_t left = pairs[c * size - 1][0];
  const uint32_t earlier = c > 1 ? pairs[(c - 1) * size - 1][0] : vocab;
  if (key == vocab || left != key || earlier == key) return;  // no run, or from an earlier border
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // The last chunk that begins with the key: 64 probes at a time.
  int64_t lo = c, hi = ceil_div(n, size);
  int64_t step = 1;  // runs are mostly short
  while (hi - lo > 1) {
    const int64_t at = lo + lane * step;
    const bool same = at < hi && pairs[at * size][0] == key;
    const int count = __popcll(__ballot(same));
    lo += (count - 1) * step;
    if (count < 64 && lo + step < hi) hi = lo + step;
    step = ceil_div(hi - lo, 64);
  }
  const int64_t count = lo - c + 2;  // chunks c - 1 .. lo
  const int64_t share = ceil_div(count, kJoinWaves);
  const int64_t from = wave * share, to = from + share < count ? from + share : count;
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * VEC;
  const bool on = col < dim;
  TO* dst = dtable + static_cast<int64_t>(key) * ostride + col;
  RawVec<TO, VEC> old;
  if (ACC && wave == 0 && on) old = *reinterpret_cast<const RawVec<TO, VEC>*>(dst);
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  if (on) {
#pragma unroll 8
    for (int64_t k = from; k < to; ++k) {
      float x[VEC];
      load_vec<float, VEC>(partial + ((c - 1 + k) * 2 + (k == 0 ? 1 : 0)) * dim + col, x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += x[i];
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) part[wave][lane * VEC + i] = acc[i];
  __syncthreads();
  if (wave == 0 && on) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      acc[i] = part[0][lane * VEC + i];
#pragma unroll
      for (int w = 1; w < kJoinWaves; ++w) acc[i] += part[w][lane * VEC + i];
    }
    finish_row<ACC, TO, VEC>(dst, acc, scale, old);
  }
}

// Small tables and few ids, in one launch and without a sort: a workgroup per
// (table row, column piece) reads all ids; each wave collects the positions of
// its share that name the row, in order, and sums their rows, then the waves'
// sums are added in order.  2048 ids x 384 into 65 rows: 7.4 us a call against
// 13.2 us for sort, sum and join, whose three launches are three latencies; 4096
// x 256 into 512 rows 8.3 against 14.1 us.  One workgroup's waves sum all of a
// row, so few rows for many ids take the sort (4096 x 1600 into 8 rows: 34
// against 19 us).  The rule knows the mean alone: ids that crowd onto one row of
// many lose to the sort (4096 x 256 into 512 rows, all ids alike 44 us, half of them
// 24, against 20 and 17 for the sort's 513 rows).
constexpr int kDirectWaves = 16;
constexpr int64_t kDirectIds = 4096, kDirectGroups = 512, kDirectMean = 32;

template <typename TI, typename TO, int VEC, bool ACC>
__global__ __launch_bounds__(kDirectWaves * 64) void direct_grad_kernel(
    const TI* __restrict__ dout, int64_t istride, const void* __restrict__ ids, int id_bits, int n,
    int64_t dim, float scale, TO* __restrict__ dtable, int64_t ostride) {
  constexpr int kShare = kDirectIds / kDirectWaves, kFetch = 8;
  __shared__ uint16_t list[kDirectWaves][kShare];
  __shared__ float part[kDirectWaves][64 * VEC];
  __shared__ int found[kDirectWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = blockIdx.x;
  const int share = (n + kDirectWaves * 64 - 1) / (kDirectWaves * 64) * 64;
  int count = 0;
#pragma unroll
  for (int k = 0; k < kShare / 64; ++k) {
    const int i = wave * share + k * 64 + lane;
    const bool mine = k * 64 < share && i < n && id_at(ids, id_bits, i) == row;
    const uint64_t mask = __ballot(mine);
    if (mine) list[wave][count + __popcll(mask & ((1ull << lane) - 1))] = static_cast<uint16_t>(i);
    count += __popcll(mask);
  }
  if (lane == 0) found[wave] = count;
  wave_fence();
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * VEC;
  const bool on = col < dim;
  const int64_t load_col = on ? col : 0;
  float acc[VEC] = {};
  for (int from = 0; from < count; from += kFetch) {
    RawVec<TI, VEC> x[kFetch];
#pragma unroll
    for (int b = 0; b < kFetch; ++b) {  // behind the last one it is read again
      const int e = from + b < count ? from + b : count - 1;
      const int at = __builtin_amdgcn_readfirstlane(list[wave][e]);
      x[b] = load_raw<false, TI, VEC>(dout + at * istride + load_col);
    }
#pragma unroll
    for (int b = 0; b < kFetch; ++b) {
      if (from + b >= count) break;
      float y[VEC];
      widen_vec<TI, VEC>(x[b], y);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += y[i];
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) part[wave][lane * VEC + i] = acc[i];
  __syncthreads();
  if (wave != 0 || !on) return;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kDirectWaves; ++w) total += found[w];
  if (ACC && total == 0) return;  // a row that no id names is not touched
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    acc[i] = part[0][lane * VEC + i];
#pragma unroll
    for (int w = 1; w < kDirectWaves; ++w) acc[i] += part[w][lane * VEC + i];
  }
  TO* dst = dtable + row * ostride + col;
  RawVec<TO, VEC> old{};
  if (ACC) old = load_raw<false, TO, VEC>(dst);
  finish_row<ACC, TO, VEC>(dst, acc, scale, old);
}

// ---------------------------------------------------------------------------
// Rows over the vocabulary.  One workgroup of NT threads per row.  The row is
// read as 16-byte vectors from its first 16-byte border on; the elements
// before and behind them (fewer than two vectors) go one to a thread, so that
// nothing outside the row is touched.
//
// NV > 0: the row is read once and kept in registers, up to NV vectors per
// thread, so that its maximum, its sums and its gradient cost one pass over
// HBM.  NV = 0, for rows too long for that: one pass for the maximum and the sums
// and one for the gradient or the top list.
//
// ONCE: nothing reads the row again after this load (non-temporal).

template <typename T, int NT, int NV, bool ONCE = false> struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* p;
  int head, nvec;     // elements before the first vector; vectors
  int edge;           // this thread's single element, or -1
  float edge_x;
  u32x4 kept[NV > 0 ? NV : 1];

  __device__ __forceinline__ Row(const T* row, int vocab) : p(row) {
    const int skip = static_cast<int>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 /
                                      sizeof(T));
    head = skip < vocab ? skip : vocab;
    nvec = (vocab - head) / E;
    const int tail0 = head + nvec * E;
    const int t = threadIdx.x;
    edge = t < head ? t : t - head < vocab - tail0 ? tail0 + t - head : -1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * NT + t;
      if (v < nvec) {
        const u32x4* at = reinterpret_cast<const u32x4*>(p + head + v * E);
        kept[j] = ONCE ? __builtin_nontemporal_load(at) : *at;
      }
    }
    edge_x = edge >= 0 ? widen(p[edge]) : 0.0f;
  }
  // The thread that holds (and in map() stores) an element.
  __device__ __forceinline__ int owner(int index) const {
    const int in = index - head, v = in / E;
    return in < 0 ? index : v < nvec ? v % NT : in - nvec * E + head;
  }
  static __device__ __forceinline__ void unpack(u32x4 u, float (&x)[E]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
    }
  }
  // f(vector's elements, index of the first, which of the thread's it is) for each
  // of this thread's vectors.
  template <typename F> __device__ __forceinline__ void vectors(F f) const {
    float x[E];
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = j * NT + static_cast<int>(threadIdx.x);
        if (v < nvec) {
          unpack(kept[j], x);
          f(x, head + v * E, j);
        }
      }
    } else {
      for (int v = threadIdx.x, j = 0; v < nvec; v += NT, ++j) {
        unpack(*reinterpret_cast<const u32x4*>(p + head + v * E), x);
        f(x, head + v * E, j);
      }
    }
  }
  // f(x, index) for each of this thread's elements.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    vectors([&](float (&x)[E], int at, int) {
#pragma unroll
      for (int i = 0; i < E; ++i) f(x[i], at + i);
    });
    if (edge >= 0) f(edge_x, edge);
  }
  // dst[index] = f(x) over the row; dst may be the row itself.  last(values, index
  // of the first, which of the thread's vectors) may change a vector's.
  template <typename F, typename L>
  __device__ __forceinline__ void map(T* dst, F f, L last) const {
    const bool vec = reinterpret_cast<uintptr_t>(dst + head) % 16 == 0;
    vectors([&](float (&x)[E], int at, int j) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = f(x[i]);
      last(x, at, j);
      if (vec) {
        store_vec<T, E, true>(dst + at, x);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) put(dst + at + i, x[i]);
      }
    });
    if (edge >= 0) put(dst + edge, f(edge_x));
  }
};

template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* dst, int vocab) {
  constexpr int E = 16 / sizeof(T);
  const int skip = static_cast<int>((16 - reinterpret_cast<uintptr_t>(dst) % 16) % 16 /
                                    sizeof(T));
  const int head = skip < vocab ? skip : vocab;
  const int nvec = (vocab - head) / E;
  for (int v = threadIdx.x; v < nvec; v += NT)
    *reinterpret_cast<u32x4*>(dst + head + v * E) = u32x4{0, 0, 0, 0};
  const int t = threadIdx.x, tail0 = head + nvec * E;
  if (t < head) dst[t] = static_cast<T>(0);
  else if (t - head < vocab - tail0) dst[tail0 + t - head] = static_cast<T>(0);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// 2^d underflows to zero far above this, so terms of 2^d * d can be cut here:
// 0 * -inf (a masked element) becomes 0.
constexpr float kLowest = -1.0e4f;
constexpr float kLowestFloat = -3.402823466e38f;

// Reductions.  A wave's in a fixed tree: four steps of lane exchanges inside
// each row of 16 lanes, then the four rows.
template <int CTRL> __device__ __forceinline__ float lane_swap(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf,
                                                     false));
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, lane_swap<kSwap1>(v));
  v = fmaxf(v, lane_swap<kSwap2>(v));
  v = fmaxf(v, lane_swap<kHalfMirror>(v));
  v = fmaxf(v, lane_swap<kMirror>(v));
  return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += lane_swap<kSwap1>(v);
  v += lane_swap<kSwap2>(v);
  v += lane_swap<kHalfMirror>(v);
  v += lane_swap<kMirror>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint64_t o = __shfl_xor(static_cast<unsigned long long>(v), s, 64);
    v = o > v ? o : v;
  }
  return v;
}

// The whole workgroup's, every thread with the result (every wave reads the
// waves' values into its lanes and repeats the exchanges).  Each call of a kernel
// has an LDS array of its own, so one barrier is enough.
template <int NT> __device__ __forceinline__ float block_max(float v, float* lds) {
  v = wave_max(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[threadIdx.x % (NT / 64)];
    v = fmaxf(v, lane_swap<kSwap1>(v));
    if constexpr (NT >= 256) v = fmaxf(v, lane_swap<kSwap2>(v));
    if constexpr (NT >= 512) v = fmaxf(v, lane_swap<kHalfMirror>(v));
    if constexpr (NT >= 1024) v = fmaxf(v, lane_swap<kMirror>(v));
  }
  return v;
}
template <int NT, int M>
__device__ __forceinline__ void block_sum(float (&v)[M], float (*lds)[M]) {
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i) lds[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      v[i] = lds[threadIdx.x % (NT / 64)][i];
      v[i] += lane_swap<kSwap1>(v[i]);
      if constexpr (NT >= 256) v[i] += lane_swap<kSwap2>(v[i]);
      if constexpr (NT >= 512) v[i] += lane_swap<kHalfMirror>(v[i]);
      if constexpr (NT >= 1024) v[i] += lane_swap<kMirror>(v[i]);
    }
  }
}
template <int NT>
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* lds) {
  v = wave_max(v);
  if constexpr (NT > 64) {
    __syncthreads();  // called in a loop on one array
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = lds[w] > v ? lds[w] : v;
  }
  return v;
}

// Waves per SIMD the kernels are built for: two workgroups of 1024 threads on a
// CU, so that one's loads and stores run beside the other's arithmetic.
constexpr int kRowWaves = 8;

// The row's exponents, in powers of two: an element's is x * l2 - at, l2 =
// log2(e) / T, with one fused rounding.  `at` = max * l2, rounded (by at most
// 1/16), cancels from everything normalised by the sum.  From |max * l2| = 10^6 on,
// where that rounding would shift the exponents out of range (huge logits, masks of
// the type's lowest value), and in rows that are not kept, whose maximum moves, the
// difference is formed first.
struct Exponent {
  float inv_tau, l2, max, at;
  bool plain;
  __device__ __forceinline__ Exponent(float m, float inv, bool fused)
      : inv_tau(inv), l2(kLog2e * inv), max(m), at(m * l2), plain(fused && fabsf(at) < 1.0e6f) {}
  __device__ __forceinline__ float far(float x) const { return (x - max) * l2; }
  __device__ __forceinline__ float near(float x) const { return fmaf(x, l2, -at); }
  __device__ __forceinline__ float of(float x) const { return plain ? near(x) : far(x); }
  // log q, finite wherever it can be: log2s counts from `at`, not from max * l2.
  __device__ __forceinline__ float log_q(float x, float log2s) const {
    return (x - max) * inv_tau - (log2s - of(max)) * kLn2;
  }
};

// each() and map() with the exponent's form chosen once for the row.
template <typename R, typename F>
__device__ __forceinline__ void each_exponent(const R& r, const Exponent& e, F f) {
  if (e.plain) r.each([&](float x, int) { f(e.near(x)); });
  else r.each([&](float x, int) { f(e.far(x)); });
}
template <typename R, typename T, typename F, typename L>
__device__ __forceinline__ void map_exponent(const R& r, T* dst, const Exponent& e, F f, L last) {
  if (e.plain) r.map(dst, [&](float x) { return f(e.near(x)); }, last);
  else r.map(dst, [&](float x) { return f(e.far(x)); }, last);
}

// The largest of a thread's elements, with S = sum 2^d and (where A) A = sum 2^d d,
// d counted from it, in one pass: a larger element that comes later shifts what
// has been summed.  For rows that are not kept in registers.
__device__ __forceinline__ void shift_sums(float by, float& s, float& a) {
  by = fmaxf(by, kLowest);  // from a thread whose elements are all masked: s = a = 0
  const float f = __builtin_amdgcn_exp2f(by);
  a = f * fmaf(by, s, a);
  s *= f;
}
template <bool A, typename R>
__device__ __forceinline__ float running_sums(const R& r, float l2, float& s, float& a) {
  float max = -INFINITY, from = kLowestFloat;  // `from` stays finite while all are masked
  auto add = [&](auto& x) {
    float most = x[0];
    for (float v : x) most = fmaxf(most, v);
    max = fmaxf(max, most);
    if (most > from) {
      shift_sums((from - most) * l2, s, a);
      from = most;
    }
    for (float v : x) {
      const float d = (v - from) * l2, p = __builtin_amdgcn_exp2f(d);
      s += p;
      if (A) a = fmaf(p, fmaxf(d, kLowest), a);
    }
  };
  r.vectors([&](auto& x, int, int) { add(x); });
  if (r.edge >= 0) {
    const float x[1] = {r.edge_x};
    add(x);
  }
  return max;
}
// Such a thread's sums, counted from the row's largest element.
__device__ __forceinline__ void join_sums(const Exponent& e, float own_max, float& s, float& a) {
  shift_sums((fmaxf(own_max, kLowestFloat) - e.max) * e.l2, s, a);
}

// The order of the top list: larger values first, then lower indices, as one
// unsigned number (larger is earlier).  -0 and +0 are equal; NaN comes before
// +inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (x == 0.0f) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_of(float x, int index) {
  return (static_cast<uint64_t>(key_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int index_of(uint64_t order) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(order));
}
// The value of a key (+0 for both zeros, a NaN for NaN's), at least -inf.
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key < 0x007fffffu) return -INFINITY;
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The top list.  The largest elements of G groups of threads are found first:
// the top-th largest of those bounds the list from below, and few elements lie
// at or above it.  They are gathered and each finds its place by counting the
// ones before it.  G is 64 for short lists and 256 for long ones, so that the
// bound stays well inside the groups' maxima.  A row with more candidates than
// fit, or with NaN, takes one search over the row per place instead.  That is a row
// with many elements at or just above the bound: fewer finite ones than places (8
// allowed tokens in each of 4096 x 50257 bf16: top 20 2.2 ms instead of 0.09, top 64
// 6.2 instead of 0.11), or fp32 values whose spread is small beside their offset
// (1000 added to such logits in fp32, top 64: 7.0 instead of 0.20 ms).
//
// What this costs is a chain of small steps, while the CU's other row streams.
// So the bound is found by the last wave beside the others' exponentials, and
// the gathering needs no barrier of its own: few lanes hold candidates, and a
// wave's put what they hold into its own LDS, where every lane searches a vector
// of it.  Measured at 4096 x 50257, 64 places: 97 us, 68 us without the list, 114 us
// with each step behind a barrier and each thread searching its own elements.

constexpr int kCandidates = 512;
constexpr int kGroups = 256, kFewGroups = 64;
constexpr int kAllListed = 128;  // a vocabulary whose every element is a candidate
constexpr int kHolders = 16;     // lanes of a wave whose elements are searched at once

template <int NT, int NV> struct TopLds {
  static constexpr int G = NT < kGroups ? NT : kGroups;
  static constexpr int kWaves = NT / 64;
  u32x4 pool[kWaves][kHolders][NV > 0 ? NV : 1];
  uint64_t found[kCandidates];
  uint64_t best[kWaves];
  uint32_t group[G];
  float bound;
  uint32_t count;
  uint8_t holder[kWaves][kHolders];
};

// A key that at least `top` of the wave's M * 64 keys are not below, and few
// more: the keys' upper 16 bits, found bit by bit.
template <int M>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&k)[M], int top) {
  uint32_t bound = 0;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t c = bound | (1u << b);
    int have = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) have += __popcll(__ballot(k[i] >= c));
    if (have >= top) bound = c;
  }
  return bound;
}

// First step, before a barrier: the groups' maxima.
template <int NT, int NV>
__device__ __forceinline__ void top_groups(float own_max, TopLds<NT, NV>& lds) {
  constexpr int S = NT / TopLds<NT, NV>::G;
  static_assert(S == 1 || S == 2 || S == 4, "groups of up to four lanes");
  float g = own_max;
  if constexpr (S >= 2) g = fmaxf(g, lane_swap<kSwap1>(g));
  if constexpr (S >= 4) g = fmaxf(g, lane_swap<kSwap2>(g));
  if (threadIdx.x % S == 0) lds.group[threadIdx.x / S] = key_of(g);
  if (threadIdx.x == 0) lds.count = 0;
}

// Second step, between two barriers, by one whole wave: the bound.
template <int NT, int NV>
__device__ __forceinline__ void top_bound(int top, TopLds<NT, NV>& lds) {
  constexpr int M = TopLds<NT, NV>::G / 64;
  const int lane = threadIdx.x & 63;
  uint32_t k[M];
#pragma unroll
  for (int i = 0; i < M; ++i) k[i] = lds.group[i * 64 + lane];
  uint32_t bound = 0;
  if (M > 1 && top <= kFewGroups / 2) {
    uint32_t most[1] = {k[0]};
#pragma unroll
    for (int i = 1; i < M; ++i) most[0] = k[i] > most[0] ? k[i] : most[0];
    bound = bound_of<1>(most, top);
  } else if (top <= M * 64) {
    bound = bound_of<M>(k, top);
  }
  if (lane == 0) lds.bound = value_of(bound);
}

// Adds a lane's elements at or above the bound to the candidates; none is NaN.
// `at`: the row's index of the first.
template <int E, typename L>
__device__ __forceinline__ void add_candidates(const float (&x)[E], int at, float bound, L& lds) {
  float most = x[0];
#pragma unroll
  for (int i = 1; i < E; ++i) most = fmaxf(most, x[i]);
  if (most < bound) return;
  uint32_t hits = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) hits += x[i] >= bound ? 1u : 0u;
  uint32_t place = atomicAdd(&lds.count, hits);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (x[i] >= bound) {
      if (place < kCandidates) {
        // order_of without its case for NaN; adding +0 leaves one zero.
        const uint32_t u = __float_as_uint(x[i] + 0.0f);
        const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
        lds.found[place] = (static_cast<uint64_t>(key) << 32) | ~static_cast<uint32_t>(at + i);
      }
      ++place;
    }
  }
}

// Third step, behind a barrier: the `top` elements that come first, handed to
// emit(place, order).  own_max: the largest of the thread's elements; exact: the
// row holds no NaN.
template <typename T, int NT, int NV, bool ONCE, typename F>
__device__ __forceinline__ void top_list(const Row<T, NT, NV, ONCE>& r, int vocab, float own_max,
                                         bool exact, int top, TopLds<NT, NV>& lds, F emit) {
  constexpr int E = Row<T, NT, NV, ONCE>::E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool every = NT == 64 && vocab <= kAllListed;
  if (every || (exact && top <= TopLds<NT, NV>::G)) {
    const float bound = lds.bound;
    if (every) {
      if (lane == 0) lds.count = static_cast<uint32_t>(vocab);
      r.each([&](float x, int index) { lds.found[index] = order_of(x, index); });
    } else if constexpr (NV > 0) {
      bool holds = own_max >= bound;
      for (uint64_t mask = __ballot(holds); mask != 0; mask = __ballot(holds)) {
        const int mine = __popcll(mask & ((1ull << lane) - 1));
        const int all = __popcll(mask), now = all < kHolders ? all : kHolders;
        if (holds && mine < kHolders) {
          holds = false;
          lds.holder[wave][mine] = static_cast<uint8_t>(lane);
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (j * NT + static_cast<int>(threadIdx.x) < r.nvec) lds.pool[wave][mine][j] = r.kept[j];
        }
        wave_fence();
        for (int v = lane; v < now * NV; v += 64) {
          const int vec = v % NV * NT + wave * 64 + lds.holder[wave][v / NV];
          if (vec < r.nvec) {
            float x[E];
            r.unpack(lds.pool[wave][v / NV][v % NV], x);
            add_candidates(x, r.head + vec * E, bound, lds);
          }
        }
        wave_fence();
      }
    } else if (own_max >= bound) {
      r.vectors([&](float (&x)[E], int at, int) { add_candidates(x, at, bound, lds); });
    }
    if (!every && r.edge >= 0) {
      const float x[1] = {r.edge_x};
      add_candidates(x, r.edge, bound, lds);
    }
    __syncthreads();
    const int count = static_cast<int>(lds.count);
    if (count <= kCandidates) {
      // `parts` neighbouring lanes share a candidate's comparisons.
      for (int c0 = 0, parts; c0 < count; c0 += NT / parts) {
        for (parts = 1; parts < 8 && parts * 2 * (count - c0) <= NT;) parts *= 2;
        if (c0 + wave * 64 / parts >= count) break;
        const int c = c0 + static_cast<int>(threadIdx.x) / parts, part = threadIdx.x % parts;
        const uint64_t mine = c < count ? lds.found[c] : ~0ull;
        int place = 0;
#pragma unroll 4
        for (int o = part; o < count; o += parts) place += lds.found[o] > mine ? 1 : 0;
        for (int s = 1; s < parts; s <<= 1) place += __shfl_xor(place, s, 64);
        if (c < count && part == 0 && place < top) emit(place, mine);
      }
      return;
    }
  }
  const Row<T, NT, 0> again(r.p, vocab);
  uint64_t most = ~0ull;  // the next place's order at most; a NaN at token 0 has this one
  for (int k = 0; k < top; ++k) {
    uint64_t best = 0;
    again.each([&](float x, int index) {
      const uint64_t o = order_of(x, index);
      if (o <= most && o > best) best = o;
    });
    best = block_max<NT>(best, lds.best);
    if (threadIdx.x == 0) emit(k, best);
    most = best - 1;  // best > 0: no order is 0, and top <= vocab
  }
}

template <typename T> struct LogprobArgs {
  int64_t row0;  // first row of the launch
  const T* x;
  int64_t stride;
  int vocab;
  const void* targets;
  int id_bits;
  int top;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  // gradient
  const float* glogprob;
  const float* gentropy;
  T* dx;
  int64_t dstride;
};

// With d the elements' exponents, S = sum 2^d and A = sum 2^d d:
// log2 q = d - log2 S, H = (log2 S - A / S) ln 2.  Without the entropy A is left out
// (4096 x 50257 bf16: 64 us against 68).  Masked elements are cut at kLowest as they
// come: summing A over again where it came out NaN saved 3 % without masks and cost
// 30-50 % with half of the row masked.
//
// Bound by HBM: 4096 x 50257 bf16 in 68 us (6.1 TB/s), its gradient in 153 us, that
// of 8192 x 32000 in 187 us (5.6 TB/s, reads and writes mixed); one workgroup of 256
// threads reading the row for each step took 307-315 us for such gradients.
template <typename T, int NT, int NV, bool GRAD>
__global__ __launch_bounds__(NT, kRowWaves) void logprob_kernel(LogprobArgs<T> a) {
  __shared__ float lds_max[NT / 64];
  __shared__ float lds_sum[NT / 64][2];
  const int64_t i = a.row0 + blockIdx.x;
  const int64_t target = a.targets != nullptr ? id_at(a.targets, a.id_bits, i) : -1;
  const bool given = target >= 0 && target < a.vocab;
  float glp = 0.0f, gent = 0.0f;
  bool flat = false;
  if constexpr (GRAD) {
    glp = given && a.glogprob != nullptr ? a.glogprob[i] : 0.0f;
    gent = a.gentropy != nullptr ? a.gentropy[i] : 0.0f;
    flat = glp == 0.0f && gent == 0.0f;
    if (flat && a.logprob == nullptr && a.entropy == nullptr) {
      zero_row<T, NT>(a.dx + i * a.dstride, a.vocab);
      return;
    }
  }
  const T* row = a.x + i * a.stride;
  const Row<T, NT, NV, true> r(row, a.vocab);
  const float xt = given ? widen(row[target]) : 0.0f;
  const bool spread = a.entropy != nullptr || (GRAD && gent != 0.0f);  // A is needed
  float own_max = -INFINITY, sum[2] = {0.0f, 0.0f};
  if constexpr (NV > 0) r.each([&](float x, int) { own_max = fmaxf(own_max, x); });
  else if (spread) own_max = running_sums<true>(r, kLog2e, sum[0], sum[1]);
  else own_max = running_sums<false>(r, kLog2e, sum[0], sum[1]);
  extern __shared__ u32x4 top_memory[];  // with a top list
  TopLds<NT, NV>& lds_top = *reinterpret_cast<TopLds<NT, NV>*>(top_memory);
  if (!GRAD && a.top > 0) top_groups(own_max, lds_top);
  const Exponent e(block_max<NT>(own_max, lds_max), 1.0f, NV > 0);
  if (NT == 64) __syncthreads();
  if (!GRAD && a.top > 0 && threadIdx.x >= NT - 64 && (NT > 64 || a.vocab > kAllListed))
    top_bound(a.top, lds_top);
  if constexpr (NV == 0) {
    join_sums(e, own_max, sum[0], sum[1]);
  } else if (spread) {
    each_exponent(r, e, [&](float d) {
      const float p = __builtin_amdgcn_exp2f(d);
      sum[0] += p;
      sum[1] = fmaf(p, fmaxf(d, kLowest), sum[1]);
    });
  } else {
    each_exponent(r, e, [&](float d) { sum[0] += __builtin_amdgcn_exp2f(d); });
  }
  block_sum<NT, 2>(sum, lds_sum);
  const float log2s = log2f(sum[0]);
  const float h = (log2s - sum[1] / sum[0]) * kLn2;
  if (threadIdx.x == 0) {
    if (a.logprob != nullptr) a.logprob[i] = given ? e.log_q(xt, log2s) : 0.0f;
    if (a.entropy != nullptr) a.entropy[i] = h;
  }
  if constexpr (GRAD) {
    T* dx = a.dx + i * a.dstride;
    if (flat) {
      zero_row<T, NT>(dx, a.vocab);
      return;
    }
    // -q (glp + gent (log q + H)), with log q in powers of two.
    const float base = glp + gent * h, slope = gent * kLn2;
    auto value = [&](float d) {
      const float lq = d - log2s;
      return -__builtin_amdgcn_exp2f(lq) * fmaf(slope, fmaxf(lq, kLowest), base);
    };
    map_exponent(r, dx, e, value, [](auto&, int, int) {});
    // Over what its thread has just stored.
    if (given && r.owner(static_cast<int>(target)) == static_cast<int>(threadIdx.x))
      put(dx + target, glp + value(e.of(xt)));
  } else if (a.top > 0) {
    if (NT == 64) __syncthreads();
    top_list(r, a.vocab, own_max, sum[0] == sum[0], a.top, lds_top, [&](int place, uint64_t order) {
      a.top_ids[i * a.top + place] = index_of(order);
      a.top_logprobs[i * a.top + place] =
          e.log_q(value_of(static_cast<uint32_t>(order >> 32)), log2s);
    });
  }
}

template <typename T> struct DistillArgs {
  int64_t row0;  // first row of the launch
  const T* x;
  int64_t stride;
  int vocab;
  const void* ids;
  int id_bits;
  const void* teacher;
  int teacher_bf16;
  int k;
  int top;  // 0: the list's length does not choose the shape
  float inv_tau;
  float tau;
  float grad_scale;
  const float* weights;
  float* loss;
  T* dx;
  int64_t dstride;
};

// p = softmax over the listed z / tau, q = softmax over the row of x / tau:
// loss = w tau^2 sum_j p_j (log p_j - log q_j), dx = w c tau (q - p).
//
// The first wave holds the list, two entries per lane; its loads go out before
// the row's, so that the list is ready when the row comes.  A listed element's
// gradient is put into its vector by the thread that holds it, which finds its
// entries through `mail`: stored by itself, behind the vector, each costs HBM a
// partial write (8192 x 32000 bf16, 64 listed: 193 us, 5.4 TB/s, against 211 us;
// 4096 x 50257, 32 listed: 145 against 149).  One listed token takes 191 us there,
// 128 take 206.
template <typename T, int NT, int NV, bool GRAD>
__global__ __launch_bounds__(NT, kRowWaves) void distill_kernel(DistillArgs<T> a) {
  constexpr int M = GRZ_MAX_TOP / 64, kNone = 255, E = Row<T, NT, NV>::E;
  __shared__ float lds_max[NT / 64];
  __shared__ float lds_sum[NT / 64][1];
  __shared__ int32_t id[GRZ_MAX_TOP];
  __shared__ float p[GRZ_MAX_TOP];       // of the entry; behind the barrier, of its token
  __shared__ float xl[GRZ_MAX_TOP];
  __shared__ int mail[GRAD ? NT : 1];    // a thread's first entry
  __shared__ int next[GRZ_MAX_TOP];      // the same thread's next one
  __shared__ int listed;
  const int64_t i = a.row0 + blockIdx.x;
  const int lane = threadIdx.x & 63;
  int64_t v[M];
  float z[M];
  if (threadIdx.x < 64) {
#pragma unroll
    for (int j = 0; j < M; ++j) {
      v[j] = -1;
      z[j] = -INFINITY;
      if (j * 64 + lane < a.k) {
        const int64_t at = i * a.k + j * 64 + lane;
        v[j] = id_at(a.ids, a.id_bits, at);
        z[j] = a.teacher_bf16 ? widen(static_cast<const uint16_t*>(a.teacher)[at])
                              : static_cast<const float*>(a.teacher)[at];
      }
    }
  }
  const float w = a.weights != nullptr ? a.weights[i] : 1.0f;
  const T* row = a.x + i * a.stride;
  T* dx = nullptr;
  if constexpr (GRAD) dx = a.dx + i * a.dstride;
  if (w == 0.0f) {
    if (threadIdx.x == 0 && a.loss != nullptr) a.loss[i] = 0.0f;
    if constexpr (GRAD) zero_row<T, NT>(dx, a.vocab);
    return;
  }
  const Row<T, NT, NV, !GRAD> r(row, a.vocab);
  if constexpr (GRAD) mail[threadIdx.x] = kNone;
  float xj[M], pj[M];
  if (threadIdx.x < 64) {
    float zm = -INFINITY;
    bool any = false;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const bool ok = v[j] >= 0 && v[j] < a.vocab;
      xj[j] = ok ? widen(row[v[j]]) : 0.0f;
      if (!ok) {
        v[j] = -1;
        z[j] = -INFINITY;
      }
      any = any || !(z[j] == -INFINITY);
      zm = fmaxf(zm, z[j]);
    }
    const bool some = __ballot(any) != 0;
    zm = wave_max(zm);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      z[j] = (z[j] - zm) * (kLog2e * a.inv_tau);
      pj[j] = v[j] >= 0 ? __builtin_amdgcn_exp2f(z[j]) : 0.0f;
      sum += pj[j];
    }
    sum = wave_sum(sum);
    const float log2z = log2f(sum), inv = 1.0f / sum;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int q = j * 64 + lane;
      pj[j] *= inv;
      z[j] -= log2z;
      if (GRAD && q < a.k) {
        id[q] = static_cast<int32_t>(v[j]);
        p[q] = pj[j];
      }
    }
    if (lane == 0) listed = some;
  }
  float own_max = -INFINITY, sum[1] = {0.0f}, unused = 0.0f;
  if constexpr (NV > 0) r.each([&](float x, int) { own_max = fmaxf(own_max, x); });
  else own_max = running_sums<false>(r, kLog2e * a.inv_tau, sum[0], unused);
  if constexpr (NT == 64) __syncthreads();
  const float m = block_max<NT>(own_max, lds_max);  // its barrier also publishes the list
  if (!listed) {
    if (threadIdx.x == 0 && a.loss != nullptr) a.loss[i] = 0.0f;
    if constexpr (GRAD) zero_row<T, NT>(dx, a.vocab);
    return;
  }
  // By the last wave, which has the fewest vectors, beside the exponentials:
  // who stores each entry's token, and the token's whole p.  Entries of one token
  // have one owner, so only those that share theirs are compared.  Each of them
  // gets the whole p and is stored, the same value each time.
  if (GRAD && threadIdx.x >= NT - 64) {
    int owner[M];
    float all[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int q = j * 64 + lane;
      owner[j] = q < a.k && id[q] >= 0 ? r.owner(id[q]) : -1;
      all[j] = owner[j] >= 0 ? p[q] : 0.0f;
      if (owner[j] >= 0) next[q] = atomicExch(&mail[owner[j]], q);
    }
    wave_fence();
    uint64_t shared[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int q = j * 64 + lane;
      const bool with = owner[j] >= 0 && (mail[owner[j]] != q || next[q] != kNone);
      if (with) all[j] = 0.0f;
      shared[j] = __ballot(with);
    }
#pragma unroll
    for (int g = 0; g < M; ++g) {
      for (uint64_t left = shared[g]; left != 0; left &= left - 1) {
        const int f = g * 64 + __builtin_ctzll(left);
        const int32_t token = id[f];
        const float pf = p[f];
#pragma unroll
        for (int j = 0; j < M; ++j)
          if ((shared[j] >> lane & 1) != 0 && id[j * 64 + lane] == token) all[j] += pf;
      }
    }
    wave_fence();
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (owner[j] >= 0) p[j * 64 + lane] = all[j];
  }
  const Exponent e(m, a.inv_tau, NV > 0);
  if constexpr (NV == 0) join_sums(e, own_max, sum[0], unused);
  else each_exponent(r, e, [&](float d) { sum[0] += __builtin_amdgcn_exp2f(d); });
  if (GRAD && threadIdx.x < 64) {
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (j * 64 + lane < a.k) xl[j * 64 + lane] = xj[j];
  }
  if constexpr (NT == 64) __syncthreads();
  block_sum<NT, 1>(sum, lds_sum);  // its barrier stands between the last read and the first write
  const float log2s = log2f(sum[0]);
  if (threadIdx.x < 64 && a.loss != nullptr) {
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (pj[j] != 0.0f) part += pj[j] * (z[j] * kLn2 - e.log_q(xj[j], log2s));
    part = wave_sum(part);
    if (lane == 0) a.loss[i] = w * a.tau * a.tau * part;
  }
  if constexpr (GRAD) {
    const float c = w * a.grad_scale * a.tau;
    auto q_of = [&](float d) { return __builtin_amdgcn_exp2f(d - log2s); };
    auto listed_of = [&](int q) { return c * (q_of(e.of(xl[q])) - p[q]); };
    const int mine = mail[threadIdx.x];
    uint32_t hit = 0;  // which of the thread's vectors hold listed tokens, modulo 32
    for (int q = mine; q != kNone; q = next[q]) hit |= 1u << ((id[q] - r.head) / (E * NT) & 31);
    map_exponent(r, dx, e, [&](float d) { return c * q_of(d); },
                 [&](float (&x)[E], int at, int j) {
      if ((hit >> (j & 31) & 1) == 0) return;
      for (int q = mine; q != kNone; q = next[q]) {
        const int in = id[q] - at;
        const float value = listed_of(q);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = in == i ? value : x[i];
      }
    });
    for (int q = mine; q != kNone; q = next[q])
      if (id[q] == r.edge) put(dx + id[q], listed_of(q));
  }
}

// One workgroup per row, kRowBatch rows per launch.
template <typename Args>
int row_launch(void (*kernel)(Args), int threads, size_t lds, Args a, int64_t n,
               hipStream_t stream) {
  for (a.row0 = 0; a.row0 < n; a.row0 += kRowBatch) {
    const int64_t rows = n - a.row0 < kRowBatch ? n - a.row0 : kRowBatch;
    const int st = launch_lds(kernel, lds, dim3(static_cast<unsigned>(rows)), dim3(threads),
                              stream, a);
    if (st != GRZ_OK) return st;
  }
  return GRZ_OK;
}

// Threads per row and kept vectors per thread, by the row's 16-byte vectors: as
// many threads as leave each about eight vectors, all on their way at once, so
// that two workgroups of 1024 (or four of 512, ...) share a CU.  The gradient of
// 4096 x 50257 logits: 154 us with 1024 threads of 8 vectors, 162 with 512 of 13
// (three workgroups on a CU), 174 with 256 of 25 (four).  One wave per row up to
// 256 vectors (its lists are at most 64 long).  Rows of more vectors are read
// again: kept by 1024 threads of 16, which leaves one workgroup on a CU, 1024 x
// 128000 took 68 us instead of 50, their distillation loss 59 instead of 48, their
// gradient 115 instead of 125.
#define GRZ_ROW_SHAPES(CALL)                                  \
  const int64_t vectors = a.vocab / (16 / (int)sizeof(T));    \
  if (vectors <= 64 * 4 && a.top <= 64) return CALL(64, 4);   \
  if (vectors <= 256 * 8) return CALL(256, 8);                \
  if (vectors <= 512 * 8) return CALL(512, 8);                \
  if (vectors <= 1024 * 8) return CALL(1024, 8);              \
  return CALL(1024, 0);

template <typename T, bool GRAD>
int logprob_launch(const LogprobArgs<T>& a, int64_t n, hipStream_t stream) {
#define GRZ_CALL(NT, NV)                                                            \
  row_launch(logprob_kernel<T, NT, NV, GRAD>, NT, a.top > 0 ? sizeof(TopLds<NT, NV>) : 0, a, n, \
             stream)
  GRZ_ROW_SHAPES(GRZ_CALL)
#undef GRZ_CALL
}

template <typename T, bool GRAD>
int distill_launch(const DistillArgs<T>& a, int64_t n, hipStream_t stream) {
#define GRZ_CALL(NT, NV) row_launch(distill_kernel<T, NT, NV, GRAD>, NT, 0, a, n, stream)
  GRZ_ROW_SHAPES(GRZ_CALL)
#undef GRZ_CALL
}

// Whether dlogits may be written while logits are read: the same matrix, or
// apart from it.
int check_pair(const void* x, int dtype, int64_t n, int64_t vocab, int64_t stride,
               const void* dx, int64_t dstride) {
  const int st = check_matrix(dx, dtype, n, vocab, dstride);
  if (st != GRZ_OK) return st;
  if (x == dx && stride == dstride) return GRZ_OK;
  return overlap(x, span_of(dtype, n, vocab, stride), dx, span_of(dtype, n, vocab, dstride))
             ? GRZ_EINVAL : GRZ_OK;
}

// A flat array of a call over the vocabulary; absent: no bytes.
struct Flat {
  const void* at;
  size_t bytes;
  bool row_value;  // one fp32 value a row
  Flat(const void* p, int64_t count, size_t size, bool row = false)
      : at(p), bytes(p != nullptr ? static_cast<size_t>(count) * size : 0), row_value(row) {}
};
Flat row_values(const float* p, int64_t n) { return Flat(p, n, 4, true); }

// Whether an array lies over elements of a row matrix; what lies between the rows
// is the caller's.
bool covers(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride, const Flat& f) {
  if (!overlap(x, span_of(dtype, rows, cols, stride), f.at, f.bytes)) return false;
  const uintptr_t base = reinterpret_cast<uintptr_t>(x), at = reinterpret_cast<uintptr_t>(f.at);
  if (at <= base) return true;
  const size_t step = elem_size(dtype) * static_cast<size_t>(stride), in = (at - base) % step;
  return in < elem_size(dtype) * static_cast<size_t>(cols) || in + f.bytes > step;
}

// The outputs may not lie over an input or each other: workgroups write their rows
// while others still read theirs.  dlogits over the logits: check_pair.  A value a
// row may replace one that comes in: its row's workgroup has read that by then.
template <size_t I, size_t O>
int check_outputs(const void* logits, const void* dlogits, int dtype, int64_t n, int64_t vocab,
                  int64_t stride, int64_t dstride, const Flat (&in)[I], const Flat (&out)[O]) {
  for (const Flat& f : in)
    if (covers(dlogits, dtype, dlogits != nullptr ? n : 0, vocab, dstride, f)) return GRZ_EINVAL;
  for (size_t o = 0; o < O; ++o) {
    const Flat& f = out[o];
    if (covers(logits, dtype, n, vocab, stride, f) ||
        covers(dlogits, dtype, dlogits != nullptr ? n : 0, vocab, dstride, f))
      return GRZ_EINVAL;
    for (const Flat& i : in)
      if (overlap(i.at, i.bytes, f.at, f.bytes) && !(i.at == f.at && i.row_value && f.row_value))
        return GRZ_EINVAL;
    for (size_t k = 0; k < o; ++k)
      if (overlap(out[k].at, out[k].bytes, f.at, f.bytes)) return GRZ_EINVAL;
  }
  return GRZ_OK;
}

template <typename T>
int logprobs_entry(const void* logits, int64_t n, int64_t vocab, int64_t stride,
                   const void* targets, int id_bits, int top, float* logprob, float* entropy,
                   int32_t* top_ids, float* top_logprobs, const float* glogprob,
                   const float* gentropy, void* dlogits, int64_t dstride, hipStream_t stream) {
  LogprobArgs<T> a{0, static_cast<const T*>(logits), stride, static_cast<int>(vocab), targets,
                   id_bits, top, logprob, entropy, top_ids, top_logprobs, glogprob, gentropy,
                   static_cast<T*>(dlogits), dstride};
  return dlogits != nullptr ? logprob_launch<T, true>(a, n, stream)
                            : logprob_launch<T, false>(a, n, stream);
}

int check_list(const float* p) { return p == nullptr || aligned(p, 4) ? GRZ_OK : GRZ_EALIGN; }

template <typename T>
int distill_run(const void* logits, int64_t n, int64_t vocab, int64_t stride, const void* ids,
                int id_bits, const void* teacher, int teacher_dtype, int k, float temperature,
                const float* weights, float grad_scale, float* loss, void* dlogits,
                int64_t dstride, hipStream_t stream) {
  DistillArgs<T> a{0, static_cast<const T*>(logits), stride, static_cast<int>(vocab), ids, id_bits,
                   teacher, teacher_dtype == GRZ_BF16, k, 0, 1.0f / temperature, temperature,
                   grad_scale, weights, loss, static_cast<T*>(dlogits), dstride};
  return dlogits != nullptr ? distill_launch<T, true>(a, n, stream)
                            : distill_launch<T, false>(a, n, stream);
}

int distill_entry(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                  const void* ids, int id_bits, const void* teacher, int teacher_dtype, int k,
                  float temperature, const float* weights, float grad_scale, float* loss,
                  bool grad, void* dlogits, int64_t dstride, hipStream_t stream) {
  int st = check_matrix(logits, dtype, n, vocab, stride);
  if (st != GRZ_OK) return st;
  if (k < 1 || k > GRZ_MAX_TOP || !float_type(teacher_dtype)) return GRZ_EINVAL;
  // T^2 and log2(e) / T stay finite.
  if (!(temperature >= kMinTemperature) || !(temperature <= kMaxTemperature)) return GRZ_EINVAL;
  if (n > kMaxRows / k) return GRZ_ERANGE;
  if ((st = check_ids(ids, id_bits, n * k)) != GRZ_OK) return st;
  if (n == 0) return GRZ_OK;
  if (vocab < 1 || teacher == nullptr) return GRZ_EINVAL;
  if (!aligned(teacher, elem_size(teacher_dtype))) return GRZ_EALIGN;
  if (check_list(weights) != GRZ_OK || check_list(loss) != GRZ_OK) return GRZ_EALIGN;
  if (grad) {
    if ((st = check_pair(logits, dtype, n, vocab, stride, dlogits, dstride)) != GRZ_OK) return st;
  } else if (loss == nullptr) {
    return GRZ_EINVAL;
  }
  const Flat in[] = {Flat(ids, n * k, id_bits / 8), Flat(teacher, n * k, elem_size(teacher_dtype)),
                     row_values(weights, n)};
  const Flat out[] = {row_values(loss, n)};
  if ((st = check_outputs(logits, dlogits, dtype, n, vocab, stride, dstride, in, out)) != GRZ_OK)
    return st;
  return dtype == GRZ_BF16
             ? distill_run<uint16_t>(logits, n, vocab, stride, ids, id_bits, teacher,
                                     teacher_dtype, k, temperature, weights, grad_scale, loss,
                                     dlogits, dstride, stream)
             : distill_run<float>(logits, n, vocab, stride, ids, id_bits, teacher, teacher_dtype,
                                  k, temperature, weights, grad_scale, loss, dlogits, dstride,
                                  stream);
}

// ---------------------------------------------------------------------------
// Embedding, host side.

int bits_of(int64_t v) {
  int b = 1;
  while (v >> b) ++b;
  return b;
}

// Workspace of the gradient: two arrays of pairs, the tiles' digit counts and
// the digits' totals, and the chunks' partial sums, each on a 256-byte border.
struct GradPlan {
  int passes, bits, chunk;
  int threads;  // of a tile's workgroup
  int64_t tiles, chunks;
  size_t pairs_b, counts, totals, partial, total;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Pairs per chunk, a power of two from 8 to 128: short chunks give few rows
// enough waves (a 2560th of the rows' pieces of 256 columns), long ones keep the
// partial sums of long runs few.  16384 x 768: 34.7 us with 16, 36.8 with 8; 4096 x
// 768: 22.4 with 8, 24.4 with 16; 16384 x 4096: 93 with 64, 102 with 16.
int chunk_of(int64_t n, int64_t dim) {
  const int64_t want = n * ceil_div(dim, 256) / 2560;
  int c = 8;
  while (c < 128 && 2 * c <= want) c *= 2;
  return c;
}

GradPlan grad_plan(int64_t n, int64_t vocab, int64_t dim) {
  GradPlan p{};
  const int need = bits_of(vocab);  // keys 0 .. vocab
  p.passes = static_cast<int>(ceil_div(need, kMaxDigitBits));
  p.bits = static_cast<int>(ceil_div(need, p.passes));
  p.chunk = chunk_of(n, dim);
  p.threads = n <= kSmallSort ? kLittleSort : kBigSort;
  p.tiles = ceil_div(n, tile_of(p.threads));
  p.chunks = ceil_div(n, p.chunk);
  p.pairs_b = up256(static_cast<size_t>(n) * 8);
  p.counts = p.pairs_b + up256(static_cast<size_t>(n) * 8);
  p.totals = p.counts + up256(static_cast<size_t>(p.tiles) * kDigits * 4);
  p.partial = p.totals + up256(kDigits * 4);
  p.total = p.partial + static_cast<size_t>(p.chunks) * 2 * static_cast<size_t>(dim) * 4;
  return p;
}

// Columns per lane that the matrices allow: 4 (8-byte bf16 and 16-byte fp32
// accesses) or 1.
template <typename T>
bool vec_ok(const void* p, int64_t dim, int64_t stride, int vec) {
  return dim % vec == 0 && stride % vec == 0 &&
         aligned(p, sizeof(T) * vec < 16 ? sizeof(T) * vec : 16);
}

// Part `k` of `parts` of the rows of a table.
template <typename T>
ZeroRows zero_part(T* data, int64_t stride, int64_t rows, int64_t dim, int k, int parts,
                   bool stream) {
  ZeroRows z{reinterpret_cast<char*>(data), stride * static_cast<int64_t>(sizeof(T)),
             dim * static_cast<int64_t>(sizeof(T)), rows * k / parts, rows * (k + 1) / parts, 16,
             stream};
  const uint64_t at = reinterpret_cast<uintptr_t>(data) | static_cast<uint64_t>(z.bytes) |
                      static_cast<uint64_t>(rows > 1 ? z.stride : 0);
  while (at % z.unit) z.unit /= 2;
  return z;
}

// Workgroups of `waves` waves for such a part: at most all the chip holds.
unsigned zero_blocks(const ZeroRows& z, int waves) {
  const int64_t want = ceil_div(z.row1 - z.row0, waves), most = 8192 / waves;
  return static_cast<unsigned>(want < most ? want : most);
}

// Sorts the ids into pairs (*sorted) and writes the table's zeros, which
// zeros(k, parts) describes, beside it.
template <typename Z>
int rank_launch(const SortSrc& src, int64_t n, u32x2* pairs, Z zeros, hipStream_t stream) {
  const ZeroRows z = zeros(0, 1);
  const unsigned own = static_cast<unsigned>(ceil_div(n, kRankLanes));
  return launch(rank_kernel, dim3(own + zero_blocks(z, kRankWaves)), dim3(kRankWaves * 64), stream,
                src, static_cast<int>(n), pairs, z);
}

template <typename Z>
int merge_launch(const SortSrc& src, int64_t n, u32x2* const (&pairs)[2], Z zeros,
                 hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>(ceil_div(n, kMergeTile));
  const ZeroRows z0 = zeros(0, 2), z1 = zeros(1, 2);
  const int st = launch(sort_tiles_kernel, dim3(tiles + zero_blocks(z0, kMergeTile / 64)),
                        dim3(kMergeTile), stream, src, static_cast<int>(n), pairs[1], z0);
  if (st != GRZ_OK) return st;
  return launch_lds(merge_tiles_kernel, tiles * kMergeTile * 4,
                    dim3(static_cast<unsigned>(ceil_div(n, 64)) + zero_blocks(z1, kRankWaves)),
                    dim3(kRankWaves * 64), stream, pairs[1], static_cast<int>(n), pairs[0], z1);
}

template <int NT, typename Z>
int sort_launch(SortSrc src, int64_t n, const GradPlan& p, u32x2* const (&pairs)[2],
                uint32_t* counts, uint32_t* totals, Z zeros, const u32x2** sorted,
                hipStream_t stream) {
  const dim3 threads(NT);
  const unsigned tiles = static_cast<unsigned>(p.tiles);
  const int digits = 1 << p.bits, waves = NT / 64;
  for (int k = 0; k < p.passes; ++k) {
    const int shift = k * p.bits;
    const ZeroRows z = zeros(k, p.passes);
    const dim3 grid(tiles + zero_blocks(z, waves));
    u32x2* out = pairs[k & 1];
    int st = launch(sort_count_kernel<NT>, dim3(tiles), threads, stream, src, n, shift, p.bits,
                    counts);
    if (st != GRZ_OK) return st;
    auto scatter = sort_scatter_kernel<NT, false>;
    if constexpr (NT == kBigSort) {  // the little tiles are kDirectTiles at most
      if (p.tiles > kDirectTiles) {
        st = launch(sort_scan_kernel, dim3(static_cast<unsigned>(ceil_div(digits, 64))),
                    dim3(kScanWaves * 64), stream, counts, totals, p.tiles, digits);
        if (st != GRZ_OK) return st;
        scatter = sort_scatter_kernel<NT, true>;
      }
    }
    st = launch(scatter, grid, threads, stream, src, n, shift, p.bits, counts, totals, out, z);
    if (st != GRZ_OK) return st;
    *sorted = out;
    src = SortSrc{nullptr, 0, out, src.vocab};
  }
  return GRZ_OK;
}

// The kernel for `pieces` pieces of columns and the waves that share them: at
// most as many a wave as its registers hold rows of on their way.
template <typename TI, typename TO, int VEC, bool ACC>
auto grad_kernel_for(int64_t pieces, int64_t* waves) {
  constexpr int most = VEC == 1 ? 2 : (sizeof(TI) == 2 ? 4 : 2) / (ACC ? 2 : 1);
  *waves = ceil_div(pieces, most);
  const int each = static_cast<int>(ceil_div(pieces, *waves));
  auto kernel = embed_grad_kernel<TI, TO, VEC, 1, ACC>;
  if constexpr (most >= 2) {
    if (each == 2) kernel = embed_grad_kernel<TI, TO, VEC, 2, ACC>;
  }
  if constexpr (most >= 4) {
    if (each == 3) kernel = embed_grad_kernel<TI, TO, VEC, 3, ACC>;
    if (each == 4) kernel = embed_grad_kernel<TI, TO, VEC, 4, ACC>;
  }
  return kernel;
}

template <typename TI, typename TO, int VEC>
int embed_grad_launch(const TI* dout, int64_t istride, const void* ids, int id_bits, int64_t n,
                      int64_t vocab, int64_t dim, float scale, int accumulate, char* ws,
                      TO* dtable, int64_t ostride, hipStream_t stream) {
  if (n == 0) {
    if (accumulate) return GRZ_OK;
    const ZeroRows z = zero_part(dtable, ostride, vocab, dim, 0, 1, true);
    return launch(zero_rows_kernel, dim3(zero_blocks(z, 4)), dim3(256), stream, z);
  }
  const int64_t pieces = ceil_div(dim, 64 * VEC);
  if (n <= kDirectIds && n <= kDirectMean * vocab && vocab * pieces <= kDirectGroups)
    return launch(accumulate ? direct_grad_kernel<TI, TO, VEC, true>
                             : direct_grad_kernel<TI, TO, VEC, false>,
                  dim3(static_cast<unsigned>(vocab), static_cast<unsigned>(pieces)),
                  dim3(kDirectWaves * 64), stream, dout, istride, ids, id_bits,
                  static_cast<int>(n), dim, scale, dtable, ostride);
  const GradPlan p = grad_plan(n, vocab, dim);
  u32x2* const pairs[2] = {reinterpret_cast<u32x2*>(ws),
                           reinterpret_cast<u32x2*>(ws + p.pairs_b)};
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + p.counts);
  uint32_t* totals = reinterpret_cast<uint32_t*>(ws + p.totals);
  float* partial = reinterpret_cast<float*>(ws + p.partial);
  const SortSrc src{ids, id_bits, nullptr, static_cast<uint32_t>(vocab)};
  auto zeros = [&](int k, int parts) {
    return zero_part(dtable, ostride, accumulate ? 0 : vocab, dim, k, parts, n > kRankIds);
  };
  const u32x2* sorted = pairs[0];
  int st;
  if (n <= kRankIds) st = rank_launch(src, n, pairs[0], zeros, stream);
  else if (n <= kMergeIds) st = merge_launch(src, n, pairs, zeros, stream);
  else st = p.threads == kBigSort
               ? sort_launch<kBigSort>(src, n, p, pairs, counts, totals, zeros, &sorted, stream)
               : sort_launch<kLittleSort>(src, n, p, pairs, counts, totals, zeros, &sorted,
                                          stream);
  if (st != GRZ_OK) return st;
  int64_t waves = 0;
  auto kernel = accumulate ? grad_kernel_for<TI, TO, VEC, true>(pieces, &waves)
                           : grad_kernel_for<TI, TO, VEC, false>(pieces, &waves);
  const uint32_t none = static_cast<uint32_t>(vocab);
  st = launch(kernel, dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(waves)),
              dim3(64), stream, dout, istride, sorted, n, p.chunk, none, dim, scale, partial,
              dtable, ostride);
  if (st != GRZ_OK || p.chunks == 1) return st;
  return launch(accumulate ? join_kernel<TO, VEC, true> : join_kernel<TO, VEC, false>,
                dim3(static_cast<unsigned>(p.chunks - 1), static_cast<unsigned>(pieces)),
                dim3(kJoinWaves * 64), stream, sorted, n, p.chunk, none, dim, scale, partial,
                dtable, ostride);
}

template <typename TI, typename TO>
int embed_grad_run(const void* dout, int64_t istride, const void* ids, int id_bits, int64_t n,
                   int64_t vocab, int64_t dim, float scale, int accumulate, void* ws,
                   void* dtable, int64_t ostride, hipStream_t stream) {
  const TI* x = static_cast<const TI*>(dout);
  TO* y = static_cast<TO*>(dtable);
  char* w = static_cast<char*>(ws);
  if (vec_ok<TI>(x, dim, istride, 4) && vec_ok<TO>(y, dim, ostride, 4))
    return embed_grad_launch<TI, TO, 4>(x, istride, ids, id_bits, n, vocab, dim, scale,
                                        accumulate, w, y, ostride, stream);
  return embed_grad_launch<TI, TO, 1>(x, istride, ids, id_bits, n, vocab, dim, scale, accumulate,
                                      w, y, ostride, stream);
}

template <typename TI, typename TO, int VEC>
int lookup_launch(const TI* table, int64_t tstride, int64_t vocab, int64_t dim, const void* ids,
                  int id_bits, int64_t n, float scale, TO* out, int64_t ostride,
                  hipStream_t stream) {
  constexpr int64_t batch = 4 * kRowBatch;  // four rows per workgroup
  for (int64_t r = 0; r < n; r += batch) {
    const int64_t rows = n - r < batch ? n - r : batch;
    const int st = launch(lookup_kernel<TI, TO, VEC>,
                          dim3(static_cast<unsigned>(ceil_div(rows, 4))), dim3(256), stream,
                          table, tstride, vocab, dim, ids, id_bits, r, n, scale, out, ostride);
    if (st != GRZ_OK) return st;
  }
  return GRZ_OK;
}

template <typename TI, typename TO>
int lookup_run(const void* table, int64_t tstride, int64_t vocab, int64_t dim, const void* ids,
               int id_bits, int64_t n, float scale, void* out, int64_t ostride,
               hipStream_t stream) {
  const TI* x = static_cast<const TI*>(table);
  TO* y = static_cast<TO*>(out);
  if (vec_ok<TI>(x, dim, tstride, 8) && vec_ok<TO>(y, dim, ostride, 8))
    return lookup_launch<TI, TO, 8>(x, tstride, vocab, dim, ids, id_bits, n, scale, y, ostride,
                                    stream);
  if (vec_ok<TI>(x, dim, tstride, 4) && vec_ok<TO>(y, dim, ostride, 4))
    return lookup_launch<TI, TO, 4>(x, tstride, vocab, dim, ids, id_bits, n, scale, y, ostride,
                                    stream);
  return lookup_launch<TI, TO, 1>(x, tstride, vocab, dim, ids, id_bits, n, scale, y, ostride,
                                  stream);
}

}  // namespace

// ---------------------------------------------------------------------------
// C ABI

extern "C" {

int dp_embed_lookup(const void* table, int table_dtype, int64_t vocab, int64_t dim,
                    int64_t table_stride, const void* ids, int id_bits, int64_t n, float scale,
                    void* out, int out_dtype, int64_t out_stride, hipStream_t stream) {
  int st = check_ids(ids, id_bits, n);
  if (st != GRZ_OK) return st;
  if ((st = check_matrix(out, out_dtype, n, dim, out_stride)) != GRZ_OK) return st;
  if (n == 0 || dim == 0) return check_matrix(nullptr, table_dtype, 0, dim, table_stride);
  if ((st = check_matrix(table, table_dtype, vocab, dim, table_stride)) != GRZ_OK) return st;
  const size_t out_bytes = span_of(out_dtype, n, dim, out_stride);
  if (overlap(table, span_of(table_dtype, vocab, dim, table_stride), out, out_bytes) ||
      overlap(ids, static_cast<size_t>(n) * (id_bits / 8), out, out_bytes))
    return GRZ_EINVAL;
  if (table_dtype == GRZ_BF16)
    return out_dtype == GRZ_BF16
               ? lookup_run<uint16_t, uint16_t>(table, table_stride, vocab, dim, ids, id_bits, n,
                                                scale, out, out_stride, stream)
               : lookup_run<uint16_t, float>(table, table_stride, vocab, dim, ids, id_bits, n,
                                             scale, out, out_stride, stream);
  return out_dtype == GRZ_BF16
             ? lookup_run<float, uint16_t>(table, table_stride, vocab, dim, ids, id_bits, n,
                                           scale, out, out_stride, stream)
             : lookup_run<float, float>(table, table_stride, vocab, dim, ids, id_bits, n, scale,
                                        out, out_stride, stream);
}

size_t dp_embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
  if (n <= 0 || vocab <= 0 || dim <= 0 || n > kGradIds || vocab > kGradRows || dim > kGradCols)
    return 0;
  return grad_plan(n, vocab, dim).total;
}

int dp_embed_grad(const void* dout, int dout_dtype, int64_t dout_stride, const void* ids,
                  int id_bits, int64_t n, int64_t vocab, int64_t dim, float scale, int flags,
                  void* workspace, void* dtable, int dtable_dtype, int64_t dtable_stride,
                  hipStream_t stream) {
  if (flags & ~GRZ_ACCUMULATE) return GRZ_EINVAL;
  int st = check_ids(ids, id_bits, n);
  if (st != GRZ_OK) return st;
  if (n > kGradIds || vocab > kGradRows || dim > kGradCols) return GRZ_ERANGE;
  if ((st = check_matrix(dout, dout_dtype, n, dim, dout_stride)) != GRZ_OK) return st;
  if ((st = check_matrix(dtable, dtable_dtype, vocab, dim, dtable_stride)) != GRZ_OK) return st;
  if (vocab == 0 || dim == 0) return GRZ_OK;
  const size_t need = dp_embed_grad_workspace(n, vocab, dim);
  if (need > 0) {
    if (workspace == nullptr) return GRZ_EINVAL;
    if (!aligned(workspace, 16)) return GRZ_EALIGN;
  }
  const size_t table_bytes = span_of(dtable_dtype, vocab, dim, dtable_stride);
  if (overlap(dout, span_of(dout_dtype, n, dim, dout_stride), dtable, table_bytes) ||
      overlap(workspace, need, dtable, table_bytes) ||
      overlap(workspace, need, dout, span_of(dout_dtype, n, dim, dout_stride)) ||
      overlap(workspace, need, ids, static_cast<size_t>(n) * (id_bits / 8)) ||
      overlap(ids, static_cast<size_t>(n) * (id_bits / 8), dtable, table_bytes))
    return GRZ_EINVAL;
  const int acc = flags & GRZ_ACCUMULATE ? 1 : 0;
  if (dout_dtype == GRZ_BF16)
    return dtable_dtype == GRZ_BF16
               ? embed_grad_run<uint16_t, uint16_t>(dout, dout_stride, ids, id_bits, n, vocab,
                                                    dim, scale, acc, workspace, dtable,
                                                    dtable_stride, stream)
               : embed_grad_run<uint16_t, float>(dout, dout_stride, ids, id_bits, n, vocab, dim,
                                                 scale, acc, workspace, dtable, dtable_stride,
                                                 stream);
  return dtable_dtype == GRZ_BF16
             ? embed_grad_run<float, uint16_t>(dout, dout_stride, ids, id_bits, n, vocab, dim,
                                               scale, acc, workspace, dtable, dtable_stride,
                                               stream)
             : embed_grad_run<float, float>(dout, dout_stride, ids, id_bits, n, vocab, dim, scale,
                                            acc, workspace, dtable, dtable_stride, stream);
}

int dp_token_logprobs(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                      const void* targets, int id_bits, int top, float* logprob, float* entropy,
                      int32_t* top_ids, float* top_logprobs, hipStream_t stream) {
  int st = check_matrix(logits, dtype, n, vocab, stride);
  if (st != GRZ_OK) return st;
  if (top < 0 || top > GRZ_MAX_TOP || top > vocab) return GRZ_EINVAL;
  if (targets != nullptr && (st = check_ids(targets, id_bits, n)) != GRZ_OK) return st;
  if (logprob != nullptr && targets == nullptr && n > 0) return GRZ_EINVAL;
  if (n == 0) return GRZ_OK;
  if (vocab < 1) return GRZ_EINVAL;
  if (top > 0 && (top_ids == nullptr || top_logprobs == nullptr)) return GRZ_EINVAL;
  if (logprob == nullptr && entropy == nullptr && top == 0) return GRZ_EINVAL;
  if (check_list(logprob) != GRZ_OK || check_list(entropy) != GRZ_OK ||
      check_list(top_logprobs) != GRZ_OK || (top_ids != nullptr && !aligned(top_ids, 4)))
    return GRZ_EALIGN;
  const Flat in[] = {Flat(targets, n, id_bits / 8)};
  const Flat out[] = {row_values(logprob, n), row_values(entropy, n), Flat(top_ids, n * top, 4),
                      Flat(top_logprobs, n * top, 4)};
  if ((st = check_outputs(logits, nullptr, dtype, n, vocab, stride, 0, in, out)) != GRZ_OK)
    return st;
  return dtype == GRZ_BF16
             ? logprobs_entry<uint16_t>(logits, n, vocab, stride, targets, id_bits, top, logprob,
                                        entropy, top_ids, top_logprobs, nullptr, nullptr, nullptr,
                                        0, stream)
             : logprobs_entry<float>(logits, n, vocab, stride, targets, id_bits, top, logprob,
                                     entropy, top_ids, top_logprobs, nullptr, nullptr, nullptr, 0,
                                     stream);
}

int dp_token_logprobs_grad(const void* logits, int dtype, int64_t n, int64_t vocab,
                           int64_t stride, const void* targets, int id_bits,
                           const float* glogprob, const float* gentropy, float* logprob,
                           float* entropy, void* dlogits, int64_t dlogits_stride,
                           hipStream_t stream) {
  int st = check_matrix(logits, dtype, n, vocab, stride);
  if (st != GRZ_OK) return st;
  if (targets != nullptr && (st = check_ids(targets, id_bits, n)) != GRZ_OK) return st;
  if (n == 0) return GRZ_OK;
  if (vocab < 1 || (glogprob == nullptr && gentropy == nullptr)) return GRZ_EINVAL;
  if (targets == nullptr && (glogprob != nullptr || logprob != nullptr)) return GRZ_EINVAL;
  if (check_list(logprob) != GRZ_OK || check_list(entropy) != GRZ_OK ||
      check_list(glogprob) != GRZ_OK || check_list(gentropy) != GRZ_OK)
    return GRZ_EALIGN;
  if ((st = check_pair(logits, dtype, n, vocab, stride, dlogits, dlogits_stride)) != GRZ_OK)
    return st;
  const Flat in[] = {Flat(targets, n, id_bits / 8), row_values(glogprob, n),
                     row_values(gentropy, n)};
  const Flat out[] = {row_values(logprob, n), row_values(entropy, n)};
  if ((st = check_outputs(logits, dlogits, dtype, n, vocab, stride, dlogits_stride, in, out)) !=
      GRZ_OK)
    return st;
  return dtype == GRZ_BF16
             ? logprobs_entry<uint16_t>(logits, n, vocab, stride, targets, id_bits, 0, logprob,
                                        entropy, nullptr, nullptr, glogprob, gentropy, dlogits,
                                        dlogits_stride, stream)
             : logprobs_entry<float>(logits, n, vocab, stride, targets, id_bits, 0, logprob,
                                     entropy, nullptr, nullptr, glogprob, gentropy, dlogits,
                                     dlogits_stride, stream);
}

int dp_distill_loss(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                    const void* teacher_ids, int id_bits, const void* teacher_logits,
                    int teacher_dtype, int k, float temperature, const float* weights,
                    float* loss, hipStream_t stream) {
  return distill_entry(logits, dtype, n, vocab, stride, teacher_ids, id_bits, teacher_logits,
                       teacher_dtype, k, temperature, weights, 1.0f, loss, false, nullptr, 0,
                       stream);
}

int dp_distill_grad(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                    const void* teacher_ids, int id_bits, const void* teacher_logits,
                    int teacher_dtype, int k, float temperature, const float* weights,
                    float grad_scale, float* loss, void* dlogits, int64_t dlogits_stride,
                    hipStream_t stream) {
  return distill_entry(logits, dtype, n, vocab, stride, teacher_ids, id_bits, teacher_logits,
                       teacher_dtype, k, temperature, weights, grad_scale, loss, true, dlogits,
                       dlogits_stride, stream);
}

}  // extern "C"
