// tensors.hip -- HIP kernels and C ABI of the gradient norm over many tensors and
// their clipping for AMD Instinct MI355X (gfx950, CDNA4, wave64):
//   dp_grad_sqnorm_tensors  squared norm and clip factor over a list of tensors
//   dp_grad_clip_tensors    the list scaled by the factor, in place or elsewhere
//
// Gradients that sit in no arena (a rank's own experts) count in the same norm as
// the arena's: the list's piece sums are formed as the reduce forms the arena's and
// go through the same tree.  The list travels in the kernel arguments, kListed
// tensors a launch: nothing is copied to the device, so a list may change from step
// to step and a captured graph holds its own.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>

#include <limits.h>
#include <stdint.h>

#include "grz.h"
#include "rows.h"

namespace {

constexpr int64_t kMaxElements = int64_t{1} << 37;  // of all tensors of a call
// Pieces of one launch, whose threads stay below 2^32; longer lists take more launches.
constexpr int64_t kLaunchPieces = int64_t{1} << 22;
constexpr int64_t kMaxPieces = int64_t{4096} * 4096 * 4096;  // of the norm's tree

template <int LISTED> struct List {
  int count;
  uint32_t pieces;         // of all its tensors
  uint32_t first[LISTED];  // the tensor's first piece in this launch
  uint8_t type[LISTED];
  int64_t numel[LISTED];
  const void* data[LISTED];
};
struct NormArgs {
  static constexpr int kListed = 184;
  List<kListed> list;
  double* pieces;
};
struct ClipArgs {
  static constexpr int kListed = 128;
  List<kListed> list;
  uint8_t out_type[kListed];
  void* out[kListed];
  const float* scale;
};
static_assert(sizeof(NormArgs) <= 4096 && sizeof(ClipArgs) <= 4096,
              "a launch's arguments exceed 4 KB");

// The tensor that holds a piece: the last one whose first piece is not behind it.  All
// first pieces are compared at once, one a lane: a launch's arguments come from far,
// so a search of one dependent read after the other costs each wave microseconds.
template <int LISTED>
__device__ __forceinline__ int tensor_of(const List<LISTED>& l, uint32_t piece, int lane) {
  int t = -1;
#pragma unroll
  for (int b = 0; b < LISTED; b += 64) {
    const int i = b + lane;
    const bool there = i < LISTED && i < l.count && l.first[i < LISTED ? i : 0] <= piece;
    t += __popcll(__ballot(there));
  }
  return __builtin_amdgcn_readfirstlane(t);
}

// The wave's piece in its tensor.
struct Piece {
  int tensor;
  int64_t at;    // its first element
  int64_t left;  // elements from there on
};
template <int LISTED>
__device__ __forceinline__ Piece piece_of(const List<LISTED>& l, uint32_t number, int lane) {
  Piece p;
  p.tensor = tensor_of(l, number, lane);
  p.at = static_cast<int64_t>(number - l.first[p.tensor]) * GRZ_PIECE;
  p.left = l.numel[p.tensor] - p.at;
  return p;
}

// 16 or 8 bytes at any element's address.
template <bool STREAM> __device__ __forceinline__ u32x4 load16(const void* p) {
  const u32x4e* q = static_cast<const u32x4e*>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool STREAM> __device__ __forceinline__ u32x2 load8(const void* p) {
  const u32x2e* q = static_cast<const u32x2e*>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool STREAM> __device__ __forceinline__ void store16(void* p, u32x4 v) {
  u32x4e* q = static_cast<u32x4e*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}
template <bool STREAM> __device__ __forceinline__ void store8(void* p, u32x2 v) {
  u32x2e* q = static_cast<u32x2e*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}

// WORDS words of the elements from `e` on, 0 where not all of them are among the first
// `left` (FULL: all are, and nothing is asked, which keeps the loads of a piece
// together: 1.04 G elements' norm 311 us instead of 341, clip 665 instead of 695).
template <bool STREAM, bool FULL, int WORDS, typename T>
__device__ __forceinline__ auto load_whole(const T* p, int e, int64_t left) {
  uint32_t __attribute__((ext_vector_type(WORDS))) u = {};
  if (FULL || e + WORDS * 4 / static_cast<int>(sizeof(T)) <= left) {
    if constexpr (WORDS == 4) u = load16<STREAM>(p + e);
    else u = load8<STREAM>(p + e);
  }
  return u;
}

// The elements behind the last whole vector of N, read one a lane (one after the other
// by the lane whose vector they are, they take microseconds).
template <typename T, int N> struct Rest {
  int at, count;
  T mine;
  __device__ __forceinline__ Rest(const T* p, int64_t left, int lane) {
    const int n = left < GRZ_PIECE ? static_cast<int>(left) : GRZ_PIECE;
    count = n % N;
    at = n - count;
    mine = lane < count ? p[at + lane] : T{};
  }
  // Puts them where a lane holds the vector that begins at `at`.
  template <typename V> __device__ __forceinline__ void into(V& u, int e) const {
    if (count == 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t bits;
      if constexpr (sizeof(T) == 2)
        bits = static_cast<uint32_t>(__builtin_amdgcn_readlane(mine, i)) << (16 * (i & 1));
      else
        bits = __builtin_amdgcn_readlane(__float_as_uint(mine), i);
      if (e == at) u[i * static_cast<int>(sizeof(T)) / 4] |= bits;
    }
  }
};

// ---------------------------------------------------------------------------
// Piece sums.  Their bits are those of the reduce's piece sums: thread t of 256 takes
// elements 1024 k + 4 t .. + 3 for k = 0 .. 3, squares added in fp64 in that order,
// then a balanced tree over each 64 threads and (w0 + w1) + (w2 + w3).  Elements behind
// a tensor's last count as 0, which changes no sum of squares.
//
//  - Many pieces: a wave a piece, without a barrier, all of it on its way at once.  A
//    lane stands for four of those threads: with fp32 elements for t = lane + 64 w (16
//    accesses of 16 bytes), with bf16 for t = 2 lane and 2 lane + 1 of each half (8 of
//    16 bytes), whose first addition is then its own.  Bound by HBM: 1.04 G bf16
//    elements in 138 tensors 311 us, 6.7 TB/s.
//  - Few: a workgroup a piece, which shortens each wave's chain of conversions and
//    additions (when first built, norms of 10.6 M elements 11.8 us bf16 and 13.5 fp32
//    against 16.1 and 20.3, of 24 M bf16 16.0 against 16.7, of 100 M 56 against 38; now
//    9.4 and 11.4, the tree's launch of 2.6 included).

template <int CTRL> __device__ __forceinline__ double add_swapped(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(b), CTRL, 0xf, 0xf,
                                                  false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(b >> 32), CTRL, 0xf,
                                                  0xf, false);
  return v + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// The wave's sum, lane by lane from neighbours outwards.
__device__ __forceinline__ double wave_sum(double v) {
  v = add_swapped<kSwap1>(v);
  v = add_swapped<kSwap2>(v);
  v = add_swapped<kHalfMirror>(v);
  v = add_swapped<kMirror>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

__device__ __forceinline__ void add_square(double& s, float x) {
  s = __fma_rn(static_cast<double>(x), static_cast<double>(x), s);
}
// A word's squares: one fp32 element's or two bf16 ones'.
template <typename T> __device__ __forceinline__ void add_squares(double& s, uint32_t word) {
  if constexpr (sizeof(T) == 2) {
    add_square(s, __uint_as_float(word << 16));
    add_square(s, __uint_as_float(word & 0xffff0000u));
  } else {
    add_square(s, __uint_as_float(word));
  }
}

template <bool STREAM, bool FULL>
__device__ __forceinline__ double piece_sum(const uint16_t* p, int64_t left, int lane) {
  u32x4 u[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      u[k][h] = load_whole<STREAM, FULL, 4>(p, 1024 * k + 512 * h + 8 * lane, left);
  if constexpr (!FULL) {
    const Rest<uint16_t, 8> rest(p, left, lane);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) rest.into(u[k][h], 1024 * k + 512 * h + 8 * lane);
  }
  double w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    double s[2] = {};  // of the lane's two threads
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) add_squares<uint16_t>(s[i >> 1], u[k][h][i]);
    // Lanes 0 .. 31 hold one wave's threads, 32 .. 63 the next one's.
    w[h] = wave_sum(s[0] + s[1]);
  }
  return w[0] + w[1];
}

template <bool STREAM, bool FULL>
__device__ __forceinline__ double piece_sum(const float* p, int64_t left, int lane) {
  u32x4 u[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int w = 0; w < 4; ++w)
      u[k][w] = load_whole<STREAM, FULL, 4>(p, 1024 * k + 256 * w + 4 * lane, left);
  if constexpr (!FULL) {
    const Rest<float, 4> rest(p, left, lane);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int w = 0; w < 4; ++w) rest.into(u[k][w], 1024 * k + 256 * w + 4 * lane);
  }
  double s[4] = {};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) add_squares<float>(s[w], u[k][w][i]);
    s[w] = wave_sum(s[w]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <bool STREAM, bool FULL>
__device__ __forceinline__ double piece_sum_of(const NormArgs& a, const Piece& p, int lane) {
  const void* data = a.list.data[p.tensor];
  return a.list.type[p.tensor] == GRZ_BF16
             ? piece_sum<STREAM, FULL>(static_cast<const uint16_t*>(data) + p.at, p.left, lane)
             : piece_sum<STREAM, FULL>(static_cast<const float*>(data) + p.at, p.left, lane);
}

template <bool STREAM> __global__ __launch_bounds__(256) void tensors_norm_kernel(
    const NormArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t number =
      blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (number >= a.list.pieces) return;
  const Piece p = piece_of(a.list, number, lane);
  const double sum = p.left >= GRZ_PIECE ? piece_sum_of<STREAM, true>(a, p, lane)
                                         : piece_sum_of<STREAM, false>(a, p, lane);
  if (lane == 0) a.pieces[number] = sum;
}

// The sum of the wave's 64 of the 256 threads.
template <bool FULL, typename T>
__device__ __forceinline__ double quarter_sum(const T* p, int64_t left) {
  constexpr int W = sizeof(T);  // words of four elements
  const int t = threadIdx.x;
  uint32_t __attribute__((ext_vector_type(W))) u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) u[k] = load_whole<false, FULL, W>(p, 1024 * k + 4 * t, left);
  if constexpr (!FULL) {
    const Rest<T, 4> rest(p, left, t & 63);
#pragma unroll
    for (int k = 0; k < 4; ++k) rest.into(u[k], 1024 * k + 4 * t);
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < W; ++i) add_squares<T>(s, u[k][i]);
  return wave_sum(s);
}

constexpr uint32_t kFewPieces = 6144;

__global__ __launch_bounds__(256) void tensors_norm_few_kernel(const NormArgs a) {
  __shared__ double sums[4];
  const Piece p = piece_of(a.list, blockIdx.x, threadIdx.x & 63);
  const void* data = a.list.data[p.tensor];
  const uint16_t* h = static_cast<const uint16_t*>(data) + p.at;
  const float* f = static_cast<const float*>(data) + p.at;
  const bool half = a.list.type[p.tensor] == GRZ_BF16;
  const double s = p.left >= GRZ_PIECE
                       ? (half ? quarter_sum<true>(h, p.left) : quarter_sum<true>(f, p.left))
                       : (half ? quarter_sum<false>(h, p.left) : quarter_sum<false>(f, p.left));
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.pieces[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// ---------------------------------------------------------------------------
// Scaling: a one-wave workgroup to a run of a piece, which leaves its CU as soon as its
// own few accesses are done.  Bound by HBM: 1.04 G bf16 elements 660 us, 6.3 TB/s (676 in
// a trace of its two launches; four waves 682; runs of 512 elements 736, of 2048 672, of
// 4096 708); 10.6 M, from the caches in part: 10.2 us, 9.5 with runs of 2048.

template <bool STREAM> constexpr int kRun = STREAM ? 1024 : 2048;  // elements

template <bool STREAM, bool FULL, typename TI, typename TO>
__device__ __forceinline__ void scale_run(const TI* p, TO* q, int64_t left, float scale,
                                          int lane) {
  constexpr int E = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
  constexpr int K = kRun<STREAM> / (64 * E);
  constexpr int IW = E * sizeof(TI) / 4, OW = E * sizeof(TO) / 4;  // words of an access
  uint32_t __attribute__((ext_vector_type(IW))) u[K];
#pragma unroll
  for (int k = 0; k < K; ++k) u[k] = load_whole<STREAM, FULL, IW>(p, 64 * E * k + E * lane, left);
  if constexpr (!FULL) {  // the elements behind the last whole vector, one a lane
    const int behind = static_cast<int>(left - left % E) + lane;
    if (behind < left) put(q + behind, widen(p[behind]) * scale);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int e = 64 * E * k + E * lane;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if constexpr (sizeof(TI) == 2)
        x[i] = __uint_as_float(i & 1 ? u[k][i / 2] & 0xffff0000u : u[k][i / 2] << 16) * scale;
      else
        x[i] = __uint_as_float(u[k][i]) * scale;
    }
    if (!FULL && e + E > left) continue;
    uint32_t __attribute__((ext_vector_type(OW))) o;
#pragma unroll
    for (int i = 0; i < OW; ++i) {
      if constexpr (sizeof(TO) == 2) o[i] = bf16_bits(x[2 * i]) | bf16_bits(x[2 * i + 1]) << 16;
      else o[i] = __float_as_uint(x[i]);
    }
    if constexpr (OW == 4) store16<STREAM>(q + e, o);
    else store8<STREAM>(q + e, o);
  }
}

template <bool STREAM, bool FULL>
__device__ __forceinline__ void scale_run_of(const ClipArgs& a, int tensor, int64_t at,
                                             int64_t left, float scale, int lane) {
  const void* in = a.list.data[tensor];
  void* out = a.out[tensor];
  const uint16_t* hi = static_cast<const uint16_t*>(in) + at;
  const float* fi = static_cast<const float*>(in) + at;
  uint16_t* ho = static_cast<uint16_t*>(out) + at;
  float* fo = static_cast<float*>(out) + at;
  if (a.list.type[tensor] == GRZ_BF16) {
    if (a.out_type[tensor] == GRZ_BF16) scale_run<STREAM, FULL>(hi, ho, left, scale, lane);
    else scale_run<STREAM, FULL>(hi, fo, left, scale, lane);
  } else {
    if (a.out_type[tensor] == GRZ_BF16) scale_run<STREAM, FULL>(fi, ho, left, scale, lane);
    else scale_run<STREAM, FULL>(fi, fo, left, scale, lane);
  }
}

template <bool STREAM>
__global__ __launch_bounds__(64) void tensors_clip_kernel(const ClipArgs a) {
  constexpr uint32_t kRuns = GRZ_PIECE / kRun<STREAM>;
  const int lane = threadIdx.x;
  const float scale = a.scale != nullptr ? *a.scale : 1.0f;
  const Piece p = piece_of(a.list, blockIdx.x / kRuns, lane);
  // A gradient in its place that is scaled by 1 is what it was.
  if (scale == 1.0f && a.list.data[p.tensor] == a.out[p.tensor]) return;
  const int skip = static_cast<int>(blockIdx.x % kRuns) * kRun<STREAM>;
  if (skip >= p.left) return;
  const int64_t at = p.at + skip, left = p.left - skip;
  if (left >= kRun<STREAM>) scale_run_of<STREAM, true>(a, p.tensor, at, left, scale, lane);
  else scale_run_of<STREAM, false>(a, p.tensor, at, left, scale, lane);
}

// ---------------------------------------------------------------------------
// Host side.

int check_tensors(const grz_tensor* t, int64_t count, int64_t* elements, int64_t* bytes) {
  if (count < 0 || (count > 0 && t == nullptr)) return GRZ_EINVAL;
  *elements = *bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].numel < 0 || !float_type(t[i].dtype)) return GRZ_EINVAL;
    if (t[i].numel > kMaxElements - *elements) return GRZ_ERANGE;
    if (t[i].numel > 0 && t[i].data == nullptr) return GRZ_EINVAL;
    if (!aligned(t[i].data, elem_size(t[i].dtype))) return GRZ_EALIGN;
    *elements += t[i].numel;
    *bytes += t[i].numel * static_cast<int64_t>(elem_size(t[i].dtype));
  }
  return GRZ_OK;
}

int64_t pieces_of(int64_t numel) { return ceil_div(numel, GRZ_PIECE); }

int64_t pieces_of(const grz_tensor* t, int64_t count) {
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) n += pieces_of(t[i].numel);
  return n;
}

// The pieces' sums and the levels of the tree over them.
size_t workspace_of(int64_t pieces) {
  return static_cast<size_t>(pieces) * sizeof(double) + dp_grad_sqnorm_workspace(pieces);
}

size_t bytes_of(const grz_tensor& t) { return static_cast<size_t>(t.numel) * elem_size(t.dtype); }

bool clash(const void* p, size_t bytes, const grz_tensor* t, int64_t count) {
  for (int64_t i = 0; i < count; ++i)
    if (overlap(p, bytes, t[i].data, bytes_of(t[i]))) return true;
  return false;
}

// Whether a tensor that is written lies over another one, read or written; only a
// gradient and its own output may be the same memory.
struct Range {
  uintptr_t from, to;
  bool out;
};

int check_apart(const grz_tensor* in, const grz_tensor* out, int64_t count) {
  Range few[64];
  Range* r = few;
  if (2 * count > 64) {
    r = new (std::nothrow) Range[static_cast<size_t>(2 * count)];
    if (r == nullptr) return GRZ_ERANGE;
  }
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (in[i].numel == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(in[i].data);
    const uintptr_t b = reinterpret_cast<uintptr_t>(out[i].data);
    r[n++] = {b, b + bytes_of(out[i]), true};
    if (a != b || in[i].dtype != out[i].dtype) r[n++] = {a, a + bytes_of(in[i]), false};
  }
  auto before = [](const Range& x, const Range& y) { return x.from < y.from; };
  if (!std::is_sorted(r, r + n, before)) std::sort(r, r + n, before);
  uintptr_t any = 0, written = 0;  // ends of the ranges so far
  int st = GRZ_OK;
  for (int64_t i = 0; i < n && st == GRZ_OK; ++i) {
    if (r[i].from < (r[i].out ? any : written)) st = GRZ_EINVAL;
    any = std::max(any, r[i].to);
    if (r[i].out) written = std::max(written, r[i].to);
  }
  if (r != few) delete[] r;
  return st;
}

// Bytes from which the tensors are streamed past the caches: what is much larger than
// the 256 MB behind the L2s is not there any more when it is read again (norm and clip of
// 55 MB: 44.1 us, 45.8 streamed; of 184 MB 114 and 107, then 98 with one-wave runs).
constexpr int64_t kStreamBytes = int64_t{96} << 20;

// Where a list goes on: element `at` (of a piece's beginning) of tensor `i`.
struct Cursor {
  int64_t i, at;
};

// Fills an empty list from there on until it or the launch is full.  `also`(entry,
// tensor, element) adds what else the launch needs.
template <int LISTED, typename F>
Cursor fill(List<LISTED>& l, const grz_tensor* t, Cursor c, int64_t count, F also) {
  l.count = 0;
  l.pieces = 0;
  while (c.i < count && l.count < LISTED && l.pieces < kLaunchPieces) {
    const int64_t left = t[c.i].numel - c.at;
    const int64_t room = (kLaunchPieces - l.pieces) * GRZ_PIECE;
    const int64_t take = left < room ? left : room;
    if (take > 0) {
      l.data[l.count] = static_cast<const char*>(t[c.i].data) + c.at * elem_size(t[c.i].dtype);
      l.numel[l.count] = take;
      l.type[l.count] = static_cast<uint8_t>(t[c.i].dtype);
      also(l.count, c);
      l.first[l.count++] = l.pieces;
      l.pieces += static_cast<uint32_t>(pieces_of(take));
    }
    c = take < left ? Cursor{c.i, c.at + take} : Cursor{c.i + 1, 0};
  }
  return c;
}

}  // namespace

// ---------------------------------------------------------------------------
// C ABI

extern "C" {

int64_t dp_tensor_pieces(const grz_tensor* tensors, int64_t count) {
  int64_t elements, bytes;
  const int st = check_tensors(tensors, count, &elements, &bytes);
  return st != GRZ_OK ? -st : pieces_of(tensors, count);
}

size_t dp_grad_sqnorm_tensors_workspace(const grz_tensor* tensors, int64_t count, int64_t lead) {
  const int64_t n = dp_tensor_pieces(tensors, count);
  if (n < 0 || lead < 0 || lead > kMaxPieces - n) return 0;
  return workspace_of(n + lead);
}

int dp_grad_sqnorm_tensors(const grz_tensor* tensors, int64_t count, double max_norm,
                           int64_t lead, void* workspace, double* sqnorm_out,
                           float* clip_scale_out, hipStream_t stream) {
  int64_t elements, bytes;
  int st = check_tensors(tensors, count, &elements, &bytes);
  if (st != GRZ_OK) return st;
  const int64_t n = pieces_of(tensors, count);
  if (lead < 0) return GRZ_EINVAL;
  if (lead > kMaxPieces - n) return GRZ_ERANGE;
  const size_t need = workspace_of(n + lead);
  if (need > 0 && workspace == nullptr) return GRZ_EINVAL;
  if (sqnorm_out == nullptr && clip_scale_out == nullptr) return GRZ_EINVAL;
  if (!aligned(workspace, 8) || !aligned(sqnorm_out, 8) || !aligned(clip_scale_out, 4))
    return GRZ_EALIGN;
  const size_t sq = sqnorm_out != nullptr ? 8 : 0, sc = clip_scale_out != nullptr ? 4 : 0;
  if (clash(workspace, need, tensors, count) || clash(sqnorm_out, sq, tensors, count) ||
      clash(clip_scale_out, sc, tensors, count) || overlap(workspace, need, sqnorm_out, sq) ||
      overlap(workspace, need, clip_scale_out, sc) || overlap(sqnorm_out, sq, clip_scale_out, sc))
    return GRZ_EINVAL;
  double* const pieces = static_cast<double*>(workspace);
  NormArgs a;
  a.pieces = pieces + lead;
  for (Cursor c{0, 0}; c.i < count;) {
    c = fill(a.list, tensors, c, count, [](int, const Cursor&) {});
    const uint32_t k = a.list.pieces;
    if (k == 0) continue;
    st = k <= kFewPieces
             ? launch(tensors_norm_few_kernel, dim3(k), dim3(256), stream, a)
             : launch(bytes >= kStreamBytes ? tensors_norm_kernel<true>
                                            : tensors_norm_kernel<false>,
                      dim3(static_cast<unsigned>(ceil_div(k, 4))), dim3(256), stream, a);
    if (st != GRZ_OK) return st;
    a.pieces += k;
  }
  return dp_grad_sqnorm(pieces, n + lead, max_norm, pieces + n + lead, sqnorm_out,
                        clip_scale_out, stream);
}

int dp_grad_clip_tensors(const grz_tensor* grads, int64_t count, const float* clip_scale,
                         const grz_tensor* out, hipStream_t stream) {
  int64_t elements, bytes, out_bytes;
  int st = check_tensors(grads, count, &elements, &bytes);
  if (st != GRZ_OK) return st;
  if (!aligned(clip_scale, 4)) return GRZ_EALIGN;
  if (out == nullptr) out = grads;
  if ((st = check_tensors(out, count, &elements, &out_bytes)) != GRZ_OK) return st;
  for (int64_t i = 0; i < count; ++i)
    if (out[i].numel != grads[i].numel) return GRZ_EINVAL;
  if (clip_scale != nullptr && clash(clip_scale, 4, out, count)) return GRZ_EINVAL;
  if ((st = check_apart(grads, out, count)) != GRZ_OK) return st;
  ClipArgs a;
  a.scale = clip_scale;
  const bool stream_past = bytes >= kStreamBytes;
  for (Cursor c{0, 0}; c.i < count;) {
    c = fill(a.list, grads, c, count, [&](int to, const Cursor& from) {
      const grz_tensor& o = out[from.i];
      a.out[to] = static_cast<char*>(o.data) + from.at * elem_size(o.dtype);
      a.out_type[to] = static_cast<uint8_t>(o.dtype);
    });
    const uint32_t k = a.list.pieces;
    if (k == 0) continue;
    const auto grid = [&](int run) { return dim3(k * static_cast<unsigned>(GRZ_PIECE / run)); };
    st = stream_past ? launch(tensors_clip_kernel<true>, grid(kRun<true>), dim3(64), stream, a)
                     : launch(tensors_clip_kernel<false>, grid(kRun<false>), dim3(64), stream, a);
    if (st != GRZ_OK) return st;
  }
  return GRZ_OK;
}

}  // extern "C"
