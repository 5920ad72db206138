// rows.h -- what the operators on row matrices share (tokens.hip, experts.hip,
// tensors.hip): launches, checks of matrices and ids, vector accesses of bf16 and
// fp32 elements, reductions of a wave.  Included once by each of them; everything
// is local to the file that includes it.
#ifndef GRZ_ROWS_H
#define GRZ_ROWS_H

#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include "grz.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same at any bf16 element's address (gfx950 takes them there).
typedef uint32_t u32x4e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2e __attribute__((ext_vector_type(2), aligned(2)));

constexpr int64_t kMaxRows = INT32_MAX;  // rows and columns of one call

template <typename T> struct NoDeduce { using type = T; };

// Returns the status of this launch alone (hipLaunchKernel's return value).  A
// dispatch counts its threads in 32 bits; the entry points' limits and batches
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

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool float_type(int dtype) { return dtype == GRZ_F32 || dtype == GRZ_BF16; }
inline size_t elem_size(int dtype) { return dtype == GRZ_F32 ? 4 : 2; }

// A row matrix as the entry points take it: `rows` x `cols` values of `dtype`,
// row r at data + r * stride elements.
inline int check_matrix(const void* data, int dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (!float_type(dtype) || rows < 0 || cols < 0) return GRZ_EINVAL;
  if (rows > kMaxRows || cols > kMaxRows) return GRZ_ERANGE;
  if (stride < cols) return GRZ_EINVAL;
  if (stride > (INT64_MAX >> 4) / (rows > 0 ? rows : 1)) return GRZ_ERANGE;
  if (rows == 0 || cols == 0) return GRZ_OK;
  if (data == nullptr) return GRZ_EINVAL;
  return aligned(data, elem_size(dtype)) ? GRZ_OK : GRZ_EALIGN;
}

// Bytes from the first element of a row matrix to behind its last one.
inline size_t span_of(int dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (rows == 0 || cols == 0) return 0;
  return elem_size(dtype) * static_cast<size_t>((rows - 1) * stride + cols);
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

inline int check_ids(const void* ids, int id_bits, int64_t n) {
  if ((id_bits != 32 && id_bits != 64) || n < 0) return GRZ_EINVAL;
  if (n > kMaxRows) return GRZ_ERANGE;
  if (n == 0) return GRZ_OK;
  if (ids == nullptr) return GRZ_EINVAL;
  return aligned(ids, id_bits / 8) ? GRZ_OK : GRZ_EALIGN;
}

// Whether rows allow accesses of `vec` columns (up to 16 bytes each).
template <typename T>
bool vec_ok(const void* p, int64_t dim, int64_t stride, int vec) {
  return dim % vec == 0 && stride % vec == 0 &&
         aligned(p, sizeof(T) * vec < 16 ? sizeof(T) * vec : 16);
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
}  // namespace

#endif  // GRZ_ROWS_H
