// Shared pieces of the per-token operators around the KDA core (gated linear
// recurrence, short convolution, q/k norm and rotation): typed vector loads
// and stores, and the packed token axis with its sequence boundaries.
// Internal header: not part of the C ABI.
#pragma once

#include <initializer_list>

#include "../../include/kda.h"
#include "kda_common.h"

namespace kda {

// Variant bits of these operators (same values as the KDA_FLAG_* constants).
constexpr unsigned FLAG_COMPLEMENT = 128;   // recurrence input scaled by 1 - a
constexpr unsigned FLAG_SILU = 256;         // convolution followed by z sigmoid(z)
constexpr unsigned FLAG_RMS_NORM = 512;     // q, k divided by their root mean square
constexpr unsigned FLAG_INTERLEAVED = 1024; // rotated pairs are channels 2i, 2i + 1
constexpr unsigned FLAG_ZERO_REST = 2048;   // rows behind the last sequence become zeros

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Token arrays are bf16 or fp32; arithmetic is fp32 in both, and a store
// rounds once, to nearest even.
template <typename T>
struct TypeOf;
template <>
struct TypeOf<__bf16> {
  typedef uint2 raw4;  // 4 elements as loaded
};
template <>
struct TypeOf<float> {
  typedef float4 raw4;
};
template <typename T>
using raw4 = typename TypeOf<T>::raw4;

__device__ __forceinline__ void widen4(const uint2 r, float (&d)[4]) {
  d[0] = __uint_as_float(r.x << 16);
  d[1] = __uint_as_float(r.x & 0xffff0000u);
  d[2] = __uint_as_float(r.y << 16);
  d[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void widen4(const float4 r, float (&d)[4]) {
  d[0] = r.x;
  d[1] = r.y;
  d[2] = r.z;
  d[3] = r.w;
}
// N (4 or 8) consecutive elements as loaded; 8 are two vectors of 4, each
// aligned to its own size.
template <typename T, int N>
struct RawN {
  raw4<T> v[N / 4];
};
template <typename T, int N>
__device__ __forceinline__ void load_raw(const T* p, RawN<T, N>& r) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) r.v[i] = reinterpret_cast<const raw4<T>*>(p)[i];
}
template <typename T, int N>
__device__ __forceinline__ void zero_raw(RawN<T, N>& r);
template <typename T, int N>
__device__ __forceinline__ void widen(const RawN<T, N>& r, float (&d)[N]);

__device__ __forceinline__ void load_f4(const float* p, float (&d)[4]) { widen4(*reinterpret_cast<const float4*>(p), d); }
__device__ __forceinline__ void store4(float* p, const float (&d)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ void store4(__bf16* p, const float (&d)[4]) {
  bf16x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (__bf16)d[i];
  *reinterpret_cast<bf16x4*>(p) = v;
}
__device__ __forceinline__ void zero4(uint2& r) { r = make_uint2(0, 0); }
__device__ __forceinline__ void zero4(float4& r) { r = make_float4(0.f, 0.f, 0.f, 0.f); }

template <typename T, int N>
__device__ __forceinline__ void zero_raw(RawN<T, N>& r) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) zero4(r.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void widen(const RawN<T, N>& r, float (&d)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float f[4];
    widen4(r.v[i], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[4 * i + j] = f[j];
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&d)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = d[4 * i + j];
    store4(p + 4 * i, f);
  }
}

template <typename T>
__device__ __forceinline__ void store_zero4(T* p) {
  const float z[4] = {0.f, 0.f, 0.f, 0.f};
  store4(p, z);
}

// The packed token axis of a call: rows 0 .. total - 1, cut into N sequences,
// by cu (int32 offsets [N + 1]) or into N of T rows each.  Rows behind the
// last sequence (cu[N] <= row < total) belong to none.
struct Axis {
  const int32_t* cu;
  int64_t T;
  int64_t total;
  int N;
  double per_row;  // 1 / T (0 for T == 0)
};
inline Axis make_axis(const int32_t* cu, int64_t T, int64_t total, int64_t N) {
  return Axis{cu, T, total, (int)N, T > 0 ? 1.0 / (double)T : 0.0};
}
// t / T for 0 <= t <= total (cu NULL): from the quotient in fp64, which is off
// by one at most, instead of a 64-bit integer division.
__device__ __forceinline__ int64_t axis_div(const Axis& ax, int64_t t) {
  int64_t n = (int64_t)((double)t * ax.per_row);
  n -= n * ax.T > t;
  n += (n + 1) * ax.T <= t;
  return n;
}
// Rows that belong to sequences.  Held to the array, the first offset to 0 and
// every other to 0 or more, so that offsets that break the contract cannot lead
// outside the arrays.
__device__ __forceinline__ int64_t axis_rows(const Axis& ax) {
  if (!ax.cu) return ax.total;
  const int64_t r = ax.cu[ax.N];
  return r < 0 ? 0 : r < ax.total ? r : ax.total;
}
__device__ __forceinline__ int64_t axis_start(const Axis& ax, int64_t n) {
  if (!ax.cu) return n * ax.T;
  const int32_t s = n > 0 ? ax.cu[n] : 0;
  return s > 0 ? s : 0;
}

// Smallest n in [0, N] with start(n) >= t (N + 1 if there is none), found by a
// whole wave: 64 candidates a step.
__device__ __forceinline__ int64_t axis_lower(const Axis& ax, int64_t t) {
  if (!ax.cu) {
    if (t <= 0) return 0;
    if (ax.T == 0) return (int64_t)ax.N + 1;
    const int64_t n = axis_div(ax, t - 1) + 1;
    return n <= ax.N ? n : (int64_t)ax.N + 1;
  }
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = (int64_t)ax.N + 1;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t i = lo + lane * step;
    const bool below = i < hi && (int64_t)ax.cu[i] < t;
    const int c = __popcll(__ballot(below));  // the candidates are sorted: a prefix of the lanes
    if (c == 0) return lo;
    const int64_t top = lo + c * step;  // first candidate that is not below, or past the range
    lo += (c - 1) * step + 1;
    hi = top < hi ? top : hi;
  }
  return lo;
}

// The sequence that row t (< axis_rows) belongs to: the largest n with
// start(n) <= t, which is not empty.  Any lane, any t.
__device__ __forceinline__ int axis_owner(const Axis& ax, int64_t t) {
  if (!ax.cu) return (int)axis_div(ax, t);
  int lo = 0, hi = ax.N - 1;
  while (lo < hi) {
    const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
    if ((int64_t)ax.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Overflow-free size checks on the host: a * b <= limit for a, b >= 0.
inline bool fits(int64_t a, int64_t b, int64_t limit) { return a == 0 || b <= limit / a; }

// Whether p is a multiple of `bytes` (NULL is).
inline bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

inline bool aligned_all(size_t bytes, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, bytes)) return false;
  return true;
}

// Whether two arrays that were given are the same one: an output that another
// workgroup's reads would still need as an input.
inline bool same(const void* a, const void* b) { return a && a == b; }

// Bytes that an element of a token array has, 0 for a type that is none.
inline size_t dtype_bytes(int dtype) { return dtype == 0 ? 2 : dtype == 1 ? 4 : 0; }

constexpr int64_t kMaxElements = (int64_t)1 << 46;  // of one token array; byte offsets stay in int64

// Workgroups that a launch can have: HIP takes fewer than 2^32 threads in a dimension of the grid.
inline int64_t most_groups(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

kda_status_t launch_status(hipError_t err, const char* what);

template <typename... P>
inline kda_status_t launch(void (*fn)(P...), int64_t grid, int threads, hipStream_t st, const char* what, P... p) {
  if (grid > most_groups(threads)) return KDA_ERR_INVALID;  // an entry point of several launches checks all of them first
  void* args[] = {(void*)&p...};
  return launch_status(
      hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)grid), dim3(threads), args, 0, st), what);
}

}  // namespace kda
