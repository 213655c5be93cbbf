// Norm of queries and keys per head, with the position rotation in the same
// pass.  Per token and head, for x of D channels at position p,
//     n = x r,  r = (sum x^2 + eps)^-1/2            (L2, as the KDA core)
//               r = (mean x^2 + eps)^-1/2           (KDA_FLAG_RMS_NORM)
//               r = 1                               (KDA_FLAG_NO_QK_NORM)
//     m = n w   (w per channel, shared by the heads, optional)
//     y = m with each of R / 2 channel pairs (i, i + R/2), or (2i, 2i + 1),
//         turned by the angle p f_i; channels from R on stay.
// Backward: dm = dy turned back, dw = sum dm n, dn = dm w,
//     dx = r (dn - n (sum dn n) [/ D]).
//
// The angle is formed in fp64 turns, p (f_i / 2 pi), and reduced to its
// fraction there: at position 2^20 an fp32 angle would be off by 1/16 radian.
//
// A row of D channels is held by D / 8 lanes of a group (of the next power of
// two), 8 channels a lane: of the rotated ones channels 4i .. 4i + 3 and their
// partners, so that a pair never leaves its lane.  A lane does up to HC heads
// of one token with the same 4 sines and cosines.  The work is bound by
// memory: 4 bytes an element forward in bf16, 0.57 ms at 32768 tokens x 192 heads
// of 128 (5.6 TB/s; fp32 1.15 ms, the same rate), and 6 backward, 53 us at 8194
// tokens x 40 heads (4.7 TB/s; 95 us with the waiting rows held as fp32, which
// left three waves a SIMD).  In fp32 four waves a SIMD leave the backward too few
// registers: the compiler spills 43, and it takes 147 us there (3.4 TB/s) and
// 1.10 ms at 16384 tokens x 192 heads (4.4 TB/s).

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_token.h"

namespace kda {
namespace {

constexpr int QT = 256;  // threads
constexpr double INV_2PI = 0.15915494309189533577;

struct QkArgs {
  const void* q;
  const void* k;
  const void* dq_out;
  const void* dk_out;
  void* q_out;  // or dq, dk
  void* k_out;
  const float* qw;
  const float* kw;
  const int32_t* pos;
  const double* freq;
  float* part;  // [blocks][2][D] sums for the weight gradients
  float* dqw;
  float* dkw;
  int64_t qs, qh, ks, kh;      // token and head strides of q and k, in elements
  int64_t qos, qoh, kos, koh;  // of q_out and k_out
  int64_t tokens;
  int Hq, Hk, D, R;
  int lanes;      // of a group
  int chunks;     // head chunks of HC of a token
  int64_t items;  // tokens * chunks
  float eps, inv_count;  // inv_count: 1 / D with the root mean square, else 1
  int norm, interleaved;
};

// Channels of a lane: [c0, c0 + 4) and [c1, c1 + 4); `turned` if they rotate.
struct Place {
  int c0, c1;
  bool in, turned;
};
__device__ __forceinline__ Place place(const QkArgs& a, int slot) {
  Place p;
  p.in = slot < a.D / 8;
  p.turned = slot < a.R / 8;
  if (p.turned && !a.interleaved) {
    p.c0 = 4 * slot;
    p.c1 = a.R / 2 + 4 * slot;
  } else {
    p.c0 = 8 * slot;
    p.c1 = p.c0 + 4;
  }
  return p;
}

// A lane's 8 channels of a row, as loaded: rows that wait for their turn take
// half the registers in bf16.
template <typename T>
__device__ __forceinline__ void load_row(const T* row, const Place& p, RawN<T, 8>& r) {
  r.v[0] = *reinterpret_cast<const raw4<T>*>(row + p.c0);
  r.v[1] = *reinterpret_cast<const raw4<T>*>(row + p.c1);
}
template <typename T>
__device__ __forceinline__ void store_row(T* row, const Place& p, const float (&v)[8]) {
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  store4(row + p.c0, a);
  store4(row + p.c1, b);
}

// Sine and cosine of `turn` turns, |turn| < 1: the hardware's for bf16 (their
// error is a few 2^-20, under the rounding), the library's for fp32.
template <typename T>
__device__ __forceinline__ void sin_cos(float turn, float& s, float& c) {
  if constexpr (sizeof(T) == 2) {
    s = __builtin_amdgcn_sinf(turn);
    c = __builtin_amdgcn_cosf(turn);
  } else {
    sincospif(2.0f * turn, &s, &c);
  }
}

// The lane's 4 sines and cosines at a position.
template <typename T>
__device__ __forceinline__ void angles(const double (&f)[4], int32_t pos, float (&s)[4], float (&c)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double t = (double)pos * f[j];
    sin_cos<T>((float)(t - __builtin_rint(t)), s[j], c[j]);
  }
}

// Turn the lane's pairs by its angles (sign -1: back).
__device__ __forceinline__ void turn(float (&v)[8], const float (&s)[4], const float (&c)[4], bool interleaved,
                                     float sign) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int x = interleaved ? 2 * j : j, y = interleaved ? 2 * j + 1 : j + 4;
    const float p = v[x], q = v[y], t = sign * s[j];
    v[x] = p * c[j] - q * t;
    v[y] = q * c[j] + p * t;
  }
}

__device__ __forceinline__ float group_sum(float s, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) s += __shfl_xor(s, m);
  return s;
}

__device__ __forceinline__ void load_weight(const float* w, const Place& p, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 1.f;
  if (w && p.in) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = w[p.c0 + j];
      v[4 + j] = w[p.c1 + j];
    }
  }
}

template <typename T, int HC, bool INTER>
__global__ void __launch_bounds__(QT) kda_qk_fwd_kernel(QkArgs a) {
  const int slot = threadIdx.x & (a.lanes - 1), per = QT / a.lanes;
  const Place p = place(a, slot);
  const int64_t item = (int64_t)blockIdx.x * per + threadIdx.x / a.lanes;
  if (item >= a.items) return;  // whole groups leave; sums stay within a group
  const int64_t t = item / a.chunks;
  const int h0 = (int)(item % a.chunks) * HC, H = a.Hq + a.Hk;
  RawN<T, 8> raw[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int h = h0 + i;
    zero_raw(raw[i]);
    if (p.in && h < H) {
      const T* row = h < a.Hq ? static_cast<const T*>(a.q) + t * a.qs + h * a.qh
                              : static_cast<const T*>(a.k) + t * a.ks + (h - a.Hq) * a.kh;
      load_row(row, p, raw[i]);
    }
  }
  float s[4], c[4];
  if (p.turned) {
    double f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = a.freq[4 * slot + j] * INV_2PI;
    angles<T>(f, a.pos[t], s, c);
  }
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int h = h0 + i;
    if (h >= H) break;
    float v[8], r = 1.0f;
    widen(raw[i], v);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
      r = __builtin_amdgcn_rsqf(group_sum(ss, a.lanes) * a.inv_count + a.eps);
    }
    const float* wp = h < a.Hq ? a.qw : a.kw;
    float w[8];
    load_weight(wp, p, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
    if (p.turned) turn(v, s, c, INTER, 1.0f);
    if (p.in) {
      T* row = h < a.Hq ? static_cast<T*>(a.q_out) + t * a.qos + h * a.qoh
                        : static_cast<T*>(a.k_out) + t * a.kos + (h - a.Hq) * a.koh;
      store_row(row, p, v);
    }
  }
}

// A persistent grid, so that the weights' sums stay in registers: every thread
// strides over items with the same slot.
template <typename T, int HC, bool INTER>
__global__ void __launch_bounds__(QT, 4) kda_qk_bwd_kernel(QkArgs a) {
  __shared__ float sm[QT][8];
  const int slot = threadIdx.x & (a.lanes - 1), per = QT / a.lanes;
  const Place p = place(a, slot);
  const int H = a.Hq + a.Hk;
  double f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = p.turned ? a.freq[4 * slot + j] * INV_2PI : 0.0;
  float sq[8], sk[8], qw[8], kw[8];
  load_weight(a.qw, p, qw);
  load_weight(a.kw, p, kw);
#pragma unroll
  for (int j = 0; j < 8; ++j) sq[j] = sk[j] = 0.f;
  for (int64_t item = (int64_t)blockIdx.x * per + threadIdx.x / a.lanes; item < a.items;
       item += (int64_t)gridDim.x * per) {
    const int64_t t = item / a.chunks;
    const int h0 = (int)(item % a.chunks) * HC;
    RawN<T, 8> vr[HC], dr[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const int h = h0 + i;
      zero_raw(vr[i]);
      zero_raw(dr[i]);
      if (p.in && h < H) {
        const bool isq = h < a.Hq;
        load_row(isq ? static_cast<const T*>(a.q) + t * a.qs + h * a.qh
                     : static_cast<const T*>(a.k) + t * a.ks + (h - a.Hq) * a.kh, p, vr[i]);
        load_row(isq ? static_cast<const T*>(a.dq_out) + (t * a.Hq + h) * a.D
                     : static_cast<const T*>(a.dk_out) + (t * a.Hk + h - a.Hq) * a.D, p, dr[i]);
      }
    }
    float s[4], c[4];
    if (p.turned) angles<T>(f, a.pos[t], s, c);
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const int h = h0 + i;
      if (h >= H) break;
      const bool isq = h < a.Hq;
      float v[8], d[8];
      widen(vr[i], v);
      widen(dr[i], d);
      if (p.turned) turn(d, s, c, INTER, -1.0f);
      float r = 1.0f;
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
        r = __builtin_amdgcn_rsqf(group_sum(ss, a.lanes) * a.inv_count + a.eps);
      }
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= r;  // n
        if (isq) sq[j] += d[j] * v[j];
        else sk[j] += d[j] * v[j];
        d[j] *= isq ? qw[j] : kw[j];
        dot += d[j] * v[j];
      }
      if (a.norm) {
        dot = group_sum(dot, a.lanes) * a.inv_count;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = r * (d[j] - v[j] * dot);
      }
      if (p.in)
        store_row(isq ? static_cast<T*>(a.q_out) + (t * a.Hq + h) * a.D
                      : static_cast<T*>(a.k_out) + (t * a.Hk + h - a.Hq) * a.D, p, d);
    }
  }
  if (!a.part) return;
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sm[threadIdx.x][j] = which ? sk[j] : sq[j];
    __syncthreads();
    if (threadIdx.x < a.lanes && p.in) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x = 0.f;
        for (int g = 0; g < per; ++g) x += sm[g * a.lanes + slot][j];
        a.part[((int64_t)blockIdx.x * 2 + which) * a.D + (j < 4 ? p.c0 + j : p.c1 + j - 4)] = x;
      }
    }
  }
}

// The weights' gradients from the workgroups' sums, in a fixed order and in
// fp64: a workgroup has 16 channels by 64 rows at a time.
constexpr int QRED = 1024, RC = 16, RR = QRED / RC;
__global__ void __launch_bounds__(QRED) kda_qk_reduce_kernel(QkArgs a, int blocks) {
  __shared__ double sm[RR][RC];
  const int ch = threadIdx.x % RC, row = threadIdx.x / RC, which = blockIdx.x & 1;
  const int c = (blockIdx.x >> 1) * RC + ch;
  float* to = which ? a.dkw : a.dqw;
  if (!to) return;
  double s = 0.0;
  if (c < a.D) {
    constexpr int U = 8;  // rows asked for at once
    for (int b0 = row; b0 < blocks; b0 += U * RR) {
      float p[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = b0 + u * RR < blocks ? a.part[((int64_t)(b0 + u * RR) * 2 + which) * a.D + c] : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) s += p[u];
    }
  }
  sm[row][ch] = s;
  for (int r = RR / 2; r >= 1; r >>= 1) {
    __syncthreads();
    if (row < r) sm[row][ch] += sm[row + r][ch];
  }
  if (row == 0 && c < a.D) to[c] = (float)sm[0][ch];
}

constexpr int HC = 4;
constexpr int64_t kQkBlocks = 1024;  // of the backward's grid: four workgroups a CU

bool strides_ok(int64_t tokens, int64_t H, int64_t D, int64_t ts, int64_t hs) {
  return ts >= 0 && hs >= 0 && ts % 4 == 0 && hs % 4 == 0 && fits(tokens, ts, kMaxElements) && fits(H, hs, kMaxElements) &&
         (H <= 1 || hs >= D) && (tokens <= 1 || ts >= D);
}

// Whether no two rows of D elements share any: heads within a token's span, or
// tokens within a head's.
bool rows_apart(int64_t tokens, int64_t H, int64_t D, int64_t ts, int64_t hs) {
  return H == 0 || tokens <= 1 || ts >= (H - 1) * hs + D || (H > 1 && hs >= (tokens - 1) * ts + D);
}

kda_status_t qk_prepare(QkArgs& a, const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
                        int64_t k_stride, int64_t k_head_stride, const float* q_weight, const float* k_weight,
                        const int32_t* positions, const double* inv_freq, float eps, int64_t tokens, int64_t Hq,
                        int64_t Hk, int64_t D, int64_t R, int dtype, unsigned flags) {
  if (tokens < 0 || Hq < 0 || Hk < 0 || Hq + Hk < 1 || D < 1 || R < 0) return KDA_ERR_INVALID;
  if (flags & ~(unsigned)(FLAG_NO_QK_NORM | FLAG_RMS_NORM | FLAG_INTERLEAVED)) return KDA_ERR_INVALID;
  if ((flags & FLAG_NO_QK_NORM) && (flags & FLAG_RMS_NORM)) return KDA_ERR_INVALID;
  if (!(eps >= 0.0f) || R > D) return KDA_ERR_INVALID;
  if (!dtype_bytes(dtype) || D % 8 != 0 || D > 512 || R % 8 != 0) return KDA_ERR_UNSUPPORTED;
  if (Hq > 1 << 20 || Hk > 1 << 20 || !fits(tokens, (Hq + Hk) * D, kMaxElements)) return KDA_ERR_INVALID;
  if (tokens > 0 && ((Hq && !q) || (Hk && !k))) return KDA_ERR_INVALID;
  if (R > 0 && (!inv_freq || (tokens > 0 && !positions))) return KDA_ERR_INVALID;
  if (!strides_ok(tokens, Hq, D, q_stride, q_head_stride) || !strides_ok(tokens, Hk, D, k_stride, k_head_stride))
    return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {q, k})) return KDA_ERR_INVALID;
  a = QkArgs{};
  a.q = q;
  a.k = k;
  a.qs = q_stride;
  a.qh = q_head_stride;
  a.ks = k_stride;
  a.kh = k_head_stride;
  a.qw = q_weight;
  a.kw = k_weight;
  a.pos = positions;
  a.freq = inv_freq;
  a.tokens = tokens;
  a.Hq = (int)Hq;
  a.Hk = (int)Hk;
  a.D = (int)D;
  a.R = (int)R;
  a.lanes = 1;
  while (a.lanes < D / 8) a.lanes *= 2;
  a.chunks = (int)((Hq + Hk + HC - 1) / HC);
  a.items = tokens * a.chunks;
  a.eps = eps;
  a.norm = flags & FLAG_NO_QK_NORM ? 0 : 1;
  a.inv_count = flags & FLAG_RMS_NORM ? 1.0f / (float)D : 1.0f;
  a.interleaved = flags & FLAG_INTERLEAVED ? 1 : 0;
  const int64_t per = QT / a.lanes;
  if ((a.items + per - 1) / per > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  return KDA_SUCCESS;
}

template <typename T, bool INTER>
kda_status_t run_fwd(const QkArgs& a, hipStream_t st) {
  const int64_t per = QT / a.lanes;
  return launch(&kda_qk_fwd_kernel<T, HC, INTER>, (a.items + per - 1) / per, QT, st, "qk forward", a);
}

int64_t bwd_blocks(int64_t items, int64_t per) {
  const int64_t b = (items + per - 1) / per;
  return b < 1 ? 1 : b < kQkBlocks ? b : kQkBlocks;
}

template <typename T, bool INTER>
kda_status_t run_bwd(const QkArgs& a, int64_t blocks, hipStream_t st) {
  const kda_status_t s = launch(&kda_qk_bwd_kernel<T, HC, INTER>, blocks, QT, st, "qk backward", a);
  if (s != KDA_SUCCESS || !a.part) return s;
  return launch(&kda_qk_reduce_kernel, (int64_t)(a.D + RC - 1) / RC * 2, QRED, st, "qk reduce", a, (int)blocks);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_qk_rope_fwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                             int64_t k_head_stride, void* q_out, void* k_out, const float* q_weight,
                             const float* k_weight, const int32_t* positions, const double* inv_freq, float eps,
                             int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int dtype, unsigned flags,
                             void* stream) {
  QkArgs a;
  const kda_status_t s = qk_prepare(a, q, q_stride, q_head_stride, k, k_stride, k_head_stride, q_weight, k_weight,
                                    positions, inv_freq, eps, tokens, Hq, Hk, D, R, dtype, flags);
  if (s != KDA_SUCCESS) return s;
  if (tokens > 0 && ((Hq && !q_out) || (Hk && !k_out))) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {q_out, k_out})) return KDA_ERR_INVALID;
  if (tokens == 0) return KDA_SUCCESS;
  a.q_out = q_out;
  a.k_out = k_out;
  const bool qin = q_out == q, kin = k_out == k;  // in place: the input's strides
  if ((qin && !rows_apart(tokens, Hq, D, q_stride, q_head_stride)) ||
      (kin && !rows_apart(tokens, Hk, D, k_stride, k_head_stride)))
    return KDA_ERR_INVALID;
  a.qos = qin ? a.qs : Hq * D;
  a.qoh = qin ? a.qh : D;
  a.kos = kin ? a.ks : Hk * D;
  a.koh = kin ? a.kh : D;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == KDA_DTYPE_BF16) return a.interleaved ? run_fwd<__bf16, true>(a, st) : run_fwd<__bf16, false>(a, st);
  return a.interleaved ? run_fwd<float, true>(a, st) : run_fwd<float, false>(a, st);
}

size_t kda_qk_rope_bwd_workspace_size(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D) {
  if (tokens < 0 || Hq < 0 || Hk < 0 || Hq + Hk < 1 || D < 8 || D % 8 != 0 || D > 512 || Hq > 1 << 20 ||
      Hk > 1 << 20 || !fits(tokens, (Hq + Hk) * D, kMaxElements))
    return 0;
  return 256 + align256((size_t)kQkBlocks * 2 * (size_t)D * sizeof(float));
}

kda_status_t kda_qk_rope_bwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                             int64_t k_head_stride, const void* d_q_out, const void* d_k_out, void* dq, void* dk,
                             float* d_q_weight, float* d_k_weight, void* workspace, size_t workspace_bytes,
                             const float* q_weight, const float* k_weight, const int32_t* positions,
                             const double* inv_freq, float eps, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
                             int64_t R, int dtype, unsigned flags, void* stream) {
  QkArgs a;
  const kda_status_t s = qk_prepare(a, q, q_stride, q_head_stride, k, k_stride, k_head_stride, q_weight, k_weight,
                                    positions, inv_freq, eps, tokens, Hq, Hk, D, R, dtype, flags);
  if (s != KDA_SUCCESS) return s;
  if (tokens > 0 && ((Hq && (!d_q_out || !dq)) || (Hk && (!d_k_out || !dk)))) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {d_q_out, d_k_out, dq, dk}) || !aligned(workspace, 16))
    return KDA_ERR_INVALID;
  const bool sums = d_q_weight || d_k_weight;
  if (sums && (!workspace || workspace_bytes < kda_qk_rope_bwd_workspace_size(tokens, Hq, Hk, D)))
    return KDA_ERR_WORKSPACE;
  if (tokens == 0 && !sums) return KDA_SUCCESS;
  a.dq_out = d_q_out;
  a.dk_out = d_k_out;
  a.q_out = dq;
  a.k_out = dk;
  a.dqw = d_q_weight;
  a.dkw = d_k_weight;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t blocks = bwd_blocks(a.items, QT / a.lanes);
  if (dtype == KDA_DTYPE_BF16)
    return a.interleaved ? run_bwd<__bf16, true>(a, blocks, st) : run_bwd<__bf16, false>(a, blocks, st);
  return a.interleaved ? run_bwd<float, true>(a, blocks, st) : run_bwd<float, false>(a, blocks, st);
}

}  // extern "C"
