// Short causal depthwise convolution: the layer in front of q, k and v,
//     z_t = bias + sum_j w_j x_{t - (W - 1) + j},   y_t = z_t or z_t sigmoid(z_t),
// per channel of [tokens][C], W = 2, 3 or 4 taps.  Rows before a sequence's
// first are its carried state [W - 1][C], the last W - 1 inputs so far, or
// zero.  A thread keeps the last W - 1 rows of its channels in registers and
// walks down a tile of rows, so every row is read once, but for the W - 1 rows
// before a tile.
//
// Backward, with dz_t = dy_t act'(z_t) and z_t computed again:
//     dx_s = sum_j w_j dz_{s + (W - 1) - j},  dw_j = sum_t dz_t x_{t - (W - 1) + j}
// the same walk, W - 1 rows past the tile: W - 1 open sums of dx ride along,
// and the one that row t completes is written.  The rows of the carried state
// get what the first W - 1 rows hand them.  dw and dbias are summed per thread,
// then over tiles in a fixed order.
//
// All arithmetic is fp32.  The forward is bound by memory, 4 bytes an element in
// bf16: 0.31 ms at 32768 rows x 12288 channels, 5.2 TB/s, a plain copy's rate
// (fp32 0.62 ms, the same rate).  The backward's 6 bytes an element come with 31
// operations and two transcendentals: 0.41 ms at 69141 x 4096, 4.1 TB/s (fp32
// 0.92 ms, 3.7 TB/s).

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_token.h"

namespace kda {
namespace {

constexpr int CT = 256;  // threads

struct ConvArgs {
  const void* x;
  const void* dy;
  void* y;  // or dx
  const float* w;
  const float* bias;
  const void* init;
  const void* d_final;
  void* fin;
  void* d_init;
  float* part;  // [tiles][W + 1][C]: sums over the tile for dw and dbias
  float* dw;
  float* dbias;
  Axis ax;
  int64_t C, xs;  // channels, elements between rows of x
  int64_t groups; // channel groups of a thread
  int64_t ntiles;
  int rows;       // rows of a tile
  int silu;
  int zero_rest;  // rows behind the last sequence: zeros (else left as they were)
};

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + fexp2(z * -LOG2E));
}

// The state rows before a sequence's first row: state[n][W - 1][C], or zeros.
template <typename T, int W, int V>
__device__ __forceinline__ void load_state(const void* init, int64_t n, int64_t C, int64_t c, float (&win)[W - 1][V]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    RawN<T, V> r;
    zero_raw(r);
    if (init) load_raw(static_cast<const T*>(init) + (n * (W - 1) + j) * C + c, r);
    widen(r, win[j]);
  }
}

// The W - 1 rows before row t of sequence n, which starts at row s.
template <typename T, int W, int V>
__device__ __forceinline__ void load_window(const ConvArgs& a, int64_t n, int64_t s, int64_t t, int64_t c,
                                            float (&win)[W - 1][V]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t r = t - (W - 1) + j;
    RawN<T, V> v;
    zero_raw(v);
    if (r >= s) load_raw(static_cast<const T*>(a.x) + r * a.xs + c, v);
    else if (a.init) load_raw(static_cast<const T*>(a.init) + (n * (W - 1) + r - s + W - 1) * a.C + c, v);
    widen(v, win[j]);
  }
}

template <typename T, int W, int V>
struct Taps {
  float w[W][V], b[V];
  __device__ __forceinline__ void load(const ConvArgs& a, int64_t c) {
    float f[V * W];  // the taps of neighbouring channels are neighbours
#pragma unroll
    for (int i = 0; i < V * W; i += 4) {
      float v[4];
      load_f4(a.w + c * W + i, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[i + j] = v[j];
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      b[k] = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][k] = f[k * W + j];
    }
    if (a.bias) {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        float v[4];
        load_f4(a.bias + c + k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[k + j] = v[j];
      }
    }
  }
  __device__ __forceinline__ float z(const float (&win)[W - 1][V], float x, int k) const {
    float s = b[k];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s += w[j][k] * win[j][k];
    return s + w[W - 1][k] * x;
  }
};

template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W - 1][V], const float (&x)[V]) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) win[j][k] = win[j + 1][k];
#pragma unroll
  for (int k = 0; k < V; ++k) win[W - 2][k] = x[k];
}

// Rows of the tile behind the last sequence.
template <typename T, int V>
__device__ __forceinline__ void zero_rest(const ConvArgs& a, int64_t t0, int64_t rows, int64_t c) {
  if (!a.zero_rest) return;
  for (int64_t t = t0 > rows ? t0 : rows; t < t0 + a.rows && t < a.ax.total; ++t)
#pragma unroll
    for (int k = 0; k < V; k += 4) store_zero4(static_cast<T*>(a.y) + t * a.C + c + k);
}

// Empty sequences hand their state, or its gradient, on.
template <typename T>
__device__ __forceinline__ void copy_empty(const Axis& ax, const void* from, void* to, int64_t n_elem) {
  if (!to) return;
  for (int64_t n = blockIdx.x; n < ax.N; n += gridDim.x) {
    if (axis_start(ax, n + 1) > axis_start(ax, n)) continue;
    for (int64_t i = threadIdx.x; i < n_elem; i += blockDim.x)
      static_cast<T*>(to)[n * n_elem + i] = from ? static_cast<const T*>(from)[n * n_elem + i] : (T)0.f;
  }
}

template <typename T>
constexpr int FV = sizeof(T) == 2 ? 8 : 4;  // channels of a forward thread: 16 bytes of a row
constexpr int CU = 8;  // rows loaded at once
template <typename T, int W>
__global__ void __launch_bounds__(CT) kda_conv_fwd_kernel(ConvArgs a) {
  constexpr int CV = FV<T>;
  const int64_t rows = axis_rows(a.ax);
  const int64_t item = (int64_t)blockIdx.x * CT + threadIdx.x;
  const int64_t tile = item / a.groups, c = (item % a.groups) * CV;
  const int64_t t0 = tile * a.rows;
  if (tile < a.ntiles && t0 < rows) {
    const int64_t t1 = t0 + a.rows < rows ? t0 + a.rows : rows;
    Taps<T, W, CV> taps;
    taps.load(a, c);
    int64_t n = axis_owner(a.ax, t0), s = axis_start(a.ax, n), e = axis_start(a.ax, n + 1);
    float win[W - 1][CV];
    load_window<T, W, CV>(a, n, s, t0, c, win);
    for (int64_t tb = t0; tb < t1; tb += CU) {
      RawN<T, CV> xr[CU];
#pragma unroll
      for (int i = 0; i < CU; ++i) {
        zero_raw(xr[i]);
        if (tb + i < t1) load_raw(static_cast<const T*>(a.x) + (tb + i) * a.xs + c, xr[i]);
      }
#pragma unroll
      for (int i = 0; i < CU; ++i) {
        const int64_t t = tb + i;
        if (t < t1) {
          if (t == e) {  // the next sequence with rows
            do {
              ++n;
              s = e;
              e = axis_start(a.ax, n + 1);
            } while (e == s && n + 1 < a.ax.N);
            load_state<T, W, CV>(a.init, n, a.C, c, win);
          }
          float xv[CV], y[CV];
          widen(xr[i], xv);
#pragma unroll
          for (int k = 0; k < CV; ++k) {
            const float z = taps.z(win, xv[k], k);
            y[k] = a.silu ? z * sigmoid(z) : z;
          }
          store_n(static_cast<T*>(a.y) + t * a.C + c, y);
          shift<W, CV>(win, xv);
          if (t == e - 1 && a.fin) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
              store_n(static_cast<T*>(a.fin) + (n * (W - 1) + j) * a.C + c, win[j]);
          }
        }
      }
    }
  }
  if (tile < a.ntiles) zero_rest<T, CV>(a, t0, rows, c);
  copy_empty<T>(a.ax, a.init, a.fin, (W - 1) * a.C);
}

// One thread per 16 bytes of channels of a sequence, its T tokens in order; the state
// may be updated in place.
template <typename T, int W>
__global__ void __launch_bounds__(CT) kda_conv_step_kernel(ConvArgs a) {
  constexpr int CV = FV<T>;
  const int64_t item = (int64_t)blockIdx.x * CT + threadIdx.x;
  const int64_t n = item / a.groups, c = (item % a.groups) * CV;
  if (n >= a.ax.N) return;
  Taps<T, W, CV> taps;
  taps.load(a, c);
  float win[W - 1][CV];
  load_state<T, W, CV>(a.init, n, a.C, c, win);
  for (int64_t t = n * a.ax.T; t < (n + 1) * a.ax.T; ++t) {
    RawN<T, CV> xr;
    load_raw(static_cast<const T*>(a.x) + t * a.xs + c, xr);
    float xv[CV], y[CV];
    widen(xr, xv);
#pragma unroll
    for (int k = 0; k < CV; ++k) {
      const float z = taps.z(win, xv[k], k);
      y[k] = a.silu ? z * sigmoid(z) : z;
    }
    store_n(static_cast<T*>(a.y) + t * a.C + c, y);
    shift<W, CV>(win, xv);
  }
  if (a.fin) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_n(static_cast<T*>(a.fin) + (n * (W - 1) + j) * a.C + c, win[j]);
  }
}

constexpr int BV = 4;  // channels of a backward thread: its open sums and partial sums double the registers
constexpr int BU = 8;  // rows loaded at once
template <typename T, int W>
__global__ void __launch_bounds__(CT) kda_conv_bwd_kernel(ConvArgs a) {
  const int64_t rows = axis_rows(a.ax);
  const int64_t item = (int64_t)blockIdx.x * CT + threadIdx.x;
  const int64_t tile = item / a.groups, c = (item % a.groups) * BV;
  const int64_t t0 = tile * a.rows;
  if (tile < a.ntiles) {
    float dw[W + 1][BV];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
      for (int k = 0; k < BV; ++k) dw[j][k] = 0.f;
    if (t0 < rows) {
      const int64_t t1 = t0 + a.rows < rows ? t0 + a.rows : rows;
      Taps<T, W, BV> taps;
      taps.load(a, c);
      int64_t n = axis_owner(a.ax, t0), s = axis_start(a.ax, n), e = axis_start(a.ax, n + 1);
      float win[W - 1][BV], open[W - 1][BV];  // open[i]: dx of row t - 1 - i so far
      load_window<T, W, BV>(a, n, s, t0, c, win);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int k = 0; k < BV; ++k) open[j][k] = 0.f;
      // dx of row r, a row of this tile, or of the state of a sequence that starts in it
      auto emit = [&](int64_t r, const float (&v)[BV]) {
        if (r >= s) {
          if (r >= t0 && r < t1) store_n(static_cast<T*>(a.y) + r * a.C + c, v);
        } else if (a.d_init && s >= t0 && s < t1) {
          store_n(static_cast<T*>(a.d_init) + (n * (W - 1) + r - s + W - 1) * a.C + c, v);
        }
      };
      // The sequence ends before row e: its last rows take d_final.
      auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          RawN<T, BV> r;
          zero_raw(r);
          if (a.d_final) load_raw(static_cast<const T*>(a.d_final) + (n * (W - 1) + W - 2 - i) * a.C + c, r);
          float v[BV];
          widen(r, v);
#pragma unroll
          for (int k = 0; k < BV; ++k) v[k] += open[i][k];
          emit(e - 1 - i, v);
        }
      };
      const int64_t te = t1 + W - 1 < rows ? t1 + W - 1 : rows;
      // row t: its dz into dw and dbias (`own` rows), into the open sums, and
      // the sum that it completes into v
      auto step = [&](const RawN<T, BV>& xw, const RawN<T, BV>& dyw, bool own, float (&v)[BV]) {
        float xv[BV], dv[BV], dz[BV];
        widen(xw, xv);
        widen(dyw, dv);
#pragma unroll
        for (int k = 0; k < BV; ++k) {
          dz[k] = dv[k];
          if (a.silu) {
            const float z = taps.z(win, xv[k], k), sg = sigmoid(z);
            dz[k] *= sg * (1.0f + z * (1.0f - sg));
          }
        }
        if (own) {
#pragma unroll
          for (int k = 0; k < BV; ++k) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][k] += dz[k] * win[j][k];
            dw[W - 1][k] += dz[k] * xv[k];
            dw[W][k] += dz[k];
          }
        }
#pragma unroll
        for (int k = 0; k < BV; ++k) {
          v[k] = open[W - 2][k] + taps.w[0][k] * dz[k];
#pragma unroll
          for (int j = W - 2; j >= 1; --j) open[j][k] = open[j - 1][k] + taps.w[W - 1 - j][k] * dz[k];
          open[0][k] = taps.w[W - 1][k] * dz[k];
        }
        shift<W, BV>(win, xv);
      };
      bool done = false;
      for (int64_t tb = t0; !done; tb += BU) {
        RawN<T, BV> xr[BU], dr[BU];
        // rows in the middle of their tile and sequence need no questions (asked
        // for every row, they took as long as the arithmetic)
        if (tb >= t0 + W - 1 && tb >= s + W - 1 && tb + BU <= e && tb + BU <= t1) {
          const T* xp = static_cast<const T*>(a.x) + tb * a.xs + c;
          const T* dp = static_cast<const T*>(a.dy) + tb * a.C + c;
          T* yp = static_cast<T*>(a.y) + (tb - (W - 1)) * a.C + c;
#pragma unroll
          for (int i = 0; i < BU; ++i) {
            load_raw(xp + i * a.xs, xr[i]);
            load_raw(dp + i * a.C, dr[i]);
          }
#pragma unroll
          for (int i = 0; i < BU; ++i) {
            float v[BV];
            step(xr[i], dr[i], true, v);
            store_n(yp + i * a.C, v);
          }
          continue;
        }
#pragma unroll 1
        for (int i = 0; i < BU; ++i) {
          const int64_t t = tb + i;
          if (t == e) {
            flush();
            if (t >= t1) {
              done = true;
              break;
            }
            do {
              ++n;
              s = e;
              e = axis_start(a.ax, n + 1);
            } while (e == s && n + 1 < a.ax.N);
            load_state<T, W, BV>(a.init, n, a.C, c, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
              for (int k = 0; k < BV; ++k) open[j][k] = 0.f;
          }
          if (t >= te) {
            done = true;
            break;
          }
          load_raw(static_cast<const T*>(a.x) + t * a.xs + c, xr[0]);
          load_raw(static_cast<const T*>(a.dy) + t * a.C + c, dr[0]);
          float v[BV];
          step(xr[0], dr[0], t < t1, v);
          emit(t - (W - 1), v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) store4(a.part + ((int64_t)tile * (W + 1) + j) * a.C + c, dw[j]);
    zero_rest<T, BV>(a, t0, rows, c);
  }
  copy_empty<T>(a.ax, a.d_final, a.d_init, (W - 1) * a.C);
}

// dw [C][W] and dbias [C] from the tiles' sums, in a fixed order and in fp64: a
// workgroup has one tap of 32 channels, a line of each row, by 32 rows at a time.
constexpr int CRED = 1024, RC = 32, RR = CRED / RC;
__global__ void __launch_bounds__(CRED) kda_conv_reduce_kernel(ConvArgs a, int W) {
  __shared__ double sm[RR][RC];
  const int ch = threadIdx.x % RC, row = threadIdx.x / RC;
  const int j = blockIdx.x % (W + 1);
  const int64_t c = (int64_t)(blockIdx.x / (W + 1)) * RC + ch;
  if (j == W && !a.dbias) return;
  double s = 0.0;
  if (c < a.C) {
    constexpr int U = 4;  // rows asked for at once
    for (int64_t t0 = row; t0 < a.ntiles; t0 += U * RR) {
      float p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u] = t0 + u * RR < a.ntiles ? a.part[((t0 + u * RR) * (W + 1) + j) * a.C + c] : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) s += p[u];
    }
  }
  sm[row][ch] = s;
  for (int r = RR / 2; r >= 1; r >>= 1) {
    __syncthreads();
    if (row < r) sm[row][ch] += sm[row + r][ch];
  }
  if (row == 0 && c < a.C) {
    if (j == W) a.dbias[c] = (float)sm[0][ch];
    else a.dw[c * W + j] = (float)sm[0][ch];
  }
}

// Rows of a tile.  Long tiles read fewer rows twice (W - 1 of each tile, also
// the rows past it in the backward) and write fewer partial sums; short ones
// give a small call enough threads.  Measured (bf16, W = 4, us): forward at
// 2048 rows x 2048 channels 7 / 15 / 25 with 8 / 32 / 64 rows; backward there 24
// / 22 / 25 / 33 with 8 / 16 / 32 / 64, at 8192 x 1536 65 / 46 / 35 / 36, at
// 65536 x 256 111 / 111 / 69 / 52.
struct TileRule {
  int most, least;
  int64_t threads;  // shorter tiles while there are fewer threads than this
};
constexpr TileRule kFwdRule{64, 8, 256 * 1024}, kBwdRule{128, 32, 64 * 1024};
int tile_rows(int64_t T_total, int64_t groups, const TileRule& rule) {
  int r = rule.most;
  while (r > rule.least && (T_total + r - 1) / r * groups < rule.threads) r >>= 1;
  return r;
}
// Tiles of any backward over at most T_total rows: full-length tiles, or as
// many shorter ones as twice the wanted threads make.
int64_t most_tiles(int64_t T_total, int64_t groups) {
  const int64_t full = (T_total + kBwdRule.most - 1) / kBwdRule.most;
  const int64_t least = (T_total + kBwdRule.least - 1) / kBwdRule.least;
  const int64_t cut = 2 * kBwdRule.threads / groups + 1;
  const int64_t some = least < cut ? least : cut;
  return full > some ? full : some;
}

bool conv_sizes_ok(int64_t T_total, int64_t C) {
  return T_total >= 0 && C >= 1 && C <= (int64_t)1 << 30 && fits(T_total, C, kMaxElements);
}

kda_status_t conv_prepare(ConvArgs& a, const void* x, int64_t x_stride, const void* w, const void* bias,
                          const void* init, const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t C, int64_t W,
                          int64_t N, int dtype, unsigned flags, bool bwd, bool step = false) {
  if (B < 1 || T < 0 || C < 1 || N < 1 || W < 1) return KDA_ERR_INVALID;
  if (flags & ~(FLAG_SILU | (step ? 0u : FLAG_ZERO_REST))) return KDA_ERR_INVALID;
  if (cu_seqlens ? B != 1 : N != B) return KDA_ERR_INVALID;
  if (!w) return KDA_ERR_INVALID;
  if (!dtype_bytes(dtype) || C % 8 != 0 || W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
  if (!fits(B, T, (int64_t)1 << 46) || !conv_sizes_ok(B * T, C)) return KDA_ERR_INVALID;
  if (N > (int64_t)1 << 30 || !fits(N, W * C, kMaxElements)) return KDA_ERR_INVALID;
  if (cu_seqlens && T > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  if (x_stride < C || x_stride % 4 != 0 || !fits(B * T, x_stride, kMaxElements)) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {x, init}) || !aligned_all(16, {w, bias})) return KDA_ERR_INVALID;
  a = ConvArgs{};
  a.x = x;
  a.xs = x_stride;
  a.w = static_cast<const float*>(w);
  a.bias = static_cast<const float*>(bias);
  a.init = init;
  a.ax = make_axis(cu_seqlens, T, B * T, N);
  a.C = C;
  a.groups = C / (bwd ? BV : dtype == KDA_DTYPE_BF16 ? FV<__bf16> : FV<float>);
  a.rows = tile_rows(B * T, a.groups, bwd ? kBwdRule : kFwdRule);
  a.ntiles = (B * T + a.rows - 1) / a.rows;
  a.zero_rest = flags & FLAG_ZERO_REST ? 1 : 0;
  a.silu = flags & FLAG_SILU ? 1 : 0;
  if (!fits(a.ntiles, a.groups, (int64_t)1 << 38)) return KDA_ERR_INVALID;
  return KDA_SUCCESS;
}

int64_t conv_grid(int64_t items) { return items < 1 ? 1 : (items + CT - 1) / CT; }

template <template <typename, int> class F, typename... P>
kda_status_t by_type(int dtype, int64_t W, P... p) {
  if (dtype == KDA_DTYPE_BF16)
    return W == 2 ? F<__bf16, 2>::run(p...) : W == 3 ? F<__bf16, 3>::run(p...) : F<__bf16, 4>::run(p...);
  return W == 2 ? F<float, 2>::run(p...) : W == 3 ? F<float, 3>::run(p...) : F<float, 4>::run(p...);
}
template <typename T, int W>
struct RunFwd {
  static kda_status_t run(const ConvArgs& a, hipStream_t st) {
    return launch(&kda_conv_fwd_kernel<T, W>, conv_grid(a.ntiles * a.groups), CT, st, "conv forward", a);
  }
};
template <typename T, int W>
struct RunStep {
  static kda_status_t run(const ConvArgs& a, hipStream_t st) {
    return launch(&kda_conv_step_kernel<T, W>, conv_grid(a.ax.N * a.groups), CT, st, "conv step", a);
  }
};
template <typename T, int W>
struct RunBwd {
  static kda_status_t run(const ConvArgs& a, hipStream_t st) {
    const kda_status_t s =
        launch(&kda_conv_bwd_kernel<T, W>, conv_grid(a.ntiles * a.groups), CT, st, "conv backward", a);
    if (s != KDA_SUCCESS) return s;
    return launch(&kda_conv_reduce_kernel, (a.C + RC - 1) / RC * (W + 1), CRED, st, "conv reduce", a, W);
  }
};

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_conv_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias, void* out,
                          const void* initial_state, void* final_state, const int32_t* cu_seqlens, int64_t B,
                          int64_t T, int64_t C, int64_t W, int64_t N, int dtype, unsigned flags, void* stream) {
  ConvArgs a;
  const kda_status_t s =
      conv_prepare(a, x, x_stride, weight, bias, initial_state, cu_seqlens, B, T, C, W, N, dtype, flags, false);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !out)) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {out, final_state})) return KDA_ERR_INVALID;
  // (rows before a tile are another thread's to write, states another tile's)
  if (same(out, x) || same(final_state, initial_state)) return KDA_ERR_INVALID;
  a.y = out;
  a.fin = final_state;
  return by_type<RunFwd>(dtype, W, a, reinterpret_cast<hipStream_t>(stream));
}

kda_status_t kda_conv_step(const void* x, int64_t x_stride, const float* weight, const float* bias, void* out,
                           const void* initial_state, void* final_state, int64_t B, int64_t T, int64_t C, int64_t W,
                           int dtype, unsigned flags, void* stream) {
  ConvArgs a;
  const kda_status_t s =
      conv_prepare(a, x, x_stride, weight, bias, initial_state, nullptr, B, T, C, W, B, dtype, flags, false, true);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !out)) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {out, final_state}) || !fits(B, a.groups, (int64_t)1 << 38)) return KDA_ERR_INVALID;
  a.y = out;
  a.fin = final_state;
  return by_type<RunStep>(dtype, W, a, reinterpret_cast<hipStream_t>(stream));
}

size_t kda_conv_bwd_workspace_size(int64_t T_total, int64_t C, int64_t W) {
  if (!conv_sizes_ok(T_total, C) || C % 8 != 0 || W < 2 || W > 4) return 0;
  return 256 + align256((size_t)most_tiles(T_total, C / BV) * (size_t)(W + 1) * (size_t)C * sizeof(float));
}

kda_status_t kda_conv_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* d_out,
                          const void* d_final, void* dx, float* d_weight, float* d_bias, void* d_initial_state,
                          void* workspace, size_t workspace_bytes, const void* initial_state,
                          const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t C, int64_t W, int64_t N, int dtype,
                          unsigned flags, void* stream) {
  ConvArgs a;
  const kda_status_t s =
      conv_prepare(a, x, x_stride, weight, bias, initial_state, cu_seqlens, B, T, C, W, N, dtype, flags, true);
  if (s != KDA_SUCCESS) return s;
  if (!d_weight || (a.ax.total > 0 && (!x || !d_out || !dx))) return KDA_ERR_INVALID;
  const size_t al = 4 * dtype_bytes(dtype);
  if (!aligned_all(al, {d_out, d_final, dx, d_initial_state}) || !aligned(workspace, 16))
    return KDA_ERR_INVALID;
  if (!workspace || workspace_bytes < kda_conv_bwd_workspace_size(a.ax.total, C, W)) return KDA_ERR_WORKSPACE;
  if (same(dx, x) || same(dx, d_out) || same(d_initial_state, d_final) || same(d_initial_state, initial_state))
    return KDA_ERR_INVALID;
  a.dy = d_out;
  a.d_final = d_final;
  a.y = dx;
  a.d_init = d_initial_state;
  a.dw = d_weight;
  a.dbias = d_bias;
  a.part = static_cast<float*>(workspace);
  return by_type<RunBwd>(dtype, W, a, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
