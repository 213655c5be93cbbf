// Gated linear recurrence: the diagonal recurrence under KDA's own decay gate,
//     g_t = lower_bound * sigmoid(exp(A_log) (raw_gate_t + dt_bias))   (or given)
//     a_t = exp(g_t),   h_t = a_t h_{t-1} + b_t x_t,   b_t = 1 or 1 - a_t,
// per channel of [tokens][H * K], its gradients, and its step for decoding.
//
// A run of tokens maps the state that enters it to h -> A h + B (A the product
// of its decays, B its result from zero), and such maps compose.  The packed
// token axis is cut into tiles of 128 rows, whatever the sequences: a tile
// that holds the first row of a sequence has a map that does not depend on the
// entering state (it is reset: the composition selects, it does not multiply
// by zero, so that a sequence's NaN or infinity stays in it).  Three launches:
//   1. the map of every tile (reads x and raw_gate);
//   2. per channel, the state entering every tile, in order;
//   3. every tile again from its entering state, writing the outputs.
// A tile is 512 threads: 32 lanes of 4 channels by 16 runs of 8 rows, each run
// in one thread's registers, the runs joined through LDS in order.
//
// Backward, with dh_t = d_out_t + a_{t+1} dh_{t+1} (d_final joins at the last
// row) and e_t = a_t dh_t, the gradient that row t hands to the row before:
//     dx_t = b_t dh_t,   dg_t = a_t dh_t (h_{t-1} [- x_t if b = 1 - a])
// the same three launches run from the right over e; h_{t-1} is recomputed
// from the states that the forward left, one per tile.
//
// All arithmetic is fp32.

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_token.h"

namespace kda {
namespace {

constexpr int GR = 8;           // rows of a run
constexpr int GS = 16;          // runs of a tile
constexpr int GL = GR * GS;     // rows of a tile
constexpr int GC = 128;         // channels of a tile
constexpr int GT = GS * GC / 4; // threads

struct GlrArgs {
  const void* x;
  const void* g;
  const void* d_out;
  void* out;  // or dx
  void* dg;
  const float* A_log;
  const float* dt_bias;
  const float* init;
  const float* d_final;
  float* fin;
  float* d_init;
  float* states;  // [tiles][C] state entering every tile
  float2* maps;   // [tiles][C] A, B of every tile (backward: of its e map)
  int* reset;     // [tiles] whether the tile's map ignores what enters
  float* ends;    // [tiles][C] e entering every tile from the right
  float2* part;   // [tiles][C] sums over the tile of d_raw and of dz z
  float* dA_log;
  float* d_dt_bias;
  Axis ax;
  int64_t C;
  int H, K;
  int nblk;       // channel blocks of GC
  int ntiles;
  int zero_rest;  // rows behind the last sequence: zeros (else left as they were)
  float lb;
};

// The gate of 4 channels.  With z = exp(A_log) (raw + dt_bias), na and nb hold
// -exp(A_log) log2(e) and na dt_bias, so that -z log2(e) = na raw + nb.
template <bool GIVEN>
struct Gate {
  float na, nb[4], lb2;
  __device__ __forceinline__ void init(const GlrArgs& a, int64_t c) {
    if constexpr (!GIVEN) {
      na = -expf(a.A_log[c / a.K]) * LOG2E;
      load_f4(a.dt_bias + c, nb);
#pragma unroll
      for (int j = 0; j < 4; ++j) nb[j] *= na;
      lb2 = a.lb * LOG2E;
    }
  }
  // g log2(e)
  __device__ __forceinline__ float g2(float raw, int j) const {
    if constexpr (GIVEN) return raw * LOG2E;
    return lb2 * __builtin_amdgcn_rcpf(1.0f + fexp2(raw * na + nb[j]));
  }
};

// 1 - exp(g) from g log2(e) and a = exp(g).  Near zero the difference would
// cancel: there the series of -expm1 to its seventh term, whose remainder is
// under 2^-24 of the value for |g| < 1/4.
__device__ __forceinline__ float one_minus(float g2, float a) {
  const float y = g2 * 0.6931471805599453f;
  const float p =
      y * (1.f + y * (1.f / 2) * (1.f + y * (1.f / 3) * (1.f + y * (1.f / 4) * (1.f + y * (1.f / 5) *
          (1.f + y * (1.f / 6) * (1.f + y * (1.f / 7)))))));
  return fabsf(y) < 0.25f ? -p : 1.0f - a;
}

// The sequences that start (S) or end (E) at each row of the tile, -1 for
// none; returns whether there is any.  Ends with a barrier.
__device__ __forceinline__ bool mark_tile(const Axis& ax, int64_t t0, int* S, int* E) {
  const int tid = threadIdx.x;
  for (int i = tid; i < GL; i += GT) S[i] = E[i] = -1;
  const int64_t t1 = t0 + GL;
  const int64_t n0 = axis_lower(ax, t0);
  int64_t n1 = axis_lower(ax, t1);
  n1 = n1 < ax.N ? n1 : ax.N;
  __syncthreads();
  bool any = false;
  // sequence n0 - 1 is the one that reaches the tile from before it
  for (int64_t n = (n0 > 0 ? n0 - 1 : 0) + tid; n < n1; n += GT) {
    const int64_t s = axis_start(ax, n), e = axis_start(ax, n + 1);
    if (e <= s) continue;
    if (s >= t0 && s < t1) {
      S[s - t0] = (int)n;
      any = true;
    }
    if (e > t0 && e <= t1) {
      E[e - 1 - t0] = (int)n;
      any = true;
    }
  }
  return __syncthreads_or(any);
}

// MAPS: write the tile's map.  Otherwise the outputs, from the entering state.
template <typename T, bool GIVEN, bool COMPL, bool MAPS>
__global__ void __launch_bounds__(GT) kda_glr_fwd_kernel(GlrArgs a) {
  __shared__ float sA[GS][GC], sB[GS][GC];
  __shared__ int sS[GL], sE[GL], sReset[GS];
  const int tid = threadIdx.x, lane = tid & 31, run = tid >> 5;
  const int64_t rows = axis_rows(a.ax);
  for (int64_t item = blockIdx.x; item < (int64_t)a.ntiles * a.nblk; item += gridDim.x) {
    const int tile = (int)(item / a.nblk), blk = (int)(item % a.nblk);
    const int64_t c = (int64_t)blk * GC + lane * 4;
    const bool in = c < a.C;
    const int64_t t0 = (int64_t)tile * GL, tr = t0 + run * GR;
    raw4<T> xr[GR], gr[GR];
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      zero4(xr[i]);
      zero4(gr[i]);
      if (in && tr + i < rows) {
        xr[i] = *reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.x) + (tr + i) * a.C + c);
        gr[i] = *reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.g) + (tr + i) * a.C + c);
      }
    }
    Gate<GIVEN> gate;
    if (in) gate.init(a, c);
    const bool marked = mark_tile(a.ax, t0, sS, sE);
    float av[GR][4], u[GR][4];
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      float xv[4], gv[4];
      widen4(xr[i], xv);
      widen4(gr[i], gv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g2 = gate.g2(gv[j], j);
        av[i][j] = fexp2(g2);
        u[i][j] = COMPL ? one_minus(g2, av[i][j]) * xv[j] : xv[j];
      }
    }
    // the run's map
    float A[4], B[4];
    bool reset = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      A[j] = 1.f;
      B[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      if (marked && sS[run * GR + i] >= 0) {
        reset = true;
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) B[j] = zero[j];
        if (a.init && in) load_f4(a.init + (int64_t)sS[run * GR + i] * a.C + c, B);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] *= av[i][j];
        B[j] = av[i][j] * B[j] + u[i][j];
      }
    }
    store4(&sA[run][lane * 4], A);
    store4(&sB[run][lane * 4], B);
    if (lane == 0) sReset[run] = reset;
    __syncthreads();
    if constexpr (MAPS) {
      if (tid < GC && (int64_t)blk * GC + tid < a.C) {
        float At = 1.f, Bt = 0.f;
        bool r = false;
        for (int k = 0; k < GS; ++k) {
          const bool rk = sReset[k];
          Bt = rk ? sB[k][tid] : sA[k][tid] * Bt + sB[k][tid];
          At *= sA[k][tid];
          r |= rk;
        }
        a.maps[(int64_t)tile * a.C + (int64_t)blk * GC + tid] = make_float2(At, Bt);
        if (tid == 0 && blk == 0) a.reset[tile] = r;
      }
    } else {
      float h[4] = {0.f, 0.f, 0.f, 0.f};
      if (in) load_f4(a.states + (int64_t)tile * a.C + c, h);
      for (int k = 0; k < run; ++k) {
        float Ak[4], Bk[4];
        load_f4(&sA[k][lane * 4], Ak);
        load_f4(&sB[k][lane * 4], Bk);
        const bool rk = sReset[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = rk ? Bk[j] : Ak[j] * h[j] + Bk[j];
      }
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        if (marked && sS[run * GR + i] >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = 0.f;
          if (a.init && in) load_f4(a.init + (int64_t)sS[run * GR + i] * a.C + c, h);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = av[i][j] * h[j] + u[i][j];
        if (in && tr + i < rows) store4(static_cast<T*>(a.out) + (tr + i) * a.C + c, h);
        else if (in && a.zero_rest && tr + i < a.ax.total) store_zero4(static_cast<T*>(a.out) + (tr + i) * a.C + c);
        if (marked && a.fin && in && sE[run * GR + i] >= 0)
          store4(a.fin + (int64_t)sE[run * GR + i] * a.C + c, h);
      }
    }
    __syncthreads();
  }
  if (!MAPS && a.fin) {  // empty sequences hand their state on
    for (int64_t n = blockIdx.x; n < a.ax.N; n += gridDim.x) {
      if (axis_start(a.ax, n + 1) > axis_start(a.ax, n)) continue;
      for (int64_t c = tid; c < a.C; c += GT) a.fin[n * a.C + c] = a.init ? a.init[n * a.C + c] : 0.f;
    }
  }
}

// Per channel: what enters every tile, in order.  REV: from the right.
template <bool REV>
__global__ void __launch_bounds__(64) kda_glr_fold_kernel(GlrArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (c >= a.C) return;
  float* to = REV ? a.ends : a.states;
  float s = 0.f;
  constexpr int U = 8;
  for (int k0 = 0; k0 < a.ntiles; k0 += U) {
    float2 m[U];
    int r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int k = k0 + u < a.ntiles ? k0 + u : a.ntiles - 1;
      k = REV ? a.ntiles - 1 - k : k;
      m[u] = a.maps[(int64_t)k * a.C + c];
      r[u] = a.reset[k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u < a.ntiles) {
        const int k = REV ? a.ntiles - 1 - k0 - u : k0 + u;
        to[(int64_t)k * a.C + c] = s;
        s = r[u] ? m[u].y : m[u].x * s + m[u].y;
      }
    }
  }
}

template <typename T, bool GIVEN, bool COMPL, bool MAPS>
__global__ void __launch_bounds__(GT) kda_glr_bwd_kernel(GlrArgs a) {
  __shared__ float sA[GS][GC], sB[GS][GC];
  __shared__ int sS[GL], sE[GL], sReset[GS];
  const int tid = threadIdx.x, lane = tid & 31, run = tid >> 5;
  const int64_t rows = axis_rows(a.ax);
  for (int64_t item = blockIdx.x; item < (int64_t)a.ntiles * a.nblk; item += gridDim.x) {
    const int tile = (int)(item / a.nblk), blk = (int)(item % a.nblk);
    const int64_t c = (int64_t)blk * GC + lane * 4;
    const bool in = c < a.C;
    const int64_t t0 = (int64_t)tile * GL, tr = t0 + run * GR;
    raw4<T> xr[GR], gr[GR], dr[GR];
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      zero4(xr[i]);
      zero4(gr[i]);
      zero4(dr[i]);
      if (in && tr + i < rows) {
        const int64_t o = (tr + i) * a.C + c;
        if (!MAPS) xr[i] = *reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.x) + o);
        gr[i] = *reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.g) + o);
        dr[i] = *reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.d_out) + o);
      }
    }
    Gate<GIVEN> gate;
    if (in) gate.init(a, c);
    const bool marked = mark_tile(a.ax, t0, sS, sE);
    float g2[GR][4];
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      float gv[4];
      widen4(gr[i], gv);
#pragma unroll
      for (int j = 0; j < 4; ++j) g2[i][j] = gate.g2(gv[j], j);
    }
    // the run's map of e, from the right
    float P[4], Q[4];
    bool reset = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      P[j] = 1.f;
      Q[j] = 0.f;
    }
#pragma unroll
    for (int i = GR - 1; i >= 0; --i) {
      if (tr + i >= rows) continue;  // rows behind the last sequence hand nothing on
      if (marked && sE[run * GR + i] >= 0) {
        reset = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) Q[j] = 0.f;
        if (a.d_final && in) load_f4(a.d_final + (int64_t)sE[run * GR + i] * a.C + c, Q);
      }
      float dv[4];
      widen4(dr[i], dv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float av = fexp2(g2[i][j]);
        P[j] *= av;
        Q[j] = av * (dv[j] + Q[j]);
      }
    }
    store4(&sA[run][lane * 4], P);
    store4(&sB[run][lane * 4], Q);
    if (lane == 0) sReset[run] = reset;
    __syncthreads();
    if constexpr (MAPS) {
      if (tid < GC && (int64_t)blk * GC + tid < a.C) {
        float Pt = 1.f, Qt = 0.f;
        bool r = false;
        for (int k = GS - 1; k >= 0; --k) {
          const bool rk = sReset[k];
          Qt = rk ? sB[k][tid] : sA[k][tid] * Qt + sB[k][tid];
          Pt *= sA[k][tid];
          r |= rk;
        }
        a.maps[(int64_t)tile * a.C + (int64_t)blk * GC + tid] = make_float2(Pt, Qt);
        if (tid == 0 && blk == 0) a.reset[tile] = r;
      }
    } else {
      float e[4] = {0.f, 0.f, 0.f, 0.f};
      if (in) load_f4(a.ends + (int64_t)tile * a.C + c, e);
      for (int k = GS - 1; k > run; --k) {
        float Pk[4], Qk[4];
        load_f4(&sA[k][lane * 4], Pk);
        load_f4(&sB[k][lane * 4], Qk);
        const bool rk = sReset[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = rk ? Qk[j] : Pk[j] * e[j] + Qk[j];
      }
      __syncthreads();
      // the run's forward map, and the state that enters the run
      float A[4], B[4];
      bool fresh = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] = 1.f;
        B[j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        if (marked && sS[run * GR + i] >= 0) {
          fresh = true;
#pragma unroll
          for (int j = 0; j < 4; ++j) B[j] = 0.f;
          if (a.init && in) load_f4(a.init + (int64_t)sS[run * GR + i] * a.C + c, B);
        }
        float xv[4];
        widen4(xr[i], xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float av = fexp2(g2[i][j]);
          A[j] *= av;
          B[j] = av * B[j] + (COMPL ? one_minus(g2[i][j], av) * xv[j] : xv[j]);
        }
      }
      store4(&sA[run][lane * 4], A);
      store4(&sB[run][lane * 4], B);
      if (lane == 0) sReset[run] = fresh;
      __syncthreads();
      float h[4] = {0.f, 0.f, 0.f, 0.f};
      if (in) load_f4(a.states + (int64_t)tile * a.C + c, h);
      for (int k = 0; k < run; ++k) {
        float Ak[4], Bk[4];
        load_f4(&sA[k][lane * 4], Ak);
        load_f4(&sB[k][lane * 4], Bk);
        const bool rk = sReset[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = rk ? Bk[j] : Ak[j] * h[j] + Bk[j];
      }
      // h_{t-1} of every row
      float hp[GR][4];
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        if (marked && sS[run * GR + i] >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = 0.f;
          if (a.init && in) load_f4(a.init + (int64_t)sS[run * GR + i] * a.C + c, h);
        }
        float xv[4];
        widen4(xr[i], xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float av = fexp2(g2[i][j]);
          hp[i][j] = h[j];
          h[j] = av * h[j] + (COMPL ? one_minus(g2[i][j], av) * xv[j] : xv[j]);
        }
      }
      float dsum[4] = {0.f, 0.f, 0.f, 0.f}, zsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = GR - 1; i >= 0; --i) {
        if (tr + i >= rows) {
          if (in && a.zero_rest && tr + i < a.ax.total) {
            store_zero4(static_cast<T*>(a.out) + (tr + i) * a.C + c);
            store_zero4(static_cast<T*>(a.dg) + (tr + i) * a.C + c);
          }
          continue;
        }
        if (marked && sE[run * GR + i] >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = 0.f;
          if (a.d_final && in) load_f4(a.d_final + (int64_t)sE[run * GR + i] * a.C + c, e);
        }
        float dv[4], xv[4], gv[4], dx[4], dg[4];
        widen4(dr[i], dv);
        widen4(xr[i], xv);
        widen4(gr[i], gv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float av = fexp2(g2[i][j]);
          const float dh = dv[j] + e[j];
          e[j] = av * dh;
          dx[j] = COMPL ? one_minus(g2[i][j], av) * dh : dh;
          dg[j] = e[j] * (COMPL ? hp[i][j] - xv[j] : hp[i][j]);
          if constexpr (!GIVEN) {
            // dg/dz = lb s (1 - s), s = 1 / (1 + w), w = exp(-z).  w is kept
            // finite (a comparison, so that NaN stays) so that w s does not
            // become infinity times zero.
            const float mz = gv[j] * gate.na + gate.nb[j];  // -z log2(e)
            const float w = fexp2(mz > 126.f ? 126.f : mz);
            const float s = __builtin_amdgcn_rcpf(1.0f + w);
            const float dz = dg[j] * (a.lb * s * (w * s));
            zsum[j] += dz * (mz * -0.6931471805599453f);
            dg[j] = dz * (gate.na * -0.6931471805599453f);  // dz/draw = exp(A_log)
            dsum[j] += dg[j];
          }
        }
        if (in) {
          const int64_t o = (tr + i) * a.C + c;
          store4(static_cast<T*>(a.out) + o, dx);
          store4(static_cast<T*>(a.dg) + o, dg);
          if (marked && a.d_init && sS[run * GR + i] >= 0)
            store4(a.d_init + (int64_t)sS[run * GR + i] * a.C + c, e);
        }
      }
      if constexpr (!GIVEN) {
        __syncthreads();
        store4(&sA[run][lane * 4], dsum);
        store4(&sB[run][lane * 4], zsum);
        __syncthreads();
        if (tid < GC && (int64_t)blk * GC + tid < a.C) {
          float d = 0.f, z = 0.f;
          for (int k = 0; k < GS; ++k) {
            d += sA[k][tid];
            z += sB[k][tid];
          }
          a.part[(int64_t)tile * a.C + (int64_t)blk * GC + tid] = make_float2(d, z);
        }
      }
    }
    __syncthreads();
  }
  if (!MAPS && a.d_init) {
    for (int64_t n = blockIdx.x; n < a.ax.N; n += gridDim.x) {
      if (axis_start(a.ax, n + 1) > axis_start(a.ax, n)) continue;
      for (int64_t c = tid; c < a.C; c += GT) a.d_init[n * a.C + c] = a.d_final ? a.d_final[n * a.C + c] : 0.f;
    }
  }
}

// Sums of the tiles' partial sums, in a fixed order and in fp64 (a long
// sequence has thousands of them): d_dt_bias per channel, dA_log per head.
constexpr int GRED = 1024;
__global__ void __launch_bounds__(GRED) kda_glr_reduce_kernel(GlrArgs a) {
  __shared__ double sd[GRED], sz[GRED];
  const int tid = threadIdx.x, h = blockIdx.x;
  double head = 0.0;
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    const int k = k0 + (tid & 63), row = tid >> 6;  // 16 rows of 64 channels
    double d = 0.0, z = 0.0;
    if (k < a.K)
      for (int t = row; t < a.ntiles; t += GRED / 64) {
        const float2 p = a.part[(int64_t)t * a.C + (int64_t)h * a.K + k];
        d += p.x;
        z += p.y;
      }
    sd[tid] = d;
    sz[tid] = z;
    __syncthreads();
    if (tid < 64 && k < a.K) {
      for (int r = 1; r < GRED / 64; ++r) {
        d += sd[r * 64 + tid];
        z += sz[r * 64 + tid];
      }
      a.d_dt_bias[(int64_t)h * a.K + k] = (float)d;
      head += z;
    }
    __syncthreads();
  }
  if (tid < 64) {
    for (int m = 32; m >= 1; m >>= 1) head += __shfl_xor(head, m);
    if (tid == 0) a.dA_log[h] = (float)head;
  }
}

// One thread per 4 channels of a sequence, its T tokens in order.
constexpr int GST = 256;
template <typename T, bool GIVEN, bool COMPL>
__global__ void __launch_bounds__(GST) kda_glr_step_kernel(GlrArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * GST + threadIdx.x) * 4;
  if (i >= a.ax.N * a.C) return;
  const int64_t n = i / a.C, c = i % a.C;
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.init) load_f4(a.init + i, h);
  Gate<GIVEN> gate;
  gate.init(a, c);
  for (int64_t t = 0; t < a.ax.T; ++t) {
    const int64_t o = (n * a.ax.T + t) * a.C + c;
    float xv[4], gv[4];
    widen4(*reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.x) + o), xv);
    widen4(*reinterpret_cast<const raw4<T>*>(static_cast<const T*>(a.g) + o), gv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float g2 = gate.g2(gv[j], j), av = fexp2(g2);
      h[j] = av * h[j] + (COMPL ? one_minus(g2, av) * xv[j] : xv[j]);
    }
    store4(static_cast<T*>(a.out) + o, h);
  }
  if (a.fin) store4(a.fin + i, h);
}

struct GlrLayout {
  size_t maps, reset, states, ends, part, total;
};
// Forward: tile maps and reset words, and the states where the caller keeps
// none.  Backward: tile maps, reset words, entering gradients, partial sums.
GlrLayout glr_layout(int64_t T_total, int64_t C, bool bwd) {
  const size_t tiles = (size_t)((T_total + GL - 1) / GL), w = tiles * (size_t)C;
  GlrLayout l;
  l.maps = 256;
  l.reset = l.maps + align256(w * sizeof(float2));
  l.states = l.reset + align256(tiles * sizeof(int));
  l.ends = l.states;
  l.part = l.states + align256(w * sizeof(float));
  l.total = l.part + (bwd ? align256(w * sizeof(float2)) : 0);
  return l;
}

bool glr_sizes_ok(int64_t T_total, int64_t H, int64_t K) {
  return T_total >= 0 && H >= 1 && K >= 1 && fits(H, K, (int64_t)1 << 30) && fits(T_total, H * K, kMaxElements);
}

// Checks shared by the entry points; fills the sizes and the gate.
kda_status_t glr_prepare(GlrArgs& a, const float* A_log, const float* dt_bias, float lower_bound,
                         const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t H, int64_t K, int64_t N,
                         int dtype, unsigned flags, bool step = false) {
  if (B < 1 || T < 0 || H < 1 || K < 1 || N < 1) return KDA_ERR_INVALID;
  if (flags & ~(unsigned)(FLAG_GATE_GIVEN | FLAG_COMPLEMENT | (step ? 0 : FLAG_ZERO_REST))) return KDA_ERR_INVALID;
  if (cu_seqlens ? B != 1 : N != B) return KDA_ERR_INVALID;
  if (!(flags & FLAG_GATE_GIVEN) && (!A_log || !dt_bias)) return KDA_ERR_INVALID;
  if (!dtype_bytes(dtype) || K % 4 != 0) return KDA_ERR_UNSUPPORTED;
  if (!(flags & FLAG_GATE_GIVEN) && !(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_UNSUPPORTED;
  if (!fits(B, T, (int64_t)1 << 46) || !glr_sizes_ok(B * T, H, K)) return KDA_ERR_INVALID;
  if (N > (int64_t)1 << 30 || !fits(N, H * K, kMaxElements)) return KDA_ERR_INVALID;
  if (cu_seqlens && T > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  if (!(flags & FLAG_GATE_GIVEN) && !aligned(dt_bias, 16)) return KDA_ERR_INVALID;
  const int64_t tiles = (B * T + GL - 1) / GL, nblk = (H * K + GC - 1) / GC;
  if (tiles > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  a = GlrArgs{};
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.ax = Axis{cu_seqlens, T, B * T, (int)N};
  a.C = H * K;
  a.H = (int)H;
  a.K = (int)K;
  a.nblk = (int)nblk;
  a.ntiles = (int)tiles;
  a.lb = lower_bound;
  a.zero_rest = flags & FLAG_ZERO_REST ? 1 : 0;
  return KDA_SUCCESS;
}

template <template <typename, bool, bool> class F, typename... P>
kda_status_t by_variant(int dtype, unsigned flags, P... p) {
  const bool g = flags & FLAG_GATE_GIVEN, c = flags & FLAG_COMPLEMENT;
  if (dtype == KDA_DTYPE_BF16)
    return g ? (c ? F<__bf16, true, true>::run(p...) : F<__bf16, true, false>::run(p...))
             : (c ? F<__bf16, false, true>::run(p...) : F<__bf16, false, false>::run(p...));
  return g ? (c ? F<float, true, true>::run(p...) : F<float, true, false>::run(p...))
           : (c ? F<float, false, true>::run(p...) : F<float, false, false>::run(p...));
}

template <typename T, bool GIVEN, bool COMPL>
struct RunFwd {
  static kda_status_t run(const GlrArgs& a, hipStream_t st) {
    const int64_t items = (int64_t)a.ntiles * a.nblk;
    if (items > 0) {
      kda_status_t s = launch(&kda_glr_fwd_kernel<T, GIVEN, COMPL, true>, grid_of(items), GT, st, "glr maps", a);
      if (s == KDA_SUCCESS) s = launch(&kda_glr_fold_kernel<false>, (a.C + 63) / 64, 64, st, "glr fold", a);
      if (s != KDA_SUCCESS) return s;
    }
    return launch(&kda_glr_fwd_kernel<T, GIVEN, COMPL, false>, grid_of(items), GT, st, "glr forward", a);
  }
};
template <typename T, bool GIVEN, bool COMPL>
struct RunBwd {
  static kda_status_t run(const GlrArgs& a, hipStream_t st) {
    const int64_t items = (int64_t)a.ntiles * a.nblk;
    kda_status_t s = KDA_SUCCESS;
    if (items > 0) {
      s = launch(&kda_glr_bwd_kernel<T, GIVEN, COMPL, true>, grid_of(items), GT, st, "glr backward maps", a);
      if (s == KDA_SUCCESS) s = launch(&kda_glr_fold_kernel<true>, (a.C + 63) / 64, 64, st, "glr fold", a);
      if (s != KDA_SUCCESS) return s;
    }
    s = launch(&kda_glr_bwd_kernel<T, GIVEN, COMPL, false>, grid_of(items), GT, st, "glr backward", a);
    if (s != KDA_SUCCESS || GIVEN) return s;
    return launch(&kda_glr_reduce_kernel, a.H, GRED, st, "glr reduce", a);
  }
};
template <typename T, bool GIVEN, bool COMPL>
struct RunStep {
  static kda_status_t run(const GlrArgs& a, int64_t grid, hipStream_t st) {
    return launch(&kda_glr_step_kernel<T, GIVEN, COMPL>, grid, GST, st, "glr step", a);
  }
};

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_glr_states_size(int64_t T_total, int64_t H, int64_t K) {
  if (!glr_sizes_ok(T_total, H, K)) return 0;
  return align256((size_t)((T_total + GL - 1) / GL) * (size_t)(H * K) * sizeof(float)) + 256;
}

size_t kda_glr_workspace_size(int64_t T_total, int64_t H, int64_t K) {
  return glr_sizes_ok(T_total, H, K) ? glr_layout(T_total, H * K, false).total : 0;
}

size_t kda_glr_bwd_workspace_size(int64_t T_total, int64_t H, int64_t K) {
  return glr_sizes_ok(T_total, H, K) ? glr_layout(T_total, H * K, true).total : 0;
}

kda_status_t kda_glr_fwd(const void* x, const void* raw_gate, void* out, void* workspace, size_t workspace_bytes,
                         const float* A_log, const float* dt_bias, float lower_bound, const float* initial_state,
                         float* final_state, float* states, const int32_t* cu_seqlens, int64_t B, int64_t T,
                         int64_t H, int64_t K, int64_t N, int dtype, unsigned flags, void* stream) {
  GlrArgs a;
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, cu_seqlens, B, T, H, K, N, dtype, flags);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !raw_gate || !out)) return KDA_ERR_INVALID;
  if (!aligned_all(4 * dtype_bytes(dtype), {x, raw_gate, out}) ||
      !aligned_all(16, {initial_state, final_state, states, workspace}))
    return KDA_ERR_INVALID;
  const GlrLayout l = glr_layout(a.ax.total, a.C, false);
  if (!workspace || workspace_bytes < l.total) return KDA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  a.x = x;
  a.g = raw_gate;
  a.out = out;
  a.init = initial_state;
  a.fin = final_state;
  a.maps = reinterpret_cast<float2*>(ws + l.maps);
  a.reset = reinterpret_cast<int*>(ws + l.reset);
  a.states = states ? states : reinterpret_cast<float*>(ws + l.states);
  return by_variant<RunFwd>(dtype, flags, a, reinterpret_cast<hipStream_t>(stream));
}

kda_status_t kda_glr_bwd(const void* x, const void* raw_gate, const float* states, const void* d_out,
                         const float* d_final, void* dx, void* d_raw_gate, float* dA_log, float* d_dt_bias,
                         float* d_initial_state, void* workspace, size_t workspace_bytes, const float* A_log,
                         const float* dt_bias, float lower_bound, const float* initial_state,
                         const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t H, int64_t K, int64_t N,
                         int dtype, unsigned flags, void* stream) {
  GlrArgs a;
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, cu_seqlens, B, T, H, K, N, dtype, flags);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !raw_gate || !states || !d_out || !dx || !d_raw_gate)) return KDA_ERR_INVALID;
  if (!(flags & FLAG_GATE_GIVEN) && (!dA_log || !d_dt_bias)) return KDA_ERR_INVALID;
  if (!aligned_all(4 * dtype_bytes(dtype), {x, raw_gate, d_out, dx, d_raw_gate}) ||
      !aligned_all(16, {states, d_final, d_initial_state, initial_state, workspace}))
    return KDA_ERR_INVALID;
  const GlrLayout l = glr_layout(a.ax.total, a.C, true);
  if (!workspace || workspace_bytes < l.total) return KDA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  a.x = x;
  a.g = raw_gate;
  a.d_out = d_out;
  a.out = dx;
  a.dg = d_raw_gate;
  a.init = initial_state;
  a.d_final = d_final;
  a.d_init = d_initial_state;
  a.dA_log = dA_log;
  a.d_dt_bias = d_dt_bias;
  a.maps = reinterpret_cast<float2*>(ws + l.maps);
  a.reset = reinterpret_cast<int*>(ws + l.reset);
  a.states = const_cast<float*>(states);
  a.ends = reinterpret_cast<float*>(ws + l.ends);
  a.part = reinterpret_cast<float2*>(ws + l.part);
  return by_variant<RunBwd>(dtype, flags, a, reinterpret_cast<hipStream_t>(stream));
}

kda_status_t kda_glr_step(const void* x, const void* raw_gate, void* out, const float* A_log, const float* dt_bias,
                          float lower_bound, const float* initial_state, float* final_state, int64_t B, int64_t T,
                          int64_t H, int64_t K, int dtype, unsigned flags, void* stream) {
  GlrArgs a;
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, nullptr, B, T, H, K, B, dtype, flags, true);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !raw_gate || !out)) return KDA_ERR_INVALID;
  if (!aligned_all(4 * dtype_bytes(dtype), {x, raw_gate, out}) || !aligned_all(16, {initial_state, final_state}))
    return KDA_ERR_INVALID;
  const int64_t grid = (B * a.C / 4 + GST - 1) / GST;
  if (grid > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  a.x = x;
  a.g = raw_gate;
  a.out = out;
  a.init = initial_state;
  a.fin = final_state;
  return by_variant<RunStep>(dtype, flags, a, grid, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
