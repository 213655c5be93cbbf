// Linear attention with one decay for each head.  Per sequence and head, with
// a = exp(g),
//     S_t = a S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Over a chunk of C tokens i that S_0 enters,
//     o_i = scale [ a^{i+1} S_0^T q_i + sum_{j<=i} a^{i-j} (q_i.k_j) v_j ],
//     S_C = a^C S_0 + sum_j a^{C-1-j} k_j v_j^T.
// The gradients are sums of the same form.  With dS_t = scale q_t do_t^T + a dS_{t+1},
//     dq_t = scale S_t do_t   (as o, of do, v, k in the place of q, k, v),
//     dv_t = dS_t^T k_t, dk_t = dS_t v_t   (as o with the time reversed, of k, q, do and of v, do, q),
// so one kernel does a sweep of all four: out_i = sum over j of (x_i.y_j) z_j
// times decays, a state [y][z] carried along, forwards or backwards in time.
//
// The decay's gradient is sum_t <dS_t/dg part>: with R_t = dS_t/dg,
//     R_t = a (R_{t-1} + S_{t-1}),   dg = sum_t scale q_t.(R_t do_t) + <R_T, dS_T>,
// carried in the dq sweep as a second state; over a chunk
//     R_C = a^C (R_0 + C S_0) + sum_j (C-1-j) a^{C-1-j} v_j k_j^T,
// and its part of o weighs the pair (i, j) by i - j.  No difference of large
// sums is taken (sum t (q_t.dq_t - k_t.dk_t) would be one).
//
// A workgroup of four waves takes one head, one slice of z's channels and a
// segment of the packed token axis, 64 tokens a step.  Each wave owns 16 or 32
// channels c of z and keeps S[d][c] in accumulators.  That layout is the A
// operand of out^T = S^T x^T and the result layout of S += y^T z, so the state
// meets no LDS; y^T and z^T come from transposing LDS reads of the row-major
// tiles.  Only the 64 x 64 products x y^T are shared, each wave forming 16 rows
// of them.
//
// Precision: products of bf16 inputs are exact in the fp32 accumulators.  Where
// an fp32 value has to be an MFMA operand it is split into bf16 parts: z times
// its decay into three (the states are fp32 results), the pair weights and the
// entering state into two (2^-16, where the bf16 output has 2^-8; the decay's
// gradient is an fp32 result again, and takes three).  A sum of one bf16 part
// would add errors as large as the output's own rounding.

#include "../../include/kda.h"
#include "kda_mix.h"

namespace kda {
namespace {

constexpr int LC = 64;          // tokens of a step
constexpr int LT = 256;         // threads
constexpr int64_t kLaWant = 512;   // workgroups to aim for: two per CU
constexpr int64_t kLaEnough = 160; // chains that fill the chip without being cut into segments
constexpr int64_t kLaMinSeg = 512; // tokens of a segment at least

// One sweep.  State element (d, c) of sequence n and head h is at
// (n H + h) K V + d sr + c sc.
struct LaPass {
  const uint16_t *x, *y, *z;
  uint16_t* out;  // [tokens][H][DZ]
  const uint16_t* w;  // the decay's gradient: q, dotted with the weighted outputs
  const float* sin;   // state that enters each sequence, or nullptr for zeros
  float* sout;        // state that leaves it, or nullptr
  const float* rend;  // the decay's gradient: d_final, dotted with R at each sequence's end
  float* seg;         // [segments][H][DX][DZ] state that enters each segment; then the same of R
  float* part;        // the decay's gradient, [H][segments][slices]
  int64_t xs, xh, ys, yh, zs, zh, ws, wh;  // token and head strides, elements
  int sr, sc;
  int rev;          // time runs backwards
  int off;          // decays of an entering state: a^{i + off}
  float c1, c2, c3;  // scale of the pairs, of the entering state's part, of what joins the state
};
struct LaArgs {
  LaPass p[2];
  Axis ax;
  const float* g;
  int64_t block, L;  // tokens of a block of the axis (a sequence, or all of it), of a segment
  int spb;           // segments per block
  int nseg, H, KV;   // segments; heads; elements of a state
  int slices, passes;
  int64_t items;     // nseg * H
  int64_t main;      // workgroups that sweep; those behind them handle empty sequences
  int zero_rest;
};

struct LaSeg {
  int64_t p0, p1;  // rows of the segment, within those that belong to sequences
};
__device__ __forceinline__ LaSeg la_seg(const LaArgs& a, int s, int64_t R) {
  const int b = s / a.spb, k = s % a.spb;
  int64_t p0 = b * a.block + k * a.L, p1 = p0 + a.L, e = (b + 1) * a.block;
  p1 = p1 < e ? p1 : e;
  return LaSeg{p0, p1 < R ? p1 : R};
}
__device__ __forceinline__ int64_t la_end(const Axis& ax, int64_t n, int64_t R) {
  const int64_t e = axis_start(ax, n + 1);
  return e < R ? e : R;
}

// exp(g n) of a token count, in fp64: a step's factor is met once for every
// step that the memory reaches over.
__device__ __forceinline__ float la_pow(float g, double n) { return n == 0 ? 1.0f : (float)exp((double)g * n); }

// The stretch of one sequence that a segment holds.
struct LaStretch {
  int64_t a, b;  // rows
  int n;
  bool starts, ends;  // the sequence starts (ends) here, in the sweep's direction
};

template <int DX, int ZW, bool OUT, bool DG>
__global__ void __launch_bounds__(LT, DG ? 1 : 2) la_sweep_kernel(const LaArgs a) {
  constexpr int NZ = 4 * ZW, XP = DX + 16, ZP = NZ + 16;  // LDS pitches: rows 8 banks (Z: 40) apart
  constexpr int NCT = ZW / 16, NDT = DX / 16, NKB = DX / 32;
  constexpr int NP = DG ? 3 : 2;  // bf16 parts of pair weights and entering states
  constexpr int XU = LC * DX / 8 / LT, ZU = LC * NZ / 8 / LT;  // 16-byte pieces a thread loads
  __shared__ __align__(16) uint16_t sX[OUT ? LC * XP : 8], sY[LC * XP], sZ[LC * ZP];
  __shared__ uint4 sP[OUT ? (DG ? 2 * NP : NP) : 1][OUT ? 8 : 1][64];  // pair weights as B operands (then times i - j)
  __shared__ float sLam[LC + 1];
  __shared__ float sRed[4];

  const int t = threadIdx.x, lane = t & 63, w = t >> 6, l16 = lane & 15, g4 = lane >> 4;
  const int64_t R = axis_rows(a.ax);

  // ---- sequences without tokens: what leaves them is what entered
  if ((int64_t)blockIdx.x >= a.main) {
    const int64_t more = gridDim.x - a.main;
    for (int64_t n = blockIdx.x - a.main; n < a.ax.N; n += more) {
      if (la_end(a.ax, n, R) > axis_start(a.ax, n)) continue;
      const int64_t at = n * a.H * a.KV;
      for (int i = 0; i < a.passes; ++i) {
        if (!a.p[i].sout) continue;
        for (int64_t e = t; e < (int64_t)a.H * a.KV; e += LT) a.p[i].sout[at + e] = a.p[i].sin ? a.p[i].sin[at + e] : 0.0f;
      }
    }
    return;
  }

  // ---- this workgroup's place.  Ids that agree mod 8 run on one XCD: the
  // slices and passes of an item, which read the same rows, are neighbours there.
  const int64_t id = blockIdx.x;
  const int kinds = a.slices * a.passes;
  const int64_t item = id / 8 / kinds * 8 + id % 8;
  if (item >= a.items) return;
  const int kind = (int)(id / 8 % kinds), slice = kind % a.slices;
  const LaPass& p = a.p[kind / a.slices];
  const int h = (int)(item % a.H), s = (int)(item / a.H);
  const int DZ = NZ * a.slices;
  const LaSeg sg = la_seg(a, s, R);
  const int rev = p.rev;

  if (OUT && a.zero_rest) {  // rows behind the last sequence, those of this segment
    const int b = s / a.spb, k = s % a.spb;
    int64_t q0 = b * a.block + k * a.L, q1 = q0 + a.L < (b + 1) * a.block ? q0 + a.L : (b + 1) * a.block;
    q0 = q0 > R ? q0 : R;
    for (int64_t e = (int64_t)t * 8; q0 * NZ + e < q1 * NZ; e += LT * 8) {
      const int64_t row = q0 + e / NZ;
      *reinterpret_cast<uint4*>(p.out + (row * a.H + h) * DZ + slice * NZ + e % NZ) = make_uint4(0, 0, 0, 0);
    }
  }
  if (DG && t == 0) p.part[((int64_t)h * a.nseg + s) * a.slices + slice] = 0.0f;
  if (sg.p0 >= sg.p1) return;

  const float gh = a.g[h];
  if (t <= LC) sLam[t] = la_pow(gh, t);
  __syncthreads();

  // ---- the first stretch.  OUT: all stretches of the segment in the sweep's
  // order; otherwise the one that goes on beyond the segment's end, if any.
  const bool tail = rev == (OUT ? 0 : 1);  // whether to begin at the segment's first row
  LaStretch c;
  auto place = [&](int n) {
    const int64_t bos = axis_start(a.ax, n), eos = la_end(a.ax, n, R);
    c.n = n;
    c.a = bos > sg.p0 ? bos : sg.p0;
    c.b = eos < sg.p1 ? eos : sg.p1;
    c.starts = rev ? eos <= sg.p1 : bos >= sg.p0;
    c.ends = rev ? bos >= sg.p0 : eos <= sg.p1;
  };
  place(axis_owner(a.ax, tail ? sg.p0 : sg.p1 - 1));
  if (!OUT && c.ends) return;
  if (c.a >= c.b) return;  // only where offsets break their contract
  int64_t done = 0;  // tokens of the stretch before the current step

  uint4 rx[OUT ? XU : 1], ry[XU], rz[ZU];
  auto rows = [&](auto& r, auto width, const uint16_t* base, int64_t ts, int64_t row0, int len) {
    constexpr int W8 = decltype(width)::value / 8;
    const uint16_t* q = base + row0 * ts;
#pragma unroll
    for (int u = 0; u < (int)(sizeof(r) / 16); ++u) {
      const int e = t + LT * u, row = e / W8;
      const int at = (rev ? -row : row) * (int)ts + e % W8 * 8;
      r[u] = row < len ? *reinterpret_cast<const uint4*>(q + at) : make_uint4(0, 0, 0, 0);
    }
  };
  auto fetch = [&]() {  // the step's rows into registers; time step i is row0 + i, or row0 - i
    const int64_t row0 = rev ? c.b - 1 - done : c.a + done;
    const int64_t left = c.b - c.a - done;
    const int len = (int)(left < LC ? left : LC);
    if constexpr (OUT) rows(rx, std::integral_constant<int, DX>{}, p.x + h * p.xh, p.xs, row0, len);
    rows(ry, std::integral_constant<int, DX>{}, p.y + h * p.yh, p.ys, row0, len);
    rows(rz, std::integral_constant<int, NZ>{}, p.z + h * p.zh + slice * NZ, p.zs, row0, len);
  };

  f32x4 S[NDT][NCT], Rs[DG ? NDT : 1][DG ? NCT : 1];
  double dg = 0.0;
  const int col = slice * NZ + w * ZW + l16;  // the lane's channel of z (+ 16 ct)
  const int64_t segat = ((int64_t)s * a.H + h) * a.KV;
  const int64_t rat = (int64_t)a.nseg * a.H * a.KV;  // R's segments lie behind S's
  // a^{i-j} of the wave's 16 rows i against each column tile, 0 above the diagonal
  float dec[OUT ? 4 : 1][4], lamo[OUT ? 4 : 1];
  if constexpr (OUT) {
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = 16 * (w - jt) + l16 - 4 * g4 - r;
        dec[jt][r] = n >= 0 ? sLam[n] * p.c1 : 0.0f;
      }
      lamo[jt] = sLam[16 * jt + l16 + p.off > LC ? LC : 16 * jt + l16 + p.off] * p.c2;
    }
  }

  fetch();
  while (true) {
    const int64_t left = c.b - c.a - done;
    const int len = (int)(left < LC ? left : LC);
    const bool first = done == 0, last = left <= LC;
    const int64_t row0 = rev ? c.b - 1 - done : c.a + done;
    const LaStretch now = c;

    // ---- tiles into LDS
#pragma unroll
    for (int u = 0; u < XU; ++u) {
      const int e = t + LT * u, at = e / (DX / 8) * XP + e % (DX / 8) * 8;
      if constexpr (OUT) *reinterpret_cast<uint4*>(sX + at) = rx[u];
      *reinterpret_cast<uint4*>(sY + at) = ry[u];
    }
#pragma unroll
    for (int u = 0; u < ZU; ++u) {
      const int e = t + LT * u;
      *reinterpret_cast<uint4*>(sZ + e / (NZ / 8) * ZP + e % (NZ / 8) * 8) = rz[u];
    }

    // ---- the state that enters a stretch
    if (first) {
      const float* src = now.starts ? p.sin : OUT ? p.seg : nullptr;
      const int64_t at = now.starts ? ((int64_t)now.n * a.H + h) * a.KV : segat;
      const int sr = now.starts ? p.sr : DZ, sc = now.starts ? p.sc : 1;
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 16 * dt + 4 * g4 + r;
            S[dt][ct][r] = src ? src[at + d * sr + (col + 16 * ct) * sc] : 0.0f;
            if constexpr (DG) Rs[dt][ct][r] = !now.starts && OUT ? p.seg[rat + segat + d * DZ + col + 16 * ct] : 0.0f;
          }
    }

    // ---- the next step, and its rows while this one runs
    bool more = true;
    done += LC;
    if (last) {
      done = 0;
      more = false;
      if (OUT) {
        int n = now.n;
        while (true) {  // the next sequence with tokens in this segment
          n += rev ? -1 : 1;
          if (n < 0 || n >= a.ax.N) break;
          if (rev ? la_end(a.ax, n, R) <= sg.p0 : axis_start(a.ax, n) >= sg.p1) break;
          place(n);
          if (c.a < c.b) {
            more = true;
            break;
          }
        }
      }
    }
    __syncthreads();
    if (more) fetch();

    if constexpr (OUT) {
      // ---- pairs: rows i of this wave, (y x^T)[j][i] with 4 consecutive j a lane
      bf16x8 xb[NKB];
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb)
        xb[kb] = *reinterpret_cast<const bf16x8*>(sX + (16 * w + l16) * XP + 32 * kb + 8 * g4);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > (w | 1)) break;
        float v[4] = {0.f, 0.f, 0.f, 0.f}, vn[4] = {0.f, 0.f, 0.f, 0.f};
        if (jt <= w) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < NKB; ++kb)
            acc = mfma_bf16(*reinterpret_cast<const bf16x8*>(sY + (16 * jt + l16) * XP + 32 * kb + 8 * g4), xb[kb], acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int n = 16 * (w - jt) + l16 - 4 * g4 - r;
            v[r] = n >= 0 ? acc[r] * dec[jt][r] : 0.0f;
            vn[r] = v[r] * (float)n;
          }
        }
#pragma unroll
        for (int m = 0; m < NP; ++m) {
          reinterpret_cast<bf16x4*>(&sP[m][2 * w + (jt >> 1)][lane])[jt & 1] = cut_part(v);
          if constexpr (DG) reinterpret_cast<bf16x4*>(&sP[NP + m][2 * w + (jt >> 1)][lane])[jt & 1] = cut_part(vn);
        }
      }
    }

    // ---- the entering state's part of the outputs: out^T[c][i] = S^T x^T
    f32x4 O[OUT ? 4 : 1][NCT], On[DG && OUT ? 4 : 1][DG && OUT ? NCT : 1];
    if constexpr (OUT) {
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
          O[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
          if constexpr (DG) On[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb) {
        bf16x8 sp[NCT][NP], rp[DG ? NCT : 1][NP];
        auto cut = [&](f32x4 u, f32x4 v, bf16x8 (&o)[NP]) {
#pragma unroll
          for (int m = 0; m < NP; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              o[m][r] = (__bf16)u[r];
              u[r] -= (float)o[m][r];
              o[m][4 + r] = (__bf16)v[r];
              v[r] -= (float)o[m][4 + r];
            }
        };
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
          cut(S[2 * kb][ct], S[2 * kb + 1][ct], sp[ct]);
          if constexpr (DG) cut(Rs[2 * kb][ct], Rs[2 * kb + 1][ct], rp[ct]);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const uint16_t* q = sX + (16 * it + l16) * XP + 32 * kb + 4 * g4;
          const bf16x8 xf = join(*reinterpret_cast<const uint2*>(q), *reinterpret_cast<const uint2*>(q + 16));
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int m = 0; m < NP; ++m) {
              O[it][ct] = mfma_bf16(sp[ct][m], xf, O[it][ct]);
              if constexpr (DG) On[it][ct] = mfma_bf16(rp[ct][m], xf, On[it][ct]);
            }
        }
      }
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (DG) On[it][ct][r] = (On[it][ct][r] + O[it][ct][r] * (float)(16 * it + l16 + 1)) * lamo[it];
            O[it][ct][r] *= lamo[it];
          }
    }

    // ---- the state: decayed, plus y^T (z times its decay), z's product in three bf16 parts
    {
      const float full = sLam[len];
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (DG) Rs[dt][ct][r] = full * (Rs[dt][ct][r] + (float)len * S[dt][ct][r]);
            S[dt][ct][r] *= full;
          }
    }
    bf16x8 zr[2][NCT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int jr = 32 * ks + 4 * g4 + (l16 >> 2);
      bf16x8 zw[NCT][3], zn[DG ? NCT : 1][3];
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) {
        const uint16_t* q = sZ + jr * ZP + w * ZW + 16 * ct + 4 * (l16 & 3);
        zr[ks][ct] = join(tr_read(q), tr_read(q + 16 * ZP));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = 32 * ks + 4 * g4 + (e & 3) + 16 * (e >> 2);
          const int n = len - j - p.off;  // len - 1 - j + (1 - off)
          const float f = (n >= 0 ? sLam[n] : 0.0f) * p.c3 * (float)zr[ks][ct][e];
          auto cut3 = [&](float v, bf16x8* o) {
            o[0][e] = (__bf16)v;
            v -= (float)o[0][e];
            o[1][e] = (__bf16)v;
            o[2][e] = (__bf16)(v - (float)o[1][e]);
          };
          cut3(f, zw[ct]);
          if constexpr (DG) cut3(f * (float)(n >= 0 ? n : 0), zn[ct]);
        }
      }
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt) {
        const uint16_t* q = sY + jr * XP + 16 * dt + 4 * (l16 & 3);
        const bf16x8 yt = join(tr_read(q), tr_read(q + 16 * XP));
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            S[dt][ct] = mfma_bf16(yt, zw[ct][m], S[dt][ct]);
            if constexpr (DG) Rs[dt][ct] = mfma_bf16(yt, zn[ct][m], Rs[dt][ct]);
          }
      }
    }

    // ---- the pairs' part of the outputs
    if constexpr (OUT) {
      __syncthreads();
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ks = 0; ks <= it >> 1; ++ks) {
#pragma unroll
          for (int m = 0; m < NP; ++m) {
            const bf16x8 pm = __builtin_bit_cast(bf16x8, sP[m][2 * it + ks][lane]);
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) O[it][ct] = mfma_bf16(zr[ks][ct], pm, O[it][ct]);
            if constexpr (DG) {
              const bf16x8 nm = __builtin_bit_cast(bf16x8, sP[NP + m][2 * it + ks][lane]);
#pragma unroll
              for (int ct = 0; ct < NCT; ++ct) On[it][ct] = mfma_bf16(zr[ks][ct], nm, On[it][ct]);
            }
          }
        }
      float sum = 0.0f;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int i = 16 * it + l16;
        if (i < len) {
          const int64_t row = rev ? row0 - i : row0 + i;
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            const int at = slice * NZ + w * ZW + 16 * ct + 4 * g4;
            bf16x4 o;
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = (__bf16)O[it][ct][r];
            *reinterpret_cast<bf16x4*>(p.out + (row * a.H + h) * DZ + at) = o;
            if constexpr (DG) {
              const bf16x4 q = *reinterpret_cast<const bf16x4*>(p.w + row * p.ws + h * p.wh + at);
#pragma unroll
              for (int r = 0; r < 4; ++r) sum += On[it][ct][r] * (float)q[r];
            }
          }
        }
      }
      if constexpr (DG) dg += sum;
    }

    // ---- the state that leaves a stretch
    if (last) {
      float* dst = OUT ? (now.ends ? p.sout : nullptr) : p.seg;
      const int64_t at = OUT ? ((int64_t)now.n * a.H + h) * a.KV : segat;
      const int sr = OUT ? p.sr : DZ, sc = OUT ? p.sc : 1;
      float sum = 0.0f;
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 16 * dt + 4 * g4 + r, cc = col + 16 * ct;
            if (dst) dst[at + d * sr + cc * sc] = S[dt][ct][r];
            if constexpr (DG) {
              if (!OUT) p.seg[rat + segat + d * DZ + cc] = Rs[dt][ct][r];
              if (OUT && now.ends && p.rend) sum += Rs[dt][ct][r] * p.rend[at + d * sr + cc * sc];
            }
          }
      if constexpr (DG) dg += sum;
    }
    if (!more) break;
    __syncthreads();
  }

  if constexpr (DG && OUT) {
    float f = (float)dg;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) f += __shfl_xor(f, m);
    if (lane == 0) sRed[w] = f;
    __syncthreads();
    if (t == 0) p.part[((int64_t)h * a.nseg + s) * a.slices + slice] = sRed[0] + sRed[1] + sRed[2] + sRed[3];
  }
}

// The states that enter the segments, from those that each of them leaves by
// itself: the stretch that goes on beyond segment s starts inside it, or
// entered it and crosses it whole.
template <bool DG>
__global__ void __launch_bounds__(LT) la_join_kernel(const LaArgs a) {
  const int per = a.KV / (LT * 4);  // workgroups per head
  const int h = blockIdx.x / per % a.H;
  const LaPass& p = a.p[blockIdx.x / per / a.H];
  const int64_t e = (int64_t)h * a.KV + ((int64_t)(blockIdx.x % per) * LT + threadIdx.x) * 4;
  const int64_t step = (int64_t)a.H * a.KV;
  const int64_t R = axis_rows(a.ax);
  const float gh = a.g[h];
  float4 E = make_float4(0.f, 0.f, 0.f, 0.f), Q = E;
  for (int k = 0; k < a.nseg; ++k) {
    const int s = p.rev ? a.nseg - 1 - k : k;
    float4* at = reinterpret_cast<float4*>(p.seg + s * step + e);
    float4* rat = reinterpret_cast<float4*>(p.seg + (a.nseg + s) * step + e);
    const LaSeg sg = la_seg(a, s, R);
    bool on = false, whole = false;
    if (sg.p0 < sg.p1) {
      const int64_t n = axis_owner(a.ax, p.rev ? sg.p0 : sg.p1 - 1);
      const int64_t bos = axis_start(a.ax, n), eos = la_end(a.ax, n, R);
      on = p.rev ? bos < sg.p0 : eos > sg.p1;
      whole = p.rev ? eos > sg.p1 : bos < sg.p0;
    }
    float4 own = make_float4(0.f, 0.f, 0.f, 0.f), rown = own;
    if (on) {
      own = *at;
      if (DG) rown = *rat;
    }
    *at = E;
    if (DG) *rat = Q;
    const float f = whole && on ? la_pow(gh, (double)(sg.p1 - sg.p0)) : 0.0f, m = (float)(sg.p1 - sg.p0);
    if (DG) {
      Q.x = f != 0.0f ? f * (Q.x + m * E.x) + rown.x : rown.x;
      Q.y = f != 0.0f ? f * (Q.y + m * E.y) + rown.y : rown.y;
      Q.z = f != 0.0f ? f * (Q.z + m * E.z) + rown.z : rown.z;
      Q.w = f != 0.0f ? f * (Q.w + m * E.w) + rown.w : rown.w;
    }
    E.x = whole && on ? f * E.x + own.x : own.x;
    E.y = whole && on ? f * E.y + own.y : own.y;
    E.z = whole && on ? f * E.z + own.z : own.z;
    E.w = whole && on ? f * E.w + own.w : own.w;
  }
}

// dg of each head: its workgroups' parts, in order.
__global__ void __launch_bounds__(64) la_reduce_kernel(const float* part, float* dg, int count) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += 64) sum += part[(int64_t)blockIdx.x * count + i];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
  if (threadIdx.x == 0) dg[blockIdx.x] = (float)sum;
}

// Token by token, for decoding: bound by the state's traffic (4 K V bytes read
// and written a sequence and head).  A workgroup has one sequence and head;
// V / 4 lanes hold one row of the state, four columns each, and every thread's
// rows are asked for before the first token.
struct LaStep {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const float* g;
  const float* init;
  float* fin;
  int64_t qs, qh, ks, kh, vs, vh;
  float scale;
  int T, H;
};
template <int K, int V>
__global__ void __launch_bounds__(LT) la_step_kernel(const LaStep a) {
  constexpr int LR = V / 4, RG = LT / LR, NR = K / RG;  // lanes a row, rows at a time, rows a thread
  __shared__ float sO[4][V];
  const int t = threadIdx.x, c4 = t % LR * 4, rg = t / LR, w = t >> 6;
  const int h = blockIdx.x % a.H;
  const int64_t b = blockIdx.x / a.H;
  const int64_t st = (int64_t)blockIdx.x * K * V;
  float4 S[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r)
    S[r] = a.init ? *reinterpret_cast<const float4*>(a.init + st + (rg + RG * r) * V + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float f = expf(a.g[h]);
  for (int i = 0; i < a.T; ++i) {
    const int64_t row = b * a.T + i;
    const uint16_t* k = a.k + row * a.ks + h * a.kh;
    const uint16_t* q = a.q + row * a.qs + h * a.qh;
    float v[4], o[4] = {0.f, 0.f, 0.f, 0.f};
    widen4(*reinterpret_cast<const uint2*>(a.v + row * a.vs + h * a.vh + c4), v);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float kd = __uint_as_float((uint32_t)k[rg + RG * r] << 16), qd = __uint_as_float((uint32_t)q[rg + RG * r] << 16);
      S[r].x = f * S[r].x + kd * v[0];
      S[r].y = f * S[r].y + kd * v[1];
      S[r].z = f * S[r].z + kd * v[2];
      S[r].w = f * S[r].w + kd * v[3];
      o[0] += qd * S[r].x;
      o[1] += qd * S[r].y;
      o[2] += qd * S[r].z;
      o[3] += qd * S[r].w;
    }
#pragma unroll
    for (int m = 32; m >= LR; m >>= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], m);
    if ((t & 63) < LR) *reinterpret_cast<float4*>(&sO[w][c4]) = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (t < LR) {
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = a.scale * (sO[0][c4 + e] + sO[1][c4 + e] + sO[2][c4 + e] + sO[3][c4 + e]);
      store4(reinterpret_cast<__bf16*>(a.out) + (row * a.H + h) * V + c4, s);
    }
    __syncthreads();
  }
  if (a.fin) {
#pragma unroll
    for (int r = 0; r < NR; ++r) *reinterpret_cast<float4*>(a.fin + st + (rg + RG * r) * V + c4) = S[r];
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// How a sweep over `blocks` blocks of `block` tokens is cut.  Each of its
// blocks' heads is a chain of steps; with few chains the blocks are cut into
// segments, whose entering states cost another pass over y and z.
struct LaPlan {
  int zw, slices, spb;
  int64_t L, nseg;
};
LaPlan la_plan(int64_t blocks, int64_t block, int64_t H, int64_t DZ, int64_t passes) {
  LaPlan pl;
  pl.zw = 16;
  pl.slices = (int)(DZ / 64);
  const int64_t chains = blocks * H * pl.slices * passes;
  int64_t spb = 1;
  if (chains < kLaEnough) {
    spb = (kLaWant + chains - 1) / chains;
    const int64_t most = (block + kLaMinSeg - 1) / kLaMinSeg;
    spb = spb < most ? spb : most;
    spb = spb < 1 ? 1 : spb;
  }
  pl.L = ((block + spb - 1) / spb + LC - 1) / LC * LC;
  pl.L = pl.L < LC ? LC : pl.L;
  pl.spb = (int)((block + pl.L - 1) / pl.L);
  pl.spb = pl.spb < 1 ? 1 : pl.spb;
  pl.nseg = blocks * pl.spb;
  return pl;
}

// Bytes of the states of a sweep's segments, at most.  Only sweeps of fewer
// than kLaEnough chains are cut, into fewer than kLaWant + kLaEnough pieces in all.
size_t la_states_bytes(int64_t H, int64_t K, int64_t V) {
  return H < kLaEnough ? (size_t)((kLaWant + kLaEnough) * K * V) * sizeof(float) : 0;
}
// Bytes of the decay gradient's parts, for at most N blocks of the axis.
size_t la_part_bytes(int64_t N, int64_t H) {
  return align256((size_t)(N * H * 2 + kLaWant + kLaEnough) * sizeof(float));
}

kda_status_t la_check(const void* q, int64_t qs, int64_t qh, const void* k, int64_t ks, int64_t kh, const void* v,
                      int64_t vs, int64_t vh, const float* g, float scale, const int32_t* cu, int64_t B, int64_t T,
                      int64_t H, int64_t K, int64_t V, int64_t N) {
  if (B < 1 || T < 0 || H < 1 || K < 1 || V < 1 || N < 1) return KDA_ERR_INVALID;
  if (cu ? B != 1 : N != B) return KDA_ERR_INVALID;
  if ((K != 64 && K != 128) || (V != 64 && V != 128)) return KDA_ERR_UNSUPPORTED;
  if (H > 1 << 20 || N > 1 << 30 || !fits(B, T, kMaxElements) || !fits(B * T, H * 128, kMaxElements) ||
      !fits(N, H * 128 * 128, kMaxElements) || (cu && T >= (int64_t)1 << 31))
    return KDA_ERR_INVALID;
  if (!(scale - scale == 0.0f)) return KDA_ERR_INVALID;  // NaN or infinite
  if (!g || (B * T > 0 && (!q || !k || !v))) return KDA_ERR_INVALID;
  if (!mix_strides_ok(qs, qh) || !mix_strides_ok(ks, kh) || !mix_strides_ok(vs, vh)) return KDA_ERR_INVALID;
  if (!aligned_all(16, {q, k, v}) || !aligned(g, 4)) return KDA_ERR_INVALID;
  return KDA_SUCCESS;
}

template <int DX, bool DG>
kda_status_t la_run(LaArgs& a, const LaPlan& pl, bool empties, hipStream_t st) {
  const int64_t groups = (a.items + 7) / 8 * 8 * a.slices * a.passes;
  const int64_t more = empties ? (a.ax.N < 1024 ? a.ax.N : 1024) : 0;
  if (groups + more > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  a.main = groups;
  if (a.spb > 1) {  // otherwise every segment starts at a sequence's start
    kda_status_t s = launch(&la_sweep_kernel<DX, 16, false, DG>, groups, LT, st, "linear attention segments", a);
    if (s != KDA_SUCCESS) return s;
    s = launch(&la_join_kernel<DG>, (int64_t)a.passes * a.H * (a.KV / (LT * 4)), LT, st, "linear attention join", a);
    if (s != KDA_SUCCESS) return s;
  }
  return launch(&la_sweep_kernel<DX, 16, true, DG>, groups + more, LT, st, "linear attention", a);
}
template <bool DG>
kda_status_t la_sweep(LaArgs& a, int64_t DX, const LaPlan& pl, bool empties, hipStream_t st) {
  return DX == 128 ? la_run<128, DG>(a, pl, empties, st) : la_run<64, DG>(a, pl, empties, st);
}

// The arguments of a sweep of `passes` passes with DZ channels of z.
LaPlan la_common(LaArgs& a, const float* g, const int32_t* cu, int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                 int64_t N, int64_t DZ, int passes, unsigned flags) {
  const LaPlan pl = la_plan(B, T, H, DZ, passes);
  a = LaArgs{};
  a.ax = make_axis(cu, T, B * T, N);
  a.g = g;
  a.block = T;
  a.L = pl.L;
  a.spb = pl.spb;
  a.nseg = (int)pl.nseg;
  a.H = (int)H;
  a.KV = (int)(K * V);
  a.slices = pl.slices;
  a.passes = passes;
  a.items = pl.nseg * H;
  a.zero_rest = flags & FLAG_ZERO_REST ? 1 : 0;
  return pl;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_la_workspace_size(int64_t T_total, int64_t H, int64_t K, int64_t V) {
  if (T_total < 0 || H < 1 || H > 1 << 20 || (K != 64 && K != 128) || (V != 64 && V != 128) ||
      !fits(T_total, H * 128, kMaxElements))
    return 0;
  return 256 + la_states_bytes(H, K, V);
}

kda_status_t kda_la_fwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                        int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                        const float* log_decay, float scale, void* out, void* workspace, size_t workspace_bytes,
                        const float* initial_state, float* final_state, const int32_t* cu_seqlens, int64_t B, int64_t T,
                        int64_t H, int64_t K, int64_t V, int64_t N, unsigned flags, void* stream) {
  kda_status_t s = la_check(q, q_stride, q_head_stride, k, k_stride, k_head_stride, v, v_stride, v_head_stride,
                            log_decay, scale, cu_seqlens, B, T, H, K, V, N);
  if (s != KDA_SUCCESS) return s;
  if (flags & ~FLAG_ZERO_REST) return KDA_ERR_INVALID;
  if (B * T > 0 && !out) return KDA_ERR_INVALID;
  if (!aligned_all(16, {out, workspace, initial_state, final_state})) return KDA_ERR_INVALID;
  if (same(q, out) || same(k, out) || same(v, out) || same(initial_state, final_state)) return KDA_ERR_INVALID;
  if (!workspace || workspace_bytes < kda_la_workspace_size(B * T, H, K, V)) return KDA_ERR_WORKSPACE;
  LaArgs a;
  const LaPlan pl = la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, V, 1, flags);
  LaPass& p = a.p[0];
  p.x = static_cast<const uint16_t*>(q);
  p.y = static_cast<const uint16_t*>(k);
  p.z = static_cast<const uint16_t*>(v);
  p.out = static_cast<uint16_t*>(out);
  p.sin = initial_state;
  p.sout = final_state;
  p.seg = static_cast<float*>(workspace);
  p.xs = q_stride, p.xh = q_head_stride, p.ys = k_stride, p.yh = k_head_stride, p.zs = v_stride, p.zh = v_head_stride;
  p.sr = (int)V, p.sc = 1;
  p.off = 1;
  p.c1 = p.c2 = scale;
  p.c3 = 1.0f;
  return la_sweep<false>(a, K, pl, final_state && (cu_seqlens || T == 0), reinterpret_cast<hipStream_t>(stream));
}

size_t kda_la_bwd_workspace_size(int64_t T_total, int64_t H, int64_t K, int64_t V, int64_t N) {
  if (!kda_la_workspace_size(T_total, H, K, V) || N < 1 || N > 1 << 30) return 0;
  return 256 + 4 * la_states_bytes(H, K, V) + la_part_bytes(N, H);
}

kda_status_t kda_la_bwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                        int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                        const float* log_decay, float scale, const void* d_out, const float* d_final, void* dq, void* dk,
                        void* dv, float* d_log_decay, float* d_initial_state, void* workspace, size_t workspace_bytes,
                        const float* initial_state, const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t H,
                        int64_t K, int64_t V, int64_t N, unsigned flags, void* stream) {
  kda_status_t s = la_check(q, q_stride, q_head_stride, k, k_stride, k_head_stride, v, v_stride, v_head_stride,
                            log_decay, scale, cu_seqlens, B, T, H, K, V, N);
  if (s != KDA_SUCCESS) return s;
  if (flags & ~FLAG_ZERO_REST) return KDA_ERR_INVALID;
  if (B * T > 0 && (!d_out || !dq || !dk || !dv)) return KDA_ERR_INVALID;
  if (!aligned_all(16, {d_out, dq, dk, dv, workspace, initial_state, d_final, d_initial_state}) ||
      !aligned(d_log_decay, 4))
    return KDA_ERR_INVALID;
  for (const void* o : {(const void*)dq, (const void*)dk, (const void*)dv})
    for (const void* i : {q, k, v, d_out})
      if (same(o, i)) return KDA_ERR_INVALID;
  if (same(dq, dk) || same(dq, dv) || same(dk, dv) || same(d_initial_state, d_final) ||
      same(d_initial_state, initial_state) || same(d_log_decay, log_decay))
    return KDA_ERR_INVALID;
  if (!workspace || workspace_bytes < kda_la_bwd_workspace_size(B * T, H, K, V, N)) return KDA_ERR_WORKSPACE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const size_t sb = la_states_bytes(H, K, V);
  char* ws = static_cast<char*>(workspace);
  const uint16_t *qp = static_cast<const uint16_t*>(q), *kp = static_cast<const uint16_t*>(k),
                 *vp = static_cast<const uint16_t*>(v), *dp = static_cast<const uint16_t*>(d_out);
  const bool none = cu_seqlens || T == 0;  // there may be sequences without tokens

  // dq: of do, v, k; the state is S^T
  LaArgs a;
  LaPlan pl = la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, K, 1, flags);
  LaPass& p = a.p[0];
  p.x = dp, p.xs = H * V, p.xh = V;
  p.y = vp, p.ys = v_stride, p.yh = v_head_stride;
  p.z = kp, p.zs = k_stride, p.zh = k_head_stride;
  p.out = static_cast<uint16_t*>(dq);
  p.sin = initial_state;
  p.sr = 1, p.sc = (int)V;
  p.off = 1;
  p.c1 = p.c2 = scale;
  p.c3 = 1.0f;
  p.seg = reinterpret_cast<float*>(ws);
  if (d_log_decay) {
    p.w = qp, p.ws = q_stride, p.wh = q_head_stride;
    p.rend = d_final;
    p.part = reinterpret_cast<float*>(ws + 4 * sb);
    s = la_sweep<true>(a, V, pl, false, st);
    if (s != KDA_SUCCESS) return s;
    s = launch(&la_reduce_kernel, H, 64, st, "linear attention decay", (const float*)p.part, d_log_decay,
               (int)(a.nseg * a.slices));
  } else {
    s = la_sweep<false>(a, V, pl, false, st);
  }
  if (s != KDA_SUCCESS) return s;

  // dv: of k, q, do backwards in time, the state is dS; dk: of v, do, q, the state is dS^T
  LaPass pv{}, pk{};
  pv.x = kp, pv.xs = k_stride, pv.xh = k_head_stride;
  pv.y = qp, pv.ys = q_stride, pv.yh = q_head_stride;
  pv.z = dp, pv.zs = H * V, pv.zh = V;
  pv.out = static_cast<uint16_t*>(dv);
  pv.sin = d_final;
  pv.sout = d_initial_state;
  pv.sr = (int)V, pv.sc = 1;
  pk.x = vp, pk.xs = v_stride, pk.xh = v_head_stride;
  pk.y = dp, pk.ys = H * V, pk.yh = V;
  pk.z = qp, pk.zs = q_stride, pk.zh = q_head_stride;
  pk.out = static_cast<uint16_t*>(dk);
  pk.sin = d_final;
  pk.sr = 1, pk.sc = (int)V;
  for (LaPass* x : {&pv, &pk}) {
    x->rev = 1;
    x->c1 = x->c3 = scale;
    x->c2 = 1.0f;
  }
  pv.seg = reinterpret_cast<float*>(ws + 2 * sb);
  pk.seg = reinterpret_cast<float*>(ws + 3 * sb);
  if (K == V) {  // one launch: both read q and do
    pl = la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, V, 2, flags);
    a.p[0] = pv;
    a.p[1] = pk;
    return la_sweep<false>(a, K, pl, d_initial_state && none, st);
  }
  pl = la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, V, 1, flags);
  a.p[0] = pv;
  s = la_sweep<false>(a, K, pl, d_initial_state && none, st);
  if (s != KDA_SUCCESS) return s;
  pl = la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, K, 1, flags);
  a.p[0] = pk;
  return la_sweep<false>(a, V, pl, false, st);
}

kda_status_t kda_la_step(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                         int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                         const float* log_decay, float scale, void* out, const float* initial_state, float* final_state,
                         int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, void* stream) {
  const kda_status_t s = la_check(q, q_stride, q_head_stride, k, k_stride, k_head_stride, v, v_stride, v_head_stride,
                                  log_decay, scale, nullptr, B, T, H, K, V, B);
  if (s != KDA_SUCCESS) return s;
  if (B * T > 0 && !out) return KDA_ERR_INVALID;
  if (!aligned_all(16, {out, initial_state, final_state})) return KDA_ERR_INVALID;
  if (same(q, out) || same(k, out) || same(v, out)) return KDA_ERR_INVALID;
  if (T > 1 << 20 || B * H > ((int64_t)1 << 31) - 1) return KDA_ERR_INVALID;
  LaStep a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
           static_cast<uint16_t*>(out), log_decay, initial_state, final_state, q_stride, q_head_stride, k_stride,
           k_head_stride, v_stride, v_head_stride, scale, (int)T, (int)H};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (K == 128)
    return V == 128 ? launch(&la_step_kernel<128, 128>, B * H, LT, st, "linear attention step", a)
                    : launch(&la_step_kernel<128, 64>, B * H, LT, st, "linear attention step", a);
  return V == 128 ? launch(&la_step_kernel<64, 128>, B * H, LT, st, "linear attention step", a)
                  : launch(&la_step_kernel<64, 64>, B * H, LT, st, "linear attention step", a);
}

}  // extern "C"
