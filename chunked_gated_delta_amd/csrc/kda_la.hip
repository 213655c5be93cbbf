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
// and the pairs within it give sum_{i>j} (i - j) a^{i-j} (do_i.v_j)(q_i.k_j), the
// fp32 scores of the sweep times those of q and k.  No difference of large sums
// is taken (sum t (q_t.dq_t - k_t.dk_t) would be one).
//
// A workgroup of four waves takes one head, one slice of z's channels and a
// segment of the packed token axis, 64 tokens a step.  Each wave owns 16
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
// would add errors as large as the output's own rounding; dropping the second
// parts would save 9 % of the time.
//
// What bounds it.  Where chains are few, the steps: 2 x 4096 tokens are 64 steps
// one after another whatever the card's width, and a step of two waves a SIMD (242
// registers, 58 KB of LDS) has two barriers.  Where they are many, memory: a prompt
// of 32768 tokens of 96 heads of 128 takes 0.92 ms in the second pass, in which the
// L2s fetch 2.8 to 3.5 GB (its arrays are 2.4: the slices of z read the same rows of
// x and y) and write 0.8: 4.0 to 4.6 TB/s, where a copy reaches 5.1 (matrix cores
// busy 38 % of the cycles, with five other vector instructions for each of theirs).
// The pass before it, that makes the segments' states, takes 0.28 ms, their join
// 0.01.  What cutting costs is that pass: unsplit there were 192 workgroups for 512
// places.

#include "../../include/kda.h"
#include "kda_mix.h"

namespace kda {
namespace {

constexpr int LC = 64;  // tokens of a step
constexpr int LT = 256;  // threads
// How sweeps are cut.  Measured, us, heads of 128: forward of 32768 tokens of 96
// heads, and of 8192 of 32; training, all gradients, on 2 x 4096 tokens of 12, and on
// 4 x 2048 of 16.  As it is: 1267, 118, 291, 342.
constexpr int64_t kLaWant = 512;    // workgroups at a time, two per CU (256: 1491, 145, 296, 360; 1024: 1269, 138, 322, 389)
constexpr int64_t kLaMost = 1024;   // workgroups that cutting leads to at most (512: 1382, 119, 289, 344; 2048: 1291, 120, 301, 345)
constexpr int64_t kLaMinSteps = 4;  // steps of a segment at least: 2 and 8 took the same time; it bounds the workspace
constexpr int64_t kLaAround = 3;    // steps that a workgroup's beginning and end cost (0: 1271, 119, 322, 357; 8: 1266, 119, 291, 346)

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

// Element (row, col) of a tile of W columns in LDS: rows are not padded; their
// 16-byte pieces are permuted by the row instead, so that 16 rows of one piece
// (MFMA rows) and 8 rows of two neighbouring ones (transposing reads) each meet
// all 64 banks once.  Padded rows can have one of the two, and cost half of the
// LDS time in the other.
template <int W>
__device__ __forceinline__ int at_lds(int row, int col) {
  static_assert(W == 64 || W == 128, "pieces of 16 bytes");
  const int f = W == 128 ? (row & 7) << 1 | (row >> 3 & 1) : (row >> 1 & 3) << 1 | (row >> 3 & 1);
  return row * W + (((col >> 3) ^ f) << 3) + (col & 7);
}

// A step's rows of one array: W channels of 64 tokens, asked for in 16-byte
// pieces by the workgroup.  Token i of the step is row i behind `p`, or, back in
// time, row 63 - i, so that every offset is positive; a step moves p by 64 rows.
template <int W>
struct LaRows {
  static constexpr int PR = LT / (W / 8), U = LC / PR;  // rows a load covers, loads
  uint4 r[U];
  const uint16_t* p;  // of the step to be fetched next
  int at, ts;         // this thread's offset in bytes in the first piece; bytes between tokens
  __device__ __forceinline__ void start(int token_stride, int rev) {
    const int rt = threadIdx.x / (W / 8);
    ts = token_stride * 2;
    at = (rev ? PR - 1 - rt : rt) * ts + (int)(threadIdx.x % (W / 8)) * 16;
  }
  __device__ __forceinline__ void seek(const uint16_t* base, int64_t row0, int rev) {
    p = base + (rev ? row0 - (LC - 1) : row0) * (ts >> 1);
  }
  // Rows from len on are zeros: their offset is behind the descriptor's end, so
  // that no load stands in a branch of its own.
  __device__ __forceinline__ void load(int len, int rev) {
    const __amdgpu_buffer_rsrc_t d = buf(p, 0x7fffffffu);
    const int rt = threadIdx.x / (W / 8);
#pragma unroll
    for (int u = 0; u < U; ++u)
      r[u] = bload<uint4>(d, rt + PR * u < len ? at : (int)0x80000000, (rev ? U - 1 - u : u) * PR * ts);
    p += (rev ? -LC : LC) * (int64_t)(ts >> 1);
  }
  __device__ __forceinline__ void store(uint16_t* lds) const {
    static_assert(PR % 16 == 0, "rows whose pieces are permuted alike");
    uint16_t* to = lds + at_lds<W>(threadIdx.x / (W / 8), threadIdx.x % (W / 8) * 8);
#pragma unroll
    for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(to + u * PR * W) = r[u];
  }
};

__device__ __forceinline__ bf16x8 cut8(float (&x)[8]) {  // the next bf16 part of eight values
  const uint32_t a = cut2(x[0], x[1]), b = cut2(x[2], x[3]), c = cut2(x[4], x[5]), d = cut2(x[6], x[7]);
  return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}

constexpr int kWaitLoads = 0x0f70;  // s_waitcnt vmcnt(0) alone

// A value that is computed where it stands: without this, the addresses of what
// is seldom done are formed once, before the loop, and hold its registers.
template <typename X>
__device__ __forceinline__ X here(X x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float uniform(float x) { return __int_as_float(uniform(__float_as_int(x))); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}

// With the decay's gradient the second state leaves one wave a SIMD (370 registers):
// 1.51 ms over 69141 packed tokens of 32 heads where the plain sweep takes 0.60.
// Instead of it, the states that enter all steps can be left in memory for the dk
// sweep, which then sums a^C <S_in, dS_out>; with two waves a SIMD, the 2.2 GB
// written and read made it 1.30 ms, and the dk sweep 1.26 in place of 0.67.
template <int DX, bool OUT, bool DG>
__global__ void __launch_bounds__(LT, DG && OUT ? 1 : 2) la_sweep_kernel(const LaArgs a) {
  constexpr int NZ = 64, NDT = DX / 16, NKB = DX / 32;  // channels of a slice of z; tiles, blocks of the state's rows
  constexpr int NP = DG ? 3 : 2;  // bf16 parts of entering states
  __shared__ __align__(16) uint16_t sX[OUT ? LC * DX : 8], sY[LC * DX], sZ[LC * NZ];
  __shared__ uint4 sP[OUT ? 2 : 1][OUT ? 8 : 1][64];  // pair weights as B operands, two parts
  __shared__ __align__(16) uint16_t sQ[OUT && DG ? LC * NZ : 8];  // the rows that the decay's gradient is dotted with
  __shared__ float sLam[LC + 1];
  __shared__ __align__(16) float sW[LC];  // decays of z's rows up to the step's end, times c3
  __shared__ float sRed[4];

  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6), l16 = lane & 15, g4 = lane >> 4;
  const int64_t R = uniform(axis_rows(a.ax));

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
  // Nothing keeps them in step, so that the L2 serves only part of what they share:
  // two slices fetch 1.2 to 1.4 times their three arrays, the four workgroups of dk
  // and dv 2.1 times their four (2.5 would be without any sharing).
  const int id = blockIdx.x;
  const int kinds = a.slices * a.passes;
  const int item = id / 8 / kinds * 8 + id % 8;
  if (item >= a.items) return;
  const int kind = id / 8 % kinds, slice = kind % a.slices;
  const LaPass& p = a.p[kind / a.slices];
  const int h = item % a.H, s = item / a.H;
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

  // ---- the first stretch.  OUT: all stretches of the segment in the sweep's
  // order; otherwise the one that goes on beyond the segment's end, if any.
  const bool tail = rev == (OUT ? 0 : 1);  // whether to begin at the segment's first row
  LaStretch c;
  auto place = [&](int n) {
    const int64_t bos = uniform(axis_start(a.ax, n)), eos = uniform(la_end(a.ax, n, R));
    c.n = n;
    c.a = bos > sg.p0 ? bos : sg.p0;
    c.b = eos < sg.p1 ? eos : sg.p1;
    c.starts = rev ? eos <= sg.p1 : bos >= sg.p0;
    c.ends = rev ? bos >= sg.p0 : eos <= sg.p1;
  };
  place(uniform(axis_owner(a.ax, tail ? sg.p0 : sg.p1 - 1)));
  if (!OUT && c.ends) return;
  if (c.a >= c.b) return;  // only where offsets break their contract
  // tokens of the stretch from the current step on; of the one whose rows are asked for
  int left = (int)(c.b - c.a), ahead = left;

  LaRows<DX> rx, ry;
  LaRows<NZ> rz, rq;
  if constexpr (OUT) rx.start((int)p.xs, rev);
  ry.start((int)p.ys, rev);
  rz.start((int)p.zs, rev);
  if constexpr (OUT && DG) rq.start((int)p.ws, rev);
  uint16_t* po = nullptr;  // the step's first token in the output
  const int os = a.H * DZ;  // elements a token
  const int o0 = (rev ? LC - 1 - l16 : l16) * os * 2 + 8 * g4, o1 = (rev ? -16 : 16) * os * 2;  // bytes: this lane, 16 tokens
  auto seek = [&]() {
    const int64_t row0 = rev ? c.b - 1 : c.a;
    if constexpr (OUT) rx.seek(p.x + h * p.xh, row0, rev);
    ry.seek(p.y + h * p.yh, row0, rev);
    rz.seek(p.z + h * p.zh + slice * NZ, row0, rev);
    if constexpr (OUT && DG) rq.seek(p.w + h * p.wh + slice * NZ, row0, rev);
  };
  auto fetch = [&]() {
    const int len = ahead < LC ? ahead : LC;
    if constexpr (OUT) rx.load(len, rev);
    ry.load(len, rev);
    rz.load(len, rev);
    if constexpr (OUT && DG) rq.load(len, rev);
  };
  int wlen = 0;  // the step length that sW belongs to
  auto stage = [&]() {  // the rows that have come, and the decays of their step, into LDS
    if constexpr (OUT) rx.store(sX);
    ry.store(sY);
    rz.store(sZ);
    if constexpr (OUT && DG) rq.store(sQ);
    const int len = ahead < LC ? ahead : LC;
    if (len != wlen) {  // seldom: steps are whole but for a stretch's last one
      wlen = len;
      const int n = len - t - p.off;  // len - 1 - j + (1 - off)
      if (t < LC) sW[t] = n >= 0 ? sLam[n] * p.c3 : 0.0f;
    }
  };

  seek();
  fetch();
  const float gh = a.g[h];
  if (t <= LC) sLam[t] = la_pow(gh, t);
  __syncthreads();

  f32x4 S[NDT], Rs[DG ? NDT : 1];
  double dg = 0.0;
  const int col = slice * NZ + 16 * w + l16;  // the lane's channel of z
  const int64_t segat = ((int64_t)s * a.H + h) * a.KV;
  const int64_t rat = (int64_t)a.nseg * a.H * a.KV;  // R's segments lie behind S's
  // a^{i-j} of the wave's 16 rows j: against the columns of its own tile (zero for
  // i < j), of the next one, and what is more for a tile further away (own: whether
  // it is its own); a^{i + off}
  float dec0[4], dec1[4], own[4], far[4], lamo[4];
  if constexpr (OUT) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = l16 - 4 * g4 - r;
      dec0[r] = n >= 0 ? sLam[n] * p.c1 : 0.0f;
      dec1[r] = sLam[16 + n] * p.c1;
      own[r] = r == w ? 1.0f : 0.0f;
      far[r] = r > w ? uniform(sLam[16 * (r - w - 1)]) : 0.0f;
      lamo[r] = sLam[16 * r + l16 + p.off] * p.c2;
    }
  }
  stage();
  __syncthreads();

  LaStretch now = c;
  bool first = true;
  while (true) {
    const int len = left < LC ? left : LC;
    const bool last = left <= LC;
    if (OUT && first) po = p.out + ((rev ? now.b - 1 : now.a) * a.H + h) * DZ + slice * NZ + 16 * w;

    // ---- the next step
    bool more = true;
    ahead = left - LC;
    if (last) {
      more = false;
      if (OUT) {
        int n = now.n;
        while (true) {  // the next sequence with tokens in this segment
          n += rev ? -1 : 1;
          if (n < 0 || n >= a.ax.N) break;
          if (rev ? uniform(la_end(a.ax, n, R)) <= sg.p0 : uniform(axis_start(a.ax, n)) >= sg.p1) break;
          place(n);
          if (c.a < c.b) {
            more = true;
            ahead = (int)(c.b - c.a);
            seek();
            break;
          }
        }
      }
    }

    // ---- the state that enters a stretch
    if (first) {
      const float* src = now.starts ? p.sin : OUT ? p.seg : nullptr;
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt) {
        S[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (DG) Rs[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (src) {
        const float* at = src + (now.starts ? ((int64_t)now.n * a.H + h) * a.KV : segat);
        const int sr = now.starts ? p.sr : DZ, sc = now.starts ? p.sc : 1;
        const int o = here(4 * g4 * sr + col * sc);
#pragma unroll
        for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            S[dt][r] = at[o + (16 * dt + r) * sr];
            if constexpr (DG && OUT)
              if (!now.starts) Rs[dt][r] = at[rat + o + (16 * dt + r) * sr];
          }
        // Waited for here: a wait behind the branch would be one for the loads
        // issued after it, on the usual path without these.
        __builtin_amdgcn_s_waitcnt(kWaitLoads);
      }
    }
    // Its rows come while this step runs.  Without a next step there are none,
    // but neither the loads nor what waits for them stands in a branch: where one
    // ends, registers would be waited for that other loads and stores hold up.
    if (!more) ahead = 0;
    fetch();

    // ---- the entering state's part of the outputs, out^T[c][i] = S^T x^T, and
    // the pairs, rows j of this wave: (y x^T)[j][i].  Both take x's rows in the
    // channel order of the state's registers.
    f32x4 O[OUT ? 4 : 1], On[DG && OUT ? 4 : 1];
    if constexpr (OUT) {
      f32x4 P[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) P[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto clear = [&](auto& o) {
#pragma unroll
        for (int it = 0; it < 4; ++it) o[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      };
      // 16 rows from row0, channels 32 kb + 4 g4 and 16 behind them
      const int at0 = at_lds<DX>(l16, 4 * g4);
      auto frag = [&](const uint16_t* tile, int row0, int kb) {
        return join(*reinterpret_cast<const uint2*>(tile + (at0 ^ 32 * kb) + row0 * DX),
                    *reinterpret_cast<const uint2*>(tile + (at0 ^ (32 * kb + 16)) + row0 * DX));
      };
      auto rows = [&](int kb, bf16x8 (&x)[4]) {
#pragma unroll
        for (int it = 0; it < 4; ++it) x[it] = frag(sX, 16 * it, kb);
      };
      auto cut = [&](const f32x4& u, const f32x4& v, bf16x8 (&o)[NP]) {
        float f[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int m = 0; m < NP; ++m) o[m] = cut8(f);
      };
      // Rows and state parts are one block of channels ahead of the products, so
      // that the parts are cut while products run.
      bf16x8 xf[2][4], yf[2], sp[2][NP], rp[DG ? 2 : 1][NP];
      clear(O);
      if constexpr (DG) clear(On);
      auto ready = [&](int kb) {
        rows(kb, xf[kb & 1]);
        yf[kb & 1] = frag(sY, 16 * w, kb);
      };
      auto parts = [&](int kb) {
        cut(S[2 * kb], S[2 * kb + 1], sp[kb & 1]);
        if constexpr (DG) cut(Rs[2 * kb], Rs[2 * kb + 1], rp[kb & 1]);
      };
      ready(0);
      __builtin_amdgcn_sched_barrier(0);
      parts(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb) {
        const int b = kb & 1;
        if (kb + 1 < NKB) {
          ready(kb + 1);
          parts(kb + 1);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) P[it] = mfma_bf16(yf[b], xf[b][it], P[it]);
#pragma unroll
        for (int m = 0; m < NP; ++m)
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            O[it] = mfma_bf16(sp[b][m], xf[b][it], O[it]);
            if constexpr (DG) On[it] = mfma_bf16(rp[b][m], xf[b][it], On[it]);
          }
        // reads first, then products with the cutting between them
        if (kb + 1 < NKB) __builtin_amdgcn_sched_group_barrier(0x100, 10, 0);
#pragma unroll
        for (int i = 0; i < 4 + (DG ? 8 : 4) * NP; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      f32x4 A[DG ? 4 : 1];  // (z q^T)[j][i] over this slice's channels
      if constexpr (DG) {
#pragma unroll
        for (int it = 0; it < 4; ++it) A[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NZ / 32; ++kb) {
          const int o = at_lds<NZ>(l16, 8 * g4) ^ 32 * kb;
          const bf16x8 zf = *reinterpret_cast<const bf16x8*>(sZ + o + 16 * w * NZ);
#pragma unroll
          for (int it = 0; it < 4; ++it)
            A[it] = mfma_bf16(zf, *reinterpret_cast<const bf16x8*>(sQ + o + 16 * it * NZ), A[it]);
        }
      }
      float pairs = 0.0f;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        if (it < (w & 2)) continue;  // nothing reads those
        float v[4];
        const float n0 = (float)(l16 - 4 * g4 - 16 * w);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float n = n0 + (float)(16 * it - r);  // i - j
          v[r] = P[it][r] * __builtin_fmaf(dec0[r], own[it], dec1[r] * far[it]);
          if constexpr (DG) pairs += n * v[r] * A[it][r];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
          reinterpret_cast<uint2*>(&sP[m][2 * it + (w >> 1)][lane])[w & 1] = cut_part(v);
      }
      if constexpr (DG) dg += pairs;
      float sum = 0.0f;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        float q[4], i1 = 0.0f;
        if constexpr (DG) {
          widen4(*reinterpret_cast<const uint2*>(sQ + at_lds<NZ>(l16, 16 * w + 4 * g4) + 16 * it * NZ), q);
          i1 = (float)l16 + (float)(16 * it + 1);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (DG) sum += (On[it][r] + O[it][r] * i1) * lamo[it] * q[r];
          O[it][r] *= lamo[it];
        }
      }
      if constexpr (DG) dg += sum;
    }

    // ---- the state: decayed, plus y^T (z times its decay), z's product in three bf16 parts
    bf16x8 zr[2];
    {
      const float full = sLam[len];
      auto column = [&](int ks, int dt) {  // channels 16 dt .. + 15 of y, 32 rows, as the A operand
        const int at1 = at_lds<DX>(4 * g4 + (l16 >> 2), 4 * (l16 & 3)) ^ 16 * dt;
        return join(tr_read(sY + at1 + 32 * ks * DX), tr_read(sY + at1 + (32 * ks + 16) * DX));
      };
      auto values = [&](int ks, float (&wz)[8]) {  // z's rows, and their decays
        lds_f32x4(sW + 32 * ks + 4 * g4, wz);
        lds_f32x4(sW + 32 * ks + 16 + 4 * g4, wz + 4);
        const uint16_t* at1 = sZ + at_lds<NZ>(4 * g4 + (l16 >> 2), 16 * w + 4 * (l16 & 3)) + 32 * ks * NZ;
        zr[ks] = join(tr_read(at1), tr_read(at1 + 16 * NZ));
      };
      float wz[2][8];
      bf16x8 yt[NDT];
      values(0, wz[0]);
      values(1, wz[1]);
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt) yt[dt] = column(0, dt);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (DG) Rs[dt][r] = full * (Rs[dt][r] + (float)len * S[dt][r]);
          S[dt][r] *= full;
        }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 zw[3], zn[3];
        const float left1 = DG ? (float)(len - 1 - 4 * g4) : 0.0f;
        float f[8], fn[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = wz[ks][e] * (float)zr[ks][e];
          if constexpr (DG)  // behind the step's end f is zero
            fn[e] = f[e] * (left1 - (float)(32 * ks + (e & 3) + 16 * (e >> 2)));
        }
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          zw[m] = cut8(f);
          if constexpr (DG) zn[m] = cut8(fn);
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int dt = 0; dt < NDT; ++dt) {
            S[dt] = mfma_bf16(yt[dt], zw[m], S[dt]);
            if constexpr (DG) Rs[dt] = mfma_bf16(yt[dt], zn[m], Rs[dt]);
          }
        __builtin_amdgcn_s_setprio(0);
        if (ks == 0) {
#pragma unroll
          for (int dt = 0; dt < NDT; ++dt) yt[dt] = column(1, dt);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    __syncthreads();  // pair weights are there, tiles are read

    // ---- the pairs' part of the outputs; the next step's tiles
    bf16x8 pf[OUT ? 6 : 1][2];
    if constexpr (OUT) {
#pragma unroll
      for (int f = 0; f < 6; ++f)
#pragma unroll
        for (int m = 0; m < 2; ++m) pf[f][m] = __builtin_bit_cast(bf16x8, sP[m][f < 2 ? 2 * f : f + 2][lane]);
      __builtin_amdgcn_sched_barrier(0);
    }
    stage();
    if constexpr (OUT) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int it = 2 * ks; it < 4; ++it) {
            const int f = it < 2 ? it : 2 * it + ks - 2;
            O[it] = mfma_bf16(zr[ks], pf[f][m], O[it]);
          }
      const __amdgpu_buffer_rsrc_t d = buf(po - (rev ? (LC - 1) * (int64_t)os : 0), 0x7fffffffu);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const uint2 o = round4(O[it][0], O[it][1], O[it][2], O[it][3]);
        // behind the step's end: an offset behind the descriptor's
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), d, 16 * it + l16 < len ? o0 + it * o1 : (int)0x80000000,
                                              0, 0);
      }
      po += (rev ? -LC : LC) * (int64_t)os;
    }

    // ---- the state that leaves a stretch
    if (last) {
      float* dst = OUT ? (now.ends ? p.sout : nullptr) : p.seg;
      const int64_t at = OUT ? ((int64_t)now.n * a.H + h) * a.KV : segat;
      const int sr = OUT ? p.sr : DZ, sc = OUT ? p.sc : 1;
      const int o = here(4 * g4 * sr + col * sc);
      if (dst) {
#pragma unroll
        for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int e = o + (16 * dt + r) * sr;
            dst[at + e] = S[dt][r];
            if constexpr (DG && !OUT) dst[rat + at + e] = Rs[dt][r];
          }
      }
      if constexpr (DG && OUT)
        if (now.ends && p.rend) {
          float sum = 0.0f;
#pragma unroll
          for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum += Rs[dt][r] * p.rend[at + o + (16 * dt + r) * sr];
          dg += sum;
        }
    }
    if (!more) break;
    first = last;
    if (last) now = c;
    left = ahead;
    __syncthreads();  // the next tiles are there, pair weights are read
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

// The states that enter the segments of a block, from those that each of them
// leaves by itself: the stretch that goes on beyond segment s starts inside it,
// or entered it and crosses it whole.  What happens at each segment is found by
// a lane of its own; the states of four segments are asked for at a time (13 us
// for 96 heads of 5 segments, a state read and written each: 4.8 TB/s).
template <bool DG>
__global__ void __launch_bounds__(LT) la_join_kernel(const LaArgs a) {
  const int per = a.KV / (LT * 4), blocks = a.nseg / a.spb;  // workgroups per head
  int id = blockIdx.x;
  const int piece = id % per, h = (id /= per) % a.H, b = (id /= a.H) % blocks;
  const LaPass& p = a.p[id / blocks];
  const int64_t e = (int64_t)h * a.KV + ((int64_t)piece * LT + threadIdx.x) * 4, step = (int64_t)a.H * a.KV;
  const int64_t R = axis_rows(a.ax);
  const int lane = threadIdx.x & 63;  // at most 64 segments a block
  bool on = false;                    // a stretch goes on beyond the segment
  float f = 0.0f, m = 0.0f;           // its decay across the segment, if it entered it, and tokens
  if (lane < a.spb) {
    const LaSeg sg = la_seg(a, b * a.spb + lane, R);
    if (sg.p0 < sg.p1) {
      const int64_t n = axis_owner(a.ax, p.rev ? sg.p0 : sg.p1 - 1);
      const int64_t bos = axis_start(a.ax, n), eos = la_end(a.ax, n, R);
      on = p.rev ? bos < sg.p0 : eos > sg.p1;
      m = (float)(sg.p1 - sg.p0);
      if (on && (p.rev ? eos > sg.p1 : bos < sg.p0)) f = la_pow(a.g[h], (double)(sg.p1 - sg.p0));
    }
  }
  constexpr int AT = 4;
  float4 E = make_float4(0.f, 0.f, 0.f, 0.f), Q = E;
  for (int k0 = 0; k0 < a.spb; k0 += AT) {
    float4 own[AT], rown[AT];
#pragma unroll
    for (int u = 0; u < AT; ++u) {
      const int k = k0 + u < a.spb ? k0 + u : a.spb - 1, s = b * a.spb + (p.rev ? a.spb - 1 - k : k);
      own[u] = *reinterpret_cast<const float4*>(p.seg + s * step + e);
      if (DG) rown[u] = *reinterpret_cast<const float4*>(p.seg + (a.nseg + s) * step + e);
    }
#pragma unroll
    for (int u = 0; u < AT; ++u) {
      const int k = k0 + u;
      if (k >= a.spb) break;
      const int l = p.rev ? a.spb - 1 - k : k, s = b * a.spb + l;
      *reinterpret_cast<float4*>(p.seg + s * step + e) = E;
      if (DG) *reinterpret_cast<float4*>(p.seg + (a.nseg + s) * step + e) = Q;
      const bool go = __shfl((int)on, l) != 0;
      const float fk = __shfl(f, l), mk = __shfl(m, l);
      // Where nothing goes on, what the segment's place holds is not a state.
      auto next = [&](float x, float y) { return !go ? 0.0f : fk != 0.0f ? fk * x + y : y; };
      if (DG) {
        Q.x = next(Q.x + mk * E.x, rown[u].x);
        Q.y = next(Q.y + mk * E.y, rown[u].y);
        Q.z = next(Q.z + mk * E.z, rown[u].z);
        Q.w = next(Q.w + mk * E.w, rown[u].w);
      }
      E.x = next(E.x, own[u].x);
      E.y = next(E.y, own[u].y);
      E.z = next(E.z, own[u].z);
      E.w = next(E.w, own[u].w);
    }
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
// rows are asked for before the first token.  64 sequences of 96 heads: 156 us,
// 5.2 TB/s, what a copy of 1 GiB reaches here.
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
  int slices, spb;
  int64_t L, nseg;
};
LaPlan la_plan(int64_t blocks, int64_t block, int64_t H, int64_t DZ, int64_t passes, bool dg) {
  LaPlan pl;
  pl.slices = (int)(DZ / 64);
  const int64_t chains = blocks * H * pl.slices * passes;
  // Steps that the busiest CU does one after another, three of the first pass
  // taken for one of the second.  With the decay's gradient the second pass has
  // one workgroup per CU, not two.
  const int64_t want = dg ? kLaWant / 2 : kLaWant;
  int64_t spb = 1, best = INT64_MAX;
  for (int64_t n = 1; n <= 64 && (n == 1 || chains * n <= kLaMost); ++n) {
    const int64_t len = (block + n * LC - 1) / (n * LC);
    if (n > 1 && len < kLaMinSteps) break;
    int64_t cost = 3 * ((chains * n + want - 1) / want * (len + kLaAround));
    if (n > 1) cost += (chains * (n - 1) + kLaWant - 1) / kLaWant * (len + kLaAround);
    if (cost < best) {
      best = cost;
      spb = n;
    }
  }
  pl.L = ((block + spb - 1) / spb + LC - 1) / LC * LC;
  pl.L = pl.L < LC ? LC : pl.L;
  pl.spb = (int)((block + pl.L - 1) / pl.L);
  pl.spb = pl.spb < 1 ? 1 : pl.spb;
  pl.nseg = blocks * pl.spb;
  return pl;
}

// Bytes of the states of a sweep's segments: at most kLaMost pieces in all,
// and, a cut block having more than 6 steps and a segment more than 3, at most
// T / 128 pieces a head.
size_t la_states_bytes(int64_t T_total, int64_t H, int64_t K, int64_t V) {
  const int64_t by_length = T_total > 6 * LC ? T_total / 128 * H : 0;
  return (size_t)((by_length < kLaMost ? by_length : kLaMost) * K * V) * sizeof(float);
}
// Bytes of the decay gradient's parts, for at most N blocks of the axis.
size_t la_part_bytes(int64_t N, int64_t H) {
  return align256((size_t)(N * H * 2 + kLaMost) * sizeof(float));
}

bool la_sizes_ok(int64_t T_total, int64_t H, int64_t K, int64_t V) {
  return T_total >= 0 && H >= 1 && H <= 1 << 16 && (K == 64 || K == 128) && (V == 64 || V == 128) &&
         fits(T_total, H * 128, kMaxElements);
}

kda_status_t la_check(const void* q, int64_t qs, int64_t qh, const void* k, int64_t ks, int64_t kh, const void* v,
                      int64_t vs, int64_t vh, const float* g, float scale, const int32_t* cu, int64_t B, int64_t T,
                      int64_t H, int64_t K, int64_t V, int64_t N) {
  if (B < 1 || T < 0 || H < 1 || K < 1 || V < 1 || N < 1) return KDA_ERR_INVALID;
  if (cu ? B != 1 : N != B) return KDA_ERR_INVALID;
  if ((K != 64 && K != 128) || (V != 64 && V != 128)) return KDA_ERR_UNSUPPORTED;
  if (H > 1 << 16 || N > 1 << 30 || !fits(B, T, kMaxElements) || !fits(B * T, H * 128, kMaxElements) ||
      !fits(N, H * 128 * 128, kMaxElements) || T >= (int64_t)1 << 31)
    return KDA_ERR_INVALID;
  if (!(scale - scale == 0.0f)) return KDA_ERR_INVALID;  // NaN or infinite
  if (!g || (B * T > 0 && (!q || !k || !v))) return KDA_ERR_INVALID;
  if (!mix_strides_ok(qs, qh) || !mix_strides_ok(ks, kh) || !mix_strides_ok(vs, vh)) return KDA_ERR_INVALID;
  if (!aligned_all(16, {q, k, v}) || !aligned(g, 4)) return KDA_ERR_INVALID;
  return KDA_SUCCESS;
}

// Workgroups of a sweep's passes, and those for sequences without tokens.
int64_t la_groups(const LaArgs& a) { return (a.items + 7) / 8 * 8 * a.slices * a.passes; }
int64_t la_more(const LaArgs& a, bool empties) { return !empties ? 0 : a.ax.N < 1024 ? a.ax.N : 1024; }
// Whether every launch of a sweep has a grid (a join has workgroups only where the
// axis is cut, and few heads then).
bool la_fits(const LaArgs& a, bool empties) { return la_groups(a) + la_more(a, empties) <= most_groups(LT); }

template <int DX, bool DG>
kda_status_t la_launch(LaArgs& a, bool empties, hipStream_t st) {
  const int64_t groups = la_groups(a), more = la_more(a, empties);
  a.main = groups;
  if (a.spb > 1) {  // otherwise every segment starts at a sequence's start
    kda_status_t s = launch(&la_sweep_kernel<DX, false, DG>, groups, LT, st, "linear attention segments", a);
    if (s != KDA_SUCCESS) return s;
    s = launch(&la_join_kernel<DG>, (int64_t)a.passes * (a.nseg / a.spb) * a.H * (a.KV / (LT * 4)), LT, st,
               "linear attention join", a);
    if (s != KDA_SUCCESS) return s;
  }
  return launch(&la_sweep_kernel<DX, true, DG>, groups + more, LT, st, "linear attention", a);
}
template <bool DG>
kda_status_t la_sweep(LaArgs& a, int64_t DX, bool empties, hipStream_t st) {
  return DX == 128 ? la_launch<128, DG>(a, empties, st) : la_launch<64, DG>(a, empties, st);
}

// The arguments of a sweep of `passes` passes with DZ channels of z.
void la_common(LaArgs& a, const float* g, const int32_t* cu, int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
               int64_t N, int64_t DZ, int passes, bool dg, unsigned flags) {
  const LaPlan pl = la_plan(B, T, H, DZ, passes, dg);
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
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_la_workspace_size(int64_t T_total, int64_t H, int64_t K, int64_t V) {
  return !la_sizes_ok(T_total, H, K, V) ? 0 : la_states_bytes(T_total, H, K, V);
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
  const size_t need = kda_la_workspace_size(B * T, H, K, V);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  LaArgs a;
  la_common(a, log_decay, cu_seqlens, B, T, H, K, V, N, V, 1, false, flags);
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
  const bool empties = final_state && (cu_seqlens || T == 0);
  return la_fits(a, empties) ? la_sweep<false>(a, K, empties, reinterpret_cast<hipStream_t>(stream)) : KDA_ERR_INVALID;
}

size_t kda_la_bwd_workspace_size(int64_t T_total, int64_t H, int64_t K, int64_t V, int64_t N) {
  if (!la_sizes_ok(T_total, H, K, V) || N < 1 || N > 1 << 30) return 0;
  return 4 * la_states_bytes(T_total, H, K, V) + la_part_bytes(N, H);
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
  const size_t sb = la_states_bytes(B * T, H, K, V);
  char* ws = static_cast<char*>(workspace);
  const uint16_t *qp = static_cast<const uint16_t*>(q), *kp = static_cast<const uint16_t*>(k),
                 *vp = static_cast<const uint16_t*>(v), *dp = static_cast<const uint16_t*>(d_out);
  const bool none = cu_seqlens || T == 0;  // there may be sequences without tokens

  // dq: of do, v, k; the state is S^T
  LaArgs aq, av, ak;
  la_common(aq, log_decay, cu_seqlens, B, T, H, K, V, N, K, 1, d_log_decay != nullptr, flags);
  LaPass& p = aq.p[0];
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
  }

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
  const bool both = K == V;  // one launch: both read q and do
  la_common(av, log_decay, cu_seqlens, B, T, H, K, V, N, V, both ? 2 : 1, false, flags);
  la_common(ak, log_decay, cu_seqlens, B, T, H, K, V, N, K, 1, false, flags);
  av.p[0] = pv;
  av.p[1] = ak.p[0] = pk;

  // nothing is enqueued unless all of it can be
  const bool empties = d_initial_state && none;
  if (!la_fits(aq, false) || !la_fits(av, empties) || !la_fits(ak, false)) return KDA_ERR_INVALID;
  s = d_log_decay ? la_sweep<true>(aq, V, false, st) : la_sweep<false>(aq, V, false, st);
  if (s == KDA_SUCCESS && d_log_decay)
    s = launch(&la_reduce_kernel, H, 64, st, "linear attention decay", (const float*)aq.p[0].part, d_log_decay,
               (int)(aq.nseg * aq.slices));
  if (s == KDA_SUCCESS) s = la_sweep<false>(av, K, empties, st);
  return s != KDA_SUCCESS || both ? s : la_sweep<false>(ak, V, false, st);
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
  if (T > 1 << 20 || !fits(B, H, most_groups(LT))) return KDA_ERR_INVALID;
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
