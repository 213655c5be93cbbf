// Causal softmax attention over whole prompts, with grouped heads and packed
// sequences.  Per sequence of nq queries and nk keys, query i sees the keys
// j <= i + nk - nq; with s_ij = scale q_i.k_j over those,
//     lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j.
// Gradients, for do and the gradient dl of lse, with d_i = do_i.o_i - dl_i:
//     dS_ij = p_ij (do_i.v_j - d_i),   dv_j = sum_i p_ij do_i,
//     dq_i = scale sum_j dS_ij k_j,    dk_j = scale sum_i dS_ij q_i,
// dk and dv summed over the query heads of a key head as well.
//
// Rows.  The G = Hq / Hk query heads of a key head share its keys, so the
// queries of a sequence are taken as nq G rows (i, g): a tile of rows is full
// for a single token's heads as for a prompt's, and the sum over a group is
// the sum over rows that a key's gradient takes anyway: no atomics.
//
// Forward.  A wave has 32 rows, in the columns of S^T = K Q^T (32x32x16 MFMA):
// a lane sees one row's scores of 32 keys a tile in its registers (its partner
// lane l ^ 32 the other half), so that maximum, sum and rescaling of the
// one-pass softmax stay in the lane, and S^T's result layout is the operand
// layout of O^T = V^T P^T: P never leaves the registers.  V^T comes from
// transposing LDS reads.  P is rounded to bf16 as an operand (2^-8 of each
// weight; their sum is taken in fp32 before), an error of the size of the
// output's own rounding.
//
// Few rows over long keys (decoding): the keys of a tile are split over
// workgroups of one wave, each leaving its o and lse in fp32; a second kernel
// joins them with weights exp(lse_s - lse).
//
// Backward.  Two kernels that both form P and dS again from lse: one over
// tiles of 128 keys holds dk and dv in accumulators and walks the rows, one
// over tiles of rows holds dq and walks the keys.  Two more products than one
// kernel with shared sums of dq would need, for results that are the same bits
// every time.  P and dS are rounded to bf16 as operands.  d is formed from
// do.(o + what o's rounding took off), which the forward keeps for a backward:
// the rounding of o alone would go into all of a row's dS alike (a sixth more
// error in dq and dk over rows of a few keys).

#include "../../include/kda.h"
#include "kda_mix.h"

namespace kda {
namespace {

constexpr float LN2 = 0.6931471805599453f;
constexpr int64_t kAttnWant = 1024;  // workgroups that a call with few rows is split into

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  uint16_t* out_lo;  // out's rounding errors, or nullptr
  float* lse;
  float* part;  // [splits][rows of q][Hq][D] partial outputs, then their lse
  const uint16_t* d_out;  // [tokens][Hq][D]
  const float* delta;     // [tokens][Hq]
  uint16_t *dq, *dk, *dv;
  int64_t qs, qh, ks, kh, vs, vh;  // token and head strides, elements
  Axis aq, ak;
  int Hq, Hk, G;
  int splits;
  int64_t slots;  // tiles of rows (dkv: of keys)
  int64_t main;   // workgroups with a tile; those behind them clear rows of no sequence
  float scale, c;  // c = scale log2(e)
};

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Sequence n's rows on an axis, held to the array.
struct Span {
  int64_t at;
  int64_t len;
};
__device__ __forceinline__ int64_t span_start(const Axis& ax, int64_t n, int64_t R) {
  const int64_t s = axis_start(ax, n);
  return s < R ? s : R;
}
__device__ __forceinline__ Span span(const Axis& ax, int n) {
  const int64_t R = axis_rows(ax), s = span_start(ax, n, R), e = span_start(ax, (int64_t)n + 1, R);
  return Span{s, e > s ? e - s : 0};
}

// Tiles of TILE rows, `mul` rows a token, sequences one after another: sequence
// n's start at slot start(n) mul / TILE + n, which leaves it enough of them
// whatever the lengths, so that no table of tiles is needed.
struct Place {
  int n;
  int64_t tile;
};
template <int TILE>
__device__ __forceinline__ Place tile_place(const Axis& ax, int64_t slot, int mul) {
  const int64_t R = axis_rows(ax);
  int lo = 0, hi = ax.N - 1;
  while (lo < hi) {  // the largest n whose first slot is not behind this one
    const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
    if (span_start(ax, mid, R) * mul / TILE + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return Place{lo, slot - (span_start(ax, lo, R) * mul / TILE + lo)};
}

// ROWS rows of D channels: NT threads ask for them in 16-byte pieces (zeros
// from `len` on), and put them into LDS rows of PITCH elements.
template <int D, int ROWS, int NT>
struct TileRegs {
  static constexpr int U = ROWS * D / 8 / NT;
  uint4 r[U];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t stride, int64_t row0, int64_t len) {
    const uint16_t* p = base + row0 * stride;
    const int left = (int)(len - row0 < ROWS ? len - row0 : ROWS);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = threadIdx.x + NT * u, row = e / (D / 8);
      r[u] = row < left ? *reinterpret_cast<const uint4*>(p + row * (int)stride + e % (D / 8) * 8) : make_uint4(0, 0, 0, 0);
    }
  }
  template <int PITCH>
  __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = threadIdx.x + NT * u;
      *reinterpret_cast<uint4*>(lds + e / (D / 8) * PITCH + e % (D / 8) * 8) = r[u];
    }
  }
};

// 32 rows of a tile as the A operand, channels 16 kk .. + 15.
template <int PITCH>
__device__ __forceinline__ bf16x8 rows_frag(const uint16_t* lds, int row0, int kk) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const bf16x8*>(lds + (row0 + (lane & 31)) * PITCH + 16 * kk + 8 * (lane >> 5));
}
// 32 channels from ch0 as the rows of the A operand, against 16 rows of the
// tile from row0 in the order of a 32x32 result's registers: a lane of half h
// has rows 4 h .. + 3 and 8 + 4 h .. + 3.
template <int PITCH>
__device__ __forceinline__ bf16x8 cols_frag(const uint16_t* lds, int row0, int ch0) {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const uint16_t* p = lds + (row0 + 4 * (lane >> 5) + (l16 >> 2)) * PITCH + ch0 + 16 * ((lane >> 4) & 1) + 4 * (l16 & 3);
  return join(tr_read(p), tr_read(p + 8 * PITCH));
}
// Registers 8 b .. 8 b + 7 of a 32x32 result, rounded, as the B operand against cols_frag's rows 16 b .. + 15.
__device__ __forceinline__ bf16x8 result_frag(const f32x16& s, int b) {
  const uint2 x = round4(s[8 * b], s[8 * b + 1], s[8 * b + 2], s[8 * b + 3]);
  return join(x, round4(s[8 * b + 4], s[8 * b + 5], s[8 * b + 6], s[8 * b + 7]));
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.0f;
  return z;
}

// Four channels of an output row, and what their rounding took off.
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t at, float (&v)[4]) {
  *reinterpret_cast<uint2*>(a.out + at) = cut_part(v);
  if (a.out_lo) *reinterpret_cast<uint2*>(a.out_lo + at) = cut_part(v);
}

// Rows behind the last sequence of an axis: H D elements each become zeros.
__device__ __forceinline__ void clear_rows(uint16_t* out, const Axis& ax, int64_t width, int64_t i, int64_t count) {
  const int64_t R = axis_rows(ax);
  for (int64_t e = R * width + (i * blockDim.x + threadIdx.x) * 8; e < ax.total * width; e += count * blockDim.x * 8)
    *reinterpret_cast<uint4*>(out + e) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <int D, int NW, int KT, bool SPLIT>
__global__ void __launch_bounds__(64 * NW, 2) attn_fwd_kernel(const AttnArgs a) {
  constexpr int NT = 64 * NW, BM = 32 * NW, ND = D / 16, NC = D / 32, NJ = KT / 32;
  constexpr int KP = D + 8, VP = D + 16;  // LDS pitches: rows 4 banks apart for row reads, 8 for transposing ones
  constexpr int NBUF = NW == 1 ? 1 : 2;
  __shared__ __align__(16) uint16_t sK[NBUF][KT * KP], sV[NBUF][KT * VP];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h2 = lane >> 5;

  if ((int64_t)blockIdx.x >= a.main) {
    const int64_t i = blockIdx.x - a.main, count = gridDim.x - a.main;
    clear_rows(a.out, a.aq, (int64_t)a.Hq * D, i, count);
    for (int64_t e = axis_rows(a.aq) * a.Hq + i * NT + threadIdx.x; e < a.aq.total * a.Hq; e += count * NT)
      a.lse[e] = -__builtin_inff();
    return;
  }
  // Longest tiles first; the key heads are neighbours in the order, so that
  // with 8 of them each has an XCD, and its L2, to itself.
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.Hk);
  const int split = SPLIT ? (int)(id / a.Hk % a.splits) : 0;
  const int64_t slot = a.slots - 1 - id / a.Hk / (SPLIT ? a.splits : 1);
  const Place at = tile_place<BM>(a.aq, slot, a.G);
  const Span sq = span(a.aq, at.n), sk = span(a.ak, at.n);
  const int64_t r0 = at.tile * BM, rows = sq.len * a.G;
  if (r0 >= rows) return;
  const int64_t off = sk.len - sq.len;

  // this lane's row, and the last key that it sees
  const int64_t row = r0 + 32 * w + (lane & 31), rc = row < rows ? row : rows - 1;
  const int64_t tok = rc / a.G;
  const int g = (int)(rc - tok * a.G);
  const int64_t see = tok + off;
  // the last keys that any row of the workgroup, of the wave sees; the first row's
  const int64_t rl = r0 + BM - 1 < rows ? r0 + BM - 1 : rows - 1;
  int64_t end = rl / a.G + off + 1;
  end = end < 0 ? 0 : end;
  int64_t j0 = 0, j1 = (end + KT - 1) / KT;
  if (SPLIT) {
    const int64_t per = (j1 + a.splits - 1) / a.splits;
    j0 = per * split < j1 ? per * split : j1;
    j1 = j0 + per < j1 ? j0 + per : j1;
  }
  const int64_t wf = r0 + 32 * w < rows ? r0 + 32 * w : rows - 1, wl = wf + 31 < rows ? wf + 31 : rows - 1;
  const int64_t wend = wl / a.G + off;   // last key of the wave's last row
  const int64_t wall = wf / a.G + off;   // every row of the wave sees the keys up to this one

  bf16x8 qf[ND];
  {
    const uint16_t* p = a.q + (sq.at + tok) * a.qs + ((int64_t)hk * a.G + g) * a.qh + 8 * h2;
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) qf[kk] = *reinterpret_cast<const bf16x8*>(p + 16 * kk);
  }
  f32x16 O[NC];
#pragma unroll
  for (int ct = 0; ct < NC; ++ct) O[ct] = zero16();
  float m = -__builtin_inff(), sum = 0.0f;  // running maximum (scores times c) and this lane's share of the sum

  const uint16_t* kb = a.k + sk.at * a.ks + hk * a.kh;
  const uint16_t* vb = a.v + sk.at * a.vs + hk * a.vh;
  TileRegs<D, KT, NT> rk, rv;
  if (j0 < j1) {
    rk.load(kb, a.ks, j0 * KT, sk.len);
    rv.load(vb, a.vs, j0 * KT, sk.len);
  }
  for (int64_t jt = j0; jt < j1; ++jt) {
    const int b = NBUF == 1 ? 0 : (int)(jt & 1);
    if (NBUF == 1) __syncthreads();
    rk.template store<KP>(sK[b]);
    rv.template store<VP>(sV[b]);
    __syncthreads();
    if (jt + 1 < j1) {
      rk.load(kb, a.ks, (jt + 1) * KT, sk.len);
      rv.load(vb, a.vs, (jt + 1) * KT, sk.len);
    }
    const int64_t key0 = jt * KT;
    if (key0 > wend) continue;
    f32x16 S[NJ];
#pragma unroll
    for (int js = 0; js < NJ; ++js) {
      S[js] = zero16();
#pragma unroll
      for (int kk = 0; kk < ND; ++kk) S[js] = mfma32(rows_frag<KP>(sK[b], 32 * js, kk), qf[kk], S[js]);
    }
    if (key0 + KT - 1 > wall) {  // some row does not see all of these keys
      const int64_t left = see - key0;
      const int last = (int)(left < KT ? left : KT);
#pragma unroll
      for (int js = 0; js < NJ; ++js)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * js + 8 * (e >> 2) + 4 * h2 + (e & 3) > last) S[js][e] = -__builtin_inff();
    }
    float top = S[0][0];
#pragma unroll
    for (int js = 0; js < NJ; ++js)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, S[js][e]);
    top = fmaxf(top, __shfl_xor(top, 32)) * a.c;
    if (__any(top > m)) {
      const float mn = fmaxf(m, top);
      const float f = mn == -__builtin_inff() ? 1.0f : fexp2(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int e = 0; e < 16; ++e) O[ct][e] *= f;
    }
    const float ms = m == -__builtin_inff() ? 0.0f : m;  // a row that has seen no key yet: all weights are 0
#pragma unroll
    for (int js = 0; js < NJ; ++js)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        S[js][e] = fexp2(S[js][e] * a.c - ms);
        sum += S[js][e];
      }
#pragma unroll
    for (int js = 0; js < NJ; ++js)
#pragma unroll
      for (int b2 = 0; b2 < 2; ++b2) {
        const bf16x8 pf = result_frag(S[js], b2);
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) O[ct] = mfma32(cols_frag<VP>(sV[b], 32 * js + 16 * b2, 32 * ct), pf, O[ct]);
      }
  }
  sum += __shfl_xor(sum, 32);
  if (row >= rows) return;
  const float inv = sum > 0.0f ? 1.0f / sum : sum;  // no key: zeros (NaN stays NaN)
  const int64_t head = (sq.at + tok) * a.Hq + (int64_t)hk * a.G + g;
  const float lse = sum == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * LN2;
  if (SPLIT) {
    const int64_t total = a.aq.total * a.Hq;
    float* po = a.part + (split * total + head) * D;
#pragma unroll
    for (int ct = 0; ct < NC; ++ct)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {O[ct][4 * q] * inv, O[ct][4 * q + 1] * inv, O[ct][4 * q + 2] * inv, O[ct][4 * q + 3] * inv};
        store4(po + 32 * ct + 8 * q + 4 * h2, v);
      }
    if (h2 == 0) a.part[a.splits * total * D + split * total + head] = lse;
    return;
  }
#pragma unroll
  for (int ct = 0; ct < NC; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4] = {O[ct][4 * q] * inv, O[ct][4 * q + 1] * inv, O[ct][4 * q + 2] * inv, O[ct][4 * q + 3] * inv};
      store_out(a, head * D + 32 * ct + 8 * q + 4 * h2, v);
    }
  if (h2 == 0) a.lse[head] = lse;
}

// The parts of split keys, joined: one row and head a D / 4 lanes.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  constexpr int LR = D / 4;
  const int64_t total = a.aq.total * a.Hq, live = axis_rows(a.aq) * a.Hq;
  const int64_t head = (int64_t)blockIdx.x * (256 / LR) + threadIdx.x / LR;
  if (head >= live) return;
  const int c4 = threadIdx.x % LR * 4;
  const float* lp = a.part + a.splits * total * D + head;
  float m = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, lp[s * total]);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float l = lp[s * total];
    if (l == -__builtin_inff()) continue;
    const float f = fexp2((l - m) * LOG2E);
    float v[4];
    load_f4(a.part + (s * total + head) * D + c4, v);
    sum += f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += f * v[e];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  store_out(a, head * D + c4, o);
  if (c4 == 0) a.lse[head] = sum == 0.0f ? -__builtin_inff() : m + __builtin_amdgcn_logf(sum) * LN2;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// d = do.o - dl for every row and head.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const uint16_t* out, const uint16_t* out_lo,
                                                         const uint16_t* d_out, const float* d_lse, float* delta,
                                                         int64_t heads) {
  constexpr int LR = D / 8;
  const int64_t head = (int64_t)blockIdx.x * (256 / LR) + threadIdx.x / LR;
  if (head >= heads) return;
  const int64_t at = head * D + threadIdx.x % LR * 8;
  float x[8], lo[8], y[8], s = 0.0f;
  unpack_bf16x8(*reinterpret_cast<const uint4*>(out + at), x);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(out_lo + at), lo);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(d_out + at), y);
#pragma unroll
  for (int e = 0; e < 8; ++e) s += (x[e] + lo[e]) * y[e];
#pragma unroll
  for (int i = LR / 2; i >= 1; i >>= 1) s += __shfl_xor(s, i);
  if (threadIdx.x % LR == 0) delta[head] = s - (d_lse ? d_lse[head] : 0.0f);
}

template <int D>
__global__ void __launch_bounds__(256, 1) attn_dq_kernel(const AttnArgs a) {
  constexpr int NT = 256, BM = 128, KT = 32, ND = D / 16, NC = D / 32;
  constexpr int KP = D + 16, VP = D + 8;
  __shared__ __align__(16) uint16_t sK[2][KT * KP], sV[2][KT * VP];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h2 = lane >> 5;
  if ((int64_t)blockIdx.x >= a.main) {
    clear_rows(a.dq, a.aq, (int64_t)a.Hq * D, blockIdx.x - a.main, gridDim.x - a.main);
    return;
  }
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.Hk);
  const Place at = tile_place<BM>(a.aq, a.slots - 1 - id / a.Hk, a.G);
  const Span sq = span(a.aq, at.n), sk = span(a.ak, at.n);
  const int64_t r0 = at.tile * BM, rows = sq.len * a.G;
  if (r0 >= rows) return;
  const int64_t off = sk.len - sq.len;
  const int64_t row = r0 + 32 * w + (lane & 31), rc = row < rows ? row : rows - 1;
  const int64_t tok = rc / a.G;
  const int g = (int)(rc - tok * a.G);
  const int64_t see = tok + off;
  const int64_t rl = r0 + BM - 1 < rows ? r0 + BM - 1 : rows - 1;
  const int64_t end = rl / a.G + off + 1;
  const int64_t j1 = end > 0 ? (end + KT - 1) / KT : 0;
  const int64_t wf = r0 + 32 * w < rows ? r0 + 32 * w : rows - 1, wl = wf + 31 < rows ? wf + 31 : rows - 1;
  const int64_t wend = wl / a.G + off, wall = wf / a.G + off;
  const int64_t head = (sq.at + tok) * a.Hq + (int64_t)hk * a.G + g;

  bf16x8 qf[ND], df[ND];
  {
    const uint16_t* p = a.q + (sq.at + tok) * a.qs + ((int64_t)hk * a.G + g) * a.qh + 8 * h2;
    const uint16_t* d = a.d_out + head * D + 8 * h2;
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      qf[kk] = *reinterpret_cast<const bf16x8*>(p + 16 * kk);
      df[kk] = *reinterpret_cast<const bf16x8*>(d + 16 * kk);
    }
  }
  const float l = a.lse[head];
  const float l2 = l == -__builtin_inff() ? 0.0f : l * LOG2E;  // a row that sees no key: all is masked
  const float dd = a.delta[head];
  f32x16 Q[NC];
#pragma unroll
  for (int ct = 0; ct < NC; ++ct) Q[ct] = zero16();
  const uint16_t* kb = a.k + sk.at * a.ks + hk * a.kh;
  const uint16_t* vb = a.v + sk.at * a.vs + hk * a.vh;
  TileRegs<D, KT, NT> rk, rv;
  if (j1 > 0) {
    rk.load(kb, a.ks, 0, sk.len);
    rv.load(vb, a.vs, 0, sk.len);
  }
  for (int64_t jt = 0; jt < j1; ++jt) {
    const int b = (int)(jt & 1);
    rk.template store<KP>(sK[b]);
    rv.template store<VP>(sV[b]);
    __syncthreads();
    if (jt + 1 < j1) {
      rk.load(kb, a.ks, (jt + 1) * KT, sk.len);
      rv.load(vb, a.vs, (jt + 1) * KT, sk.len);
    }
    const int64_t key0 = jt * KT;
    if (key0 > wend) continue;
    f32x16 S = zero16(), P = zero16();
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      S = mfma32(rows_frag<KP>(sK[b], 0, kk), qf[kk], S);
      P = mfma32(rows_frag<VP>(sV[b], 0, kk), df[kk], P);
    }
    const int64_t left = see - key0;
    const int last = key0 + KT - 1 > wall ? (int)(left < KT ? left : KT) : KT;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p = fexp2(S[e] * a.c - l2);
      S[e] = 8 * (e >> 2) + 4 * h2 + (e & 3) > last ? 0.0f : p * (P[e] - dd);
    }
#pragma unroll
    for (int b2 = 0; b2 < 2; ++b2) {
      const bf16x8 sf = result_frag(S, b2);
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) Q[ct] = mfma32(cols_frag<KP>(sK[b], 16 * b2, 32 * ct), sf, Q[ct]);
    }
  }
  if (row >= rows) return;
  __bf16* po = reinterpret_cast<__bf16*>(a.dq) + head * D;
#pragma unroll
  for (int ct = 0; ct < NC; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a.scale * Q[ct][4 * q + e];
      store4(po + 32 * ct + 8 * q + 4 * h2, v);
    }
}

template <int D>
__global__ void __launch_bounds__(256, 1) attn_dkv_kernel(const AttnArgs a) {
  constexpr int NT = 256, BN = 128, RT = 32, ND = D / 16, NC = D / 32;
  constexpr int QP = D + 16;
  __shared__ __align__(16) uint16_t sQ[2][RT * QP], sD[2][RT * QP];
  __shared__ __align__(16) float sL[2][RT], sE[2][RT];  // lse log2(e) and d of the rows
  __shared__ int sT[2][RT];                             // the last key that each row sees, from this tile's first
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h2 = lane >> 5;
  if ((int64_t)blockIdx.x >= a.main) {
    clear_rows(a.dk, a.ak, (int64_t)a.Hk * D, blockIdx.x - a.main, gridDim.x - a.main);
    clear_rows(a.dv, a.ak, (int64_t)a.Hk * D, blockIdx.x - a.main, gridDim.x - a.main);
    return;
  }
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.Hk);
  const Place at = tile_place<BN>(a.ak, id / a.Hk, 1);  // the first keys are seen by the most rows
  const Span sq = span(a.aq, at.n), sk = span(a.ak, at.n);
  const int64_t key0 = at.tile * BN;
  if (key0 >= sk.len) return;
  const int64_t off = sk.len - sq.len, rows = sq.len * a.G;
  const int64_t key = key0 + 32 * w + (lane & 31), kc = key < sk.len ? key : sk.len - 1;
  const int64_t t0 = key0 > off ? key0 - off : 0;  // first token that sees a key of the tile
  const int64_t i0 = t0 * a.G / RT, i1 = (rows + RT - 1) / RT;

  bf16x8 kf[ND], vf[ND];
  {
    const uint16_t* p = a.k + (sk.at + kc) * a.ks + hk * a.kh + 8 * h2;
    const uint16_t* q = a.v + (sk.at + kc) * a.vs + hk * a.vh + 8 * h2;
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      kf[kk] = *reinterpret_cast<const bf16x8*>(p + 16 * kk);
      vf[kk] = *reinterpret_cast<const bf16x8*>(q + 16 * kk);
    }
  }
  f32x16 K[NC], V[NC];
#pragma unroll
  for (int ct = 0; ct < NC; ++ct) {
    K[ct] = zero16();
    V[ct] = zero16();
  }

  constexpr int U = RT * D / 8 / NT;
  uint4 rq[U], rd[U];
  float rl = 0.0f, re = 0.0f;
  int rt = -1;
  auto fetch = [&](int64_t it) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = threadIdx.x + NT * u;
      const int64_t r = it * RT + e / (D / 8);
      const int c8 = e % (D / 8) * 8;
      rq[u] = rd[u] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int64_t tok = r / a.G, h = (int64_t)hk * a.G + (r - tok * a.G);
        rq[u] = *reinterpret_cast<const uint4*>(a.q + (sq.at + tok) * a.qs + h * a.qh + c8);
        rd[u] = *reinterpret_cast<const uint4*>(a.d_out + ((sq.at + tok) * a.Hq + h) * D + c8);
      }
    }
    if (threadIdx.x < RT) {
      const int64_t r = it * RT + threadIdx.x;
      rl = re = 0.0f;
      rt = -1;
      if (r < rows) {
        const int64_t tok = r / a.G, h = (sq.at + tok) * a.Hq + (int64_t)hk * a.G + (r - tok * a.G);
        const float l = a.lse[h];
        rl = l == -__builtin_inff() ? 0.0f : l * LOG2E;
        re = a.delta[h];
        const int64_t last = tok + off - key0;
        rt = (int)(last < BN ? last : BN);
      }
    }
  };
  if (i0 < i1) fetch(i0);
  for (int64_t it = i0; it < i1; ++it) {
    const int b = (int)((it - i0) & 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = threadIdx.x + NT * u, to = e / (D / 8) * QP + e % (D / 8) * 8;
      *reinterpret_cast<uint4*>(sQ[b] + to) = rq[u];
      *reinterpret_cast<uint4*>(sD[b] + to) = rd[u];
    }
    if (threadIdx.x < RT) {
      sL[b][threadIdx.x] = rl;
      sE[b][threadIdx.x] = re;
      sT[b][threadIdx.x] = rt;
    }
    __syncthreads();
    if (it + 1 < i1) fetch(it + 1);
    f32x16 S = zero16(), P = zero16();
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      S = mfma32(rows_frag<QP>(sQ[b], 0, kk), kf[kk], S);
      P = mfma32(rows_frag<QP>(sD[b], 0, kk), vf[kk], P);
    }
    const int mine = 32 * w + (lane & 31);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 l4 = *reinterpret_cast<const float4*>(&sL[b][8 * q + 4 * h2]);
      const float4 e4 = *reinterpret_cast<const float4*>(&sE[b][8 * q + 4 * h2]);
      const int4 t4 = *reinterpret_cast<const int4*>(&sT[b][8 * q + 4 * h2]);
      const float lv[4] = {l4.x, l4.y, l4.z, l4.w}, ev[4] = {e4.x, e4.y, e4.z, e4.w};
      const int tv[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool on = mine <= tv[e];
        const float p = on ? fexp2(S[4 * q + e] * a.c - lv[e]) : 0.0f;
        S[4 * q + e] = p;
        P[4 * q + e] = on ? p * (P[4 * q + e] - ev[e]) : 0.0f;
      }
    }
#pragma unroll
    for (int b2 = 0; b2 < 2; ++b2) {
      const bf16x8 pf = result_frag(S, b2), sf = result_frag(P, b2);
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        V[ct] = mfma32(cols_frag<QP>(sD[b], 16 * b2, 32 * ct), pf, V[ct]);
        K[ct] = mfma32(cols_frag<QP>(sQ[b], 16 * b2, 32 * ct), sf, K[ct]);
      }
    }
  }
  if (key >= sk.len) return;
  const int64_t to = ((sk.at + key) * a.Hk + hk) * D;
#pragma unroll
  for (int ct = 0; ct < NC; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = a.scale * K[ct][4 * q + e];
        y[e] = V[ct][4 * q + e];
      }
      store4(reinterpret_cast<__bf16*>(a.dk) + to + 32 * ct + 8 * q + 4 * h2, x);
      store4(reinterpret_cast<__bf16*>(a.dv) + to + 32 * ct + 8 * q + 4 * h2, y);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// How a forward is cut: rows of a tile (32 or 128), parts of the keys.
struct AttnPlan {
  int bm;
  int64_t slots;
  int splits;
  size_t bytes;
};
AttnPlan attn_plan(int64_t tq, int64_t tk, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  AttnPlan p;
  const int64_t rows = tq * (Hq / Hk);
  p.bm = rows <= 64 * N ? 32 : 128;
  p.slots = rows / p.bm + N;
  // tiles that hold rows, as far as the host knows, and keys of a sequence
  const int64_t tiles = ((rows + p.bm - 1) / p.bm > N ? (rows + p.bm - 1) / p.bm : (rows < N ? rows : N)) * Hk;
  const int64_t most = (tk / N + 255) / 256;
  int64_t s = tiles > 0 ? kAttnWant / tiles : 1;
  s = s < most ? s : most;
  p.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  p.bytes = p.splits > 1 ? align256((size_t)p.splits * (size_t)(tq * Hq) * (size_t)(D + 1) * sizeof(float)) : 0;
  return p;
}

kda_status_t attn_check(AttnArgs& a, const void* q, int64_t qs, int64_t qh, const void* k, int64_t ks, int64_t kh,
                        const void* v, int64_t vs, int64_t vh, float scale, const int32_t* cq, const int32_t* ck,
                        int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t N, unsigned flags) {
  if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hk < 1 || N < 1 || Hq % Hk != 0) return KDA_ERR_INVALID;
  if ((cq == nullptr) != (ck == nullptr)) return KDA_ERR_INVALID;
  if (cq ? B != 1 : N != B) return KDA_ERR_INVALID;
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  if (flags & ~FLAG_ZERO_REST) return KDA_ERR_INVALID;
  if (Hq > 1 << 16 || N > 1 << 30 || !fits(B, Tq, kMaxElements) || !fits(B, Tk, kMaxElements) ||
      !fits(B * Tq, Hq * D, kMaxElements) || !fits(B * Tk, Hk * D, kMaxElements) || Tq >= (int64_t)1 << 31 ||
      Tk >= (int64_t)1 << 31)
    return KDA_ERR_INVALID;
  if (!(scale > 0.0f) || !(scale - scale == 0.0f)) return KDA_ERR_INVALID;
  if ((B * Tq > 0 && !q) || (B * Tk > 0 && (!k || !v))) return KDA_ERR_INVALID;
  if (!mix_strides_ok(qs, qh) || !mix_strides_ok(ks, kh) || !mix_strides_ok(vs, vh)) return KDA_ERR_INVALID;
  if (!aligned_all(16, {q, k, v})) return KDA_ERR_INVALID;
  a = AttnArgs{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.qs = qs, a.qh = qh, a.ks = ks, a.kh = kh, a.vs = vs, a.vh = vh;
  a.aq = make_axis(cq, Tq, B * Tq, N);
  a.ak = make_axis(ck, Tk, B * Tk, N);
  a.Hq = (int)Hq;
  a.Hk = (int)Hk;
  a.G = (int)(Hq / Hk);
  a.scale = scale;
  a.c = scale * LOG2E;
  a.splits = 1;
  return KDA_SUCCESS;
}

// Workgroups that clear the rows of no sequence.
int64_t attn_clear(const int32_t* cu, unsigned flags) { return cu && (flags & FLAG_ZERO_REST) ? 64 : 0; }

constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;

template <int D>
kda_status_t attn_run_fwd(AttnArgs& a, const AttnPlan& p, int64_t clear, hipStream_t st) {
  a.slots = p.slots;
  a.splits = p.splits;
  if (p.slots > kMaxGrid / a.Hk / p.splits - 64) return KDA_ERR_INVALID;
  a.main = p.slots * a.Hk * p.splits;
  if (p.splits == 1)
    return p.bm == 32 ? launch(&attn_fwd_kernel<D, 1, 32, false>, a.main + clear, 64, st, "attention", a)
                      : launch(&attn_fwd_kernel<D, 4, 64, false>, a.main + clear, 256, st, "attention", a);
  const kda_status_t s = p.bm == 32 ? launch(&attn_fwd_kernel<D, 1, 32, true>, a.main + clear, 64, st, "attention parts", a)
                                    : launch(&attn_fwd_kernel<D, 4, 64, true>, a.main + clear, 256, st, "attention parts", a);
  if (s != KDA_SUCCESS) return s;
  const int64_t per = 256 / (D / 4);
  return launch(&attn_join_kernel<D>, (a.aq.total * a.Hq + per - 1) / per, 256, st, "attention join", a);
}

template <int D>
kda_status_t attn_run_bwd(AttnArgs& a, const void* out, const void* out_lo, const float* d_lse, float* delta, int64_t clear, hipStream_t st) {
  const int64_t heads = a.aq.total * a.Hq, per = 256 / (D / 8);
  a.delta = delta;
  if (heads > 0) {
    const kda_status_t s = launch(&attn_delta_kernel<D>, (heads + per - 1) / per, 256, st, "attention delta",
                                  static_cast<const uint16_t*>(out), static_cast<const uint16_t*>(out_lo), a.d_out, d_lse,
                                  delta, heads);
    if (s != KDA_SUCCESS) return s;
  }
  a.slots = a.ak.total / 128 + a.ak.N;
  if (a.slots > (kMaxGrid - 64) / a.Hk) return KDA_ERR_INVALID;
  a.main = a.slots * a.Hk;
  const kda_status_t s = launch(&attn_dkv_kernel<D>, a.main + clear, 256, st, "attention dk, dv", a);
  if (s != KDA_SUCCESS) return s;
  a.slots = a.aq.total * a.G / 128 + a.aq.N;
  if (a.slots > (kMaxGrid - 64) / a.Hk) return KDA_ERR_INVALID;
  a.main = a.slots * a.Hk;
  return launch(&attn_dq_kernel<D>, a.main + clear, 256, st, "attention dq", a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_attn_workspace_size(int64_t Tq_total, int64_t Tk_total, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  if (Tq_total < 0 || Tk_total < 0 || Hq < 1 || Hk < 1 || Hq > 1 << 16 || Hq % Hk != 0 || (D != 64 && D != 128) ||
      N < 1 || N > 1 << 30 || !fits(Tq_total, Hq * D, kMaxElements) || !fits(Tk_total, Hk * D, kMaxElements))
    return 0;
  return 256 + attn_plan(Tq_total, Tk_total, Hq, Hk, D, N).bytes;
}

kda_status_t kda_attn_fwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                          int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride, float scale,
                          void* out, void* out_lo, float* lse, void* workspace, size_t workspace_bytes, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                          int64_t D, int64_t N, unsigned flags, void* stream) {
  AttnArgs a;
  const kda_status_t s = attn_check(a, q, q_stride, q_head_stride, k, k_stride, k_head_stride, v, v_stride,
                                    v_head_stride, scale, cu_seqlens_q, cu_seqlens_k, B, Tq, Tk, Hq, Hk, D, N, flags);
  if (s != KDA_SUCCESS) return s;
  if (B * Tq > 0 && (!out || !lse)) return KDA_ERR_INVALID;
  if (!aligned_all(16, {out, out_lo, workspace}) || !aligned(lse, 4)) return KDA_ERR_INVALID;
  for (const void* i : {q, k, v})
    if (same(out, i) || same(out_lo, i)) return KDA_ERR_INVALID;
  if (same(out, out_lo)) return KDA_ERR_INVALID;
  if (!workspace || workspace_bytes < kda_attn_workspace_size(B * Tq, B * Tk, Hq, Hk, D, N)) return KDA_ERR_WORKSPACE;
  if (B * Tq == 0) return KDA_SUCCESS;
  a.out = static_cast<uint16_t*>(out);
  a.out_lo = static_cast<uint16_t*>(out_lo);
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  const AttnPlan p = attn_plan(B * Tq, B * Tk, Hq, Hk, D, N);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t clear = attn_clear(cu_seqlens_q, flags);
  return D == 128 ? attn_run_fwd<128>(a, p, clear, st) : attn_run_fwd<64>(a, p, clear, st);
}

size_t kda_attn_bwd_workspace_size(int64_t Tq_total, int64_t Hq) {
  if (Tq_total < 0 || Hq < 1 || Hq > 1 << 16 || !fits(Tq_total, Hq * 128, kMaxElements)) return 0;
  return 256 + align256((size_t)(Tq_total * Hq) * sizeof(float));
}

kda_status_t kda_attn_bwd(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                          int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride, float scale,
                          const void* out, const void* out_lo, const float* lse, const void* d_out, const float* d_lse, void* dq, void* dk,
                          void* dv, void* workspace, size_t workspace_bytes, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                          int64_t D, int64_t N, unsigned flags, void* stream) {
  AttnArgs a;
  const kda_status_t s = attn_check(a, q, q_stride, q_head_stride, k, k_stride, k_head_stride, v, v_stride,
                                    v_head_stride, scale, cu_seqlens_q, cu_seqlens_k, B, Tq, Tk, Hq, Hk, D, N, flags);
  if (s != KDA_SUCCESS) return s;
  if ((B * Tq > 0 && (!out || !out_lo || !lse || !d_out || !dq)) || (B * Tk > 0 && (!dk || !dv))) return KDA_ERR_INVALID;
  if (!aligned_all(16, {out, out_lo, d_out, dq, dk, dv, workspace}) || !aligned_all(4, {lse, d_lse})) return KDA_ERR_INVALID;
  for (const void* o : {(const void*)dq, (const void*)dk, (const void*)dv})
    for (const void* i : {q, k, v, out, out_lo, d_out})
      if (same(o, i)) return KDA_ERR_INVALID;
  if (same(dq, dk) || same(dq, dv) || same(dk, dv)) return KDA_ERR_INVALID;
  if (!workspace || workspace_bytes < kda_attn_bwd_workspace_size(B * Tq, Hq)) return KDA_ERR_WORKSPACE;
  a.lse = const_cast<float*>(lse);
  a.d_out = static_cast<const uint16_t*>(d_out);
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t clear = attn_clear(cu_seqlens_q, flags);
  float* delta = static_cast<float*>(workspace);
  return D == 128 ? attn_run_bwd<128>(a, out, out_lo, d_lse, delta, clear, st)
                  : attn_run_bwd<64>(a, out, out_lo, d_lse, delta, clear, st);
}

}  // extern "C"
