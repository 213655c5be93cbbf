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

#include <type_traits>

#include "../../include/kda.h"
#include "kda_mix.h"

namespace kda {
namespace {

constexpr float LN2 = 0.6931471805599453f;
constexpr int64_t kAttnRound = 256;  // CUs

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  uint16_t* out_lo;  // out's rounding errors, or nullptr
  float* lse;
  float* part;  // forward: [splits][rows of q][Hq][D] outputs, then their lse; backward: [splits] dk, dv sums in fp32
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

constexpr int64_t kNoTile = (int64_t)1 << 40;  // behind every sequence's last tile
struct Place {
  int n;
  int64_t tile;
};
__device__ __forceinline__ int wave_sum(int x) {
  auto add = [&](auto ctrl) { x += __builtin_amdgcn_update_dpp(0, x, decltype(ctrl)::value, 0xf, 0xf, true); };
  add(std::integral_constant<int, 0xB1>{});   // quad_perm [1, 0, 3, 2]
  add(std::integral_constant<int, 0x4E>{});   // quad_perm [2, 3, 0, 1]
  add(std::integral_constant<int, 0x141>{});  // row_half_mirror
  add(std::integral_constant<int, 0x140>{});  // row_mirror
  return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) + __builtin_amdgcn_readlane(x, 32) +
         __builtin_amdgcn_readlane(x, 48);
}
// The id-th tile of TILE rows, `mul` rows a token.  up: tiles further into their
// sequence take more work (rows see more keys), otherwise tiles further from its
// end do (keys are seen by more rows); those come first, so that a launch does not
// end with a long tile.
// Of up to 64 packed sequences a lane has one: the tiles of level L, as many
// before (behind) them in their sequence, go before those of level L - 1, and the
// level is found by counting.  16 ragged prompts in 16411 tokens, 12 heads of 64,
// forward: 77 us; sequences one after another 93.  Equal lengths come one sequence
// after another (2 x 4097 tokens, 12 heads of 128, with gradients: 613 us; by level
// 620), as do more than 64: sequence n's tiles start at slot start(n) mul / TILE + n,
// which leaves it enough of them whatever the lengths.  No table of tiles is
// needed in any of the three.
template <int TILE>
__device__ __forceinline__ Place tile_place(const Axis& ax, int64_t id, int64_t slots, int mul, bool up) {
  if (!ax.cu) {
    const int64_t tiles = (ax.T * mul + TILE - 1) / TILE, n = tiles > 0 ? id / tiles : ax.N, tile = id - n * tiles;
    return n < ax.N ? Place{(int)n, up ? tiles - 1 - tile : tile} : Place{0, kNoTile};
  }
  const int64_t R = axis_rows(ax);
  if (ax.N > 1 && ax.N <= 64) {
    const int lane = threadIdx.x & 63;
    int tiles = 0;
    if (lane < ax.N) {
      const int64_t a = span_start(ax, lane, R), e = span_start(ax, (int64_t)lane + 1, R);
      tiles = e > a ? (int)(((e - a) * mul + TILE - 1) / TILE) : 0;
    }
    auto from = [&](int level) { return wave_sum(tiles > level ? tiles - level : 0); };  // tiles of this level and more
    if (id >= from(0)) return Place{0, kNoTile};
    int lo = 0, hi = (int)slots;
    while (hi - lo > 1) {  // from(lo) > id >= from(hi)
      const int mid = lo + ((hi - lo) >> 1);
      if (from(mid) > id) lo = mid; else hi = mid;
    }
    const int k = (int)id - from(lo + 1);  // the k-th sequence with more tiles than lo
    const uint64_t has = __ballot(tiles > lo);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(has >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)has, 0));
    const uint64_t is = __ballot(tiles > lo && before == k);
    const int n = is ? __builtin_ctzll(is) : 0;
    return Place{n, up ? lo : __builtin_amdgcn_readlane(tiles, n) - 1 - lo};
  }
  const int64_t slot = up ? slots - 1 - id : id;
  int lo = 0, hi = ax.N - 1;
  while (lo < hi) {  // the largest n whose first slot is not behind this one
    const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
    if (span_start(ax, mid, R) * mul / TILE + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return Place{lo, slot - (span_start(ax, lo, R) * mul / TILE + lo)};
}

// Element (row, col) of a tile of W columns in LDS: the 16-byte pieces of a row
// are permuted by the row, so that both 16 rows of one piece (row operands) and
// 4 rows of four neighbouring ones (transposing reads) meet all 64 banks once.
template <int W>
__device__ __forceinline__ int at_tile(int row, int col) {
  static_assert(W == 64 || W == 128, "pieces of 16 bytes");
  const int f = W == 128 ? (row & 3) << 2 | (row >> 2 & 3) : (row >> 1 & 1) << 2 | (row >> 2 & 3);
  return row * W + (((col >> 3) ^ f) << 3) + (col & 7);
}

// ROWS rows of D channels: NT threads ask for them in 16-byte pieces (zeros
// from `len` on), and put them into a tile in LDS.
template <int D, int ROWS, int NT>
struct TileRegs {
  static constexpr int PR = NT / (D / 8), U = ROWS / PR;  // rows a load covers, loads
  uint4 r[U];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t stride, int64_t row0, int64_t len) {
    const __amdgpu_buffer_rsrc_t d = buf(base + row0 * stride, 0x7fffffffu);
    const int left = (int)(len - row0 < ROWS ? len - row0 : ROWS);
    const int rt = threadIdx.x / (D / 8), at = rt * (int)stride * 2 + (int)(threadIdx.x % (D / 8)) * 16;
#pragma unroll
    for (int u = 0; u < U; ++u)  // a row from len on: an offset behind the descriptor's end
      r[u] = bload<uint4>(d, rt + PR * u < left ? at : (int)0x80000000, u * PR * (int)stride * 2);
  }
  __device__ __forceinline__ void store(uint16_t* lds) const {
    const int rt = threadIdx.x / (D / 8), c = threadIdx.x % (D / 8) * 8;
#pragma unroll
    for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(lds + at_tile<D>(rt + PR * u, c)) = r[u];
  }
};

// 32 rows of a tile as the A operand, channels 16 kk .. + 15.  The permutation
// is one by xor, so a lane keeps one place for all of a tile's operands.
template <int D>
__device__ __forceinline__ int rows_place() {
  const int lane = threadIdx.x & 63;
  return at_tile<D>(lane & 31, 8 * (lane >> 5));
}
template <int D>
__device__ __forceinline__ bf16x8 rows_frag(const uint16_t* lds, int place, int row0, int kk) {
  return *reinterpret_cast<const bf16x8*>(lds + (place ^ 16 * kk) + row0 * D);
}
// 32 channels from 32 ct as the rows of the A operand, against 16 rows of the
// tile from row0 in the order of a 32x32 result's registers: a lane of half h
// has rows 4 h .. + 3 and 8 + 4 h .. + 3.
template <int D>
__device__ __forceinline__ int cols_place() {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  return at_tile<D>(4 * (lane >> 5) + (l16 >> 2), 16 * ((lane >> 4) & 1) + 4 * (l16 & 3));
}
template <int D>
__device__ __forceinline__ bf16x8 cols_frag(const uint16_t* lds, int place, int row0, int ct) {
  const int at = place ^ 32 * ct;
  return join(tr_read(lds + at + row0 * D), tr_read(lds + (at ^ 16) + (row0 + 8) * D));
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
// Tiles of 128 rows, 64 keys and two buffers (64 KB of LDS for D = 128, two
// workgroups on a CU), or of one wave's 32 rows and 32 keys in one buffer, eight
// on a CU.  A prompt of 16384 tokens, 32 heads on 8 of 128: 2194 us, 1000 TFLOP/s,
// where a library product of 16384^3 reaches 1395.  The matrix cores are
// busy 51 % of the cycles, the exponentials and sums take about as many issue slots
// as they do, and LDS reads (32 KB a wave and tile) as much time; the clock falls
// as they overlap better (11 % fewer cycles by reading ahead saved 4.5 % of the
// time).  Three waves a SIMD where D = 64 has registers for them (168, all but one
// value that goes to memory): 89 us in place of 95 on 16 ragged prompts in 16411
// tokens, 12 heads.
template <int D, int NW, int KT, bool SPLIT>
__global__ void __launch_bounds__(64 * NW, D == 64 ? 3 : 2) attn_fwd_kernel(const AttnArgs a) {
  constexpr int NT = 64 * NW, BM = 32 * NW, ND = D / 16, NC = D / 32, NJ = KT / 32;
  constexpr int NBUF = NW == 1 ? 1 : 2;
  __shared__ __align__(16) uint16_t sK[NBUF][KT * D], sV[NBUF][KT * D];
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
  const Place at = tile_place<BM>(a.aq, id / a.Hk / (SPLIT ? a.splits : 1), a.slots, a.G, true);
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
  const int kp = rows_place<D>(), cp = cols_place<D>();  // of K's rows, of V's columns
  for (int64_t jt = j0; jt < j1; ++jt) {
    const int b = NBUF == 1 ? 0 : (int)(jt & 1);
    if (NBUF == 1) __syncthreads();
    rk.store(sK[b]);
    rv.store(sV[b]);
    __syncthreads();
    if (jt + 1 < j1) {
      rk.load(kb, a.ks, (jt + 1) * KT, sk.len);
      rv.load(vb, a.vs, (jt + 1) * KT, sk.len);
    }
    const int64_t key0 = jt * KT;
    if (key0 > wend) continue;
    f32x16 S[NJ];
    // Operands are asked for AH products ahead, those of V behind the last of K's:
    // with each read waited for at its product a prompt of 16384 tokens, 32 heads on
    // 8 of 128, took 2297 us in place of 2194.
    constexpr int AH = NW == 4 ? D / 32 : 1, NS = NJ * ND, NP = 2 * NJ * NC;
    bf16x8 kf[AH], vf[AH];
    auto key = [&](int i) { return rows_frag<D>(sK[b], kp, 32 * (i % NJ), i / NJ); };
    auto value = [&](int i) { return cols_frag<D>(sV[b], cp, 16 * (i / NC), i % NC); };
    if constexpr (AH > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int js = 0; js < NJ; ++js) S[js] = zero16();
#pragma unroll
    for (int i = 0; i < AH; ++i) kf[i] = key(i);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      S[i % NJ] = mfma32(kf[i % AH], qf[i / NJ], S[i % NJ]);
      if (i + AH < NS) kf[i % AH] = key(i + AH);
      else vf[i + AH - NS] = value(i + AH - NS);
    }
    if constexpr (AH > 1) {
      __builtin_amdgcn_sched_group_barrier(0x100, AH, 0);
#pragma unroll
      for (int i = AH; i < NS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < AH; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
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
    for (int i = 0; i < NP; ++i) {
      const bf16x8 pf = result_frag(S[i / NC / 2], i / NC % 2);
      O[i % NC] = mfma32(vf[i % AH], pf, O[i % NC]);
      if (i + AH < NP) vf[i % AH] = value(i + AH);
    }
    if constexpr (AH > 1)
#pragma unroll
      for (int i = AH; i < NP; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
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

// The parts of split keys, joined: a row and head has D / 4 lanes for each of GRP
// groups of splits, four of which are asked for at a time: one after another, 64
// parts took 0.6 us each.  What a group has seen is again sums and a maximum, so
// groups are joined as splits are.
template <int D, int GRP>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  constexpr int LR = D / 4, ROWS = 256 / (LR * GRP), U = 4;
  __shared__ float sO[GRP > 1 ? 256 : 1][4], sM[GRP > 1 ? 256 : 1], sS[GRP > 1 ? 256 : 1];
  const int64_t total = a.aq.total * a.Hq, live = axis_rows(a.aq) * a.Hq;
  const int lane = threadIdx.x % LR, grp = threadIdx.x / LR % GRP, c4 = lane * 4;
  const int64_t head = (int64_t)blockIdx.x * ROWS + threadIdx.x / (LR * GRP), hc = head < live ? head : live - 1;
  if (live == 0) return;
  const float *po = a.part + hc * D + c4, *pl = a.part + a.splits * total * D + hc;
  float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.0f, m = -__builtin_inff();
  // takes in sums w, v of weights exp(lse - l)
  auto take = [&](float l, float w, const float (&v)[4]) {
    const float mn = fmaxf(m, l), ms = mn == -__builtin_inff() ? 0.0f : mn;  // no key yet: all weights are 0
    const float f = fexp2((m - ms) * LOG2E), g = fexp2((l - ms) * LOG2E);
    m = mn;
    sum = f * sum + g * w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = f * o[e] + g * v[e];
  };
  for (int s0 = grp; s0 < a.splits; s0 += GRP * U) {
    float l[U], v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t s = s0 + u * GRP < a.splits ? s0 + u * GRP : s0;
      load_f4(po + s * total * D, v[u]);
      l[u] = pl[s * total];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + u * GRP < a.splits) take(l[u], 1.0f, v[u]);
  }
  if constexpr (GRP > 1) {
    const int at = threadIdx.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) sO[at][e] = o[e];
    sM[at] = m;
    sS[at] = sum;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int i = 1; i < GRP; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = sO[at + i * LR][e];
      take(sM[at + i * LR], sS[at + i * LR], v);
    }
  }
  if (head >= live) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  store_out(a, head * D + c4, o);
  if (c4 == 0) a.lse[head] = sum == 0.0f ? -__builtin_inff() : m + __builtin_amdgcn_logf(sum) * LN2;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// d = do.o - dl for every row and head: three arrays read once (30 us for 8219 tokens
// of 32 heads of 128, 6.7 TB/s).
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

// dq: a tile of 128 rows, 32 a wave, which walks the keys 32 at a time.  q and do
// stay in registers as operands, P and dS never leave them.  166 us for 2 x 4097
// tokens of 12 heads of 128 (three products: 930 TFLOP/s; matrix cores busy 53 % of
// the cycles).  With one wave a SIMD and a tile ahead it took 235 us, and reading
// operands ahead as the forward does made no difference.
template <int D>
__global__ void __launch_bounds__(256, 2) attn_dq_kernel(const AttnArgs a) {
  constexpr int NT = 256, BM = 128, KT = 32, ND = D / 16, NC = D / 32;
  __shared__ __align__(16) uint16_t sK[2][KT * D], sV[2][KT * D];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h2 = lane >> 5;
  if ((int64_t)blockIdx.x >= a.main) {
    clear_rows(a.dq, a.aq, (int64_t)a.Hq * D, blockIdx.x - a.main, gridDim.x - a.main);
    return;
  }
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.Hk);
  const Place at = tile_place<BM>(a.aq, id / a.Hk, a.slots, a.G, true);
  const Span sq = span(a.aq, at.n), sk = span(a.ak, at.n);
  const int64_t r0 = at.tile * BM, rows = sq.len * a.G;
  if (r0 >= rows) return;
  const int64_t off = sk.len - sq.len;
  const int64_t row = r0 + 32 * w + (lane & 31), rc = row < rows ? row : rows - 1;
  const int64_t tok = rc / a.G;
  const int g = (int)(rc - tok * a.G);
  const int64_t rl = r0 + BM - 1 < rows ? r0 + BM - 1 : rows - 1;
  const int64_t end = rl / a.G + off + 1;
  const int j1 = end > 0 ? (int)((end + KT - 1) / KT) : 0;
  const int64_t wf = r0 + 32 * w < rows ? r0 + 32 * w : rows - 1;
  const int64_t wall = wf / a.G + off;  // every row of the wave sees the keys up to this one
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
  const int64_t see = tok + off;  // the last key that this lane's row sees
  f32x16 Q[NC];
#pragma unroll
  for (int ct = 0; ct < NC; ++ct) Q[ct] = zero16();
  const uint16_t* kb = a.k + sk.at * a.ks + hk * a.kh;
  const uint16_t* vb = a.v + sk.at * a.vs + hk * a.vh;
  TileRegs<D, KT, NT> rk, rv;
  auto fetch = [&](int jt) {
    rk.load(kb, a.ks, (int64_t)jt * KT, sk.len);
    rv.load(vb, a.vs, (int64_t)jt * KT, sk.len);
  };
  auto stage = [&](int b) {
    rk.store(sK[b]);
    rv.store(sV[b]);
  };
  const int kp = rows_place<D>(), cp = cols_place<D>();
  if (j1 > 0) fetch(0);
  for (int jt = 0; jt < j1; ++jt) {
    const int b = jt & 1;
    stage(b);
    __syncthreads();
    fetch(jt + 1);  // nothing but zeros behind the last key
    f32x16 S = zero16(), P = zero16();
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      S = mfma32(rows_frag<D>(sK[b], kp, 0, kk), qf[kk], S);
      P = mfma32(rows_frag<D>(sV[b], kp, 0, kk), df[kk], P);
    }
    const int64_t key0 = (int64_t)jt * KT;
    if (key0 + KT - 1 > wall) {  // some row does not see all of these keys
      const int64_t left = see - key0;
      const int last = (int)(left < -1 ? -1 : left < KT ? left : KT);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (8 * (e >> 2) + 4 * h2 + (e & 3) > last) S[e] = -__builtin_inff(), P[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) S[e] = fexp2(S[e] * a.c - l2) * (P[e] - dd);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bf16x8 sf = result_frag(S, s);
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) Q[ct] = mfma32(cols_frag<D>(sK[b], cp, 16 * s, ct), sf, Q[ct]);
    }
  }
  if (row >= rows) return;
  __bf16* po = reinterpret_cast<__bf16*>(a.dq) + head * D;
#pragma unroll
  for (int ct = 0; ct < NC; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint2*>(po + 32 * ct + 8 * q + 4 * h2) = round4(
          a.scale * Q[ct][4 * q], a.scale * Q[ct][4 * q + 1], a.scale * Q[ct][4 * q + 2], a.scale * Q[ct][4 * q + 3]);
}

// A tile of 128 keys, 32 a wave, and two streams of rows: waves 0..3 take the
// even tiles of 32 rows, waves 4..7 the odd ones, each with its own sums of dk
// and dv, which are added at the end.  The 128 registers of sums leave room for
// two waves a SIMD, whose products and weights overlap, as long as k and v are
// read from LDS as operands: held in registers (one wave a SIMD, a tile ahead)
// the same work took 384 us in place of 264 (2 x 4097 tokens x 12 heads of 128: 780
// TFLOP/s of the four products).
//
// With few tiles (few key heads, whose groups make each tile's rows many) the rows
// of a tile are split over workgroups, which leave fp32 sums to be added (for 128
// channels one value a lane goes to memory there).
template <int D, bool SPLIT>
__global__ void __launch_bounds__(512, 2) attn_dkv_kernel(const AttnArgs a) {
  constexpr int NT = 256, BN = 128, RT = 32, ND = D / 16, NC = D / 32;
  __shared__ __align__(16) uint16_t sKV[2][BN * D], sR[2][2][2][RT * D];  // k, v; q, do of a stream's two buffers
  __shared__ __align__(16) float sL[2][2][RT], sE[2][2][RT];              // lse log2(e) and d of the rows
  __shared__ __align__(16) int sT[2][2][RT];  // the last key that each row sees, from this tile's first
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6 & 3, h2 = lane >> 5, st = threadIdx.x >> 8, t = threadIdx.x & 255;
  if ((int64_t)blockIdx.x >= a.main) {
    clear_rows(a.dk, a.ak, (int64_t)a.Hk * D, blockIdx.x - a.main, gridDim.x - a.main);
    clear_rows(a.dv, a.ak, (int64_t)a.Hk * D, blockIdx.x - a.main, gridDim.x - a.main);
    return;
  }
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.Hk);
  const int split = SPLIT ? (int)(id / a.Hk % a.splits) : 0;
  const Place at = tile_place<BN>(a.ak, id / a.Hk / (SPLIT ? a.splits : 1), a.slots, 1, false);
  const Span sq = span(a.aq, at.n), sk = span(a.ak, at.n);
  const int64_t key0 = at.tile * BN;
  if (key0 >= sk.len) return;
  const int64_t off = sk.len - sq.len, rows = sq.len * a.G;
  const int64_t t0 = key0 > off ? key0 - off : 0;  // first token that sees a key of the tile
  int64_t i0 = t0 * a.G / RT, i1 = (rows + RT - 1) / RT;
  if (SPLIT) {  // pairs of tiles, one for each stream
    const int64_t pairs = i1 > i0 ? (i1 - i0 + 1) / 2 : 0, per = (pairs + a.splits - 1) / a.splits * 2;
    i0 += per * split;
    i1 = i0 + per < i1 ? i0 + per : i1;
  }
  {
    TileRegs<D, BN, 512> r;
    r.load(a.k + sk.at * a.ks + hk * a.kh, a.ks, key0, sk.len);
    r.store(sKV[0]);
    r.load(a.v + sk.at * a.vs + hk * a.vh, a.vs, key0, sk.len);
    r.store(sKV[1]);
  }
  f32x16 K[NC], V[NC];
#pragma unroll
  for (int ct = 0; ct < NC; ++ct) {
    K[ct] = zero16();
    V[ct] = zero16();
  }

  // The next tile's first row is head ng of token nt; a row of the tile is
  // (ng + row) / G tokens further (by a multiplication: (G + 32) G < 2^32).
  constexpr int PR = NT / (D / 8), U = RT / PR;
  const uint32_t recip = a.G > 1 ? (uint32_t)((((uint64_t)1 << 32) + a.G - 1) / a.G) : 0;
  const int stepT = 2 * RT / a.G, stepG = 2 * RT % a.G;
  int64_t nrow = (i0 + st) * RT, nt = nrow / a.G;
  int ng = (int)(nrow - nt * a.G);
  uint4 rq[U], rd[U];
  uint32_t rl = 0, re = 0;
  int rt = -1;
  const int mine = t / (D / 8), c16 = t % (D / 8) * 16;
  auto fetch = [&]() {
    const __amdgpu_buffer_rsrc_t dq = buf(a.q + (sq.at + nt) * a.qs + (int64_t)hk * a.G * a.qh, 0x7fffffffu);
    const int64_t h0 = (sq.at + nt) * a.Hq + (int64_t)hk * a.G;
    const __amdgpu_buffer_rsrc_t dd = buf(a.d_out + h0 * D, 0x7fffffffu);
    const int left = (int)(rows - nrow < RT ? rows - nrow : RT);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = mine + PR * u, n = ng + r;
      const int tk = a.G > 1 ? (int)__umulhi((uint32_t)n, recip) : n, g = n - tk * a.G;
      rq[u] = bload<uint4>(dq, r < left ? (tk * (int)a.qs + g * (int)a.qh) * 2 + c16 : (int)0x80000000, 0);
      rd[u] = bload<uint4>(dd, r < left ? (tk * a.Hq + g) * D * 2 + c16 : (int)0x80000000, 0);
    }
    if (t < RT) {
      const int n = ng + t;
      const int tk = a.G > 1 ? (int)__umulhi((uint32_t)n, recip) : n, g = n - tk * a.G;
      const int o = t < left ? (tk * a.Hq + g) * 4 : (int)0x80000000;
      rl = __builtin_amdgcn_raw_buffer_load_b32(buf(a.lse + h0, 0x7fffffffu), o, 0, 0);
      re = __builtin_amdgcn_raw_buffer_load_b32(buf(a.delta + h0, 0x7fffffffu), o, 0, 0);
      const int64_t last = nt + tk + off - key0;
      rt = t < left ? (int)(last < -1 ? -1 : last < BN ? last : BN) : -1;
    }
    nrow += 2 * RT;
    nt += stepT;
    ng += stepG;
    if (ng >= a.G) ng -= a.G, ++nt;
  };
  auto stage = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int to = at_tile<D>(mine + PR * u, c16 / 2);
      *reinterpret_cast<uint4*>(sR[st][b][0] + to) = rq[u];
      *reinterpret_cast<uint4*>(sR[st][b][1] + to) = rd[u];
    }
    if (t < RT) {
      const float l = __uint_as_float(rl);
      sL[st][b][t] = l == -__builtin_inff() ? 0.0f : l * LOG2E;  // a row that sees no key: all is masked
      sE[st][b][t] = __uint_as_float(re);
      sT[st][b][t] = rt;
    }
  };
  int64_t first = (i0 + st) * RT / a.G;  // the current tile's first token, and its first row's head
  int fg = (int)((i0 + st) * RT - first * a.G);
  const int kp = rows_place<D>(), cp = cols_place<D>();
  if (i0 < i1) fetch();
  for (int64_t it = i0; it < i1; it += 2) {  // the streams keep step: one may end with a tile behind the last row
    const int b = (int)((it - i0) >> 1 & 1);
    stage(b);
    __syncthreads();
    fetch();  // nothing but zeros behind the last row
    const uint16_t *tq = sR[st][b][0], *td = sR[st][b][1];
    f32x16 S = zero16(), P = zero16();
#pragma unroll
    for (int kk = 0; kk < ND; ++kk) {
      S = mfma32(rows_frag<D>(tq, kp, 0, kk), rows_frag<D>(sKV[0], kp, 32 * w, kk), S);
      P = mfma32(rows_frag<D>(td, kp, 0, kk), rows_frag<D>(sKV[1], kp, 32 * w, kk), P);
    }
    // Rows that do not see all keys of the tile; those behind the last one need
    // no mask, their q, do and d are zeros.
    if (first + off - key0 < BN - 1) {
      const int my = 32 * w + (lane & 31);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int4 t4 = *reinterpret_cast<const int4*>(&sT[st][b][8 * q + 4 * h2]);
        const int tv[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (my > tv[e]) S[4 * q + e] = -__builtin_inff(), P[4 * q + e] = 0.0f;
      }
    }
    first += stepT;
    fg += stepG;
    if (fg >= a.G) fg -= a.G, ++first;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float lv[4], ev[4];
      lds_f32x4(&sL[st][b][8 * q + 4 * h2], lv);
      lds_f32x4(&sE[st][b][8 * q + 4 * h2], ev);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[4 * q + e] = fexp2(S[4 * q + e] * a.c - lv[e]);
        P[4 * q + e] = S[4 * q + e] * (P[4 * q + e] - ev[e]);
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bf16x8 pf = result_frag(S, s), sf = result_frag(P, s);
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        V[ct] = mfma32(cols_frag<D>(td, cp, 16 * s, ct), pf, V[ct]);
        K[ct] = mfma32(cols_frag<D>(tq, cp, 16 * s, ct), sf, K[ct]);
      }
    }
  }

  // ---- the second stream's sums to the first, dv and then dk through the LDS of k and v
  float4* box = reinterpret_cast<float4*>(&sKV[0][0]) + w * 64 * NC * 4 + lane;  // 16 NC floats a lane: BN D halves in all
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    f32x16* X = part == 0 ? V : K;
    __syncthreads();
    if (st == 1) {
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          box[(4 * ct + q) * 64] = make_float4(X[ct][4 * q], X[ct][4 * q + 1], X[ct][4 * q + 2], X[ct][4 * q + 3]);
    }
    __syncthreads();
    if (st == 0) {
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 y = box[(4 * ct + q) * 64];
          X[ct][4 * q] += y.x, X[ct][4 * q + 1] += y.y, X[ct][4 * q + 2] += y.z, X[ct][4 * q + 3] += y.w;
        }
    }
  }
  const int64_t key = key0 + 32 * w + (lane & 31);
  if (st == 1 || key >= sk.len) return;
  const int64_t to = ((sk.at + key) * a.Hk + hk) * D;
  if (SPLIT) {
    const int64_t size = a.ak.total * a.Hk * D;
    float* pk = a.part + 2 * split * size + to;
#pragma unroll
    for (int ct = 0; ct < NC; ++ct)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int o = 32 * ct + 8 * q + 4 * h2;
        *reinterpret_cast<float4*>(pk + o) = make_float4(K[ct][4 * q], K[ct][4 * q + 1], K[ct][4 * q + 2], K[ct][4 * q + 3]);
        *reinterpret_cast<float4*>(pk + size + o) = make_float4(V[ct][4 * q], V[ct][4 * q + 1], V[ct][4 * q + 2], V[ct][4 * q + 3]);
      }
    return;
  }
#pragma unroll
  for (int ct = 0; ct < NC; ++ct)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = 32 * ct + 8 * q + 4 * h2;
      *reinterpret_cast<uint2*>(a.dk + to + o) = round4(a.scale * K[ct][4 * q], a.scale * K[ct][4 * q + 1],
                                                        a.scale * K[ct][4 * q + 2], a.scale * K[ct][4 * q + 3]);
      *reinterpret_cast<uint2*>(a.dv + to + o) = round4(V[ct][4 * q], V[ct][4 * q + 1], V[ct][4 * q + 2], V[ct][4 * q + 3]);
    }
}

// The sums of split rows, added in order: four values of dk and dv a thread.
__global__ void __launch_bounds__(256) attn_sum_kernel(const AttnArgs a, int64_t row) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, size = a.ak.total * row;
  if (at >= axis_rows(a.ak) * row) return;
  float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    float x[4], y[4];
    load_f4(a.part + 2 * s * size + at, x);
    load_f4(a.part + (2 * s + 1) * size + at, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k[e] += x[e];
      v[e] += y[e];
    }
  }
  *reinterpret_cast<uint2*>(a.dk + at) = round4(a.scale * k[0], a.scale * k[1], a.scale * k[2], a.scale * k[3]);
  *reinterpret_cast<uint2*>(a.dv + at) = round4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// How a forward is cut: rows of a tile (32, a wave, or 128, four waves), and parts
// of the keys.  Measured, us, on 8 key heads of 128 with 4 query heads each, both
// sides of each rule:
// - Rows of a tile.  One wave where it has all rows of a sequence, or where keys
//   are few: 64 sequences of 24 tokens by themselves, 12.6 (128 rows: 16.4).  More
//   rows on long keys share what they read: 16 sequences, 14 tokens behind 4096,
//   55 (32 rows: 87).
// - Parts.  One round of 128-row workgroups, two on a CU (16 sequences, 18 tokens
//   behind 4096: 59, two rounds 75), or of single waves, eight on a CU (64 tokens
//   behind 8191 each: 370, half of that 412), as long as the parts' own traffic is a
//   sixteenth of the keys' or most CUs would be idle without (16 sequences, 8 tokens
//   behind 4096: 57, without this limit 73).  At most 64 (1 token behind 65535: 45,
//   with 256 parts 53), of 128 or 256 keys at least (1 token of 8 heads on one key
//   head behind 8191: 12.7, with 256 16.3; 24 tokens behind 8000: 20.2, with 128 22.4).
// The host knows the mean of the keys alone, and every sequence gets as many parts.
// Packed single tokens with very unequal keys wait for the longest: one of 131072
// keys among 63 of 16 takes 1041 (by itself 104), 8 of 16384 among 56 of 16 148, where
// 64 of 2064 take 110 and 64 of 1 to 4127 120.
struct AttnPlan {
  int bm;
  int64_t slots;
  int splits;
  size_t bytes;
};
AttnPlan attn_plan(int64_t tq, int64_t tk, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  AttnPlan p;
  const int64_t rows = tq * (Hq / Hk);
  const int64_t keys = tk / N;
  p.bm = rows <= 32 * N || (rows <= 128 * N && keys <= 256) ? 32 : 128;
  p.slots = rows / p.bm + N;
  // tiles that hold rows, as far as the host knows
  const int64_t tiles = ((rows + p.bm - 1) / p.bm > N ? (rows + p.bm - 1) / p.bm : (rows < N ? rows : N)) * Hk;
  int64_t s = 1;
  if (tiles > 0) {
    s = p.bm == 128 ? 2 * kAttnRound / tiles : 8 * kAttnRound / tiles;
    const int64_t least = p.bm == 128 ? 256 : 128, most = (keys + least - 1) / least;
    const int64_t few = kAttnRound / tiles, light = keys * N / (32 * rows);
    if (p.bm == 32 && s > few && s > light) s = few > light ? few : light;
    s = s < most ? s : most;
  }
  p.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  p.bytes = p.splits > 1 ? align256((size_t)p.splits * (size_t)(tq * Hq) * (size_t)(D + 1) * sizeof(float)) : 0;
  return p;
}

// Workgroups that the rows of a backward's tile of keys are split over: two
// rounds of the card's CUs in all (a workgroup's LDS fills one), each with 8
// pairs of row tiles at least.  A whole backward, us, unsplit and split: 1 x 1500
// tokens of 16 heads on 2 key heads of 128, 434 and 98; 1 x 2000, 32 on 8, 337
// and 189 (four rounds 217); 1 x 4096, 32 on 8, 765 and 570 (610); 2 x 1024, 8 on
// 8, 79 and 73 (with 4 pairs at least 82).
int attn_bwd_splits(int64_t tq, int64_t tk, int64_t Hq, int64_t Hk, int64_t N) {
  const int64_t tiles = (tk + 127) / 128 * Hk, most = tq / N * (Hq / Hk) / 512;
  int64_t s = tiles > 0 ? (kAttnRound * 2 + tiles / 2) / tiles : 1;
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}
size_t attn_delta_bytes(int64_t tq, int64_t Hq) { return align256((size_t)(tq * Hq) * sizeof(float)); }

kda_status_t attn_check(AttnArgs& a, const void* q, int64_t qs, int64_t qh, const void* k, int64_t ks, int64_t kh,
                        const void* v, int64_t vs, int64_t vh, float scale, const int32_t* cq, const int32_t* ck,
                        int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t N, unsigned flags) {
  if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hk < 1 || N < 1 || Hq % Hk != 0) return KDA_ERR_INVALID;
  if ((cq == nullptr) != (ck == nullptr)) return KDA_ERR_INVALID;
  if (cq ? B != 1 : N != B) return KDA_ERR_INVALID;
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  if (flags & ~FLAG_ZERO_REST) return KDA_ERR_INVALID;
  if (Hq > 1 << 15 || N > 1 << 30 || !fits(B, Tq, kMaxElements) || !fits(B, Tk, kMaxElements) ||
      !fits(B * Tq, Hq * D, kMaxElements) || !fits(B * Tk, Hk * D, kMaxElements) || Tq >= (int64_t)1 << 31 ||
      Tk >= (int64_t)1 << 31)
    return KDA_ERR_INVALID;
  if (!(scale > 0.0f) || !(scale - scale == 0.0f)) return KDA_ERR_INVALID;
  if ((B * Tq > 0 && !q) || (B * Tk > 0 && (!k || !v))) return KDA_ERR_INVALID;
  if (!mix_strides_ok(qs, qh) || !mix_strides_ok(ks, kh) || !mix_strides_ok(vs, vh)) return KDA_ERR_INVALID;
  // 32-bit byte offsets within 32 rows of q
  if (Hq / Hk * qh + 33 * qs >= (int64_t)1 << 30) return KDA_ERR_INVALID;
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

bool attn_sizes_ok(int64_t tq, int64_t tk, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  return tq >= 0 && tk >= 0 && Hq >= 1 && Hk >= 1 && Hq <= 1 << 15 && Hq % Hk == 0 && (D == 64 || D == 128) && N >= 1 &&
         N <= 1 << 30 && fits(tq, Hq * D, kMaxElements) && fits(tk, Hk * D, kMaxElements);
}

// Workgroups that clear the rows of no sequence.
int64_t attn_clear(const int32_t* cu, unsigned flags) { return cu && (flags & FLAG_ZERO_REST) ? 64 : 0; }

// Whether tiles times heads times splits workgroups of `threads`, and those that
// clear, are a grid.
bool attn_fits(int64_t tiles, int64_t heads, int64_t splits, int64_t clear, int threads) {
  return tiles <= (most_groups(threads) - clear) / heads / splits;
}

template <int D>
kda_status_t attn_run_fwd(AttnArgs& a, const AttnPlan& p, int64_t clear, hipStream_t st) {
  a.slots = p.slots;
  a.splits = p.splits;
  // (keys are split for few rows only: the join's grid is small)
  if (!attn_fits(p.slots, a.Hk, p.splits, clear, p.bm == 32 ? 64 : 256)) return KDA_ERR_INVALID;
  a.main = p.slots * a.Hk * p.splits;
  if (p.splits == 1)
    return p.bm == 32 ? launch(&attn_fwd_kernel<D, 1, 32, false>, a.main + clear, 64, st, "attention", a)
                      : launch(&attn_fwd_kernel<D, 4, 64, false>, a.main + clear, 256, st, "attention", a);
  const kda_status_t s = p.bm == 32 ? launch(&attn_fwd_kernel<D, 1, 32, true>, a.main + clear, 64, st, "attention parts", a)
                                    : launch(&attn_fwd_kernel<D, 4, 64, true>, a.main + clear, 256, st, "attention parts", a);
  if (s != KDA_SUCCESS) return s;
  const int64_t heads = a.aq.total * a.Hq, per = 256 / (D / 4);
  return p.splits <= 8 ? launch(&attn_join_kernel<D, 1>, (heads + per - 1) / per, 256, st, "attention join", a)
                       : launch(&attn_join_kernel<D, 8>, (heads + per / 8 - 1) / (per / 8), 256, st, "attention join", a);
}

template <int D>
kda_status_t attn_run_bwd(AttnArgs& a, const void* out, const void* out_lo, const float* d_lse, float* delta, int64_t clear, hipStream_t st) {
  const int64_t heads = a.aq.total * a.Hq, per = 256 / (D / 8);
  a.delta = delta;
  a.slots = a.ak.total / 128 + a.ak.N;
  a.splits = attn_bwd_splits(a.aq.total, a.ak.total, a.Hq, a.Hk, a.ak.N);
  const int64_t rows = a.aq.total * a.G / 128 + a.aq.N;  // tiles of rows
  // Nothing is enqueued unless all of it can be (rows are split for few tiles of keys
  // only: the sums' grid is small).
  if ((heads + per - 1) / per > most_groups(256) || !attn_fits(a.slots, a.Hk, a.splits, clear, 512) ||
      !attn_fits(rows, a.Hk, 1, clear, 256))
    return KDA_ERR_INVALID;
  if (heads > 0) {
    const kda_status_t s = launch(&attn_delta_kernel<D>, (heads + per - 1) / per, 256, st, "attention delta",
                                  static_cast<const uint16_t*>(out), static_cast<const uint16_t*>(out_lo), a.d_out, d_lse,
                                  delta, heads);
    if (s != KDA_SUCCESS) return s;
  }
  a.main = a.slots * a.Hk * a.splits;
  kda_status_t s = a.splits == 1 ? launch(&attn_dkv_kernel<D, false>, a.main + clear, 512, st, "attention dk, dv", a)
                                 : launch(&attn_dkv_kernel<D, true>, a.main + clear, 512, st, "attention dk, dv parts", a);
  if (s != KDA_SUCCESS) return s;
  if (a.splits > 1) {
    const int64_t row = (int64_t)a.Hk * D;
    s = launch(&attn_sum_kernel, (a.ak.total * row / 4 + 255) / 256, 256, st, "attention dk, dv sums", a, row);
    if (s != KDA_SUCCESS) return s;
  }
  a.slots = rows;
  a.main = a.slots * a.Hk;
  return launch(&attn_dq_kernel<D>, a.main + clear, 256, st, "attention dq", a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_attn_workspace_size(int64_t Tq_total, int64_t Tk_total, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  if (!attn_sizes_ok(Tq_total, Tk_total, Hq, Hk, D, N)) return 0;
  return attn_plan(Tq_total, Tk_total, Hq, Hk, D, N).bytes;
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
  const AttnPlan p = attn_plan(B * Tq, B * Tk, Hq, Hk, D, N);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return KDA_ERR_WORKSPACE;
  if (B * Tq == 0) return KDA_SUCCESS;
  a.out = static_cast<uint16_t*>(out);
  a.out_lo = static_cast<uint16_t*>(out_lo);
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t clear = attn_clear(cu_seqlens_q, flags);
  return D == 128 ? attn_run_fwd<128>(a, p, clear, st) : attn_run_fwd<64>(a, p, clear, st);
}

size_t kda_attn_bwd_workspace_size(int64_t Tq_total, int64_t Tk_total, int64_t Hq, int64_t Hk, int64_t D, int64_t N) {
  if (!attn_sizes_ok(Tq_total, Tk_total, Hq, Hk, D, N)) return 0;
  const int splits = attn_bwd_splits(Tq_total, Tk_total, Hq, Hk, N);
  return 256 + attn_delta_bytes(Tq_total, Hq) +
         (splits > 1 ? align256((size_t)splits * 2 * (size_t)(Tk_total * Hk * D) * sizeof(float)) : 0);
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
  if (!workspace || workspace_bytes < kda_attn_bwd_workspace_size(B * Tq, B * Tk, Hq, Hk, D, N)) return KDA_ERR_WORKSPACE;
  a.lse = const_cast<float*>(lse);
  a.d_out = static_cast<const uint16_t*>(d_out);
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t clear = attn_clear(cu_seqlens_q, flags);
  float* delta = static_cast<float*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + attn_delta_bytes(B * Tq, Hq));
  return D == 128 ? attn_run_bwd<128>(a, out, out_lo, d_lse, delta, clear, st)
                  : attn_run_bwd<64>(a, out, out_lo, d_lse, delta, clear, st);
}

}  // extern "C"
