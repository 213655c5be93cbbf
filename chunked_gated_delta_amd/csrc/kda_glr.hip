// Gated linear recurrence: the diagonal recurrence under KDA's own decay gate,
//     g_t = lower_bound * sigmoid(exp(A_log) (raw_gate_t + dt_bias))   (or given)
//     a_t = exp(g_t),   h_t = a_t h_{t-1} + b_t x_t,   b_t = 1 or 1 - a_t,
// per channel of [tokens][H * K], its gradients, and its step for decoding.
//
// A run of tokens maps the state that enters it to h -> A h + B (A the product
// of its decays, B its result from zero), and such maps compose.  The packed
// token axis is cut into tiles of rows by 64 channels, whatever the sequences: a
// tile that holds the first row of a sequence has a map that does not depend on
// the entering state (it is reset: the composition selects, it does not multiply
// by zero, so that a sequence's NaN or infinity stays in it).  A tile is 512
// threads, one workgroup a CU: seven waves hold 28 runs of 8 rows (bf16; 4 in
// fp32 and in the backward) in registers, 16 lanes of 4 channels each, and one
// wave joins the runs, a lane a channel.
//
// One pass over the data: a workgroup takes the tiles in order from a counter,
// loads its tile once, publishes the tile's map, finds the state that enters it
// and writes the outputs from registers.  To find that state it looks for the
// nearest of the 32 tiles before it whose entering state is known and applies
// the maps of the tiles in between, in order.  The leaving state of a tile is
// always its map applied to its entering state, so the result has the same bits
// however far back the search ends.  A tile waits only for tiles that running
// workgroups took before it; the wait is bounded all the same, and one that
// gives up sets the workspace's fault word and takes NaN for the state.
//
// What bounds it: memory, where there are many columns.  At 32768 rows x 12288
// channels of bf16 the pass takes 0.47 ms, 5.1 TB/s of its 6 bytes an element (a
// copy reaches 5.2 on the same card); reading the inputs twice, with the states
// folded between two launches, took 1.20 ms.  With few columns every column has
// more tiles in flight than its entering states can travel through, at two or
// three round trips of about 1 us a hop: 262144 x 1024 takes 0.42 ms (3.8 TB/s).
// Measured on the way there: 64-row tiles with two workgroups a CU 0.72 ms; all
// tickets from one counter 13 ns a tile, whatever it did; the joining wave at
// default priority 0.65 ms; rows that ask for marks one by one 0.57 ms.
//
// Backward, with dh_t = d_out_t + a_{t+1} dh_{t+1} (d_final joins at the last
// row) and e_t = a_t dh_t, the gradient that row t hands to the row before:
//     dx_t = b_t dh_t,   dg_t = a_t dh_t (h_{t-1} [- x_t if b = 1 - a])
// the same pass runs over e from the right; h_{t-1} is recomputed from the
// states entering every 112 rows, which the forward leaves.  At 32768 x 12288 it
// takes 0.94 ms, 4.3 TB/s of its 10 bytes an element (1.03 ms with the slopes of
// the gates formed twice and the gates' parameters loaded by every wave); at
// 69141 x 4096, with four tiles of a column at work, 0.84 ms, 3.4 TB/s: 0.73 of
// them without the waits for entering states, 0.53 if rows and results also
// stayed in the caches.
//
// In fp32: forward 32768 x 6144 0.48 ms and 69141 x 4096 0.72 ms (4.8 TB/s),
// backward there 1.10 ms (5.1 TB/s).
//
// Registers: the data waves' rows fill them.  The compiler spills two in the
// bf16 forwards with formed gates, five and six in the fp32 backwards with
// formed gates, none in the others; 50 to 97 scalar registers a kernel live in
// lanes of a vector register instead of memory.
//
// All arithmetic is fp32.

#include <limits.h>

#include <type_traits>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_token.h"

namespace kda {
namespace {

constexpr int GS = 28;           // runs of a tile
constexpr int GC = 64;           // channels of a tile
constexpr int GW = GC / 4;       // lanes of a row
constexpr int GD = GS * GW;      // threads that hold data: seven waves
constexpr int GT = GD + GC;      // and one, a lane a channel, that finds what enters the tile
static_assert(GD % 64 == 0 && GT == 512 && GS <= 32, "whole waves, runs in a 32-bit mask");
// Rows of a run: as many as the registers of one workgroup a CU hold.  More
// rows a tile mean fewer tiles in flight on a column, and so less waiting, for
// the same bytes.  The forward has 8 of bf16 and 4 of fp32, tiles of 224 and 112
// rows; the backward, which holds three arrays and h_{t-1}, has 4 of both.
constexpr int BR = 4, BL = BR * GS;
template <typename T>
constexpr int FR = sizeof(T) == 2 ? 2 * BR : BR;
template <typename T>
constexpr int FL = FR<T> * GS;
constexpr int L_MAX = 2 * BL;
constexpr int64_t kMaxChannels = (int64_t)1 << 21;  // a tile's rows span less than 2^30 bytes

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
  const float* states;  // [backward tiles][C] state entering every BL rows
  // the pass's own, tiles counted in its order (the backward from the right):
  uint64_t* enter; // [tiles][C] what enters every tile, with KNOWN above it
  uint64_t* maps;  // [tiles][C] A (with KNOWN_MAP) and B of every tile's map
  float* keep;     // forward: what enters every BL rows, for the backward, or NULL
  int* tickets;   // [sets] the next tile of each set of columns, TICKET_LINE apart
  int sets;
  unsigned* faults;
  float2* part;   // [tiles][C] sums over the tile of d_raw and of dz z
  double* zsum;   // [C] sums of dz z
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

// The gates of a tile's columns, by the wave that joins: asked for a tile ahead
// of their use, and written where the seven waves find them.
template <bool STAGED>
struct Gates {
  int blk = -1;  // the column block that is in hand: a workgroup's tiles are often of one
  float al, dt;
  __device__ __forceinline__ void ask(const GlrArgs& a, int2 item, int ch) {
    if (!STAGED || item.x >= a.ntiles || item.y == blk) return;
    blk = item.y;
    const uint32_t c = (uint32_t)blk * GC + ch;
    const bool in = c < (uint32_t)a.C;
    al = in ? a.A_log[c / (uint32_t)a.K] : 0.f;
    dt = in ? a.dt_bias[c] : 0.f;
  }
  __device__ __forceinline__ void put(float (&gate)[2][GC], int ch) const {
    if constexpr (STAGED) {
      const float na = -expf(al) * LOG2E;
      gate[0][ch] = na;
      gate[1][ch] = na * dt;
    }
  }
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
  // The same out of LDS, where the wave that joins has put it: a load here
  // would come back behind every row that the wave has asked for.
  __device__ __forceinline__ void init(const GlrArgs& a, const float (&gate)[2][GC], int at) {
    if constexpr (!GIVEN) {
      na = gate[0][at];
      load_f4(&gate[1][at], nb);
      lb2 = a.lb * LOG2E;
    }
  }
  // g log2(e)
  __device__ __forceinline__ float g2(float raw, int j) const {
    if constexpr (GIVEN) return raw * LOG2E;
    return lb2 * __builtin_amdgcn_rcpf(1.0f + fexp2(raw * na + nb[j]));
  }
  // and s (1 - s) = w s^2, with s = sigmoid(z) and w = exp(-z), its slope but
  // for constants.  The w outside of s is kept finite so that w s does not
  // become infinity times zero (a NaN is in s as well).
  __device__ __forceinline__ float g2(float raw, int j, float& slope) const {
    const float w = fexp2(raw * na + nb[j]), s = __builtin_amdgcn_rcpf(1.0f + w);
    slope = fminf(w, 0x1p126f) * s * s;
    return lb2 * s;
  }
  // the slope alone, from -z log2(e) (held finite by a comparison: NaN stays)
  __device__ __forceinline__ float slope(float mz) const {
    const float w = fexp2(mz > 126.f ? 126.f : mz), s = __builtin_amdgcn_rcpf(1.0f + w);
    return s * (w * s);
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

// The sequences that start (S) or end (E) at each row of the tile at t0, -1 for
// none, and whether there is any, or any row behind the last sequence; by one
// wave.  S and E are only written where there is.
struct Marks {
  int S[L_MAX], E[L_MAX], any;
};
__device__ __forceinline__ void mark_tile(const Axis& ax, int64_t t0, int tile_len, int64_t rows, Marks& m) {
  const int lane = threadIdx.x & 63;
  const int64_t t1 = t0 + tile_len;
  if (!ax.cu && ax.N == 1 && t0 > 0 && t1 < rows) {  // inside the one sequence
    if (lane == 0) m.any = 0;
    return;
  }
  // n0, n1: first sequences that start at t0, t1 or behind
  const int64_t n0 = axis_lower(ax, t0);
  int64_t n1 = n0;
  if (ax.cu) {
    const bool before = n0 + lane <= ax.N && axis_start(ax, n0 + lane) < t1;
    n1 += __popcll(__ballot(before));
    if (n1 == n0 + 64) n1 = axis_lower(ax, t1);
  } else {
    n1 = axis_lower(ax, t1);
  }
  // (an end is the next one's start, so one at the very end of the tile is no start of it)
  const bool any = n1 > n0 || (n0 <= ax.N && axis_start(ax, n0) == t1) || t1 > rows;
  if (lane == 0) m.any = any;
  if (!any) return;
  for (int i = lane; i < tile_len; i += 64) m.S[i] = m.E[i] = -1;
  n1 = n1 < ax.N ? n1 : ax.N;
  __builtin_amdgcn_wave_barrier();
  // sequence n0 - 1 is the one that reaches the tile from before it
  for (int64_t n = (n0 > 0 ? n0 - 1 : 0) + lane; n < n1; n += 64) {
    const int64_t s = axis_start(ax, n), e = axis_start(ax, n + 1);
    if (e <= s) continue;
    if (s >= t0 && s < t1) m.S[s - t0] = (int)n;
    if (e > t0 && e <= t1) m.E[e - 1 - t0] = (int)n;
  }
}

// Loads and stores of a tile by 32-bit offsets from its first row.  The
// descriptor ends behind the last row that belongs to a sequence: rows behind
// it load as zeros and are not stored, and so does an offset of OUTSIDE.  All of
// an offset is in the lane's register: the intrinsics leave the scalar offset
// out of the check against the descriptor's end, so that with a row's offset
// there the last tile read rows behind the array.  (No slower: 32704 x 12288 of
// bf16 472 us forward and 936 backward, 470 and 940 with scalar offsets.)
constexpr int OUTSIDE = 0x40000000;  // past any tile, also with a row's offset added
template <typename T, int L>
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Rows(const void* base, int64_t t0, int64_t rows, int64_t C) {
    const int64_t left = rows - t0 < L ? rows - t0 : L;
    r = buf(static_cast<const T*>(base) + t0 * C, (uint32_t)((left > 0 ? left : 0) * C * sizeof(T)));
  }
  __device__ __forceinline__ raw4<T> load(int voff, int off) const {
    if constexpr (sizeof(T) == 2) {
      return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, voff + off, 0, 0));
    } else {
      return __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(r, voff + off, 0, 0));
    }
  }
  // With the row's offset in a scalar register, one build of the 16-byte store
  // gave single wrong fp32 outputs: the first element of a lane's four.  The
  // assembly of that build wrote the store's first data register in the very
  // next instruction.  The compiler keeps such writes away from stores of more
  // than 8 bytes, except from those with a scalar offset, which the public ISA
  // guides exempt; that the exemption does not hold here is inferred from this
  // one build and not otherwise established.  Without a scalar offset the
  // question does not arise.
  __device__ __forceinline__ void store(int voff, int off, const float (&d)[4]) const {
    if constexpr (sizeof(T) == 2) {
      bf16x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (__bf16)d[i];
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), r, voff + off, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, make_float4(d[0], d[1], d[2], d[3])), r,
                                             voff + off, 0, 0);
    }
  }
};

// Device-scope words that other workgroups write while this kernel runs, all by
// relaxed atomics, which go to where the XCDs agree.  A word carries its value
// and the sign that it is there, so nothing has to be ordered: what leaves a
// tile has KNOWN above it, and a map has KNOWN_MAP in the sign of its A, a
// product of exponentials, which has none of its own.  A round trip takes
// microseconds under load, so none is spent on waiting for a store and then
// flagging it.
constexpr uint64_t KNOWN = (uint64_t)1 << 32;
constexpr uint32_t KNOWN_MAP = 0x80000000u;
template <typename W>
__device__ __forceinline__ W peek(const W* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ void post(W* p, W v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Rounds before a wait gives up (more than a second: each is a round trip to memory).
constexpr int kPolls = 1 << 21;

// What enters tile k (tiles counted in the pass's order) at channel c: its own
// word, or the word of a tile up to REACH before it with the maps in between
// applied, in order.  `word` is a first look at its own.  Where that is not
// there yet, the maps of the tiles before are collected in LDS, the nearest
// first and a batch a round, and every round looks at the words of several
// distances at once, so that a value that arrives anywhere in reach is taken up
// in one round trip.
constexpr int REACH = 32, BATCH = 8;
typedef uint64_t Maps[REACH][GC];
// Of a row of words (a wave-uniform address) the one of channel c.
__device__ __forceinline__ uint64_t peek_row(const uint64_t* row, uint32_t c) { return peek(row + c); }
__device__ __forceinline__ float look_back(const GlrArgs& a, Maps& maps, int k, int64_t c, bool in, uint64_t word) {
  constexpr int ND = 7;
  if (__all((word & KNOWN) != 0)) return __uint_as_float((uint32_t)word);
  const int ch = threadIdx.x & 63;
  const uint32_t at = in ? (uint32_t)c : 0;
  const int before = k < REACH ? k : REACH;  // tiles in reach
  const uint64_t* enter = a.enter + (int64_t)k * a.C;
  uint32_t have = 0;  // maps that are there, in all channels: bit u, of tile k - 1 - u
  for (int poll = 0; poll < kPolls; ++poll) {
    // one round trip: the words, and the nearest BATCH maps that are not all there yet
    const int u0 = have == ~0u ? REACH : __builtin_ctz(~have) & -BATCH;
    const int reach = u0 + BATCH < before ? u0 + BATCH : before;
    uint64_t w[ND], m[BATCH];  // entering words at distances 0, 1, 2, 4, 8, 16, 32
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = i == 0 ? 0 : 1 << (i - 1);
      w[i] = d <= reach ? peek_row(enter - d * a.C, at) : 0;
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) m[u] = u0 + u < reach ? peek_row(a.maps + (int64_t)(k - 1 - u0 - u) * a.C, at) : 0;
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (u0 + u < reach) {
        maps[u0 + u][ch] = m[u];
        if (__all(!in || (m[u] & KNOWN_MAP) != 0)) have |= 1u << (u0 + u);
      }
    float s = 0.f;
    int found = -1;
#pragma unroll
    for (int i = ND - 1; i >= 0; --i) {
      const int d = i == 0 ? 0 : 1 << (i - 1);
      const uint32_t need = d == 32 ? ~0u : (1u << (d & 31)) - 1;
      if (d <= reach && (have & need) == need && __all(!in || (w[i] & KNOWN) != 0)) {
        s = __uint_as_float((uint32_t)w[i]);
        found = d;
      }
    }
    if (found >= 0) {
#pragma unroll 4
      for (int u = found - 1; u >= 0; --u) {
        const uint64_t m = maps[u][ch];
        s = __uint_as_float((uint32_t)m & ~KNOWN_MAP) * s + __uint_as_float((uint32_t)(m >> 32));
      }
      return s;
    }
  }
  // Not a state that could be taken for one: the fault word is in a workspace
  // that the caller may have let go of, a NaN stays to the sequence's end.
  if (ch == 0) atomicOr(a.faults, FAULT_WAIT_TIMEOUT);
  return __builtin_nanf("");
}

struct Tile {
  float A[GS][GC], B[GS][GC];  // the runs' maps; then, in A, what enters every run
  int reset[GS];
};

// Joins the runs of a tile, in the pass's order (REV: from the last run), by
// the wave that holds no data: finds what enters the tile (not where the tile
// begins `fresh`, with a sequence's first row), hands on what leaves it, and
// puts what enters every run into t.A.
// HALVES: keep what enters every half (2) or whole (1) tile for the backward.
template <bool REV, bool MARKED, int HALVES>
__device__ __forceinline__ void join_runs(const GlrArgs& a, Tile& t, Maps& maps, int k, int blk, bool fresh) {
  const int ch = threadIdx.x & 63;
  const int64_t c = (int64_t)blk * GC + ch;
  const bool in = c < a.C;
  const bool ask = k > 0 && !fresh, last = k + 1 == a.ntiles;
  const uint64_t word = ask && in ? peek(a.enter + (int64_t)k * a.C + c) : KNOWN;
  float At = 1.f, Bt = 0.f;
  uint32_t resets = 0;  // runs that hold a sequence's first row (REV: last row)
  if (MARKED) resets = (uint32_t)__ballot(ch < GS && t.reset[ch < GS ? ch : 0]);
  float A[GS], B[GS];
#pragma unroll
  for (int i = 0; i < GS; ++i) {
    A[i] = t.A[i][ch];
    B[i] = t.B[i][ch];
  }
#pragma unroll
  for (int i = 0; i < GS; ++i) {
    const int run = REV ? GS - 1 - i : i;
    Bt = MARKED && (resets >> run & 1) ? B[run] : A[run] * Bt + B[run];
    At *= A[run];
  }
  float s = 0.f, leave = Bt;
  if (!resets && ask && !last && in)  // for the tiles behind, should they have to wait
    post(a.maps + (int64_t)k * a.C + c, (uint64_t)__float_as_uint(Bt) << 32 | __float_as_uint(At) | KNOWN_MAP);
  // what leaves a reset tile does not depend on what enters it: it is handed on first
  if (!resets) {
    if (ask) s = look_back(a, maps, k, c, in, word);
    leave = At * s + Bt;
  }
  if (!last && in) post(a.enter + (int64_t)(k + 1) * a.C + c, KNOWN | __float_as_uint(leave));
  if (resets && ask) s = look_back(a, maps, k, c, in, word);
  // (what enters a fresh tile is not asked for, and what is kept for it not used)
  float* keep = HALVES > 0 && a.keep && in ? a.keep + (int64_t)k * HALVES * a.C + c : nullptr;
#pragma unroll
  for (int i = 0; i < GS; ++i) {
    const int run = REV ? GS - 1 - i : i;
    if (HALVES > 0 && i % (GS / (HALVES > 0 ? HALVES : 1)) == 0 && keep) keep[i / (GS / (HALVES > 0 ? HALVES : 1)) * a.C] = s;
    t.A[run][ch] = s;
    s = MARKED && (resets >> run & 1) ? B[run] : A[run] * s + B[run];
  }
}

constexpr int ASKS = 64;  // the thread that asks for tickets (wave 0 makes the marks)

// Tiles are handed out in order by counters.  One counter serves a tile each
// 13 ns at best (measured), which is near what memory allows, so columns are
// split into equal sets of neighbours where their number is even (two, four or
// eight), each with its counter and its share of the workgroups.  A tile waits
// only for tiles of its own column with lower tickets, which running workgroups
// drew and work on in the order they drew them: the lowest unfinished ticket is
// always being worked on.
constexpr int SETS = 8;
constexpr int TICKET_LINE = 64;  // ints: counters on lines of their own
struct Drawer {
  int* counter;
  int first, n;  // columns of the set
  double per;    // 1 / n
  __device__ __forceinline__ Drawer(const GlrArgs& a) {
    const int set = blockIdx.x % a.sets;
    counter = a.tickets + set * TICKET_LINE;
    n = a.nblk / a.sets;
    first = n * set;
    per = 1.0 / n;
  }
  // A ticket is asked for by ask() and turned into a tile (x: its number in the
  // pass's order, at least ntiles for none; y: its column block) by answer(),
  // later: the round trip lies between.  The address is given in a vector
  // register: at one that is known to be the wave's the compiler adds up over
  // lanes first and so takes the answer at once.  `after` is an answer that has
  // to be there before.
  __device__ __forceinline__ int ask(int after = 0) const {
    int zero = 0;
    asm("" : "+v"(zero) : "v"(after));
    return __hip_atomic_fetch_add(counter + zero, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ int2 answer(int t) const {
    int q = (int)(t * per);  // t / n, off by one at most
    q -= q * n > t;
    q += (q + 1) * n <= t;
    return make_int2(q, first + t - q * n);
  }
};

// The first N tiles and the ticket after them, by one thread.  One at a time, so
// that the workgroups' first tiles come first, then their second ones: asked for
// at once, a workgroup holds neighbours, and the next waits for its last
// (262144 x 1024 680 us instead of 430).
// With one tile a column nothing waits for anything: there is a workgroup for
// every column, and no counter.
template <int N>
__device__ __forceinline__ int draw_first(const GlrArgs& a, const Drawer& d, int2* slot) {
  if (a.ntiles == 1) {
    for (int i = 0; i < N; ++i) slot[i] = make_int2(i, blockIdx.x);
    return INT_MAX / 2;
  }
  int t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = d.ask(i > 0 ? t[i - 1] : 0);
  const int asked = d.ask(t[N - 1]);
#pragma unroll
  for (int i = 0; i < N; ++i) slot[i] = d.answer(t[i]);
  return asked;
}

// Clears the fault word, the counters and the words that other workgroups wait
// for (a kernel rather than a memset, so that a captured graph
// replays it as a kernel node).
__global__ void __launch_bounds__(256) kda_glr_clear_kernel(unsigned* faults, uint4* words, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i == 0) *faults = 0;
  for (int64_t j = i; j < n; j += (int64_t)gridDim.x * 256) words[j] = make_uint4(0, 0, 0, 0);
}

// State (or gradient) of sequence n at 4 channels, zeros where there is none.
__device__ __forceinline__ void state4(const float* p, int n, int64_t C, int64_t c, bool in, float (&s)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = 0.f;
  if (p && in) load_f4(p + (int64_t)n * C + c, s);
}

// One run in one thread: decays and inputs.
template <typename T>
struct Run {
  float a[FR<T>][4], u[FR<T>][4];
};
template <typename T>
struct Raw {
  raw4<T> x[FR<T>], g[FR<T>];
};

// Seven waves hold the data and one finds what enters the tiles, so that rows
// are under way while it waits for other workgroups (loads come back in order:
// a wave that had asked for rows could not see a word before they arrive).
// They run a tile apart, with one barrier a tile: while the one joins tile i,
// the seven write the outputs of tile i - 1, form the maps of tile i + 1 from
// rows that have arrived, and ask for the rows of tile i + 3.  A workgroup
// holds the tickets of those tiles and works on them in order.
template <typename T, bool GIVEN, bool COMPL>
__global__ void __launch_bounds__(GT, 2) kda_glr_fwd_kernel(GlrArgs a) {
  constexpr int R = FR<T>, L = FL<T>;
  // Gates out of LDS (see Gates), where a tile has many rows: 32768 x 12288 of
  // bf16 takes 480 us so and 490 to 515 with loads; fp32, whose tiles have half
  // as many, 540 us and 475 at 32768 x 6144.
  constexpr bool STAGED = sizeof(T) == 2 && !GIVEN;
  __shared__ Tile tiles[2];
  __shared__ Maps maps;
  __shared__ Marks marks[4];
  __shared__ float gates[4][2][GC];
  __shared__ int2 slot[8];  // tiles, by turns
  const int tid = threadIdx.x, lane = tid % GW, run = tid / GW;
  const int64_t rows = axis_rows(a.ax);
  Drawer drawer(a);
  int asked = 0;
  if (tid == ASKS) asked = draw_first<4>(a, drawer, slot);
  __syncthreads();  // tickets
  if (tid >= GD) {
    // everything else waits for this wave: its instructions go first
    __builtin_amdgcn_s_setprio(3);
    const int ch = tid - GD;
    Gates<STAGED> gate;
    for (int i = 0; i < 2; ++i) {
      gate.ask(a, slot[i], ch);
      gate.put(gates[i], ch);
    }
    __syncthreads();  // marks
    __syncthreads();  // the maps of the first tile
    for (int i = 0;; ++i) {
      const int2 item = slot[i & 7];
      if (item.x >= a.ntiles) break;
      const Marks& m = marks[i & 3];
      const int k = item.x, blk = item.y;
      gate.ask(a, slot[(i + 2) & 7], ch);
      if (m.any) join_runs<false, true, FR<T> / BR>(a, tiles[i & 1], maps, k, blk, m.S[0] >= 0);
      else join_runs<false, false, FR<T> / BR>(a, tiles[i & 1], maps, k, blk, false);
      gate.put(gates[(i + 2) & 3], ch);
      __syncthreads();  // what enters tile i, the maps of tile i + 1
    }
  } else {
    const int row_bytes = (int)(a.C * sizeof(T));
    auto place = [&](int2 item, int64_t& t0, int64_t& c) {
      t0 = (int64_t)item.x * L;
      c = (int64_t)item.y * GC + lane * 4;
      return c < a.C ? run * R * row_bytes + (int)(c * sizeof(T)) : OUTSIDE;
    };
    auto fetch = [&](int2 item, Raw<T>& w) {
      if (item.x >= a.ntiles) return;
      int64_t t0, c;
      const int voff = place(item, t0, c);
      const Rows<T, L> xs(a.x, t0, rows, a.C), gs(a.g, t0, rows, a.C);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        w.g[i] = gs.load(voff, i * row_bytes);
        w.x[i] = xs.load(voff, i * row_bytes);
      }
    };
    // the marks of tile i, by the first wave, before anybody needs them
    auto mark = [&](int2 item, int i) {
      if (tid < 64 && item.x < a.ntiles) mark_tile(a.ax, (int64_t)item.x * L, L, rows, marks[i & 3]);
    };
    // the maps of tile i, from rows that were asked for
    auto map_ = [&](auto marked, int2 item, int i, const Raw<T>& w, Run<T>& r) {
      int64_t t0, c;
      place(item, t0, c);
      const bool in = c < a.C;
      Gate<GIVEN> gate;
      if constexpr (STAGED) gate.init(a, gates[i & 3], lane * 4);
      else gate.init(a, in ? c : 0);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        float xv[4], gv[4];
        widen4(w.x[q], xv);
        widen4(w.g[q], gv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float g2 = gate.g2(gv[j], j);
          r.a[q][j] = fexp2(g2);
          r.u[q][j] = COMPL ? one_minus(g2, r.a[q][j]) * xv[j] : xv[j];
        }
      }
      const Marks& m = marks[i & 3];
      Tile& t = tiles[i & 1];
      float A[4], B[4];
      bool reset = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] = 1.f;
        B[j] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (marked() && m.S[run * R + q] >= 0) {
          reset = true;
          state4(a.init, m.S[run * R + q], a.C, c, in, B);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          A[j] *= r.a[q][j];
          B[j] = r.a[q][j] * B[j] + r.u[q][j];
        }
      }
      store4(&t.A[run][lane * 4], A);
      store4(&t.B[run][lane * 4], B);
      if (lane == 0) t.reset[run] = reset;
    };
    auto map = [&](int2 item, int i, const Raw<T>& w, Run<T>& r) {
      if (item.x >= a.ntiles) return;
      if (marks[i & 3].any) map_(std::true_type{}, item, i, w, r);
      else map_(std::false_type{}, item, i, w, r);
    };
    // the outputs of tile i
    auto finish_ = [&](auto marked, int2 item, int i, const Run<T>& r) {
      int64_t t0, c;
      const int voff = place(item, t0, c);
      const bool in = c < a.C;
      const Marks& m = marks[i & 3];
      float h[4];
      load_f4(&tiles[i & 1].A[run][lane * 4], h);
      const Rows<T, L> os(a.out, t0, rows, a.C);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (marked() && m.S[run * R + q] >= 0) state4(a.init, m.S[run * R + q], a.C, c, in, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = r.a[q][j] * h[j] + r.u[q][j];
        os.store(voff, q * row_bytes, h);
        if (marked() && a.fin && in && m.E[run * R + q] >= 0) store4(a.fin + (int64_t)m.E[run * R + q] * a.C + c, h);
      }
      if (a.zero_rest && t0 + L > rows && in) {
        for (int q = 0; q < R; ++q) {
          const int64_t t = t0 + run * R + q;
          if (t >= rows && t < a.ax.total) store_zero4(static_cast<T*>(a.out) + t * a.C + c);
        }
      }
    };
    auto finish = [&](int2 item, int i, const Run<T>& r) {
      if (marks[i & 3].any) finish_(std::true_type{}, item, i, r);
      else finish_(std::false_type{}, item, i, r);
    };
    Run<T> r0, r1;
    Raw<T> w0, w1;
    // tile i: its run `now` is ready; tile i + 1 is made from `w`, which then takes tile i + 3
    auto turn = [&](int i, Run<T>& now, Run<T>& then, Raw<T>& w) {
      const int2 item = slot[i & 7];
      if (item.x >= a.ntiles) return false;
      mark(slot[(i + 2) & 7], i + 2);
      map(slot[(i + 1) & 7], i + 1, w, then);
      if (tid == ASKS) {  // the ticket that was asked for a tile ago
        slot[(i + 4) & 7] = drawer.answer(asked);
        asked = drawer.ask();
      }
      fetch(slot[(i + 3) & 7], w);
      __syncthreads();  // what enters tile i, the maps of tile i + 1
      finish(item, i, now);
      return true;
    };
    mark(slot[0], 0);
    mark(slot[1], 1);
    fetch(slot[0], w0);
    fetch(slot[1], w1);
    __syncthreads();  // marks
    map(slot[0], 0, w0, r0);
    fetch(slot[2], w0);
    __syncthreads();  // the maps of the first tile
    for (int i = 0; turn(i, r0, r1, w1) && turn(i + 1, r1, r0, w0); i += 2) {}
  }
  if (a.fin) {  // empty sequences hand their state on
    for (int64_t n = blockIdx.x; n < a.ax.N; n += gridDim.x) {
      if (axis_start(a.ax, n + 1) > axis_start(a.ax, n)) continue;
      for (int64_t c = tid; c < a.C; c += GT) a.fin[n * a.C + c] = a.init ? a.init[n * a.C + c] : 0.f;
    }
  }
}

// The backward's run keeps its rows as loaded, its decays and (SLOPE) the slopes
// of its gates: they are needed again.
template <typename T, bool SLOPE>
struct Kept {
  float a[BR][4], slope[SLOPE ? BR : 1][4];
  raw4<T> x[BR], g[BR], d[BR];
};

// As the forward, from the right, with a second set of maps for h, whose
// entering states are given: the wave that joins does both.  Rows are asked for
// when a tile is finished, into its registers.
template <typename T, bool GIVEN, bool COMPL>
__global__ void __launch_bounds__(GT, 2) kda_glr_bwd_kernel(GlrArgs a) {
  constexpr int R = BR, L = BL;
  // With b = 1 - a the registers do not hold the slopes too: they are formed again.
  constexpr bool SLOPE = !GIVEN && !COMPL;
  __shared__ Tile et[2], ht[2];  // maps of e, from the right, and of h
  __shared__ float dsums[GIVEN ? 1 : 2][GS][GC], zsums[GIVEN ? 1 : 2][GS][GC];
  __shared__ Maps maps;
  __shared__ Marks marks[4];
  __shared__ float gates[4][2][GC];
  __shared__ int2 slot[8];
  const int tid = threadIdx.x, lane = tid % GW, run = tid / GW;
  const int64_t rows = axis_rows(a.ax);
  Drawer drawer(a);
  int asked = 0;
  if (tid == ASKS) asked = draw_first<3>(a, drawer, slot);
  __syncthreads();  // tickets
  if (tid >= GD) {
    __builtin_amdgcn_s_setprio(3);
    const int ch = tid - GD;
    auto state_of = [&](int2 item) {  // h entering the tile
      const int64_t c = (int64_t)item.y * GC + ch;
      return item.x < a.ntiles && c < a.C ? a.states[(int64_t)(a.ntiles - 1 - item.x) * a.C + c] : 0.f;
    };
    // d_raw and dz z over the tile, from the runs' sums of tile i, a tile behind
    auto add_up = [&](int2 item, int i) {
      const int64_t c = (int64_t)item.y * GC + ch;
      if (c >= a.C) return;
      float d = 0.f, z = 0.f;
#pragma unroll
      for (int q = 0; q < GS; ++q) {
        d += dsums[i & (GIVEN ? 0 : 1)][q][ch];
        z += zsums[i & (GIVEN ? 0 : 1)][q][ch];
      }
      a.part[(int64_t)(a.ntiles - 1 - item.x) * a.C + c] = make_float2(d, z);
    };
    float s = state_of(slot[0]);
    Gates<!GIVEN> gate;
    for (int i = 0; i < 2; ++i) {
      gate.ask(a, slot[i], ch);
      gate.put(gates[i], ch);
    }
    int last = -1;
    __syncthreads();  // marks
    __syncthreads();  // the maps of the first tile
    for (int i = 0;; ++i) {
      const int2 item = slot[i & 7];
      if (item.x >= a.ntiles) break;
      const Marks& m = marks[i & 3];
      const int k = item.x, blk = item.y;
      gate.ask(a, slot[(i + 2) & 7], ch);
      if (m.any) join_runs<true, true, 0>(a, et[i & 1], maps, k, blk, m.E[L - 1] >= 0);
      else join_runs<true, false, 0>(a, et[i & 1], maps, k, blk, false);
      Tile& t = ht[i & 1];
      const uint32_t resets = m.any ? (uint32_t)__ballot(ch < GS && t.reset[ch < GS ? ch : 0]) : 0;
#pragma unroll
      for (int q0 = 0; q0 < GS; q0 += 14) {
        float A[14], B[14];
#pragma unroll
        for (int q = 0; q < 14; ++q) {
          A[q] = t.A[q0 + q][ch];
          B[q] = t.B[q0 + q][ch];
        }
#pragma unroll
        for (int q = 0; q < 14; ++q) {
          t.A[q0 + q][ch] = s;
          s = (resets >> (q0 + q) & 1) ? B[q] : A[q] * s + B[q];
        }
      }
      s = state_of(slot[(i + 1) & 7]);
      gate.put(gates[(i + 2) & 3], ch);
      __syncthreads();  // what enters tile i, the maps of tile i + 1
      if (!GIVEN && i > 0) add_up(slot[(i - 1) & 7], i - 1);
      last = i;
    }
    __syncthreads();  // the sums of the last tile
    if (!GIVEN && last >= 0) add_up(slot[last & 7], last);
  } else {
    const int row_bytes = (int)(a.C * sizeof(T));
    auto place = [&](int2 item, int64_t& t0, int64_t& c) {
      t0 = (int64_t)(a.ntiles - 1 - item.x) * L;
      c = (int64_t)item.y * GC + lane * 4;
      return c < a.C ? run * R * row_bytes + (int)(c * sizeof(T)) : OUTSIDE;
    };
    auto fetch = [&](int2 item, Kept<T, SLOPE>& r) {
      if (item.x >= a.ntiles) return;
      int64_t t0, c;
      const int voff = place(item, t0, c);
      const Rows<T, L> xs(a.x, t0, rows, a.C), gs(a.g, t0, rows, a.C), ds(a.d_out, t0, rows, a.C);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        r.g[i] = gs.load(voff, i * row_bytes);
        r.d[i] = ds.load(voff, i * row_bytes);
        r.x[i] = xs.load(voff, i * row_bytes);
      }
    };
    auto mark = [&](int2 item, int i) {
      if (tid < 64 && item.x < a.ntiles)
        mark_tile(a.ax, (int64_t)(a.ntiles - 1 - item.x) * L, L, rows, marks[i & 3]);
    };
    auto map_ = [&](auto marked, int2 item, int i, Kept<T, SLOPE>& r) {
      int64_t t0, c;
      place(item, t0, c);
      const bool in = c < a.C;
      const int64_t tr = t0 + run * R;
      Gate<GIVEN> gate;
      gate.init(a, gates[i & 3], lane * 4);
      const Marks& m = marks[i & 3];
      {  // of h
        Tile& t = ht[i & 1];
        float A[4], B[4];
        bool reset = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          A[j] = 1.f;
          B[j] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
          if (marked() && m.S[run * R + q] >= 0) {
            reset = true;
            state4(a.init, m.S[run * R + q], a.C, c, in, B);
          }
          float xv[4], gv[4];
          widen4(r.x[q], xv);
          widen4(r.g[q], gv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float g2;
            if constexpr (SLOPE) g2 = gate.g2(gv[j], j, r.slope[q][j]);
            else g2 = gate.g2(gv[j], j);
            r.a[q][j] = fexp2(g2);
            A[j] *= r.a[q][j];
            B[j] = r.a[q][j] * B[j] + (COMPL ? one_minus(g2, r.a[q][j]) * xv[j] : xv[j]);
          }
        }
        store4(&t.A[run][lane * 4], A);
        store4(&t.B[run][lane * 4], B);
        if (lane == 0) t.reset[run] = reset;
      }
      {  // of e; rows behind the last sequence hand nothing on
        Tile& t = et[i & 1];
        float P[4], Q[4];
        bool reset = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          P[j] = 1.f;
          Q[j] = 0.f;
        }
#pragma unroll
        for (int q = R - 1; q >= 0; --q) {
          if (!marked() || tr + q < rows) {
            if (marked() && m.E[run * R + q] >= 0) {
              reset = true;
              state4(a.d_final, m.E[run * R + q], a.C, c, in, Q);
            }
            float dv[4];
            widen4(r.d[q], dv);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              P[j] *= r.a[q][j];
              Q[j] = r.a[q][j] * (dv[j] + Q[j]);
            }
          }
        }
        store4(&t.A[run][lane * 4], P);
        store4(&t.B[run][lane * 4], Q);
        if (lane == 0) t.reset[run] = reset;
      }
    };
    auto map = [&](int2 item, int i, Kept<T, SLOPE>& r) {
      if (item.x >= a.ntiles) return;
      if (marks[i & 3].any) map_(std::true_type{}, item, i, r);
      else map_(std::false_type{}, item, i, r);
    };
    auto finish_ = [&](auto marked, int2 item, int i, const Kept<T, SLOPE>& r) {
      int64_t t0, c;
      const int voff = place(item, t0, c);
      const bool in = c < a.C;
      const int64_t tr = t0 + run * R;
      Gate<GIVEN> gate;
      gate.init(a, gates[i & 3], lane * 4);
      const Marks& m = marks[i & 3];
      const float to_raw = GIVEN ? 1.f : a.lb * (gate.na * -0.6931471805599453f);
      float h[4], e[4], hp[R][4], dsum[4], zsum[4];
      load_f4(&ht[i & 1].A[run][lane * 4], h);
      load_f4(&et[i & 1].A[run][lane * 4], e);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (marked() && m.S[run * R + q] >= 0) state4(a.init, m.S[run * R + q], a.C, c, in, h);
        float xv[4], gv[4];
        widen4(r.x[q], xv);
        widen4(r.g[q], gv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hp[q][j] = COMPL ? h[j] - xv[j] : h[j];
          h[j] = r.a[q][j] * h[j] + (COMPL ? one_minus(gate.g2(gv[j], j), r.a[q][j]) * xv[j] : xv[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) dsum[j] = zsum[j] = 0.f;
      const Rows<T, L> dxs(a.out, t0, rows, a.C), dgs(a.dg, t0, rows, a.C);
#pragma unroll
      for (int q = R - 1; q >= 0; --q) {
        if (!marked() || tr + q < rows) {
          if (marked() && m.E[run * R + q] >= 0) state4(a.d_final, m.E[run * R + q], a.C, c, in, e);
          float dv[4], gv[4], dx[4], dg[4];
          widen4(r.d[q], dv);
          widen4(r.g[q], gv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float dh = dv[j] + e[j];
            e[j] = r.a[q][j] * dh;
            dx[j] = COMPL ? one_minus(gate.g2(gv[j], j), r.a[q][j]) * dh : dh;
            dg[j] = e[j] * hp[q][j];
            if constexpr (!GIVEN) {
              // dg/dz = lb slope, dz/draw = exp(A_log)
              const float mz = gv[j] * gate.na + gate.nb[j];  // -z log2(e)
              float slope;
              if constexpr (SLOPE) slope = r.slope[q][j];
              else slope = gate.slope(mz);
              const float dz = dg[j] * slope;  // (the constants come behind)
              zsum[j] += dz * mz;
              dg[j] = dz * to_raw;
              dsum[j] += dg[j];
            }
          }
          dxs.store(voff, q * row_bytes, dx);
          dgs.store(voff, q * row_bytes, dg);
          if (marked() && a.d_init && in && m.S[run * R + q] >= 0)
            store4(a.d_init + (int64_t)m.S[run * R + q] * a.C + c, e);
        } else if (in && a.zero_rest && tr + q < a.ax.total) {
          store_zero4(static_cast<T*>(a.out) + (tr + q) * a.C + c);
          store_zero4(static_cast<T*>(a.dg) + (tr + q) * a.C + c);
        }
      }
      if constexpr (!GIVEN) {
#pragma unroll
        for (int j = 0; j < 4; ++j) zsum[j] *= a.lb * -0.6931471805599453f;
        store4(&dsums[i & 1][run][lane * 4], dsum);
        store4(&zsums[i & 1][run][lane * 4], zsum);
      }
    };
    auto finish = [&](int2 item, int i, const Kept<T, SLOPE>& r) {
      if (marks[i & 3].any) finish_(std::true_type{}, item, i, r);
      else finish_(std::false_type{}, item, i, r);
    };
    // tile i is ready in `now`; tile i + 1 is made in `then`; `now` takes tile i + AHEAD
    constexpr int AHEAD = sizeof(T) == 2 ? 3 : 2;
    auto turn = [&](int i, Kept<T, SLOPE>& now, Kept<T, SLOPE>& then) {
      const int2 item = slot[i & 7];
      if (item.x >= a.ntiles) return false;
      mark(slot[(i + 2) & 7], i + 2);
      map(slot[(i + 1) & 7], i + 1, then);
      if (tid == ASKS) {
        slot[(i + 3) & 7] = drawer.answer(asked);
        asked = drawer.ask();
      }
      __syncthreads();  // what enters tile i, the maps of tile i + 1
      finish(item, i, now);
      fetch(slot[(i + AHEAD) & 7], now);
      return true;
    };
    Kept<T, SLOPE> r0, r1;
    mark(slot[0], 0);
    mark(slot[1], 1);
    fetch(slot[0], r0);
    fetch(slot[1], r1);
    if constexpr (AHEAD == 3) {
      Kept<T, SLOPE> r2;
      fetch(slot[2], r2);
      __syncthreads();  // marks
      map(slot[0], 0, r0);
      __syncthreads();  // the maps of the first tile
      for (int i = 0; turn(i, r0, r1) && turn(i + 1, r1, r2) && turn(i + 2, r2, r0); i += 3) {}
    } else {
      __syncthreads();  // marks
      map(slot[0], 0, r0);
      __syncthreads();  // the maps of the first tile
      for (int i = 0; turn(i, r0, r1) && turn(i + 1, r1, r0); i += 2) {}
    }
    __syncthreads();  // the sums of the last tile
  }
  if (a.d_init) {
    for (int64_t n = blockIdx.x; n < a.ax.N; n += gridDim.x) {
      if (axis_start(a.ax, n + 1) > axis_start(a.ax, n)) continue;
      for (int64_t c = tid; c < a.C; c += GT) a.d_init[n * a.C + c] = a.d_final ? a.d_final[n * a.C + c] : 0.f;
    }
  }
}

// Sums of the tiles' partial sums, in a fixed order and in fp64 (a long
// sequence has thousands of them): d_dt_bias per channel, and per channel what
// dA_log adds up per head.  A workgroup has 16 channels, a line of each row, by
// 64 rows at a time: few channels still make enough workgroups to be done in a
// few round trips (64 channels by 16 rows took 37 us at 618 tiles of 4096
// channels).
constexpr int GRED = 1024, RC = 16, RR = GRED / RC;
__global__ void __launch_bounds__(GRED) kda_glr_reduce_kernel(GlrArgs a) {
  __shared__ double sd[RR][RC], sz[RR][RC];
  const int ch = threadIdx.x % RC, row = threadIdx.x / RC;
  const int64_t c = (int64_t)blockIdx.x * RC + ch;
  double d = 0.0, z = 0.0;
  if (c < a.C) {
    constexpr int U = 4;  // rows asked for at once
    for (int t0 = row; t0 < a.ntiles; t0 += U * RR) {
      float2 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = t0 + u * RR < a.ntiles ? a.part[(int64_t)(t0 + u * RR) * a.C + c] : make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        d += p[u].x;
        z += p[u].y;
      }
    }
  }
  sd[row][ch] = d;
  sz[row][ch] = z;
  for (int r = RR / 2; r >= 1; r >>= 1) {
    __syncthreads();
    if (row < r) {
      sd[row][ch] += sd[row + r][ch];
      sz[row][ch] += sz[row + r][ch];
    }
  }
  if (row == 0 && c < a.C) {
    a.d_dt_bias[c] = (float)sd[0][ch];
    a.zsum[c] = sz[0][ch];
  }
}
__global__ void __launch_bounds__(64) kda_glr_head_kernel(GlrArgs a) {
  double z = 0.0;
  for (int k = threadIdx.x; k < a.K; k += 64) z += a.zsum[(int64_t)blockIdx.x * a.K + k];
  for (int m = 32; m >= 1; m >>= 1) z += __shfl_xor(z, m);
  if (threadIdx.x == 0) a.dA_log[blockIdx.x] = (float)z;
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

// The fault word comes where kda_workspace_faults looks for it, then what is
// cleared: the counters and the words that tiles hand each other.
struct GlrLayout {
  size_t faults, tickets, enter, maps, part, zsum, total;
};
GlrLayout glr_layout(int64_t T_total, int64_t C, bool bwd) {
  const size_t tiles = (size_t)((T_total + BL - 1) / BL);  // of the shorter kind
  const size_t w = tiles * (size_t)C;
  GlrLayout l;
  l.faults = 4;
  l.tickets = 256;
  l.enter = l.tickets + SETS * TICKET_LINE * sizeof(int);
  l.maps = l.enter + align256(w * sizeof(uint64_t));
  l.part = l.maps + align256(w * sizeof(uint64_t));
  l.zsum = l.part + (bwd ? align256(w * sizeof(float2)) : 0);
  l.total = l.zsum + (bwd ? align256((size_t)C * sizeof(double)) : 0);
  return l;
}

bool glr_sizes_ok(int64_t T_total, int64_t H, int64_t K) {
  return T_total >= 0 && H >= 1 && K >= 1 && fits(H, K, kMaxChannels) && fits(T_total, H * K, kMaxElements);
}

// Checks shared by the entry points; fills the sizes and the gate.
kda_status_t glr_prepare(GlrArgs& a, const float* A_log, const float* dt_bias, float lower_bound,
                         const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t H, int64_t K, int64_t N,
                         int dtype, unsigned flags, bool bwd, bool step = false) {
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
  const int64_t L = bwd || dtype == KDA_DTYPE_FP32 ? BL : L_MAX, tiles = (B * T + L - 1) / L, nblk = (H * K + GC - 1) / GC;
  if (!fits(tiles, nblk, (int64_t)1 << 30)) return KDA_ERR_INVALID;  // tile numbers are 32-bit
  a = GlrArgs{};
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.ax = make_axis(cu_seqlens, T, B * T, N);
  a.C = H * K;
  a.H = (int)H;
  a.K = (int)K;
  a.nblk = (int)nblk;
  a.ntiles = (int)tiles;
  a.sets = nblk % 8 == 0 ? 8 : nblk % 4 == 0 ? 4 : nblk % 2 == 0 ? 2 : 1;
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

// Workgroups of a pass: as many as run at once, one on a CU.
int64_t pass_grid(const GlrArgs& a) {
  const int64_t items = (int64_t)a.ntiles * a.nblk, most = a.ntiles == 1 ? a.nblk : 256;  // (draw_first)
  return items < 1 ? 1 : items < most ? items : most;
}
kda_status_t clear(const GlrArgs& a, hipStream_t st) {
  const int64_t n = (reinterpret_cast<char*>(a.maps + (int64_t)a.ntiles * a.C) - reinterpret_cast<char*>(a.tickets)) / sizeof(uint4);
  const int64_t blocks = (n + 255) / 256, most = 2048;
  return launch(&kda_glr_clear_kernel, blocks < 1 ? 1 : blocks < most ? blocks : most, 256, st, "glr clear",
                a.faults, reinterpret_cast<uint4*>(a.tickets), n);
}
template <typename T, bool GIVEN, bool COMPL>
struct RunFwd {
  static kda_status_t run(const GlrArgs& a, hipStream_t st) {
    const kda_status_t s = clear(a, st);
    return s != KDA_SUCCESS ? s : launch(&kda_glr_fwd_kernel<T, GIVEN, COMPL>, pass_grid(a), GT, st, "glr forward", a);
  }
};
template <typename T, bool GIVEN, bool COMPL>
struct RunBwd {
  static kda_status_t run(const GlrArgs& a, hipStream_t st) {
    kda_status_t s = clear(a, st);
    if (s == KDA_SUCCESS) s = launch(&kda_glr_bwd_kernel<T, GIVEN, COMPL>, pass_grid(a), GT, st, "glr backward", a);
    if (s != KDA_SUCCESS || GIVEN) return s;
    s = launch(&kda_glr_reduce_kernel, (a.C + RC - 1) / RC, GRED, st, "glr reduce", a);
    return s != KDA_SUCCESS ? s : launch(&kda_glr_head_kernel, a.H, 64, st, "glr heads", a);
  }
};
template <typename T, bool GIVEN, bool COMPL>
struct RunStep {
  static kda_status_t run(const GlrArgs& a, int64_t grid, hipStream_t st) {
    return launch(&kda_glr_step_kernel<T, GIVEN, COMPL>, grid, GST, st, "glr step", a);
  }
};

void carve(GlrArgs& a, char* ws, const GlrLayout& l) {
  a.tickets = reinterpret_cast<int*>(ws + l.tickets);
  a.faults = reinterpret_cast<unsigned*>(ws + l.faults);
  a.enter = reinterpret_cast<uint64_t*>(ws + l.enter);
  a.maps = reinterpret_cast<uint64_t*>(ws + l.maps);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_glr_states_size(int64_t T_total, int64_t H, int64_t K) {
  if (!glr_sizes_ok(T_total, H, K)) return 0;
  return align256((size_t)((T_total + L_MAX - 1) / L_MAX * 2) * (size_t)(H * K) * sizeof(float)) + 256;
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
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, cu_seqlens, B, T, H, K, N, dtype, flags, false);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !raw_gate || !out)) return KDA_ERR_INVALID;
  if (!aligned_all(4 * dtype_bytes(dtype), {x, raw_gate, out}) ||
      !aligned_all(16, {initial_state, final_state, states, workspace}))
    return KDA_ERR_INVALID;
  const GlrLayout l = glr_layout(a.ax.total, a.C, false);
  if (!workspace || workspace_bytes < l.total) return KDA_ERR_WORKSPACE;
  // (a sequence's last tile may be written before its first reads the state again)
  if (same(final_state, initial_state)) return KDA_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  a.x = x;
  a.g = raw_gate;
  a.out = out;
  a.init = initial_state;
  a.fin = final_state;
  carve(a, ws, l);
  a.keep = states;
  return by_variant<RunFwd>(dtype, flags, a, reinterpret_cast<hipStream_t>(stream));
}

kda_status_t kda_glr_bwd(const void* x, const void* raw_gate, const float* states, const void* d_out,
                         const float* d_final, void* dx, void* d_raw_gate, float* dA_log, float* d_dt_bias,
                         float* d_initial_state, void* workspace, size_t workspace_bytes, const float* A_log,
                         const float* dt_bias, float lower_bound, const float* initial_state,
                         const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t H, int64_t K, int64_t N,
                         int dtype, unsigned flags, void* stream) {
  GlrArgs a;
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, cu_seqlens, B, T, H, K, N, dtype, flags, true);
  if (s != KDA_SUCCESS) return s;
  if (a.ax.total > 0 && (!x || !raw_gate || !states || !d_out || !dx || !d_raw_gate)) return KDA_ERR_INVALID;
  if (!(flags & FLAG_GATE_GIVEN) && (!dA_log || !d_dt_bias)) return KDA_ERR_INVALID;
  if (!aligned_all(4 * dtype_bytes(dtype), {x, raw_gate, d_out, dx, d_raw_gate}) ||
      !aligned_all(16, {states, d_final, d_initial_state, initial_state, workspace}))
    return KDA_ERR_INVALID;
  const GlrLayout l = glr_layout(a.ax.total, a.C, true);
  if (!workspace || workspace_bytes < l.total) return KDA_ERR_WORKSPACE;
  if (same(d_initial_state, d_final) || same(d_initial_state, initial_state)) return KDA_ERR_INVALID;
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
  carve(a, ws, l);
  a.states = states;
  a.part = reinterpret_cast<float2*>(ws + l.part);
  a.zsum = reinterpret_cast<double*>(ws + l.zsum);
  return by_variant<RunBwd>(dtype, flags, a, reinterpret_cast<hipStream_t>(stream));
}

kda_status_t kda_glr_step(const void* x, const void* raw_gate, void* out, const float* A_log, const float* dt_bias,
                          float lower_bound, const float* initial_state, float* final_state, int64_t B, int64_t T,
                          int64_t H, int64_t K, int dtype, unsigned flags, void* stream) {
  GlrArgs a;
  const kda_status_t s = glr_prepare(a, A_log, dt_bias, lower_bound, nullptr, B, T, H, K, B, dtype, flags, false, true);
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
