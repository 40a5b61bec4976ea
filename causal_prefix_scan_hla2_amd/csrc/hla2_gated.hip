// hla2_gated.hip -- the gated linear recurrence s_t = a_t s_{t-1} + b_t: forward over a sequence,
// backward, and the single-token step.
#include "hla2.h"
#include "hla2_internal.h"
#include "hla2_mfma.h"

#include <initializer_list>
#include <type_traits>

namespace hla2 {
namespace {

static_assert(GATED_TILE == HLA2_GATED_SCAN_TILE, "marks are a tile apart");

// A gate in one register, "held": the factor a, 0 <= a <= 1, as -a where it is small and as z = 1 - a, which
// is formed by itself and not by subtraction, where it is not.  A gate that holds its state for 1/z tokens
// is off by z's relative error then, whatever z; 1 - a from a rounded a is off by 2^-25 / z, and every token
// adds that (states after 9000 tokens of a constant sigmoid gate near logit 12: 4e-3 off, near 18: 0.7).  The
// factor not held is 1 minus the one that is, good to half a step.  The sign is the whole sign bit: -0 is
// a = 0, +0 is z = 0.
__device__ __forceinline__ bool held_a_itself(float h) { return __builtin_bit_cast(int, h) < 0; }
__device__ __forceinline__ float held_z(float h) { return held_a_itself(h) ? 1.f + h : h; }
// a s + y
__device__ __forceinline__ float scale_add(float h, float s, float y) {
  return fmaf(-h, s, y) + (held_a_itself(h) ? 0.f : s);
}
// a u
__device__ __forceinline__ float scale(float h, float u) { return fmaf(-h, u, held_a_itself(h) ? 0.f : u); }

// The gate of one token and channel.  fp32 takes the library's exp and an IEEE division.  bf16 takes the
// hardware's exp2 and reciprocal, each good to one fp32 step of its result (and the argument's rounding, |g| half
// steps): with the exact forms the walk was bound by the vector units (forward over 65536 tokens x 2048
// channels, sigmoid: 215 us against 181 us when it was measured).
constexpr float LOG2E = 1.44269504088896340736f;
// exp(m), m <= 0.  Near 0 (a > 0.94) by the series of 1 - exp(m), whose first term left out is 2^-22.9 of it at
// m = -1/16; farther, 1 minus a rounded a is good to 2^-20.
template <bool FAST> __device__ __forceinline__ float hold_exp(float m) {
  const float a = FAST ? __builtin_amdgcn_exp2f(m * LOG2E) : expf(m);
  const float z = m * fmaf(m, fmaf(m, fmaf(m, 1.f / 24, 1.f / 6), 0.5f), 1.f);
  return m > -0.0625f ? fabsf(z) : -a;  // of a NaN, a
}
// What the gate is formed from: log gates above 0 count as 0 (a NaN stays).
template <int GATE> __device__ __forceinline__ float gate_arg(float g) {
  return GATE == HLA2_GATE_LOG && g > 0.f ? 0.f : g;
}
template <typename T, int GATE> __device__ __forceinline__ float hold(float arg) {
  constexpr bool FAST = sizeof(T) == 2;
  if constexpr (GATE == HLA2_GATE_LOG) {
    return hold_exp<FAST>(arg);
  } else {
    const float e = FAST ? __builtin_amdgcn_exp2f(-fabsf(arg) * LOG2E) : expf(-fabsf(arg));
    const float r = FAST ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e);
    return copysignf(e * r, arg);  // the smaller of a and z
  }
}
constexpr float HELD_ONE = 0.f;  // a = 1
// s_t from s_{t-1}: the sigmoid gate moves s towards x by a part z of the way, from the nearer end
template <int GATE> __device__ __forceinline__ float advance(float h, float x, float s) {
  return GATE == HLA2_GATE_LOG ? scale_add(h, s, x) : fmaf(-h, s - x, held_a_itself(h) ? x : s);
}

// The factor of a run of tokens, both ways: A, and Z = 1 - A as the sum of z times the A before it.
struct Decay {
  float A = 1.f, Z = 0.f;
  __device__ __forceinline__ void then(float h) {
    Z = fmaf(-h, Z, (held_a_itself(h) ? 1.f : Z) + h);
    A = scale(h, A);
  }
  __device__ __forceinline__ float held() const { return A >= 0.5f ? Z : -A; }
};
// A thread's run of tokens: log gates add up.
template <int GATE> struct Run {
  Decay all;
  __device__ __forceinline__ void then(float, float h) { all.then(h); }
  __device__ __forceinline__ float held() const { return all.held(); }
};
template <> struct Run<HLA2_GATE_LOG> {
  float sum = 0.f;
  __device__ __forceinline__ void then(float arg, float) { sum += arg; }
  __device__ __forceinline__ float held() const { return hold_exp<false>(sum); }
};

__device__ __forceinline__ int seq_len(const int *lens, int b, int n) {
  const int m = lens ? lens[b] : n;
  return m < 0 ? 0 : (m > n ? n : m);
}

// ---------------------------------------------------------------------------
// Tiles.  A workgroup takes GATED_TILE tokens of CS channels of one sequence: thread (tt, cg) holds R
// consecutive tokens of V channels in registers, so x and g are read from memory once.  V channels
// are 16 bytes; the scalar form (V = 1) serves rows that are not whole 16-byte vectors.
template <typename T, bool VEC> struct Shape {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  static constexpr int CG = VEC ? 8 : 32, TT = 256 / CG, R = GATED_TILE / TT, CS = CG * V;
  static constexpr int Q = 256 / CS, PQ = TT / Q;  // quarters of the thread rows, thread rows in each
};

template <int V, typename T> struct Pack { T e[V]; };

// V consecutive values at byte offset `off` of a buffer (past its end: zeros / dropped)
template <typename T, int V> __device__ __forceinline__ Pack<V, T> ld_pack(__amdgpu_buffer_rsrc_t r, int off) {
  if constexpr (V * sizeof(T) == 16)
    return __builtin_bit_cast(Pack<V, T>, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  else if constexpr (sizeof(T) == 4)
    return __builtin_bit_cast(Pack<V, T>, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
  else
    return __builtin_bit_cast(Pack<V, T>, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
}
template <typename T, int V> __device__ __forceinline__ void st_pack(__amdgpu_buffer_rsrc_t r, int off, Pack<V, T> x) {
  if constexpr (V * sizeof(T) == 16)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, off, 0, 0);
  else if constexpr (sizeof(T) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), r, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, x), r, off, 0, 0);
}

// Values the compiler takes for new.  What was formed from them before (gates, values widened to
// fp32) is formed again instead of being kept across the wait for the carry: registers for a second
// workgroup on the compute unit are worth more than the arithmetic.
template <int R, int V, typename T> __device__ __forceinline__ void fresh(Pack<V, T> (&x)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (V * sizeof(T) == 16) {
      u32x4 w = __builtin_bit_cast(u32x4, x[r]);
      asm volatile("" : "+v"(w));
      x[r] = __builtin_bit_cast(Pack<V, T>, w);
    } else if constexpr (sizeof(T) == 4) {
      asm volatile("" : "+v"(x[r].e[0]));
    } else {
      unsigned w = __builtin_bit_cast(unsigned short, x[r]);
      asm volatile("" : "+v"(w));
      x[r] = __builtin_bit_cast(Pack<V, T>, (unsigned short)w);
    }
  }
}

template <int R, int V> __device__ __forceinline__ void fresh(float (&x)[R][V]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < V; ++e) asm volatile("" : "+v"(x[r][e]));
}

// ---------------------------------------------------------------------------
// Carries between the tiles of one sequence.  A tile is the map s -> A s + H of the state it starts
// from, A held like a gate.  Its workgroup publishes (A, H), then looks back for the newest tile whose
// outgoing state is known and folds the maps in between onto it, oldest first: the same multiply-adds in
// the same order as the tiles in between make themselves, so the result does not depend on what was found.
// What is published is one 64-bit word, written and read whole, so no ordering between words is needed:
// a state beside a mark that it is there, or a map as H beside A's inverted bits, which are not zero.
// The words are cleared by a launch before.
// Tiles are dealt by counters, in sequence order, so every tile waited for belongs to a workgroup
// that already runs, and whose tile does not wait for a later one.  Only a workspace that another call
// uses at the same time can leave a wait without an answer: it ends all the same, with a state of NaN,
// which goes on to the tiles after.
typedef unsigned long long Word;
constexpr int LOOK = 8;            // words read at once
constexpr int PATIENCE = 1 << 20;  // reads of a wait that find nothing, a microsecond or more each

__device__ __forceinline__ void publish(Word *w, unsigned low, float high) {
  __hip_atomic_store(w, (Word)__builtin_bit_cast(unsigned, high) << 32 | low, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(Word *w, float s) { publish(w, 1u, s); }
__device__ __forceinline__ void publish_map(Word *w, float A, float H) {
  if (A != A) A = NAN;  // the one NaN whose inverted bits are not zero
  publish(w, ~__builtin_bit_cast(unsigned, A), H);
}
__device__ __forceinline__ Word peek(const Word *w) {
  return __hip_atomic_load(const_cast<Word *>(w), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool there(Word w) { return (unsigned)w != 0; }
__device__ __forceinline__ float value(Word w) { return __builtin_bit_cast(float, (unsigned)(w >> 32)); }  // the state, H
__device__ __forceinline__ float map_a(Word w) { return __builtin_bit_cast(float, ~(unsigned)w); }

// `own`: this lane's words of the tile, its map and its outgoing state, CS apart; the tile before lies `step`
// words below.  k >= 1 tiles come before.  Called by the CS first lanes of a wave together.
template <int CS> __device__ float look_back(const Word *own, long step, int k) {
  int back = 1, found = 0, left = PATIENCE;
  float s = 0.f;
  while (!found) {
    Word w[LOOK];
#pragma unroll
    for (int m = 0; m < LOOK; ++m) w[m] = back + m <= k ? peek(own - (back + m) * step + CS) : 0;
#pragma unroll
    for (int m = LOOK - 1; m >= 0; --m)
      if (__all(there(w[m]))) {
        found = back + m;
        s = value(w[m]);
      }
    back += LOOK;
    if (!found && (back > k || back > 4 * LOOK)) {
      if (--left == 0) return NAN;
      back = 1;
      __builtin_amdgcn_s_sleep(1);
    }
  }
  for (int i = found - 1; i >= 1; i -= LOOK) {
    Word map[LOOK];
    bool all;
    do {
      if (left-- == 0) return NAN;
      all = true;
#pragma unroll
      for (int m = 0; m < LOOK; ++m)
        if (i - m >= 1) map[m] = peek(own - (i - m) * step);
#pragma unroll
      for (int m = 0; m < LOOK; ++m)
        if (i - m >= 1) all = all && there(map[m]);
    } while (!__all(all));
#pragma unroll
    for (int m = 0; m < LOOK; ++m)
      if (i - m >= 1) s = scale_add(map_a(map[m]), s, value(map[m]));
  }
  return s;
}

// The workgroup's tile in dealing order: `turn` counts a sequence's tiles in the order of the scan.
// Workgroups reach the eight XCDs in turn.  Each XCD has a run of neighbouring slabs and a counter that
// deals their tiles, so that the memory lines two slabs share, and the words of a sequence, are in one
// L2 (3 x 1999 tokens x 1001 channels, fp32, forward: 23 -> 17 us; 8 x 16 heads x 2048 x 128, fp32,
// backward: 155 -> 131 us).  A workgroup that finds its own counter spent goes on to the next; there are
// as many workgroups as tiles, so each gets one.  Few slabs of many tiles have one counter (32 slabs of
// 256 tiles, bf16: 192 us against 202 us; at 48 of 128 and below the counters are even or ahead).
struct Deal {
  int turn, slab;
};
constexpr int XCDS = 8, COUNTERS = 16;  // 64-bit words from one counter to the next: a line of memory
static_assert(XCDS * COUNTERS <= GATED_WORD0, "the counters lie before the tiles' words");
__device__ __forceinline__ Deal deal(const GatedArgs &p, int slabs, int tiles) {
  const int parts = tiles >= 4 * (long)slabs ? 1 : XCDS, q = slabs / parts, rest = slabs % parts, home = blockIdx.x % parts;
  if (!p.words) return Deal{0, home * q + min(home, rest) + (int)blockIdx.x / parts};
  __shared__ int s_turn, s_slab;
  if (threadIdx.x == 0) {
    Deal got{tiles, 0};  // no tile: only when another call uses the workspace at the same time
    for (int j = 0; j < parts; ++j) {
      const int x = (home + j) % parts, count = q + (x < rest);
      if (count == 0) continue;
      const unsigned ticket = atomicAdd((unsigned *)p.words + 2 * COUNTERS * x, 1u);
      if (ticket / (unsigned)count >= (unsigned)tiles) continue;
      got = Deal{(int)(ticket / (unsigned)count), x * q + min(x, rest) + (int)(ticket % (unsigned)count)};
      break;
    }
    s_turn = got.turn;
    s_slab = got.slab;
  }
  __syncthreads();
  return Deal{s_turn, s_slab};
}
// this lane's words of a sequence's `turn`-th tile
template <int CS> __device__ __forceinline__ Word *words_of(const GatedArgs &p, int slab, int turn, int tiles, int lane) {
  return (Word *)p.words + GATED_WORD0 + ((long)slab * tiles + turn) * 2 * CS + lane;
}

// Forward.  A thread forms the map of its R tokens, (A, H) with s -> A s + H, A held; the thread rows' maps are
// folded in LDS in quarters by all threads, the quarters by the first CS, which also carry the state in
// from the tile before; then every thread walks its tokens again from the state it starts with.
// Bound by HBM and, in bf16, as nearly by the vector units: x and g read once, out written once.  8 x 16 heads x
// 8192 tokens, d = 128, bf16, log gate: 163 us, 4.9 TB/s, where a large copy reaches 5.1 (two passes over x and
// g would move 5/3 of that) and vector instructions issue in every cycle; 65536 tokens x 2048 channels,
// sigmoid: 178 us, in 86% of them.  256 tokens to a tile: a thread's 8 rows of 16 bytes keep 64 KB of
// loads in flight to a workgroup, and a tile's words are 1% of its data.  Three workgroups to a compute
// unit or, where 128 registers are enough, four.
template <typename T, int GATE, bool VEC>
__global__ void __launch_bounds__(256, 3) gated_forward_kernel(GatedArgs p) {
  using S = Shape<T, VEC>;
  constexpr bool HOLD = sizeof(T) == 4 || !VEC;  // the gate takes g's registers; bf16 vectors would need twice as many
  constexpr int V = S::V, CG = S::CG, TT = S::TT, R = S::R, CS = S::CS, Q = S::Q, PQ = S::PQ;
  __shared__ float sA[TT][CS], sH[TT][CS], qA[Q][CS], qH[Q][CS], qC[Q][CS];
  const int groups = (p.d + CS - 1) / CS, tiles = (p.n + GATED_TILE - 1) / GATED_TILE;
  const Deal at = deal(p, p.BH * groups, tiles);
  const int bh = at.slab / groups, c0 = (at.slab % groups) * CS, k = at.turn, tid = threadIdx.x;
  const int len = seq_len(p.lens, bh / p.H, p.n), used = (len + GATED_TILE - 1) / GATED_TILE;
  if (k >= used) {
    if (k == 0 && p.s_last && tid < CS && c0 + tid < p.d) {  // an empty sequence
      const long o = (long)bh * p.d + c0 + tid;
      p.s_last[o] = p.s0 ? p.s0[o] : 0.f;
    }
    return;
  }
  const int cg = tid % CG, tt = tid / CG, ch = c0 + cg * V, t0 = k * GATED_TILE + tt * R;
  const long base = (long)bh * p.n * p.d;
  const int bytes = len * p.d * (int)sizeof(T), row = p.d * (int)sizeof(T);
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc((const T *)p.x + base, bytes), rg = buf_rsrc((const T *)p.g + base, bytes),
                               ro = buf_rsrc((const T *)p.out + base, bytes);
  Pack<V, T> x[R], g[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // rows and channels past the end read as zeros
    const int off = ch < p.d && t0 + r < len ? (t0 + r) * row + ch * (int)sizeof(T) : OOB_OFFSET;
    g[r] = ld_pack<T, V>(rg, off);
    x[r] = ld_pack<T, V>(rx, off);
  }
  Run<GATE> A[V];
  float Hs[V], held[R][V];
#pragma unroll
  for (int e = 0; e < V; ++e) Hs[e] = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // row by row, as the loads arrive (log gates, 8 x 16 heads x 8192 x 128: 174 -> 166 us)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // past the end the state stays; a log gate read as zero there is that by itself
      float arg = 0.f, h;
      if constexpr (GATE == HLA2_GATE_LOG) {
        arg = gate_arg<GATE>((float)g[r].e[e]);
        h = hold<T, GATE>(arg);
      } else {
        h = t0 + r < len ? hold<T, GATE>((float)g[r].e[e]) : HELD_ONE;
      }
      if constexpr (HOLD) held[r][e] = h;
      A[e].then(arg, h);
      Hs[e] = advance<GATE>(h, (float)x[r].e[e], Hs[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) sA[tt][cg * V + e] = A[e].held(), sH[tt][cg * V + e] = Hs[e];
  __syncthreads();
  {  // exclusive prefixes of the thread rows within each quarter
    const int c = tid % CS, q = tid / CS;
    Decay fA;
    float fH = 0.f;
#pragma unroll
    for (int m = 0; m < PQ; ++m) {
      const float mA = sA[q * PQ + m][c], mH = sH[q * PQ + m][c];
      sA[q * PQ + m][c] = fA.held();
      sH[q * PQ + m][c] = fH;
      fH = scale_add(mA, fH, mH);
      fA.then(mA);
    }
    qA[q][c] = fA.held();
    qH[q][c] = fH;
  }
  __syncthreads();
  if (tid < CS) {
    const bool in = c0 + tid < p.d;
    const long o = (long)bh * p.d + c0 + tid;
    Decay run;
    float tH = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      tH = scale_add(qA[q][tid], tH, qH[q][tid]);
      run.then(qA[q][tid]);
    }
    const float tA = run.held();
    float s;
    if (k == 0) {
      s = p.s0 && in ? p.s0[o] : 0.f;
    } else {
      Word *w = words_of<CS>(p, at.slab, k, tiles, tid);
      publish_map(w, tA, tH);
      s = look_back<CS>(w, 2 * CS, k);
    }
    const float last = scale_add(tA, s, tH);
    if (k + 1 < used) publish_state(words_of<CS>(p, at.slab, k, tiles, tid) + CS, last);
    if (in) {
      if (p.marks_out) p.marks_out[((long)bh * tiles + k) * p.d + c0 + tid] = s;
      if (p.s_last && k + 1 == used) p.s_last[o] = last;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      qC[q][tid] = s;
      s = scale_add(qA[q][tid], s, qH[q][tid]);
    }
  }
  __syncthreads();
  fresh(x);
  if constexpr (HOLD) fresh(held);
  else fresh(g);
  float s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = scale_add(sA[tt][cg * V + e], qC[tt / PQ][cg * V + e], sH[tt][cg * V + e]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    Pack<V, T> y;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float h = HOLD ? held[r][e] : hold<T, GATE>(gate_arg<GATE>((float)g[r].e[e]));
      s[e] = advance<GATE>(h, (float)x[r].e[e], s[e]);  // rows past the end are dropped
      y.e[e] = (T)s[e];
    }
    st_pack<T, V>(ro, ch < p.d && t0 + r < len ? (t0 + r) * row + ch * (int)sizeof(T) : OOB_OFFSET, y);
  }
}

// Backward.  Bound by HBM: x, g and dout read once, dx and dg written once (65536 tokens x 2048 channels,
// bf16, sigmoid: 280 us, 4.8 TB/s; with the gate formed anew at each use 18% more).  The tile's states are
// recomputed from its mark, so the only carry is the adjoint's, u = a r, which runs from the last tile to
// the first: turn 0 is the sequence's last tile.
template <typename T, int GATE, bool VEC>
__global__ void __launch_bounds__(256, 2) gated_backward_kernel(GatedArgs p) {
  using S = Shape<T, VEC>;
  constexpr int V = S::V, CG = S::CG, TT = S::TT, R = S::R, CS = S::CS, Q = S::Q, PQ = S::PQ;
  __shared__ float sA[TT][CS], sH[TT][CS], sU[TT][CS], sB[TT][CS], qA[Q][CS], qH[Q][CS], qU[Q][CS], qC[Q][CS], qD[Q][CS];
  const int groups = (p.d + CS - 1) / CS, tiles = (p.n + GATED_TILE - 1) / GATED_TILE;
  const Deal at = deal(p, p.BH * groups, tiles);
  const int bh = at.slab / groups, c0 = (at.slab % groups) * CS, turn = at.turn, tid = threadIdx.x;
  const int len = seq_len(p.lens, bh / p.H, p.n), used = (len + GATED_TILE - 1) / GATED_TILE;
  if (turn >= used) {
    if (turn == 0 && p.ds0 && tid < CS && c0 + tid < p.d) {
      const long o = (long)bh * p.d + c0 + tid;
      p.ds0[o] = p.ds_last ? p.ds_last[o] : 0.f;
    }
    return;
  }
  const int k = used - 1 - turn;
  const int cg = tid % CG, tt = tid / CG, ch = c0 + cg * V, t0 = k * GATED_TILE + tt * R;
  const long base = (long)bh * p.n * p.d;
  const int bytes = len * p.d * (int)sizeof(T), row = p.d * (int)sizeof(T);
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc((const T *)p.x + base, bytes), rg = buf_rsrc((const T *)p.g + base, bytes),
                               rd = buf_rsrc((const T *)p.dout + base, bytes),
                               rdx = buf_rsrc((const T *)p.dx + base, bytes), rdg = buf_rsrc((const T *)p.dg + base, bytes);
  Pack<V, T> x[R], y[R];
  float h[R][V];  // the gates
  Run<GATE> A[V];
  {
    Pack<V, T> g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int off = ch < p.d && t0 + r < len ? (t0 + r) * row + ch * (int)sizeof(T) : OOB_OFFSET;
      g[r] = ld_pack<T, V>(rg, off);
      x[r] = ld_pack<T, V>(rx, off);
      y[r] = ld_pack<T, V>(rd, off);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float gv = (float)g[r].e[e], arg = gate_arg<GATE>(gv);
        h[r][e] = GATE == HLA2_GATE_LOG || t0 + r < len ? hold<T, GATE>(arg) : HELD_ONE;  // past the end: the states stay
        if constexpr (GATE == HLA2_GATE_LOG) {
          A[e].then(arg, h[r][e]);
          // +0 says that a gate above 0 has no gradient; z is 2^-126 or more (by the bits: -a is left alone), which
          // moves nothing
          const unsigned bits = __builtin_bit_cast(unsigned, h[r][e]);
          h[r][e] = gv > 0.f ? 0.f : __builtin_bit_cast(float, bits < 0x00800000u ? 0x00800000u : bits);
        }
      }
  }
  {
    float Hs[V], U[V];
#pragma unroll
    for (int e = 0; e < V; ++e) Hs[e] = 0.f, U[e] = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (GATE == HLA2_GATE_SIGMOID) A[e].then(0.f, h[r][e]);
        Hs[e] = advance<GATE>(h[r][e], (float)x[r].e[e], Hs[e]);
      }
    }
    fresh(h);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) U[e] = scale(h[r][e], (float)y[r].e[e] + U[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sA[tt][cg * V + e] = A[e].held(), sH[tt][cg * V + e] = Hs[e], sU[tt][cg * V + e] = U[e];
  }
  __syncthreads();
  {
    const int c = tid % CS, q = tid / CS;
    Decay fA, bA;
    float mA[PQ], fH = 0.f, bU = 0.f;
#pragma unroll
    for (int m = 0; m < PQ; ++m) {
      mA[m] = sA[q * PQ + m][c];
      const float mH = sH[q * PQ + m][c];
      sA[q * PQ + m][c] = fA.held();
      sH[q * PQ + m][c] = fH;
      fH = scale_add(mA[m], fH, mH);
      fA.then(mA[m]);
    }
    qA[q][c] = fA.held();
    qH[q][c] = fH;
#pragma unroll
    for (int m = PQ - 1; m >= 0; --m) {
      const float mU = sU[q * PQ + m][c];
      sB[q * PQ + m][c] = bA.held();
      sU[q * PQ + m][c] = bU;
      bU = scale_add(mA[m], bU, mU);
      bA.then(mA[m]);
    }
    qU[q][c] = bU;
  }
  __syncthreads();
  if (tid < CS) {
    const bool in = c0 + tid < p.d;
    const long o = (long)bh * p.d + c0 + tid;
    float s = 0.f;
    if (in) s = p.marks ? p.marks[((long)bh * tiles + k) * p.d + c0 + tid] : (p.s0 ? p.s0[o] : 0.f);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      qC[q][tid] = s;
      s = scale_add(qA[q][tid], s, qH[q][tid]);
    }
    Decay run;
    float tU = 0.f;
#pragma unroll
    for (int q = Q - 1; q >= 0; --q) {
      tU = scale_add(qA[q][tid], tU, qU[q][tid]);
      run.then(qA[q][tid]);
    }
    const float tA = run.held();
    float u;
    if (turn == 0) {
      u = p.ds_last && in ? p.ds_last[o] : 0.f;
    } else {
      Word *w = words_of<CS>(p, at.slab, turn, tiles, tid);
      publish_map(w, tA, tU);
      u = look_back<CS>(w, 2 * CS, turn);
    }
    const float first = scale_add(tA, u, tU);
    if (k > 0) publish_state(words_of<CS>(p, at.slab, turn, tiles, tid) + CS, first);
    if (in && p.ds0 && k == 0) p.ds0[o] = first;
#pragma unroll
    for (int q = Q - 1; q >= 0; --q) {
      qD[q][tid] = u;
      u = scale_add(qA[q][tid], u, qU[q][tid]);
    }
  }
  __syncthreads();
  fresh(x);
  fresh(y);
  fresh(h);
  float before[R][V], s[V], u[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = cg * V + e, q = tt / PQ;
    s[e] = scale_add(sA[tt][c], qC[q][c], sH[tt][c]);
    u[e] = scale_add(sB[tt][c], qD[q][c], sU[tt][c]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float xv = (float)x[r].e[e];
      before[r][e] = GATE == HLA2_GATE_LOG ? s[e] : s[e] - xv;
      s[e] = advance<GATE>(h[r][e], xv, s[e]);
    }
  fresh(h);
#pragma unroll
  for (int r = R - 1; r >= 0; --r) {
    Pack<V, T> ox, og;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = (float)y[r].e[e] + u[e];
      u[e] = scale(h[r][e], d);
      if constexpr (GATE == HLA2_GATE_LOG) {
        ox.e[e] = (T)d;
        og.e[e] = (T)(__builtin_bit_cast(int, h[r][e]) == 0 ? 0.f : u[e] * before[r][e]);
      } else {
        const float z = held_z(h[r][e]);
        ox.e[e] = (T)(z * d);
        og.e[e] = (T)(u[e] * z * before[r][e]);
      }
    }
    const int off = ch < p.d && t0 + r < len ? (t0 + r) * row + ch * (int)sizeof(T) : OOB_OFFSET;
    st_pack<T, V>(rdx, off, ox);
    st_pack<T, V>(rdg, off, og);
  }
}

__global__ void __launch_bounds__(256) gated_clear_kernel(u32x4 *w, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) w[i] = u32x4{0, 0, 0, 0};
}

// A thread to a channel.  A step of 256 x 32 heads x 64 channels takes as long as its launch.
template <typename T, int GATE>
__global__ void __launch_bounds__(256) gated_step_kernel(GatedStepArgs p) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)p.N * p.Hd || (p.pos && p.pos[i / p.Hd] < 0)) return;
  const float s = advance<GATE>(hold<T, GATE>(gate_arg<GATE>((float)((const T *)p.g)[i])), (float)((const T *)p.x)[i], p.state[i]);
  p.state[i] = s;
  ((T *)p.out)[i] = (T)s;
}

// f(type tag, gate constant) for the runtime type and gate
template <typename F> hipError_t by_kind(int dtype, int gate, F &&f) {
  if (dtype == 0) {
    if (gate == HLA2_GATE_LOG) f(float{}, std::integral_constant<int, HLA2_GATE_LOG>{});
    else f(float{}, std::integral_constant<int, HLA2_GATE_SIGMOID>{});
  } else {
    if (gate == HLA2_GATE_LOG) f(bf16{}, std::integral_constant<int, HLA2_GATE_LOG>{});
    else f(bf16{}, std::integral_constant<int, HLA2_GATE_SIGMOID>{});
  }
  return hipGetLastError();
}

}  // namespace

// Vectors when every row of every array starts on 16 bytes and is a whole number of them.
static bool whole_vectors(int dtype, int d, std::initializer_list<const void *> arrays) {
  const int V = dtype == 0 ? 4 : 8;
  uintptr_t bits = 0;
  for (const void *p : arrays) bits |= (uintptr_t)p;
  return d % V == 0 && bits % 16 == 0;
}

template <typename F> static hipError_t launch_tiles(int dtype, int gate, bool vec, const GatedArgs &a, hipStream_t s, F &&f) {
  const int cs = vec && dtype != 0 ? 64 : 32, tiles = (a.n + GATED_TILE - 1) / GATED_TILE;
  const unsigned grid = (unsigned)a.BH * ((a.d + cs - 1) / cs) * tiles;
  if (a.words) {
    const long n = (long)gated_words_bytes(a.BH, a.n, a.d) / 16;
    const long blocks = (n + 1023) / 1024;
    hipLaunchKernelGGL(gated_clear_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s,
                       (u32x4 *)a.words, n);
  }
  return by_kind(dtype, gate, [&](auto t, auto k) {
    if (vec) f(t, k, std::true_type{}, grid);
    else f(t, k, std::false_type{}, grid);
  });
}

size_t gated_words_bytes(int BH, int n, int d) {
  const size_t tiles = ((size_t)n + GATED_TILE - 1) / GATED_TILE;
  if (tiles < 2) return 0;
  return 8 * ((size_t)GATED_WORD0 + (size_t)BH * tiles * 2 * (((size_t)d + 63) / 64 * 64));
}

hipError_t launch_gated_forward(int dtype, int gate, const GatedArgs &a, hipStream_t s) {
  return launch_tiles(dtype, gate, whole_vectors(dtype, a.d, {a.x, a.g, a.out}), a, s, [&](auto t, auto k, auto v, unsigned grid) {
    hipLaunchKernelGGL((gated_forward_kernel<decltype(t), k.value, v.value>), dim3(grid), dim3(256), 0, s, a);
  });
}

hipError_t launch_gated_backward(int dtype, int gate, const GatedArgs &a, hipStream_t s) {
  return launch_tiles(dtype, gate, whole_vectors(dtype, a.d, {a.x, a.g, a.dout, a.dx, a.dg}), a, s,
                      [&](auto t, auto k, auto v, unsigned grid) {
    hipLaunchKernelGGL((gated_backward_kernel<decltype(t), k.value, v.value>), dim3(grid), dim3(256), 0, s, a);
  });
}

hipError_t launch_gated_step(int dtype, int gate, const GatedStepArgs &a, hipStream_t s) {
  const unsigned grid = (unsigned)(((long)a.N * a.Hd + 255) / 256);
  return by_kind(dtype, gate, [&](auto t, auto k) {
    hipLaunchKernelGGL((gated_step_kernel<decltype(t), k.value>), dim3(grid), dim3(256), 0, s, a);
  });
}

}  // namespace hla2
