// hla2_window_bwd.hip -- backward pass of windowed attention.
//
// Two walks, each recomputing the weights p = exp(scale q.k - lse) tile by tile: one holds a block of
// queries and passes over the keys they see (dq, and D = dout . out on the way), one holds a block of
// keys and passes over the queries that see them (dk, dv).  That is seven products where one walk with
// shared sums would do with five, but every sum has one owner: no atomics, and the same bits on every
// run.
// The sinks' keys are seen by every later query.  Their far queries (t - j >= window) are cut into
// runs, each head's run summed by a workgroup of its own, in the same launch, into the workspace, where the
// walk of those keys leaves its sums too; a launch of one thread to four sums adds them up, in order.
//
// Measured at 16 heads (4 key heads) x 65536 tokens, d = dv = 128, window 2048, 16 sinks: dq 1.90 ms (1.2
// PFLOP/s with ds in two operands), dk and dv with the far queries 2.68 ms (0.9), their sum 0.02 ms.  dq has the
// matrix units busy in 57% of the cycles and vector issue in 54%; dk and dv 38% and 36%, with LDS at 53%: a wave
// holds 16 keys at d = 128 (registers), so each fragment feeds one product.  Slower there: 32 keys to a wave with
// one wave to a SIMD (3.3 against 2.5 ms), or with v in LDS and one buffer (4.7, spills); below, 32 keys fit.
#include "hla2.h"
#include "hla2_window.h"

namespace hla2 {
namespace {

constexpr float LOG2E = 1.44269504088896340736f;

// the first tile of far queries
__host__ __device__ __forceinline__ int far_first(int window) { return window / WIN_KEYS * WIN_KEYS; }

constexpr int DOT_TILES = 5;  // tiles of a block of queries up to which D is formed from the weights

// ds as two operands of a product, hi + lo, each rounded to bf16 (fp32: as one).  Rounded once, ds is
// the largest error of dq and dk: the terms of a row of dq cancel (sum_j ds_tj = 0).  On the training
// workload of 4 x 8 heads x 2048 tokens, relative to the 64-bit gradients and with the result's own
// rounding at 1.66e-3: dq 2.8e-3 with one operand, 2.1e-3 with two; dk 2.5e-3 with one.  dq takes two
// everywhere (d = dv = 128, 65536 tokens: 1.59 -> 1.98 ms); dk takes two on edge tiles, which hold the
// rows that see few keys and so the largest weights, and one elsewhere (two everywhere: 2.7 -> 3.0 ms).
// dv takes the weights so too, with 16 keys to a wave (window 18, eight heads to a key head: 2.7e-3 -> 1.7e-3).
__device__ __forceinline__ void split_frag(const f32x4 *s, bf16x8 &hi, bf16x8 &lo) {
  hi = frag_from_acc(s[0], s[1]);
  f32x4 r0, r1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r0[e] = s[0][e] - (float)hi[e];
    r1[e] = s[1][e] - (float)hi[4 + e];
  }
  lo = frag_from_acc(r0, r1);
}
__device__ __forceinline__ void split_frag(const f32x4 *s, f32x4 &hi, f32x4 &) { hi = s[0]; }

// The scores s of QW x 16 queries with 16 NS keys from row0 of a tile, and dp = dout . v with their values.
template <typename TK, typename TV, typename FR, int QW, int NS, int NK, int NV, typename T>
__device__ __forceinline__ void scores(f32x4 (&s)[QW][NS], f32x4 (&dp)[QW][NS], const FR (&qf)[QW][NK],
                                       const FR (&df)[QW][NV], const T *K, const T *V, int row0, int lane) {
  constexpr int KT = Ktile<T>::ROWS;
  stream<T, NS * (NK + NV)>(
      [&](int x) {
        const int row = row0 + 16 * (x / (NK + NV)), m = x % (NK + NV);
        return m < NK ? TK::rows(K, row, m * KT, lane) : TV::rows(V, row, (m - NK) * KT, lane);
      },
      [&](int x, const FR &f) {
        const int c = x / (NK + NV), m = x % (NK + NV);
#pragma unroll
        for (int i = 0; i < QW; ++i) {
          if (m < NK) s[i][c] = mma1(f, qf[i][m], m ? s[i][c] : zero4());
          else dp[i][c] = mma1(f, df[i][m - NK], m > NK ? dp[i][c] : zero4());
        }
      });
  feed<T, 1, QW, NS * (NK + NV)>();
}

// dq: the forward walk with the queries' rows of q and dout held in registers.
template <typename T, int DK, int DV, int QW>
__global__ void __launch_bounds__(256, 2) window_dq_kernel(WindowBwdArgs p) {
  typedef Tile64<T, DK> TK;
  typedef Tile64<T, DV> TV;
  constexpr int KT = Ktile<T>::ROWS, NK = DK / KT, NV = DV / KT, QB = 64 * QW, NPF = WIN_KEYS / KT;
  constexpr int HT = DK + DV > 192 ? 1 : NPF, NS = HT * KT / 16;
  typedef typename Ktile<T>::frag frag;
  __shared__ __align__(16) T sK[2][WIN_KEYS * DK], sV[2][WIN_KEYS * DV];
  const int G = p.H / p.Hkv, nqb = (p.n + QB - 1) / QB, total = p.B * p.H * nqb;
  int id = xcd_order(blockIdx.x, total);
  if (id >= total) return;
  const int gh = id % G;
  id /= G;
  const int qb = id % nqb, bk = id / nqb, b = bk / p.Hkv, bh = b * p.H + (bk % p.Hkv) * G + gh;
  const int len = win_len(p.lens, b, p.n), q0 = qb * QB;
  if (q0 >= len) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, col = lane & 15;
  const T *q = (const T *)p.q + (long)bh * p.n * p.d, *k = (const T *)p.k + (long)bk * p.n * p.d,
          *v = (const T *)p.v + (long)bk * p.n * p.dv, *dout = (const T *)p.dout + (long)bh * p.n * p.dv,
          *out = (const T *)p.out + (long)bh * p.n * p.dv;
  const WinTiles tiles(q0, min(q0 + QB, len) - 1, p.window, p.sinks);
  const int qa = q0 + wave * 16 * QW, qz = qa + 16 * QW - 1;
  TK fk;
  TV fv;
  fk.init(p.d, tid);
  fv.init(p.dv, tid);
  frag qf[QW][NK], df[QW][NV];
  float lse2[QW], dot[QW];
  const __amdgpu_buffer_rsrc_t rq = buf_rsrc(q, len * p.d * (int)sizeof(T)), rd = buf_rsrc(dout, len * p.dv * (int)sizeof(T)),
                               ro = buf_rsrc(out, len * p.dv * (int)sizeof(T));
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    const int t = qa + 16 * i + col;
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < NK; ++m) qf[i][m] = ldg_rows<T>(rq, p.d, qa + 16 * i, m * KT, lane);
#pragma unroll
    for (int m = 0; m < NV; ++m) {
      df[i][m] = ldg_rows<T>(rd, p.dv, qa + 16 * i, m * KT, lane);
      const frag of = ldg_rows<T>(ro, p.dv, qa + 16 * i, m * KT, lane);
#pragma unroll
      for (int e = 0; e < KT / 4; ++e) s = fmaf((float)df[i][m][e], (float)of[e], s);
    }
    dot[i] = add_groups(s);
    lse2[i] = t < len ? p.lse[(long)bh * p.n + t] * LOG2E : INFINITY;  // rows past the end: p = 0
  }
  auto needs = [&](int j0) { return j0 <= qz && (j0 + WIN_KEYS > qa - p.window + 1 || j0 < p.sinks); };
  // whether every key of the tile is seen by every query of the wave
  auto whole = [&](int j0) {
    return j0 + WIN_KEYS - 1 <= qa && (qz - j0 < p.window || j0 + WIN_KEYS <= p.sinks);
  };
  auto mask = [&](auto &s, int j0) {  // the scores of keys j0 ..
#pragma unroll
    for (int i = 0; i < QW; ++i)
#pragma unroll
      for (int c = 0; c < (int)(sizeof(s[0]) / sizeof(s[0][0])); ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!win_sees(qa + 16 * i + col, j0 + 16 * c + 4 * g + e, p.window, p.sinks)) s[i][c][e] = -INFINITY;
  };
  // Here D = dout . out has the rounding of out as it was saved, which counts where a row sees few keys: over
  // 280 drawn shapes dq was up to 4.0e-3 off (8 to 90 tokens), 2.5e-3 at a window of 70.  A block of few tiles
  // therefore passes over them once more for bf16 and takes D = sum_j p_tj (dout_t . v_j): then 1.7 to 2.1e-3.
  // It costs most where every block is one of these (a training pass of 4 x 16 heads x 4096 tokens, window 128:
  // 232 -> 274 us).
  if (sizeof(T) == 2 && tiles.count <= DOT_TILES) {
#pragma unroll
    for (int i = 0; i < QW; ++i) dot[i] = 0.f;
    for (int it = 0; it < tiles.count; ++it) {
      const int j0 = tiles.tile(it), ln = fresh(lane);
      fk.fetch(k, p.d, j0, len);
      fv.fetch(v, p.dv, j0, len);
      fk.put(sK[0], tid);
      fv.put(sV[0], tid);
      __syncthreads();
      if (needs(j0)) {
#pragma unroll
        for (int h = 0; h < NPF; ++h) {
          f32x4 s[QW][KT / 16], dp[QW][KT / 16];
          scores<TK, TV>(s, dp, qf, df, sK[0], sV[0], h * KT, ln);
          __builtin_amdgcn_sched_barrier(0);
          if (!whole(j0)) mask(s, j0 + h * KT);
#pragma unroll
          for (int i = 0; i < QW; ++i)
#pragma unroll
            for (int c = 0; c < KT / 16; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dot[i] = fmaf(__builtin_amdgcn_exp2f(fmaf(s[i][c][e], p.scale2, -lse2[i])), dp[i][c][e], dot[i]);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < QW; ++i) dot[i] = add_groups(dot[i]);
  }
  fk.fetch(k, p.d, tiles.tile(0), len);
  fv.fetch(v, p.dv, tiles.tile(0), len);
  f32x4 o[QW][DK / 16];
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    const int t = qa + 16 * i + col;
    if (g == 0 && t < len) p.dot[(long)bh * p.n + t] = dot[i];
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) o[i][c] = zero4();
  }
  fk.put(sK[0], tid);
  fv.put(sV[0], tid);
  __syncthreads();

  // A tile, HT k-tiles of keys at a time.  At d = dv = 128 one at a time, so that the scores and ds of few
  // keys are live and nothing spills (1.70 -> 1.59 ms, ds in one operand); below, all of them.
  auto pass = [&](bool masked, const T *K, const T *V, int j0, int lane) {
#pragma unroll
    for (int h = 0; h < NPF; h += HT) {
      f32x4 s[QW][NS], dp[QW][NS];
      scores<TK, TV>(s, dp, qf, df, K, V, h * KT, lane);
      __builtin_amdgcn_sched_barrier(0);
      if (masked) mask(s, j0 + h * KT);
      frag hi[QW][HT], lo[QW][HT];
#pragma unroll
      for (int i = 0; i < QW; ++i) {
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = __builtin_amdgcn_exp2f(fmaf(s[i][c][e], p.scale2, -lse2[i]));
            s[i][c][e] = w * (dp[i][c][e] - dot[i]);
          }
#pragma unroll
        for (int m = 0; m < HT; ++m) split_frag(s[i] + m * KT / 16, hi[i][m], lo[i][m]);
      }
      __builtin_amdgcn_sched_barrier(0);
      stream<T, DK / 16 * HT>([&](int x) { return TK::cols(K, (h + x % HT) * KT, 16 * (x / HT), lane); },
                              [&](int x, const frag &f) {
                                const int c = x / HT, m = x % HT;
#pragma unroll
                                for (int i = 0; i < QW; ++i) {
                                  o[i][c] = mma1(f, hi[i][m], o[i][c]);
                                  if constexpr (sizeof(T) == 2) o[i][c] = mma1(f, lo[i][m], o[i][c]);
                                }
                              });
      feed<T, 2, 2 * QW, DK / 16 * HT>();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int it = 0; it < tiles.count; ++it) {
    const int j0 = tiles.tile(it), jn = tiles.tile(min(it + 1, tiles.count - 1));
    fk.fetch(k, p.d, jn, len);  // after the last tile: that tile again, not used
    fv.fetch(v, p.dv, jn, len);
    // fresh where the addresses, held, would make these registers spill; elsewhere held (1.95 -> 1.91 ms)
    if (needs(j0)) pass(!whole(j0), sK[it & 1], sV[it & 1], j0, QW == 2 && DK + DV <= 192 ? fresh(lane) : lane);
    fk.put(sK[(it + 1) & 1], tid);
    fv.put(sV[(it + 1) & 1], tid);
    __syncthreads();
  }
  T *dq = (T *)p.dq + (long)bh * p.n * p.d;
#pragma unroll
  for (int i = 0; i < QW; ++i)
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) st_out(dq, p.d, qa + 16 * i + col, 16 * c + 4 * g, len, o[i][c] * p.scale);
}

// A workgroup's sums over the sinks' far queries: for each 16 keys that hold sinks (a wave's share) the
// accumulator vectors of dk and dv, a lane's side by side with its neighbours'.
__host__ __device__ constexpr int far_vectors(int DK, int DV, int sinks) { return (sinks + 15) / 16 * ((DK + DV) / 16) * 64; }

// blocks of keys to walk; with heads apart, each query head's
__host__ __device__ __forceinline__ int dkv_blocks(const WindowBwdArgs &p, int KB) {
  return (p.parts ? p.B * p.H : p.B * p.Hkv) * ((p.n + KB - 1) / KB);
}

template <typename T, int DK, int DV> struct DkvShared {
  T Q[2][WIN_KEYS * DK], D[2][WIN_KEYS * DV];
  float L[2][WIN_KEYS], dot[2][WIN_KEYS];
};

// dk, dv: a block of KB keys held in registers, the queries that see them passed over, head by head of
// the group.  FAR: the first WIN_KEYS keys and one run of one head's far queries, into the workspace.
template <typename T, int DK, int DV, int KW, bool FAR>
__device__ __forceinline__ void dkv_walk(const WindowBwdArgs &p, DkvShared<T, DK, DV> &sh, int block) {
  typedef Tile64<T, DK> TQ;
  typedef Tile64<T, DV> TD;
  static_assert(!FAR || KW == 1, "a run's sums are those of 64 keys");
  constexpr int KT = Ktile<T>::ROWS, NK = DK / KT, NV = DV / KT, KB = 64 * KW, NQT = WIN_KEYS / 16, NPF = WIN_KEYS / KT;
  constexpr int ND = (DK + DV) / 16;
  typedef typename Ktile<T>::frag frag;
  auto &sQ = sh.Q;
  auto &sD = sh.D;
  auto &sL = sh.L, &sDot = sh.dot;
  const int G = p.H / p.Hkv, nkb = (p.n + KB - 1) / KB;
  const bool alone = !FAR && p.parts;  // one query head of the group, its sums into the workspace
  const int total = FAR ? p.B * p.H * p.runs : dkv_blocks(p, KB);
  const int id = xcd_order(block, total);
  if (id >= total) return;
  // FAR: run `id % runs` of query head `id / runs`, whose sums are the id-th
  const int bk = FAR ? id / p.runs / G : alone ? id / nkb / G : id / nkb, b = bk / p.Hkv, len = win_len(p.lens, b, p.n);
  const int k0 = FAR ? 0 : id % nkb * KB;
  if (k0 >= len) return;
  const int qfirst = FAR ? far_first(p.window) + id % p.runs * p.run : k0;
  const int reach = p.window < p.n ? k0 + KB - 1 + p.window : p.n;
  const int qend = min(FAR ? qfirst + p.run : reach, len);
  const int nt = qend > qfirst ? (qend - qfirst + WIN_KEYS - 1) / WIN_KEYS : 0, count = FAR || alone ? nt : nt * G;
  if (count == 0) return;  // a run behind the sequence's end
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, col = lane & 15;
  const T *k = (const T *)p.k + (long)bk * p.n * p.d, *v = (const T *)p.v + (long)bk * p.n * p.dv;
  const long bh0 = FAR ? id / p.runs : alone ? id / nkb : (long)bk * G;
  const int ka = k0 + wave * 16 * KW, kz = ka + 16 * KW - 1;

  TQ fq;
  TD fd;
  fq.init(p.d, tid);
  fd.init(p.dv, tid);
  float fl = 0.f, fdot = 0.f;
  long bh = bh0;  // the tile being fetched
  int t0 = qfirst;
  auto fetch = [&]() {
    fq.fetch((const T *)p.q + bh * p.n * p.d, p.d, t0, len);
    fd.fetch((const T *)p.dout + bh * p.n * p.dv, p.dv, t0, len);
    const int t = t0 + (tid & 63);
    fl = t < len ? p.lse[bh * p.n + t] * LOG2E : INFINITY;  // rows past the end: p = 0
    fdot = t < len ? p.dot[bh * p.n + t] : 0.f;
  };
  auto put = [&](int to) {
    fq.put(sQ[to], tid);
    fd.put(sD[to], tid);
    if (tid < WIN_KEYS) {
      sL[to][tid] = fl;
      sDot[to][tid] = fdot;
    }
  };
  fetch();
  frag kf[KW][NK], vf[KW][NV];
  f32x4 ok[KW][DK / 16], ov[KW][DV / 16];
  const __amdgpu_buffer_rsrc_t rk = buf_rsrc(k, len * p.d * (int)sizeof(T)), rv = buf_rsrc(v, len * p.dv * (int)sizeof(T));
#pragma unroll
  for (int i = 0; i < KW; ++i) {
#pragma unroll
    for (int m = 0; m < NK; ++m) kf[i][m] = ldg_rows<T>(rk, p.d, ka + 16 * i, m * KT, lane);
#pragma unroll
    for (int m = 0; m < NV; ++m) vf[i][m] = ldg_rows<T>(rv, p.dv, ka + 16 * i, m * KT, lane);
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) ok[i][c] = zero4();
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) ov[i][c] = zero4();
  }
  put(0);
  __syncthreads();

  auto pass = [&](bool masked, const T *Q, const T *D, const float *L, const float *E, int t0, int lane) {
    frag wf[KW][NPF], sf[KW][NPF];
    f32x4 s[KW][NQT], dp[KW][NQT];
    stream<T, NQT * (NK + NV)>(
        [&](int x) {
          const int row = 16 * (x / (NK + NV)), m = x % (NK + NV);
          return m < NK ? TQ::rows(Q, row, m * KT, lane) : TD::rows(D, row, (m - NK) * KT, lane);
        },
        [&](int x, const frag &f) {
          const int c = x / (NK + NV), m = x % (NK + NV);
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            if (m < NK) s[i][c] = mma1(f, kf[i][m], m ? s[i][c] : zero4());
            else dp[i][c] = mma1(f, vf[i][m - NK], m > NK ? dp[i][c] : zero4());
          }
        });
    feed<T, 1, KW, NQT * (NK + NV)>();
    __builtin_amdgcn_sched_barrier(0);
    if (masked) {
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int c = 0; c < NQT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + 16 * c + 4 * g + e, j = ka + 16 * i + col;
            const bool in = FAR ? t - j >= p.window && j < p.sinks : j <= t && t - j < p.window;
            if (!in) s[i][c][e] = -INFINITY;
          }
    }
#pragma unroll
    for (int c = 0; c < NQT; ++c) {
      const f32x4 l4 = *(const f32x4 *)(L + 16 * c + 4 * g), e4 = *(const f32x4 *)(E + 16 * c + 4 * g);
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][c][e] = __builtin_amdgcn_exp2f(fmaf(s[i][c][e], p.scale2, -l4[e]));
          dp[i][c][e] = s[i][c][e] * (dp[i][c][e] - e4[e]);
        }
    }
#pragma unroll
    for (int i = 0; i < KW; ++i)
#pragma unroll
      for (int m = 0; m < NPF; ++m) {
        wf[i][m] = acc_frag(s[i], m, T{});
        sf[i][m] = acc_frag(dp[i], m, T{});
      }
    if (sizeof(T) == 2 && masked) {  // what the operands' rounding left
      constexpr bool W = KW == 1;     // the weights' too: with 32 keys to a wave their registers spill (41 -> 88 us)
      const int ln = fresh(lane);     // its addresses stay in this rare branch (2.77 -> 2.73 ms)
#pragma unroll
      for (int i = 0; i < KW; ++i) {
#pragma unroll
        for (int c = 0; c < NQT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dp[i][c][e] -= (float)(T)dp[i][c][e];
            if constexpr (W) s[i][c][e] -= (float)(T)s[i][c][e];
          }
#pragma unroll
        for (int m = 0; m < NPF; ++m) {
          const frag lo = acc_frag(dp[i], m, T{});
#pragma unroll
          for (int c = 0; c < DK / 16; ++c) ok[i][c] = mma1(TQ::cols(Q, m * KT, 16 * c, ln), lo, ok[i][c]);
          if constexpr (W) {
            const frag wl = acc_frag(s[i], m, T{});
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) ov[i][c] = mma1(TD::cols(D, m * KT, 16 * c, ln), wl, ov[i][c]);
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // fp32 sums a tile by itself first: a key's sum may run over every later query (3057 tokens, all visible:
    // dk off by 1.1e-6 of its norm in one chain, by 5.0e-7 so)
    constexpr int CV = DV / 16, CK = DK / 16;
    constexpr bool PART = sizeof(T) == 4;
    f32x4 tk[KW][CK], tv[KW][CV];
    stream<T, NPF * (CK + CV)>(
        [&](int x) {
          const int row = x / (CK + CV) * KT, c = x % (CK + CV);
          return c < CV ? TD::cols(D, row, 16 * c, lane) : TQ::cols(Q, row, 16 * (c - CV), lane);
        },
        [&](int x, const frag &f) {
          const int m = x / (CK + CV), c = x % (CK + CV);
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            f32x4 &to = c < CV ? (PART ? tv[i][c % CV] : ov[i][c % CV]) : PART ? tk[i][(c - CV) % CK] : ok[i][(c - CV) % CK];
            to = mma1(f, c < CV ? wf[i][m] : sf[i][m], PART && m == 0 ? zero4() : to);
          }
        });
    feed<T, 2, KW, NPF * (DK + DV) / 16>();
    if constexpr (PART) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
#pragma unroll
        for (int c = 0; c < CV; ++c) ov[i][c] += tv[i][c];
#pragma unroll
        for (int c = 0; c < CK; ++c) ok[i][c] += tk[i][c];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int it = 0; it < count; ++it) {
    const int now = t0;
    if (it + 1 < count) {  // after the last tile: that tile again, not used
      t0 += WIN_KEYS;
      if (t0 >= qend) {
        t0 = qfirst;
        ++bh;
      }
    }
    fetch();
    const int at = it & 1;
    if (FAR ? ka < p.sinks : now + WIN_KEYS > ka && now - kz < p.window) {
      const bool whole = !FAR && now >= kz && now + WIN_KEYS - 1 - ka < p.window;
      // as in window_dq_kernel (2.66 -> 2.58 ms; 32 keys to a wave would spill: 40.4 -> 42.6 us)
      pass(!whole, sQ[at], sD[at], sL[at], sDot[at], now, KW == 2 ? fresh(lane) : lane);
    }
    put(at ^ 1);
    __syncthreads();
  }
  // vectors of 16 keys' sums in the workspace: a run's, or behind the runs this walk's, where runs are added
  auto save = [&](long slot, int i) {
    f32x4 *to = (f32x4 *)p.far + slot * far_vectors(DK, DV, p.sinks) + (wave * KW + i) * ND * 64 + lane;
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) to[c * 64] = ok[i][c];
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) to[(DK / 16 + c) * 64] = ov[i][c];
  };
  if constexpr (FAR) {
    if (ka < p.sinks) save(id, 0);
  } else {
    const bool shared = k0 == 0 && p.runs > 0 && far_first(p.window) < len && !alone;
#pragma unroll
    for (int i = 0; i < KW; ++i) {
      const int j = ka + 16 * i + col;
      if (alone) {
        float *dk = p.parts + bh0 * p.n * (p.d + p.dv), *dvp = dk + (long)p.n * p.d;
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) st_out(dk, p.d, j, 16 * c + 4 * g, len, ok[i][c] * p.scale);
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) st_out(dvp, p.dv, j, 16 * c + 4 * g, len, ov[i][c]);
      } else if (shared && ka + 16 * i < p.sinks) {
        save((long)p.B * p.H * p.runs + bk, i);
      } else {
        T *dk = (T *)p.dk + (long)bk * p.n * p.d, *dvp = (T *)p.dv_out + (long)bk * p.n * p.dv;
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) st_out(dk, p.d, j, 16 * c + 4 * g, len, ok[i][c] * p.scale);
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) st_out(dvp, p.dv, j, 16 * c + 4 * g, len, ov[i][c]);
      }
    }
  }
}

// The blocks of keys, then the runs of far queries, which are shorter and fill up what the blocks leave
// idle (a launch of their own before: 4 x 8 heads x 2048 tokens, d = dv = 64, window 512, 4 sinks: 7 us more).
template <typename T, int DK, int DV, int KW>
__global__ void __launch_bounds__(256, 2) window_dkv_kernel(WindowBwdArgs p) {
  __shared__ __align__(16) DkvShared<T, DK, DV> sh;
  const int blocks = xcd_grid(dkv_blocks(p, 64 * KW));
  if ((int)blockIdx.x < blocks) dkv_walk<T, DK, DV, KW, false>(p, sh, blockIdx.x);
  else dkv_walk<T, DK, DV, 1, true>(p, sh, blockIdx.x - blocks);
}

// The sum of the far runs of a key head's query heads, vector x of them.
template <int DK, int DV> __device__ __forceinline__ f32x4 far_sum(const WindowBwdArgs &p, int bk, int len, int x) {
  const int NV = far_vectors(DK, DV, p.sinks), G = p.H / p.Hkv, far = len - far_first(p.window);
  const int used = far > 0 ? (far + p.run - 1) / p.run : 0;  // runs before the sequence's end
  f32x4 s = zero4();
  for (int h = 0; h < G; ++h) {
    const f32x4 *from = (const f32x4 *)p.far + ((long)bk * G + h) * p.runs * NV + x;
#pragma unroll 8
    for (int r = 0; r < used; ++r) s += from[(long)r * NV];
  }
  return s;
}

// dk and dv from the sums of the query heads that share a key head: a thread to four columns of a row.
template <typename T, int DK, int DV> __global__ void __launch_bounds__(256) window_heads_kernel(WindowBwdArgs p) {
  const int per = (p.d + p.dv) / 4, G = p.H / p.Hkv;
  const long x = (long)blockIdx.x * 256 + threadIdx.x, row = x / per;
  if (row >= (long)p.B * p.Hkv * p.n) return;
  const int t = (int)(row % p.n), c = (int)(x % per) * 4;
  const long bk = row / p.n, size = (long)p.n * (p.d + p.dv);
  const int len = win_len(p.lens, (int)(bk / p.Hkv), p.n);
  if (t >= len) return;
  const bool k = c < p.d;
  const int cc = k ? c : c - p.d;  // the column within dk or dv
  const long at = k ? (long)t * p.d + cc : (long)p.n * p.d + (long)t * p.dv + cc;
  f32x4 s = zero4();
#pragma unroll 4
  for (int h = 0; h < G; ++h) s += *(const f32x4 *)(p.parts + (bk * G + h) * size + at);
  if (p.runs > 0 && t < p.sinks) {
    const f32x4 far = far_sum<DK, DV>(p, (int)bk, len,
                                      (t / 16 * ((DK + DV) / 16) + (k ? 0 : DK / 16) + cc / 16) * 64 + cc % 16 / 4 * 16 + t % 16);
    s += k ? far * p.scale : far;
  }
  if (k) st4g((T *)p.dk + row * p.d + cc, s);
  else st4g((T *)p.dv_out + row * p.dv + cc, s);
}

// dk and dv of the sinks' keys: the runs' sums and the walk's, a thread to a vector.
template <typename T, int DK, int DV> __global__ void __launch_bounds__(256) window_far_kernel(WindowBwdArgs p) {
  const int NV = far_vectors(DK, DV, p.sinks);  // a multiple of 256
  const int bk = blockIdx.x / (NV / 256), x = blockIdx.x % (NV / 256) * 256 + threadIdx.x;
  const int len = win_len(p.lens, bk / p.Hkv, p.n);
  if (len <= far_first(p.window)) return;  // no far queries: the walk wrote its rows
  const f32x4 s = ((const f32x4 *)p.far)[((long)p.B * p.H * p.runs + bk) * NV + x] + far_sum<DK, DV>(p, bk, len, x);
  const int lane = x % 64, c = x / 64 % ((DK + DV) / 16), j = x / 64 / ((DK + DV) / 16) * 16 + lane % 16, e = lane / 16 * 4;
  if (c < DK / 16) st_out((T *)p.dk + (long)bk * p.n * p.d, p.d, j, 16 * c + e, len, s * p.scale);
  else st_out((T *)p.dv_out + (long)bk * p.n * p.dv, p.dv, j, 16 * (c - DK / 16) + e, len, s);
}

template <typename T, int DK, int DV, int QW, int KW> hipError_t run_backward(const WindowBwdArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((window_dq_kernel<T, DK, DV, QW>), dim3(xcd_grid(a.B * a.H * ((a.n + 64 * QW - 1) / (64 * QW)))),
                     dim3(256), 0, s, a);
  hipLaunchKernelGGL((window_dkv_kernel<T, DK, DV, KW>),
                     dim3(xcd_grid(dkv_blocks(a, 64 * KW)) + (a.runs > 0 ? xcd_grid(a.B * a.H * a.runs) : 0)), dim3(256), 0,
                     s, a);
  if (a.parts) {
    const long x = (long)a.B * a.Hkv * a.n * ((a.d + a.dv) / 4);
    hipLaunchKernelGGL((window_heads_kernel<T, DK, DV>), dim3((unsigned)((x + 255) / 256)), dim3(256), 0, s, a);
  } else if (a.runs > 0) {
    hipLaunchKernelGGL((window_far_kernel<T, DK, DV>), dim3((unsigned)a.B * a.Hkv * (far_vectors(DK, DV, a.sinks) / 256)),
                       dim3(256), 0, s, a);
  }
  return hipGetLastError();
}
// Fewer than a workgroup to a compute unit with 128 rows to a workgroup: 64, which ends sooner.  Rows that
// see fewer than NARROW keys in their window: 16 keys to a wave, for dv's precision (a training pass
// of 4 x 16 heads x 4096 tokens, window 64: the same time, 238 us; window 200: 292 against 281).
constexpr int NARROW = 128;
template <typename T, int DK, int DV, int KW> hipError_t by_rows(const WindowBwdArgs &a, hipStream_t s) {
  if (few_rows(a.B * a.H, a.n)) return run_backward<T, DK, DV, 1, 1>(a, s);
  if (KW == 2 && a.window < NARROW) return run_backward<T, DK, DV, 2, 1>(a, s);
  return run_backward<T, DK, DV, 2, KW>(a, s);
}

}  // namespace

// The far queries' runs: about 1024 workgroups over all heads, two tiles or more to a run.
int window_far_run(long heads, int n, int window) {
  const long tiles = (n - far_first(window) + WIN_KEYS - 1) / WIN_KEYS;
  const long run = (tiles * heads + 1023) / 1024;
  return (int)(run < 2 ? 2 : run) * WIN_KEYS;
}
int window_far_runs(long heads, int n, int window, int sinks) {
  if (sinks == 0 || window >= n) return 0;
  const int run = window_far_run(heads, n, window);
  return (n - far_first(window) + run - 1) / run;
}
size_t window_far_bytes(int dtype, int d, int dv, int sinks) {
  return 16 * (size_t)far_vectors(dtype == 0 || d <= 64 ? 64 : 128, dtype == 0 || dv <= 64 ? 64 : 128, sinks);
}

// Whether each query head's dk and dv are summed by workgroups of their own and added up in a launch
// after: where the key heads' blocks are fewer than the compute units (2 x 6 heads on 2 x 2, 1371 tokens,
// fp32: 58 us against 114 us).
bool window_heads_apart(int B, int H, int Hkv, int n) {
  return H > Hkv && (long)B * Hkv * ((n + WIN_KEYS - 1) / WIN_KEYS) < 256;
}

hipError_t launch_window_backward(int dtype, const WindowBwdArgs &a, hipStream_t s) {
  if (dtype == 0) return run_backward<float, 64, 64, 1, 1>(a, s);
  const bool k64 = a.d <= 64, v64 = a.dv <= 64;
  if (k64 && v64) return by_rows<bf16, 64, 64, 2>(a, s);
  if (k64) return by_rows<bf16, 64, 128, 1>(a, s);
  if (v64) return by_rows<bf16, 128, 64, 1>(a, s);
  return by_rows<bf16, 128, 128, 1>(a, s);
}

}  // namespace hla2
