// hla2_window.hip -- attention over a sliding window with visible first tokens: the forward pass over
// a sequence and the fill of the streaming cache.
//
// One pass over the keys a block of queries sees, with the running maximum and sum of the softmax.
// Scores are formed transposed, S^T = K Q^T: a lane then holds four keys of one query, so the maximum
// and the sum are a lane's own but for two exchanges between its four lane groups, the exponentials
// feed the product with V from registers (out^T = V^T P^T, operand order of hla2_mfma.h), and the
// accumulated rows are rescaled by a lane's own factor.
//
// A workgroup holds 128 rows of a head (64 where the grid would be small), a wave 32 of them, so that a
// fragment of K or V read from LDS feeds two products; the next tile of 64 keys is on its way from
// memory meanwhile.  At d = 64, dv = 128 a wave's tile is 48 matrix and 200 vector instructions (the
// exponentials twice), at d = dv = 128 64 and 200.
// Measured: 8 x 16 heads x 8192 tokens, d = 64, dv = 128, window 1024: 0.59 ms, 0.66 PFLOP/s; 16 heads x
// 65536 tokens, d = dv = 128, window 2048: 1.21 ms, 0.90 PFLOP/s, where a library product of 8192 x 8192
// matrices reaches 1.2.  No unit is full: matrix units 32% and 43% of the cycles, vector issue 53% and 51%, LDS
// 25% and 33%.  What is left are waits that the two waves of a SIMD do not cover for each other: without the
// tiles' loads and stores, through registers into LDS, it would be 25% faster, without barriers 6%.
// Sizes of d and dv between the instantiations are padded to the next, products and all.
// Slower: 16 rows to a wave and four waves to a SIMD (764 against 706 us at the first shape), 64 rows to a wave
// (1092), 256 rows to a workgroup (773), the next tile's scores formed during this one's softmax (730), two
// tiles on their way (711).
#include "hla2.h"
#include "hla2_window.h"

namespace hla2 {
namespace {

// Reference maximum: the weights are exp2(x - ref), x the scores in base 2.  The reference follows the
// running maximum only when that passes it by GROW, so the accumulated rows are rarely rescaled; the
// weights stay below 2^GROW, which fp32 sums and bf16 weights hold as exactly as weights below 1.
constexpr float GROW = 8.f;

template <typename T, int DK, int DV, int QW>
__global__ void __launch_bounds__(256, 2) window_forward_kernel(WindowArgs p) {
  typedef Tile64<T, DK> TK;
  typedef Tile64<T, DV> TV;
  constexpr int KT = Ktile<T>::ROWS, NK = DK / KT, QB = 64 * QW, NKT = WIN_KEYS / 16, NPF = WIN_KEYS / KT;
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
          *v = (const T *)p.v + (long)bk * p.n * p.dv;
  const WinTiles tiles(q0, min(q0 + QB, len) - 1, p.window, p.sinks);
  const int qa = q0 + wave * 16 * QW, qz = qa + 16 * QW - 1;  // this wave's queries

  TK fk;
  TV fv;
  fk.init(p.d, tid);
  fv.init(p.dv, tid);
  fk.fetch(k, p.d, tiles.tile(0), len);
  fv.fetch(v, p.dv, tiles.tile(0), len);
  frag qf[QW][NK];
  const __amdgpu_buffer_rsrc_t rq = buf_rsrc(q, len * p.d * (int)sizeof(T));
#pragma unroll
  for (int i = 0; i < QW; ++i)
#pragma unroll
    for (int m = 0; m < NK; ++m) qf[i][m] = ldg_rows<T>(rq, p.d, qa + 16 * i, m * KT, lane);
  f32x4 o[QW][DV / 16];
  float ref[QW], sum[QW];
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    ref[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) o[i][c] = zero4();
  }
  fk.put(sK[0], tid);
  fv.put(sV[0], tid);
  __syncthreads();

  auto pass = [&](bool masked, const T *K, const T *V, int j0, int lane) {
    frag pf[QW][NPF];
    f32x4 s[QW][NKT];
    __builtin_amdgcn_s_setprio(1);
    stream<T, NKT * NK>([&](int x) { return TK::rows(K, 16 * (x / NK), x % NK * KT, lane); },
                        [&](int x, const frag &f) {
                          const int c = x / NK, m = x % NK;
#pragma unroll
                          for (int i = 0; i < QW; ++i) s[i][c] = mma1(f, qf[i][m], m ? s[i][c] : zero4());
                        });
    feed<T, 1, QW, NKT * NK>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    if (masked) {
#pragma unroll
      for (int i = 0; i < QW; ++i)
#pragma unroll
        for (int c = 0; c < NKT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!win_sees(qa + 16 * i + col, j0 + 16 * c + 4 * g + e, p.window, p.sinks)) s[i][c][e] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < QW; ++i) {
      float top = s[i][0][0];
#pragma unroll
      for (int c = 0; c < NKT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i][c][e]);
      top = max_groups(top) * p.scale2;
      if (__any(top > ref[i] + GROW)) {  // also the first visible keys, from a reference of -inf
        const float next = top > ref[i] + GROW ? top : ref[i];
        const float f = ref[i] == -INFINITY ? 0.f : exp2f(ref[i] - next);
        ref[i] = next;
        sum[i] *= f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) o[i][c] *= f;
      }
      const float base = ref[i] == -INFINITY ? 0.f : ref[i];  // a query that has seen no key yet
#pragma unroll
      for (int c = 0; c < NKT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][c][e] = __builtin_amdgcn_exp2f(fmaf(s[i][c][e], p.scale2, -base));
          sum[i] += s[i][c][e];
        }
#pragma unroll
      for (int m = 0; m < NPF; ++m) pf[i][m] = acc_frag(s[i], m, T{});
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    stream<T, DV / 16 * NPF>([&](int x) { return TV::cols(V, x % NPF * KT, 16 * (x / NPF), lane); },
                             [&](int x, const frag &f) {
                               const int c = x / NPF, m = x % NPF;
#pragma unroll
                               for (int i = 0; i < QW; ++i) o[i][c] = mma1(f, pf[i][m], o[i][c]);
                             });
    feed<T, 2, QW, DV / 16 * NPF>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };
  for (int it = 0; it < tiles.count; ++it) {
    const int j0 = tiles.tile(it), jn = tiles.tile(min(it + 1, tiles.count - 1));
    fk.fetch(k, p.d, jn, len);  // after the last tile: that tile again, not used
    fv.fetch(v, p.dv, jn, len);
    if (j0 <= qz && (j0 + WIN_KEYS > qa - p.window + 1 || j0 < p.sinks)) {
      const bool whole = j0 + WIN_KEYS - 1 <= qa && (qz - j0 < p.window || j0 + WIN_KEYS <= p.sinks);
      pass(!whole, sK[it & 1], sV[it & 1], j0, lane);
    }
    fk.put(sK[(it + 1) & 1], tid);
    fv.put(sV[(it + 1) & 1], tid);
    __syncthreads();
  }
  T *out = (T *)p.out + (long)bh * p.n * p.dv;
#pragma unroll
  for (int i = 0; i < QW; ++i) {
    const int t = qa + 16 * i + col;
    const float l = add_groups(sum[i]), inv = 1.f / l;
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) st_out(out, p.dv, t, 16 * c + 4 * g, len, o[i][c] * inv);
    if (p.lse && g == 0 && t < len)
      p.lse[(long)bh * p.n + t] = (ref[i] + log2f(l)) * 0.693147180559945309f;
  }
}

// One 16-byte vector a thread, over the slots of every sequence and key head.
__global__ void __launch_bounds__(256) window_cache_kernel(WindowCacheArgs p) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const int per = p.vk + p.vv;
  const long slot_row = i / per;
  const int c = (int)(i % per), slots = p.window + p.sinks;
  if (slot_row >= (long)p.B * p.Hkv * slots) return;
  const int slot = (int)(slot_row % slots);
  const long bk = slot_row / slots;
  const int len = win_len(p.lens, (int)(bk / p.Hkv), p.n);
  if (slot >= len) return;
  const int token = slot < p.sinks ? slot : slot + (len - 1 - slot) / p.window * p.window;
  if (c < p.vk)
    ((u32x4 *)p.cache_k)[slot_row * p.vk + c] = ((const u32x4 *)p.k)[(bk * p.n + token) * p.vk + c];
  else
    ((u32x4 *)p.cache_v)[slot_row * p.vv + c - p.vk] = ((const u32x4 *)p.v)[(bk * p.n + token) * p.vv + c - p.vk];
}

template <typename T, int DK, int DV, int QW> hipError_t run_forward(const WindowArgs &a, hipStream_t s) {
  const int total = a.B * a.H * ((a.n + 64 * QW - 1) / (64 * QW));
  hipLaunchKernelGGL((window_forward_kernel<T, DK, DV, QW>), dim3(xcd_grid(total)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Fewer than a workgroup to a compute unit with 128 rows to a workgroup: 64, which ends sooner (8 heads
// x 333 tokens, d = dv = 64: 12.6 -> 8.6 us).
template <int DK, int DV> hipError_t by_rows(const WindowArgs &a, hipStream_t s) {
  return few_rows(a.B * a.H, a.n) ? run_forward<bf16, DK, DV, 1>(a, s) : run_forward<bf16, DK, DV, 2>(a, s);
}

}  // namespace

hipError_t launch_window_forward(int dtype, const WindowArgs &a, hipStream_t s) {
  if (dtype == 0) return run_forward<float, 64, 64, 1>(a, s);
  const bool k64 = a.d <= 64, v64 = a.dv <= 64;
  if (k64 && v64) return by_rows<64, 64>(a, s);
  if (k64) return by_rows<64, 128>(a, s);
  if (v64) return by_rows<128, 64>(a, s);
  return by_rows<128, 128>(a, s);
}

hipError_t launch_window_cache(const WindowCacheArgs &a, hipStream_t s) {
  const long n = (long)a.B * a.Hkv * (a.window + a.sinks) * (a.vk + a.vv);
  hipLaunchKernelGGL(window_cache_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace hla2
