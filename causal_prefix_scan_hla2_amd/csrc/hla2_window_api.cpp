// hla2_window_api.cpp -- the C ABI of windowed attention: argument checks on the host, before any HIP
// call, workspace layout and the launches.
#include <math.h>
#include <stdint.h>

#include "hla2.h"
#include "hla2_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int check_kind(int B, int H, int Hkv, int d, int dv, int window, int sinks, int dtype) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || d <= 0 || dv <= 0 || window <= 0 || sinks < 0) return HLA2_ERR_INVALID;
  if (dtype != HLA2_F32 && dtype != HLA2_BF16) return HLA2_ERR_INVALID;
  if (H % Hkv) return HLA2_ERR_INVALID;
  const int top = dtype == HLA2_F32 ? 64 : 128;
  if (d % 16 || dv % 16 || d > top || dv > top || sinks > HLA2_WINDOW_MAX_SINKS) return HLA2_ERR_UNSUPPORTED;
  if ((long)B * H > (1L << 24)) return HLA2_ERR_UNSUPPORTED;
  return HLA2_OK;
}

int check_shape(int B, int H, int Hkv, int n, int d, int dv, int window, int sinks, int dtype) {
  if (n <= 0) return HLA2_ERR_INVALID;
  const int rc = check_kind(B, H, Hkv, d, dv, window, sinks, dtype);
  if (rc != HLA2_OK) return rc;
  if ((long)n > (1L << 30) || (long)B * H * n > (1L << 40)) return HLA2_ERR_UNSUPPORTED;
  // one head's rows are addressed with 32-bit byte offsets
  if ((long)n * ((d > dv ? d : dv) + 16) * 4 > 0x7fffff00L) return HLA2_ERR_UNSUPPORTED;
  // launches of 256 threads to 64 rows of a head stay below 2^32 work-items
  if (((long)B * H * (((long)n + 63) / 64) + 8) * 256 > 0xFFFFFFFFL) return HLA2_ERR_UNSUPPORTED;
  return HLA2_OK;
}

constexpr float kLog2e = 1.44269504088896340736f;
bool good_scale(float s) { return s > 0.0f && isfinite(s * kLog2e); }

// workspace of the backward pass: dout . out, the sinks' far sums, the query heads' own sums
struct BwdSpace {
  size_t far, parts, total;  // offsets
  bool apart;
};
BwdSpace backward_space(int B, int H, int Hkv, int n, int d, int dv, int window, int sinks, int dt) {
  BwdSpace w;
  w.far = align256((size_t)B * H * n * 4);
  w.apart = hla2::window_heads_apart(B, H, Hkv, n);
  const size_t runs = hla2::window_far_runs((long)B * H, n, window, sinks);
  w.parts = w.far + align256(((size_t)B * H * runs + (runs && !w.apart ? (size_t)B * Hkv : 0)) *
                             hla2::window_far_bytes(dt, d, dv, sinks));
  w.total = w.parts + (w.apart ? (size_t)B * H * n * (d + dv) * 4 : 0);
  return w;
}

int check_backward(int B, int H, int Hkv, int n, int d, int dv, int window, int sinks, int dtype) {
  const int rc = check_shape(B, H, Hkv, n, d, dv, window, sinks, dtype);
  if (rc != HLA2_OK) return rc;
  const long runs = hla2::window_far_runs((long)B * H, n, window, sinks);
  // the launch that adds the far runs up: up to four workgroups' worth of 16 for each key head
  if (runs > 0 && (long)B * Hkv * 64 * 256 > 0xFFFFFFFFL) return HLA2_ERR_UNSUPPORTED;
  // the keys' walk and the far runs in one launch
  if (((long)B * H * (((long)n + 63) / 64 + runs) + 16) * 256 > 0xFFFFFFFFL) return HLA2_ERR_UNSUPPORTED;
  return HLA2_OK;
}

// window + sinks slots of one head, addressed with 32-bit offsets
int check_slots(int N, int Hkv, int d, int dv, int window, int sinks) {
  const long slots = (long)window + sinks;
  if (slots >= (1L << 24) || slots * (d > dv ? d : dv) * 4 > 0x7fffff00L) return HLA2_ERR_UNSUPPORTED;
  return (long)N * Hkv * 64 < (1L << 24) ? HLA2_OK : HLA2_ERR_UNSUPPORTED;
}
int check_step(int N, int H, int Hkv, int d, int dv, int window, int sinks, int dtype) {
  int rc = check_kind(N, H, Hkv, d, dv, window, sinks, dtype);
  if (rc == HLA2_OK) rc = check_slots(N, Hkv, d, dv, window, sinks);
  if (rc != HLA2_OK) return rc;
  return H / Hkv <= 16 ? HLA2_OK : HLA2_ERR_UNSUPPORTED;
}
size_t step_bytes(int N, int Hkv, int dv, int window, int sinks) {
  const int splits = hla2::window_step_splits((long)N * Hkv, window + sinks);
  return splits > 1 ? (size_t)N * Hkv * splits * hla2::window_step_part_floats(dv) * 4 : 0;
}

}  // namespace

extern "C" {

int hla2_window_forward(const void *q, const void *k, const void *v, void *out, float *lse, const int *lens, int B,
                        int H, int Hkv, int n, int d, int dv, int window, int sinks, float scale, hla2_dtype_t dtype,
                        hipStream_t stream) {
  if (!q || !k || !v || !out || !good_scale(scale)) return HLA2_ERR_INVALID;
  const int rc = check_shape(B, H, Hkv, n, d, dv, window, sinks, (int)dtype);
  if (rc != HLA2_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)) return HLA2_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(lens, 4)) return HLA2_ERR_INVALID;
  hla2::WindowArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.lens = lens;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.n = n;
  a.d = d;
  a.dv = dv;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  a.scale2 = scale * kLog2e;
  const hipError_t e = hla2::launch_window_forward(dtype == HLA2_F32 ? 0 : 1, a, stream);
  return e == hipSuccess ? HLA2_OK : HLA2_ERR_LAUNCH;
}

size_t hla2_window_backward_workspace_bytes(int B, int H, int Hkv, int n, int d, int dv, int window, int sinks,
                                            hla2_dtype_t dtype) {
  if (check_backward(B, H, Hkv, n, d, dv, window, sinks, (int)dtype) != HLA2_OK) return 0;
  return backward_space(B, H, Hkv, n, d, dv, window, sinks, (int)dtype == HLA2_F32 ? 0 : 1).total;
}

int hla2_window_backward(const void *q, const void *k, const void *v, const void *out, const float *lse,
                         const void *dout, void *dq, void *dk, void *dv_out, const int *lens, int B, int H, int Hkv,
                         int n, int d, int dv, int window, int sinks, float scale, hla2_dtype_t dtype, void *workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv_out || !good_scale(scale)) return HLA2_ERR_INVALID;
  const int rc = check_backward(B, H, Hkv, n, d, dv, window, sinks, (int)dtype);
  if (rc != HLA2_OK) return rc;
  const void *tens[] = {q, k, v, out, dout, dq, dk, dv_out};
  for (const void *t : tens)
    if (!aligned(t, 16)) return HLA2_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(lens, 4)) return HLA2_ERR_INVALID;
  const int dt = dtype == HLA2_F32 ? 0 : 1;
  const BwdSpace w = backward_space(B, H, Hkv, n, d, dv, window, sinks, dt);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 256)) return HLA2_ERR_WORKSPACE;
  hla2::WindowBwdArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.dout = dout;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv_out = dv_out;
  a.lens = lens;
  a.dot = (float *)workspace;
  a.far = (float *)((char *)workspace + w.far);
  a.parts = w.apart ? (float *)((char *)workspace + w.parts) : nullptr;
  a.runs = hla2::window_far_runs((long)B * H, n, window, sinks);
  a.run = a.runs > 0 ? hla2::window_far_run((long)B * H, n, window) : 0;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.n = n;
  a.d = d;
  a.dv = dv;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  a.scale2 = scale * kLog2e;
  const hipError_t e = hla2::launch_window_backward(dt, a, stream);
  return e == hipSuccess ? HLA2_OK : HLA2_ERR_LAUNCH;
}

int hla2_window_cache(const void *k, const void *v, void *cache_k, void *cache_v, const int *lens, int B, int Hkv,
                      int n, int d, int dv, int window, int sinks, hla2_dtype_t dtype, hipStream_t stream) {
  if (!k || !v || !cache_k || !cache_v) return HLA2_ERR_INVALID;
  int rc = check_shape(B, Hkv, Hkv, n, d, dv, window, sinks, (int)dtype);
  if (rc == HLA2_OK) rc = check_slots(B, Hkv, d, dv, window, sinks);
  if (rc != HLA2_OK) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache_k, 16) || !aligned(cache_v, 16) || !aligned(lens, 4))
    return HLA2_ERR_INVALID;
  const int per16 = dtype == HLA2_F32 ? 4 : 8;
  hla2::WindowCacheArgs a = {k, v, cache_k, cache_v, lens, B, Hkv, n, window, sinks, d / per16, dv / per16};
  if ((long)B * Hkv * ((long)window + sinks) * (a.vk + a.vv) > 0xFFFFFF00L) return HLA2_ERR_UNSUPPORTED;
  const hipError_t e = hla2::launch_window_cache(a, stream);
  return e == hipSuccess ? HLA2_OK : HLA2_ERR_LAUNCH;
}

size_t hla2_window_step_workspace_bytes(int N, int H, int Hkv, int d, int dv, int window, int sinks,
                                        hla2_dtype_t dtype) {
  if (check_step(N, H, Hkv, d, dv, window, sinks, (int)dtype) != HLA2_OK) return 0;
  return step_bytes(N, Hkv, dv, window, sinks);
}

int hla2_window_step(void *cache_k, void *cache_v, const long long *pos, const void *q, const void *k, const void *v,
                     void *out, int N, int H, int Hkv, int d, int dv, int window, int sinks, float scale,
                     hla2_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!cache_k || !cache_v || !pos || !q || !k || !v || !out || !good_scale(scale)) return HLA2_ERR_INVALID;
  const int rc = check_step(N, H, Hkv, d, dv, window, sinks, (int)dtype);
  if (rc != HLA2_OK) return rc;
  const void *tens[] = {cache_k, cache_v, q, k, v, out};
  for (const void *t : tens)
    if (!aligned(t, 16)) return HLA2_ERR_INVALID;
  if (!aligned(pos, 8)) return HLA2_ERR_INVALID;
  const size_t need = step_bytes(N, Hkv, dv, window, sinks);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return HLA2_ERR_WORKSPACE;
  hla2::WindowStepArgs a = {};
  a.cache_k = cache_k;
  a.cache_v = cache_v;
  a.pos = pos;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.parts = need > 0 ? (float *)workspace : nullptr;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.dv = dv;
  a.window = window;
  a.sinks = sinks;
  a.splits = hla2::window_step_splits((long)N * Hkv, window + sinks);
  a.scale2 = scale * kLog2e;
  const hipError_t e = hla2::launch_window_step(dtype == HLA2_F32 ? 0 : 1, a, stream);
  return e == hipSuccess ? HLA2_OK : HLA2_ERR_LAUNCH;
}

}  // extern "C"
