// C ABI of libwbmm: argument validation (host only, before anything is enqueued), the thread-local
// error message, and dispatch to the kernel launchers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "../../include/wbmm.h"
#include "wbmm_adamw.hpp"
#include "wbmm_delta.hpp"
#include "wbmm_launch.hpp"
#include "wbmm_norm.hpp"
#include "wbmm_scan.hpp"

#define WBMM_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local std::string g_err;
thread_local hipEvent_t g_ev_before = nullptr, g_ev_after = nullptr;

wbmm_status fail(wbmm_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

wbmm_status ok() {
  g_err.clear();
  return WBMM_OK;
}

wbmm_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(WBMM_E_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

constexpr int kMaxW = 32;
constexpr long long kMaxDim = 1 << 20;
constexpr long long kMaxElems = 1ll << 38;

bool valid_dtype(int dt) { return dt == WBMM_F32 || dt == WBMM_BF16; }
bool valid_layout(int l) { return l == WBMM_NCHW || l == WBMM_NHWC; }
size_t dtype_size(int dt) { return dt == WBMM_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Byte ranges [p, p + n) and [q, q + m) intersect.
bool overlaps(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + m && b < a + n;
}

wbmm_status check_map(int B, int C, int H, int W, int w, int layout) {
  if (w < 1 || w > kMaxW) return fail(WBMM_E_INVALID, "window size w=%d outside [1, %d]", w, kMaxW);
  if (B < 1 || C < 1 || H < 1 || W < 1)
    return fail(WBMM_E_INVALID, "sizes must be >= 1 (B=%d C=%d H=%d W=%d)", B, C, H, W);
  if (C > 65535) return fail(WBMM_E_UNSUPPORTED, "C=%d exceeds 65535", C);
  if (B > kMaxDim || H > kMaxDim || W > kMaxDim)
    return fail(WBMM_E_UNSUPPORTED, "a dimension exceeds 2^20");
  const long long Hp = (H + w - 1) / w * (long long)w, Wp = (W + w - 1) / w * (long long)w;
  if ((long long)B * C * Hp * Wp > kMaxElems) return fail(WBMM_E_UNSUPPORTED, "map too large");
  if ((long long)B * (Hp / w) * (Wp / w) >= (1ll << 31))
    return fail(WBMM_E_UNSUPPORTED, "too many windows per channel");
  if (!valid_layout(layout)) return fail(WBMM_E_INVALID, "unknown layout %d", layout);
  return WBMM_OK;
}

}  // namespace

namespace wbmm {
void take_main_events(hipEvent_t* before, hipEvent_t* after) {
  *before = g_ev_before;
  *after = g_ev_after;
  g_ev_before = g_ev_after = nullptr;  // one call only
}
}  // namespace wbmm

WBMM_API int wbmm_abi_version(void) { return WBMM_ABI_VERSION; }

WBMM_API wbmm_status wbmm_set_launch_events(void* before, void* after) {
  if ((before == nullptr) != (after == nullptr))
    return fail(WBMM_E_INVALID, "give both events or neither");
  g_ev_before = (hipEvent_t)before;
  g_ev_after = (hipEvent_t)after;
  return ok();
}

WBMM_API const char* wbmm_last_error(void) { return g_err.c_str(); }

WBMM_API wbmm_status wbmm_build_index(int w, int32_t* idx, void* stream) {
  if (w < 1 || w > kMaxW) return fail(WBMM_E_INVALID, "window size w=%d outside [1, %d]", w, kMaxW);
  if (!idx) return fail(WBMM_E_INVALID, "idx is NULL");
  if (!aligned(idx, 4)) return fail(WBMM_E_UNSUPPORTED, "idx not 4-byte aligned");
  return hip_status(wbmm::launch_build_index(w, idx, (hipStream_t)stream), "wbmm_build_index");
}

WBMM_API wbmm_status wbmm_build_matrix(const void* T, int C, int w, int dtype, void* M,
                                       void* stream) {
  if (w < 1 || w > kMaxW) return fail(WBMM_E_INVALID, "window size w=%d outside [1, %d]", w, kMaxW);
  if (C < 1) return fail(WBMM_E_INVALID, "C=%d must be >= 1", C);
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (!T || !M) return fail(WBMM_E_INVALID, "T and M must be non-NULL");
  const size_t es = dtype_size(dtype);
  if (!aligned(T, es) || !aligned(M, es)) return fail(WBMM_E_UNSUPPORTED, "misaligned pointer");
  const size_t L = (size_t)(2 * w - 1) * (2 * w - 1), d = (size_t)w * w;
  if (overlaps(T, (size_t)C * L * es, M, (size_t)C * d * d * es))
    return fail(WBMM_E_INVALID, "M overlaps T");
  return hip_status(wbmm::launch_build_matrix(T, C, w, dtype == WBMM_BF16, M, (hipStream_t)stream),
                    "wbmm_build_matrix");
}

WBMM_API wbmm_status wbmm_fold_hier(const void* M_in, const void* T_sub, int C, int w, int s,
                                    int dtype, void* M_out, void* stream) {
  if (w < 1 || w > kMaxW) return fail(WBMM_E_INVALID, "window size w=%d outside [1, %d]", w, kMaxW);
  if (C < 1) return fail(WBMM_E_INVALID, "C=%d must be >= 1", C);
  if (s < 1 || s >= w || w % s != 0)
    return fail(WBMM_E_INVALID, "sub-window s=%d must divide w=%d with 1 <= s < w", s, w);
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (!M_in || !T_sub || !M_out) return fail(WBMM_E_INVALID, "NULL pointer");
  const size_t es = dtype_size(dtype);
  if (!aligned(M_in, es) || !aligned(T_sub, es) || !aligned(M_out, es))
    return fail(WBMM_E_UNSUPPORTED, "misaligned pointer");
  const size_t mbytes = (size_t)C * w * w * w * w * es;
  if (M_in != M_out && overlaps(M_in, mbytes, M_out, mbytes))
    return fail(WBMM_E_INVALID, "M_out partially overlaps M_in");
  const size_t tbytes = (size_t)C * (2 * s - 1) * (2 * s - 1) * es;
  if (overlaps(T_sub, tbytes, M_out, mbytes)) return fail(WBMM_E_INVALID, "M_out overlaps T_sub");
  return hip_status(
      wbmm::launch_fold(M_in, T_sub, C, w, s, dtype == WBMM_BF16, M_out, (hipStream_t)stream),
      "wbmm_fold_hier");
}

namespace {

wbmm_status check_forward(const wbmm::FwdRequest& r, int in_dtype, int out_dtype) {
  wbmm_status st = check_map(r.B, r.C, r.H, r.W, r.w, r.layout);
  if (st != WBMM_OK) return st;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(WBMM_E_INVALID, "unknown dtype (in %d, out %d)", in_dtype, out_dtype);
  if (!r.x || !r.y) return fail(WBMM_E_INVALID, "x and y must be non-NULL");
  if ((r.T == nullptr) == (r.M == nullptr))
    return fail(WBMM_E_INVALID, "exactly one of T (table) and M (cached matrix) must be given");
  const size_t ies = dtype_size(in_dtype), oes = dtype_size(out_dtype);
  if (!aligned(r.x, ies) || (r.T && !aligned(r.T, ies)) || (r.M && !aligned(r.M, ies)) ||
      !aligned(r.y, oes) || (r.zsave && !aligned(r.zsave, oes)) || (r.mixw && !aligned(r.mixw, 4)))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t elems = (size_t)r.B * r.C * r.H * r.W;
  const size_t d = (size_t)r.w * r.w, L = (size_t)(2 * r.w - 1) * (2 * r.w - 1);
  const size_t ybytes = elems * oes;
  if (overlaps(r.y, ybytes, r.x, elems * ies)) return fail(WBMM_E_INVALID, "y overlaps x");
  if (overlaps(r.y, ybytes, r.T, (size_t)r.C * L * ies)) return fail(WBMM_E_INVALID, "y overlaps T");
  if (overlaps(r.y, ybytes, r.M, (size_t)r.C * d * d * ies))
    return fail(WBMM_E_INVALID, "y overlaps M");
  if (overlaps(r.y, ybytes, r.mixw, (size_t)r.C * 9 * 4))
    return fail(WBMM_E_INVALID, "y overlaps mix_w");
  if (overlaps(r.y, ybytes, r.zsave, ybytes)) return fail(WBMM_E_INVALID, "y overlaps z_save");
  if (r.zsave && overlaps(r.zsave, ybytes, r.x, elems * ies))
    return fail(WBMM_E_INVALID, "z_save overlaps x");
  if (!wbmm::forward_plan_ok(r))
    return fail(WBMM_E_UNSUPPORTED, "no launch shape fits this problem (w=%d)", r.w);
  return WBMM_OK;
}

wbmm::FwdRequest make_fwd(int B, int C, int H, int W, int w, int layout, int in_dtype,
                          int out_dtype, const void* x, const void* T, const void* M,
                          const float* mix_w, void* z_save, void* y, void* ws, size_t ws_bytes) {
  wbmm::FwdRequest r{};
  r.B = B; r.C = C; r.H = H; r.W = W; r.w = w; r.layout = layout;
  r.in_bf16 = in_dtype == WBMM_BF16;
  r.out_bf16 = out_dtype == WBMM_BF16;
  r.x = x; r.T = T; r.M = M; r.mixw = mix_w; r.zsave = z_save; r.y = y;
  r.ws = ws; r.ws_bytes = ws_bytes;
  return r;
}

}  // namespace

namespace {

bool offsets_ok(int w, int oy, int ox) { return oy >= 0 && ox >= 0 && oy < w && ox < w; }

size_t forward_ws_bytes(int B, int C, int H, int W, int w, int oy, int ox, int layout, int has_mix,
                        int has_z_save) {
  if (check_map(B, C, H + oy, W + ox, w, layout) != WBMM_OK || !offsets_ok(w, oy, ox)) return 0;
  static const float dummy = 0.f;
  wbmm::FwdRequest r = make_fwd(B, C, H, W, w, layout, WBMM_F32, WBMM_F32, &dummy, &dummy, nullptr,
                                has_mix ? &dummy : nullptr, has_z_save ? (void*)&dummy : nullptr,
                                (void*)&dummy, nullptr, 0);
  r.oy = oy;
  r.ox = ox;
  if (!wbmm::forward_plan_ok(r)) return 0;
  // the dtypes and the operand kind are not arguments: the largest need over fp32 / bf16 inputs
  // and outputs, with a table or a cached matrix
  size_t need = 0;
  for (int cached = 0; cached < 2; ++cached)
    for (int ib = 0; ib < 2; ++ib)
      for (int ob = 0; ob < 2; ++ob) {
        r.T = cached ? nullptr : (const void*)&dummy;
        r.M = cached ? (const void*)&dummy : nullptr;
        r.in_bf16 = ib;
        r.out_bf16 = ob;
        if (cached && !wbmm::forward_plan_ok(r)) continue;
        const size_t n = wbmm::forward_workspace(r);
        if (n > need) need = n;
      }
  return need;
}

wbmm_status forward_call(int B, int C, int H, int W, int w, int oy, int ox, int layout,
                         int in_dtype, int out_dtype, const void* x, const void* T, const void* M,
                         const float* mix_w, void* z_save, void* y, void* workspace,
                         size_t workspace_bytes, void* stream, const char* name) {
  if (!offsets_ok(w, oy, ox))
    return fail(WBMM_E_INVALID, "grid offset (%d, %d) outside [0, w=%d)", oy, ox, w);
  const wbmm_status sm = check_map(B, C, H + oy, W + ox, w, layout);
  if (sm != WBMM_OK) return sm;
  wbmm::FwdRequest r = make_fwd(B, C, H, W, w, layout, in_dtype, out_dtype, x, T, M, mix_w, z_save,
                                y, workspace, workspace_bytes);
  r.oy = oy;
  r.ox = ox;
  wbmm_status st = check_forward(r, in_dtype, out_dtype);
  if (st != WBMM_OK) return st;
  const size_t need = wbmm::forward_workspace(r);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 16-byte aligned");
  return hip_status(wbmm::launch_forward(r, (hipStream_t)stream), name);
}

}  // namespace

WBMM_API size_t wbmm_forward_workspace_bytes(int B, int C, int H, int W, int w, int layout,
                                             int has_mix, int has_z_save) {
  return forward_ws_bytes(B, C, H, W, w, 0, 0, layout, has_mix, has_z_save);
}

WBMM_API wbmm_status wbmm_forward(int B, int C, int H, int W, int w, int layout, int in_dtype,
                                  int out_dtype, const void* x, const void* T, const void* M,
                                  const float* mix_w, void* z_save, void* y, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return forward_call(B, C, H, W, w, 0, 0, layout, in_dtype, out_dtype, x, T, M, mix_w, z_save, y,
                      workspace, workspace_bytes, stream, "wbmm_forward");
}

WBMM_API size_t wbmm_forward_shifted_workspace_bytes(int B, int C, int H, int W, int w, int oy,
                                                     int ox, int layout, int has_mix,
                                                     int has_z_save) {
  return forward_ws_bytes(B, C, H, W, w, oy, ox, layout, has_mix, has_z_save);
}

WBMM_API wbmm_status wbmm_forward_shifted(int B, int C, int H, int W, int w, int oy, int ox,
                                          int layout, int in_dtype, int out_dtype, const void* x,
                                          const void* T, const void* M, const float* mix_w,
                                          void* z_save, void* y, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return forward_call(B, C, H, W, w, oy, ox, layout, in_dtype, out_dtype, x, T, M, mix_w, z_save,
                      y, workspace, workspace_bytes, stream, "wbmm_forward_shifted");
}

namespace {

wbmm::BwdRequest make_bwd(int B, int C, int H, int W, int w, int layout, const float* x,
                          const float* T, const float* M, const float* mix_w, const float* z_saved,
                          const float* dy, float* dx, float* dT, float* dmix_w, void* ws,
                          size_t ws_bytes) {
  wbmm::BwdRequest r{};
  r.B = B; r.C = C; r.H = H; r.W = W; r.w = w; r.layout = layout;
  r.x = x; r.T = T; r.M = M; r.mixw = mix_w; r.zsaved = z_saved; r.dy = dy;
  r.dx = dx; r.dT = dT; r.dmixw = mix_w ? dmix_w : nullptr;
  r.ws = ws; r.ws_bytes = ws_bytes;
  return r;
}

}  // namespace

namespace {

size_t backward_ws_bytes(int B, int C, int H, int W, int w, int oy, int ox, int layout,
                         int has_mix) {
  if (check_map(B, C, H + oy, W + ox, w, layout) != WBMM_OK || !offsets_ok(w, oy, ox)) return 0;
  static const float dummy = 0.f;
  wbmm::BwdRequest r = make_bwd(B, C, H, W, w, layout, &dummy, &dummy, nullptr,
                                has_mix ? &dummy : nullptr, has_mix ? &dummy : nullptr, &dummy,
                                nullptr, nullptr, nullptr, nullptr, 0);
  r.oy = oy;
  r.ox = ox;
  if (!wbmm::backward_plan_ok(r)) return 0;
  // the operand kind is not an argument: the larger need of a table and a cached matrix
  size_t need = wbmm::backward_workspace(r);
  r.T = nullptr;
  r.M = &dummy;
  if (wbmm::backward_plan_ok(r)) {
    const size_t n = wbmm::backward_workspace(r);
    if (n > need) need = n;
  }
  return need;
}

}  // namespace

// Scratch of the allocation-free backward: one copy per GPU, in the library's code object, held
// until the process ends. Host code never passes `scratch` itself to a kernel (on the host it is
// only a stand-in for the symbol); it asks for the device address once per device.
static __device__ __align__(256) unsigned char scratch[WBMM_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr size_t kScratchBytes = WBMM_NOALLOC_SCRATCH_BYTES;
std::mutex g_scratch_mu;
void* g_scratch_dev[64];  // device address of `scratch` per device id, once looked up

// The current device's copy of `scratch` (looked up on first use with that device current).
wbmm_status scratch_ptr(void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e, "hipGetDevice");
  if (dev < 0 || dev >= 64) return fail(WBMM_E_UNSUPPORTED, "device id %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_scratch_mu);
  if (!g_scratch_dev[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_status(e, "hipGetSymbolAddress(scratch)");
    if (!p) return fail(WBMM_E_HIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_dev[dev] = p;
  }
  *out = g_scratch_dev[dev];
  return WBMM_OK;
}

// no_alloc: the workspace is the current device's `scratch` (workspace arguments ignored).
wbmm_status backward_call(int B, int C, int H, int W, int w, int oy, int ox, int layout,
                          const float* x, const float* T, const float* M, const float* mix_w,
                          const float* z_saved, const float* dy, float* dx, float* dT,
                          float* dmix_w, void* workspace, size_t workspace_bytes, void* stream,
                          const char* name, bool no_alloc = false) {
  if (!offsets_ok(w, oy, ox))
    return fail(WBMM_E_INVALID, "grid offset (%d, %d) outside [0, w=%d)", oy, ox, w);
  wbmm_status st = check_map(B, C, H + oy, W + ox, w, layout);
  if (st != WBMM_OK) return st;
  if (!x || !dy) return fail(WBMM_E_INVALID, "x and dy must be non-NULL");
  if ((T == nullptr) == (M == nullptr))
    return fail(WBMM_E_INVALID, "exactly one of T (table) and M (cached matrix) must be given");
  if ((mix_w == nullptr) != (z_saved == nullptr))
    return fail(WBMM_E_INVALID, "z_saved is required exactly when mix_w is given");
  const void* ptrs[] = {x, T, M, mix_w, z_saved, dy, dx, dT, dmix_w};
  for (const void* p : ptrs)
    if (p && !aligned(p, 4)) return fail(WBMM_E_UNSUPPORTED, "pointer not 4-byte aligned");
  const size_t mb = (size_t)B * C * H * W * 4;
  const size_t tb = (size_t)C * (2 * w - 1) * (2 * w - 1) * 4;
  if (dx && (overlaps(dx, mb, x, mb) || overlaps(dx, mb, dy, mb) || overlaps(dx, mb, z_saved, mb)))
    return fail(WBMM_E_INVALID, "dx overlaps an input");
  if (dT && (overlaps(dT, tb, T, tb) || overlaps(dT, tb, dx, mb)))
    return fail(WBMM_E_INVALID, "dT overlaps T or dx");
  wbmm::BwdRequest r = make_bwd(B, C, H, W, w, layout, x, T, M, mix_w, z_saved, dy, dx, dT, dmix_w,
                                workspace, workspace_bytes);
  r.oy = oy;
  r.ox = ox;
  if (!wbmm::backward_plan_ok(r))
    return fail(WBMM_E_UNSUPPORTED, "no launch shape fits this problem (w=%d)", w);
  const size_t need = wbmm::backward_workspace(r);
  if (no_alloc) {
    if (need > kScratchBytes)
      return fail(WBMM_E_UNSUPPORTED,
                  "this problem needs %zu bytes of scratch; the allocation-free backward holds "
                  "%zu (use wbmm_backward with a workspace)", need, kScratchBytes);
    const wbmm_status sp = scratch_ptr(&r.ws);
    if (sp != WBMM_OK) return sp;
    r.ws_bytes = kScratchBytes;
    return hip_status(wbmm::launch_backward(r, (hipStream_t)stream), name);
  }
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 256))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 256-byte aligned");
  return hip_status(wbmm::launch_backward(r, (hipStream_t)stream), name);
}

}  // namespace

WBMM_API size_t wbmm_backward_workspace_bytes(int B, int C, int H, int W, int w, int layout,
                                              int has_mix) {
  return backward_ws_bytes(B, C, H, W, w, 0, 0, layout, has_mix);
}

WBMM_API wbmm_status wbmm_backward(int B, int C, int H, int W, int w, int layout, const float* x,
                                   const float* T, const float* M, const float* mix_w,
                                   const float* z_saved, const float* dy, float* dx, float* dT,
                                   float* dmix_w, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return backward_call(B, C, H, W, w, 0, 0, layout, x, T, M, mix_w, z_saved, dy, dx, dT, dmix_w,
                       workspace, workspace_bytes, stream, "wbmm_backward");
}

WBMM_API wbmm_status wbmm_backward_noalloc(int B, int C, int H, int W, int w, int layout,
                                           const float* x, const float* T, const float* M,
                                           const float* mix_w, const float* z_saved,
                                           const float* dy, float* dx, float* dT, float* dmix_w,
                                           void* stream) {
  return backward_call(B, C, H, W, w, 0, 0, layout, x, T, M, mix_w, z_saved, dy, dx, dT, dmix_w,
                       nullptr, 0, stream, "wbmm_backward_noalloc", true);
}

WBMM_API size_t wbmm_backward_shifted_workspace_bytes(int B, int C, int H, int W, int w, int oy,
                                                      int ox, int layout, int has_mix) {
  return backward_ws_bytes(B, C, H, W, w, oy, ox, layout, has_mix);
}

WBMM_API wbmm_status wbmm_backward_shifted(int B, int C, int H, int W, int w, int oy, int ox,
                                           int layout, const float* x, const float* T,
                                           const float* M, const float* mix_w,
                                           const float* z_saved, const float* dy, float* dx,
                                           float* dT, float* dmix_w, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  return backward_call(B, C, H, W, w, oy, ox, layout, x, T, M, mix_w, z_saved, dy, dx, dT, dmix_w,
                       workspace, workspace_bytes, stream, "wbmm_backward_shifted");
}
namespace {
// Shared checks of the hierarchical entry points: fp32 tables, s x s sub-windows tiling the
// w x w window (s divides w, s < w).
bool hier_sizes_ok(int w, int s) { return s >= 1 && s < w && w % s == 0; }
wbmm_status check_hier(int w, int s, const float* T, const float* T_sub) {
  if (!hier_sizes_ok(w, s))
    return fail(WBMM_E_INVALID, "the sub-window side must divide the window side and be smaller "
                "(w=%d, s=%d)", w, s);
  if (!T || !T_sub) return fail(WBMM_E_INVALID, "T and T_sub must be non-NULL");
  if (!aligned(T, 4) || !aligned(T_sub, 4)) return fail(WBMM_E_UNSUPPORTED, "misaligned pointer");
  return WBMM_OK;
}
}  // namespace
WBMM_API size_t wbmm_forward_hier_workspace_bytes(int B, int C, int H, int W, int w, int s,
                                                  int layout, int has_mix, int has_z_save) {
  if (check_map(B, C, H, W, w, layout) != WBMM_OK || !hier_sizes_ok(w, s)) return 0;
  static const float dummy = 0.f;
  wbmm::FwdRequest r = make_fwd(B, C, H, W, w, layout, WBMM_F32, WBMM_F32, &dummy, &dummy, nullptr,
                                has_mix ? &dummy : nullptr, has_z_save ? (void*)&dummy : nullptr,
                                (void*)&dummy, nullptr, 0);
  r.Tsub = &dummy;
  r.s = s;
  if (!wbmm::forward_plan_ok(r)) return 0;
  return wbmm::forward_workspace(r);
}
WBMM_API wbmm_status wbmm_forward_hier(int B, int C, int H, int W, int w, int s, int layout,
                                       const float* x, const float* T, const float* T_sub,
                                       const float* mix_w, float* z_save, float* y,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  wbmm_status st = check_map(B, C, H, W, w, layout);
  if (st != WBMM_OK) return st;
  st = check_hier(w, s, T, T_sub);
  if (st != WBMM_OK) return st;
  wbmm::FwdRequest r = make_fwd(B, C, H, W, w, layout, WBMM_F32, WBMM_F32, x, T, nullptr, mix_w,
                                z_save, y, workspace, workspace_bytes);
  r.Tsub = T_sub;
  r.s = s;
  st = check_forward(r, WBMM_F32, WBMM_F32);
  if (st != WBMM_OK) return st;
  const size_t elems = (size_t)B * C * H * W;
  if (overlaps(y, elems * 4, T_sub, (size_t)C * (2 * s - 1) * (2 * s - 1) * 4))
    return fail(WBMM_E_INVALID, "y overlaps T_sub");
  const size_t need = wbmm::forward_workspace(r);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 16-byte aligned");
  return hip_status(wbmm::launch_forward(r, (hipStream_t)stream), "wbmm_forward_hier");
}
WBMM_API size_t wbmm_backward_hier_workspace_bytes(int B, int C, int H, int W, int w, int s,
                                                   int layout, int has_mix) {
  if (check_map(B, C, H, W, w, layout) != WBMM_OK || !hier_sizes_ok(w, s)) return 0;
  static const float dummy = 0.f;
  wbmm::BwdRequest r = make_bwd(B, C, H, W, w, layout, &dummy, &dummy, nullptr,
                                has_mix ? &dummy : nullptr, has_mix ? &dummy : nullptr, &dummy,
                                nullptr, nullptr, nullptr, nullptr, 0);
  r.Tsub = &dummy;
  r.s = s;
  if (!wbmm::backward_plan_ok(r)) return 0;
  return wbmm::backward_workspace(r);
}
WBMM_API wbmm_status wbmm_backward_hier(int B, int C, int H, int W, int w, int s, int layout,
                                        const float* x, const float* T, const float* T_sub,
                                        const float* mix_w, const float* z_saved, const float* dy,
                                        float* dx, float* dT, float* dT_sub, float* dmix_w,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  wbmm_status st = check_map(B, C, H, W, w, layout);
  if (st != WBMM_OK) return st;
  st = check_hier(w, s, T, T_sub);
  if (st != WBMM_OK) return st;
  if (!x || !dy) return fail(WBMM_E_INVALID, "x and dy must be non-NULL");
  if ((mix_w == nullptr) != (z_saved == nullptr))
    return fail(WBMM_E_INVALID, "z_saved is required exactly when mix_w is given");
  const void* ptrs[] = {x, mix_w, z_saved, dy, dx, dT, dT_sub, dmix_w};
  for (const void* p : ptrs)
    if (p && !aligned(p, 4)) return fail(WBMM_E_UNSUPPORTED, "pointer not 4-byte aligned");
  const size_t mb = (size_t)B * C * H * W * 4;
  const size_t tb = (size_t)C * (2 * w - 1) * (2 * w - 1) * 4;
  const size_t sb = (size_t)C * (2 * s - 1) * (2 * s - 1) * 4;
  if (dx && (overlaps(dx, mb, x, mb) || overlaps(dx, mb, dy, mb) || overlaps(dx, mb, z_saved, mb)))
    return fail(WBMM_E_INVALID, "dx overlaps an input");
  if (dT && (overlaps(dT, tb, T, tb) || overlaps(dT, tb, T_sub, sb) || overlaps(dT, tb, dx, mb)))
    return fail(WBMM_E_INVALID, "dT overlaps T, T_sub or dx");
  if (dT_sub && (overlaps(dT_sub, sb, T, tb) || overlaps(dT_sub, sb, T_sub, sb) ||
                 overlaps(dT_sub, sb, dx, mb) || overlaps(dT_sub, sb, dT, tb)))
    return fail(WBMM_E_INVALID, "dT_sub overlaps T, T_sub, dx or dT");
  wbmm::BwdRequest r = make_bwd(B, C, H, W, w, layout, x, T, nullptr, mix_w, z_saved, dy, dx, dT,
                                dmix_w, workspace, workspace_bytes);
  r.Tsub = T_sub;
  r.s = s;
  r.dTsub = dT_sub;
  if (!wbmm::backward_plan_ok(r))
    return fail(WBMM_E_UNSUPPORTED, "no launch shape fits this problem (w=%d)", w);
  const size_t need = wbmm::backward_workspace(r);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 256))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 256-byte aligned");
  return hip_status(wbmm::launch_backward(r, (hipStream_t)stream), "wbmm_backward_hier");
}

WBMM_API wbmm_status wbmm_dwconv_forward(int B, int C, int H, int W, int k, const float* x,
                                         const float* w_dw, float* y, void* stream) {
  if (B < 1 || C < 1 || H < 1 || W < 1)
    return fail(WBMM_E_INVALID, "sizes must be >= 1 (B=%d C=%d H=%d W=%d)", B, C, H, W);
  if (k < 1 || k % 2 == 0) return fail(WBMM_E_INVALID, "kernel size k=%d must be odd and >= 1", k);
  if (!x || !w_dw || !y) return fail(WBMM_E_INVALID, "x, w_dw and y must be non-NULL");
  if (!aligned(x, 4) || !aligned(w_dw, 4) || !aligned(y, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not 4-byte aligned");
  if (!wbmm::dwconv_supported(B, C, H, W, k))
    return fail(WBMM_E_UNSUPPORTED,
                "the depthwise convolution is provided for odd k in 3..13 and rows up to ~600 "
                "pixels (k=%d, W=%d)", k, W);
  const size_t mb = (size_t)B * C * H * W * 4;
  if (overlaps(y, mb, x, mb)) return fail(WBMM_E_INVALID, "y overlaps x");
  if (overlaps(y, mb, w_dw, (size_t)C * k * k * 4)) return fail(WBMM_E_INVALID, "y overlaps w_dw");
  return hip_status(wbmm::launch_dwconv(B, C, H, W, k, x, w_dw, y, (hipStream_t)stream),
                    "wbmm_dwconv_forward");
}

WBMM_API double wbmm_probe_mfma_flops(int dtype, int blocks, int iters) {
  if (!valid_dtype(dtype) || blocks < 1 || iters < 1) return 0.0;
  return wbmm::probe_mfma_flops(dtype == WBMM_BF16, blocks, iters);
}

WBMM_API wbmm_status wbmm_probe_mfma(int dtype, int blocks, int iters, float* out, void* stream) {
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (blocks < 1 || iters < 1 || blocks > 1 << 20)
    return fail(WBMM_E_INVALID, "blocks=%d and iters=%d must be >= 1 (blocks <= 2^20)", blocks,
                iters);
  if (!out || !aligned(out, 4)) return fail(WBMM_E_INVALID, "out must be a 4-byte aligned pointer");
  return hip_status(wbmm::launch_probe_mfma(dtype == WBMM_BF16, blocks, iters, out,
                                            (hipStream_t)stream),
                    "wbmm_probe_mfma");
}

WBMM_API size_t wbmm_backward_bf16_workspace_bytes(int B, int C, int H, int W, int w, int layout,
                                                   int has_mix) {
  if (check_map(B, C, H, W, w, layout) != WBMM_OK ||
      !wbmm::bf16_backward_plan_ok(B, C, H, W, w, layout))
    return 0;
  return wbmm::bf16_backward_workspace(B, C, H, W, w, layout, has_mix);
}

WBMM_API wbmm_status wbmm_backward_bf16(int B, int C, int H, int W, int w, int layout,
                                        const void* x, const void* T, const float* mix_w,
                                        const void* z_saved, const void* dy, void* dx, float* dT,
                                        float* dmix_w, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  wbmm_status st = check_map(B, C, H, W, w, layout);
  if (st != WBMM_OK) return st;
  if (!wbmm::bf16_backward_plan_ok(B, C, H, W, w, layout))
    return fail(WBMM_E_UNSUPPORTED, "no launch shape fits this problem (w=%d)", w);
  if (!x || !T || !dy) return fail(WBMM_E_INVALID, "x, T and dy must be non-NULL");
  if ((mix_w == nullptr) != (z_saved == nullptr))
    return fail(WBMM_E_INVALID, "z_saved is required exactly when mix_w is given");
  const void* ptrs[] = {x, T, z_saved, dy, dx};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return fail(WBMM_E_UNSUPPORTED, "bf16 maps and T must be 16-byte aligned");
  const void* fptrs[] = {mix_w, dT, dmix_w};
  for (const void* p : fptrs)
    if (p && !aligned(p, 4)) return fail(WBMM_E_UNSUPPORTED, "pointer not 4-byte aligned");
  const size_t mb = (size_t)B * C * H * W * 2;
  const size_t tb = (size_t)C * (2 * w - 1) * (2 * w - 1);
  if (dx && (overlaps(dx, mb, x, mb) || overlaps(dx, mb, dy, mb) || overlaps(dx, mb, z_saved, mb) ||
             overlaps(dx, mb, T, tb * 2)))
    return fail(WBMM_E_INVALID, "dx overlaps an input");
  if (dT && (overlaps(dT, tb * 4, T, tb * 2) || overlaps(dT, tb * 4, dx, mb)))
    return fail(WBMM_E_INVALID, "dT overlaps T or dx");
  if (dmix_w && mix_w && overlaps(dmix_w, (size_t)C * 36, mix_w, (size_t)C * 36))
    return fail(WBMM_E_INVALID, "dmix_w overlaps mix_w");
  const size_t need = wbmm::bf16_backward_workspace(B, C, H, W, w, layout, mix_w != nullptr);
  if (!workspace || workspace_bytes < need)
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256)) return fail(WBMM_E_UNSUPPORTED, "workspace not 256-byte aligned");
  wbmm::BwdBf16Request r{};
  r.B = B; r.C = C; r.H = H; r.W = W; r.w = w; r.layout = layout;
  r.x = (const uint16_t*)x; r.T = (const uint16_t*)T; r.mixw = mix_w;
  r.zsaved = (const uint16_t*)z_saved; r.dy = (const uint16_t*)dy; r.dx = (uint16_t*)dx;
  r.dT = dT; r.dmixw = mix_w ? dmix_w : nullptr; r.ws = workspace;
  return hip_status(wbmm::launch_backward_bf16(r, (hipStream_t)stream), "wbmm_backward_bf16");
}

// ---------------------------------------------------------------------------- 8-bit checkpoints
namespace {

constexpr int64_t kMaxCkpt = 1ll << 35;

bool valid_fmt(int f) { return f == WBMM_CKPT_INT8 || f == WBMM_CKPT_E4M3; }

// A buffer of a call: outputs must not overlap inputs or one another.
struct Span {
  const void* p;
  size_t n;
  const char* name;
};
wbmm_status check_spans(const Span* in, int nin, const Span* out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n))
        return fail(WBMM_E_INVALID, "%s overlaps %s", out[i].name, in[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(WBMM_E_INVALID, "%s overlaps %s", out[i].name, out[j].name);
  }
  return WBMM_OK;
}

wbmm_status check_ckpt(int64_t n, int dtype, int fmt) {
  if (n < 1) return fail(WBMM_E_INVALID, "n=%lld must be >= 1", (long long)n);
  if (n > kMaxCkpt) return fail(WBMM_E_UNSUPPORTED, "n=%lld exceeds 2^35", (long long)n);
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (!valid_fmt(fmt)) return fail(WBMM_E_INVALID, "unknown checkpoint format %d", fmt);
  return WBMM_OK;
}

size_t ckpt_scales(int64_t n) {
  return (size_t)(n + WBMM_CKPT_GROUP - 1) / WBMM_CKPT_GROUP;
}

}  // namespace

WBMM_API wbmm_status wbmm_ckpt_pack(const void* x, int64_t n, int dtype, int fmt, uint8_t* codes,
                                    uint8_t* scales, void* stream) {
  wbmm_status st = check_ckpt(n, dtype, fmt);
  if (st != WBMM_OK) return st;
  if (!x || !codes || !scales) return fail(WBMM_E_INVALID, "x, codes and scales must be non-NULL");
  if (!aligned(x, dtype_size(dtype)))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const Span in[] = {{x, (size_t)n * dtype_size(dtype), "x"}};
  const Span out[] = {{codes, (size_t)n, "codes"}, {scales, ckpt_scales(n), "scales"}};
  st = check_spans(in, 1, out, 2);
  if (st != WBMM_OK) return st;
  return hip_status(wbmm::launch_ckpt_pack(x, (size_t)n, dtype == WBMM_BF16, fmt, codes, scales,
                                           (hipStream_t)stream),
                    "wbmm_ckpt_pack");
}

WBMM_API wbmm_status wbmm_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                      int dtype, int fmt, void* x, void* stream) {
  wbmm_status st = check_ckpt(n, dtype, fmt);
  if (st != WBMM_OK) return st;
  if (!x || !codes || !scales) return fail(WBMM_E_INVALID, "x, codes and scales must be non-NULL");
  if (!aligned(x, dtype_size(dtype)))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const Span in[] = {{codes, (size_t)n, "codes"}, {scales, ckpt_scales(n), "scales"}};
  const Span out[] = {{x, (size_t)n * dtype_size(dtype), "x"}};
  st = check_spans(in, 2, out, 1);
  if (st != WBMM_OK) return st;
  return hip_status(wbmm::launch_ckpt_unpack(codes, scales, (size_t)n, dtype == WBMM_BF16, fmt, x,
                                             (hipStream_t)stream),
                    "wbmm_ckpt_unpack");
}

namespace {

wbmm_status check_bwd_ckpt(const wbmm::BwdCkptRequest& r, int dtype) {
  wbmm_status st = check_map(r.B, r.C, r.H, r.W, r.w, r.layout);
  if (st != WBMM_OK) return st;
  return check_ckpt((int64_t)r.B * r.C * r.H * r.W, dtype, r.fmt);
}

}  // namespace

WBMM_API size_t wbmm_backward_ckpt_workspace_bytes(int B, int C, int H, int W, int w, int layout,
                                                   int dtype, int has_mix) {
  static const float dummy = 0.f;
  wbmm::BwdCkptRequest r{};
  r.B = B; r.C = C; r.H = H; r.W = W; r.w = w; r.layout = layout;
  r.bf16 = dtype == WBMM_BF16;
  r.mixw = has_mix ? &dummy : nullptr;
  if (check_bwd_ckpt(r, dtype) != WBMM_OK || !wbmm::backward_ckpt_plan_ok(r)) return 0;
  // the buffers' addresses are not arguments: the larger need of an aligned and a misaligned call
  const size_t fused = wbmm::backward_ckpt_workspace(r);
  r.xc = (const uint8_t*)1;
  const size_t general = wbmm::backward_ckpt_workspace(r);
  return fused > general ? fused : general;
}

WBMM_API wbmm_status wbmm_backward_ckpt(int B, int C, int H, int W, int w, int layout, int dtype,
                                        int fmt, const uint8_t* x_codes, const uint8_t* x_scales,
                                        const void* T, const float* mix_w, const uint8_t* z_codes,
                                        const uint8_t* z_scales, const void* dy, void* dx,
                                        float* dT, float* dmix_w, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  wbmm::BwdCkptRequest r{};
  r.B = B; r.C = C; r.H = H; r.W = W; r.w = w; r.layout = layout;
  r.bf16 = dtype == WBMM_BF16;
  r.fmt = fmt;
  r.xc = x_codes; r.xs = x_scales; r.T = T; r.mixw = mix_w; r.zc = z_codes; r.zs = z_scales;
  r.dy = dy; r.dx = dx; r.dT = dT; r.dmixw = mix_w ? dmix_w : nullptr;
  r.ws = workspace;
  wbmm_status st = check_bwd_ckpt(r, dtype);
  if (st != WBMM_OK) return st;
  if (!x_codes || !x_scales || !T || !dy)
    return fail(WBMM_E_INVALID, "x_codes, x_scales, T and dy must be non-NULL");
  if ((mix_w == nullptr) != (z_codes == nullptr) || (mix_w == nullptr) != (z_scales == nullptr))
    return fail(WBMM_E_INVALID, "z_codes and z_scales are required exactly when mix_w is given");
  const size_t es = dtype_size(dtype);
  if (!aligned(T, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(mix_w, 4) ||
      !aligned(dT, 4) || !aligned(dmix_w, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t n = (size_t)B * C * H * W, L = (size_t)C * (2 * w - 1) * (2 * w - 1);
  const size_t wb = (size_t)C * 36;
  const Span in[] = {{x_codes, n, "x_codes"}, {x_scales, ckpt_scales((int64_t)n), "x_scales"},
                     {T, L * es, "T"}, {mix_w, wb, "mix_w"}, {z_codes, n, "z_codes"},
                     {z_scales, ckpt_scales((int64_t)n), "z_scales"}, {dy, n * es, "dy"}};
  const Span out[] = {{dx, n * es, "dx"}, {dT, L * 4, "dT"}, {r.dmixw, wb, "dmix_w"}};
  st = check_spans(in, 7, out, 3);
  if (st != WBMM_OK) return st;
  if (!wbmm::backward_ckpt_plan_ok(r))
    return fail(WBMM_E_UNSUPPORTED, "no launch shape fits this problem (w=%d)", w);
  const size_t need = wbmm::backward_ckpt_workspace(r);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 256))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 256-byte aligned");
  if (!r.dx && !r.dT && !r.dmixw) return ok();
  return hip_status(wbmm::launch_backward_ckpt(r, (hipStream_t)stream), "wbmm_backward_ckpt");
}

// ---------------------------------------------------------------------------- recurrence
namespace {

constexpr int64_t kMaxScanLen = 1ll << 30, kMaxScanCols = (1ll << 26) - 1;

wbmm_status check_scan_sizes(int64_t outer, int64_t len, int64_t inner) {
  if (outer < 1 || len < 1 || inner < 1)
    return fail(WBMM_E_INVALID, "sizes must be >= 1 (outer=%lld len=%lld inner=%lld)",
                (long long)outer, (long long)len, (long long)inner);
  if (len > kMaxScanLen) return fail(WBMM_E_UNSUPPORTED, "len=%lld exceeds 2^30", (long long)len);
  if (outer > kMaxScanCols || inner > kMaxScanCols || outer * inner > kMaxScanCols)
    return fail(WBMM_E_UNSUPPORTED, "outer * inner must be below 2^26");
  if (outer * inner > kMaxElems / len) return fail(WBMM_E_UNSUPPORTED, "tensor too large");
  return WBMM_OK;
}

wbmm_status check_scan_ws(const wbmm::ScanRequest& r, size_t need, size_t bytes) {
  if (need > 0 && (!r.ws || bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                r.ws ? bytes : (size_t)0);
  if (need > 0 && !aligned(r.ws, 16))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 16-byte aligned");
  return WBMM_OK;
}

wbmm_status check_scan_lens(const int32_t* lens, int64_t n_lens, int64_t outer) {
  if (!lens) return WBMM_OK;
  if (n_lens < 1 || outer % n_lens != 0)
    return fail(WBMM_E_INVALID, "n_lens=%lld must divide outer=%lld", (long long)n_lens,
                (long long)outer);
  if (!aligned(lens, 4)) return fail(WBMM_E_UNSUPPORTED, "lens not 4-byte aligned");
  return WBMM_OK;
}

}  // namespace

WBMM_API size_t wbmm_scan_forward_workspace_bytes(int64_t outer, int64_t len, int64_t inner) {
  if (check_scan_sizes(outer, len, inner) != WBMM_OK) return 0;
  return wbmm::scan_workspace(outer, len, inner);
}

WBMM_API size_t wbmm_scan_backward_workspace_bytes(int64_t outer, int64_t len, int64_t inner,
                                                   int has_states) {
  if (check_scan_sizes(outer, len, inner) != WBMM_OK) return 0;
  return wbmm::scan_backward_workspace(outer, len, inner, has_states != 0);
}

WBMM_API wbmm_status wbmm_scan_forward(int64_t outer, int64_t len, int64_t inner, int dtype,
                                       int reverse, const void* g, const void* u, const float* h0,
                                       const int32_t* lens, int64_t n_lens, void* h, float* h_last,
                                       float* states, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  wbmm_status st = check_scan_sizes(outer, len, inner);
  if (st != WBMM_OK) return st;
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (!g || !u || !h) return fail(WBMM_E_INVALID, "g, u and h must be non-NULL");
  st = check_scan_lens(lens, n_lens, outer);
  if (st != WBMM_OK) return st;
  const size_t es = dtype_size(dtype);
  if (!aligned(g, es) || !aligned(u, es) || !aligned(h, es) || !aligned(h0, 4) ||
      !aligned(h_last, 4) || !aligned(states, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t cols = (size_t)outer * inner, n = cols * len * es, cb = cols * 4;
  const size_t sb = cb * ((len + WBMM_SCAN_CHUNK - 1) / WBMM_SCAN_CHUNK);
  const Span in[] = {{g, n, "g"}, {u, n, "u"}, {lens, lens ? (size_t)n_lens * 4 : 0, "lens"},
                     {h0 == h_last ? nullptr : h0, cb, "h0"}};   // in place: exactly the same
  const Span out[] = {{h, n, "h"}, {h_last, cb, "h_last"}, {states, sb, "states"}};
  st = check_spans(in, 4, out, 3);
  if (st != WBMM_OK) return st;
  wbmm::ScanRequest r{};
  r.outer = outer; r.len = len; r.inner = inner; r.n_lens = n_lens;
  r.bf16 = dtype == WBMM_BF16;
  r.reverse = reverse != 0;
  r.g = g; r.u = u; r.carry_in = h0; r.lens = lens;
  r.out0 = h; r.carry_out = h_last; r.states = states; r.ws = workspace;
  st = check_scan_ws(r, wbmm::scan_workspace(outer, len, inner), workspace_bytes);
  if (st != WBMM_OK) return st;
  return hip_status(wbmm::launch_scan_forward(r, (hipStream_t)stream), "wbmm_scan_forward");
}

WBMM_API wbmm_status wbmm_scan_backward(int64_t outer, int64_t len, int64_t inner, int dtype,
                                        int reverse, int u_fmt, const void* g, const void* u,
                                        const uint8_t* u_scales, const float* states,
                                        const float* h0, const void* dh, const float* dh_last,
                                        const int32_t* lens, int64_t n_lens, void* dg, void* du, float* dh0,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  wbmm_status st = check_scan_sizes(outer, len, inner);
  if (st != WBMM_OK) return st;
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (u_scales && !valid_fmt(u_fmt))
    return fail(WBMM_E_INVALID, "unknown checkpoint format %d", u_fmt);
  if (!g || !u || !dh || !dg || !du)
    return fail(WBMM_E_INVALID, "g, u, dh, dg and du must be non-NULL");
  if (states && h0) return fail(WBMM_E_INVALID, "h0 goes with states == NULL only");
  st = check_scan_lens(lens, n_lens, outer);
  if (st != WBMM_OK) return st;
  const size_t es = dtype_size(dtype);
  if (!aligned(g, es) || !aligned(dh, es) || !aligned(dg, es) || !aligned(du, es) ||
      (!u_scales && !aligned(u, es)) || !aligned(states, 4) || !aligned(h0, 4) ||
      !aligned(dh_last, 4) || !aligned(dh0, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t cols = (size_t)outer * inner, e = cols * len, cb = cols * 4;
  const size_t sb = cb * ((len + WBMM_SCAN_CHUNK - 1) / WBMM_SCAN_CHUNK);
  const Span in[] = {{g, e * es, "g"}, {u, u_scales ? e : e * es, "u"},
                     {u_scales, ckpt_scales((int64_t)e), "u_scales"}, {states, sb, "states"},
                     {dh, e * es, "dh"}, {dh_last, cb, "dh_last"},
                     {lens, lens ? (size_t)n_lens * 4 : 0, "lens"}, {h0, cb, "h0"}};
  const Span out[] = {{dg, e * es, "dg"}, {du, e * es, "du"}, {dh0, cb, "dh0"}};
  st = check_spans(in, 8, out, 3);
  if (st != WBMM_OK) return st;
  wbmm::ScanRequest r{};
  r.outer = outer; r.len = len; r.inner = inner; r.n_lens = n_lens;
  r.bf16 = dtype == WBMM_BF16;
  r.reverse = reverse != 0;
  r.fmt = u_fmt;
  r.g = g; r.u = u; r.us = u_scales; r.states = const_cast<float*>(states);
  r.dh = dh; r.carry_in = dh_last; r.h0 = h0; r.lens = lens;
  r.out0 = dg; r.out1 = du; r.carry_out = dh0; r.ws = workspace;
  st = check_scan_ws(r, wbmm::scan_backward_workspace(outer, len, inner, states != nullptr),
                     workspace_bytes);
  if (st != WBMM_OK) return st;
  return hip_status(wbmm::launch_scan_backward(r, (hipStream_t)stream), "wbmm_scan_backward");
}

// ---------------------------------------------------------------------------- RMS norm
namespace {

// A row takes up to 64 lanes, one longer than a wave's registers 256, and grids hold 2^32 threads.
constexpr int64_t kMaxNormRows = 1ll << 25;

wbmm_status check_norm(int64_t outer, int64_t len, int64_t inner, int dtype, double eps) {
  if (outer < 1 || len < 1 || inner < 1)
    return fail(WBMM_E_INVALID, "sizes must be >= 1 (outer=%lld len=%lld inner=%lld)",
                (long long)outer, (long long)len, (long long)inner);
  if (len > kMaxDim) return fail(WBMM_E_UNSUPPORTED, "len=%lld exceeds 2^20", (long long)len);
  if (outer > kMaxNormRows || inner > kMaxNormRows || outer * inner > kMaxNormRows)
    return fail(WBMM_E_UNSUPPORTED, "outer * inner exceeds 2^25");
  if (outer * inner > kMaxCkpt / len) return fail(WBMM_E_UNSUPPORTED, "tensor too large");
  if (inner == 1 && len > wbmm::kNormWaveLen && outer > kMaxNormRows / 4)
    return fail(WBMM_E_UNSUPPORTED, "more than 2^23 rows of over %d elements", wbmm::kNormWaveLen);
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  if (!(eps >= 0) || eps > 3e38) return fail(WBMM_E_INVALID, "eps must be finite and not negative");
  return WBMM_OK;
}

}  // namespace

WBMM_API wbmm_status wbmm_rmsnorm_forward(int64_t outer, int64_t len, int64_t inner, int dtype,
                                          float eps, const void* x, const void* residual,
                                          const float* weight, void* s, void* y, int fmt,
                                          uint8_t* codes, uint8_t* scales, void* stream) {
  wbmm_status st = check_norm(outer, len, inner, dtype, eps);
  if (st != WBMM_OK) return st;
  if (!x || !y) return fail(WBMM_E_INVALID, "x and y must be non-NULL");
  if ((codes == nullptr) != (scales == nullptr))
    return fail(WBMM_E_INVALID, "codes and scales go together");
  if (codes && !valid_fmt(fmt)) return fail(WBMM_E_INVALID, "unknown checkpoint format %d", fmt);
  const size_t es = dtype_size(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, 4) || !aligned(s, es) ||
      !aligned(y, es))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t n = (size_t)outer * len * inner;
  // s may be x or the residual itself: an element is written after it has been read
  const Span in[] = {{x == s ? nullptr : x, n * es, "x"},
                     {residual == s ? nullptr : residual, n * es, "residual"},
                     {weight, (size_t)len * 4, "weight"}};
  const Span out[] = {{s, n * es, "s"}, {y, n * es, "y"}, {codes, n, "codes"},
                      {scales, ckpt_scales((int64_t)n), "scales"}};
  st = check_spans(in, 3, out, 4);
  if (st != WBMM_OK) return st;
  wbmm::NormRequest r{};
  r.outer = outer; r.len = len; r.inner = inner;
  r.bf16 = dtype == WBMM_BF16;
  r.fmt = fmt; r.eps = eps;
  r.x = x; r.res = residual; r.w = weight; r.s = s; r.y = y; r.codes = codes; r.scales = scales;
  return hip_status(wbmm::launch_norm_forward(r, (hipStream_t)stream), "wbmm_rmsnorm_forward");
}

WBMM_API size_t wbmm_rmsnorm_backward_workspace_bytes(int64_t outer, int64_t len, int64_t inner) {
  if (check_norm(outer, len, inner, WBMM_F32, 0) != WBMM_OK) return 0;
  return wbmm::norm_backward_workspace(outer, len, inner);
}

WBMM_API wbmm_status wbmm_rmsnorm_backward(int64_t outer, int64_t len, int64_t inner, int dtype,
                                           float eps, const void* s, const float* weight,
                                           const void* dy, const void* ds, void* dx,
                                           float* dweight, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  wbmm_status st = check_norm(outer, len, inner, dtype, eps);
  if (st != WBMM_OK) return st;
  if (!s || !dy) return fail(WBMM_E_INVALID, "s and dy must be non-NULL");
  const size_t es = dtype_size(dtype);
  if (!aligned(s, es) || !aligned(dy, es) || !aligned(ds, es) || !aligned(dx, es) ||
      !aligned(weight, 4) || !aligned(dweight, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const size_t n = (size_t)outer * len * inner * es;
  const Span in[] = {{s, n, "s"}, {dy, n, "dy"}, {ds, n, "ds"}, {weight, (size_t)len * 4, "weight"}};
  const Span out[] = {{dx, n, "dx"}, {dweight, (size_t)len * 4, "dweight"}};
  st = check_spans(in, 4, out, 2);
  if (st != WBMM_OK) return st;
  if (!dx && !dweight) return ok();
  const size_t need = dweight ? wbmm::norm_backward_workspace(outer, len, inner) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 16-byte aligned");
  wbmm::NormRequest r{};
  r.outer = outer; r.len = len; r.inner = inner;
  r.bf16 = dtype == WBMM_BF16;
  r.eps = eps;
  r.x = s; r.res = ds; r.w = weight; r.dy = dy; r.y = dx; r.dw = dweight; r.ws = workspace;
  return hip_status(wbmm::launch_norm_backward(r, (hipStream_t)stream), "wbmm_rmsnorm_backward");
}

// ---------------------------------------------------------------------------- AdamW
namespace {

constexpr int64_t kMaxAdamChunks = (1ll << 24) - 1;   // grids hold 2^32 threads

int64_t adam_chunks(int64_t n) { return (n + wbmm::kAdamChunk - 1) / wbmm::kAdamChunk; }

wbmm_status adam_sizes(const wbmm_adamw_tensor* t, int64_t count, int64_t* chunks) {
  if (!t) return fail(WBMM_E_INVALID, "tensors must be non-NULL");
  if (count < 1) return fail(WBMM_E_INVALID, "count=%lld must be >= 1", (long long)count);
  if (count > kMaxAdamChunks) return fail(WBMM_E_UNSUPPORTED, "more than 2^24 - 1 tensors");
  int64_t sum = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 1)
      return fail(WBMM_E_INVALID, "tensor %lld: n=%lld must be >= 1", (long long)i,
                  (long long)t[i].n);
    if (t[i].n > kMaxAdamChunks * wbmm::kAdamChunk ||
        (sum += adam_chunks(t[i].n)) > kMaxAdamChunks)
      return fail(WBMM_E_UNSUPPORTED, "more than 2^36 elements");
  }
  *chunks = sum;
  return WBMM_OK;
}

size_t adam_bytes(int64_t count, int64_t chunks) {
  return sizeof(wbmm::AdamHead) + (size_t)count * sizeof(wbmm::AdamEntry) + (size_t)chunks * 4;
}

wbmm_status adam_tensor(const wbmm_adamw_tensor& t, long long i) {
  if (!t.p || !t.g || !t.m || !t.v)
    return fail(WBMM_E_INVALID, "tensor %lld: p, g, m and v must be non-NULL", i);
  if ((t.m_scales == nullptr) != (t.v_scales == nullptr))
    return fail(WBMM_E_INVALID, "tensor %lld: m_scales and v_scales go together", i);
  if (!valid_dtype(t.g_dtype))
    return fail(WBMM_E_INVALID, "tensor %lld: unknown gradient dtype %d", i, t.g_dtype);
  if (!std::isfinite(t.weight_decay) || t.weight_decay < 0)
    return fail(WBMM_E_INVALID, "tensor %lld: weight_decay must be finite and not negative", i);
  const bool small = t.m_scales != nullptr;
  if (!aligned(t.p, 4) || !aligned(t.g, dtype_size(t.g_dtype)) || !aligned(t.p_bf16, 2) ||
      (!small && (!aligned(t.m, 4) || !aligned(t.v, 4))))
    return fail(WBMM_E_UNSUPPORTED, "tensor %lld: pointer not aligned to its element size", i);
  return WBMM_OK;
}

}  // namespace

WBMM_API size_t wbmm_adamw_plan_bytes(const wbmm_adamw_tensor* tensors, int64_t count) {
  int64_t chunks = 0;
  return adam_sizes(tensors, count, &chunks) == WBMM_OK ? adam_bytes(count, chunks) : 0;
}

WBMM_API wbmm_status wbmm_adamw_plan(const wbmm_adamw_tensor* tensors, int64_t count, void* table,
                                     size_t table_bytes, int64_t* chunks) {
  int64_t total = 0;
  wbmm_status st = adam_sizes(tensors, count, &total);
  if (st != WBMM_OK) return st;
  if (!table || !chunks) return fail(WBMM_E_INVALID, "table and chunks must be non-NULL");
  if (table_bytes < adam_bytes(count, total))
    return fail(WBMM_E_WORKSPACE, "table of %zu bytes required, %zu given",
                adam_bytes(count, total), table_bytes);
  if (!aligned(table, 8)) return fail(WBMM_E_UNSUPPORTED, "table not 8-byte aligned");
  // nothing that a step writes may be another tensor's, or its own gradient
  struct Range { uintptr_t a, b; int64_t i; bool written; };
  try {
    std::vector<Range> all;
    all.reserve((size_t)count * 7);
    for (int64_t i = 0; i < count; ++i) {
      const wbmm_adamw_tensor& t = tensors[i];
      st = adam_tensor(t, (long long)i);
      if (st != WBMM_OK) return st;
      const size_t n = (size_t)t.n, e = t.m_scales ? 1 : 4, sc = ckpt_scales(t.n);
      auto add = [&](const void* p, size_t bytes, bool written) {
        if (p) all.push_back({(uintptr_t)p, (uintptr_t)p + bytes, i, written});
      };
      add(t.p, n * 4, true);
      add(t.g, n * dtype_size(t.g_dtype), false);
      add(t.m, n * e, true);
      add(t.v, n * e, true);
      add(t.m_scales, sc, true);
      add(t.v_scales, sc, true);
      add(t.p_bf16, n * 2, true);
    }
    std::sort(all.begin(), all.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
    uintptr_t end = 0, wend = 0;       // of all ranges so far, and of the written ones
    int64_t at = 0, wat = 0;
    for (const Range& r : all) {
      if (r.a < wend || (r.written && r.a < end))
        return fail(WBMM_E_INVALID, "tensors %lld and %lld overlap",
                    (long long)(r.a < wend ? wat : at), (long long)r.i);
      if (r.b > end) end = r.b, at = r.i;
      if (r.written && r.b > wend) wend = r.b, wat = r.i;
    }
  } catch (const std::bad_alloc&) {
    return fail(WBMM_E_UNSUPPORTED, "out of host memory for %lld tensors", (long long)count);
  }
  wbmm::AdamHead* head = (wbmm::AdamHead*)table;
  *head = {wbmm::kAdamMagic, (uint64_t)count, (uint64_t)total, 0};
  wbmm::AdamEntry* entries = (wbmm::AdamEntry*)(head + 1);
  uint32_t* owner = (uint32_t*)(entries + count);
  uint32_t first = 0;
  for (int64_t i = 0; i < count; ++i) {
    const wbmm_adamw_tensor& t = tensors[i];
    const bool small = t.m_scales != nullptr;
    wbmm::AdamEntry e{};
    e.p = t.p; e.g = t.g; e.m = t.m; e.v = t.v; e.ms = t.m_scales; e.vs = t.v_scales;
    e.copy = t.p_bf16; e.n = t.n; e.decay = t.weight_decay; e.first = first;
    const size_t sa = small ? 8 : 16;
    if (t.g_dtype == WBMM_BF16) e.flags |= wbmm::kAdamG16;
    if (small) e.flags |= wbmm::kAdam8;
    if (aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.m, sa) && aligned(t.v, sa) &&
        aligned(t.p_bf16, 16))
      e.flags |= wbmm::kAdamWide;
    entries[i] = e;
    const uint32_t c = (uint32_t)adam_chunks(t.n);
    for (uint32_t k = 0; k < c; ++k) owner[first + k] = (uint32_t)i;
    first += c;
  }
  *chunks = total;
  return ok();
}

WBMM_API wbmm_status wbmm_adamw_step(const void* table, int64_t count, int64_t chunks, double lr,
                                     double beta1, double beta2, double eps, int64_t step,
                                     const int32_t* step_dev, const float* lr_factor,
                                     const float* grad_factor, uint64_t seed, void* stream) {
  if (!table) return fail(WBMM_E_INVALID, "table must be non-NULL");
  if (count < 1 || chunks < count || chunks > kMaxAdamChunks)
    return fail(WBMM_E_INVALID, "count=%lld and chunks=%lld are not a plan's", (long long)count,
                (long long)chunks);
  if (!std::isfinite(lr)) return fail(WBMM_E_INVALID, "lr must be finite");
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
    return fail(WBMM_E_INVALID, "beta1 and beta2 must lie in [0, 1)");
  if (!(eps >= 0) || !std::isfinite(eps))
    return fail(WBMM_E_INVALID, "eps must be finite and not negative");
  if (!step_dev && (step < 1 || step > INT32_MAX))
    return fail(WBMM_E_INVALID, "step=%lld outside [1, 2^31)", (long long)step);
  if (!aligned(table, 8) || !aligned(step_dev, 4) || !aligned(lr_factor, 4) ||
      !aligned(grad_factor, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  wbmm::AdamRequest r{};
  r.table = table; r.count = (uint32_t)count; r.chunks = (uint32_t)chunks;
  r.lr = lr; r.beta1 = beta1; r.beta2 = beta2; r.eps = eps;
  r.step = step; r.step_dev = step_dev; r.lr_factor = lr_factor; r.grad_factor = grad_factor;
  r.seed = seed;
  return hip_status(wbmm::launch_adamw(r, (hipStream_t)stream), "wbmm_adamw_step");
}

// ---------------------------------------------------------------------------- delta rule
namespace {

constexpr int64_t kMaxDeltaChunks = 1ll << 22;   // chunks of heads: grids hold 2^32 threads

wbmm_status check_delta(int64_t B, int64_t L, int Hk, int H, int dk, int dv, int dtype) {
  if (B < 1 || L < 1 || Hk < 1 || H < 1 || dk < 1 || dv < 1)
    return fail(WBMM_E_INVALID, "sizes must be >= 1 (B=%lld L=%lld Hk=%d H=%d dk=%d dv=%d)",
                (long long)B, (long long)L, Hk, H, dk, dv);
  if (H % Hk != 0) return fail(WBMM_E_INVALID, "Hk=%d must divide H=%d", Hk, H);
  if (dk > 128 || dv > 128)
    return fail(WBMM_E_UNSUPPORTED, "dk=%d and dv=%d must not exceed 128", dk, dv);
  if ((int64_t)Hk * dk > (1 << 22) || (int64_t)H * dv > (1 << 22))
    return fail(WBMM_E_UNSUPPORTED, "rows of more than 2^22 elements");
  if (L > (1ll << 28) || B > kMaxDeltaChunks || H > kMaxDeltaChunks ||
      B * H > kMaxDeltaChunks ||
      B * H * ((L + WBMM_DELTA_CHUNK - 1) / WBMM_DELTA_CHUNK) > kMaxDeltaChunks)
    return fail(WBMM_E_UNSUPPORTED, "more than 2^22 chunks of %d steps of a head, or L > 2^28",
                WBMM_DELTA_CHUNK);
  if (!valid_dtype(dtype)) return fail(WBMM_E_INVALID, "unknown dtype %d", dtype);
  return WBMM_OK;
}

wbmm_status check_delta_ws(size_t need, const void* ws, size_t bytes) {
  if (need > 0 && (!ws || bytes < need))
    return fail(WBMM_E_WORKSPACE, "workspace of %zu bytes required, %zu given", need,
                ws ? bytes : (size_t)0);
  if (need > 0 && !aligned(ws, 16))
    return fail(WBMM_E_UNSUPPORTED, "workspace not 16-byte aligned");
  return WBMM_OK;
}

// Byte sizes of the tensors of a call.
struct DeltaBytes {
  size_t qk, v, gate, state, states;
  DeltaBytes(int64_t B, int64_t L, int Hk, int H, int dk, int dv, int dtype) {
    const size_t es = dtype_size(dtype), t = (size_t)B * L;
    qk = t * Hk * dk * es;
    v = t * H * dv * es;
    gate = t * H * es;
    state = (size_t)B * H * dk * dv * 4;
    states = state * ((L + WBMM_DELTA_CHUNK - 1) / WBMM_DELTA_CHUNK);
  }
};

}  // namespace

WBMM_API size_t wbmm_delta_forward_workspace_bytes(int64_t B, int64_t L, int Hk, int H, int dk,
                                                   int dv, int dtype) {
  if (check_delta(B, L, Hk, H, dk, dv, dtype) != WBMM_OK) return 0;
  return wbmm::delta_forward_workspace(B, L, H, dtype == WBMM_BF16);
}

WBMM_API wbmm_status wbmm_delta_forward(int64_t B, int64_t L, int Hk, int H, int dk, int dv,
                                        int dtype, int reverse, float scale, const void* q,
                                        const void* k, const void* v, const void* g,
                                        const void* beta, const float* s0, const int32_t* lens,
                                        void* o, float* s_last, float* states, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  wbmm_status st = check_delta(B, L, Hk, H, dk, dv, dtype);
  if (st != WBMM_OK) return st;
  if (!std::isfinite(scale)) return fail(WBMM_E_INVALID, "scale must be finite");
  if (!q || !k || !v || !g || !beta || !o)
    return fail(WBMM_E_INVALID, "q, k, v, g, beta and o must be non-NULL");
  const size_t es = dtype_size(dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(g, es) ||
      !aligned(beta, es) || !aligned(o, es) || !aligned(s0, 4) || !aligned(lens, 4) ||
      !aligned(s_last, 4) || !aligned(states, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const DeltaBytes n(B, L, Hk, H, dk, dv, dtype);
  const Span in[] = {{q, n.qk, "q"}, {k, n.qk, "k"}, {v, n.v, "v"}, {g, n.gate, "g"},
                     {beta, n.gate, "beta"}, {lens, (size_t)B * 4, "lens"},
                     {s0 == s_last ? nullptr : s0, n.state, "s0"}};   // in place: exactly the same
  const Span out[] = {{o, n.v, "o"}, {s_last, n.state, "s_last"}, {states, n.states, "states"}};
  st = check_spans(in, 7, out, 3);
  if (st != WBMM_OK) return st;
  st = check_delta_ws(wbmm::delta_forward_workspace(B, L, H, dtype == WBMM_BF16), workspace,
                      workspace_bytes);
  if (st != WBMM_OK) return st;
  wbmm::DeltaRequest r{};
  r.B = B; r.L = L; r.Hk = Hk; r.H = H; r.dk = dk; r.dv = dv;
  r.bf16 = dtype == WBMM_BF16;
  r.reverse = reverse != 0;
  r.scale = scale;
  r.q = q; r.k = k; r.v = v; r.g = g; r.beta = beta; r.s0 = s0; r.lens = lens;
  r.o = o; r.s_last = s_last; r.states = states; r.ws = workspace;
  return hip_status(wbmm::launch_delta_forward(r, (hipStream_t)stream), "wbmm_delta_forward");
}

WBMM_API size_t wbmm_delta_backward_workspace_bytes(int64_t B, int64_t L, int Hk, int H, int dk,
                                                    int dv, int dtype, int has_states) {
  if (check_delta(B, L, Hk, H, dk, dv, dtype) != WBMM_OK) return 0;
  return wbmm::delta_backward_workspace(B, L, H, dk, dv, dtype == WBMM_BF16, has_states != 0);
}

WBMM_API wbmm_status wbmm_delta_backward(
    int64_t B, int64_t L, int Hk, int H, int dk, int dv, int dtype, int reverse, float scale,
    const void* q, const void* k, const void* v, const void* g, const void* beta,
    const float* states, const float* s0, const void* dout, const float* ds_last,
    const int32_t* lens, void* dq, void* dkey, void* dval, void* dg, void* dbeta, float* ds0,
    void* workspace, size_t workspace_bytes, void* stream) {
  wbmm_status st = check_delta(B, L, Hk, H, dk, dv, dtype);
  if (st != WBMM_OK) return st;
  if (!std::isfinite(scale)) return fail(WBMM_E_INVALID, "scale must be finite");
  if (!q || !k || !v || !g || !beta || !dout || !dq || !dkey || !dval || !dg || !dbeta)
    return fail(WBMM_E_INVALID,
                "q, k, v, g, beta, do, dq, dk, dv, dg and dbeta must be non-NULL");
  if (states && s0) return fail(WBMM_E_INVALID, "s0 goes with states == NULL only");
  const size_t es = dtype_size(dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(g, es) ||
      !aligned(beta, es) || !aligned(dout, es) || !aligned(dq, es) || !aligned(dkey, es) ||
      !aligned(dval, es) || !aligned(dg, es) || !aligned(dbeta, es) || !aligned(s0, 4) ||
      !aligned(lens, 4) || !aligned(ds_last, 4) || !aligned(ds0, 4) || !aligned(states, 4))
    return fail(WBMM_E_UNSUPPORTED, "pointer not aligned to its element size");
  const DeltaBytes n(B, L, Hk, H, dk, dv, dtype);
  const Span in[] = {{q, n.qk, "q"}, {k, n.qk, "k"}, {v, n.v, "v"}, {g, n.gate, "g"},
                     {beta, n.gate, "beta"}, {lens, (size_t)B * 4, "lens"},
                     {states, n.states, "states"}, {s0, n.state, "s0"}, {dout, n.v, "do"},
                     {ds_last == ds0 ? nullptr : ds_last, n.state, "ds_last"}};
  const Span out[] = {{dq, n.qk, "dq"}, {dkey, n.qk, "dk"}, {dval, n.v, "dv"}, {dg, n.gate, "dg"},
                      {dbeta, n.gate, "dbeta"}, {ds0, n.state, "ds0"}};
  st = check_spans(in, 10, out, 6);
  if (st != WBMM_OK) return st;
  st = check_delta_ws(wbmm::delta_backward_workspace(B, L, H, dk, dv, dtype == WBMM_BF16,
                                                     states != nullptr),
                      workspace, workspace_bytes);
  if (st != WBMM_OK) return st;
  wbmm::DeltaRequest r{};
  r.B = B; r.L = L; r.Hk = Hk; r.H = H; r.dk = dk; r.dv = dv;
  r.bf16 = dtype == WBMM_BF16;
  r.reverse = reverse != 0;
  r.scale = scale;
  r.q = q; r.k = k; r.v = v; r.g = g; r.beta = beta; r.dout = dout; r.lens = lens;
  r.states = const_cast<float*>(states); r.s0 = s0; r.ds_last = ds_last;
  r.dq = dq; r.dkey = dkey; r.dval = dval; r.dg = dg; r.dbeta = dbeta; r.ds0 = ds0;
  r.ws = workspace;
  return hip_status(wbmm::launch_delta_backward(r, (hipStream_t)stream), "wbmm_delta_backward");
}
