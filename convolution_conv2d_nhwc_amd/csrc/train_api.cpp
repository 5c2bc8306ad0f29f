// train_api.cpp -- C entry points of the training-side operators
// (include/conv_train.h): argument checks on the host, then the launchers.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "train.h"

using namespace convnhwc;

namespace {

constexpr int64_t kMaxBytes = (int64_t)1 << 31;

// The byte alignment an address has, up to 16 (16 for NULL).
int align_of(const void* p) {
  const uintptr_t v = (uintptr_t)p;
  return v & 15 ? (int)(v & (~v + 1)) : 16;
}

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether any output overlaps an input or another output.
template <int NI, int NO>
bool aliased(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (ranges_overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

// ---- group norm ---------------------------------------------------------------

conv_status norm_check(const conv_norm_desc* d) {
  if (!d) return CONV_E_NULL;
  if (d->n <= 0 || d->h <= 0 || d->w <= 0 || d->c <= 0 || d->groups <= 0 || d->c % d->groups ||
      d->x_pixel_stride < 0 || (d->x_pixel_stride && d->x_pixel_stride < d->c) || !(d->eps >= 0.0f) ||
      !std::isfinite(d->eps))
    return CONV_E_SHAPE;
  if (d->dtype != CONV_F32 && d->dtype != CONV_BF16) return CONV_E_UNSUPPORTED;
  if (d->act < CONV_ACT_NONE || d->act > CONV_ACT_SILU) return CONV_E_UNSUPPORTED;
  const int64_t esz = d->dtype == CONV_F32 ? 4 : 2, pitch = d->x_pixel_stride ? d->x_pixel_stride : d->c;
  // each factor bounded before the product, so that it cannot wrap
  if (d->n > 65535 || d->h >= kMaxBytes || d->w >= kMaxBytes || pitch >= kMaxBytes) return CONV_E_UNSUPPORTED;
  if (d->h * d->w >= kMaxBytes || d->h * d->w * d->n >= kMaxBytes ||
      (double)d->h * d->w * d->n * pitch * esz >= (double)kMaxBytes)
    return CONV_E_UNSUPPORTED;
  // channel tiles are a grid dimension
  if (d->c > 65535) return CONV_E_UNSUPPORTED;
  return CONV_OK;
}

// Scratch that is enough whatever the pointers' alignment.
int64_t norm_ws(const conv_norm_desc& d, bool grad) {
  int64_t most = 0;
  for (int align = 2; align <= 16; align *= 2)
    most = std::max(most, norm_ws_bytes(d, norm_plan(d, grad, align), grad));
  return most;
}

NormArgs norm_args(const conv_norm_desc& d) {
  NormArgs a = {};
  a.pitch = d.x_pixel_stride ? d.x_pixel_stride : d.c;
  a.n = (int)d.n;
  a.hw = (int)(d.h * d.w);
  a.c = (int)d.c;
  a.groups = d.groups;
  a.cg = (int)(d.c / d.groups);
  a.eps = d.eps;
  a.inv_count = (float)(1.0 / ((double)a.hw * a.cg));
  a.act = d.act;
  return a;
}

// ---- head loss ----------------------------------------------------------------

conv_status head_check(const conv_head_desc* d) {
  if (!d) return CONV_E_NULL;
  if (d->rows <= 0 || d->c <= 0 || d->classes <= 0) return CONV_E_SHAPE;
  if (d->dtype != CONV_BF16 || (d->label_bytes != 4 && d->label_bytes != 8)) return CONV_E_UNSUPPORTED;
  // below 2^22 - 64 rows and classes the copies' grids (64 a workgroup) and the
  // smallest piece of the gradient (256 classes by rows) stay in range
  if (d->c > 65536 || d->rows > (1 << 22) - 64 || d->classes > (1 << 22) - 64) return CONV_E_UNSUPPORTED;
  const int64_t c = (d->c + 7) / 8 * 8, most = (std::max(d->rows, d->classes) + 63) / 64 * 64;
  if (most * c * 2 >= kMaxBytes) return CONV_E_UNSUPPORTED;
  // a launch has fewer than 2^32 lanes, 256 a workgroup
  if (head_workgroups(*d) >= 1 << 24) return CONV_E_UNSUPPORTED;
  return CONV_OK;
}

conv_status head_run(const conv_head_desc* d, const void* x, const void* w, const void* labels, const float* weights,
                     float* loss, float* total, void* dx, void* dw, void* ws, int64_t ws_bytes, void* stream,
                     bool grad) {
  if (!d || !x || !w || !labels || !loss || !total || (grad && (!dx || !dw))) return CONV_E_NULL;
  const conv_status st = head_check(d);
  if (st != CONV_OK) return st;
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)dx | (uintptr_t)dw) & 1) return CONV_E_ALIGN;
  if ((uintptr_t)labels & (d->label_bytes - 1)) return CONV_E_ALIGN;
  if (((uintptr_t)weights | (uintptr_t)loss | (uintptr_t)total) & 3) return CONV_E_ALIGN;
  if (!ws) return CONV_E_NULL;
  if ((uintptr_t)ws & 255) return CONV_E_ALIGN;
  HeadArgs a = {};
  a.p = head_plan(*d, grad, d->c % 8 || ((uintptr_t)x & 15), d->c % 8 || ((uintptr_t)w & 15));
  if (a.p.bytes > ws_bytes) return CONV_E_SCRATCH;
  const int64_t xb = d->rows * d->c * 2, wb = d->classes * d->c * 2;
  const Range in[] = {{x, xb}, {w, wb}, {labels, d->rows * d->label_bytes}, {weights, d->rows * 4}};
  const Range out[] = {{loss, d->rows * 4}, {total, 4}, {dx, xb}, {dw, wb}, {ws, a.p.bytes}};
  if (aliased(in, out)) return CONV_E_ALIAS;
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.labels = labels;
  a.weights = weights;
  a.loss = loss;
  a.total = total;
  a.dx = static_cast<uint16_t*>(dx);
  a.dw = static_cast<uint16_t*>(dw);
  a.ws = static_cast<char*>(ws);
  a.rows = d->rows;
  a.c = d->c;
  a.classes = d->classes;
  a.label_bytes = d->label_bytes;
  return hip_status(launch_head_loss(a, grad, static_cast<hipStream_t>(stream)));
}

// ---- orthogonalisation ----------------------------------------------------------

conv_status ortho_check(const conv_ortho_desc* d) {
  if (!d) return CONV_E_NULL;
  if (d->batch <= 0 || d->rows <= 0 || d->cols <= 0 || d->steps < 1 || d->steps > 100 || !std::isfinite(d->a) ||
      !std::isfinite(d->b) || !std::isfinite(d->c) || !(d->eps >= 0.0f) || !std::isfinite(d->eps))
    return CONV_E_SHAPE;
  if (d->dtype != CONV_F32 && d->dtype != CONV_BF16) return CONV_E_UNSUPPORTED;
  if (d->batch > 65535 || d->rows > 32768 || d->cols > 32768) return CONV_E_UNSUPPORTED;
  const int64_t esz = d->dtype == CONV_F32 ? 4 : 2;
  const int64_t rp = (d->rows + 63) / 64 * 64, cp = (d->cols + 63) / 64 * 64;
  // one padded matrix is a product's operand; g is a tensor of its own
  if (rp * cp * 2 >= kMaxBytes || d->batch * d->rows * d->cols * esz >= kMaxBytes) return CONV_E_UNSUPPORTED;
  return CONV_OK;
}

}  // namespace

extern "C" {

int64_t conv_head_loss_ws_bytes(const conv_head_desc* d, int32_t grad) {
  const conv_status st = head_check(d);
  // operands that need a copy only for their alignment are counted in
  return st != CONV_OK ? (int64_t)st : head_plan(*d, grad != 0, true, true).bytes;
}

conv_status conv_head_loss_describe(const conv_head_desc* d, int32_t grad, int32_t align, char* buf, int32_t len) {
  if (!d || !buf || len <= 0) return CONV_E_NULL;
  const conv_status st = head_check(d);
  if (st != CONV_OK) return st;
  const bool copy = d->c % 8 || align % 16;
  head_describe(*d, grad != 0, head_plan(*d, grad != 0, copy, copy), buf, len);
  return CONV_OK;
}

conv_status conv_head_loss(const conv_head_desc* d, const void* x, const void* w, const void* labels,
                           const float* weights, float* loss, float* total, void* ws, int64_t ws_bytes,
                           void* stream) {
  return head_run(d, x, w, labels, weights, loss, total, nullptr, nullptr, ws, ws_bytes, stream, false);
}

conv_status conv_head_loss_grad(const conv_head_desc* d, const void* x, const void* w, const void* labels,
                                const float* weights, float* loss, float* total, void* dx, void* dw, void* ws,
                                int64_t ws_bytes, void* stream) {
  return head_run(d, x, w, labels, weights, loss, total, dx, dw, ws, ws_bytes, stream, true);
}

int64_t conv_orthogonalize_ws_bytes(const conv_ortho_desc* d) {
  const conv_status st = ortho_check(d);
  return st != CONV_OK ? (int64_t)st : ortho_ws_bytes(*d);
}

conv_status conv_orthogonalize_describe(const conv_ortho_desc* d, char* buf, int32_t len) {
  if (!d || !buf || len <= 0) return CONV_E_NULL;
  const conv_status st = ortho_check(d);
  if (st != CONV_OK) return st;
  ortho_describe(*d, buf, len);
  return CONV_OK;
}

conv_status conv_orthogonalize(const conv_ortho_desc* d, const void* g, void* out, void* ws, int64_t ws_bytes,
                               void* stream) {
  if (!d || !g || !out) return CONV_E_NULL;
  const int64_t need = conv_orthogonalize_ws_bytes(d);
  if (need < 0) return (conv_status)need;
  if (need > 0 && !ws) return CONV_E_NULL;
  const int64_t esz = d->dtype == CONV_F32 ? 4 : 2, count = d->batch * d->rows * d->cols;
  if ((uintptr_t)g & (esz - 1) || (uintptr_t)out & 1 || (uintptr_t)ws & 255) return CONV_E_ALIGN;
  if (need > ws_bytes) return CONV_E_SCRATCH;
  const Range in[] = {{g, count * esz}};
  const Range res[] = {{out, count * 2}, {ws, need}};
  if (aliased(in, res)) return CONV_E_ALIAS;
  OrthoArgs a = {};
  a.g = g;
  a.out = static_cast<uint16_t*>(out);
  a.ws = static_cast<char*>(ws);
  a.batch = (int)d->batch;
  a.rows = (int)d->rows;
  a.cols = (int)d->cols;
  a.steps = d->steps;
  a.a = d->a;
  a.b = d->b;
  a.c = d->c;
  a.eps = d->eps;
  a.g_f32 = d->dtype == CONV_F32;
  return hip_status(launch_ortho(a, static_cast<hipStream_t>(stream)));
}

int64_t conv_group_norm_ws_bytes(const conv_norm_desc* d, int32_t grad) {
  const conv_status st = norm_check(d);
  if (st != CONV_OK) return st;
  const int64_t b = norm_ws(*d, grad != 0);
  return b >= kMaxBytes ? (int64_t)CONV_E_UNSUPPORTED : b;
}

conv_status conv_group_norm_describe(const conv_norm_desc* d, int32_t grad, int32_t align, char* buf, int32_t len) {
  if (!d || !buf || len <= 0) return CONV_E_NULL;
  const conv_status st = norm_check(d);
  if (st != CONV_OK) return st;
  const NormPlan p = norm_plan(*d, grad != 0, align_of(reinterpret_cast<const void*>((uintptr_t)align)));
  std::snprintf(buf, len,
                "group_norm%s %s dtype=%s vec=%d ct=%d gpt=%d tpg=%d ctiles=%d ppi=%d r=%d threads=%d chunks=%d "
                "cpix=%d",
                grad ? "_grad" : "", p.r ? "whole" : "streamed", d->dtype == CONV_F32 ? "f32" : "bf16", p.vec, p.ct,
                p.gpt, p.tpg, p.ctiles, p.ppi, p.r, p.threads, p.chunks, p.cpix);
  return CONV_OK;
}

conv_status conv_group_norm(const conv_norm_desc* d, const void* x, const float* gamma, const float* beta, void* y,
                            float* stats, void* ws, int64_t ws_bytes, void* stream) {
  if (!d || !x || !y) return CONV_E_NULL;
  const conv_status st = norm_check(d);
  if (st != CONV_OK) return st;
  const int esz = d->dtype == CONV_F32 ? 4 : 2;
  if (((uintptr_t)x | (uintptr_t)y) & (esz - 1)) return CONV_E_ALIGN;
  if (((uintptr_t)gamma | (uintptr_t)beta | (uintptr_t)stats) & 3) return CONV_E_ALIGN;
  const NormPlan plan = norm_plan(*d, false, std::min(align_of(x), align_of(y)));
  const int64_t need = norm_ws_bytes(*d, plan, false);
  if (need >= kMaxBytes) return CONV_E_UNSUPPORTED;
  if (need > 0 && !ws) return CONV_E_NULL;
  if ((uintptr_t)ws & 255) return CONV_E_ALIGN;
  if (need > ws_bytes) return CONV_E_SCRATCH;
  NormArgs a = norm_args(*d);
  const int64_t px = d->n * a.hw;
  const Range in[] = {{x, ((px - 1) * a.pitch + a.c) * esz}, {gamma, a.c * 4}, {beta, a.c * 4}};
  const Range out[] = {{y, px * a.c * esz}, {stats, (int64_t)a.n * a.groups * 8}, {ws, need}};
  if (aliased(in, out)) return CONV_E_ALIAS;
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.stats = stats;
  a.part = static_cast<float*>(ws);
  a.p = plan;
  return hip_status(launch_norm(a, d->dtype, static_cast<hipStream_t>(stream)));
}

conv_status conv_group_norm_grad(const conv_norm_desc* d, const void* x, const void* dy, const float* stats,
                                 const float* gamma, const float* beta, void* dx, float* dgamma, float* dbeta,
                                 void* ws, int64_t ws_bytes, void* stream) {
  if (!d || !x || !dy || !stats || !dx) return CONV_E_NULL;
  const conv_status st = norm_check(d);
  if (st != CONV_OK) return st;
  const int esz = d->dtype == CONV_F32 ? 4 : 2;
  if (((uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx) & (esz - 1)) return CONV_E_ALIGN;
  if (((uintptr_t)gamma | (uintptr_t)beta | (uintptr_t)stats | (uintptr_t)dgamma | (uintptr_t)dbeta) & 3)
    return CONV_E_ALIGN;
  const NormPlan plan = norm_plan(*d, true, std::min(align_of(x), std::min(align_of(dy), align_of(dx))));
  const int64_t need = norm_ws_bytes(*d, plan, true);
  if (need >= kMaxBytes) return CONV_E_UNSUPPORTED;
  if (need > 0 && !ws) return CONV_E_NULL;
  if ((uintptr_t)ws & 255) return CONV_E_ALIGN;
  if (need > ws_bytes) return CONV_E_SCRATCH;
  NormArgs a = norm_args(*d);
  const int64_t px = d->n * a.hw, st_bytes = (int64_t)a.n * a.groups * 8;
  const Range in[] = {{x, ((px - 1) * a.pitch + a.c) * esz}, {dy, px * a.c * esz}, {stats, st_bytes},
                      {gamma, a.c * 4}, {beta, a.c * 4}};
  const Range out[] = {{dx, px * a.c * esz}, {dgamma, a.c * 4}, {dbeta, a.c * 4}, {ws, need}};
  if (aliased(in, out)) return CONV_E_ALIAS;
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.y = dx;
  a.stats = const_cast<float*>(stats);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.p = plan;
  a.part = static_cast<float*>(ws);
  return hip_status(launch_norm_grad(a, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
