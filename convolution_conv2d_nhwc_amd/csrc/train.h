// train.h -- internal declarations of the training-side operators
// (include/conv_train.h): plans computed on the host, kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/conv_train.h"

namespace convnhwc {

// Keeps the text of a HIP error for conv_status_str; CONV_OK for hipSuccess.
conv_status hip_status(hipError_t err);
bool ranges_overlap(const void* a, int64_t an, const void* b, int64_t bn);

// ---- group norm ---------------------------------------------------------------

// How a (n, h*w, c) map is cut: channel tiles of whole groups (tpg == 1) or
// parts of one group (gpt == 1, tpg > 1), and pixel chunks.
struct NormPlan {
  int vec;     // elements per load
  int ct;      // channels per tile (a multiple of vec)
  int gpt;     // groups per tile
  int tpg;     // tiles per group
  int ctiles;  // channel tiles
  int ppi;     // pixels a workgroup covers per step
  int r;       // one launch: vectors a lane keeps in registers; 0: streamed
  int threads; // lanes of a workgroup: 512, or 1024 for one launch with the most vectors a lane
  int chunks;  // pixel chunks per image (one launch: 1)
  int cpix;    // pixels per chunk, whole blocks
};

struct NormArgs {
  const void* x;
  const void* dy;
  const float* gamma;
  const float* beta;
  void* y;       // y, or dx of the gradient
  float* stats;  // [n][groups][2]: written by the forward pass when not null, read by the gradient
  float* part;   // ws: forward [n][groups][chunks * tpg][2]; gradient [n][chunks][c][2]
  float* dgamma;
  float* dbeta;
  int64_t pitch;  // elements per pixel of x
  int n, hw, c, groups, cg;
  float eps, inv_count;
  int act;
  NormPlan p;
};

// align: the byte alignment that x, dy and y share (a power of two, at most 16).
NormPlan norm_plan(const conv_norm_desc& d, bool grad, int align);
int64_t norm_ws_bytes(const conv_norm_desc& d, const NormPlan& p, bool grad);
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_grad(const NormArgs& a, int dtype, hipStream_t s);

// ---- head loss ----------------------------------------------------------------

// A product's tile side and the splits of its reduction.
struct GemmShape {
  int tile, splits;
};

// Tiles, pieces and the layout of ws (byte offsets; -1: not used).
struct HeadPlan {
  int64_t cpad;    // channels of the copies, a multiple of 8
  int64_t cq;      // pitch of the fp32 partial sums, a multiple of 4
  int64_t vp;      // classes per piece of the gradient, a multiple of 256
  int slots;       // (max, sum) pairs per row
  int stat_tile, ds_tile;
  bool copy_x, pair;
  GemmShape dx, dw;
  int64_t o_stat, o_lab, o_x, o_w;                       // forward, copies
  int64_t o_lse, o_inv, o_delta, o_ds, o_dxp, o_dwp;     // gradient
  int64_t bytes;
};

struct HeadArgs {
  const uint16_t* x;
  const uint16_t* w;
  const void* labels;
  const float* weights;
  float* loss;
  float* total;
  uint16_t* dx;
  uint16_t* dw;
  char* ws;
  int64_t rows, c, classes;
  int label_bytes;
  HeadPlan p;
};

// Workgroups of the logits' product, the widest launch.
int64_t head_workgroups(const conv_head_desc& d);
// copy_x, copy_w: the operand cannot be read in place (c % 8 or alignment).
HeadPlan head_plan(const conv_head_desc& d, bool grad, bool copy_x, bool copy_w);
// The plan in words: each product's tile side x workgroups a CU, and its splits.
void head_describe(const conv_head_desc& d, bool grad, const HeadPlan& p, char* buf, int len);
hipError_t launch_head_loss(const HeadArgs& a, bool grad, hipStream_t s);

// ---- orthogonalisation ----------------------------------------------------------

struct OrthoArgs {
  const void* g;
  uint16_t* out;
  char* ws;
  int batch, rows, cols;
  int steps;
  float a, b, c, eps;
  int g_f32;
};

int64_t ortho_ws_bytes(const conv_ortho_desc& d);
void ortho_describe(const conv_ortho_desc& d, char* buf, int len);
hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s);

}  // namespace convnhwc
