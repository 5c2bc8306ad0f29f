// head_loss.hip -- softmax cross entropy of a 1x1 head over a large set of
// classes, and its gradients, without storing the logits.
//
// Mathematics. s[r][v] = x[r] . w[v]; with the row's maximum m and
// sum = sum_v e^(s - m): loss = log(sum) - (s[label] - m), and with
// lse = m + log(sum) and the row's weight k:
//   g[r][v] = k (e^(s - lse) - [v == label]),  dx = g w,  dw = g^T x.
//
// Forward: one matrix product whose epilogue keeps a (maximum, sum) pair per
// row and half tile of classes, then one wave per row merges the pairs. A
// lane of the MFMA result holds four consecutive classes of one row, so the
// reduction is in registers but for two exchanges between lanes.
//
// Gradients: per piece of the classes the same product again, its epilogue
// writing g in bf16 both row-major (for dx) and transposed (for dw; a 4x4
// exchange within quads of lanes makes its stores vectors), then the two
// products. Computing the logits twice costs 2 of 8 products' worth of
// operations; the alternative, keeping e^(s - m) of each tile from the first
// pass, rounds twice to bf16 and stores rows * classes values all the same.
// What bounds it: the matrix cores at large sizes, launches at small ones.
#include "gemm_nt.h"
#include "train.h"

namespace convnhwc {
namespace {

constexpr int kMaxSplit = 16;

__device__ __forceinline__ int label_at(const void* labels, int bytes, int64_t r, int64_t classes) {
  const int64_t l = bytes == 8 ? static_cast<const int64_t*>(labels)[r] : static_cast<const int32_t*>(labels)[r];
  return l >= 0 && l < classes ? (int)l : -1;
}

// ---- copies ---------------------------------------------------------------------

// src [rows][c] -> dst [rows][cpad] (zero past c; not when null) and
// dst_t [c][pitch_t] (zero past rows; not when null), 64x64 tiles through
// LDS. With labels, rows that are left out become zeros: their x, NaN or
// not, then adds nothing to dw.
template <int VEC>
__global__ __launch_bounds__(256) void copy_kernel(const uint16_t* src, int64_t rows, int c, const void* labels,
                                                   int label_bytes, int64_t classes, uint16_t* dst, int cpad,
                                                   uint16_t* dst_t, int64_t pitch_t) {
  __shared__ uint16_t t[64][66];
  const int tid = threadIdx.x;
  const int c0 = blockIdx.x * 64;
  const int64_t r0 = (int64_t)blockIdx.y * 64;
  constexpr int PER = 64 / VEC;  // vectors per tile row
  for (int i = tid; i < 64 * PER; i += 256) {
    const int r = i / PER, k = (i % PER) * VEC;
    const int64_t row = r0 + r;
    uint16_t v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = 0;
    const bool in = row < rows && (!labels || label_at(labels, label_bytes, row, classes) >= 0);
    if constexpr (VEC == 8) {
      if (in && c0 + k < c) {
        const uint4 q = *reinterpret_cast<const uint4*>(src + row * c + c0 + k);
        __builtin_memcpy(v, &q, 16);
      }
      if (dst && row < rows && c0 + k < cpad) {
        uint4 q;
        __builtin_memcpy(&q, v, 16);
        *reinterpret_cast<uint4*>(dst + row * cpad + c0 + k) = q;
      }
    } else {
      if (in && c0 + k < c) v[0] = src[row * c + c0 + k];
      if (dst && row < rows && c0 + k < cpad) dst[row * cpad + c0 + k] = v[0];
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[r][k + j] = v[j];
  }
  if (!dst_t) return;
  __syncthreads();
  for (int i = tid; i < 64 * 8; i += 256) {
    const int k = i / 8, r = (i % 8) * 8;
    if (c0 + k >= c || r0 + r >= pitch_t) continue;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = t[r + j][k];
    uint4 q;
    __builtin_memcpy(&q, v, 16);
    *reinterpret_cast<uint4*>(dst_t + (int64_t)(c0 + k) * pitch_t + r0 + r) = q;
  }
}

// ---- forward ----------------------------------------------------------------------

struct StatEpi {
  static constexpr bool kSymmetric = false;
  struct Args {
    float2* stat;  // [rows][slots]
    float* lab;    // [rows]: the label's logit
    const void* labels;
    int label_bytes, rows, classes, slots;
  };
  template <int TQ, int TP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[TQ / 32][TP / 32], const TileAt& at, const Args& e) {
    constexpr int FQ = TQ / 32, FP = TP / 32;
    const int slot = (at.tq / TQ) * 2 + at.wq;
    const bool ragged = at.tq + TQ > e.classes;
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      const int lab = r < e.rows ? label_at(e.labels, e.label_bytes, r, e.classes) : -1;
      if (ragged) {
#pragma unroll
        for (int i = 0; i < FQ; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (at.q0 + 16 * i + k >= e.classes) acc[i][j][k] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < FQ; ++i) m = fmaxf(fmaxf(m, fmaxf(acc[i][j][0], acc[i][j][1])), fmaxf(acc[i][j][2], acc[i][j][3]));
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      // a run without a finite value has no exponentials to sum
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < FQ; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s += __expf(acc[i][j][k] - base);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (r < e.rows) {
        if (at.lane < 16) e.stat[(int64_t)r * e.slots + slot] = float2{m, s};
        const int d = lab - at.q0;  // this lane's classes: q0 + 16 i + 0..3
        if (lab >= 0 && d >= 0 && d < 16 * FQ && (d & 15) < 4) {
          float v = 0.0f;
#pragma unroll
          for (int i = 0; i < FQ; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (d == 16 * i + k) v = acc[i][j][k];
          e.lab[r] = v;
        }
      }
    });
  }
};

// One wave per row: the slots' pairs to lse and loss.
__global__ __launch_bounds__(256) void rows_kernel(const float2* stat, int slots, const float* lab,
                                                   const void* labels, int label_bytes, int64_t rows, int64_t classes,
                                                   float* lse, float* loss) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;
  const float2* q = stat + r * slots;
  float m = -INFINITY;
  for (int i = lane; i < slots; i += 64) m = fmaxf(m, q[i].x);
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
  for (int i = lane; i < slots; i += 64) s += q[i].y * __expf(q[i].x - base);
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) s += __shfl_xor(s, k);
  if (lane == 0) {
    const float ls = logf(s);
    const bool kept = label_at(labels, label_bytes, r, classes) >= 0;
    if (lse) lse[r] = base + ls;
    loss[r] = kept ? ls - (lab[r] - base) : 0.0f;
  }
}

// One workgroup: the count of rows that are not left out, every row's weight
// and the weighted total (64-bit partial sums, a fixed order).
__global__ __launch_bounds__(1024) void total_kernel(const void* labels, int label_bytes, int64_t rows,
                                                     int64_t classes, const float* weights, const float* loss,
                                                     float* scale, float* total) {
  __shared__ double sum[16];
  __shared__ int cnt[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n = 0;
  double t = 0.0;
  for (int64_t r = tid; r < rows; r += 1024) {
    const bool kept = label_at(labels, label_bytes, r, classes) >= 0;
    n += kept;
    if (kept) t += (double)loss[r] * (weights ? (double)weights[r] : 1.0);
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) {
    n += __shfl_xor(n, k);
    t += __shfl_xor(t, k);
  }
  if (lane == 0) {
    sum[wave] = t;
    cnt[wave] = n;
  }
  __syncthreads();
  n = 0;
  t = 0.0;
  for (int i = 0; i < 16; ++i) {
    n += cnt[i];
    t += sum[i];
  }
  const double inv = 1.0 / (double)max(n, 1);
  if (tid == 0) total[0] = (float)(weights ? t : t * inv);
  if (scale) {
    for (int64_t r = tid; r < rows; r += 1024) {
      const bool kept = label_at(labels, label_bytes, r, classes) >= 0;
      scale[r] = kept ? (weights ? weights[r] : (float)inv) : 0.0f;
    }
  }
}

// ---- gradients -----------------------------------------------------------------

struct GradEpi {
  static constexpr bool kSymmetric = false;
  struct Args {
    const float* lse;
    const float* scale;
    const void* labels;
    int label_bytes;
    int rows, classes;   // of the whole problem
    int v0, nv;          // the piece: classes v0 .. v0 + nv - 1
    uint16_t* ds;        // [rows][vp]
    uint16_t* dst;       // [vp][rpad]
    int64_t vp, rpad;
  };
  template <int TQ, int TP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[TQ / 32][TP / 32], const TileAt& at, const Args& e) {
    constexpr int FQ = TQ / 32, FP = TP / 32;
    const bool ragged = at.tq + TQ > e.nv;
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      float lse = 0.0f, k = 0.0f;
      int d = -1;
      if (r < e.rows) {
        k = e.scale[r];
        lse = e.lse[r];
        const int lab = label_at(e.labels, e.label_bytes, r, e.classes);
        d = lab >= 0 ? lab - e.v0 - at.q0 : -1;
      }
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        float g[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          g[z] = __expf(acc[i][j][z] - lse);
          if (d == 16 * i + z) g[z] -= 1.0f;
          g[z] *= k;
          // rows past the last, rows left out and classes past the last: zeros
          if (k == 0.0f || (ragged && at.q0 + 16 * i + z >= e.nv)) g[z] = 0.0f;
        }
        const uint2 v = {bf16x2_bits(g[0], g[1]), bf16x2_bits(g[2], g[3])};
        const int q = at.q0 + 16 * i;
        if (r < e.rows) *reinterpret_cast<uint2*>(e.ds + (int64_t)r * e.vp + q) = v;
        const uint2 t = quad_transpose(v, at.lane);
        if ((r & ~3) < e.rpad)
          *reinterpret_cast<uint2*>(e.dst + (int64_t)(q + (at.lane & 3)) * e.rpad + (r & ~3)) = t;
      });
    });
  }
};

// bf16 out [p][q] (pitch c).
struct StoreEpi {
  static constexpr bool kSymmetric = false;
  struct Args {
    uint16_t* out;
    int rows, c;
    int vec;  // c % 4 == 0 and out 8-byte aligned
  };
  template <int TQ, int TP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[TQ / 32][TP / 32], const TileAt& at, const Args& e) {
    StaticFor<0, TP / 32>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      if (r >= e.rows) return;
      StaticFor<0, TQ / 32>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        uint16_t* o = e.out + (int64_t)r * e.c + q;
        const f32x4 v = acc[i][j];
        if (e.vec) {
          if (q < e.c) *reinterpret_cast<uint2*>(o) = uint2{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
        } else {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (q + z < e.c) o[z] = f32_to_bf16_bits(v[z]);
        }
      });
    });
  }
};

// fp32 partial sums [split][p][cq], added to what an earlier piece left.
struct PartEpi {
  static constexpr bool kSymmetric = false;
  struct Args {
    float* part;
    int64_t split_stride;
    int rows, cq;
    int add;
  };
  template <int TQ, int TP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[TQ / 32][TP / 32], const TileAt& at, const Args& e) {
    float* base = e.part + at.split * e.split_stride;
    StaticFor<0, TP / 32>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      if (r >= e.rows) return;
      StaticFor<0, TQ / 32>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        if (q >= e.cq) return;
        f32x4* o = reinterpret_cast<f32x4*>(base + (int64_t)r * e.cq + q);
        *o = e.add ? *o + acc[i][j] : acc[i][j];
      });
    });
  }
};

// out [rows][c] bf16 = the splits' sums, added in split order.
__global__ __launch_bounds__(256) void part_sum_kernel(const float* part, int64_t split_stride, int splits,
                                                       int64_t rows, int c, int cq, uint16_t* out, int vec) {
  const int64_t quads = rows * (cq / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 v[kMaxSplit];
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k)
      if (k < splits) v[k] = *reinterpret_cast<const f32x4*>(part + k * split_stride + 4 * i);
    f32x4 s = v[0];
#pragma unroll
    for (int k = 1; k < kMaxSplit; ++k)
      if (k < splits) s += v[k];
    const int64_t r = i / (cq / 4);
    const int q = (int)(i - r * (cq / 4)) * 4;
    uint16_t* o = out + r * c + q;
    if (vec) {
      *reinterpret_cast<uint2*>(o) = uint2{bf16x2_bits(s[0], s[1]), bf16x2_bits(s[2], s[3])};
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (q + z < c) o[z] = f32_to_bf16_bits(s[z]);
    }
  }
}

// Tile and splits of a product: whole reductions where the tiles fill the
// chip, else splits of at least 8 K-tiles (512 values of K).
GemmShape shape_for(int64_t q, int64_t p, int64_t k) {
  auto tiles = [&](int t) { return (int64_t)cdiv(q, t) * cdiv(p, t); };
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxSplit, k / 512));
  if (tiles(256) >= 192) return {256, 1};
  if (tiles(128) * most >= 128) return {128, (int)std::min<int64_t>(most, cdiv(512, tiles(128)))};
  return {64, (int)std::min<int64_t>(most, cdiv(512, tiles(64)))};
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace

HeadPlan head_plan(const conv_head_desc& d, bool grad, bool copy_x, bool copy_w) {
  HeadPlan p = {};
  const int64_t rows = d.rows, c = d.c, v = d.classes;
  p.cpad = up(c, 8);
  p.rpad = up(rows, 64);
  p.vpad = up(v, 64);
  p.cq = up(c, 4);
  p.stat_tile = gemm_tile(v, rows, 1, false);
  p.slots = 2 * cdiv(v, p.stat_tile);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  p.o_stat = take(rows * p.slots * 8);
  p.o_lab = take(rows * 4);
  p.o_lse = p.o_scale = p.o_x = p.o_w = p.o_xt = p.o_wt = p.o_ds = p.o_dst = p.o_dxp = p.o_dwp = -1;
  // the gradient reads x with the rows left out as zeros: always a copy
  if (grad || copy_x) p.o_x = take(rows * p.cpad * 2);
  if (copy_w) p.o_w = take(v * p.cpad * 2);
  if (grad) {
    p.o_lse = take(rows * 4);
    p.o_scale = take(rows * 4);
    p.o_xt = take(c * p.rpad * 2);
    p.o_wt = take(c * p.vpad * 2);
    // pieces of at most 512 MiB of g (and as much transposed)
    p.vp = std::min(up(v, 256), std::max<int64_t>(256, ((int64_t)1 << 28) / p.rpad / 256 * 256));
    const bool pieces = p.vp < v;
    const int64_t pv = std::min(p.vp, v);
    p.ds_tile = gemm_tile(pv, rows, 1, false);
    p.dx = shape_for(c, rows, pv);
    p.dw = shape_for(c, pv, rows);
    p.o_ds = take(rows * p.vp * 2);
    p.o_dst = take(p.vp * p.rpad * 2);
    if (pieces || p.dx.splits > 1) p.o_dxp = take(p.dx.splits * rows * p.cq * 4);
    if (p.dw.splits > 1) p.o_dwp = take(p.dw.splits * pv * p.cq * 4);
  }
  p.bytes = at;
  return p;
}

namespace {

hipError_t launch_copy(const uint16_t* src, int64_t rows, int64_t c, const HeadArgs* mask, uint16_t* dst,
                       int64_t cpad, uint16_t* dst_t, int64_t pitch_t, hipStream_t s) {
  const dim3 grid(cdiv(cpad, 64), cdiv(dst_t ? pitch_t : rows, 64));
  const void* labels = mask ? mask->labels : nullptr;
  const int lb = mask ? mask->label_bytes : 4;
  const int64_t cls = mask ? mask->classes : 0;
  if (c % 8 == 0 && ((uintptr_t)src & 15) == 0)
    hipLaunchKernelGGL(copy_kernel<8>, grid, dim3(256), 0, s, src, rows, (int)c, labels, lb, cls, dst, (int)cpad,
                       dst_t, pitch_t);
  else
    hipLaunchKernelGGL(copy_kernel<1>, grid, dim3(256), 0, s, src, rows, (int)c, labels, lb, cls, dst, (int)cpad,
                       dst_t, pitch_t);
  return hipGetLastError();
}

hipError_t launch_part_sum(const float* part, int64_t stride, int splits, int64_t rows, int64_t c, int64_t cq,
                           uint16_t* out, int vec, hipStream_t s) {
  const int blocks = (int)std::min<int64_t>((rows * (cq / 4) + 255) / 256, 4096);
  hipLaunchKernelGGL(part_sum_kernel, dim3(blocks), dim3(256), 0, s, part, stride, splits, rows, (int)c, (int)cq, out,
                     vec);
  return hipGetLastError();
}

}  // namespace

#define CONV_TRY(call)                        \
  do {                                        \
    const hipError_t try_err = (call);        \
    if (try_err != hipSuccess) return try_err; \
  } while (0)

hipError_t launch_head_loss(const HeadArgs& a, bool grad, hipStream_t s) {
  const HeadPlan& p = a.p;
  auto at = [&](int64_t o) { return a.ws + o; };
  const uint16_t* x = a.x;
  const uint16_t* w = a.w;
  uint16_t* xt = grad ? reinterpret_cast<uint16_t*>(at(p.o_xt)) : nullptr;
  uint16_t* wt = grad ? reinterpret_cast<uint16_t*>(at(p.o_wt)) : nullptr;
  if (p.o_x >= 0) {
    uint16_t* xc = reinterpret_cast<uint16_t*>(at(p.o_x));
    CONV_TRY(launch_copy(a.x, a.rows, a.c, grad ? &a : nullptr, xc, p.cpad, xt, p.rpad, s));
    x = xc;
  }
  if (p.o_w >= 0 || grad) {
    uint16_t* wc = p.o_w >= 0 ? reinterpret_cast<uint16_t*>(at(p.o_w)) : nullptr;
    CONV_TRY(launch_copy(a.w, a.classes, a.c, nullptr, wc, p.cpad, wt, p.vpad, s));
    if (wc) w = wc;
  }
  // x and w read in place have c % 8 == 0, so cpad is their pitch too
  GemmArgs g = {};
  g.a = reinterpret_cast<const char*>(w);
  g.b = reinterpret_cast<const char*>(x);
  g.a_pitch = g.b_pitch = g.kbytes = (int)p.cpad * 2;
  g.q = (int)a.classes;
  g.p = (int)a.rows;
  float* lab = reinterpret_cast<float*>(at(p.o_lab));
  float2* stat = reinterpret_cast<float2*>(at(p.o_stat));
  float* lse = grad ? reinterpret_cast<float*>(at(p.o_lse)) : nullptr;
  float* scale = grad ? reinterpret_cast<float*>(at(p.o_scale)) : nullptr;
  const StatEpi::Args se = {stat, lab, a.labels, a.label_bytes, (int)a.rows, (int)a.classes, p.slots};
  CONV_TRY((gemm_launch<BF16, StatEpi>(g, se, p.stat_tile, 1, 1, s)));
  hipLaunchKernelGGL(rows_kernel, dim3(cdiv(a.rows, 4)), dim3(256), 0, s, stat, p.slots, lab, a.labels, a.label_bytes,
                     a.rows, a.classes, lse, a.loss);
  CONV_TRY(hipGetLastError());
  hipLaunchKernelGGL(total_kernel, dim3(1), dim3(1024), 0, s, a.labels, a.label_bytes, a.rows, a.classes, a.weights,
                     a.loss, scale, a.total);
  CONV_TRY(hipGetLastError());
  if (!grad) return hipSuccess;

  uint16_t* ds = reinterpret_cast<uint16_t*>(at(p.o_ds));
  uint16_t* dst = reinterpret_cast<uint16_t*>(at(p.o_dst));
  const int vec_dx = a.c % 4 == 0 && ((uintptr_t)a.dx & 7) == 0;
  const int vec_dw = a.c % 4 == 0 && ((uintptr_t)a.dw & 7) == 0;
  const int64_t dx_stride = a.rows * p.cq;
  for (int64_t v0 = 0; v0 < a.classes; v0 += p.vp) {
    const int64_t nv = std::min(p.vp, a.classes - v0);
    GemmArgs gg = g;
    gg.a = reinterpret_cast<const char*>(w + v0 * p.cpad);
    gg.q = (int)nv;
    const GradEpi::Args ge = {lse, scale, a.labels, a.label_bytes, (int)a.rows, (int)a.classes, (int)v0, (int)nv, ds,
                              dst, p.vp, p.rpad};
    CONV_TRY((gemm_launch<BF16, GradEpi>(gg, ge, p.ds_tile, 1, 1, s)));
    // dx [rows][c] (+)= ds . (wt piece)^T
    GemmArgs gx = {};
    gx.a = reinterpret_cast<const char*>(wt + v0);
    gx.b = reinterpret_cast<const char*>(ds);
    gx.a_pitch = (int)p.vpad * 2;
    gx.b_pitch = (int)p.vp * 2;
    gx.kbytes = (int)up(nv, 8) * 2;
    gx.q = (int)a.c;
    gx.p = (int)a.rows;
    if (p.o_dxp >= 0) {
      const PartEpi::Args pe = {reinterpret_cast<float*>(at(p.o_dxp)), dx_stride, (int)a.rows, (int)p.cq, v0 > 0};
      CONV_TRY((gemm_launch<BF16, PartEpi>(gx, pe, p.dx.tile, p.dx.splits, 1, s)));
    } else {
      const StoreEpi::Args st = {a.dx, (int)a.rows, (int)a.c, vec_dx};
      CONV_TRY((gemm_launch<BF16, StoreEpi>(gx, st, p.dx.tile, 1, 1, s)));
    }
    // dw piece [nv][c] = dst . xt^T
    GemmArgs gw = {};
    gw.a = reinterpret_cast<const char*>(xt);
    gw.b = reinterpret_cast<const char*>(dst);
    gw.a_pitch = gw.b_pitch = (int)p.rpad * 2;
    gw.kbytes = (int)up(a.rows, 8) * 2;
    gw.q = (int)a.c;
    gw.p = (int)nv;
    uint16_t* dw = a.dw + v0 * a.c;
    if (p.o_dwp >= 0) {
      float* part = reinterpret_cast<float*>(at(p.o_dwp));
      const int64_t stride = std::min(p.vp, a.classes) * p.cq;
      const PartEpi::Args pe = {part, stride, (int)nv, (int)p.cq, 0};
      CONV_TRY((gemm_launch<BF16, PartEpi>(gw, pe, p.dw.tile, p.dw.splits, 1, s)));
      CONV_TRY(launch_part_sum(part, stride, p.dw.splits, nv, a.c, p.cq, dw, vec_dw, s));
    } else {
      const StoreEpi::Args st = {dw, (int)nv, (int)a.c, vec_dw};
      CONV_TRY((gemm_launch<BF16, StoreEpi>(gw, st, p.dw.tile, 1, 1, s)));
    }
  }
  if (p.o_dxp >= 0)
    CONV_TRY(launch_part_sum(reinterpret_cast<float*>(at(p.o_dxp)), dx_stride, p.dx.splits, a.rows, a.c, p.cq, a.dx,
                             vec_dx, s));
  return hipSuccess;
}

}  // namespace convnhwc
