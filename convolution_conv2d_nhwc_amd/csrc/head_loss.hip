// head_loss.hip -- softmax cross entropy of a 1x1 head over a large set of
// classes, and its gradients, without storing the logits.
//
// Mathematics. s[r][v] = x[r] . w[v]; with the row's maximum m and
// sum = sum_v e^(s - m): loss = log(sum) - (s[label] - m), and with
// lse = m + log(sum) and the row's weight k:
//   g[r][v] = k (e^(s - lse) - [v == label]),  dx = g w,  dw = g^T x.
// Exponentials run in base 2 (e^s = 2^(s L), L = log2 e, one fused multiply-add
// and one instruction a value); m and lse are kept in those units too, so that
// the rounding of m L cancels out of every term.
//
// Forward: one matrix product whose epilogue keeps a (maximum, sum) pair per
// row and wave's run of classes, then a reduction over the row's pairs. A
// lane of the MFMA result holds four consecutive classes of one row, so the
// epilogue's reduction is in registers but for two exchanges between lanes.
//
// Gradients: per piece of the classes the same product again, its epilogue
// writing g in bf16, then the two products, which read g, w and x as they lie
// (see gemm.h: no transposed copies). Computing the logits twice costs 2 of 8
// products' worth of operations; the alternative, keeping e^(s - m) of each
// tile from the first pass, rounds twice to bf16 and stores rows * classes
// values all the same.
//
// What bounds it: the matrix cores at large sizes (6400 x 1024 x 65536, all
// gradients: 3.15 ms, of which logits 0.78, logits again with g 0.92, dx 0.76, dw
// 0.66 ms), the fixed cost of eight launches at small ones (1521 x 250 x 10007:
// 92 us as a call, 99 us of kernels under a profiler).
//
// Precision. Rounding g to bf16 would cost as much as the rounding of the
// results, nearly all of it from the one large entry of a row, its label's.
// What that rounding left out, delta[r], is kept in fp32 and put back: in dx as
// delta[r] w[label] in the epilogue, in dw as the product's sparse term.
#include <cstdio>

#include "gemm.h"
#include "train.h"

namespace convnhwc {
namespace {

constexpr int kMaxSplit = 16;
constexpr float kLog2e = 1.44269504088896f;

__device__ __forceinline__ float exp2_f32(float v) { return __builtin_amdgcn_exp2f(v); }

__device__ __forceinline__ int label_at(const void* labels, int bytes, int64_t r, int64_t classes) {
  const int64_t l = label_raw(labels, bytes, r);
  return l >= 0 && l < classes ? (int)l : -1;
}

// ---- copies ---------------------------------------------------------------------

// src [rows][c] -> dst [rows][cpad], zeros past c, eight values a lane. With
// labels, rows that are left out become zeros: their x, NaN or not, then
// adds nothing to dw.
__device__ __forceinline__ void pad_chunk(const uint16_t* src, int64_t row, int c, int chunk, bool keep, uint16_t* dst,
                                          int cpad) {
  const uint16_t* p = src + row * c + chunk * 8;
  const int left = keep ? c - chunk * 8 : 0;
  uint16_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : (uint16_t)0;
  uint4 q;
  __builtin_memcpy(&q, v, 16);
  *reinterpret_cast<uint4*>(dst + row * cpad + chunk * 8) = q;
}

// x (nx rows, labels) and w (nw rows) in one launch; a count of 0 leaves one out.
__global__ __launch_bounds__(256) void pad_kernel(const uint16_t* x, int64_t nx, const void* labels, int label_bytes,
                                                  int64_t classes, uint16_t* xd, const uint16_t* w, int64_t nw,
                                                  uint16_t* wd, int c, int cpad) {
  const int chunks = cpad / 8;
  const int64_t total = (nx + nw) * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / chunks;
    const int k = (int)(i - row * chunks);
    if (row < nx)
      pad_chunk(x, row, c, k, label_at(labels, label_bytes, row, classes) >= 0, xd, cpad);
    else
      pad_chunk(w, row - nx, c, k, true, wd, cpad);
  }
}

// What an epilogue reads of a row (one p), besides the accumulators: before
// the product where a lane has one row.
template <int FP, class Epi>
struct RowPre {
  typename Epi::Row first;
  __device__ __forceinline__ void load(const TileAt& at, const typename Epi::Args& e) {
    if constexpr (FP == 1) first.load(at, e, 0);
  }
  __device__ __forceinline__ typename Epi::Row row(const TileAt& at, const typename Epi::Args& e, int j) const {
    if constexpr (FP == 1) return first;
    typename Epi::Row r;
    r.load(at, e, j);
    return r;
  }
};

// ---- forward ----------------------------------------------------------------------

struct StatEpi {
  static constexpr bool kSymmetric = false, kSparse = false;
  struct Args {
    float2* stat;  // [rows][slots]: (m L, sum 2^(s L - m L)) of the slot's classes
    float* lab;    // [rows]: the label's logit
    const void* labels;
    int label_bytes, rows, classes, slots;
  };
  struct Row {
    int label;
    __device__ __forceinline__ void load(const TileAt& at, const Args& e, int j) {
      const int r = at.p0 + 16 * j;
      label = r < e.rows ? label_at(e.labels, e.label_bytes, r, e.classes) : -1;
    }
  };
  template <int FQ, int FP>
  using Pre = RowPre<FP, StatEpi>;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e,
                                             const Pre<FQ, FP>& pre) {
    if (at.wq + 16 * FQ > e.classes)
      rows_of<FQ, FP, true>(acc, at, e, pre);
    else
      rows_of<FQ, FP, false>(acc, at, e, pre);
  }
  template <int FQ, int FP, bool RAGGED>
  static __device__ __forceinline__ void rows_of(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e,
                                                 const Pre<FQ, FP>& pre) {
    const int slot = at.wq / (16 * FQ);
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      asm volatile("" ::: "memory");  // one row at a time: keeps the registers within bounds
      const int r = at.p0 + 16 * j;
      auto val = [&](int i, int k) {
        return RAGGED && at.q0 + 16 * i + k >= e.classes ? -INFINITY : acc[i][j][k];
      };
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < FQ; ++i) m = fmaxf(fmaxf(fmaxf(fmaxf(m, val(i, 0)), val(i, 1)), val(i, 2)), val(i, 3));
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      // a run without a finite value has no exponentials to sum
      const float base = m == -INFINITY ? 0.0f : m * kLog2e;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < FQ; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s += exp2_f32(__builtin_fmaf(val(i, k), kLog2e, -base));
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (r < e.rows) {
        if (at.lane < 16) e.stat[(int64_t)r * e.slots + slot] = float2{m == -INFINITY ? m : base, s};
        // the label's logit, where it is one of this lane's: q0 + 16 i + 0..3
        const int d = pre.row(at, e, j).label - at.q0;
        if (d >= 0 && d < 16 * FQ && (d & 15) < 4) {
          float u = 0.0f;
#pragma unroll
          for (int i = 0; i < FQ; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (d == 16 * i + k) u = acc[i][j][k];
          e.lab[r] = u;
        }
      }
    });
  }
};

struct FinishArgs {
  const float2* stat;
  const float* lab;
  const void* labels;
  const float* weights;
  const uint16_t* x;  // to be copied to xd, rows left out as zeros; null: not
  uint16_t* xd;
  float* lse;   // null without gradients
  float* loss;
  float* inv;   // 1 / rows not left out; null without gradients
  float* total;
  int64_t rows, classes;
  int slots, label_bytes, c;
};

// One row's loss and lse from its sum over the classes (in units of 2^base).
__device__ __forceinline__ float row_loss(const FinishArgs& a, int64_t r, float base, float s, float lab, bool kept,
                                          bool store) {
  const float ls = __log2f(s);
  const float loss = kept ? (ls - __builtin_fmaf(lab, kLog2e, -base)) * 0.693147180559945f : 0.0f;
  if (store) {
    a.loss[r] = loss;
    // a left out row's logits are zeros in the gradient's product: 2^(0 - 0), times 0
    if (a.lse) a.lse[r] = kept ? base + ls : 0.0f;
  }
  return loss;
}

// One wave per row.
__global__ __launch_bounds__(256) void rows_kernel(FinishArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  const bool kept = label_at(a.labels, a.label_bytes, r, a.classes) >= 0;
  if (a.x)
    for (int k = lane; k < a.c / 8; k += 64)
      reinterpret_cast<uint4*>(a.xd + r * a.c)[k] =
          kept ? reinterpret_cast<const uint4*>(a.x + r * a.c)[k] : uint4{0, 0, 0, 0};
  const float2* q = a.stat + r * a.slots;
  float m = -INFINITY;
  for (int i = lane; i < a.slots; i += 64) m = fmaxf(m, q[i].x);
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
  for (int i = lane; i < a.slots; i += 64) s += q[i].y * exp2_f32(q[i].x - base);
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) s += __shfl_xor(s, k);
  row_loss(a, r, base, s, kept ? a.lab[r] : 0.0f, kept, lane == 0);
}

// The weighted total and the count from the lanes' sums (64-bit, a fixed order).
__device__ __forceinline__ void total_store(const FinishArgs& a, double t, int n, double* sum, int* cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
  if (wave) return;
  n = lane < 16 ? cnt[lane] : 0;
  t = lane < 16 ? sum[lane] : 0.0;
#pragma unroll
  for (int k = 8; k >= 1; k >>= 1) {
    n += __shfl_xor(n, k);
    t += __shfl_xor(t, k);
  }
  if (lane == 0) {
    const double inv = 1.0 / (double)max(n, 1);
    a.total[0] = (float)(a.weights ? t : t * inv);
    if (a.inv) a.inv[0] = (float)inv;
  }
}

__global__ __launch_bounds__(1024) void total_kernel(FinishArgs a) {
  __shared__ double sum[16];
  __shared__ int cnt[16];
  int n = 0;
  double t = 0.0;
#pragma unroll 4
  for (int64_t r = threadIdx.x; r < a.rows; r += 1024) {
    const bool kept = label_at(a.labels, a.label_bytes, r, a.classes) >= 0;
    const double l = a.loss[r], w = a.weights ? a.weights[r] : 1.0f;
    n += kept;
    t += kept ? l * w : 0.0;
  }
  total_store(a, t, n, sum, cnt);
}

// Few rows with few pairs: everything in one launch, the rows in the first
// workgroup (eight lanes each, up to four rows, all loads before the first
// use: one latency), the copy of x in the others.
constexpr int kFinishRows = 512, kFinishSlots = 64;

__global__ __launch_bounds__(1024) void finish_kernel(FinishArgs a) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int chunks = a.c / 8;
    const int i = (blockIdx.x - 1) * 1024 + tid;
    if (i < (int)a.rows * chunks)
      reinterpret_cast<uint4*>(a.xd)[i] = label_at(a.labels, a.label_bytes, i / chunks, a.classes) >= 0
                                              ? reinterpret_cast<const uint4*>(a.x)[i]
                                              : uint4{0, 0, 0, 0};
    return;
  }
  __shared__ double sum[16];
  __shared__ int cnt[16];
  constexpr int N = kFinishRows / 128, S = kFinishSlots / 8;
  const int rows = (int)a.rows, sub = tid & 7;
  int label[N];
  float w[N], lab[N];
  float2 q[N][S];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int r = (tid >> 3) + 128 * u;
    label[u] = r < rows ? label_at(a.labels, a.label_bytes, r, a.classes) : -1;
    w[u] = r < rows && a.weights ? a.weights[r] : 1.0f;
    lab[u] = r < rows ? a.lab[r] : 0.0f;  // of a row left out: not set, not used
#pragma unroll
    for (int i = 0; i < S; ++i)
      q[u][i] = r < rows && sub + 8 * i < a.slots ? a.stat[(int64_t)r * a.slots + sub + 8 * i] : float2{-INFINITY, 0.0f};
  }
  int n = 0;
  double t = 0.0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int r = (tid >> 3) + 128 * u;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) m = fmaxf(m, q[u][i].x);
#pragma unroll
    for (int k = 4; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
    const float base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) s += q[u][i].y * exp2_f32(q[u][i].x - base);
#pragma unroll
    for (int k = 4; k >= 1; k >>= 1) s += __shfl_xor(s, k);
    const bool kept = label[u] >= 0;
    const float loss = row_loss(a, r, base, s, lab[u], kept, sub == 0 && r < rows);
    if (sub == 0 && kept) {
      ++n;
      t += (double)loss * w[u];
    }
  }
  total_store(a, t, n, sum, cnt);
}

// ---- gradients -----------------------------------------------------------------

struct GradEpi {
  static constexpr bool kSymmetric = false, kSparse = false;
  struct Args {
    const float* lse;
    const float* weights;
    const float* inv;
    const void* labels;
    int label_bytes;
    int rows, classes;   // of the whole problem
    int v0, nv;          // the piece: classes v0 .. v0 + nv - 1
    uint16_t* ds;        // [rows][vp]
    float* delta;        // [rows]
    int64_t vp;
  };
  // rows past the last and rows left out: logits 0, lse 0, weight 0
  struct Row {
    float lse, k;
    int d;  // the label, from the wave's first class
    __device__ __forceinline__ void load(const TileAt& at, const Args& e, int j) {
      const int r = at.p0 + 16 * j;
      lse = k = 0.0f;
      d = -1;
      if (r >= e.rows) return;
      const int lab = label_at(e.labels, e.label_bytes, r, e.classes);
      lse = e.lse[r];
      if (lab >= 0) {
        k = e.weights ? e.weights[r] : e.inv[0];
        d = lab - e.v0 - at.wq;
      }
    }
  };
  template <int FQ, int FP>
  using Pre = RowPre<FP, GradEpi>;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e,
                                             const Pre<FQ, FP>& pre) {
    const bool ragged = at.wq + 16 * FQ > e.nv;
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      const Row in = pre.row(at, e, j);
      const float lse = in.lse, k = in.k;
      int d = in.d;
      const Rows<FQ> rows(at.lane);
      rows.fence();
      if (ragged || __any(d >= 0 && d < 16 * FQ)) {
        d -= at.q0 - at.wq;
        StaticFor<0, FQ>::run([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          float g[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const bool hit = d == 16 * i + z;
            g[z] = exp2_f32(__builtin_fmaf(acc[i][j][z], kLog2e, -lse));
            if (hit) g[z] -= 1.0f;
            g[z] *= k;
            if (at.q0 + 16 * i + z >= e.nv) g[z] = 0.0f;
            if (hit) e.delta[r] = g[z] - bf16_bits_to_f32(f32_to_bf16_bits(g[z]));
          }
          rows.put16(at, i, uint2{bf16x2_bits(g[0], g[1]), bf16x2_bits(g[2], g[3])});
        });
      } else {
        StaticFor<0, FQ>::run([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          float g[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) g[z] = k * exp2_f32(__builtin_fmaf(acc[i][j][z], kLog2e, -lse));
          rows.put16(at, i, uint2{bf16x2_bits(g[0], g[1]), bf16x2_bits(g[2], g[3])});
        });
      }
      rows.fence();
#pragma unroll
      for (int s = 0; s < rows.kPasses; ++s) {
        const int p = rows.p(at, j, s);
        if (p < e.rows) *reinterpret_cast<uint4*>(e.ds + (int64_t)p * e.vp + rows.q(at)) = rows.take16(at, s);
      }
    });
  }
};

// The label's part of dx that bf16 g left out, for the rows whose label is one
// of the piece's classes.
struct LabelTerm {
  const uint16_t* w;    // [classes][cpad]
  const void* labels;
  const float* delta;
  int label_bytes, classes, cpad;
  int v0, nv;
};

struct LabelRow {
  const uint16_t* w;
  float delta;
};
__device__ __forceinline__ LabelRow label_row(const LabelTerm& t, int r) {
  const int lab = label_at(t.labels, t.label_bytes, r, t.classes);
  const bool in = lab >= t.v0 && lab < t.v0 + t.nv;
  return {in ? t.w + (int64_t)lab * t.cpad : t.w, in ? t.delta[r] : 0.0f};
}
__device__ __forceinline__ f32x4 label_add(f32x4 v, const LabelRow& l, int q) {
  if (l.delta != 0.0f) {
    const uint2 u = *reinterpret_cast<const uint2*>(l.w + q);
    v[0] += l.delta * bf16_bits_to_f32(u.x & 0xffffu);
    v[1] += l.delta * bf16_bits_to_f32(u.x >> 16);
    v[2] += l.delta * bf16_bits_to_f32(u.y & 0xffffu);
    v[3] += l.delta * bf16_bits_to_f32(u.y >> 16);
  }
  return v;
}

// bf16 out [p][q] (pitch c). DX: with the label's term; else the product has a
// sparse term.
template <bool DX>
struct StoreEpi {
  static constexpr bool kSymmetric = false, kSparse = !DX;
  struct Args {
    uint16_t* out;
    int rows, c;
    int vec;  // c % 8 == 0 and out 16-byte aligned
    LabelTerm lt;
    SparseTerm st;
  };
  static __device__ __forceinline__ SparseTerm sparse(const Args& e) { return e.st; }
  template <int FQ, int FP>
  using Pre = NoPre;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e, NoPre) {
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      LabelRow l = {};
      if constexpr (DX)
        if (r < e.rows) l = label_row(e.lt, r);
      const Rows<FQ> rows(at.lane);
      rows.fence();
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        f32x4 v = acc[i][j];
        if constexpr (DX)
          if (q < e.c) v = label_add(v, l, q);
        rows.put16(at, i, uint2{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])});
      });
      rows.fence();
#pragma unroll
      for (int s = 0; s < rows.kPasses; ++s) {
        const int p = rows.p(at, j, s), q = rows.q(at);
        if (p >= e.rows || q >= e.c) continue;
        const uint4 v = rows.take16(at, s);
        uint16_t* o = e.out + (int64_t)p * e.c + q;
        if (e.vec) {
          *reinterpret_cast<uint4*>(o) = v;
        } else {
          uint16_t u[8];
          __builtin_memcpy(u, &v, 16);
#pragma unroll
          for (int z = 0; z < 8; ++z)
            if (q + z < e.c) o[z] = u[z];
        }
      }
    });
  }
};

// fp32 partial sums [split][p][cq], added to what an earlier piece left.
template <bool DX>
struct PartEpi {
  static constexpr bool kSymmetric = false, kSparse = !DX;
  struct Args {
    float* part;
    int64_t split_stride;
    int rows, cq;
    int add;
    LabelTerm lt;
    SparseTerm st;
  };
  static __device__ __forceinline__ SparseTerm sparse(const Args& e) { return e.st; }
  template <int FQ, int FP>
  using Pre = NoPre;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e, NoPre) {
    float* base = e.part + at.split * e.split_stride;
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int r = at.p0 + 16 * j;
      if (r >= e.rows) return;
      LabelRow l = {};
      if constexpr (DX)
        if (at.split == 0) l = label_row(e.lt, r);
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        if (q >= e.cq) return;
        f32x4* o = reinterpret_cast<f32x4*>(base + (int64_t)r * e.cq + q);
        f32x4 v = acc[i][j];
        if constexpr (DX) v = label_add(v, l, q);
        *o = e.add ? *o + v : v;
      });
    });
  }
};

struct DxProduct {
  static constexpr bool KSA = true, KSB = false;
  typedef StoreEpi<true> Epi;
};
struct DwProduct {
  static constexpr bool KSA = true, KSB = true;
  typedef StoreEpi<false> Epi;
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

// Tile and splits of a product of k values of K: the least of an estimate in us,
// rounds of workgroups times (K-tiles of 64 + what a tile costs besides), and
// for a split the writing and adding of its sums at 3.5 TB/s. The figures are
// measured ones: a K-tile of a 256 tile 1.65, of a 128 tile 0.8 alone on its CU
// and 1.3 beside another, of a 64 tile 0.3 and 0.5. (1521 x 250 x 10007: dx in ten
// splits of 128 tiles 20 us, dw in whole 128 tiles 25 us, in two splits 17 + 7;
// 6400 x 1024 x 32768: dx in five splits of 256 tiles 390 us, unsplit 128 tiles
// 690.)
GemmShape shape_for(int64_t q, int64_t p, int64_t k) {
  const int64_t kt = cdiv(k, kKV), most = std::max<int64_t>(1, std::min<int64_t>(kMaxSplit, k / 512));
  GemmShape best = {64, 1};
  double least = 1e30;
  for (int t = 64; t <= 256; t *= 2) {
    const int64_t tiles = gemm_tiles(q, p, t, false);
    for (int64_t s = 1; s <= most; ++s) {
      const bool alone = t == 256 || tiles * s <= 256;
      const double tile = t == 256 ? 1.65 : t == 128 ? (alone ? 0.8 : 1.3) : alone ? 0.3 : 0.5;
      const double fixed = t == 256 ? 8.0 : t == 128 ? (alone ? 6.0 : 8.0) : alone ? 4.5 : 6.0;
      double us = cdiv(tiles * s, alone ? 256 : 512) * (cdiv(kt, s) * tile + fixed);
      if (s > 1) us += 3.0 + 8.0 * s * q * p / 3.5e6;
      if (us < least) {
        least = us;
        best = {t, (int)s};
      }
    }
  }
  return best;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace

// Tile of the logits' products. Over few channels the epilogue is most of the
// work, and two workgroups a CU hide one's behind the other's product (with
// gradients, 128 / 256 tiles: 6400 x 128 x 30000 582 / 659 us, 4096 x 256 x
// 16384 318 / 338, 4096 x 512 x 16384 457 / 453).
static int logits_tile(int64_t classes, int64_t rows, int64_t c) {
  const int t = gemm_tile(classes, rows, 1, false);
  return t == 256 && c <= 256 ? 128 : t;
}

int64_t head_workgroups(const conv_head_desc& d) {
  return gemm_tiles(d.classes, d.rows, logits_tile(d.classes, d.rows, d.c), false);
}

HeadPlan head_plan(const conv_head_desc& d, bool grad, bool copy_x, bool copy_w) {
  HeadPlan p = {};
  const int64_t rows = d.rows, c = d.c, v = d.classes;
  p.cpad = up(c, 8);
  p.cq = up(c, 4);
  p.stat_tile = logits_tile(v, rows, c);
  p.slots = p.stat_tile == 64 ? cdiv(v, 64) : 2 * cdiv(v, p.stat_tile);  // one per wave along the classes
  p.copy_x = copy_x;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  p.o_stat = take(rows * p.slots * 8);
  p.o_lab = take(rows * 4);
  p.o_lse = p.o_inv = p.o_delta = p.o_x = p.o_w = p.o_ds = p.o_dxp = p.o_dwp = -1;
  // the gradient reads x with the rows left out as zeros: always a copy
  if (grad || copy_x) p.o_x = take(rows * p.cpad * 2);
  if (copy_w) p.o_w = take(v * p.cpad * 2);
  if (grad) {
    p.o_lse = take(rows * 4);
    p.o_delta = take(rows * 4);
    p.o_inv = take(4);
    // equal pieces of at most 512 MiB of g (or 256 classes)
    const int64_t most = std::max<int64_t>(256, ((int64_t)1 << 28) / rows / 256 * 256);
    p.vp = up(cdiv(v, cdiv(v, most)), 256);
    const bool pieces = p.vp < v;
    const int64_t pv = std::min(p.vp, v);
    p.ds_tile = logits_tile(pv, rows, c);
    p.dx = shape_for(c, rows, pv);
    p.dw = shape_for(c, pv, rows);
    // short products in few tiles: both in one launch
    p.pair = !pieces && p.dx.tile == 64 && p.dw.tile == 64 && p.dw.splits == 1 && pv <= 2048;
    if (p.pair) p.dx.splits = 1;
    p.o_ds = take(rows * p.vp * 2);
    if (pieces || p.dx.splits > 1) p.o_dxp = take(p.dx.splits * rows * p.cq * 4);
    if (p.dw.splits > 1) p.o_dwp = take(p.dw.splits * pv * p.cq * 4);
  }
  p.bytes = at;
  return p;
}

void head_describe(const conv_head_desc& d, bool grad, const HeadPlan& p, char* buf, int len) {
  auto per_cu = [](int64_t q, int64_t r, const GemmShape& g) { return gemm_deep(q, r, g.tile, g.splits, false) ? 1 : 2; };
  const int n = std::snprintf(buf, len, "head_loss%s logits=%dx%d slots=%d finish=%d copy_x=%d copy_w=%d",
                              grad ? "_grad" : "", p.stat_tile, per_cu(d.classes, d.rows, {p.stat_tile, 1}), p.slots,
                              d.rows <= kFinishRows && p.slots <= kFinishSlots ? 1 : 2, p.copy_x, p.o_w >= 0);
  if (!grad || n < 0 || n >= len) return;
  const int64_t pv = std::min(p.vp, d.classes);
  // a pair's products share a launch built for one workgroup a CU
  const int dx = p.pair ? 1 : per_cu(p.cpad, d.rows, p.dx), dw = p.pair ? 1 : per_cu(p.cpad, up(pv, 8), p.dw);
  std::snprintf(buf + n, len - n,
                " pieces=%d g=%dx%d pair=%d dx=%dx%d dx_splits=%d dx_part=%d dw=%dx%d dw_splits=%d dw_part=%d",
                cdiv(d.classes, p.vp), p.ds_tile, per_cu(pv, d.rows, {p.ds_tile, 1}), p.pair, p.dx.tile, dx,
                p.dx.splits, p.o_dxp >= 0, p.dw.tile, dw, p.dw.splits, p.o_dwp >= 0);
}

namespace {

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
  auto f32_at = [&](int64_t o) { return o < 0 ? nullptr : reinterpret_cast<float*>(a.ws + o); };
  const uint16_t* x = a.x;
  const uint16_t* w = a.w;
  uint16_t* xc = p.o_x >= 0 ? reinterpret_cast<uint16_t*>(at(p.o_x)) : nullptr;
  if (p.copy_x || p.o_w >= 0) {
    uint16_t* wc = p.o_w >= 0 ? reinterpret_cast<uint16_t*>(at(p.o_w)) : nullptr;
    const int64_t nx = p.copy_x ? a.rows : 0, nw = wc ? a.classes : 0;
    const int blocks = (int)std::min<int64_t>(((nx + nw) * (p.cpad / 8) + 255) / 256, 65536);
    hipLaunchKernelGGL(pad_kernel, dim3(blocks), dim3(256), 0, s, a.x, nx, a.labels, a.label_bytes, a.classes, xc, a.w,
                       nw, wc, (int)a.c, (int)p.cpad);
    CONV_TRY(hipGetLastError());
    if (p.copy_x) x = xc;
    if (wc) w = wc;
  }
  // x and w read in place have c % 8 == 0, so cpad is their pitch too
  GemmArgs g = {};
  g.a = reinterpret_cast<const char*>(w);
  g.b = reinterpret_cast<const char*>(x);
  g.a_pitch = g.b_pitch = (int)p.cpad * 2;
  g.k = (int)p.cpad;
  g.q = (int)a.classes;
  g.p = (int)a.rows;
  FinishArgs f = {};
  f.stat = reinterpret_cast<const float2*>(at(p.o_stat));
  f.lab = f32_at(p.o_lab);
  f.labels = a.labels;
  f.weights = a.weights;
  if (grad && !p.copy_x) {
    f.x = a.x;
    f.xd = xc;
  }
  f.lse = f32_at(p.o_lse);
  f.loss = a.loss;
  f.inv = f32_at(p.o_inv);
  f.total = a.total;
  f.rows = a.rows;
  f.classes = a.classes;
  f.slots = p.slots;
  f.label_bytes = a.label_bytes;
  f.c = (int)a.c;
  const StatEpi::Args se = {reinterpret_cast<float2*>(at(p.o_stat)), f32_at(p.o_lab), a.labels, a.label_bytes,
                            (int)a.rows, (int)a.classes, p.slots};
  CONV_TRY((gemm_launch<BF16, false, false, StatEpi>(g, se, p.stat_tile, 1, 1, s)));
  if (a.rows <= kFinishRows && p.slots <= kFinishSlots) {
    const int copies = f.x ? cdiv(a.rows * (a.c / 8), 1024) : 0;
    hipLaunchKernelGGL(finish_kernel, dim3(1 + copies), dim3(1024), 0, s, f);
  } else {
    hipLaunchKernelGGL(rows_kernel, dim3(cdiv(a.rows, 4)), dim3(256), 0, s, f);
    CONV_TRY(hipGetLastError());
    hipLaunchKernelGGL(total_kernel, dim3(1), dim3(1024), 0, s, f);
  }
  CONV_TRY(hipGetLastError());
  if (!grad) return hipSuccess;

  uint16_t* ds = reinterpret_cast<uint16_t*>(at(p.o_ds));
  float* delta = f32_at(p.o_delta);
  const int vec_dx = a.c % 8 == 0 && ((uintptr_t)a.dx & 15) == 0;
  const int vec_dw = a.c % 8 == 0 && ((uintptr_t)a.dw & 15) == 0;
  const int sum_vec_dx = a.c % 4 == 0 && ((uintptr_t)a.dx & 7) == 0;
  const int sum_vec_dw = a.c % 4 == 0 && ((uintptr_t)a.dw & 7) == 0;
  const int64_t dx_stride = a.rows * p.cq;
  for (int64_t v0 = 0; v0 < a.classes; v0 += p.vp) {
    const int64_t nv = std::min(p.vp, a.classes - v0);
    GemmArgs gg = g;
    gg.a = reinterpret_cast<const char*>(w + v0 * p.cpad);
    gg.b = reinterpret_cast<const char*>(xc);
    gg.q = (int)nv;
    const GradEpi::Args ge = {f.lse, a.weights, f.inv, a.labels, a.label_bytes, (int)a.rows, (int)a.classes, (int)v0,
                              (int)nv, ds, delta, p.vp};
    CONV_TRY((gemm_launch<BF16, false, false, GradEpi>(gg, ge, p.ds_tile, 1, 1, s)));
    const LabelTerm lt = {w, a.labels, delta, a.label_bytes, (int)a.classes, (int)p.cpad, (int)v0, (int)nv};
    const SparseTerm st = {a.labels, a.label_bytes, (int)v0, delta};
    // dx [rows][c] (+)= g . w of the piece
    GemmArgs gx = {};
    gx.a = gg.a;
    gx.b = reinterpret_cast<const char*>(ds);
    gx.a_pitch = (int)p.cpad * 2;
    gx.b_pitch = (int)p.vp * 2;
    gx.k = (int)nv;
    gx.q = (int)p.cpad;
    gx.p = (int)a.rows;
    // dw of the piece [nv][c] = g^T x
    GemmArgs gw = {};
    gw.a = reinterpret_cast<const char*>(xc);
    gw.b = reinterpret_cast<const char*>(ds);
    gw.a_pitch = (int)p.cpad * 2;
    gw.b_pitch = (int)p.vp * 2;
    gw.k = (int)a.rows;
    gw.q = (int)p.cpad;
    gw.p = (int)up(nv, 8);
    uint16_t* dw = a.dw + v0 * a.c;
    if (p.pair) {
      const StoreEpi<true>::Args ex = {a.dx, (int)a.rows, (int)a.c, vec_dx, lt, st};
      const StoreEpi<false>::Args ew = {dw, (int)nv, (int)a.c, vec_dw, lt, st};
      CONV_TRY((gemm_launch_pair<BF16, 64, DxProduct, DwProduct>(gx, ex, gw, ew, s)));
      continue;
    }
    if (p.o_dxp >= 0) {
      const PartEpi<true>::Args pe = {f32_at(p.o_dxp), dx_stride, (int)a.rows, (int)p.cq, v0 > 0, lt, st};
      CONV_TRY((gemm_launch<BF16, true, false, PartEpi<true>>(gx, pe, p.dx.tile, p.dx.splits, 1, s)));
    } else {
      const StoreEpi<true>::Args ee = {a.dx, (int)a.rows, (int)a.c, vec_dx, lt, st};
      CONV_TRY((gemm_launch<BF16, true, false, StoreEpi<true>>(gx, ee, p.dx.tile, 1, 1, s)));
    }
    if (p.o_dwp >= 0) {
      float* part = f32_at(p.o_dwp);
      const int64_t stride = std::min(p.vp, a.classes) * p.cq;
      const PartEpi<false>::Args pe = {part, stride, (int)nv, (int)p.cq, 0, lt, st};
      CONV_TRY((gemm_launch<BF16, true, true, PartEpi<false>>(gw, pe, p.dw.tile, p.dw.splits, 1, s)));
      CONV_TRY(launch_part_sum(part, stride, p.dw.splits, nv, a.c, p.cq, dw, sum_vec_dw, s));
    } else {
      const StoreEpi<false>::Args ee = {dw, (int)nv, (int)a.c, vec_dw, lt, st};
      CONV_TRY((gemm_launch<BF16, true, true, StoreEpi<false>>(gw, ee, p.dw.tile, 1, 1, s)));
    }
  }
  if (p.o_dxp >= 0)
    CONV_TRY(launch_part_sum(f32_at(p.o_dxp), dx_stride, p.dx.splits, a.rows, a.c, p.cq, a.dx, sum_vec_dx, s));
  return hipSuccess;
}

}  // namespace convnhwc
