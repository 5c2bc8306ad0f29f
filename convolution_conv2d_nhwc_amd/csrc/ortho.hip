// ortho.hip -- the orthogonalised update of weight matrices by Newton-Schulz
// products.
//
// Mathematics. G is m x n with m <= n (a tall matrix is read transposed).
// X0 = G / (|G|_F + eps); a step is
//   A = X X^T,  Q = a I + b A + c A A,  X <- Q X,
// which maps every singular value t to a t + b t^3 + c t^5.
//
// Precision. The products run on fp16 matrix instructions (11 significant
// bits, fp32 sums; bf16's 8 bits would leave an error of several bf16 steps in
// the result). What the rounding of the operands costs most is the diagonal of
// A and Q and the Q_ii X_i term, so these are kept apart:
//   * A = D + O with D the diagonal in fp32 and O the rest in fp16;
//     A A = O O + (D_i + D_j) O_ij + D_i^2 [i = j];
//   * Q = E + R likewise, Q X = E_i X_i + R X, the first term in fp32 from
//     X held as a pair hi + lo of fp16 (22 bits).
// Against 64 bits the result is then within a third of its own bf16
// rounding. X, O and R are stored scaled by 2^8, 2^12 and 2^10: entries of
// order 1 / sqrt(m n) would otherwise be subnormal in fp16, and singular
// values up to 2 still stay in range.
//
// Work. A and A A are symmetric: only the tiles of the lower triangle are
// computed and each is stored twice (the second time transposed by exchanges
// between lanes), so a step costs m m n + m m m + 2 m m n operations. All
// sides are padded to multiples of 64 with zeros, which the iteration keeps
// zero. What bounds it: the matrix cores at large sizes; at small ones the
// 3 steps + 2 launches.
#include "gemm.h"
#include "train.h"

namespace convnhwc {
namespace {

constexpr float kSx = 256.0f, kSo = 4096.0f, kSr = 1024.0f;
constexpr int kNormBlocks = 256;  // partial sums of |G|^2 per matrix, at most

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, (f16x2{(_Float16)lo, (_Float16)hi}));
}
__device__ __forceinline__ void half4(uint2 v, float (&f)[4]) {
  const f16x2 a = __builtin_bit_cast(f16x2, v.x), b = __builtin_bit_cast(f16x2, v.y);
  f[0] = (float)a[0];
  f[1] = (float)a[1];
  f[2] = (float)b[0];
  f[3] = (float)b[1];
}

// Per matrix, in elements: mp, np the padded sides.
struct Layout {
  int m, n, mp, np;
  int tall;  // rows > cols: G is read, and the result written, transposed
};

template <typename T>
__device__ __forceinline__ float g_at(const T* g, int64_t i) {
  if constexpr (sizeof(T) == 4)
    return g[i];
  else
    return bf16_bits_to_f32(g[i]);
}

// part[batch][kNormBlocks] = sums of squares in 64 bits (gridDim.x blocks fill them)
template <typename T>
__global__ __launch_bounds__(256) void norm_part_kernel(const T* g, int64_t count, double* part) {
  __shared__ double red[4];
  const T* gb = g + (int64_t)blockIdx.y * count;
  const int64_t stride = (int64_t)gridDim.x * 256;
  double s = 0.0;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (; i + 7 * stride < count; i += 8 * stride) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = g_at(gb, i + k * stride);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += (double)v[k] * v[k];
  }
  for (; i < count; i += stride) {
    const double v = g_at(gb, i);
    s += v * v;
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kNormBlocks + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// hi, lo [mp][np] of G / (|G| + eps), 64x64 tiles; a tall G is transposed in LDS.
template <typename T>
__global__ __launch_bounds__(256) void start_kernel(const T* g, Layout l, const double* part, int parts, float eps,
                                                    _Float16* hi, _Float16* lo) {
  __shared__ float t[64][65];
  __shared__ double red[4];
  const int tid = threadIdx.x;
  const int b = blockIdx.z;
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  double s = tid < parts ? part[(int64_t)b * kNormBlocks + tid] : 0.0;
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) s += __shfl_xor(s, k);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  const T* gb = g + (int64_t)b * l.m * l.n;
  // t[i][j] = X[m0 + i][n0 + j], read along G's rows either way round
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int u = (tid >> 6) + 4 * i, v = tid & 63;
    if (l.tall) {
      t[v][u] = n0 + u < l.n && m0 + v < l.m ? g_at(gb, (int64_t)(n0 + u) * l.m + m0 + v) : 0.0f;
    } else {
      t[u][v] = m0 + u < l.m && n0 + v < l.n ? g_at(gb, (int64_t)(m0 + u) * l.n + n0 + v) : 0.0f;
    }
  }
  __syncthreads();
  // in 64 bits: the factor for a tiny G would leave fp32's range
  const double inv = (double)kSx / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)eps);
  const int64_t xb = (int64_t)b * l.mp * l.np;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = (tid >> 4) + 16 * i, v = (tid & 15) * 4;
    float f[4], h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = (float)((double)t[u][v + k] * inv);
    const uint2 hv = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3])};
    half4(hv, h);
    const int64_t o = xb + (int64_t)(m0 + u) * l.np + n0 + v;
    *reinterpret_cast<uint2*>(hi + o) = hv;
    *reinterpret_cast<uint2*>(lo + o) = uint2{half2_bits(f[0] - h[0], f[1] - h[1]), half2_bits(f[2] - h[2], f[3] - h[3])};
  }
}

// Stores v (four consecutive q of row p) to out[p][q], and where `both` to
// out[q][p]: pitch mp, in bounds for p, q < mp (multiples of 64, as 16-wide
// fragments are whole).
__device__ __forceinline__ void store_both(_Float16* out, int pitch, int p, int q, uint2 v, bool both, int lane) {
  *reinterpret_cast<uint2*>(out + (int64_t)p * pitch + q) = v;
  const uint2 t = quad_transpose(v, lane);
  if (both) *reinterpret_cast<uint2*>(out + (int64_t)(q + (lane & 3)) * pitch + (p & ~3)) = t;
}

// The rows (one p each) that an epilogue reads besides the accumulators: where
// a wave has one, it is loaded before the product; else the next one before
// the current one's stores (which may alias loads, so the compiler would wait
// out a latency a row).
template <int FQ, int FP, class Epi>
struct RowsPre {
  typename Epi::template Row<FQ> row[FP == 1 ? 1 : 2];
  __device__ __forceinline__ void load(const TileAt& at, const typename Epi::Args& e) {
    if constexpr (FP == 1) row[0].load(at, e, 0);
  }
  template <int J>
  __device__ __forceinline__ typename Epi::template Row<FQ> next(const TileAt& at, const typename Epi::Args& e) {
    if constexpr (FP > 1 && J == 0) row[0].load(at, e, 0);
    if constexpr (J + 1 < FP) row[(J + 1) & 1].load(at, e, J + 1);
    return row[J & 1];
  }
};

// A = X X^T: O scaled by kSo, D.
struct GramEpi {
  static constexpr bool kSymmetric = true, kSparse = false;
  struct Args {
    _Float16* o;
    float* d;
    int mp;
  };
  template <int FQ, int FP>
  using Pre = NoPre;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e, NoPre) {
    _Float16* o = e.o + (int64_t)at.batch * e.mp * e.mp;
    float* d = e.d + (int64_t)at.batch * e.mp;
    const float k = kSo / (kSx * kSx);
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const int p = at.p0 + 16 * j;
      if (p >= e.mp) return;  // whole fragments: the same for all lanes
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        if (q >= e.mp) return;
        float f[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          f[z] = acc[i][j][z] * k;
          if (p == q + z) {
            d[p] = f[z] * (1.0f / kSo);
            f[z] = 0.0f;
          }
        }
        store_both(o, e.mp, p, q, uint2{half2_bits(f[0], f[1]), half2_bits(f[2], f[3])}, at.mirror, at.lane);
      });
    });
  }
};

// Q = a I + b A + c A A: R scaled by kSr, E.
struct PolyEpi {
  static constexpr bool kSymmetric = true, kSparse = false;
  struct Args {
    const _Float16* o;
    const float* d;
    _Float16* r;
    float* e;
    int mp;
    float a, b, c;
  };
  // O of one p, and D there and at the lane's q
  template <int FQ>
  struct Row {
    uint2 o[FQ];
    float dp;
    __device__ __forceinline__ void load(const TileAt& at, const Args& e, int j) {
      const int p = at.p0 + 16 * j;
      if (p >= e.mp) return;
      const int64_t b = (int64_t)at.batch * e.mp;
      dp = e.d[b + p];
#pragma unroll
      for (int i = 0; i < FQ; ++i)
        if (at.q0 + 16 * i < e.mp) o[i] = *reinterpret_cast<const uint2*>(e.o + (b + p) * e.mp + at.q0 + 16 * i);
    }
  };
  template <int FQ, int FP>
  using Pre = RowsPre<FQ, FP, PolyEpi>;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e,
                                             Pre<FQ, FP>& pre) {
    const int64_t mb = (int64_t)at.batch * e.mp * e.mp;
    const float* d = e.d + (int64_t)at.batch * e.mp;
    float* ed = e.e + (int64_t)at.batch * e.mp;
    f32x4 dq[FQ];
#pragma unroll
    for (int i = 0; i < FQ; ++i)
      if (at.q0 + 16 * i < e.mp) dq[i] = *reinterpret_cast<const f32x4*>(d + at.q0 + 16 * i);
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const Row<FQ> row = pre.template next<j>(at, e);
      const int p = at.p0 + 16 * j;
      if (p >= e.mp) return;
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        if (q >= e.mp) return;
        float of[4], f[4];
        half4(row.o[i], of);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float oo = acc[i][j][z] * (1.0f / (kSo * kSo)), o = of[z] * (1.0f / kSo);
          f[z] = (e.b * o + e.c * (oo + (row.dp + dq[i][z]) * o)) * kSr;
          if (p == q + z) {
            ed[p] = e.a + e.b * row.dp + e.c * (oo + row.dp * row.dp);
            f[z] = 0.0f;
          }
        }
        store_both(e.r + mb, e.mp, p, q, uint2{half2_bits(f[0], f[1]), half2_bits(f[2], f[3])}, at.mirror, at.lane);
      });
    });
  }
};

// X <- E_p X_p + R X, from hi (which the product reads) to the next hi, lo in
// place, or to the result of the last step.
struct StepEpi {
  static constexpr bool kSymmetric = false, kSparse = false;
  struct Args {
    const float* e;
    const _Float16* hi;
    _Float16* next;
    _Float16* lo;
    uint16_t* out;    // last step: [m][n], or [n][m] when tall; else null
    int out_vec;      // rows of out are whole 8-byte vectors
    Layout l;
  };
  template <int FQ>
  struct Row {
    uint2 h[FQ], g[FQ];
    float ep;
    __device__ __forceinline__ void load(const TileAt& at, const Args& e, int j) {
      const int p = at.p0 + 16 * j;
      if (p >= e.l.mp) return;
      const int64_t b = (int64_t)at.batch * e.l.mp;
      ep = e.e[b + p];
#pragma unroll
      for (int i = 0; i < FQ; ++i) {
        const int64_t o = (b + p) * e.l.np + at.q0 + 16 * i;
        if (at.q0 + 16 * i < e.l.np) {
          h[i] = *reinterpret_cast<const uint2*>(e.hi + o);
          g[i] = *reinterpret_cast<const uint2*>(e.lo + o);
        }
      }
    }
  };
  template <int FQ, int FP>
  using Pre = RowsPre<FQ, FP, StepEpi>;
  template <int FQ, int FP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[FQ][FP], const TileAt& at, const Args& e,
                                             Pre<FQ, FP>& pre) {
    const Layout l = e.l;
    const int64_t xb = (int64_t)at.batch * l.mp * l.np;
    uint16_t* out = e.out ? e.out + (int64_t)at.batch * l.m * l.n : nullptr;
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const Row<FQ> row = pre.template next<j>(at, e);
      const int p = at.p0 + 16 * j;
      if (p >= l.mp) return;
      StaticFor<0, FQ>::run([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int q = at.q0 + 16 * i;
        if (q >= l.np) return;
        const int64_t o = xb + (int64_t)p * l.np + q;
        float h[4], g[4], f[4];
        half4(row.h[i], h);
        half4(row.g[i], g);
#pragma unroll
        for (int z = 0; z < 4; ++z) f[z] = row.ep * (h[z] + g[z]) + acc[i][j][z] * (1.0f / kSr);
        if (!out) {
          const uint2 hv = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3])};
          half4(hv, h);
          *reinterpret_cast<uint2*>(e.next + o) = hv;
          *reinterpret_cast<uint2*>(e.lo + o) =
              uint2{half2_bits(f[0] - h[0], f[1] - h[1]), half2_bits(f[2] - h[2], f[3] - h[3])};
        } else {
          const float k = 1.0f / kSx;
          const uint2 v = {bf16x2_bits(f[0] * k, f[1] * k), bf16x2_bits(f[2] * k, f[3] * k)};
          if (l.tall) {
            const uint2 t = quad_transpose(v, at.lane);
            const int row = q + (at.lane & 3), col = p & ~3;
            if (row < l.n) put4(out + (int64_t)row * l.m + col, t, l.m - col, e.out_vec);
          } else if (p < l.m) {
            put4(out + (int64_t)p * l.n + q, v, l.n - q, e.out_vec);
          }
        }
      });
    });
  }
  // `left` of the four values, as one vector where rows allow
  static __device__ __forceinline__ void put4(uint16_t* o, uint2 v, int left, int vec) {
    if (vec && left >= 4) {
      *reinterpret_cast<uint2*>(o) = v;
    } else {
      if (left > 0) o[0] = (uint16_t)v.x;
      if (left > 1) o[1] = (uint16_t)(v.x >> 16);
      if (left > 2) o[2] = (uint16_t)v.y;
      if (left > 3) o[3] = (uint16_t)(v.y >> 16);
    }
  }
};

Layout layout_of(int64_t rows, int64_t cols) {
  Layout l;
  l.tall = rows > cols;
  l.m = (int)std::min(rows, cols);
  l.n = (int)std::max(rows, cols);
  l.mp = (l.m + 63) / 64 * 64;
  l.np = (l.n + 63) / 64 * 64;
  return l;
}

struct OrthoWs {
  int64_t part, hi0, hi1, lo, o, r, d, e, bytes;
};

OrthoWs ortho_layout(int64_t batch, const Layout& l) {
  OrthoWs w;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at = (at + bytes + 255) / 256 * 256;
    return o;
  };
  const int64_t x = batch * l.mp * l.np * 2, a = batch * l.mp * l.mp * 2, v = batch * l.mp * 4;
  w.part = take(batch * kNormBlocks * 8);
  w.hi0 = take(x);
  w.hi1 = take(x);
  w.lo = take(x);
  w.o = take(a);
  w.r = take(a);
  w.d = take(v);
  w.e = take(v);
  w.bytes = at;
  return w;
}

template <typename T>
hipError_t launch_start(const OrthoArgs& a, const Layout& l, const OrthoWs& w, hipStream_t s) {
  const T* g = static_cast<const T*>(a.g);
  double* part = reinterpret_cast<double*>(a.ws + w.part);
  const int64_t count = (int64_t)l.m * l.n;
  const int parts = (int)std::min<int64_t>(kNormBlocks, cdiv(count, 2048));
  hipLaunchKernelGGL(norm_part_kernel<T>, dim3(parts, a.batch), dim3(256), 0, s, g, count, part);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(start_kernel<T>, dim3(l.np / 64, l.mp / 64, a.batch), dim3(256), 0, s, g, l, part, parts, a.eps,
                     reinterpret_cast<_Float16*>(a.ws + w.hi0), reinterpret_cast<_Float16*>(a.ws + w.lo));
  return hipGetLastError();
}

}  // namespace

int64_t ortho_ws_bytes(const conv_ortho_desc& d) { return ortho_layout(d.batch, layout_of(d.rows, d.cols)).bytes; }

hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s) {
  const Layout l = layout_of(a.rows, a.cols);
  const OrthoWs w = ortho_layout(a.batch, l);
  hipError_t err = a.g_f32 ? launch_start<float>(a, l, w, s) : launch_start<uint16_t>(a, l, w, s);
  if (err != hipSuccess) return err;
  _Float16* lo = reinterpret_cast<_Float16*>(a.ws + w.lo);
  _Float16* o = reinterpret_cast<_Float16*>(a.ws + w.o);
  _Float16* r = reinterpret_cast<_Float16*>(a.ws + w.r);
  float* d = reinterpret_cast<float*>(a.ws + w.d);
  float* e = reinterpret_cast<float*>(a.ws + w.e);
  const int sym_tile = gemm_tile(l.mp, l.mp, a.batch, true);
  const int step_tile = gemm_tile(l.np, l.mp, a.batch, false);
  const int out_row = l.tall ? l.m : l.n;
  const int out_vec = out_row % 4 == 0 && ((uintptr_t)a.out & 7) == 0;
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    _Float16* hi = reinterpret_cast<_Float16*>(a.ws + (k % 2 ? w.hi1 : w.hi0));
    _Float16* next = reinterpret_cast<_Float16*>(a.ws + (k % 2 ? w.hi0 : w.hi1));
    GemmArgs g = {};
    g.a = g.b = reinterpret_cast<const char*>(hi);
    g.k = l.np;
    g.a_pitch = g.b_pitch = l.np * 2;
    g.a_batch = g.b_batch = (int64_t)l.mp * l.np * 2;
    g.q = g.p = l.mp;
    const GramEpi::Args ga = {o, d, l.mp};
    err = gemm_launch<FP16, false, false, GramEpi>(g, ga, sym_tile, 1, a.batch, s);
    if (err != hipSuccess) return err;
    g.a = g.b = reinterpret_cast<const char*>(o);
    g.k = l.mp;
    g.a_pitch = g.b_pitch = l.mp * 2;
    g.a_batch = g.b_batch = (int64_t)l.mp * l.mp * 2;
    const PolyEpi::Args pa = {o, d, r, e, l.mp, a.a, a.b, a.c};
    err = gemm_launch<FP16, false, false, PolyEpi>(g, pa, sym_tile, 1, a.batch, s);
    if (err != hipSuccess) return err;
    g.a = reinterpret_cast<const char*>(hi);
    g.b = reinterpret_cast<const char*>(r);
    g.a_pitch = l.np * 2;
    g.a_batch = (int64_t)l.mp * l.np * 2;
    g.q = l.np;
    const StepEpi::Args sa = {e, hi, next, lo, last ? a.out : nullptr, out_vec, l};
    err = gemm_launch<FP16, true, false, StepEpi>(g, sa, step_tile, 1, a.batch, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace convnhwc
