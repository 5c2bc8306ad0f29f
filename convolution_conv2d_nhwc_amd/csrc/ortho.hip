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
// Against 64 bits, five steps then add a fifth to three quarters of the result's
// own bf16 rounding (700 x 900: 0.21, 64 x 576: 0.30, 65 x 70: 0.43); with the
// pair's second half or Q's diagonal given up, 700 x 900 adds 2.0 of it, with
// A's diagonal given up 64 x 576 adds 0.39. X, O and R are stored scaled by 2^8,
// 2^12 and 2^10: entries of order 1 / sqrt(m n) would otherwise be subnormal in
// fp16, and singular values up to 2 still stay in range.
//
// Work. A and A A are symmetric: only the tiles of the lower triangle are
// computed and each is stored twice (the second time transposed by exchanges
// between lanes), so a step costs m m n + m m m + 2 m m n operations. All
// sides are padded to multiples of 64 with zeros, which the iteration keeps
// zero. What bounds it: the matrix cores at large sizes; at small ones the
// 3 steps + 2 launches. 1024 x 4608 in five steps: 255 us, a step 18 (A) + 9 (Q)
// + 22 (Q X), and 14 before the first; six of 250 x 1000: 122 us.
#include <cstdio>

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

// The exponent of a finite v > 0, else 0 (infinities and NaN stay themselves).
__device__ __forceinline__ int ilogb_f64(double v) {
  return v > 0.0 && v < __builtin_inf() ? __builtin_amdgcn_frexp_exp(v) - 1 : 0;
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
  // t[i][j] = X[m0 + i][n0 + j], read along G's rows either way round; all loads
  // before the first store (one latency)
  const int u0 = tid >> 6, v = tid & 63;
  float r[16];
  if (l.tall) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int u = u0 + 4 * i;
      r[i] = n0 + u < l.n && m0 + v < l.m ? g_at(gb, (int64_t)(n0 + u) * l.m + m0 + v) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) t[v][u0 + 4 * i] = r[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int u = u0 + 4 * i;
      r[i] = m0 + u < l.m && n0 + v < l.n ? g_at(gb, (int64_t)(m0 + u) * l.n + n0 + v) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) t[u0 + 4 * i][v] = r[i];
  }
  __syncthreads();
  // as inv_m 2^inv_k: the factor for a tiny G would leave fp32's range
  const double inv = (double)kSx / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)eps);
  const int inv_k = ilogb_f64(inv);
  const float inv_m = (float)__builtin_ldexp(inv, -inv_k);
  const int64_t xb = (int64_t)b * l.mp * l.np;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = (tid >> 4) + 16 * i, v = (tid & 15) * 4;
    float f[4], h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __builtin_ldexpf(t[u][v + k] * inv_m, inv_k);
    const uint2 hv = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3])};
    half4(hv, h);
    const int64_t o = xb + (int64_t)(m0 + u) * l.np + n0 + v;
    *reinterpret_cast<uint2*>(hi + o) = hv;
    *reinterpret_cast<uint2*>(lo + o) = uint2{half2_bits(f[0] - h[0], f[1] - h[1]), half2_bits(f[2] - h[2], f[3] - h[3])};
  }
}

// `left` of the four values, as one vector where rows allow
__device__ __forceinline__ void put4(uint16_t* o, uint2 v, int left, int vec) {
  if (vec && left >= 4) {
    *reinterpret_cast<uint2*>(o) = v;
  } else {
    if (left > 0) o[0] = (uint16_t)v.x;
    if (left > 1) o[1] = (uint16_t)(v.x >> 16);
    if (left > 2) o[2] = (uint16_t)v.y;
    if (left > 3) o[3] = (uint16_t)(v.y >> 16);
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

__device__ __forceinline__ void half8(uint4 v, float (&f)[8]) {
  float a[4], b[4];
  half4(uint2{v.x, v.y}, a);
  half4(uint2{v.z, v.w}, b);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[k] = a[k];
    f[4 + k] = b[k];
  }
}

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
    int out_vec;      // rows of out are whole 16-byte vectors
    Layout l;
  };
  // hi, lo and E of the 16 p of one j, as Rows has them
  template <int FQ>
  struct Row {
    uint4 h[Rows<FQ>::kPasses], g[Rows<FQ>::kPasses];
    float ep[Rows<FQ>::kPasses];
    __device__ __forceinline__ void load(const TileAt& at, const Args& e, int j) {
      const Rows<FQ> rows(at.lane);
      const int q = rows.q(at);
#pragma unroll
      for (int s = 0; s < rows.kPasses; ++s) {
        const int p = rows.p(at, j, s);
        if (p < e.l.mp && q < e.l.np) {
          const int64_t b = (int64_t)at.batch * e.l.mp + p;
          ep[s] = e.e[b];
          h[s] = *reinterpret_cast<const uint4*>(e.hi + b * e.l.np + q);
          g[s] = *reinterpret_cast<const uint4*>(e.lo + b * e.l.np + q);
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
    uint16_t* out = e.out ? e.out + (int64_t)at.batch * l.m * l.n : nullptr;
    const Rows<FQ> rows(at.lane);
    const int q = rows.q(at);
    StaticFor<0, FP>::run([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const Row<FQ> row = pre.template next<j>(at, e);
      rows.put(at, acc, j);
#pragma unroll
      for (int s = 0; s < rows.kPasses; ++s) {
        const int p = rows.p(at, j, s);
        float f[8], h[8], g[8];
        rows.take(at, s, f);
        if (p >= l.mp || q >= l.np) continue;
        half8(row.h[s], h);
        half8(row.g[s], g);
#pragma unroll
        for (int z = 0; z < 8; ++z) f[z] = row.ep[s] * (h[z] + g[z]) + f[z] * (1.0f / kSr);
        if (!out) {
          const int64_t o = ((int64_t)at.batch * l.mp + p) * l.np + q;
          const uint4 hv = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3]), half2_bits(f[4], f[5]),
                            half2_bits(f[6], f[7])};
          half8(hv, h);
          *reinterpret_cast<uint4*>(e.next + o) = hv;
          *reinterpret_cast<uint4*>(e.lo + o) =
              uint4{half2_bits(f[0] - h[0], f[1] - h[1]), half2_bits(f[2] - h[2], f[3] - h[3]),
                    half2_bits(f[4] - h[4], f[5] - h[5]), half2_bits(f[6] - h[6], f[7] - h[7])};
        } else if (p < l.m) {
          const float k = 1.0f / kSx;
          if (!l.tall && e.out_vec) {
            if (q < l.n)
              *reinterpret_cast<uint4*>(out + (int64_t)p * l.n + q) =
                  uint4{bf16x2_bits(f[0] * k, f[1] * k), bf16x2_bits(f[2] * k, f[3] * k),
                        bf16x2_bits(f[4] * k, f[5] * k), bf16x2_bits(f[6] * k, f[7] * k)};
          } else {
#pragma unroll
            for (int z = 0; z < 8; ++z)
              if (q + z < l.n) out[l.tall ? (int64_t)(q + z) * l.m + p : (int64_t)p * l.n + q + z] = f32_to_bf16_bits(f[z] * k);
          }
        }
      }
    });
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

// ---- small matrices: everything in one launch ---------------------------------------

// m <= 64 and n <= 1024 in one workgroup of 16 waves per matrix, all in LDS and
// registers: 64 x 576 takes 30 us against 78 in 17 launches. X lives in fp32
// in the lanes that compute it (up to four blocks of 16 columns a wave, in the
// MFMA result's layout: p = lane % 16 of four row blocks, four consecutive
// columns; a fourth block, above 768 columns, leaves 22 registers in scratch memory:
// 64 x 768 takes 36 us, 64 x 1024 48) and in fp16 in LDS for the products; O and
// R as above. Of A and A A
// ten waves compute one 16 x 16 block of the lower triangle each and store
// both halves. Rows in LDS are 16 bytes longer than their values, so that the 16
// rows of one read fall on different banks.
constexpr int kSmallM = 64, kSmallN = 1024, kSmallWaves = 16;
constexpr int kSmallPitch = kSmallM + 8;                  // of O and R, in values

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ f32x4 mfma_f16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Four values of G from i on; vec: as one load.
template <typename T>
__device__ __forceinline__ f32x4 g_at4(const T* g, int64_t i, int left, bool vec) {
  f32x4 v = {0, 0, 0, 0};
  if (vec) {
    if (left > 0) {
      if constexpr (sizeof(T) == 4) {
        v = *reinterpret_cast<const f32x4*>(g + i);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(g + i);
        v = f32x4{bf16_bits_to_f32(u.x & 0xffffu), bf16_bits_to_f32(u.x >> 16), bf16_bits_to_f32(u.y & 0xffffu),
                  bf16_bits_to_f32(u.y >> 16)};
      }
    }
  } else {
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (z < left) v[z] = g_at(g, i + z);
  }
  return v;
}

// NB: column blocks per wave. in_vec, out_vec: G (not tall) and out take vectors of four.
template <typename T, int NB>
__global__ __launch_bounds__(64 * kSmallWaves) void small_kernel(const T* g, uint16_t* out, Layout l, int steps,
                                                                 float ca, float cb, float cc, float eps, int in_vec,
                                                                 int out_vec) {
  __shared__ __attribute__((aligned(16))) _Float16 x[kSmallM * (kSmallN + 8)];
  __shared__ __attribute__((aligned(16))) _Float16 o[kSmallM * kSmallPitch], r[kSmallM * kSmallPitch];
  __shared__ __attribute__((aligned(16))) float d[kSmallM], e[kSmallM];
  __shared__ double red[kSmallWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lp = lane & 15, lq = 4 * (lane >> 4), lk = 8 * (lane >> 4);
  const int pitch = l.np + 8;  // of x
  const int64_t mat = (int64_t)blockIdx.x * l.m * l.n;
  const int nb = l.np / 16;

  // block u of the wave: columns 16 (wave + 16 u) ..
  f32x4 xr[NB][4];
  double sq = 0.0;
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    const int q = 16 * (wave + kSmallWaves * u) + lq;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 16 * i + lp;
      f32x4 v = {0, 0, 0, 0};
      if (p < l.m) {
        if (l.tall) {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (q + z < l.n) v[z] = g_at(g, mat + (int64_t)(q + z) * l.m + p);
        } else {
          v = g_at4(g, mat + (int64_t)p * l.n + q, l.n - q, in_vec);
        }
      }
      xr[u][i] = v;
    }
  }
#pragma unroll
  for (int u = 0; u < NB; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int z = 0; z < 4; ++z) sq += (double)xr[u][i][z] * xr[u][i][z];
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) sq += __shfl_xor(sq, k);
  if (lane == 0) red[wave] = sq;
  __syncthreads();
  sq = 0.0;
#pragma unroll
  for (int k = 0; k < kSmallWaves; ++k) sq += red[k];
  // as inv_m 2^inv_k: the factor for a tiny G would leave fp32's range
  const double inv = (double)kSx / (sqrt(sq) + (double)eps);
  const int inv_k = ilogb_f64(inv);
  const float inv_m = (float)__builtin_ldexp(inv, -inv_k);

  auto put_x = [&]() {
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int b = wave + kSmallWaves * u;
      if (b < nb) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint2*>(x + (16 * i + lp) * pitch + 16 * b + lq) =
              uint2{half2_bits(xr[u][i][0], xr[u][i][1]), half2_bits(xr[u][i][2], xr[u][i][3])};
      }
    }
  };
#pragma unroll
  for (int u = 0; u < NB; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int z = 0; z < 4; ++z) xr[u][i][z] = __builtin_ldexpf(xr[u][i][z] * inv_m, inv_k);
  put_x();
  // the wave's block of the lower triangle: pb (pb + 1) / 2 + qb = wave
  int pb = 0, qb = wave;
  while (qb > pb) {
    ++pb;
    qb -= pb;
  }
  const bool tri = wave < 10;
  // 16 x 16 values of a symmetric 64 x 64 matrix, both ways round
  auto put_both = [&](_Float16* to, const float (&f)[4]) {
    const int p = 16 * pb + lp, q = 16 * qb + lq;
    const uint2 v = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3])};
    *reinterpret_cast<uint2*>(to + p * kSmallPitch + q) = v;
    if (pb != qb)
      *reinterpret_cast<uint2*>(to + (q + (lane & 3)) * kSmallPitch + (p & ~3)) = quad_transpose(v, lane);
  };
  __syncthreads();

  for (int step = 0; step < steps; ++step) {
    if (tri) {  // A = X X^T
      const _Float16* xa = x + (16 * qb + lp) * pitch + lk;
      const _Float16* xb = x + (16 * pb + lp) * pitch + lk;
      f32x4 a0 = {0, 0, 0, 0}, a1 = {0, 0, 0, 0};
#pragma unroll 4
      for (int k = 0; k < l.np; k += 64) {
        a0 = mfma_f16(*reinterpret_cast<const f16x8*>(xa + k), *reinterpret_cast<const f16x8*>(xb + k), a0);
        a1 = mfma_f16(*reinterpret_cast<const f16x8*>(xa + k + 32), *reinterpret_cast<const f16x8*>(xb + k + 32), a1);
      }
      float f[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        f[z] = (a0[z] + a1[z]) * (kSo / (kSx * kSx));
        if (pb == qb && lp == lq + z) {
          d[16 * pb + lp] = f[z] * (1.0f / kSo);
          f[z] = 0.0f;
        }
      }
      put_both(o, f);
    }
    __syncthreads();
    if (tri) {  // Q = a I + b A + c A A
      f32x4 a0 = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kSmallM; k += 32)
        a0 = mfma_f16(*reinterpret_cast<const f16x8*>(o + (16 * qb + lp) * kSmallPitch + lk + k),
                      *reinterpret_cast<const f16x8*>(o + (16 * pb + lp) * kSmallPitch + lk + k), a0);
      const int p = 16 * pb + lp, q = 16 * qb + lq;
      float of[4], f[4];
      half4(*reinterpret_cast<const uint2*>(o + p * kSmallPitch + q), of);
      const float dp = d[p];
      const f32x4 dq = *reinterpret_cast<const f32x4*>(d + q);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float oo = a0[z] * (1.0f / (kSo * kSo)), ov = of[z] * (1.0f / kSo);
        f[z] = (cb * ov + cc * (oo + (dp + dq[z]) * ov)) * kSr;
        if (p == q + z) {
          e[p] = ca + cb * dp + cc * (oo + dp * dp);
          f[z] = 0.0f;
        }
      }
      put_both(r, f);
    }
    __syncthreads();
    // X <- E_p X_p + R X, the wave's own columns, two row blocks at a time (registers)
#pragma unroll
    for (int h = 0; h < 4; h += 2) {
      f16x8 rf[2][2];
      float ep[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ep[i] = e[16 * (h + i) + lp];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          rf[i][k] = *reinterpret_cast<const f16x8*>(r + (16 * (h + i) + lp) * kSmallPitch + lk + 32 * k);
      }
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int b = wave + kSmallWaves * u;
        if (b < nb) {
          f16x8 xt[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const _Float16* at = x + (32 * k + lk + ((lane >> 2) & 3)) * pitch + 16 * b + 4 * (lane & 3);
            struct {
              s16x4 lo, hi;
            } v;
            v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
            v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * pitch));
            xt[k] = __builtin_bit_cast(f16x8, v);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f32x4 a0 = {0, 0, 0, 0};
            a0 = mfma_f16(xt[0], rf[i][0], a0);
            a0 = mfma_f16(xt[1], rf[i][1], a0);
#pragma unroll
            for (int z = 0; z < 4; ++z)
              xr[u][h + i][z] = ep[i] * xr[u][h + i][z] + a0[z] * (1.0f / kSr);
          }
        }
      }
    }
    // a wave reads and writes its own columns of x only, and the next step's
    // product reads it behind the barrier
    if (step + 1 < steps) {
      put_x();
      __syncthreads();
    }
  }

#pragma unroll
  for (int u = 0; u < NB; ++u) {
    const int q = 16 * (wave + kSmallWaves * u) + lq;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 16 * i + lp;
      float f[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) f[z] = xr[u][i][z] * (1.0f / kSx);
      if (l.tall) {
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (p < l.m && q + z < l.n) out[mat + (int64_t)(q + z) * l.m + p] = f32_to_bf16_bits(f[z]);
      } else if (p < l.m && q < l.n) {
        put4(out + mat + (int64_t)p * l.n + q, uint2{bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3])}, l.n - q,
             out_vec);
      }
    }
  }
}

struct OrthoWs {
  int64_t part, hi0, hi1, lo, o, r, d, e, bytes;
};

// ws.bytes is 0 for matrices that small_kernel takes
OrthoWs ortho_layout(int64_t batch, const Layout& l) {
  OrthoWs w = {};
  if (l.mp <= kSmallM && l.np <= kSmallN) return w;
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

template <typename T, int NB>
void launch_small_nb(const OrthoArgs& a, const Layout& l, int out_vec, hipStream_t s) {
  const T* g = static_cast<const T*>(a.g);
  const int in_vec = !l.tall && l.n % 4 == 0 && ((uintptr_t)g & (4 * sizeof(T) - 1)) == 0;
  hipLaunchKernelGGL((small_kernel<T, NB>), dim3(a.batch), dim3(64 * kSmallWaves), 0, s, g, a.out, l, a.steps, a.a,
                     a.b, a.c, a.eps, in_vec, out_vec);
}

template <typename T>
void launch_small(const OrthoArgs& a, const Layout& l, int out_vec, hipStream_t s) {
  switch (cdiv(l.np, 16 * kSmallWaves)) {
    case 1: return launch_small_nb<T, 1>(a, l, out_vec, s);
    case 2: return launch_small_nb<T, 2>(a, l, out_vec, s);
    case 3: return launch_small_nb<T, 3>(a, l, out_vec, s);
    default: return launch_small_nb<T, 4>(a, l, out_vec, s);
  }
}

}  // namespace

int64_t ortho_ws_bytes(const conv_ortho_desc& d) { return ortho_layout(d.batch, layout_of(d.rows, d.cols)).bytes; }

// Tiles of the symmetric products and of the step's.
static int sym_tile_of(const Layout& l, int64_t batch) { return gemm_tile(l.mp, l.mp, batch, true); }
static int step_tile_of(const Layout& l, int64_t batch) { return gemm_tile(l.np, l.mp, batch, false); }

void ortho_describe(const conv_ortho_desc& d, char* buf, int len) {
  const Layout l = layout_of(d.rows, d.cols);
  if (!ortho_layout(d.batch, l).bytes) {
    std::snprintf(buf, len, "ortho small m=%d n=%d tall=%d blocks=%d", l.m, l.n, l.tall, cdiv(l.np, 16 * kSmallWaves));
    return;
  }
  const int sym = sym_tile_of(l, d.batch), step = step_tile_of(l, d.batch);
  std::snprintf(buf, len, "ortho m=%d n=%d tall=%d sym=%dx%d step=%dx%d", l.m, l.n, l.tall, sym,
                gemm_deep(l.mp, l.mp, sym, d.batch, true) ? 1 : 2, step,
                gemm_deep(l.np, l.mp, step, d.batch, false) ? 1 : 2);
}

hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s) {
  const Layout l = layout_of(a.rows, a.cols);
  const int out_row = l.tall ? l.m : l.n;
  const int out_vec = out_row % 4 == 0 && ((uintptr_t)a.out & 7) == 0;
  const int out_vec8 = l.n % 8 == 0 && ((uintptr_t)a.out & 15) == 0;
  const OrthoWs w = ortho_layout(a.batch, l);
  if (!w.bytes) {
    if (a.g_f32)
      launch_small<float>(a, l, out_vec, s);
    else
      launch_small<uint16_t>(a, l, out_vec, s);
    return hipGetLastError();
  }
  hipError_t err = a.g_f32 ? launch_start<float>(a, l, w, s) : launch_start<uint16_t>(a, l, w, s);
  if (err != hipSuccess) return err;
  _Float16* lo = reinterpret_cast<_Float16*>(a.ws + w.lo);
  _Float16* o = reinterpret_cast<_Float16*>(a.ws + w.o);
  _Float16* r = reinterpret_cast<_Float16*>(a.ws + w.r);
  float* d = reinterpret_cast<float*>(a.ws + w.d);
  float* e = reinterpret_cast<float*>(a.ws + w.e);
  const int sym_tile = sym_tile_of(l, a.batch), step_tile = step_tile_of(l, a.batch);
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
    const StepEpi::Args sa = {e, hi, next, lo, last ? a.out : nullptr, out_vec8, l};
    err = gemm_launch<FP16, true, false, StepEpi>(g, sa, step_tile, 1, a.batch, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace convnhwc
