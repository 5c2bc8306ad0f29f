// group_norm.hip -- group norm with its activation over NHWC maps, and its
// gradients.
//
// Mathematics. For one image and one group of cg channels, N = h w cg:
//   mean = sum x / N, var = sum (x - mean)^2 / N, rstd = 1/sqrt(var + eps),
//   xhat = (x - mean) rstd, z = gamma xhat + beta, y = act(z);
//   dz = dy act'(z), dbeta = sum dz, dgamma = sum dz xhat,
//   dx = rstd (gamma dz - m1 - xhat m2), m1 = sum gamma dz / N,
//   m2 = sum gamma dz xhat / N.
// All in fp32; the only rounding to fewer bits is the bf16 store of y or dx.
// The variance is taken about the mean (two sweeps over values held in
// registers, chunks merged by mean and squared deviation), never as
// E[x^2] - mean^2, so a large common offset costs no digits.
//
// What bounds it: memory. A workgroup of 512 lanes owns a channel tile of
// whole groups and a chunk of pixels and keeps it in registers (up to 16
// vectors of 16 bytes a lane), so where a whole map of a tile fits, one launch
// reads x once and writes y once. Larger maps take a sweep for the chunk
// statistics and a second one that applies them; the second read of x comes
// from the last-level cache as far as the map fits there. The gradient does the
// same with two tensors and per-channel sums.
#include <algorithm>

#include "device_common.h"
#include "train.h"

namespace convnhwc {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxCt = 512;    // channels of a tile: one LDS word each
constexpr int kFwdSteps = 16;  // vectors of x a lane holds when a map fits one launch
constexpr int kGradSteps = 8;  // the same of x and of dy

template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  typedef uint4 t;
};
template <>
struct Raw<8> {
  typedef uint2 t;
};
template <>
struct Raw<4> {
  typedef uint32_t t;
};
template <>
struct Raw<2> {
  typedef uint16_t t;
};

// VEC values of type float or bf16 (uint16_t) in one load or store.
template <typename T, int VEC>
struct Vec {
  typedef typename Raw<VEC * sizeof(T)>::t raw;
  static __device__ __forceinline__ raw load(const void* base, int64_t off) {
    return *reinterpret_cast<const raw*>(static_cast<const T*>(base) + off);
  }
  static __device__ __forceinline__ void unpack(const raw& r, float (&f)[VEC]) {
    T t[VEC];
    __builtin_memcpy(t, &r, sizeof(raw));
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if constexpr (sizeof(T) == 4)
        f[k] = t[k];
      else
        f[k] = bf16_bits_to_f32(t[k]);
    }
  }
  static __device__ __forceinline__ void store(void* base, int64_t off, const float (&f)[VEC]) {
    raw r;
    if constexpr (sizeof(T) == 4) {
      __builtin_memcpy(&r, f, sizeof(raw));
    } else if constexpr (VEC == 1) {
      r = f32_to_bf16_bits(f[0]);
    } else {
      uint32_t w[VEC / 2];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) w[k] = bf16x2_bits(f[2 * k], f[2 * k + 1]);
      __builtin_memcpy(&r, w, sizeof(raw));
    }
    *reinterpret_cast<raw*>(static_cast<T*>(base) + off) = r;
  }
};

// act(z). SiLU(z) = z / (1 + e^-z): e^-z overflows to infinity for z << 0 and
// the quotient is then -0, the limit.
template <int ACT>
__device__ __forceinline__ float norm_act(float z) {
  if constexpr (ACT == CONV_ACT_SILU)
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  else
    return act_t<ACT>(z);
}

// act'(z). SiLU: q (1 + z (1 - q)) with q = 1 / (1 + e^-z). Mish, with
// t = e^z, u = t (t + 2), h = u / (u + 2) = tanh(ln(1 + t)):
// h + z (1 - h^2) t / (1 + t), and 1 - h^2 = 4 (u + 1) / (u + 2)^2 =
// 4 (1 + t)^2 / (u + 2)^2, so the second term is z 4 t (1 + t) / (u + 2)^2
// (no difference of near-equal numbers). t is clamped as in mish_f32.
template <int ACT>
__device__ __forceinline__ float norm_slope(float z) {
  if constexpr (ACT == CONV_ACT_SILU) {
    const float q = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    // past +-88 the product z (1 - q) could be inf * 0; the slope is q there
    return __builtin_fabsf(z) > 88.0f ? q : q * (1.0f + z * (1.0f - q));
  } else if constexpr (ACT == ACT_MISH) {
    const float t = __expf(fminf(z, 20.0f));
    const float u = t * (t + 2.0f);
    const float r = __builtin_amdgcn_rcpf(u + 2.0f);
    // t is 0 below, 1 - h^2 is 0 above; a NaN stays one
    const float zc = z < -104.0f ? -104.0f : z > 104.0f ? 104.0f : z;
    return u * r + zc * (4.0f * t * (1.0f + t)) * (r * r);
  } else if constexpr (ACT == ACT_RELU) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_RELU6) {
    return z > 0.0f && z < 6.0f ? 1.0f : 0.0f;
  } else {
    return 1.0f;
  }
}

template <class F>
__device__ __forceinline__ void with_norm_act(int act, F&& f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
    case ACT_RELU6: f(std::integral_constant<int, ACT_RELU6>{}); break;
    case ACT_MISH: f(std::integral_constant<int, ACT_MISH>{}); break;
    case CONV_ACT_SILU: f(std::integral_constant<int, CONV_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}); break;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sums of v[VEC] over the lanes that hold the same channels, into
// chan[0 .. ct-1]; red has kThreads * VEC floats. All lanes call it; lanes
// outside the tile pass zeros (pl >= ppi: they write nothing).
template <int VEC>
__device__ __forceinline__ void channel_sums(const float (&v)[VEC], int pl, int vc, const NormPlan& p, float* red,
                                             float* red2, float* chan) {
  const int tid = threadIdx.x;
  if (pl < p.ppi) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[pl * p.ct + vc * VEC + k] = v[k];
  }
  __syncthreads();
  const int parts = kThreads / p.ct;  // ct <= kMaxCt = kThreads
  const int ch = tid % p.ct, part = tid / p.ct;
  if (part < parts) {
    float s = 0.0f;
    for (int j = part; j < p.ppi; j += parts) s += red[j * p.ct + ch];
    red2[part * p.ct + ch] = s;
  }
  __syncthreads();
  if (tid < p.ct) {
    float s = 0.0f;
    for (int j = 0; j < parts; ++j) s += red2[j * p.ct + tid];
    chan[tid] = s;
  }
  __syncthreads();
}

// Group sums of chan over `width` channels per group (ng groups).
__device__ __forceinline__ void group_sums(const float* chan, int ng, int width, float* gs) {
  const int tid = threadIdx.x;
  if (width <= 32) {
    if (tid < ng) {
      float s = 0.0f;
      for (int j = 0; j < width; ++j) s += chan[tid * width + j];
      gs[tid] = s;
    }
  } else {
    for (int g = tid >> 6; g < ng; g += kWaves) {
      float s = 0.0f;
      for (int j = tid & 63; j < width; j += 64) s += chan[g * width + j];
      s = wave_sum(s);
      if ((tid & 63) == 0) gs[g] = s;
    }
  }
  __syncthreads();
}

// The channel tile of a workgroup: groups g0 .. g0+ng-1 (whole, gw = cg
// channels each) or gw channels of group g0 (part `sub` of tpg).
struct Tile {
  int c0, width, g0, ng, gw, sub;
};
__device__ __forceinline__ Tile tile_of(const NormArgs& a, int t) {
  Tile r;
  if (a.p.tpg == 1) {
    r.g0 = t * a.p.gpt;
    r.ng = min(a.p.gpt, a.groups - r.g0);
    r.gw = a.cg;
    r.c0 = r.g0 * a.cg;
    r.width = r.ng * a.cg;
    r.sub = 0;
  } else {
    r.g0 = t / a.p.tpg;
    r.sub = t - r.g0 * a.p.tpg;
    r.ng = 1;
    r.c0 = r.g0 * a.cg + r.sub * a.p.ct;
    r.gw = r.width = min(a.p.ct, a.cg - r.sub * a.p.ct);
  }
  return r;
}

enum { WHOLE = 0, SUMS = 1, APPLY = 2 };

template <typename T, int VEC, int R, int MODE>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a) {
  typedef Vec<T, VEC> V;
  __shared__ float red[kThreads * VEC], red2[kThreads], chan[kMaxCt], gmean[kMaxCt], grstd[kMaxCt];
  const NormPlan& p = a.p;
  const int tid = threadIdx.x;
  const int n = blockIdx.z, chunk = blockIdx.x;
  const Tile t = tile_of(a, blockIdx.y);
  const int ctv = p.ct / VEC;
  const int pl = tid / ctv, vc = tid - pl * ctv;
  const bool on = pl < p.ppi && vc * VEC < t.width;
  const int per = p.ppi * R;
  const int pix0 = chunk * per;
  const int npix = min(per, a.hw - pix0);

  typename V::raw raw[R];
  const int64_t xo = ((int64_t)n * a.hw + pix0 + pl) * a.pitch + t.c0 + vc * VEC;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    raw[i] = typename V::raw{};
    if (on && pl + i * p.ppi < npix) raw[i] = V::load(a.x, xo + (int64_t)i * p.ppi * a.pitch);
  }
  int gi[VEC];  // group of each channel, within the tile
#pragma unroll
  for (int k = 0; k < VEC; ++k) gi[k] = on ? (vc * VEC + k) / t.gw : 0;

  if constexpr (MODE != APPLY) {
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[VEC];
      V::unpack(raw[i], f);
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[k] += f[k];
    }
    channel_sums<VEC>(s, pl, vc, p, red, red2, chan);
    group_sums(chan, t.ng, t.gw, gmean);
    const float inv = 1.0f / ((float)npix * (float)t.gw);
    float mu[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      mu[k] = gmean[gi[k]] * inv;
      s[k] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[VEC];
      V::unpack(raw[i], f);
      if (on && pl + i * p.ppi < npix) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] += (f[k] - mu[k]) * (f[k] - mu[k]);
      }
    }
    channel_sums<VEC>(s, pl, vc, p, red, red2, chan);
    group_sums(chan, t.ng, t.gw, grstd);
    if (tid < t.ng) {
      const float mean = gmean[tid] * inv;
      if constexpr (MODE == SUMS) {
        const int np = p.chunks * p.tpg;
        float* o = a.part + (((int64_t)n * a.groups + t.g0 + tid) * np + chunk * p.tpg + t.sub) * 2;
        o[0] = mean;
        o[1] = grstd[tid];
      } else {
        const float rstd = rsqrtf(grstd[tid] * inv + a.eps);
        gmean[tid] = mean;
        grstd[tid] = rstd;
        if (a.stats) {
          float* o = a.stats + ((int64_t)n * a.groups + t.g0 + tid) * 2;
          o[0] = mean;
          o[1] = rstd;
        }
      }
    }
    if constexpr (MODE == SUMS) return;
  } else {
    // merge the chunks' (mean, squared deviation): mean = sum n_i mean_i / N,
    // M2 = sum (M2_i + n_i (mean_i - mean)^2)
    const int np = p.chunks * p.tpg;
    for (int g = tid >> 6; g < t.ng; g += kWaves) {
      const float* q = a.part + ((int64_t)n * a.groups + t.g0 + g) * np * 2;
      auto count = [&](int j) {
        const int cj = j / p.tpg, sj = j - cj * p.tpg;
        const int w = p.tpg == 1 ? a.cg : min(p.ct, a.cg - sj * p.ct);
        return (float)min(per, a.hw - cj * per) * (float)w;
      };
      float s = 0.0f;
      for (int j = tid & 63; j < np; j += 64) s += count(j) * q[2 * j];
      const float mean = wave_sum(s) * a.inv_count;
      s = 0.0f;
      for (int j = tid & 63; j < np; j += 64) {
        const float d = q[2 * j] - mean;
        s += q[2 * j + 1] + count(j) * d * d;
      }
      const float rstd = rsqrtf(wave_sum(s) * a.inv_count + a.eps);
      if ((tid & 63) == 0) {
        gmean[g] = mean;
        grstd[g] = rstd;
        if (a.stats && chunk == 0 && t.sub == 0) {
          float* o = a.stats + ((int64_t)n * a.groups + t.g0 + g) * 2;
          o[0] = mean;
          o[1] = rstd;
        }
      }
    }
  }
  __syncthreads();
  if (!on) return;
  float mu[VEC], sc[VEC], sh[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const int ch = t.c0 + vc * VEC + k;
    mu[k] = gmean[gi[k]];
    sc[k] = grstd[gi[k]] * (a.gamma ? a.gamma[ch] : 1.0f);
    sh[k] = a.beta ? a.beta[ch] : 0.0f;
  }
  const int64_t yo = ((int64_t)n * a.hw + pix0 + pl) * a.c + t.c0 + vc * VEC;
  with_norm_act(a.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (pl + i * p.ppi < npix) {
        float f[VEC];
        V::unpack(raw[i], f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = norm_act<ACT>((f[k] - mu[k]) * sc[k] + sh[k]);
        V::store(a.y, yo + (int64_t)i * p.ppi * a.c, f);
      }
    }
  });
}

template <typename T, int VEC, int R, int MODE>
__global__ __launch_bounds__(kThreads) void norm_grad_kernel(NormArgs a) {
  typedef Vec<T, VEC> V;
  __shared__ float red[kThreads * VEC], red2[kThreads], chan1[kMaxCt], chan2[kMaxCt], gm1[kMaxCt], gm2[kMaxCt];
  const NormPlan& p = a.p;
  const int tid = threadIdx.x;
  const int n = blockIdx.z, chunk = blockIdx.x;
  const Tile t = tile_of(a, blockIdx.y);
  const int ctv = p.ct / VEC;
  const int pl = tid / ctv, vc = tid - pl * ctv;
  const bool on = pl < p.ppi && vc * VEC < t.width;
  const int per = p.ppi * R;
  const int pix0 = chunk * per;
  const int npix = min(per, a.hw - pix0);

  typename V::raw rx[R], rg[R];
  const int64_t xo = ((int64_t)n * a.hw + pix0 + pl) * a.pitch + t.c0 + vc * VEC;
  const int64_t yo = ((int64_t)n * a.hw + pix0 + pl) * a.c + t.c0 + vc * VEC;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    rx[i] = rg[i] = typename V::raw{};
    if (on && pl + i * p.ppi < npix) {
      rx[i] = V::load(a.x, xo + (int64_t)i * p.ppi * a.pitch);
      rg[i] = V::load(a.dy, yo + (int64_t)i * p.ppi * a.c);
    }
  }
  int gi[VEC];
  float mu[VEC], rs[VEC], gm[VEC], bt[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    gi[k] = on ? (vc * VEC + k) / t.gw : 0;
    const int ch = on ? t.c0 + vc * VEC + k : 0;
    const float* st = a.stats + ((int64_t)n * a.groups + t.g0 + gi[k]) * 2;
    mu[k] = st[0];
    rs[k] = st[1];
    gm[k] = a.gamma ? a.gamma[ch] : 1.0f;
    bt[k] = a.beta ? a.beta[ch] : 0.0f;
  }

  if constexpr (MODE != APPLY) {
    float s1[VEC], s2[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s1[k] = s2[k] = 0.0f;
    with_norm_act(a.act, [&](auto ac) {
      constexpr int ACT = decltype(ac)::value;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (on && pl + i * p.ppi < npix) {
          float f[VEC], g[VEC];
          V::unpack(rx[i], f);
          V::unpack(rg[i], g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float xh = (f[k] - mu[k]) * rs[k];
            const float dz = g[k] * norm_slope<ACT>(xh * gm[k] + bt[k]);
            s1[k] += dz;
            s2[k] += dz * xh;
          }
        }
      }
    });
    channel_sums<VEC>(s1, pl, vc, p, red, red2, chan1);
    channel_sums<VEC>(s2, pl, vc, p, red, red2, chan2);
    if (tid < t.width) {
      const int ch = t.c0 + tid;
      if constexpr (MODE == SUMS) {
        float* o = a.part + (((int64_t)n * p.chunks + chunk) * a.c + ch) * 2;
        o[0] = chan1[tid];
        o[1] = chan2[tid];
      } else {
        if (a.n == 1) {
          if (a.dbeta) a.dbeta[ch] = chan1[tid];
          if (a.dgamma) a.dgamma[ch] = chan2[tid];
        } else {
          float* o = a.tot + ((int64_t)n * a.c + ch) * 2;
          o[0] = chan1[tid];
          o[1] = chan2[tid];
        }
        const float w = a.gamma ? a.gamma[ch] : 1.0f;
        chan1[tid] *= w;
        chan2[tid] *= w;
      }
    }
    if constexpr (MODE == SUMS) return;
    __syncthreads();
    group_sums(chan1, t.ng, t.gw, gm1);
    group_sums(chan2, t.ng, t.gw, gm2);
  } else {
    if (tid < t.ng) {
      const float* m = a.means + ((int64_t)n * a.groups + t.g0 + tid) * 2;
      gm1[tid] = m[0];
      gm2[tid] = m[1];
    }
    // one workgroup per channel tile also adds the images' channel sums
    if (n == 0 && chunk == 0 && tid < t.width) {
      const int ch = t.c0 + tid;
      float s1 = 0.0f, s2 = 0.0f;
      for (int i = 0; i < a.n; ++i) {
        s1 += a.tot[((int64_t)i * a.c + ch) * 2];
        s2 += a.tot[((int64_t)i * a.c + ch) * 2 + 1];
      }
      if (a.dbeta) a.dbeta[ch] = s1;
      if (a.dgamma) a.dgamma[ch] = s2;
    }
    __syncthreads();
  }
  if (!on) return;
  float m1[VEC], m2[VEC];
  // gm1, gm2: the sums (WHOLE) or the means (APPLY) of the groups
  const float inv = MODE == APPLY ? 1.0f : a.inv_count;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    m1[k] = gm1[gi[k]] * inv;
    m2[k] = gm2[gi[k]] * inv;
  }
  with_norm_act(a.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (pl + i * p.ppi < npix) {
        float f[VEC], g[VEC];
        V::unpack(rx[i], f);
        V::unpack(rg[i], g);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float xh = (f[k] - mu[k]) * rs[k];
          const float dz = g[k] * norm_slope<ACT>(xh * gm[k] + bt[k]);
          f[k] = rs[k] * (gm[k] * dz - m1[k] - xh * m2[k]);
        }
        V::store(a.y, yo + (int64_t)i * p.ppi * a.c, f);
      }
    }
  });
}

// The chunks' channel sums of one image and a run of whole groups, added in
// chunk order by eight waves of interleaved chunks: tot[n][c], means[n][g].
__global__ __launch_bounds__(kThreads) void norm_grad_merge_kernel(NormArgs a, int gper) {
  __shared__ float l1[kWaves][64], l2[kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = blockIdx.y;
  const int g0 = blockIdx.x * gper, ng = min(gper, a.groups - g0);
  const int c0 = g0 * a.cg, c1 = c0 + ng * a.cg;
  for (int cb = c0; cb < c1; cb += 64) {
    const int ch = cb + lane;
    float s1 = 0.0f, s2 = 0.0f;
    if (ch < c1) {
#pragma unroll 4
      for (int j = wave; j < a.p.chunks; j += kWaves) {
        const float2 q = *reinterpret_cast<const float2*>(a.part + (((int64_t)n * a.p.chunks + j) * a.c + ch) * 2);
        s1 += q.x;
        s2 += q.y;
      }
    }
    l1[wave][lane] = s1;
    l2[wave][lane] = s2;
    __syncthreads();
    if (wave == 0 && ch < c1) {
      s1 = s2 = 0.0f;
#pragma unroll
      for (int j = 0; j < kWaves; ++j) {
        s1 += l1[j][lane];
        s2 += l2[j][lane];
      }
      float2* o = reinterpret_cast<float2*>(a.tot + ((int64_t)n * a.c + ch) * 2);
      *o = float2{s1, s2};
    }
    __syncthreads();
  }
  for (int g = wave; g < ng; g += kWaves) {
    float s1 = 0.0f, s2 = 0.0f;
    for (int j = lane; j < a.cg; j += 64) {
      const int ch = c0 + g * a.cg + j;
      const float w = a.gamma ? a.gamma[ch] : 1.0f;
      const float2 q = *reinterpret_cast<const float2*>(a.tot + ((int64_t)n * a.c + ch) * 2);
      s1 += w * q.x;
      s2 += w * q.y;
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (lane == 0) {
      float* o = a.means + ((int64_t)n * a.groups + g0 + g) * 2;
      o[0] = s1 * a.inv_count;
      o[1] = s2 * a.inv_count;
    }
  }
}

// dgamma, dbeta from the images' channel sums (one-launch maps of several images).
__global__ __launch_bounds__(256) void norm_grad_params_kernel(NormArgs a) {
  const int ch = blockIdx.x * 256 + threadIdx.x;
  if (ch >= a.c) return;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 8
  for (int i = 0; i < a.n; ++i) {
    const float2 q = *reinterpret_cast<const float2*>(a.tot + ((int64_t)i * a.c + ch) * 2);
    s1 += q.x;
    s2 += q.y;
  }
  if (a.dbeta) a.dbeta[ch] = s1;
  if (a.dgamma) a.dgamma[ch] = s2;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <typename T, int VEC, int R>
hipError_t launch_fwd(const NormArgs& a, hipStream_t s) {
  const dim3 grid(a.p.chunks, a.p.ctiles, a.n);
  if (a.p.chunks == 1 && a.p.tpg == 1) {
    hipLaunchKernelGGL((norm_kernel<T, VEC, R, WHOLE>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_kernel<T, VEC, R, SUMS>), grid, dim3(kThreads), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((norm_kernel<T, VEC, R, APPLY>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T, int VEC, int R>
hipError_t launch_bwd(const NormArgs& a, hipStream_t s) {
  const dim3 grid(a.p.chunks, a.p.ctiles, a.n);
  if (a.p.chunks == 1 && a.p.tpg == 1) {
    hipLaunchKernelGGL((norm_grad_kernel<T, VEC, R, WHOLE>), grid, dim3(kThreads), 0, s, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.n == 1 || (!a.dgamma && !a.dbeta)) return err;
    hipLaunchKernelGGL(norm_grad_params_kernel, dim3((a.c + 255) / 256), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_grad_kernel<T, VEC, R, SUMS>), grid, dim3(kThreads), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int gper = a.cg >= 64 ? 1 : 64 / a.cg;
  hipLaunchKernelGGL(norm_grad_merge_kernel, dim3((a.groups + gper - 1) / gper, a.n), dim3(kThreads), 0, s, a, gper);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((norm_grad_kernel<T, VEC, R, APPLY>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t dispatch(const NormArgs& a, bool grad, hipStream_t s) {
  if (grad) {
    switch (a.p.r) {
      case 1: return launch_bwd<T, VEC, 1>(a, s);
      case 2: return launch_bwd<T, VEC, 2>(a, s);
      case 4: return launch_bwd<T, VEC, 4>(a, s);
      case 8: return launch_bwd<T, VEC, 8>(a, s);
    }
  } else {
    switch (a.p.r) {
      case 1: return launch_fwd<T, VEC, 1>(a, s);
      case 2: return launch_fwd<T, VEC, 2>(a, s);
      case 4: return launch_fwd<T, VEC, 4>(a, s);
      case 8: return launch_fwd<T, VEC, 8>(a, s);
      case 16: return launch_fwd<T, VEC, 16>(a, s);
    }
  }
  return hipErrorInvalidValue;
}

hipError_t launch_any(const NormArgs& a, int dtype, bool grad, hipStream_t s) {
  if (dtype == CONV_F32) {
    switch (a.p.vec) {
      case 4: return dispatch<float, 4>(a, grad, s);
      case 2: return dispatch<float, 2>(a, grad, s);
      default: return dispatch<float, 1>(a, grad, s);
    }
  }
  switch (a.p.vec) {
    case 8: return dispatch<uint16_t, 8>(a, grad, s);
    case 2: return dispatch<uint16_t, 2>(a, grad, s);
    default: return dispatch<uint16_t, 1>(a, grad, s);
  }
}

}  // namespace

// vec: the widest load that c, the pixel pitch and the pointers allow and
// whose tiles of whole groups stay within kMaxCt channels.
NormPlan norm_plan(const conv_norm_desc& d, bool grad, int align) {
  NormPlan p;
  const int esz = d.dtype == CONV_F32 ? 4 : 2;
  const int c = (int)d.c, g = d.groups, cg = c / g;
  const int64_t hw = d.h * d.w;
  const int64_t pitch = d.x_pixel_stride ? d.x_pixel_stride : d.c;
  for (p.vec = 16 / esz; p.vec > 1; p.vec = p.vec > 2 ? 2 : 1) {
    if (c % p.vec || pitch % p.vec || align % (p.vec * esz)) continue;
    if (cg % p.vec == 0 || cg * (p.vec / gcd(cg, p.vec)) <= kMaxCt) break;
  }
  const int gpt0 = p.vec / gcd(cg, p.vec);  // groups that make whole vectors
  if (cg > kMaxCt) {
    p.gpt = 1;
    p.ct = kMaxCt;
    p.tpg = (cg + kMaxCt - 1) / kMaxCt;
    p.ctiles = g * p.tpg;
  } else {
    // 128-byte runs of channels per pixel, where whole groups allow it
    const int unit = gpt0 * cg, want = 128 / esz;
    int k = std::min((want + unit - 1) / unit, (g + gpt0 - 1) / gpt0);
    while (k > 1 && k * unit > kMaxCt) --k;
    p.gpt = k * gpt0;
    p.ct = p.gpt * cg;
    p.tpg = 1;
    p.ctiles = (g + p.gpt - 1) / p.gpt;
  }
  p.ppi = kThreads / (p.ct / p.vec);
  const int most = grad ? kGradSteps : kFwdSteps;
  const int64_t need = (hw + p.ppi - 1) / p.ppi;
  p.r = 1;
  while (p.r < most && p.r < need) p.r *= 2;
  if (need > most) p.r = most / 2;
  p.chunks = (int)((hw + (int64_t)p.ppi * p.r - 1) / ((int64_t)p.ppi * p.r));
  return p;
}

int64_t norm_ws_bytes(const conv_norm_desc& d, const NormPlan& p, bool grad) {
  const bool whole = p.chunks == 1 && p.tpg == 1;
  if (!grad) return whole ? 0 : 8 * d.n * d.groups * p.chunks * p.tpg;
  if (whole) return d.n == 1 ? 0 : 8 * d.n * d.c;
  return 8 * d.n * (d.c * p.chunks + d.c + d.groups);
}

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) { return launch_any(a, dtype, false, s); }
hipError_t launch_norm_grad(const NormArgs& a, int dtype, hipStream_t s) { return launch_any(a, dtype, true, s); }

}  // namespace convnhwc
