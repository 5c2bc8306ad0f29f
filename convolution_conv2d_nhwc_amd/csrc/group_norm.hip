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
// The variance is taken about the mean, never as E[x^2] - mean^2, so a large
// common offset costs no digits: a lane takes the mean and the squared
// deviation of the values it holds in registers, and runs of values (n, mean,
// M2) merge by M2 = M2a + M2b + (mean_a - mean_b)^2 n_a n_b / (n_a + n_b).
//
// What bounds it: memory. A workgroup of 512 lanes or more owns a channel tile of
// whole groups. Where the tile's map fits its registers (8 vectors of 16 bytes
// for each of up to 1024 lanes, of x or of x and dy), one launch reads once and
// writes once; a narrower tile (runs of 64 or 32 bytes a pixel instead of 128)
// makes larger maps fit and gives more workgroups when images are few. Larger maps take one
// sweep for the statistics and one that applies them, each workgroup
// streaming its share of the pixels a block ahead of its arithmetic; the second
// read comes from the last-level cache as far as the map fits there. 16 x 160 x
// 160 x 128 bf16: 20 us for the statistics (5.1 TB/s), 39 to apply them
// (5.4 TB/s); over inputs that the cache does not hold 30 + 43, 73 as a call. 20 x
// 20 x 512 in one launch 7 us.
//
// Registers: 1024 lanes leave 128 each, so the one-launch gradient of eight
// bf16 a vector keeps 23 of its values in scratch memory, 51 where vectors straddle
// groups (16 x 30 x 30 x 256: 27 us, 0.8 TB/s; 22 x 22 in 512 lanes 11 us, 1.1 TB/s),
// and so does the streamed gradient of straddling vectors, 19 and 33 (16 x 80 x
// 80 x 80 in 8 groups: 16 + 25 us; 96 channels, where none straddles, 15 + 17).
#include <algorithm>

#include "device_common.h"
#include "train.h"

namespace convnhwc {
namespace {

constexpr int kThreads = 512;  // lanes of a workgroup; twice as many for the largest one-launch maps
constexpr int kMaxCt = 512;    // channels of a tile: one LDS word each
constexpr int kSteps = 8;      // vectors a lane holds when a map fits one launch
constexpr int kBlock = 4;    // vectors of x a lane holds of a streamed map
constexpr int kGradBlock = 2;  // vectors of x and of dy

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

// act(z), NaN staying NaN. SiLU(z) = z / (1 + e^-z): e^-z overflows to infinity
// for z << 0 and the quotient is then -0, the limit.
template <int ACT>
__device__ __forceinline__ float norm_act(float z) {
  if constexpr (ACT == CONV_ACT_SILU)
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  else if constexpr (ACT == ACT_RELU)
    return z < 0.0f ? 0.0f : z;
  else if constexpr (ACT == ACT_RELU6)
    return z < 0.0f ? 0.0f : z > 6.0f ? 6.0f : z;
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
    return q * (1.0f + z * (1.0f - q));
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

// A lane's place: pixel pl of each step of ppi pixels, VEC channels from c.
// SAME: these lie in one group.
template <int VEC>
struct Lane {
  int pl, vc, c;
  bool on;
  __device__ __forceinline__ Lane(const NormPlan& p, const Tile& t) {
    const int ctv = p.ct / VEC, tid = threadIdx.x;
    pl = tid / ctv;
    vc = tid - pl * ctv;
    c = t.c0 + vc * VEC;
    on = pl < p.ppi && vc * VEC < t.width;
  }
  __device__ __forceinline__ int group(const Tile& t, int k) const { return on ? (vc * VEC + k) / t.gw : 0; }
};

// n values with their mean and squared deviation, one of each per group that
// the lane's channels belong to (SAME: one) or per channel.
template <int VEC, bool SAME>
struct Run {
  static constexpr int U = SAME ? 1 : VEC;
  float n, mean[U], m2[U];
  __device__ __forceinline__ void clear() {
    n = 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) mean[k] = m2[k] = 0.0f;
  }
  // the first cnt of R vectors, the others zeros
  template <class V, int R>
  __device__ __forceinline__ void add(const typename V::raw (&raw)[R], int cnt) {
    if (cnt <= 0) return;
    float s[U];
#pragma unroll
    for (int k = 0; k < U; ++k) s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[VEC];
      V::unpack(raw[i], f);
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[SAME ? 0 : k] += f[k];
    }
    const float nb = (float)cnt * (VEC / U), inv = 1.0f / nb;
    float q[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      s[k] *= inv;
      q[k] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < cnt) {
        float f[VEC];
        V::unpack(raw[i], f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float d = f[k] - s[SAME ? 0 : k];
          q[SAME ? 0 : k] += d * d;
        }
      }
    }
    const float w = nb / (n + nb);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float d = s[k] - mean[k];
      mean[k] += d * w;
      m2[k] += q[k] + d * d * (n * w);
    }
    n += nb;
  }
};

// Group statistics of the workgroup's runs: gmean[g], gm2[g] for the tile's
// groups; inv is 1 / their values. red: NT * (2 U + 1) floats.
template <int NT, int VEC, bool SAME>
__device__ __forceinline__ void merge_runs(const Run<VEC, SAME>& r, const Lane<VEC>& l, const Tile& t,
                                           const NormPlan& p, float inv, float* red, float* gmean, float* gm2) {
  constexpr int U = Run<VEC, SAME>::U, W = VEC / U;  // channels per run
  float* const mean = red;
  float* const m2 = red + NT * U;
  float* const cnt = red + 2 * NT * U;
  const int units = p.ct / W;  // runs per pixel
  if (l.pl < p.ppi) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int at = l.pl * units + l.vc * U + k;
      mean[at] = r.mean[k];
      m2[at] = r.m2[k];
    }
    if (l.vc == 0) cnt[l.pl] = l.on ? r.n : 0.0f;
  }
  __syncthreads();
  // one wave per group in turn: its runs are gu neighbours of each pixel
  const int lane = threadIdx.x & 63, gu = t.gw / W, all = gu * p.ppi;
  const float rgu = 1.0f / (float)gu;  // (i + 1/2) / gu truncates to i / gu: all < 2^13
  for (int g = threadIdx.x >> 6; g < t.ng; g += NT / 64) {
    float s = 0.0f;
    for (int i = lane; i < all; i += 64) {
      const int px = (int)(((float)i + 0.5f) * rgu), at = px * units + g * gu + (i - px * gu);
      s += cnt[px] * mean[at];
    }
    const float mu = wave_sum(s) * inv;
    s = 0.0f;
    for (int i = lane; i < all; i += 64) {
      const int px = (int)(((float)i + 0.5f) * rgu), at = px * units + g * gu + (i - px * gu);
      const float d = mean[at] - mu;
      s += m2[at] + cnt[px] * d * d;
    }
    s = wave_sum(s);
    if (lane == 0) {
      gmean[g] = mu;
      gm2[g] = s;
    }
  }
  __syncthreads();
}

// The pixels of a workgroup: pix0 .. pix0 + npix - 1 of the image, one R-vector
// block after another.
template <class V, int R>
struct Source {
  const void* base;
  int64_t off, pitch;  // of the lane's first vector; from one pixel to the next
  // the block whose first pixel is `first`
  __device__ __forceinline__ void load(typename V::raw (&raw)[R], int first, int pl, int ppi, int npix,
                                       bool on) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      raw[i] = typename V::raw{};
      const int px = first + i * ppi;
      if (on && px + pl < npix) raw[i] = V::load(base, off + px * pitch);
    }
  }
};

enum { WHOLE = 0, SUMS = 1, APPLY = 2 };

// Vectors of the lane in a block that starts at pixel `first` (a multiple of ppi) of npix.
__device__ __forceinline__ int block_count(int first, int pl, int npix, int ppi, int r) {
  const int left = npix - first - pl;
  return left <= 0 ? 0 : min(r, (left + ppi - 1) / ppi);
}

template <typename T, int VEC, bool SAME, int R, int MODE, int NT = kThreads>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(MODE == WHOLE && NT == kThreads ? 2 : 4))) void norm_kernel(NormArgs a) {
  typedef Vec<T, VEC> V;
  typedef Run<VEC, SAME> Stat;
  __shared__ float red[MODE == APPLY ? 1 : NT * (2 * Stat::U + 1)], gmean[kMaxCt], grstd[kMaxCt];
  const NormPlan& p = a.p;
  const int tid = threadIdx.x;
  const int n = blockIdx.z, chunk = blockIdx.x;
  const Tile t = tile_of(a, blockIdx.y);
  const Lane<VEC> l(p, t);
  const int pix0 = chunk * p.cpix, npix = min(p.cpix, a.hw - pix0);
  const int64_t px0 = (int64_t)n * a.hw + pix0 + l.pl;
  const Source<V, R> src = {a.x, px0 * a.pitch + l.c, a.pitch};
  const int per = p.ppi * R;

  typename V::raw raw[R];
  src.load(raw, 0, l.pl, p.ppi, npix, l.on);

  if constexpr (MODE != APPLY) {
    Stat st;
    st.clear();
    if constexpr (MODE == WHOLE) {
      st.template add<V, R>(raw, block_count(0, l.pl, npix, p.ppi, R));
    } else {
      for (int first = 0; first < npix; first += per) {
        typename V::raw next[R];
        src.load(next, first + per, l.pl, p.ppi, npix, l.on);
        st.template add<V, R>(raw, block_count(first, l.pl, npix, p.ppi, R));
#pragma unroll
        for (int i = 0; i < R; ++i) raw[i] = next[i];
      }
    }
    const float inv = 1.0f / ((float)npix * (float)t.gw);
    merge_runs<NT, VEC, SAME>(st, l, t, p, inv, red, gmean, grstd);
    if constexpr (MODE == SUMS) {
      if (tid < t.ng) {
        const int np = p.chunks * p.tpg;
        float* o = a.part + (((int64_t)n * a.groups + t.g0 + tid) * np + chunk * p.tpg + t.sub) * 2;
        o[0] = gmean[tid];
        o[1] = grstd[tid];
      }
      return;
    }
    if (tid < t.ng) {
      const float rstd = rsqrtf(grstd[tid] * inv + a.eps);
      grstd[tid] = rstd;
      if (a.stats) {
        float* o = a.stats + ((int64_t)n * a.groups + t.g0 + tid) * 2;
        o[0] = gmean[tid];
        o[1] = rstd;
      }
    }
  } else {
    // merge the chunks' (mean, squared deviation)
    const int np = p.chunks * p.tpg;
    for (int g = tid >> 6; g < t.ng; g += NT / 64) {
      const float2* q = reinterpret_cast<const float2*>(a.part) + ((int64_t)n * a.groups + t.g0 + g) * np;
      auto count = [&](int j) {
        const int cj = j / p.tpg, sj = j - cj * p.tpg;
        const int w = p.tpg == 1 ? a.cg : min(p.ct, a.cg - sj * p.ct);
        return (float)min(p.cpix, a.hw - cj * p.cpix) * (float)w;
      };
      float s = 0.0f;
      for (int j = tid & 63; j < np; j += 64) s += count(j) * q[j].x;
      const float mean = wave_sum(s) * a.inv_count;
      s = 0.0f;
      for (int j = tid & 63; j < np; j += 64) {
        const float2 v = q[j];
        const float d = v.x - mean;
        s += v.y + count(j) * d * d;
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
  if (!l.on) return;
  float mu[Stat::U], sc[VEC], sh[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const int g = l.group(t, SAME ? 0 : k);
    mu[SAME ? 0 : k] = gmean[g];
    sc[k] = grstd[g] * (a.gamma ? a.gamma[l.c + k] : 1.0f);
    sh[k] = a.beta ? a.beta[l.c + k] : 0.0f;
  }
  const int64_t yo = px0 * a.c + l.c;
  with_norm_act(a.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    for (int first = 0; first < npix; first += per) {
      typename V::raw next[R];
      if constexpr (MODE == APPLY) src.load(next, first + per, l.pl, p.ppi, npix, true);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int px = first + i * p.ppi;
        if (px + l.pl < npix) {
          float f[VEC];
          V::unpack(raw[i], f);
#pragma unroll
          for (int k = 0; k < VEC; ++k) f[k] = norm_act<ACT>((f[k] - mu[SAME ? 0 : k]) * sc[k] + sh[k]);
          V::store(a.y, yo + (int64_t)px * a.c, f);
        }
      }
      if constexpr (MODE == APPLY) {
#pragma unroll
        for (int i = 0; i < R; ++i) raw[i] = next[i];
      } else {
        break;
      }
    }
  });
}

// Sums of s1 and s2 over the lanes that hold the same channels, into chan1 and
// chan2[0 .. ct-1]. red: NT * VEC pairs. All lanes call it, those
// outside the tile with zeros.
template <int NT, int VEC>
__device__ __forceinline__ void channel_sums(const float (&s1)[VEC], const float (&s2)[VEC], const Lane<VEC>& l,
                                             const NormPlan& p, float2* red, float2* red2, float* chan1,
                                             float* chan2) {
  const int tid = threadIdx.x;
  if (l.pl < p.ppi) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[l.pl * p.ct + l.vc * VEC + k] = float2{s1[k], s2[k]};
  }
  __syncthreads();
  // two stages of about the same length
  int parts = NT / p.ct;  // ct <= kMaxCt <= NT
  while (parts > 1 && parts * parts > 2 * p.ppi) parts >>= 1;
  const int ch = tid % p.ct, part = tid / p.ct;
  if (part < parts) {
    float2 s = {0.0f, 0.0f};
#pragma unroll 4
    for (int j = part; j < p.ppi; j += parts) {
      s.x += red[j * p.ct + ch].x;
      s.y += red[j * p.ct + ch].y;
    }
    red2[part * p.ct + ch] = s;
  }
  __syncthreads();
  if (tid < p.ct) {
    float2 s = {0.0f, 0.0f};
#pragma unroll 4
    for (int j = 0; j < parts; ++j) {
      s.x += red2[j * p.ct + tid].x;
      s.y += red2[j * p.ct + tid].y;
    }
    chan1[tid] = s.x;
    chan2[tid] = s.y;
  }
  __syncthreads();
}

// Sums over each group's `width` channels of w chan1 and w chan2 (w = gamma).
template <int NT>
__device__ __forceinline__ void group_sums(const float* chan1, const float* chan2, const float* gamma, const Tile& t,
                                           float* g1, float* g2) {
  const int tid = threadIdx.x;
  auto add = [&](int ch, float& s1, float& s2) {
    const float w = gamma ? gamma[t.c0 + ch] : 1.0f;
    s1 += w * chan1[ch];
    s2 += w * chan2[ch];
  };
  if (t.gw <= 32) {
    if (tid < t.ng) {
      float s1 = 0.0f, s2 = 0.0f;
      for (int j = 0; j < t.gw; ++j) add(tid * t.gw + j, s1, s2);
      g1[tid] = s1;
      g2[tid] = s2;
    }
  } else {
    for (int g = tid >> 6; g < t.ng; g += NT / 64) {
      float s1 = 0.0f, s2 = 0.0f;
      for (int j = tid & 63; j < t.gw; j += 64) add(g * t.gw + j, s1, s2);
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if ((tid & 63) == 0) {
        g1[g] = s1;
        g2[g] = s2;
      }
    }
  }
  __syncthreads();
}

// The images' or chunks' channel sums: sum over j < count of in[j * stride + ch]
// for the tile's channels, by all lanes, into chan1 and chan2.
template <int NT>
__device__ __forceinline__ void fold_sums(const float2* in, int count, int64_t stride, int width, float2* red2,
                                          float* chan1, float* chan2) {
  const int tid = threadIdx.x, parts = NT / width, ch = tid % width, part = tid / width;
  if (part < parts) {
    float2 s = {0.0f, 0.0f};
#pragma unroll 4
    for (int j = part; j < count; j += parts) {
      const float2 q = in[(int64_t)j * stride + ch];
      s.x += q.x;
      s.y += q.y;
    }
    red2[part * width + ch] = s;
  }
  __syncthreads();
  if (tid < width) {
    float2 s = {0.0f, 0.0f};
    for (int j = 0; j < parts; ++j) {
      s.x += red2[j * width + tid].x;
      s.y += red2[j * width + tid].y;
    }
    chan1[tid] = s.x;
    chan2[tid] = s.y;
  }
  __syncthreads();
}

template <typename T, int VEC, bool SAME, int R, int MODE, int NT = kThreads>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(MODE == WHOLE && NT == kThreads ? 2 : 4))) void norm_grad_kernel(NormArgs a) {
  typedef Vec<T, VEC> V;
  __shared__ float2 red[MODE == APPLY ? 1 : NT * VEC], red2[NT];
  __shared__ float chan1[kMaxCt], chan2[kMaxCt], gm1[kMaxCt], gm2[kMaxCt];
  const NormPlan& p = a.p;
  const int tid = threadIdx.x;
  const int n = blockIdx.z, chunk = blockIdx.x;
  const Tile t = tile_of(a, blockIdx.y);
  if constexpr (MODE == APPLY) {
    if (chunk == p.chunks) {  // one more workgroup per tile: dgamma and dbeta
      if (n > 0) return;
      fold_sums<NT>(reinterpret_cast<const float2*>(a.part) + t.c0, a.n * p.chunks, a.c, t.width, red2, chan1, chan2);
      if (tid < t.width) {
        if (a.dbeta) a.dbeta[t.c0 + tid] = chan1[tid];
        if (a.dgamma) a.dgamma[t.c0 + tid] = chan2[tid];
      }
      return;
    }
  }
  const Lane<VEC> l(p, t);
  const int pix0 = chunk * p.cpix, npix = min(p.cpix, a.hw - pix0);
  const int64_t px0 = (int64_t)n * a.hw + pix0 + l.pl;
  const int64_t yo = px0 * a.c + l.c;
  const Source<V, R> sx = {a.x, px0 * a.pitch + l.c, a.pitch};
  const Source<V, R> sg = {a.dy, yo, a.c};
  const int per = p.ppi * R;

  typename V::raw rx[R], rg[R];
  sx.load(rx, 0, l.pl, p.ppi, npix, l.on);
  sg.load(rg, 0, l.pl, p.ppi, npix, l.on);
  constexpr int U = SAME ? 1 : VEC;
  float mu[U], rs[U], gm[VEC], bt[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const int ch = l.on ? l.c + k : 0;
    const float* st = a.stats + ((int64_t)n * a.groups + t.g0 + l.group(t, SAME ? 0 : k)) * 2;
    mu[SAME ? 0 : k] = st[0];
    rs[SAME ? 0 : k] = st[1];
    gm[k] = a.gamma ? a.gamma[ch] : 1.0f;
    bt[k] = a.beta ? a.beta[ch] : 0.0f;
  }

  if constexpr (MODE != APPLY) {
    float s1[VEC], s2[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s1[k] = s2[k] = 0.0f;
    with_norm_act(a.act, [&](auto ac) {
      constexpr int ACT = decltype(ac)::value;
      for (int first = 0; first < npix; first += per) {
        typename V::raw nx[R], ng[R];
        if constexpr (MODE == SUMS) {
          sx.load(nx, first + per, l.pl, p.ppi, npix, l.on);
          sg.load(ng, first + per, l.pl, p.ppi, npix, l.on);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (l.on && first + l.pl + i * p.ppi < npix) {
            float f[VEC], g[VEC];
            V::unpack(rx[i], f);
            V::unpack(rg[i], g);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              const float xh = (f[k] - mu[SAME ? 0 : k]) * rs[SAME ? 0 : k];
              const float dz = g[k] * norm_slope<ACT>(xh * gm[k] + bt[k]);
              s1[k] += dz;
              s2[k] += dz * xh;
            }
          }
        }
        if constexpr (MODE == SUMS) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            rx[i] = nx[i];
            rg[i] = ng[i];
          }
        } else {
          break;
        }
      }
    });
    channel_sums<NT, VEC>(s1, s2, l, p, red, red2, chan1, chan2);
    if (tid < t.width) {
      const int ch = t.c0 + tid;
      if (MODE == WHOLE && a.n == 1) {
        if (a.dbeta) a.dbeta[ch] = chan1[tid];
        if (a.dgamma) a.dgamma[ch] = chan2[tid];
      } else {
        reinterpret_cast<float2*>(a.part)[((int64_t)n * p.chunks + chunk) * a.c + ch] = float2{chan1[tid], chan2[tid]};
      }
    }
    if constexpr (MODE == SUMS) return;
    group_sums<NT>(chan1, chan2, a.gamma, t, gm1, gm2);
  } else if (p.tpg == 1) {
    const float2* in = reinterpret_cast<const float2*>(a.part) + (int64_t)n * p.chunks * a.c + t.c0;
    fold_sums<NT>(in, p.chunks, a.c, t.width, red2, chan1, chan2);
    group_sums<NT>(chan1, chan2, a.gamma, t, gm1, gm2);
  } else {
    // a group of several tiles: all of its channels, lane by lane
    float s1 = 0.0f, s2 = 0.0f;
    for (int j = tid; j < a.cg; j += NT) {
      const int ch = t.g0 * a.cg + j;
      const float w = a.gamma ? a.gamma[ch] : 1.0f;
      float2 s = {0.0f, 0.0f};
      for (int k = 0; k < p.chunks; ++k) {
        const float2 q = reinterpret_cast<const float2*>(a.part)[((int64_t)n * p.chunks + k) * a.c + ch];
        s.x += q.x;
        s.y += q.y;
      }
      s1 += w * s.x;
      s2 += w * s.y;
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if ((tid & 63) == 0) red2[tid >> 6] = float2{s1, s2};
    __syncthreads();
    if (tid == 0) {
      s1 = s2 = 0.0f;
      for (int j = 0; j < NT / 64; ++j) {
        s1 += red2[j].x;
        s2 += red2[j].y;
      }
      gm1[0] = s1;
      gm2[0] = s2;
    }
    __syncthreads();
  }
  if (!l.on) return;
  float m1[U], m2[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int g = l.group(t, k);
    m1[k] = gm1[g] * a.inv_count;
    m2[k] = gm2[g] * a.inv_count;
  }
  with_norm_act(a.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    for (int first = 0; first < npix; first += per) {
      typename V::raw nx[R], ng[R];
      if constexpr (MODE == APPLY) {
        sx.load(nx, first + per, l.pl, p.ppi, npix, true);
        sg.load(ng, first + per, l.pl, p.ppi, npix, true);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int px = first + i * p.ppi;
        if (px + l.pl < npix) {
          float f[VEC], g[VEC];
          V::unpack(rx[i], f);
          V::unpack(rg[i], g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float xh = (f[k] - mu[SAME ? 0 : k]) * rs[SAME ? 0 : k];
            const float dz = g[k] * norm_slope<ACT>(xh * gm[k] + bt[k]);
            f[k] = rs[SAME ? 0 : k] * (gm[k] * dz - m1[SAME ? 0 : k] - xh * m2[SAME ? 0 : k]);
          }
          V::store(a.y, yo + (int64_t)px * a.c, f);
        }
      }
      if constexpr (MODE == APPLY) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          rx[i] = nx[i];
          rg[i] = ng[i];
        }
      } else {
        break;
      }
    }
  });
}

// dgamma, dbeta from the images' channel sums (one-launch maps of several images).
__global__ __launch_bounds__(256) void norm_grad_params_kernel(NormArgs a) {
  const int ch = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  __shared__ float2 red[4][64];
  float2 s = {0.0f, 0.0f};
  if (ch < a.c) {
#pragma unroll 4
    for (int i = part; i < a.n; i += 4) {
      const float2 q = reinterpret_cast<const float2*>(a.part)[(int64_t)i * a.c + ch];
      s.x += q.x;
      s.y += q.y;
    }
  }
  red[part][threadIdx.x & 63] = s;
  __syncthreads();
  if (part || ch >= a.c) return;
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    s.x += red[j][threadIdx.x].x;
    s.y += red[j][threadIdx.x].y;
  }
  if (a.dbeta) a.dbeta[ch] = s.x;
  if (a.dgamma) a.dgamma[ch] = s.y;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <typename T, int VEC, bool SAME, int R, int NT = kThreads>
hipError_t launch_whole(const NormArgs& a, bool grad, hipStream_t s) {
  const dim3 grid(1, a.p.ctiles, a.n);
  if (!grad) {
    hipLaunchKernelGGL((norm_kernel<T, VEC, SAME, R, WHOLE, NT>), grid, dim3(NT), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_grad_kernel<T, VEC, SAME, R, WHOLE, NT>), grid, dim3(NT), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.n == 1 || (!a.dgamma && !a.dbeta)) return err;
  hipLaunchKernelGGL(norm_grad_params_kernel, dim3((a.c + 63) / 64), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T, int VEC, bool SAME>
hipError_t launch_vec(const NormArgs& a, bool grad, hipStream_t s) {
  switch (a.p.r) {
    case 1: return launch_whole<T, VEC, SAME, 1>(a, grad, s);
    case 2: return launch_whole<T, VEC, SAME, 2>(a, grad, s);
    case 4: return launch_whole<T, VEC, SAME, 4>(a, grad, s);
    case kSteps:
      return a.p.threads == kThreads ? launch_whole<T, VEC, SAME, kSteps>(a, grad, s)
                                     : launch_whole<T, VEC, SAME, kSteps, 2 * kThreads>(a, grad, s);
  }
  const dim3 grid(a.p.chunks, a.p.ctiles, a.n);
  const dim3 more(a.p.chunks + (a.dgamma || a.dbeta), a.p.ctiles, a.n);
  if (!grad) {
    hipLaunchKernelGGL((norm_kernel<T, VEC, SAME, kBlock, SUMS>), grid, dim3(kThreads), 0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((norm_kernel<T, VEC, SAME, kBlock, APPLY>), grid, dim3(kThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((norm_grad_kernel<T, VEC, SAME, kGradBlock, SUMS>), grid, dim3(kThreads), 0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((norm_grad_kernel<T, VEC, SAME, kGradBlock, APPLY>), more, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t launch_same(const NormArgs& a, bool grad, hipStream_t s) {
  if (VEC == 1 || a.cg % VEC == 0) return launch_vec<T, VEC, true>(a, grad, s);
  if constexpr (VEC > 1) return launch_vec<T, VEC, false>(a, grad, s);
  return hipErrorInvalidValue;
}

hipError_t launch_any(const NormArgs& a, int dtype, bool grad, hipStream_t s) {
  if (dtype == CONV_F32) {
    switch (a.p.vec) {
      case 4: return launch_same<float, 4>(a, grad, s);
      case 2: return launch_same<float, 2>(a, grad, s);
      default: return launch_same<float, 1>(a, grad, s);
    }
  }
  switch (a.p.vec) {
    case 8: return launch_same<uint16_t, 8>(a, grad, s);
    case 4: return launch_same<uint16_t, 4>(a, grad, s);
    case 2: return launch_same<uint16_t, 2>(a, grad, s);
    default: return launch_same<uint16_t, 1>(a, grad, s);
  }
}

}  // namespace

// vec: the widest load that c, the pixel pitch and the pointers allow; one of 16
// or 8 bytes within a group, if there is one, else one that may straddle
// groups, whose tiles of whole groups stay within kMaxCt channels.
NormPlan norm_plan(const conv_norm_desc& d, bool grad, int align) {
  NormPlan p;
  const int esz = d.dtype == CONV_F32 ? 4 : 2;
  const int c = (int)d.c, g = d.groups, cg = c / g;
  const int64_t hw = d.h * d.w;
  const int64_t pitch = d.x_pixel_stride ? d.x_pixel_stride : d.c;
  auto fits = [&](int v) { return c % v == 0 && pitch % v == 0 && align % (v * esz) == 0; };
  p.vec = 0;
  for (int v = 16 / esz; v * esz >= 8 && !p.vec; v /= 2)
    if (fits(v) && cg % v == 0) p.vec = v;
  if (!p.vec)
    for (p.vec = 16 / esz; p.vec > 1; p.vec /= 2)
      if (fits(p.vec) && cg * (p.vec / gcd(cg, p.vec)) <= kMaxCt) break;
  const int gpt0 = p.vec / gcd(cg, p.vec);  // groups that make whole vectors
  p.r = 0;
  p.threads = kThreads;
  p.chunks = 1;
  p.cpix = (int)hw;
  if (cg > kMaxCt) {
    p.gpt = 1;
    p.ct = kMaxCt;
    p.tpg = (cg + kMaxCt - 1) / kMaxCt;
    p.ctiles = g * p.tpg;
    p.ppi = kThreads / (p.ct / p.vec);
  } else {
    // `run` bytes of channels per pixel, where whole groups allow it
    auto cut = [&](int run) {
      const int unit = gpt0 * cg, want = run / esz;
      int k = std::min((want + unit - 1) / unit, (g + gpt0 - 1) / gpt0);
      while (k > 1 && k * unit > kMaxCt) --k;
      p.gpt = k * gpt0;
      p.ct = p.gpt * cg;
      p.tpg = 1;
      p.ctiles = (g + p.gpt - 1) / p.gpt;
      p.ppi = kThreads / (p.ct / p.vec);
      return (hw + p.ppi - 1) / p.ppi;  // vectors per lane of a whole map
    };
    // One launch: the widest runs that give every CU a workgroup, or else the
    // narrowest. Above 4 MB, where bandwidth counts, runs of 32 bytes cost more
    // than the second sweep of a streamed map, and so do 64 in the gradient (16 x
    // 40 x 40 x 512 bf16, 64 bytes / streamed: forward 19 / 23 us, gradient
    // 42 / 37; 32 bytes: 28, 60)
    for (int run = 128; run >= 32; run /= 2) {
      if (run < (grad ? 128 : 64) && d.n * hw * c * esz > 4 << 20) break;
      const int64_t need = cut(run);
      if (need > 2 * kSteps) continue;
      p.threads = kThreads;
      if (need > kSteps) {
        // 1024 lanes take at least two pixels a step for each that 512 took, so kSteps
        // vectors suffice; their kernel has that many also where fewer would do
        p.threads *= 2;
        p.ppi = p.threads / (p.ct / p.vec);
        p.r = kSteps;
      } else {
        for (p.r = 1; p.r < need;) p.r *= 2;
      }
      if (d.n * p.ctiles >= 256) break;
    }
    if (p.r) return p;
    cut(128);
  }
  // streamed: two workgroups a CU, blocks of kBlock vectors a lane
  const int64_t blocks = (hw + (int64_t)p.ppi * kBlock - 1) / ((int64_t)p.ppi * kBlock);
  const int64_t want = std::max<int64_t>(1, 512 / (d.n * p.ctiles));
  const int64_t per = (blocks + want - 1) / want;  // blocks a chunk
  p.cpix = (int)std::min<int64_t>(per * p.ppi * kBlock, hw);
  p.chunks = (int)((hw + p.cpix - 1) / p.cpix);
  return p;
}

int64_t norm_ws_bytes(const conv_norm_desc& d, const NormPlan& p, bool grad) {
  if (!grad) return p.r ? 0 : 8 * d.n * d.groups * p.chunks * p.tpg;
  return p.r && d.n == 1 ? 0 : 8 * d.n * p.chunks * d.c;
}

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) { return launch_any(a, dtype, false, s); }
hipError_t launch_norm_grad(const NormArgs& a, int dtype, hipStream_t s) { return launch_any(a, dtype, true, s); }

}  // namespace convnhwc
