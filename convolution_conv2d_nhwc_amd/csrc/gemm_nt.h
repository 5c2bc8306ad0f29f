// gemm_nt.h -- the matrix product of the training-side operators:
//   out[p][q] = sum_k B[p][k] A[q][k]
// with both operands 16-bit (bf16 or fp16), K-contiguous rows, fp32
// accumulators, and an epilogue functor that takes the accumulators in
// registers (softmax statistics, the softmax gradient, the polynomial of the
// orthogonalisation, plain stores).
//
// Shape. A workgroup of four waves (2 x 2) owns a TQ x TP tile; the A operand
// runs along the MFMA's rows, so a lane holds four consecutive q of one p and
// stores them as one vector. Operands go from memory straight into LDS in
// 128-byte K-tiles (16 bytes a lane, XOR-swizzled rows), two LDS buffers, one
// barrier a K-tile; a K-tile's operand reads are spread over the MFMAs of the
// half before (the pipeline of igemm_xl.hip, whose measurements hold here: an
// output block of 128x128 a wave reads a quarter of the LDS bytes per MFMA
// that 32x32 does).
//
// Rows past an operand's last and K past its end read as zeros (buffer
// bounds), so sizes need no padding; row pitches are multiples of 16 bytes.
#pragma once

#include <algorithm>

#include "device_common.h"

namespace convnhwc {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kKB = 128;                     // bytes of K per tile row
constexpr uint32_t kPastEnd = 0x80000000u;   // buffer offset past any tensor: reads 0

struct GemmArgs {
  const char* a;     // [q][K]
  const char* b;     // [p][K]
  int a_pitch, b_pitch;      // bytes from row to row, multiples of 16
  int64_t a_batch, b_batch;  // bytes from one batch entry (gridDim.z) to the next
  int q, p;          // rows
  int kbytes;        // bytes of K, a multiple of 16
  int nq;            // tiles along q; symmetric products: tiles along either side
  int group;         // tile order: q tiles per group
  int kt_per;        // K-tiles per split (gridDim.y splits)
};

enum { BF16 = 0, FP16 = 1 };

// The accumulator stays in one AGPR quad and is updated in place (see
// igemm_xl.hip: the compiler's own selection copies it every iteration).
template <int DT>
__device__ __forceinline__ void mfma_acc(f32x4& c, const i32x4& a, const i32x4& b) {
  if constexpr (DT == BF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b) : "memory");
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b) : "memory");
}

// Wait states between a VALU access of an accumulator and an MFMA on it.
__device__ __forceinline__ void acc_guard(f32x4& c) { asm volatile("s_nop 4" : "+a"(c)); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gemm_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

__device__ __forceinline__ int kt_off(int r, int c) { return r * kKB + ((c ^ (r & 7)) << 4); }

// What an epilogue sees: q of accumulator (i, r) is q0 + 16 i + r, p of
// accumulator j is p0 + 16 j; p0 and q0 are the lane's.
struct TileAt {
  int q0, p0;        // the lane's first q and p
  int tq, tp;        // the tile's first q and p
  int wq, wp;        // the wave within the tile
  int split, batch;
  int lane;
  bool mirror;       // a symmetric product's tile off the diagonal
};

// 4x4 transpose within each quad of lanes: v = four 16-bit values of
// consecutive q at the lane's p; the result is four consecutive p (the quad's)
// at q = the run's first + lane % 4. Two exchanges: lane ^ 1 on the pairs,
// then lane ^ 2.
__device__ __forceinline__ uint2 quad_transpose(uint2 v, int lane) {
  const bool odd = lane & 1, up = lane & 2;
  const uint32_t ox = __builtin_amdgcn_mov_dpp((int)v.x, 0xB1, 0xf, 0xf, true);  // quad_perm [1,0,3,2]
  const uint32_t oy = __builtin_amdgcn_mov_dpp((int)v.y, 0xB1, 0xf, 0xf, true);
  // even lanes: (own.lo, other.lo); odd lanes: (other.hi, own.hi)
  const uint32_t a = odd ? ((v.x & 0xffff0000u) | (ox >> 16)) : ((v.x & 0xffffu) | (ox << 16));
  const uint32_t b = odd ? ((v.y & 0xffff0000u) | (oy >> 16)) : ((v.y & 0xffffu) | (oy << 16));
  const uint32_t keep = up ? b : a, send = up ? a : b;
  const uint32_t got = __builtin_amdgcn_mov_dpp((int)send, 0x4E, 0xf, 0xf, true);  // quad_perm [2,3,0,1]
  return up ? uint2{got, keep} : uint2{keep, got};
}

// Residency: a 256x256 tile's LDS fills a CU (one wave a SIMD, all registers);
// smaller tiles share it.
constexpr int gemm_waves(int tq, int tp) { return tq + tp >= 512 ? 1 : tq + tp >= 256 ? 2 : 4; }

template <int DT, int TQ, int TP, class Epi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(gemm_waves(TQ, TP), gemm_waves(TQ, TP)))) void
gemm_nt_kernel(GemmArgs g, typename Epi::Args e) {
  constexpr int FQ = TQ / 32;  // 16-row fragments per wave
  constexpr int FP = TP / 32;
  constexpr int ACH = TQ / 32;  // 16-byte chunks per thread per K-tile
  constexpr int BCH = TP / 32;
  constexpr int NMF = FQ * FP;
  __shared__ __attribute__((aligned(16))) char smem[2 * (TQ + TP) * kKB];
  char* const As = smem;
  char* const Bs = smem + 2 * TQ * kKB;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  TileAt at;
  at.wq = wave >> 1;
  at.wp = wave & 1;
  at.lane = lane;
  at.split = blockIdx.y;
  at.batch = blockIdx.z;

  // Each XCD (blockIdx.x % 8 under round-robin dispatch) walks a contiguous
  // run of tiles, `group` q tiles by all p tiles at a time, so that its L2
  // holds the rows it re-reads.
  const int nwg = gridDim.x, xcd = blockIdx.x & 7;
  const int lin = xcd * (nwg >> 3) + min(xcd, nwg & 7) + (blockIdx.x >> 3);
  int qt, pt;
  at.mirror = false;
  if constexpr (Epi::kSymmetric) {
    // the lower triangle, row by row: lin = pt (pt + 1) / 2 + qt, qt <= pt
    pt = (int)((__builtin_sqrtf(8.0f * (float)lin + 1.0f) - 1.0f) * 0.5f);
    while ((pt + 1) * (pt + 2) / 2 <= lin) ++pt;
    while (pt * (pt + 1) / 2 > lin) --pt;
    qt = lin - pt * (pt + 1) / 2;
    at.mirror = qt != pt;
  } else {
    const int npt = nwg / g.nq;
    const int span = g.group * npt;
    const int grp = lin / span;
    const int first = grp * g.group;
    const int gsz = min(g.nq - first, g.group);
    const int rem = lin - grp * span;
    qt = first + rem % gsz;
    pt = rem / gsz;
  }
  at.tq = qt * TQ;
  at.tp = pt * TP;

  const __amdgpu_buffer_rsrc_t ra = gemm_rsrc(g.a + at.batch * g.a_batch, g.q * g.a_pitch);
  const __amdgpu_buffer_rsrc_t rb = gemm_rsrc(g.b + at.batch * g.b_batch, g.p * g.b_pitch);
  // lane l of a wave's 1 KiB load fills chunk l % 8 of row l / 8; fetching
  // chunk (l % 8) ^ (l / 8) lands the swizzled layout
  const int row0 = tid >> 3;
  const int c16 = ((tid & 7) ^ ((tid >> 3) & 7)) * 16;
  uint32_t va[ACH], vb[BCH];
#pragma unroll
  for (int j = 0; j < ACH; ++j) va[j] = (uint32_t)(at.tq + row0 + 32 * j) * (uint32_t)g.a_pitch + c16;
#pragma unroll
  for (int j = 0; j < BCH; ++j) vb[j] = (uint32_t)(at.tp + row0 + 32 * j) * (uint32_t)g.b_pitch + c16;
  // rows past the last start at or past the buffer's end: they read zeros
  // (an offset that would not fit 32 bits is pinned past the end as well)
#pragma unroll
  for (int j = 0; j < ACH; ++j)
    if (at.tq + row0 + 32 * j >= g.q) va[j] = kPastEnd;
#pragma unroll
  for (int j = 0; j < BCH; ++j)
    if (at.tp + row0 + 32 * j >= g.p) vb[j] = kPastEnd;

  const int kt0 = blockIdx.y * g.kt_per;
  const int nkt_all = (g.kbytes + kKB - 1) / kKB;
  const int nkt = min(g.kt_per, nkt_all - kt0);  // <= 0: a split past the end, its sums are zeros
  const int wave_blk = wave * 1024;
  // chunk c of K-tile kt into LDS buffer buf; K past the end reads zeros
  auto dma_chunk = [&](int kt, int buf, auto cc) {
    constexpr int c = decltype(cc)::value;
    const bool in = kt * kKB + c16 < g.kbytes;
    const int so = kt < nkt_all ? kt * kKB : 0;  // a scalar offset past the buffer could wrap its bounds check
    if constexpr (c < ACH) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ra, (__attribute__((address_space(3))) void*)(As + buf * TQ * kKB + c * 4096 + wave_blk), 16,
          (int)(in ? va[c] : kPastEnd), so, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (__attribute__((address_space(3))) void*)(Bs + buf * TP * kKB + (c - ACH) * 4096 + wave_blk), 16,
          (int)(in ? vb[c - ACH] : kPastEnd), so, 0, 0);
    }
  };
  auto dma_all = [&](int kt, int buf) {
    StaticFor<0, ACH + BCH>::run([&](auto cc) { dma_chunk(kt, buf, cc); });
  };

  const int ar = at.wq * (TQ / 2) + (lane & 15);
  const int br = at.wp * (TP / 2) + (lane & 15);
  auto read_frag = [&](int buf, int s, auto rc, i32x4(&af)[FQ], i32x4(&bf)[FP]) {
    constexpr int r = decltype(rc)::value;
    const int c = 4 * s + (lane >> 4);
    if constexpr (r < FQ)
      af[r] = *reinterpret_cast<const i32x4*>(As + buf * TQ * kKB + kt_off(ar + 16 * r, c));
    else
      bf[r - FQ] = *reinterpret_cast<const i32x4*>(Bs + buf * TP * kKB + kt_off(br + 16 * (r - FQ), c));
  };
  auto read_all = [&](int buf, int s, i32x4(&af)[FQ], i32x4(&bf)[FP]) {
    StaticFor<0, FQ + FP>::run([&](auto rc) { read_frag(buf, s, rc, af, bf); });
  };

  f32x4 acc[FQ][FP];
#pragma unroll
  for (int i = 0; i < FQ; ++i)
#pragma unroll
    for (int j = 0; j < FP; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto guard_all = [&]() {
    StaticFor<0, FQ>::run([&](auto ic) {
      StaticFor<0, FP>::run([&](auto jc) { acc_guard(acc[decltype(ic)::value][decltype(jc)::value]); });
    });
  };
  guard_all();
  auto mfma_range = [&](auto bc, auto ec, const i32x4(&af)[FQ], const i32x4(&bf)[FP]) {
    StaticFor<decltype(bc)::value, decltype(ec)::value>::run([&](auto kc) {
      constexpr int k = decltype(kc)::value;
      mfma_acc<DT>(acc[k / FP][k % FP], af[k / FP], bf[k % FP]);
    });
  };

  auto wait_loads = [&]() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
  i32x4 a0[FQ], b0[FP], a1[FQ], b1[FP];
  dma_all(kt0, 0);
  dma_all(kt0 + 1, 1);
  wait_loads();
  __syncthreads();
  read_all(0, 0, a0, b0);

  constexpr int CH = ACH + BCH;
  constexpr int NR = FQ + FP;
  static_assert(CH <= NR, "every load has a slot in half 2");
  int t = 0;
  for (; t + 1 < nkt; ++t) {
    const int buf = t & 1;
    StaticFor<0, NR>::run([&](auto rc) {
      constexpr int r = decltype(rc)::value;
      mfma_range(std::integral_constant<int, r * NMF / NR>{}, std::integral_constant<int, (r + 1) * NMF / NR>{}, a0,
                 b0);
      read_frag(buf, 1, rc, a1, b1);
    });
    wait_loads();
    __syncthreads();
    StaticFor<0, NR>::run([&](auto rc) {
      constexpr int r = decltype(rc)::value;
      if constexpr (r < CH) dma_chunk(kt0 + t + 2, buf, rc);
      read_frag(buf ^ 1, 0, rc, a0, b0);
      mfma_range(std::integral_constant<int, r * NMF / NR>{}, std::integral_constant<int, (r + 1) * NMF / NR>{}, a1,
                 b1);
    });
  }
  read_all(t & 1, 1, a1, b1);
  mfma_range(std::integral_constant<int, 0>{}, std::integral_constant<int, NMF>{}, a0, b0);
  mfma_range(std::integral_constant<int, 0>{}, std::integral_constant<int, NMF>{}, a1, b1);
  wait_loads();
  guard_all();

  at.q0 = at.tq + at.wq * (TQ / 2) + 4 * (lane >> 4);
  at.p0 = at.tp + at.wp * (TP / 2) + (lane & 15);
  Epi::template run<TQ, TP>(acc, at, e);
}

// ---- host side --------------------------------------------------------------

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int DT, int T, class Epi>
hipError_t gemm_launch_t(GemmArgs g, const typename Epi::Args& e, int splits, int batch, hipStream_t s) {
  const int nq = cdiv(g.q, T), np = cdiv(g.p, T);
  g.nq = nq;
  // about the square root of an XCD's run of tiles
  g.group = 1;
  while (g.group < nq && 8 * g.group * g.group < nq * np) ++g.group;
  const int nkt = cdiv(g.kbytes, kKB);
  g.kt_per = cdiv(nkt, splits);
  const int tiles = Epi::kSymmetric ? np * (np + 1) / 2 : nq * np;
  hipLaunchKernelGGL((gemm_nt_kernel<DT, T, T, Epi>), dim3(tiles, splits, batch), dim3(256), 0, s, g, e);
  return hipGetLastError();
}

// Tile: 256x256 when that fills the chip (one workgroup a CU), else 128x128 when it
// gives at least half a chip, else 64x64.
inline int gemm_tile(int64_t q, int64_t p, int64_t others, bool symmetric) {
  auto tiles = [&](int t) {
    const int64_t a = cdiv(q, t), b = cdiv(p, t);
    return (symmetric ? a * (a + 1) / 2 : a * b) * others;
  };
  return tiles(256) >= 192 ? 256 : tiles(128) >= 128 ? 128 : 64;
}

template <int DT, class Epi>
hipError_t gemm_launch(const GemmArgs& g, const typename Epi::Args& e, int tile, int splits, int batch,
                       hipStream_t s) {
  switch (tile) {
    case 256: return gemm_launch_t<DT, 256, Epi>(g, e, splits, batch, s);
    case 128: return gemm_launch_t<DT, 128, Epi>(g, e, splits, batch, s);
    default: return gemm_launch_t<DT, 64, Epi>(g, e, splits, batch, s);
  }
}

}  // namespace
}  // namespace convnhwc
