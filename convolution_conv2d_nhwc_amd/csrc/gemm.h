// gemm.h -- the matrix product of the training-side operators:
//   out[p][q] = sum_k B[p][k] A[q][k]
// with both operands 16-bit (bf16 or fp16), fp32 accumulators, and an epilogue
// functor that takes the accumulators in registers (softmax statistics, the
// softmax gradient, the polynomial of the orthogonalisation, plain stores).
//
// Operands. Each lies in memory either row by row, [q][K] (K contiguous), or
// column by column, [K][q] (KS: K strided), so no product needs a transposed
// copy of what another one reads or writes. A tile of 64 values of K goes
// from memory straight into LDS, 16 bytes a lane, as rows of 128 bytes
// ([q][64]) or of 2 T bytes ([64][T]); a KS tile is transposed by the LDS read
// itself (ds_read_b64_tr_b16: each group of 16 lanes reads four K rows of 16
// columns and every lane receives its column's four values). Rows are swizzled
// so that the lanes of one read fall on different banks.
//
// Shape. A workgroup of four waves owns a T x T tile; the A operand runs along
// the MFMA's rows, so a lane holds four consecutive q of one p and stores them
// as one vector. For T = 256 and 128 each wave owns a quarter of the tile; for
// T = 64, where a quarter would read twice the LDS bytes per MFMA and products
// are short of workgroups, each wave owns the whole tile for a quarter of the K
// values and the four sums meet in LDS at the end.
//
// Pipeline. K-tiles wait in an LDS ring: five operand tiles (two K-tiles and a
// half) for T = 256, where that is all that fits, and for T = 128 when two
// workgroups share a CU; four K-tiles for T = 128 alone on its CU; two or four
// pairs of K-tiles for T = 64. One barrier a stage; operand reads and
// loads go out over the first three quarters of the MFMAs before the ones that
// need them, so that LDS latency and the barrier fall behind matrix work. Tried
// and slower: K-tiles of 32 in a ring of four (rows of 64 bytes: twice the
// requests; 6400 x 65536 x 1024 logits 855 against 788 us).
//
// What bounds it: the matrix cores, as far as a T = 256 tile keeps them fed.
// A K-tile takes 1.65 us of it; at the rate that a large library product reaches
// (1.62 PFLOP/s at 16384^3) it would be 1.33. The difference is the first reads
// after a barrier and loads that arrive late. 6400 x 1024 x 65536 (0.86 TFLOP a
// product): 1.09 PFLOP/s for the logits with their statistics, 1.11 for the
// product over the classes, 1.29 for the one over the rows. Small
// products are bound by what a tile costs besides (4 to 8 us: launch, first
// loads, epilogue).
//
// Rows past an operand's last and K past its end read as zeros, so sizes need
// no padding; row pitches are multiples of 16 bytes.
#pragma once

#include <algorithm>

#include "device_common.h"

namespace convnhwc {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kKV = 64;                      // values of K per tile
constexpr int kKB = 2 * kKV;                 // and their bytes
constexpr uint32_t kPastEnd = 0x80000000u;   // buffer offset past any tensor: reads 0

struct GemmArgs {
  const char* a;     // [q][K], or [K][q] when KS
  const char* b;     // [p][K], or [K][p]
  int a_pitch, b_pitch;      // bytes from one row in memory to the next, multiples of 16
  int64_t a_batch, b_batch;  // bytes from one batch entry (gridDim.z) to the next
  int q, p;          // values along either side; KS: multiples of 8 (readable columns)
  int k;             // values of K; unless KS a multiple of 8
  int nq;            // tiles along q; symmetric products: tiles along either side
  int group;         // tile order: q tiles per group
  int splits;        // of K, each
  int kt_per;        // this many K-tiles
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

// The accumulators as one point in the program: between it and an MFMA, or an
// MFMA and it, go the wait states that the hardware asks for (a VALU write
// before an MFMA's read: at most 4; an MFMA's result before a VALU or store
// reads it: at most 18).
template <int FQ, int FP>
__device__ __forceinline__ void acc_pin(f32x4 (&c)[FQ][FP]) {
#pragma unroll
  for (int i = 0; i < FQ; ++i)
#pragma unroll
    for (int j = 0; j < FP; ++j) asm volatile("" : "+a"(c[i][j]));
}

// Operands that the compiler may just have moved: a VALU write needs two wait
// states before an MFMA reads it, and it does not know the ones above for MFMAs.
template <int F>
__device__ __forceinline__ void operands_ready(i32x4 (&a)[F], i32x4 (&b)[F]) {
#pragma unroll
  for (int k = 0; k < F; ++k) asm volatile("" : "+v"(a[k]), "+v"(b[k]));
  asm volatile("s_nop 1");
}

// A raw buffer of `bytes` at p, in scalar registers.
__device__ __forceinline__ i32x4 gemm_rsrc(const void* p, int bytes) {
  const uint64_t v = (uint64_t)p;
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)v),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// 16 bytes a lane from buffer r at voff + soff into LDS, lane after lane from
// address `to` + OFF (the wave's). Written out because the compiler, which sees
// the builtin as a store to any LDS, would wait for it before every transposing
// read; the waits are wait_loads. It has no destination register.
template <int OFF>
__device__ __forceinline__ void load_lds(const i32x4& r, uint32_t to, uint32_t voff, int soff) {
  asm volatile(
      "s_add_u32 m0, %0, %4\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to),
      "v"(voff), "s"(r), "s"(soff), "n"(OFF)
      : "scc", "memory");  // m0 is reserved: nothing keeps a value in it
}

// At most N loads of this wave in flight, and its LDS reads done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wg_barrier() { asm volatile("s_barrier" ::: "memory"); }

typedef __attribute__((address_space(3))) const char* lds_ptr;

// One operand's T-wide side of the product: how lanes load its K-tiles of 64
// values (N loads a lane) and read their wave's NF fragments (16 wide, 32 of
// K) from them. v: the loads' offsets in the first K-tile.
template <int T, bool KS, int NF>
struct Side;

// [q][64]: 128-byte rows, 16-byte chunk c of row r at c ^ (r & 7).
template <int T, int NF>
struct Side<T, false, NF> {
  static constexpr int N = T / 32;
  uint32_t v[N];
  int rd;
  __device__ __forceinline__ void init(int t0, int rows, int pitch, int tid, int frag0) {
    const int row = t0 + (tid >> 3), c16 = ((tid & 7) ^ ((tid >> 3) & 7)) * 16;
#pragma unroll
    for (int j = 0; j < N; ++j)
      v[j] = row + 32 * j < rows ? (uint32_t)(row + 32 * j) * (uint32_t)pitch + c16 : kPastEnd;
    const int lane = tid & 63;
    rd = (frag0 * 16 + (lane & 15)) * kKB + (((lane >> 4) ^ (lane & 7)) << 4);
  }
  static __device__ __forceinline__ int step(int) { return kKB; }
  // the last K-tile's `left` values only
  __device__ __forceinline__ void cut(int left, int tid) {
    const bool in = ((tid & 7) ^ ((tid >> 3) & 7)) * 8 < left;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = in ? v[j] : kPastEnd;
  }
  __device__ __forceinline__ i32x4 read(lds_ptr tile, int s, int r) const {
    // chunk 4 s + lane / 16 of the row, swizzled: s flips bit 2 of the chunk
    return *reinterpret_cast<__attribute__((address_space(3))) const i32x4*>(tile + (rd ^ (s << 6)) + r * 16 * kKB);
  }
};

// [64][T]: rows of 2 T bytes, 32-byte block b of K row k at b ^ swz(k). The four K rows
// that 16 lanes read (k & 3) and those of the next 16 (k >> 3) lie on different banks.
template <int T, int NF>
struct Side<T, true, NF> {
  static constexpr int N = T / 32;
  static constexpr int CPR = T / 8;      // 16-byte chunks per row
  static constexpr int RPL = 256 / CPR;  // rows per load of the workgroup
  uint32_t v[N];
  int rd[NF];
  static __device__ __forceinline__ int swz(int kk) {
    return T >= 128 ? (kk & 3) | ((kk >> 3) & 1) << 2 : ((kk >> 1) & 1) | ((kk >> 3) & 1) << 1;
  }
  // the K row of load j and the lane's first column in it
  static __device__ __forceinline__ int row_of(int tid, int j) { return tid / CPR + j * RPL; }
  static __device__ __forceinline__ int col_of(int tid, int j) {
    const int pos = tid % CPR;
    return ((((pos >> 1) ^ swz(row_of(tid, j))) << 1) | (pos & 1)) * 8;
  }
  __device__ __forceinline__ void init(int t0, int cols, int pitch, int tid, int frag0) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int col = t0 + col_of(tid, j);
      v[j] = col < cols ? (uint32_t)row_of(tid, j) * (uint32_t)pitch + (uint32_t)col * 2 : kPastEnd;
    }
    const int lane = tid & 63;
    const int kk = 8 * (lane >> 4) + ((lane >> 2) & 3);
#pragma unroll
    for (int r = 0; r < NF; ++r) rd[r] = kk * 2 * T + ((frag0 + r) ^ swz(kk)) * 32 + 8 * (lane & 3);
  }
  static __device__ __forceinline__ int step(int pitch) { return kKV * pitch; }
  __device__ __forceinline__ void cut(int left, int tid) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = row_of(tid, j) < left ? v[j] : kPastEnd;
  }
  __device__ __forceinline__ i32x4 read(lds_ptr tile, int s, int r) const {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const lds_ptr at = tile + rd[r] + s * 64 * T;
    struct {
      s16x4 lo, hi;
    } f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at));
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 8 * T));
    return __builtin_bit_cast(i32x4, f);
  }
};

// What an epilogue sees: q of accumulator (i, r) is q0 + 16 i + r, p of
// accumulator j is p0 + 16 j; p0 and q0 are the lane's.
struct TileAt {
  int q0, p0;        // the lane's first q and p
  int tq, wq;        // the tile's and the wave's first q
  int split, batch;
  int lane;
  char* lds;         // kRelay bytes of the wave's own, free
  bool mirror;       // a symmetric product's tile off the diagonal
};

// The accumulators of one j, 16 p by 16 FQ q, as whole rows: eight consecutive q
// a lane instead of four, 16 FQ / 8 lanes a row, through the wave's LDS (rows 16
// bytes longer than their values: no two lanes of an access on a bank). Memory
// then sees runs of 128 or 256 bytes; the accumulators' own layout gives runs of
// 32 in sixteen rows an instruction (X of the 1024 x 4608 update, read and
// written in its products' epilogue: 30 us a product that way, 22 this way).
constexpr int kRelay = 16 * (128 + 4) * 4;
template <int FQ>
struct Rows {
  static constexpr int kLanes = 2 * FQ;            // lanes per row
  static constexpr int kPer = 64 / kLanes;         // rows per pass
  static constexpr int kPasses = 16 / kPer;
  int row, col;  // the lane's row in a pass, its first q in the wave's run
  __device__ __forceinline__ explicit Rows(int lane) : row(lane / kLanes), col(lane % kLanes * 8) {}
  // p of pass s of j, and q
  __device__ __forceinline__ int p(const TileAt& at, int j, int s) const {
    return at.p0 - (at.lane & 15) + 16 * j + row + s * kPer;
  }
  __device__ __forceinline__ int q(const TileAt& at) const { return at.wq + col; }
  static __device__ __forceinline__ void fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // 32-bit values: put acc[0..FQ-1][j], then take row `row` of pass s
  template <int FP>
  static __device__ __forceinline__ void put(const TileAt& at, const f32x4 (&acc)[FQ][FP], int j) {
    float* to = reinterpret_cast<float*>(at.lds) + (at.lane & 15) * (16 * FQ + 4) + 4 * (at.lane >> 4);
    fence();
#pragma unroll
    for (int i = 0; i < FQ; ++i) *reinterpret_cast<f32x4*>(to + 16 * i) = acc[i][j];
    fence();
  }
  __device__ __forceinline__ void take(const TileAt& at, int s, float (&f)[8]) const {
    const f32x4* from =
        reinterpret_cast<const f32x4*>(reinterpret_cast<float*>(at.lds) + (row + s * kPer) * (16 * FQ + 4) + col);
    const f32x4 a = from[0], b = from[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = a[k];
      f[4 + k] = b[k];
    }
  }
  // 16-bit values: put four of fragment i at the lane's p, take eight
  static __device__ __forceinline__ void put16(const TileAt& at, int i, uint2 v) {
    *reinterpret_cast<uint2*>(at.lds + (at.lane & 15) * (32 * FQ + 16) + 8 * (at.lane >> 4) + 32 * i) = v;
  }
  __device__ __forceinline__ uint4 take16(const TileAt& at, int s) const {
    return *reinterpret_cast<const uint4*>(at.lds + (row + s * kPer) * (32 * FQ + 16) + 2 * col);
  }
};

// What an epilogue loads before the product (here nothing).
struct NoPre {
  template <class Args>
  __device__ __forceinline__ void load(const TileAt&, const Args&) {}
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

// The sparse term that a product may add to the dense one before its epilogue:
//   out[p][q] += sum over K rows r of delta[r] [label(r) == p] A[r][q]
// (both operands KS), as K-tiles of 64 gathered rows of A against a tile of
// zeros with one value per row.
struct SparseTerm {
  const void* labels;
  int label_bytes;
  int p_base;           // the label of p = 0
  const float* delta;   // [K]
};
constexpr int kSparseCap = 4096;  // rows listed at a time
// a listed row: its number (the K of a product with a sparse term is below 2^22) and its p in the tile
constexpr int kSparseRowBits = 22, kSparseRow = (1 << kSparseRowBits) - 1;

__device__ __forceinline__ int64_t label_raw(const void* labels, int bytes, int64_t r) {
  return bytes == 8 ? static_cast<const int64_t*>(labels)[r] : static_cast<const int32_t*>(labels)[r];
}

// How a T x T tile is cut. DEEP: a CU's LDS for one workgroup; else half of it,
// for two. A 256 tile takes all of it either way.
template <int T, bool DEEP>
struct Cut {
  static constexpr bool kSplitK = T == 64;       // waves share the tile, not K
  static constexpr int SUB = kSplitK ? 2 : 1;    // K-tiles of 64 per stage
  static constexpr int NST = T == 256 || !DEEP ? 2 : 4;
  static constexpr bool kUnits = T == 256 || (T == 128 && !DEEP);  // a ring of operand tiles, not of stages
  static constexpr int NF = kSplitK ? 4 : T / 32;  // fragments of a wave along either side
  static constexpr int CH = SUB * 2 * (T / 32);    // loads per lane per stage
  static constexpr int TILE = T * kKB;             // bytes of one operand's K-tile
  static constexpr int STAGE = SUB * 2 * TILE;
  static constexpr int LDS = kUnits ? 5 * TILE : NST * STAGE;
  static constexpr int FP = kSplitK ? 1 : NF;      // the epilogue's accumulators: [NF][FP]
};

// One tile of a product: the workgroup `block` of nwg.
template <int DT, int T, bool DEEP, bool KSA, bool KSB, class Epi>
__device__ __forceinline__ void gemm_tile_run(const GemmArgs& g, const typename Epi::Args& e, char* smem, int block,
                                              int nwg) {
  typedef Cut<T, DEEP> C;
  constexpr int F = C::NF, NMF = F * F, NST = C::NST, CH = C::CH, TILE = C::TILE, STAGE = C::STAGE, SUB = C::SUB;
  constexpr int NL = T / 32;  // loads per lane per K-tile and operand
  const lds_ptr lds = (lds_ptr)smem;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  TileAt at;
  at.lane = lane;
  at.batch = blockIdx.z;

  // Each XCD (block % 8 under round-robin dispatch) walks a contiguous
  // run of tiles, split after split, `group` q tiles by all p tiles at a time, so
  // that its L2 holds the rows it re-reads.
  const int xcd = block & 7;
  int lin = xcd * (nwg >> 3) + min(xcd, nwg & 7) + (block >> 3);
  const int tiles = nwg / g.splits;
  at.split = lin / tiles;
  lin -= at.split * tiles;
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
    const int npt = tiles / g.nq;
    const int span = g.group * npt;
    const int grp = lin / span;
    const int first = grp * g.group;
    const int gsz = min(g.nq - first, g.group);
    const int rem = lin - grp * span;
    qt = first + rem % gsz;
    pt = rem / gsz;
  }
  const int wq = C::kSplitK ? 0 : wave >> 1, wp = C::kSplitK ? 0 : wave & 1;
  const int tp = pt * T;
  at.tq = qt * T;
  at.wq = at.tq + wq * F * 16;
  at.q0 = at.wq + 4 * (lane >> 4);
  at.p0 = tp + (C::kSplitK ? wave : wp * F) * 16 + (lane & 15);
  typename Epi::template Pre<F, C::FP> pre;
  pre.load(at, e);

  const i32x4 ra = gemm_rsrc(g.a + at.batch * g.a_batch, (KSA ? g.k : g.q) * g.a_pitch);
  const i32x4 rb = gemm_rsrc(g.b + at.batch * g.b_batch, (KSB ? g.k : g.p) * g.b_pitch);
  Side<T, KSA, F> sa;
  Side<T, KSB, F> sb;
  sa.init(at.tq, g.q, g.a_pitch, tid, wq * F);
  sb.init(tp, g.p, g.b_pitch, tid, wp * F);
  const int step_a = sa.step(g.a_pitch), step_b = sb.step(g.b_pitch);

  // stages of SUB K-tiles: kt0 is this split's first K-tile
  const int kt0 = at.split * g.kt_per;
  const int kt_all = (g.k + kKV - 1) / kKV, kt_end = min(kt0 + g.kt_per, kt_all);
  const int nst = kt0 < kt_end ? (kt_end - kt0 + SUB - 1) / SUB : 0;  // 0: a split past the end, its sums are zeros
  const uint32_t lds_wave = (uint32_t)(uintptr_t)lds + wave * 1024;

  // load c of the stage whose first K-tile is kt, into LDS at `to` (A) and to_b. Only the
  // last stage (not `inner`) can hold K's last tile, whose first load cuts off
  // the values past the end, and K-tiles past the split's end, loaded with
  // every lane past the buffer's.
  const int left = g.k - (kt_all - 1) * kKV;
  auto dma_chunk = [&](int kt, uint32_t to, uint32_t to_b, auto inner, auto cc) {
    constexpr int c = decltype(cc)::value, sub = c / (2 * NL), k = c % (2 * NL);
    constexpr bool in = decltype(inner)::value;
    const int at_kt = in ? kt + sub : min(kt + sub, kt_all - 1);
    const bool past = !in && SUB > 1 && kt + sub >= kt_end;
    if constexpr (!in && (k == 0 || k == NL)) {
      if (left < kKV && kt + sub == kt_all - 1) {
        if constexpr (k == 0)
          sa.cut(left, tid);
        else
          sb.cut(left, tid);
      }
    }
    if constexpr (k < NL)
      load_lds<sub * 2 * TILE + k * 4096>(ra, to, past ? kPastEnd : sa.v[k], at_kt * step_a);
    else
      load_lds<sub * 2 * TILE + (k - NL) * 4096>(rb, to_b, past ? kPastEnd : sb.v[k - NL], at_kt * step_b);
  };
  auto read_frag2 = [&](lds_ptr st, lds_ptr st_b, int s, auto rc, i32x4(&af)[F], i32x4(&bf)[F]) {
    constexpr int r = decltype(rc)::value;
    // in the order of use: a[0], all of b, the rest of a
    if constexpr (r == 0)
      af[0] = sa.read(st, s, 0);
    else if constexpr (r <= F)
      bf[r - 1] = sb.read(st_b, s, r - 1);
    else
      af[r - F] = sa.read(st, s, r - F);
  };
  auto read_frag = [&](lds_ptr st, int s, auto rc, i32x4(&af)[F], i32x4(&bf)[F]) {
    read_frag2(st, st + TILE, s, rc, af, bf);
  };
  auto read_all = [&](lds_ptr st, int s, i32x4(&af)[F], i32x4(&bf)[F]) {
    StaticFor<0, 2 * F>::run([&](auto rc) { read_frag(st, s, rc, af, bf); });
  };

  f32x4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  acc_pin(acc);
  asm volatile("s_nop 4");
  auto mfma_range = [&](auto bc, auto ec, const i32x4(&af)[F], const i32x4(&bf)[F]) {
    StaticFor<decltype(bc)::value, decltype(ec)::value>::run([&](auto kc) {
      constexpr int k = decltype(kc)::value;
      mfma_acc<DT>(acc[k / F][k % F], af[k / F], bf[k % F]);
    });
  };
  auto mfma_all = [&](i32x4(&af)[F], i32x4(&bf)[F]) {
    operands_ready(af, bf);
    mfma_range(std::integral_constant<int, 0>{}, std::integral_constant<int, NMF>{}, af, bf);
  };
  // one slot's reads and loads, then W MFMAs; the MFMAs left over at the end
  constexpr int NR = 2 * F, W = 3 * NMF / 4 / NR;
  auto slots = [&](auto&& mem, const i32x4(&af)[F], const i32x4(&bf)[F]) {
    StaticFor<0, NR>::run([&](auto rc) {
      constexpr int r = decltype(rc)::value;
      mem(rc);
      mfma_range(std::integral_constant<int, r * W>{}, std::integral_constant<int, (r + 1) * W>{}, af, bf);
    });
    mfma_range(std::integral_constant<int, NR * W>{}, std::integral_constant<int, NMF>{}, af, bf);
  };

  // the sparse term's first labels, loaded behind the product (as p of this tile, or -1)
  constexpr int LR = Epi::kSparse ? 8 : 1;
  int lab[LR];
  auto load_labels = [&](int base) {
    if constexpr (Epi::kSparse) {
      const SparseTerm sp = Epi::sparse(e);
      const int r1 = min(kt_end * kKV, g.k);
#pragma unroll
      for (int u = 0; u < LR; ++u) {
        const int r = base + 64 * LR * wave + 64 * u + lane;
        const int64_t l = r < r1 ? label_raw(sp.labels, sp.label_bytes, r) - sp.p_base - tp : -1;
        lab[u] = l >= 0 && l < T && l + tp < g.p ? (int)l : -1;
      }
    }
  };
  load_labels(kt0 * kKV);

  i32x4 a0[F], b0[F], a1[F], b1[F];
  if (nst > 0) {
#pragma unroll
    for (int k = 0; k < NST; ++k) {
      if (k < nst) {
        const int kt = kt0 + k * SUB;
        StaticFor<0, CH>::run([&](auto cc) { dma_chunk(kt, lds_wave + k * STAGE, lds_wave + k * STAGE + TILE, std::false_type{}, cc); });
      }
    }
    if (nst >= NST)
      wait_loads<(NST - 1) * CH>();
    else
      wait_loads<0>();
    wg_barrier();
    int cur = 0;  // byte offset of stage t
    if constexpr (C::kSplitK) {
      // a wave's quarter of a stage: K-tile wave / 2, half wave % 2
      const lds_ptr mine = lds + (wave >> 1) * 2 * TILE;
      const int half = wave & 1;
      read_all(mine, half, a0, b0);
      auto body = [&](int t, auto inner, i32x4(&af)[F], i32x4(&bf)[F], i32x4(&an)[F], i32x4(&bn)[F]) {
        const int next = cur + STAGE == NST * STAGE ? 0 : cur + STAGE;
        if (t + NST <= nst)
          wait_loads<(NST - 2) * CH>();
        else
          wait_loads<0>();
        wg_barrier();  // stage t + 1 is in LDS, stage t is in registers
        slots(
            [&](auto rc) {
              if (decltype(inner)::value || t + NST < nst) dma_chunk(kt0 + (t + NST) * SUB, lds_wave + cur, lds_wave + cur + TILE, inner, rc);
              read_frag(mine + next, half, rc, an, bn);
            },
            af, bf);
        cur = next;
      };
      int t = 0;
      for (; t + 2 + NST < nst; t += 2) {
        body(t, std::true_type{}, a0, b0, a1, b1);
        body(t + 1, std::true_type{}, a1, b1, a0, b0);
      }
      for (; t + 1 < nst; ++t) {
        body(t, std::false_type{}, a0, b0, a1, b1);
        StaticFor<0, F>::run([&](auto kc) {
          constexpr int k = decltype(kc)::value;
          a0[k] = a1[k];
          b0[k] = b1[k];
        });
      }
      mfma_all(a0, b0);
    } else if constexpr (C::kUnits) {
      // Five units of one operand's K-tile: A(t) in unit 2 t mod 5, B(t) in the next. A(t + 2)
      // is loaded in the first half of K-tile t (its unit held B(t - 1)), B(t + 2) in the second
      // (its unit held A(t)): a load has at least a K-tile and a half, or a K-tile, to arrive.
      auto after = [](int u, int n) { return u + n * TILE >= 5 * TILE ? u + n * TILE - 5 * TILE : u + n * TILE; };
      int ua = 0, ub = TILE;
      read_all(lds, 0, a0, b0);
      constexpr int LW = NMF / NL;  // one load per so many MFMAs
      auto body = [&](int t, auto inner) {
        const int na = after(ua, 2), nb = after(ub, 2);
        const uint32_t fa = lds_wave + after(ua, 4), fb = lds_wave + ua;
        const bool more = decltype(inner)::value || t + 2 < nst;
        StaticFor<0, NMF>::run([&](auto kc) {
          constexpr int m = decltype(kc)::value;
          if constexpr (m % LW == 0)
            if (more) dma_chunk(kt0 + t + 2, fa, 0, inner, std::integral_constant<int, m / LW>{});
          if constexpr (m % W == 0 && m / W < NR)
            read_frag2(lds + ua, lds + ub, 1, std::integral_constant<int, m / W>{}, a1, b1);
          mfma_range(kc, std::integral_constant<int, m + 1>{}, a0, b0);
        });
        if (more)
          wait_loads<NL>();
        else
          wait_loads<0>();
        wg_barrier();  // K-tile t + 1 is in LDS, K-tile t is in registers
        StaticFor<0, NMF>::run([&](auto kc) {
          constexpr int m = decltype(kc)::value;
          if constexpr (m % LW == 0)
            if (more) dma_chunk(kt0 + t + 2, 0, fb, inner, std::integral_constant<int, NL + m / LW>{});
          if constexpr (m % W == 0 && m / W < NR)
            read_frag2(lds + na, lds + nb, 0, std::integral_constant<int, m / W>{}, a0, b0);
          mfma_range(kc, std::integral_constant<int, m + 1>{}, a1, b1);
        });
        ua = na;
        ub = nb;
      };
      int t = 0;
      for (; t + 3 < nst; ++t) body(t, std::true_type{});
      for (; t + 1 < nst; ++t) body(t, std::false_type{});
      slots([&](auto rc) { read_frag2(lds + ua, lds + ub, 1, rc, a1, b1); }, a0, b0);
      mfma_all(a1, b1);
    } else {
      read_all(lds, 0, a0, b0);
      auto body = [&](int t, auto inner) {
        const int next = cur + STAGE == NST * STAGE ? 0 : cur + STAGE;
        slots([&](auto rc) { read_frag(lds + cur, 1, rc, a1, b1); }, a0, b0);
        if (NST > 2 && t + NST <= nst)
          wait_loads<(NST - 2) * CH>();
        else
          wait_loads<0>();
        wg_barrier();  // K-tile t + 1 is in LDS, K-tile t is in registers
        // a load keeps the CU's memory path busy for 64 cycles (four waves of 16), as
        // long as four MFMAs
        constexpr int LW = NMF / CH;
        StaticFor<0, NMF>::run([&](auto kc) {
          constexpr int m = decltype(kc)::value;
          if constexpr (m % LW == 0)
            if (decltype(inner)::value || t + NST < nst)
              dma_chunk(kt0 + t + NST, lds_wave + cur, lds_wave + cur + TILE, inner, std::integral_constant<int, m / LW>{});
          if constexpr (m % W == 0 && m / W < NR) read_frag(lds + next, 0, std::integral_constant<int, m / W>{}, a0, b0);
          mfma_range(kc, std::integral_constant<int, m + 1>{}, a1, b1);
        });
        cur = next;
      };
      int t = 0;
      for (; t + 1 + NST < nst; ++t) body(t, std::true_type{});
      for (; t + 1 < nst; ++t) body(t, std::false_type{});
      slots([&](auto rc) { read_frag(lds + cur, 1, rc, a1, b1); }, a0, b0);
      mfma_all(a1, b1);
    }
    wait_loads<0>();
  }

  if constexpr (Epi::kSparse) {
    static_assert(KSA && KSB, "the sparse term gathers rows of A");
    const SparseTerm sp = Epi::sparse(e);
    int* const list = reinterpret_cast<int*>(smem + STAGE);  // stage 1: [kSparseCap], then [4] counts
    int* const counts = list + kSparseCap;
    const int r0 = kt0 * kKV, r1 = min(kt_end * kKV, g.k);
    int n = 0;
    wg_barrier();  // all waves have read the last stage
    for (int base = r0; base < r1; base += 256 * LR) {
      // rows whose label lies in this tile's p, in order: wave w takes 64 LR rows from
      // base + 64 LR w on
      if (base > r0) load_labels(base);
      int own[LR], cnt = 0;
#pragma unroll
      for (int u = 0; u < LR; ++u) {
        const uint64_t m = __ballot(lab[u] >= 0);
        own[u] = m >> lane & 1 ? cnt + __popcll(m & ((1ull << lane) - 1)) : -1;
        cnt += __popcll(m);
      }
      if (lane == 0) counts[wave] = cnt;
      __syncthreads();
      int at0 = n, all = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w < wave) at0 += counts[w];
        all += counts[w];
      }
#pragma unroll
      for (int u = 0; u < LR; ++u)
        if (own[u] >= 0) list[at0 + own[u]] = (base + 64 * LR * wave + 64 * u + lane) | lab[u] << kSparseRowBits;
      n += all;
      __syncthreads();
      // room for another 256 LR: list on; else, or at the end, multiply what is listed
      if (base + 256 * LR < r1 && n + 256 * LR <= kSparseCap) continue;
      for (int first = 0; first < n; first += SUB * kKV) {
        StaticFor<0, SUB * NL>::run([&](auto cc) {
          constexpr int sub = decltype(cc)::value / NL, c = decltype(cc)::value % NL;
          typedef Side<T, true, F> S;
          const int kk = first + sub * kKV + S::row_of(tid, c);
          const int col = at.tq + S::col_of(tid, c);
          const uint32_t off = kk < n && col < g.q ? (uint32_t)(list[kk] & kSparseRow) * (uint32_t)g.a_pitch + (uint32_t)col * 2 : kPastEnd;
          load_lds<sub * 2 * TILE + c * 4096>(ra, lds_wave, off, 0);
          *reinterpret_cast<i32x4*>(smem + sub * 2 * TILE + TILE + c * 4096 + tid * 16) = i32x4{0, 0, 0, 0};
        });
        __syncthreads();
        if (tid < SUB * kKV && first + tid < n) {
          const int r = list[first + tid] & kSparseRow, kk = tid % kKV;
          const int pl = (int)((uint32_t)list[first + tid] >> kSparseRowBits);
          const int off = kk * 2 * T + ((pl >> 4) ^ Side<T, true, F>::swz(kk)) * 32 + (pl & 15) * 2;
          *reinterpret_cast<uint16_t*>(smem + (tid / kKV) * 2 * TILE + TILE + off) = f32_to_bf16_bits(sp.delta[r]);
        }
        wait_loads<0>();
        __syncthreads();
        if constexpr (C::kSplitK) {
          read_all(lds + (wave >> 1) * 2 * TILE, wave & 1, a0, b0);
        } else {
          read_all(lds, 1, a1, b1);
          read_all(lds, 0, a0, b0);
          mfma_all(a1, b1);
        }
        mfma_all(a0, b0);
        wait_loads<0>();
        wg_barrier();
      }
      n = 0;
    }
  }
  asm volatile("s_nop 15\n\ts_nop 3");
  acc_pin(acc);

  wg_barrier();  // all waves have read the last stage
  at.lds = smem + wave * kRelay;
  if constexpr (C::kSplitK) {
    // the waves' sums, in the waves' order: wave w ends with the 16 p of fragment w
    i32x4* const sums = reinterpret_cast<i32x4*>(smem);
    StaticFor<0, F>::run([&](auto ic) {
      StaticFor<0, F>::run([&](auto jc) {
        constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
        sums[((wave * F + j) * F + i) * 64 + lane] = __builtin_bit_cast(i32x4, acc[i][j]);
      });
    });
    __syncthreads();
    f32x4 sum[F][1];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      sum[i][0] = __builtin_bit_cast(f32x4, sums[(wave * F + i) * 64 + lane]);
#pragma unroll
      for (int w = 1; w < 4; ++w) sum[i][0] += __builtin_bit_cast(f32x4, sums[((w * F + wave) * F + i) * 64 + lane]);
    }
    __syncthreads();
    Epi::template run<F, 1>(sum, at, e, pre);
  } else {
    Epi::template run<F, F>(acc, at, e, pre);
  }
}

template <int DT, int T, bool DEEP, bool KSA, bool KSB, class Epi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(DEEP ? 1 : 2, DEEP ? 1 : 2))) void
gemm_kernel(GemmArgs g, typename Epi::Args e) {
  __shared__ __attribute__((aligned(16))) char smem[Cut<T, DEEP>::LDS];
  gemm_tile_run<DT, T, DEEP, KSA, KSB, Epi>(g, e, smem, blockIdx.x, gridDim.x);
}

// Two products that do not wait for each other in one launch: the first n0
// workgroups run P0's, the others P1's. P: { KSA, KSB, Epi }.
template <int DT, int T, class P0, class P1>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void
gemm_pair_kernel(GemmArgs g0, typename P0::Epi::Args e0, int n0, GemmArgs g1, typename P1::Epi::Args e1) {
  __shared__ __attribute__((aligned(16))) char smem[Cut<T, true>::LDS];
  if ((int)blockIdx.x < n0)
    gemm_tile_run<DT, T, true, P0::KSA, P0::KSB, typename P0::Epi>(g0, e0, smem, blockIdx.x, n0);
  else
    gemm_tile_run<DT, T, true, P1::KSA, P1::KSB, typename P1::Epi>(g1, e1, smem, blockIdx.x - n0, gridDim.x - n0);
}

// ---- host side --------------------------------------------------------------

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Workgroups of a product with tiles of side t.
inline int64_t gemm_tiles(int64_t q, int64_t p, int t, bool symmetric) {
  const int64_t a = cdiv(q, t), b = cdiv(p, t);
  return symmetric ? a * (a + 1) / 2 : a * b;
}

// The tile order and the K-tiles per split.
inline void gemm_order(GemmArgs& g, int t, int splits) {
  g.nq = cdiv(g.q, t);
  // the 32 or 64 tiles that an XCD works on together make a block that is about
  // as wide as high: fewest rows fetched into its L2
  g.group = std::min(g.nq, t == 256 ? 6 : 8);
  g.splits = splits;
  g.kt_per = cdiv(cdiv(g.k, kKV), splits);
}

template <int DT, int T, bool DEEP, bool KSA, bool KSB, class Epi>
hipError_t gemm_launch_t(GemmArgs g, const typename Epi::Args& e, int splits, int batch, hipStream_t s) {
  gemm_order(g, T, splits);
  const int tiles = (int)gemm_tiles(g.q, g.p, T, Epi::kSymmetric);
  hipLaunchKernelGGL((gemm_kernel<DT, T, DEEP, KSA, KSB, Epi>), dim3(tiles * splits, 1, batch), dim3(256), 0, s, g, e);
  return hipGetLastError();
}

// Both in tiles of T, unsplit.
template <int DT, int T, class P0, class P1>
hipError_t gemm_launch_pair(GemmArgs g0, const typename P0::Epi::Args& e0, GemmArgs g1,
                            const typename P1::Epi::Args& e1, hipStream_t s) {
  gemm_order(g0, T, 1);
  gemm_order(g1, T, 1);
  const int n0 = (int)gemm_tiles(g0.q, g0.p, T, false), n1 = (int)gemm_tiles(g1.q, g1.p, T, false);
  hipLaunchKernelGGL((gemm_pair_kernel<DT, T, P0, P1>), dim3(n0 + n1), dim3(256), 0, s, g0, e0, n0, g1, e1);
  return hipGetLastError();
}

// Tile: 256 from 192 workgroups on (one a CU, three quarters of the CUs), else 128
// from 128 on, else 64. A wider tile reads less and has fewer workgroups. Head
// loss forward, 1024 channels, 4096 classes: 2816 rows (176 tiles of 256, 704 of
// 128) 36 us in 256 tiles, 34 in 128; 3200 rows (208 of 256) 37 and 40; 1024 rows
// (256 of 128, 1024 of 64) 20 us in 128 tiles, 24 in 64; below that the two are level
// up to 1024 channels. Update's symmetric products: 2048 x 4608 (136 of 128) 581 us a
// call in 128 tiles, 702 in 64; 1024 x 4608 (36 of 128) 358 and 249. Where most of
// a tile is padding or the 256 tiles are few over a round the rule is off: six
// matrices of 260 x 4608 take 316 us with steps in 256 tiles (216 of them, a third
// padding), 253 in 128; two of 2048 x 4608 (288) 1232 and 1023.
inline int gemm_tile(int64_t q, int64_t p, int64_t others, bool symmetric) {
  return gemm_tiles(q, p, 256, symmetric) * others >= 192   ? 256
         : gemm_tiles(q, p, 128, symmetric) * others >= 128 ? 128
                                                            : 64;
}

// Deep: as many workgroups as CUs or fewer have a CU's LDS each. A 256 tile always has.
inline bool gemm_deep(int64_t q, int64_t p, int tile, int64_t others, bool symmetric) {
  return tile == 256 || gemm_tiles(q, p, tile, symmetric) * others <= 256;
}

template <int DT, bool KSA, bool KSB, class Epi>
hipError_t gemm_launch(const GemmArgs& g, const typename Epi::Args& e, int tile, int splits, int batch,
                       hipStream_t s) {
  const bool deep = gemm_deep(g.q, g.p, tile, (int64_t)splits * batch, Epi::kSymmetric);
  switch (tile) {
    case 256: return gemm_launch_t<DT, 256, true, KSA, KSB, Epi>(g, e, splits, batch, s);
    case 128:
      return deep ? gemm_launch_t<DT, 128, true, KSA, KSB, Epi>(g, e, splits, batch, s)
                  : gemm_launch_t<DT, 128, false, KSA, KSB, Epi>(g, e, splits, batch, s);
    default:
      return deep ? gemm_launch_t<DT, 64, true, KSA, KSB, Epi>(g, e, splits, batch, s)
                  : gemm_launch_t<DT, 64, false, KSA, KSB, Epi>(g, e, splits, batch, s);
  }
}

}  // namespace
}  // namespace convnhwc
