// gemm16.h -- the dense matrix product on 16-bit operands (bf16 or f16, FP32
// sums) under the orthogonalised update and the vocabulary loss, gfx950.
//
// C[m][n] = sum_k A(m, k) B(n, k), per batch entry.  Either operand may be
// stored K-contiguous (rows of k, "row" form) or with k as its slow axis
// ("column" form, TA / TB = true), so no caller transposes a matrix:
//
//     row form      A(m, k) = A[m lda + k]     LDS stage [BM][64 k], 128 B rows
//     column form   A(m, k) = A[k lda + m]     LDS stage [64 k][BM]
//
// A row-form stage is read 16 bytes (8 k) a lane; a column-form stage through
// the transposing LDS read (within 16 lanes, lane i element j receives element
// i % 4 of the 8 bytes that lane 4 j + i / 4 addresses; checked on gfx950), so
// both give the MFMA 16 x 16 x 32 the same fragment: lane l holds row l % 16 and
// k = 8 (l / 16) .. + 7 of a 32-deep part.
//
// A workgroup owns one BM x BN tile (WM x WN waves) and walks K in steps of 64
// through LDS stages (three of A, two of B: with 256 x 256 tiles the whole 160 KiB)
// filled by 16-byte LDS-direct buffer loads.  The buffer descriptor is rebased
// every step (64-bit), its range ending with the matrix: rows past the end read as
// zeros, so K and the tile edges need no masks as long as a row-form operand is
// stored with its k padded to a multiple of 64 by zeros.  In a column-form operand
// columns past the edge may read a neighbouring row's values: they feed only output
// rows or columns that are not stored.
//
// Tiles of 256 x 256 by 8 waves, one workgroup a CU, are the fastest where there
// are enough of them: the tile's bytes per flop are the least that LDS and the
// registers allow, and moving bytes costs the power that the MFMA runs on.  8192^3
// in bf16, calls in a row: 817 us (1,345 TFLOP/s; the library's product on the same
// board 733 us), MFMA 82% busy at 1.65 GHz.  By the fit below a step costs 1.45 us and
// a tile 11 us besides, most of them the burst of everyone's stores.
//
// The MFMA's first operand is B, so a lane ends with 4 consecutive n of one m:
// register r of block (mi, ni) in lane l is m = 16 mi + l % 16,
// n = 16 ni + 4 (l / 16) + r of the wave's part.
#ifndef MXW_GEMM16_H
#define MXW_GEMM16_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxw {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kGemmStep = 64;  // k per LDS stage: 128 bytes, one cache line a row

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// a buffer's range for so many bytes left
__device__ __forceinline__ uint32_t range_of(int64_t left) {
  return left <= 0 ? 0u : left > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)left;
}

// LDS-direct load: lane l's 16 bytes at byte offset voff of the buffer land at
// LDS byte lds + 16 l; lanes out of the buffer's range write zeros.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const __amdgpu_buffer_rsrc_t& rsrc, uint32_t lds, uint32_t voff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// all but the last N loads of this wave have landed and every LDS read has
// returned, then the workgroup's barrier; no memory access moves across
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ v4f mfma16(const v4i& a, const v4i& b, const v4f& c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma16(const v4i& a, const v4i& b, const v4f& c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// two floats rounded to nearest even, packed
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __bf16) {
  f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, _Float16) {
  f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
}

__device__ __forceinline__ v2i lds_read_tr(const uint8_t* p) {
  return __builtin_bit_cast(
      v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p)));
}

struct GemmArgs {
  const uint16_t* A;
  const uint16_t* B;
  int64_t strideA, strideB;  // elements from one batch entry to the next
  int lda, ldb;              // elements from one row (row form) or one k (column form) to the next
  int M, N, K;               // M (N) a multiple of 8 where A (B) is in column form
  int tilesM, tilesN;
  int tiles;    // tiles per (batch entry, split)
  int batch, splits;
  int ksplit;   // k per split, a multiple of 64
  int first;    // this launch's first of all batch * splits * tiles
  int cut;      // a workgroup's tile is one of 2^cut x 2^cut that such a tile is cut into
};

// Where the 16-byte chunks of a stage's rows lie, so that a fragment read, which
// takes 256 bytes at a time, meets every LDS bank once.  Row form (128-byte
// rows, 16 lanes at one chunk of 16 rows): chunk c of row r at c ^ (r / 2) % 8.
// Column form (32 lanes at 32 bytes of 8 different k, 0 .. 3 and 8 .. 11 after the
// first): chunk c of row k at c ^ (4 (k % 4) + 2 (k / 8 % 2)); in 128-byte rows
// (W = 64), of which two fill the banks, at c ^ (2 (k / 2 % 2) + 4 (k / 8 % 2)).
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }
template <int W>
__device__ __forceinline__ int col_swizzle(int k) {
  static_assert(W >= 64, "8 chunks a row");
  return W == 64 ? (k & 2) | ((k >> 1) & 4) : ((k & 3) << 2) | ((k >> 2) & 2);
}

// what an epilogue gets to know of its tile
struct TileAt {
  int batch, split, m0, n0;
  int wave, lane, wm, wn;  // the wave's part of the tile starts at row wm, column wn
  bool mirror;             // symmetric product, off the diagonal: the transposed tile is wanted too
};

// A tile of 16-bit values staged in LDS [BM][BN]: 16-byte chunk c of row r at
// position c ^ (r % chunks), so rows and columns are both read without bank
// conflicts that matter.
template <int BN>
__device__ __forceinline__ uint32_t tile_at(int r, int chunk) {
  constexpr int kChunks = BN / 8;
  return (uint32_t)(r * BN * 2 + ((chunk ^ (r & (kChunks - 1))) << 4));
}

// The workgroup's block index dealt so that each XCD (block index mod 8) gets
// one contiguous run of work, for its L2.
__device__ __forceinline__ int xcd_run(int b, int n) {
  const int q = n >> 3, r = n & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

// DEEP = 0: the rolling pipeline below.  DEEP > 0, for tiles whose step is shorter
// than a load's latency: a ring of DEEP stages of both operands, filled DEEP - 1
// steps ahead.
template <typename T, int BM, int BN, int WM, int WN, int DEEP, bool TA, bool TB, bool SYM, class Epi>
__global__ __launch_bounds__(WM* WN * 64, BM * BN / (WM * WN) > 8192 ? 1 : 2) void gemm16_kernel(GemmArgs p, typename Epi::Args ea) {
  constexpr int kWaves = WM * WN;
  constexpr int kPartM = BM / WM, kPartN = BN / WN;
  constexpr int MI = kPartM / 16, NI = kPartN / 16;
  constexpr int kBytesA = BM * 128, kBytesB = BN * 128;  // a stage of A, of B
  constexpr int kLoadsA = BM / 8, kLoadsB = BN / 8;  // 1 KiB loads per stage
  constexpr int LA = (kLoadsA + kWaves - 1) / kWaves, LB = (kLoadsB + kWaves - 1) / kWaves;
  // three stages of A and two of B, or the ring; the epilogue's tile takes their place
  constexpr int kLds = DEEP ? DEEP * (kBytesA + kBytesB) : 3 * kBytesA + 2 * kBytesB;
  static_assert(!Epi::kStaged || BM * BN * 2 <= kLds, "the staged tile fits");
  __shared__ __align__(1024) uint8_t lds[kLds];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  TileAt at;
  {
    const int run = xcd_run(blockIdx.x, gridDim.x);
    const int id = p.first + (run >> (2 * p.cut));
    const int t = id % p.tiles, bs = id / p.tiles;
    at.split = bs % p.splits;
    at.batch = bs / p.splits;
    int tm, tn;
    if (SYM) {  // the lower triangle, row by row
      tm = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
      while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
      while (tm * (tm + 1) / 2 > t) --tm;
      tn = t - tm * (tm + 1) / 2;
    } else {  // bands of 4 tile rows
      const int per = 4 * p.tilesN, band = t / per, in = t - band * per;
      const int rows = p.tilesM - 4 * band < 4 ? p.tilesM - 4 * band : 4;
      tn = in / rows;
      tm = 4 * band + in - tn * rows;
    }
    if (p.cut) {
      const int mask = (1 << p.cut) - 1;
      tm = (tm << p.cut) + ((run >> p.cut) & mask);
      tn = (tn << p.cut) + (run & mask);
      if (tm * BM >= p.M || tn * BN >= p.N || (SYM && tn > tm)) return;  // the whole workgroup
    }
    at.mirror = SYM && tm != tn;
    at.m0 = tm * BM;
    at.n0 = tn * BN;
  }
  at.wave = wave;
  at.lane = lane;
  at.wm = (wave / WN) * kPartM;
  at.wn = (wave % WN) * kPartN;
  const int kbeg = at.split * p.ksplit;
  const int kend = kbeg + p.ksplit < p.K ? kbeg + p.ksplit : p.K;
  const int steps = (kend - kbeg + kGemmStep - 1) / kGemmStep;

  // operand addressing: the tile's first byte, the bytes left in the matrix
  // from there, and the bytes a step advances
  const uint8_t *baseA, *baseB;
  int64_t leftA, leftB;
  uint32_t voA[LA], voB[LB];
  {
    const uint8_t* A = (const uint8_t*)(p.A + at.batch * p.strideA);
    const uint8_t* B = (const uint8_t*)(p.B + at.batch * p.strideB);
    const int64_t la = 2 * (int64_t)p.lda, lb = 2 * (int64_t)p.ldb;
    if (TA) {
      baseA = A + kbeg * la + 2 * at.m0;
      leftA = (kend - 1 - kbeg) * la + 2 * (int64_t)(p.M - at.m0);
    } else {
      baseA = A + at.m0 * la + 2 * kbeg;
      leftA = (p.M - at.m0 - 1) * la + 128 * (int64_t)steps;
    }
    if (TB) {
      baseB = B + kbeg * lb + 2 * at.n0;
      leftB = (kend - 1 - kbeg) * lb + 2 * (int64_t)(p.N - at.n0);
    } else {
      baseB = B + at.n0 * lb + 2 * kbeg;
      leftB = (p.N - at.n0 - 1) * lb + 128 * (int64_t)steps;
    }
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int u = wave + i * kWaves;
      if (TA) {
        constexpr int kLanes = BM / 8;  // lanes (16-byte chunks) a k
        const int k = u * (64 / kLanes) + lane / kLanes, c = lane % kLanes;
        voA[i] = (uint32_t)(k * la + ((c ^ col_swizzle<TA ? BM : 64>(k)) << 4));
      } else {
        const int r = u * 8 + (lane >> 3), c = lane & 7;
        voA[i] = (uint32_t)(r * la + ((c ^ row_swizzle(r)) << 4));
      }
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int u = wave + i * kWaves;
      if (TB) {
        constexpr int kLanes = BN / 8;
        const int k = u * (64 / kLanes) + lane / kLanes, c = lane % kLanes;
        voB[i] = (uint32_t)(k * lb + ((c ^ col_swizzle<TB ? BN : 64>(k)) << 4));
      } else {
        const int r = u * 8 + (lane >> 3), c = lane & 7;
        voB[i] = (uint32_t)(r * lb + ((c ^ row_swizzle(r)) << 4));
      }
    }
  }
  const int64_t stepA = TA ? 2 * (int64_t)kGemmStep * p.lda : 2 * kGemmStep;
  const int64_t stepB = TB ? 2 * (int64_t)kGemmStep * p.ldb : 2 * kGemmStep;
  const uint32_t ldsBase = (uint32_t)(uintptr_t)lds;

  // this wave's loads [from, to) of a stage of A (B); the last one moves on to
  // the next step
  auto fillA = [&](uint32_t at, int from, int to) {
#pragma unroll
    for (int i = from; i < to; ++i)
      if (kLoadsA % kWaves == 0 || wave + i * kWaves < kLoadsA)
        load_lds16(buffer_of(baseA, range_of(leftA)), at + i * kWaves * 1024, voA[i]);
    if (to == LA && from < to) {
      baseA += stepA;
      leftA -= stepA;
    }
  };
  auto fillB = [&](uint32_t at, int from, int to) {
#pragma unroll
    for (int i = from; i < to; ++i)
      if (kLoadsB % kWaves == 0 || wave + i * kWaves < kLoadsB)
        load_lds16(buffer_of(baseB, range_of(leftB)), at + i * kWaves * 1024, voB[i]);
    if (to == LB && from < to) {
      baseB += stepB;
      leftB -= stepB;
    }
  };

  // fragment addresses within a stage: of each 32-deep part (row form) or each
  // block of 16 rows (column form)
  uint32_t fa[TA ? MI : 2], fb[TB ? NI : 2];
  {
    const int g = lane >> 4, r = lane & 15;
    const int tk = 8 * g + (r >> 2), tc = (lane & 3) >> 1;
    if (TA) {
#pragma unroll
      for (int i = 0; i < (TA ? MI : 0); ++i)
        fa[i] = tk * BM * 2 + (((((at.wm >> 4) + i) * 2 + tc) ^ col_swizzle<TA ? BM : 64>(tk)) << 4) + ((lane & 1) << 3);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) fa[j] = (at.wm + r) * 128 + (((4 * j + g) ^ row_swizzle(r)) << 4);
    }
    if (TB) {
#pragma unroll
      for (int i = 0; i < (TB ? NI : 0); ++i)
        fb[i] = tk * BN * 2 + (((((at.wn >> 4) + i) * 2 + tc) ^ col_swizzle<TB ? BN : 64>(tk)) << 4) + ((lane & 1) << 3);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j] = (at.wn + r) * 128 + (((4 * j + g) ^ row_swizzle(r)) << 4);
    }
  }

  v4f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;

  // fragment i of part j (32 k) of the stage at byte `from`
  auto readA = [&](uint32_t from, int j, int i) -> v4i {
    const uint8_t* st = lds + from;
    if (TA) {
      const v2i lo = lds_read_tr(st + fa[TA ? i : 0] + 32 * j * BM * 2);
      const v2i hi = lds_read_tr(st + fa[TA ? i : 0] + (32 * j + 4) * BM * 2);
      return (v4i){lo.x, lo.y, hi.x, hi.y};
    }
    return *(const v4i*)(st + fa[TA ? 0 : j] + i * 16 * 128);
  };
  auto readB = [&](uint32_t from, int j, int i) -> v4i {
    const uint8_t* st = lds + from;
    if (TB) {
      const v2i lo = lds_read_tr(st + fb[TB ? i : 0] + 32 * j * BN * 2);
      const v2i hi = lds_read_tr(st + fb[TB ? i : 0] + (32 * j + 4) * BN * 2);
      return (v4i){lo.x, lo.y, hi.x, hi.y};
    }
    return *(const v4i*)(st + fb[TB ? 0 : j] + i * 16 * 128);
  };

  // The pipeline, in rows of NI MFMAs (one A fragment against all of B's): after
  // a row its A fragment is replaced by the next part's, and B's fragments of
  // the next part come in meanwhile, so every read has about a part's MFMAs to
  // return.  A step's only barrier stands kBefore rows into its second part (the
  // last reads return under those; 8192^3: 828 us with none before, 815 with two,
  // A by columns 845 and, with one, 839): it certifies that the next step's stages
  // have landed and that everyone has read this one's.
  // The loads are spread thinly (a CU's vector memory path takes a 1 KiB load
  // per ~16 clocks, and a wave that waits for it issues no MFMA): B's of the step
  // after next in the second part, into the stage just read, and A's of the step
  // after next in the first part, into the third A stage, so that they may be in
  // flight across the next barrier.
  constexpr int kOldest = kLoadsA % kWaves == 0 ? LA : 0;  // loads a barrier leaves in flight
  constexpr int kBefore = MI >= 8 && !TA ? 2 : 1, kAfter = MI - kBefore;
  constexpr int kBRow = (NI + kAfter - 1) / kAfter;  // B reads a row after the barrier
  if constexpr (DEEP > 0) {
    static_assert(kLoadsA % kWaves == 0 && kLoadsB % kWaves == 0, "every wave has the same loads");
    constexpr int kSlot = kBytesA + kBytesB;
    const uint32_t ldsWave = ldsBase + wave * 1024;
    auto fill = [&](int slot) {
      fillA(ldsWave + slot * kSlot, 0, LA);
      fillB(ldsWave + slot * kSlot + kBytesA, 0, LB);
    };
#pragma unroll
    for (int i = 0; i < DEEP - 1; ++i) fill(i);
    int slot = 0, next = DEEP - 1;
    for (int s = 0; s < steps; ++s) {
      stage_barrier<(DEEP - 2) * (LA + LB)>();  // this step's loads are here, the slot before it is free
      fill(next);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v4i a[MI], b[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) b[i] = readB(slot * kSlot + kBytesA, j, i);
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = readA(slot * kSlot, j, i);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = mfma16(b[ni], a[mi], acc[mi][ni], T());
      }
      slot = slot + 1 == DEEP ? 0 : slot + 1;
      next = next + 1 == DEEP ? 0 : next + 1;
    }
  } else {
    static_assert(NI <= MI && kBefore <= kAfter, "the rows hold the reads");
    const uint32_t ldsWave = ldsBase + wave * 1024;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fillA(ldsWave + i * kBytesA, 0, LA);
      fillB(ldsWave + 3 * kBytesA + i * kBytesB, 0, LB);
    }
    stage_barrier<kLoadsA % kWaves == 0 && kLoadsB % kWaves == 0 ? LA + LB : 0>();
    // in the order of the loop: a read's age tells the wait before its use
    v4i a[MI], b[2][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < NI) b[0][i] = readB(3 * kBytesA, 0, i);
      __builtin_amdgcn_sched_barrier(0);
      a[i] = readA(0, 0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    // every MFMA shares an operand with the one before it, across rows too: less
    // toggling, and under the power limit 1.5% more clock (8192^3: 849 -> 832 us on
    // one board)
    auto row = [&](int mi, const v4i& av, const v4i(&bv)[NI]) {
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int ni = mi & 1 ? NI - 1 - n : n;
        acc[mi][ni] = mfma16(bv[ni], av, acc[mi][ni], T());
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    uint32_t a0 = 0, a1 = kBytesA, a2 = 2 * kBytesA, b0 = 3 * kBytesA, b1 = b0 + kBytesB;
    for (int s = 0; s < steps; ++s) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        if (mi < NI) b[1][mi] = readB(b0, 1, mi);
        fillA(ldsWave + a2, mi * LA / MI, (mi + 1) * LA / MI);
        row(mi, a[mi], b[0]);
        a[mi] = readA(a0, 1, mi);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        const int after = mi - kBefore;
        if (after == 0) stage_barrier<kOldest>();
        if (after >= 0) {
#pragma unroll
          for (int i = after * kBRow; i < (after + 1) * kBRow && i < NI; ++i) b[0][i] = readB(b1, 0, i);
          if (after < kBefore) a[after] = readA(a1, 0, after);
          fillB(ldsWave + b0, after * LB / kAfter, (after + 1) * LB / kAfter);
        }
        row(mi, a[mi], b[1]);
        if (after >= 0) a[mi] = readA(a1, 0, mi);
        __builtin_amdgcn_sched_barrier(0);
      }
      uint32_t t = a0;
      a0 = a1;
      a1 = a2;
      a2 = t;
      t = b0;
      b0 = b1;
      b1 = t;
    }
  }
  // the loads past the last step (their range is empty: zeros) have landed too,
  // and the stages are free for the epilogue
  stage_barrier<0>();
  Epi::template run<BM, BN, WM, WN, MI, NI>(p, ea, at, acc, lds);
}

// ---- helpers for epilogues that stage a 16-bit tile -------------------------

// where the 4 values of row r from column c (a multiple of 4) on are staged
template <int BN>
__device__ __forceinline__ uint32_t staged_at(int r, int c) {
  return tile_at<BN>(r, c >> 3) + ((c & 4) << 1);
}

// a matrix's tile (16-byte aligned rows of ld elements, `rows` of them; what lies
// outside is not defined) to where one is staged; the caller waits for the loads
template <int BM, int BN, int WAVES>
__device__ __forceinline__ void load_tile(const TileAt& at, const uint8_t* lds, const uint16_t* src, int ld, int rows) {
  constexpr int kChunks = BN / 8, kRows = 64 / kChunks;  // rows a load
  static_assert(kChunks <= 64 && BM % (kRows * WAVES) == 0, "every wave has the same loads");
  const auto rsrc = buffer_of((const uint8_t*)(src + (int64_t)at.m0 * ld + at.n0),
                              range_of(2 * ((int64_t)(rows - at.m0) * ld - at.n0)));
#pragma unroll
  for (int u = at.wave; u < BM / kRows; u += WAVES) {
    const int r = u * kRows + at.lane / kChunks, c = at.lane % kChunks;
    load_lds16(rsrc, (uint32_t)(uintptr_t)lds + u * 1024, 2 * (r * ld + ((c ^ (r & (kChunks - 1))) << 3)));
  }
}

// the wave's part of the tile, its sums passed four at a time (row m, columns
// n .. n + 3, n a multiple of 4; i: the row's 16-row block in the part) through
// quad(i, m, n, v), rounded to T and staged
template <typename T, int BN, int MI, int NI, class F>
__device__ __forceinline__ void stage_part(const TileAt& at, const v4f (&acc)[MI][NI], uint8_t* lds, F quad) {
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = at.wm + 16 * i + (at.lane & 15);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int c = at.wn + 16 * j + 4 * (at.lane >> 4);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e];
      quad(i, at.m0 + r, at.n0 + c, v);
      const v2i w = {(int)pack2(v[0], v[1], T()), (int)pack2(v[2], v[3], T())};
      *(v2i*)(lds + staged_at<BN>(r, c)) = w;
    }
  }
}

// the staged tile to rows of dst: rows below nrows, columns below ncols.  Rows may
// start at any element: 16-byte stores need no alignment beyond it.  ONCE: nobody reads
// them soon, they need no place in the caches.
template <int BM, int BN, int WAVES, bool ONCE = false>
__device__ __forceinline__ void store_rows(const TileAt& at, const uint8_t* lds, uint16_t* dst, int64_t ld, int nrows,
                                           int ncols) {
  constexpr int kChunks = BN / 8;
  const int tid = at.wave * 64 + at.lane;
#pragma unroll 4
  for (int i = tid; i < BM * kChunks; i += WAVES * 64) {
    const int r = i / kChunks, c = i % kChunks;
    const int m = at.m0 + r, n = at.n0 + 8 * c;
    if (m >= nrows || n >= ncols) continue;
    const v4i v = *(const v4i*)(lds + tile_at<BN>(r, c));
    uint16_t* to = dst + m * ld + n;
    if (n + 8 <= ncols) {
      if (ONCE) __builtin_nontemporal_store(v, (v4i*)to);
      else __builtin_memcpy(to, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < ncols) to[e] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// the staged tile's transpose: dst[n][m], 16 bytes (8 m) a lane
template <int BM, int BN, int WAVES>
__device__ __forceinline__ void store_cols(const TileAt& at, const uint8_t* lds, uint16_t* dst, int64_t ld, int nrows,
                                           int ncols) {
  const int g = at.lane >> 4, i = at.lane & 15;
#pragma unroll 2
  for (int u = at.wave; u < (BM / 32) * (BN / 16); u += WAVES) {
    const int r0 = (u % (BM / 32)) * 32 + 8 * g, c0 = (u / (BM / 32)) * 16;
    const int r = r0 + (i >> 2), c = c0 + 4 * (i & 3);
    const v2i lo = lds_read_tr(lds + staged_at<BN>(r, c));
    const v2i hi = lds_read_tr(lds + staged_at<BN>(r + 4, c));
    const int n = at.n0 + c0 + i, m = at.m0 + r0;
    if (n < nrows && m < ncols) *(v4i*)(dst + n * ld + m) = (v4i){lo.x, lo.y, hi.x, hi.y};
  }
}

// ---- host: which tile -----------------------------------------------------------

// Hundredths of a us that `tiles` tiles of s steps take on `cus` CUs, fitted to the
// products of the two operators that use this at 35 shapes, forced to one tile (1 to
// 4,781 rows, 75 to 127,930 columns, 1 to 112 steps; most are met within a tenth).
// 256 x 256 and 128 x 256 stand alone on a CU: every round pays its first loads and
// its stores, and a step is shorter while CUs are idle (the clock is the power
// limit's).  Of the others two share a CU and hide that from each other; a last
// round that leaves a CU one is faster.
template <int BM, int BN>
inline int64_t tiles_cost(int64_t tiles, int64_t s, int64_t cus) {
  constexpr bool kAlone = BN == 256;
  const int64_t slots = kAlone ? cus : 2 * cus, full = tiles / slots, rest = tiles % slots;
  const bool single = rest <= cus;
  if (BM == 256) return full * (1100 + 145 * s) + (rest ? 1100 + s * (105 + 40 * rest / cus) : 0);
  if (kAlone) return full * (600 + 110 * s) + (rest ? 600 + s * (58 + 42 * rest / cus) : 0);
  if (BM == 128)
    return 500 + full * (400 + 95 * s) + (rest ? 100 + s * (single ? 48 : 80 + 25 * (rest - cus) / cus) : 0);
  if (BM == 64) return 100 + full * (220 + 43 * s) + (rest ? 200 + s * (single ? 37 : 50) : 0);
  return 300 + full * (250 + 31 * s) + (rest ? 200 + s * (single ? 20 : 29) : 0);  // 32 x 64
}

}  // namespace mxw

#endif  // MXW_GEMM16_H
