// linear4.hip -- products of a few tokens with 4-bit weights (mxw_linear_4bit,
// declared in include/mxfp8_wgrad.h), for gfx950.
//
//     out[t][n] = sum_k x[t][k] v[n][k]
//     MXFP4:    v = e2m1(code) 2^(scale - 127), a scale for each 32 along k
//     integers: v = (code - zero) scale, a scale (and a zero) for each group of k
//
// Every weight is read once and nothing else is large: bound by reading HBM.  The
// products run on the bf16 MFMA 16 x 16 x 32 with up to 16 tokens as the first operand
// and 16 weight rows as the second, so that a lane holds sums of one weight row and its
// group's scale is a number of the lane's own.
//
// Measured (one MI355X, other weights from call to call, 300 calls in a row): 128,000 rows of K
// 7168, one token 87 us (MXFP4, 5.6 TB/s of codes and scales; reading alone reaches 7.0), 96
// (integers, groups of 128), 123 (groups of 32); 64 tokens 144, 210 and 316 (the first hundred
// calls after a pause up to a third longer, until the clock has settled): there operations
// bound it, not memory.  A step's products (96 of 16 cycles a wave, a third of them the tokens'
// own sums for the zeros) keep the matrix unit busy for 40% of the time and its other
// operations (340 of 4 to 5 cycles) the vector unit for about as much; other orders of the same
// work (products and decoding alternating, deeper prefetch of either operand, priorities, 16
// waves) gained nothing or lost.  32,000 rows of K 2048, one token: 8.9 us, of which launch and
// first loads take half.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"
#include "gemm16.h"
#include "mx.h"
#include "mxfp8_wgrad.h"

namespace {

using mxw::check_device;
using mxw::i4;
using mxw::v4f;
using mxw::v8bf;

typedef unsigned int u2v __attribute__((ext_vector_type(2)));

struct LinArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  int T, K, N, group;
  int steps;      // of 256 k, the last one may be partly past K
  int split;      // waves that share a row tile's steps
  int chunk;      // steps of x that LDS holds at a time, a multiple of split
  int chunks;
  int items;      // row tiles of a workgroup's size
  int f32;        // out is FP32
  void* out;
};

__device__ __forceinline__ v4f mfma(const i4& a, const i4& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// 8 E2M1 codes times 2^(scale - 127) as bf16, exactly
__device__ __forceinline__ i4 decode_fp4(uint32_t c, float scale) {
  i4 r;
  r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
  r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
  r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
  r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  return r;
}
// 8 codes n as the bf16 numbers n.  The bytes 0 .. 15 are E4M3's first 16 numbers,
// n 2^-9 (its subnormals and the binade above them have one step), so that the scaled
// conversion makes them whole numbers: 9 operations, where putting n into the bits of
// 16 + n takes 11 and leaves 16 to be taken off again.
__device__ __forceinline__ i4 decode_int(uint32_t c) {
  const uint32_t even = c & 0x0F0F0F0Fu, odd = c >> 4 & 0x0F0F0F0Fu;
  const int lo = (int)__builtin_amdgcn_perm(odd, even, 0x05010400u), hi = (int)__builtin_amdgcn_perm(odd, even, 0x07030602u);
  i4 r;
  r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return r;
}

// 4 x 4 words turned over between the 4 rows of 16 lanes: of lane (n, b), word i
// becomes word b of lane (n, i)
__device__ __forceinline__ i4 turn(i4 v) {
  const u2v p = __builtin_amdgcn_permlane32_swap((uint32_t)v.x, (uint32_t)v.z, false, false);
  const u2v q = __builtin_amdgcn_permlane32_swap((uint32_t)v.y, (uint32_t)v.w, false, false);
  const u2v r = __builtin_amdgcn_permlane16_swap(p.x, q.x, false, false);
  const u2v s = __builtin_amdgcn_permlane16_swap(p.y, q.y, false, false);
  return (i4){(int)r.x, (int)r.y, (int)s.x, (int)s.y};
}

// LDS-direct load of BYTES (1, 2, 16) a lane from offset voff + soff of the buffer, to 4 (16)
// bytes l of LDS byte `lds`; the range check leaves soff out, lanes out of the range write
// zeros
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void load_lds(const __amdgpu_buffer_rsrc_t& rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  static_assert(BYTES == 1 || BYTES == 2 || BYTES == 16, "a byte, a 16-bit word or four words");
  if (BYTES == 1)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
  else if (BYTES == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// all but the last N loads of this wave have landed
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}
// every LDS read of this wave has returned
__device__ __forceinline__ void wait_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
}

constexpr uint32_t kOut = 0xC0000000u;   // an offset past every buffer's range: loads give 0 and read nothing

// What a wave's slot of the ring holds for each 16 rows of a step of 256 k: 2 KiB of codes,
// and a word for every scale and zero.
template <int GC, int RT>
struct Slot {
  static constexpr int kScaleLoads = GC == 0 || GC == 4 ? 2 * RT : GC == 2 ? RT : (RT + 1) / 2;
  static constexpr int kLoads = 2 * RT + kScaleLoads * (GC == 0 ? 1 : 2);
  static constexpr int kScales = 2048 * RT, kZeros = kScales + 256 * kScaleLoads;
  static constexpr int kBytes = kZeros + (GC == 0 ? 0 : 256 * kScaleLoads);
};

// A workgroup: WAVES / split row tiles of 16 RT, each by `split` waves that take steps of
// 256 k in turn.  GC: groups of 128 k of integers (128 / group), 0: MXFP4.  R: how many of
// its 4 tokens a lane sums up (1 for a single token).
//
// The tokens are held in LDS, all of K (CH = 0), or CH steps at a time in two buffers,
// loaded straight to LDS a piece ahead.  16 bytes of token t at place p of its row lie at
// p' ^ t % 16 (p': place_of below): the LDS takes 256 bytes at a time, from lanes 0 .. 3 and
// 12 .. 15 of 16 and 4 .. 11 of the next 16, and their reads meet every bank once (with p
// itself half of them met another: a fifth of the kernel's time at 64 tokens).
//
// A wave brings its own rows' codes to its own ring of D slots in LDS, whole cache lines
// a load: read straight into the MFMA's layout, 16 lanes touch 16 lines, which makes the
// vector memory path the bound (one token, 128,000 x 7168: 143 us; this 88).  The ring runs on across
// pieces and row tiles.  Every step issues the same number of loads, which the waits count:
// what is past the end gets an offset out of its buffer's range and lands as zeros.
template <int GC, int TT, int RT, int D, int WAVES, int R, int CH>
__global__ __launch_bounds__(WAVES * 64) void linear4_kernel(LinArgs a) {
  constexpr bool FP4 = GC == 0, TURN = GC > 1, PIECES = CH > 0;
  using S = Slot<GC, RT>;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % a.split, sub = wave / a.split, subs = WAVES / a.split;
  const int n = lane & 15, b = lane >> 4;
  const int blocks = a.K >> 5, groups = FP4 ? blocks : a.K / a.group;
  const uint32_t wrow = (uint32_t)a.K >> 1;
  const uint32_t ring = wave * (D * S::kBytes), tokens0 = WAVES * (D * S::kBytes);

  // ---- tokens to LDS -----------------------------------------------------------
  // place in 128 k of the 16 bytes that lane b reads q-th
  auto place_of = [](int b, int q) { return TURN ? 4 * q + b : 4 * (2 * (b & 1) + ((b ^ b >> 1) & 1)) + q; };
  // and which of the row's 16 bytes lie at a place
  auto source_of = [](int p) {
    const int u = p >> 2;
    return TURN ? p : (p & ~12) | 4 * ((u >> 1 & 1) + 2 * ((u ^ u >> 1) & 1));
  };
  const int chunk = PIECES ? CH : a.chunk, per_row = chunk * 32;   // steps, and 16 bytes of a token, that LDS holds
  const int pieces = (PIECES ? 16 * TT : a.T) * per_row;
  const int rounds = PIECES ? TT * CH * 8 / WAVES : (pieces + WAVES * 64 - 1) / (WAVES * 64);
  const uint32_t buf = rounds * (WAVES * 1024);
  const __amdgpu_buffer_rsrc_t xr =
      mxw::buffer_of(a.x, mxw::range_of(((int64_t)(a.T - 1) * a.ldx + a.K) * 2));
  auto token_piece = [&](int h, int c, bool whole) {   // its offset, without the piece's
    const int i = (h * WAVES + wave) * 64 + lane, t = i / per_row, p = source_of((i - t * per_row) ^ (t & 15));
    return t < a.T && (whole || (c * per_row + p) * 8 < a.K) ? (uint32_t)(t * (int)a.ldx + 8 * p) * 2u : kOut;
  };
  constexpr int kRounds = PIECES ? TT * CH * 8 / WAVES : 1;
  uint32_t xo[kRounds];
  if (PIECES) {
#pragma unroll
    for (int h = 0; h < kRounds; ++h) xo[h] = token_piece(h, 0, true);
  }
  auto fetch = [&](int c, uint32_t to) {
    const bool whole = (c + 1) * chunk * 256 <= a.K;
    if (PIECES && whole) {
#pragma unroll
      for (int h = 0; h < kRounds; ++h) load_lds<16>(xr, to + (h * WAVES + wave) * 1024, xo[h], c * chunk * 512);
    } else {
      for (int h = 0; h < rounds; ++h)
        load_lds<16>(xr, to + (h * WAVES + wave) * 1024, token_piece(h, c, whole), c * chunk * 512);
    }
  };

  // ---- weights: a cursor that runs D steps ahead --------------------------------
  const int ends = a.chunks * chunk;       // steps of a row tile, rounded up
  int item = blockIdx.x, at = part;
  __amdgpu_buffer_rsrc_t wr, sr, zr;
  auto seek = [&] {
    // the ranges end with the tile's rows, so that an offset of kOut / 2 is past them too
    const int64_t row0 = ((int64_t)item * subs + sub) * (16 * RT), left = item < a.items ? a.N - row0 : 0;
    const int64_t base = left > 0 ? row0 : 0, rows = left < 16 * RT ? left : 16 * RT;
    wr = mxw::buffer_of(a.w + base * wrow, mxw::range_of(rows * wrow));
    sr = mxw::buffer_of((const uint8_t*)a.scales + base * groups * (FP4 ? 1 : 2),
                        mxw::range_of(rows * groups * (FP4 ? 1 : 2)));
    if (!FP4) zr = mxw::buffer_of(a.zeros + base * groups, a.zeros ? mxw::range_of(rows * groups) : 0u);
  };
  // codes: 8 rows of 128 bytes a load, 16 bytes c of row i at c ^ (i / 2) % 8; scales and
  // zeros: a word each, g of row i at g ^ 4 where i / 8 is odd and a row has 8 (bank conflicts)
  constexpr int kPer = FP4 ? 8 : 2 * GC;   // scales of a row and step
  uint32_t wo[2 * RT], so[S::kScaleLoads];
#pragma unroll
  for (int j = 0; j < 2 * RT; ++j) {
    const int row = 8 * j + (lane >> 3);
    wo[j] = row * wrow + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  auto group_of = [&](int j) { return (lane % kPer) ^ (kPer == 8 ? 4 * (j & 1) : 0); };
#pragma unroll
  for (int j = 0; j < S::kScaleLoads; ++j) {
    const int row = (j * 64 + lane) / kPer;
    so[j] = row < 16 * RT ? (uint32_t)(row * groups + group_of(j)) : kOut >> 1;
  }
  auto load = [&](int d) {
    const uint32_t to = ring + d * S::kBytes;
    const bool whole = 8 * at + 8 <= blocks;
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j) {
      uint32_t o = wo[j];
      if (!whole) o = 8 * at + ((lane & 7) ^ ((8 * j + (lane >> 3)) >> 1 & 7)) < blocks ? o : kOut;
      load_lds<16>(wr, to + 1024 * j, o, 128 * at);
    }
#pragma unroll
    for (int j = 0; j < S::kScaleLoads; ++j) {
      uint32_t o = so[j];
      if (!whole) o = kPer * at + group_of(j) < groups ? o : kOut >> 1;
      load_lds<FP4 ? 1 : 2>(sr, to + S::kScales + 256 * j, FP4 ? o : 2 * o, kPer * at * (FP4 ? 1 : 2));
      if (!FP4) load_lds<1>(zr, to + S::kZeros + 256 * j, o, kPer * at);
    }
    at += a.split;
    if (at >= ends) {
      at = part;
      item += gridDim.x;
      seek();
    }
  };

  v4f sum[RT][TT];
  const i4 ones = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
  // this lane's token rows in LDS (past T: the last, whose sums are not stored), and in
  // 128 k its 16 bytes of q
  uint32_t token[TT], place[4];
#pragma unroll
  for (int i = 0; i < TT; ++i)
    token[i] = (uint32_t)((PIECES ? 16 * i : min(16 * i + n, a.T - 1)) * per_row * 16);
#pragma unroll
  for (int q = 0; q < 4; ++q) place[q] = (uint32_t)((PIECES ? n * per_row * 16 : 0) + (place_of(b, q) ^ n) * 16);
  // A step's codes, and of its groups the scale and minus the zero, from slot d
  constexpr int G = FP4 ? 1 : GC, Q = 4 / G;
  i4 codes[2][RT];
  float scale[2][RT][G], zero[2][RT][G];
  auto take = [&](int d) {
    const uint8_t* slot = lds + (ring + d * S::kBytes);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        codes[h][j] = *(const i4*)(slot + 2048 * j + 128 * n + (((4 * h + b) ^ (n >> 1)) << 4));
        const int flip = kPer == 8 ? n >> 3 : 0;   // the half of the row's words
        const uint8_t* words = slot + 4 * ((16 * j + n) * kPer + (kPer == 8 ? 4 * (h ^ flip) + (FP4 ? b : 0) : GC * h));
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t s = *(const uint32_t*)(words + S::kScales + 4 * g);
          scale[h][j][g] = __uint_as_float(FP4 ? s << 23 : s << 16);
          if (!FP4)
            zero[h][j][g] = a.zeros ? -(float)*(const uint32_t*)(words + S::kZeros + 4 * g) : -8.0f;
        }
      }
  };
  // Its products with the tokens from LDS byte `from` on, 16 tokens of 128 k at a time.  The
  // reads of the next ones are set before the products: left to itself the compiler reads
  // each operand when it needs it, and waits.
  auto use = [&](uint32_t from) {
    i4 v[RT][4], x[2][4];
    auto read = [&](int u) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[u & 1][q] = *(const i4*)(lds + (from + place[q]) + (token[u % TT] + 256 * (u / TT)));
    };
    read(0);
#pragma unroll
    for (int u = 0; u < 2 * TT; ++u) {
      const int h = u / TT, i = u % TT;
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const i4 c = TURN ? turn(codes[h][j]) : codes[h][j];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[j][q] = FP4 ? decode_fp4((uint32_t)c[q], scale[h][j][0]) : decode_int((uint32_t)c[q]);
        }
      }
      if (u + 1 < 2 * TT) read(u + 1);
      __builtin_amdgcn_sched_barrier(0);
      const i4(&xu)[4] = x[u & 1];
      if (FP4) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < RT; ++j) sum[j][i] = mfma(xu[q], v[j][q], sum[j][i]);
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          v4f all = none, dot[RT];
#pragma unroll
          for (int j = 0; j < RT; ++j) dot[j] = none;
#pragma unroll
          for (int q = g * Q; q < (g + 1) * Q; ++q) {
            all = mfma(xu[q], ones, all);
#pragma unroll
            for (int j = 0; j < RT; ++j) dot[j] = mfma(xu[q], v[j][q], dot[j]);
          }
#pragma unroll
          for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int r = 0; r < R; ++r)
              // the scale last: times a zero it may leave FP32's range where the sum does not
              sum[j][i][r] = fmaf(scale[h][j][g], fmaf(zero[h][j][g], all[r], dot[j][r]), sum[j][i][r]);
        }
      }
    }
  };
  auto put = [&](int64_t row0) {
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int64_t row = row0 + 16 * j + n;
      if (row >= a.N) continue;
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int t = 16 * i + 4 * b + r;
          if (t >= a.T) continue;
          if (a.f32)
            ((float*)a.out)[(int64_t)t * a.N + row] = sum[j][i][r];
          else
            ((uint16_t*)a.out)[(int64_t)t * a.N + row] = (uint16_t)mxw::bf16_bits(sum[j][i][r]);
        }
    }
  };

  seek();
  fetch(0, tokens0);
#pragma unroll
  for (int d = 0; d < D; ++d) load(d);
  mxw::stage_barrier<D * S::kLoads>();
  uint32_t now = 0;   // the buffer of the piece
  int slot = 0;
  for (int it = blockIdx.x; it < a.items; it += gridDim.x) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < TT; ++i) sum[j][i] = none;
    for (int c = 0; c < a.chunks; ++c) {
      // the next piece of x, or the first again for the next row tile
      const bool more = PIECES && (c + 1 < a.chunks || it + (int)gridDim.x < a.items);
#pragma unroll 1
      for (int of = part; of < chunk; of += a.split) {
        const bool real = c * chunk + of < a.steps;
        wait_loads<(D - 1) * S::kLoads>();
        if (real) take(slot);
        // the slot is free, and its load has D - 1 steps and this one's products to land; the
        // next piece's loads go before it, so that the wait for them leaves it out
        wait_reads();
        if (more && of == part) fetch(c + 1 < a.chunks ? c + 1 : 0, tokens0 + (buf - now));
        load(slot);
        if (real) use(tokens0 + now + 512 * of);
        slot = slot + 1 == D ? 0 : slot + 1;
      }
      if (more) {
        // loads after the piece's: at least a step's
        mxw::stage_barrier<S::kLoads>();
        now = buf - now;
      }
    }
    const int64_t row0 = ((int64_t)it * subs + sub) * (16 * RT);
    if (RT == 1 && a.split > 1) {   // the parts are added in their order
      float* red = (float*)(lds + tokens0 + (PIECES ? 2 : 1) * buf) + sub * (a.split - 1) * (TT * 256);
      mxw::stage_barrier<D * S::kLoads>();
      if (part > 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r) red[(((part - 1) * TT + i) * 4 + r) * 64 + lane] = sum[0][i][r];
      }
      mxw::stage_barrier<D * S::kLoads>();
      if (part == 0) {
        for (int p = 1; p < a.split; ++p)
#pragma unroll
          for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) sum[0][i][r] += red[(((p - 1) * TT + i) * 4 + r) * 64 + lane];
        put(row0);
      }
    } else {
      put(row0);
    }
  }
  wait_loads<0>();   // no load outlives the ring's use
}

bool on(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

constexpr int kLds = 160 * 1024;

// CH: the steps of a piece where x does not fit in LDS, and then the most that a tile's steps
// are split
template <int GC, int TT, int RT, int D, int WAVES, int CH, int R = 4>
int launch(LinArgs a, hipStream_t st) {
  const int tiles = (a.N + 15) / 16;
  constexpr int ring = WAVES * D * Slot<GC, RT>::kBytes;
  a.split = 1;
  while (RT == 1 && a.split < WAVES && tiles * a.split < 256 * WAVES && a.steps >= 2 * a.split) a.split *= 2;
  auto joined = [&] { return a.split > 1 ? (WAVES - WAVES / a.split) * TT * 1024 : 0; };
  a.chunk = (a.steps + a.split - 1) / a.split * a.split;
  a.chunks = 1;
  int lds = ring + (a.T * a.chunk * 512 + WAVES * 1024 - 1) / (WAVES * 1024) * (WAVES * 1024) + joined();
  const bool pieces = lds > kLds;
  if (pieces) {
    while (a.split > CH) a.split /= 2;
    a.chunk = CH;
    a.chunks = (a.steps + CH - 1) / CH;
    lds = ring + 2 * TT * CH * 8192 + joined();
    static_assert(ring + 2 * TT * CH * 8192 + (RT == 1 ? (WAVES - WAVES / CH) * TT * 1024 : 0) <= kLds, "LDS");
  }
  const int rows = WAVES / a.split * RT;   // 16-row tiles of a workgroup
  a.items = (tiles + rows - 1) / rows;
  const dim3 grid(a.items < 256 ? a.items : 256), block(WAVES * 64);
  if (pieces)
    linear4_kernel<GC, TT, RT, D, WAVES, R, CH><<<grid, block, lds, st>>>(a);
  else
    linear4_kernel<GC, TT, RT, D, WAVES, R, 0><<<grid, block, lds, st>>>(a);
  return hipGetLastError() == hipSuccess ? MXW_OK : MXW_ERR_LAUNCH;
}
template <int GC>
int launch(const LinArgs& a, hipStream_t st) {
  const int tiles = (a.N + 15) / 16;
  // More tiles than one for each wave of a full device: two a wave, so that each read of the
  // tokens serves both (64 tokens, K 7168: 34,000 rows of MXFP4 60 us, with one 76; 32,000 rows
  // of integers, one round either way, 90 and 65).  A round is then 65,536 rows, and row counts
  // between rounds pay for a whole one, up to twice a full one's time a row: MXFP4, 64 tokens,
  // 34,000 rows 60 us, 66,000 126, 100,000 132, 128,000 144; one token 38, 74, 81 and 87.
  const bool wide = tiles > 2048;
  if (a.T == 1) return wide ? launch<GC, 1, 2, 1, 8, 4, 1>(a, st) : launch<GC, 1, 1, 2, 8, 4, 1>(a, st);
  if (a.T <= 16) return wide ? launch<GC, 1, 2, 1, 8, 4>(a, st) : launch<GC, 1, 1, 2, 8, 4>(a, st);
  // Half as many waves a workgroup where few tiles meet tokens that only fit in pieces: pieces
  // leave room for few parts of K, and more workgroups take the tiles (64 tokens, K 7168: 8,192
  // rows 22 us, with 8 waves 39; 20,000 rows 55 and 40.  24 tokens, 4,096 rows: K 7168 15 us
  // and 25, K 2048, which fits, 8.7 and 7.4).
  const bool few = tiles <= 1024 && a.T * a.steps * 512 + 8 * 2 * Slot<GC, 1>::kBytes > kLds;
  if (a.T <= 32)
    return wide  ? launch<GC, 2, 2, 1, 8, 2>(a, st)
           : few ? launch<GC, 2, 1, 2, 4, 4>(a, st)
                 : launch<GC, 2, 1, 2, 8, 2>(a, st);
  return wide  ? launch<GC, 4, 2, 1, 8, 1>(a, st)
         : few ? launch<GC, 4, 1, 2, 4, 2>(a, st)
               : launch<GC, 4, 1, 2, 8, 1>(a, st);
}

}  // namespace

extern "C" int mxw_linear_4bit(const uint16_t* x, int64_t ldx, const uint8_t* codes, const void* scales,
                               const uint8_t* zeros, int format, int group, int T, int K, int N, void* out,
                               int out_type, void* stream) {
  const bool fp4 = format == MXW_MXFP4;
  if ((!fp4 && format != MXW_INT4) || T < 0 || T > MXW_MOE_MAX_TOKENS || K < 32 || K > 65536 || N < 1 ||
      N > (1 << 20) || ldx < K || (ldx & 7) || ldx > (1 << 23) || (out_type != MXW_BF16 && out_type != MXW_F32) ||
      (fp4 ? group != 32 || zeros : group != 32 && group != 64 && group != 128) || K % group)
    return MXW_ERR_DIM;
  if (!codes || !scales || (T && (!x || !out))) return MXW_ERR_NULL;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, fp4 ? 1 : 2) || !on(out, out_type == MXW_F32 ? 4 : 2))
    return MXW_ERR_ALIGN;
  const int64_t groups = (int64_t)N * (K / group);
  if (mxw::overlap<5>({{out, (int64_t)T * N * (out_type == MXW_F32 ? 4 : 2)}, {x, T, ldx, K, 2}, {codes, (int64_t)N * K / 2},
                       {scales, groups * (fp4 ? 1 : 2)}, {zeros, groups}}, 1))
    return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  if (T == 0) return MXW_OK;
  LinArgs a = {};
  a.x = x, a.ldx = ldx, a.w = codes, a.scales = scales, a.zeros = zeros;
  a.T = T, a.K = K, a.N = N, a.group = group, a.steps = (K + 255) / 256, a.f32 = out_type == MXW_F32, a.out = out;
  hipStream_t st = (hipStream_t)stream;
  return fp4 ? launch<0>(a, st) : group == 128 ? launch<1>(a, st) : group == 64 ? launch<2>(a, st) : launch<4>(a, st);
}
