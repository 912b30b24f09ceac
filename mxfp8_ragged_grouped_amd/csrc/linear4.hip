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
// group's scale is a number of the lane's own.  A lane loads 32 codes of its row at a
// time (16 bytes), 4 lanes a 128-wide step of k.
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

struct LinArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  int T, K, N, group;
  int split;      // waves that share a row tile's steps
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
// 8 codes n as the bf16 numbers 16 + n (0x4180 + 8 n), in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ i4 decode_int(uint32_t c) {
  i4 r;
  r.x = (int)((c << 3 & 0x00780078u) | 0x41804180u);
  r.y = (int)((c >> 1 & 0x00780078u) | 0x41804180u);
  r.z = (int)((c >> 5 & 0x00780078u) | 0x41804180u);
  r.w = (int)((c >> 9 & 0x00780078u) | 0x41804180u);
  return r;
}
// 8 tokens' values in that order
__device__ __forceinline__ i4 like_codes(const i4& v) {
  i4 r;
  r.x = (int)__builtin_amdgcn_perm((uint32_t)v.z, (uint32_t)v.x, 0x05040100u);
  r.y = (int)__builtin_amdgcn_perm((uint32_t)v.z, (uint32_t)v.x, 0x07060302u);
  r.z = (int)__builtin_amdgcn_perm((uint32_t)v.w, (uint32_t)v.y, 0x05040100u);
  r.w = (int)__builtin_amdgcn_perm((uint32_t)v.w, (uint32_t)v.y, 0x07060302u);
  return r;
}

// 4 x 4 words turned over between the 4 rows of 16 lanes: of lane (n, b), word i
// becomes word b of lane (n, i)
__device__ __forceinline__ i4 turn(i4 v) {
  typedef unsigned int u2 __attribute__((ext_vector_type(2)));
  u2 p = __builtin_amdgcn_permlane32_swap((uint32_t)v.x, (uint32_t)v.z, false, false);
  u2 q = __builtin_amdgcn_permlane32_swap((uint32_t)v.y, (uint32_t)v.w, false, false);
  u2 r = __builtin_amdgcn_permlane16_swap(p.x, q.x, false, false);
  u2 s = __builtin_amdgcn_permlane16_swap(p.y, q.y, false, false);
  return (i4){(int)r.x, (int)r.y, (int)s.x, (int)s.y};
}

template <bool OUT32>
__device__ __forceinline__ void put(const LinArgs& a, int t, int n, float v) {
  if (t < a.T && n < a.N) {
    if (OUT32)
      ((float*)a.out)[(int64_t)t * a.N + n] = v;
    else
      ((uint16_t*)a.out)[(int64_t)t * a.N + n] = (uint16_t)mxw::bf16_bits(v);
  }
}

// A workgroup: 4 / split row tiles of 16, each by `split` waves that take steps in turn.
template <bool FP4, int TT, int D, bool OUT32>
__global__ __launch_bounds__(256) void linear4_kernel(LinArgs a) {
  __shared__ float red[3][TT * 4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % a.split;
  const int n0 = (blockIdx.x * (4 / a.split) + wave / a.split) * 16;
  const int n = lane & 15, b = lane >> 4;
  const int64_t row = min(n0 + n, a.N - 1);
  const uint8_t* w = a.w + row * (a.K >> 1) + 16 * b;
  const int blocks = a.K >> 5, steps = (blocks + 3) >> 2;
  const uint16_t* x[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) x[i] = a.x + min(16 * i + n, a.T - 1) * a.ldx + (FP4 ? 32 * b : 8 * b);
  const int groups = FP4 ? blocks : a.K / a.group;
  const int per = FP4 ? 1 : a.group >> 5;  // blocks of a group
  const uint8_t* s8 = (const uint8_t*)a.scales + row * groups;
  const uint16_t* s16 = (const uint16_t*)a.scales + row * groups;
  const uint8_t* zero = a.zeros ? a.zeros + row * groups : nullptr;

  v4f sum[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) sum[i] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  i4 codes[D], xv[D][TT][4];
  uint32_t sc[D][4], ze[D][4];
  auto load = [&](int d, int step) {
    const bool in = 4 * step + b < blocks;
    codes[d] = (i4){0, 0, 0, 0};
    if (in) codes[d] = __builtin_nontemporal_load((const i4*)(w + 64 * step));
    if (FP4) {
      sc[d][0] = in ? s8[4 * step + b] : 0;
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[d][i][q] = in ? *(const i4*)(x[i] + 128 * step + 8 * q) : (i4){0, 0, 0, 0};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int block = 4 * step + q < blocks ? 4 * step + q : 0;
        sc[d][q] = s16[block / per];
        ze[d][q] = zero ? zero[block / per] : 8;
#pragma unroll
        for (int i = 0; i < TT; ++i) xv[d][i][q] = *(const i4*)(x[i] + 32 * block);
      }
    }
  };
  const i4 ones = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
  auto use = [&](int d, int step) {
    if (FP4) {
      const float s = __uint_as_float(sc[d][0] << 23);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i4 v = decode_fp4((uint32_t)codes[d][q], s);
#pragma unroll
        for (int i = 0; i < TT; ++i) sum[i] = mfma(xv[d][i][q], v, sum[i]);
      }
    } else {
      const i4 c = turn(codes[d]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * step + q >= blocks) continue;
        const i4 v = decode_int((uint32_t)c[q]);
        const float s = __uint_as_float(sc[d][q] << 16), z = s * (float)(16 + ze[d][q]);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
          const i4 xp = like_codes(xv[d][i][q]);
          const v4f dot = mfma(xp, v, none), all = mfma(xp, ones, none);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[i][r] = fmaf(s, dot[r], fmaf(-z, all[r], sum[i][r]));
        }
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (part + d * a.split < steps) load(d, part + d * a.split);
  for (int step = part; step < steps; step += D * a.split) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int now = step + d * a.split;
      if (now >= steps) break;
      use(d, now);
      if (now + D * a.split < steps) load(d, now + D * a.split);
    }
  }
  if (a.split > 1) {
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave - 1][4 * i + r][lane] = sum[i][r];
    }
    __syncthreads();
    if (part > 0) return;
    for (int p = 1; p < a.split; ++p)
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[i][r] += red[wave + p - 1][4 * i + r][lane];
  }
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) put<OUT32>(a, 16 * i + 4 * b + r, n0 + n, sum[i][r]);
}

bool on(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

}  // namespace

extern "C" int mxw_linear_4bit(const uint16_t* x, int64_t ldx, const uint8_t* codes, const void* scales,
                               const uint8_t* zeros, int format, int group, int T, int K, int N, void* out,
                               int out_type, void* stream) {
  const bool fp4 = format == MXW_MXFP4;
  if ((!fp4 && format != MXW_INT4) || T < 0 || T > MXW_MOE_MAX_TOKENS || K < 32 || K > 65536 || N < 1 ||
      N > (1 << 20) || ldx < K || (ldx & 7) || (out_type != MXW_BF16 && out_type != MXW_F32) ||
      (fp4 ? group != 32 || zeros : group != 32 && group != 64 && group != 128) || K % group)
    return MXW_ERR_DIM;
  if (!codes || !scales || (T && (!x || !out))) return MXW_ERR_NULL;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, fp4 ? 1 : 2) || !on(out, out_type == MXW_F32 ? 4 : 2))
    return MXW_ERR_ALIGN;
  if (const int rc = check_device()) return rc;
  if (T == 0) return MXW_OK;
  const int tiles = (N + 15) / 16, steps = (K + 127) / 128;
  int split = 1;
  while (split < 4 && tiles * split < 2048 && steps >= 4 * split) split *= 2;
  LinArgs a = {x, ldx, codes, scales, zeros, T, K, N, group, split, out};
  const dim3 grid((tiles + 4 / split - 1) / (4 / split)), block(256);
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto f, auto o) {
    constexpr bool F = decltype(f)::value, O = decltype(o)::value;
    switch ((T + 15) / 16) {
      case 1: linear4_kernel<F, 1, 4, O><<<grid, block, 0, st>>>(a); break;
      case 2: linear4_kernel<F, 2, 2, O><<<grid, block, 0, st>>>(a); break;
      case 3: linear4_kernel<F, 3, 2, O><<<grid, block, 0, st>>>(a); break;
      default: linear4_kernel<F, 4, 2, O><<<grid, block, 0, st>>>(a); break;
    }
  };
  using Y = std::true_type;
  using No = std::false_type;
  const bool o32 = out_type == MXW_F32;
  if (fp4)
    o32 ? go(Y{}, Y{}) : go(Y{}, No{});
  else
    o32 ? go(No{}, Y{}) : go(No{}, No{});
  return hipGetLastError() == hipSuccess ? MXW_OK : MXW_ERR_LAUNCH;
}
