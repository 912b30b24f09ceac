// mx.h -- MXFP8 and MXFP4 encoding of values that lie 8 to a lane, and loads and
// stores of any element alignment, shared by the kernels that write such rows.
#ifndef MXW_MX_H
#define MXW_MX_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxw {

// The bytes of a host call's argument (none: NULL, or no rows), to find outputs that overlap
// themselves or an input.
struct Span {
  uintptr_t lo = 0, hi = 0;
  Span() {}
  Span(const void* p, int64_t bytes) {
    if (p && bytes > 0) lo = (uintptr_t)p, hi = lo + (uintptr_t)bytes;
  }
  // rows of H elements, ld apart
  Span(const void* p, int64_t rows, int64_t ld, int64_t H, int size)
      : Span(p, rows > 0 ? (int64_t)((((uint64_t)rows - 1) * (uint64_t)ld + (uint64_t)H) * (uint64_t)size) : 0) {}
};
// whether one of the first `outs` meets another of them or any span behind them
template <int N>
bool overlap(const Span (&s)[N], int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < N; ++j)
      if (s[i].lo < s[j].hi && s[j].lo < s[i].hi) return true;
  return false;
}

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
// the same on an element's alignment (a vector access of any address is legal)
typedef int i4_a2 __attribute__((ext_vector_type(4), aligned(2)));

// bf16 of f, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const __bf16 h = (__bf16)f;
  return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 h = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, h);
}

// 8 elements of a row as they are stored
template <bool F32>
struct Raw8 {
  i4 v[F32 ? 2 : 1];
};

// NT: past the caches (data that is not met again before they have turned over)
template <bool F32, bool NT = false>
__device__ __forceinline__ Raw8<F32> load8(const void* base, int64_t at) {
  Raw8<F32> r;
  const i4_a2* p = (const i4_a2*)((const char*)base + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.v[i] = NT ? __builtin_nontemporal_load(p + i) : p[i];
  return r;
}
template <bool NT, class T>
__device__ __forceinline__ void store(T* p, const T& v) {
  if (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool F32, bool NT = false>
__device__ __forceinline__ void store8(void* base, int64_t at, const Raw8<F32>& r) {
  i4_a2* p = (i4_a2*)((char*)base + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    if (NT)
      __builtin_nontemporal_store(r.v[i], p + i);
    else
      p[i] = r.v[i];
  }
}
// 0 < n < 8 elements at an end (the others are 0).  All 7 loads are made, past the end of the
// last element again: in branches of their own each would wait for the one before.
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_some(const void* base, int64_t at, int n) {
  Raw8<F32> r;
  r.v[0] = (i4){0, 0, 0, 0};
  if (F32) r.v[F32 ? 1 : 0] = (i4){0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const int64_t from = at + min(i, n - 1);
    if (F32) {
      const int v = ((const int*)base)[from];
      r.v[F32 ? i >> 2 : 0][i & 3] = i < n ? v : 0;
    } else {
      const uint32_t v = ((const uint16_t*)base)[from];
      r.v[0][i >> 1] |= (int)(i < n ? v << (16 * (i & 1)) : 0u);
    }
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void store_some(void* base, int64_t at, const Raw8<F32>& r, int n) {
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) {
      if (F32)
        ((int*)base)[at + i] = r.v[F32 ? i >> 2 : 0][i & 3];
      else
        ((uint16_t*)base)[at + i] = (uint16_t)((uint32_t)r.v[0][i >> 1] >> (16 * (i & 1)));
    }
}

// The lane at column c of a row of H takes the 8 columns from c on.  SHARED, for rows of 8 and
// more: at the row's end the last 8, some of which are the lane's before it too: one access
// without a branch, and both lanes store the same bytes (by elements, each its own load, a
// gradient of 5,000 tokens x 3951 bf16, 4 rows each, took 109 us, now 75, of 3952 67; 264 of
// 501 joined from 8 rows 7.0 and 3.9; rows of whole lanes lose up to 1%).  Otherwise, for
// shorter rows and outputs of which another lane may still read what it shares, the columns
// that there are.
template <bool F32, bool NT, bool SHARED>
__device__ __forceinline__ Raw8<F32> load_row(const void* base, int64_t row, int c, int H) {
  if (SHARED) return load8<F32, NT>(base, row + min(c, H - 8));
  return c + 8 <= H ? load8<F32, NT>(base, row + c) : load_some<F32>(base, row + c, H - c);
}
template <bool F32, bool NT, bool SHARED>
__device__ __forceinline__ void store_row(void* base, int64_t row, int c, int H, const Raw8<F32>& r) {
  if (SHARED)
    store8<F32, NT>(base, row + min(c, H - 8), r);
  else if (c + 8 <= H)
    store8<F32, NT>(base, row + c, r);
  else
    store_some<F32>(base, row + c, r, H - c);
}

template <bool F32>
__device__ __forceinline__ void values(const Raw8<F32>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = F32 ? __int_as_float(r.v[F32 ? i >> 2 : 0][i & 3])
               : __uint_as_float((i & 1) ? (uint32_t)r.v[0][i >> 1] & 0xFFFF0000u : (uint32_t)r.v[0][i >> 1] << 16);
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> rounded(const float* f) {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (F32) {
      r.v[0][i] = __float_as_int(f[i]);
      r.v[F32 ? 1 : 0][i] = __float_as_int(f[4 + i]);
    } else {
      r.v[0][i] = (int)bf16_pair(f[2 * i], f[2 * i + 1]);
    }
  return r;
}

// The largest magnitude of a block of 32, 8 values in each of 4 neighbouring
// lanes, as its bits: of the magnitudes' bits the largest as whole numbers, so that
// a NaN comes out above infinity.
__device__ __forceinline__ uint32_t block_top(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
  return m;
}
// E8M0 byte of a block whose top binade the format's 2^BIN takes: 127 for zeros,
// 255 (NaN) if the block holds an infinity or a NaN.
template <int BIN>
__device__ __forceinline__ int block_scale(uint32_t top) {
  if (top == 0) return 127;
  if (top >= 0x7F800000u) return 255;
  // floor(log2 top) = frexp exponent - 1 (exact, subnormals included)
  return max(__builtin_amdgcn_frexp_expf(__uint_as_float(top)) - 1 - BIN + 127, 0);
}

// 8 E4M3 codes of a lane's values under its block's scale byte: to nearest, ties to
// even, saturated at 448, zeros as +0; 0x7F (NaN) under a NaN scale.  The scaling is a
// product with a power of two from 2^-119 to 2^127: exact wherever it counts.
__device__ __forceinline__ i2 encode_e4m3(const float* f, int s) {
  const float up = __uint_as_float((uint32_t)(254 - min(s, 253)) << 23);
  i2 q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_amdgcn_fmed3f(f[4 * h + i] * up, -448.0f, 448.0f);
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
    const uint32_t some = (((uint32_t)c & 0x7F7F7F7Fu) + 0x7F7F7F7Fu & 0x80808080u) >> 7;  // codes that are not +-0
    q[h] = s == 255 ? 0x7F7F7F7F : (int)((uint32_t)c & some * 0xFFu);
  }
  return q;
}

// 8 E2M1 codes, the first in the lowest half byte: to nearest, ties to even,
// saturated at 6, zeros as +0 (also under a NaN scale).
__device__ __forceinline__ uint32_t encode_e2m1(const float* f, int s) {
  const float up = __uint_as_float((uint32_t)(254 - min(s, 253)) << 23);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(f[i] * up, -6.0f, 6.0f);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
  const uint32_t some = ((c & 0x77777777u) + 0x77777777u & 0x88888888u) >> 3;
  return s == 255 ? 0u : c & some * 0xFu;
}

}  // namespace mxw

#endif  // MXW_MX_H
