// Row access shared by the norm and the 8-bit checkpoint kernels: a row is read and written in
// chunks of 8 elements (one lane each), in bf16 or f32, at any element alignment, with a short
// last chunk; 16 consecutive chunks (16 consecutive lanes) are one 1x128 tile.
#pragma once

#include "device_common.h"

namespace moe {

// 16 and 8 bytes at element alignment (rows of odd widths): gfx950 reads and writes global memory
// at any byte address, so these stay single wide instructions.
typedef u32x4 u32x4_u __attribute__((aligned(2)));
typedef f32x4 f32x4_u __attribute__((aligned(4)));
typedef u32x2 u32x2_u __attribute__((aligned(1)));

enum { ROW_BF16 = 0, ROW_F32 = 1 };  // the values of MOE_BF16 and MOE_F32

template <int DT>
struct Raw8;
template <>
struct Raw8<ROW_BF16> {
  u32x4 v;
};
template <>
struct Raw8<ROW_F32> {
  f32x4 lo, hi;
};

// In the accessors below FULL says that rows are whole chunks (d % 8 == 0): without the short last
// chunk's element loads and stores the norm's backward kernel needs 30 registers less.

// Elements [c, c + 8) of a row of d elements; those at or past d read as zero.
template <int DT, bool FULL>
__device__ __forceinline__ Raw8<DT> load8(const void* row, int c, int d) {
  Raw8<DT> r;
  if constexpr (DT == ROW_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + c;
    if (FULL || c + 8 <= d) {
      r.v = *reinterpret_cast<const u32x4_u*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 2 * i < d ? p[2 * i] : 0u, hi = c + 2 * i + 1 < d ? p[2 * i + 1] : 0u;
        r.v[i] = lo | (hi << 16);
      }
    }
  } else {
    const float* p = static_cast<const float*>(row) + c;
    if (FULL || c + 8 <= d) {
      r.lo = *reinterpret_cast<const f32x4_u*>(p);
      r.hi = *reinterpret_cast<const f32x4_u*>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r.lo[i] = c + i < d ? p[i] : 0.f;
        r.hi[i] = c + 4 + i < d ? p[4 + i] : 0.f;
      }
    }
  }
  return r;
}

__device__ __forceinline__ void values8(const Raw8<ROW_BF16>& r, float f[8]) { unpack_bf16x8(r.v, f); }
__device__ __forceinline__ void values8(const Raw8<ROW_F32>& r, float f[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = r.lo[i];
    f[4 + i] = r.hi[i];
  }
}

// The same with the type known at run time only (it is uniform over the launch).
template <bool FULL>
__device__ __forceinline__ void load8_any(int dtype, const void* row, int c, int d, float f[8]) {
  if (dtype == ROW_BF16)
    values8(load8<ROW_BF16, FULL>(row, c, d), f);
  else
    values8(load8<ROW_F32, FULL>(row, c, d), f);
}

__device__ __forceinline__ u32x4 pack_bf16x8(const float f[8]) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16_rne(f[2 * i]) | (f32_to_bf16_rne(f[2 * i + 1]) << 16);
  return o;
}

// Stores 8 values at [c, c + 8) of a row of d elements (bf16: rounded to nearest even).
// With NT the stores are non-temporal: whole 16-byte pieces of lines that nothing reads again soon.
template <bool FULL, bool NT = false>
__device__ __forceinline__ void store8_any(int dtype, void* row, int c, int d, const float f[8]) {
  if (dtype == ROW_BF16) {
    uint16_t* p = static_cast<uint16_t*>(row) + c;
    const u32x4 o = pack_bf16x8(f);
    if (FULL || c + 8 <= d) {
      if constexpr (NT) __builtin_nontemporal_store(o, reinterpret_cast<u32x4_u*>(p));
      else *reinterpret_cast<u32x4_u*>(p) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < d) p[i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(row) + c;
    if (FULL || c + 8 <= d) {
      const f32x4 lo = {f[0], f[1], f[2], f[3]}, hi = {f[4], f[5], f[6], f[7]};
      if constexpr (NT) {
        __builtin_nontemporal_store(lo, reinterpret_cast<f32x4_u*>(p));
        __builtin_nontemporal_store(hi, reinterpret_cast<f32x4_u*>(p + 4));
      } else {
        *reinterpret_cast<f32x4_u*>(p) = lo;
        *reinterpret_cast<f32x4_u*>(p + 4) = hi;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < d) p[i] = f[i];
    }
  }
}

// 8 codes of a row of d bytes; bytes at or past d read as zero (the code of +0).
template <bool FULL>
__device__ __forceinline__ u32x2 load_codes8(const uint8_t* row, int c, int d) {
  if (FULL || c + 8 <= d) return *reinterpret_cast<const u32x2_u*>(row + c);
  u32x2 r = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < d) r[i / 4] |= (uint32_t)row[c + i] << (8 * (i & 3));
  return r;
}

template <bool FULL, bool NT = false>
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int d, const u32x2& q) {
  if (FULL || c + 8 <= d) {
    if constexpr (NT) __builtin_nontemporal_store(q, reinterpret_cast<u32x2_u*>(row + c));
    else *reinterpret_cast<u32x2_u*>(row + c) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) row[c + i] = (uint8_t)(q[i / 4] >> (8 * (i & 3)));
  }
}

// Lane exchanges inside the 16-lane rows of a wave (DPP row rotations): no LDS traffic.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  return max(v, row_ror<1>(v));
}

// One lane's 8 values of a 1x128 tile (the tile's 16 lanes in step, one DPP row) -> its E4M3 codes
// and the tile's E8M0 scale code, by the rule of fp8_quant_1x128_e8m0: the least 2^k with
// amax <= 448 * 2^k, v * 2^-k an exact product, RNE.  No scaled value exceeds 448, where the
// hardware conversion gives the codes of f32_to_e4m3 for every float (checked over all of them);
// a tile that holds an infinity or a NaN (its largest bit pattern says so) takes f32_to_e4m3,
// which saturates infinities and keeps NaN, with the scale of its other values.
__device__ __forceinline__ u32x2 ckpt_encode8(const float f[8], uint32_t& code) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  top = max16_u32(top);
  u32x2 q = {0u, 0u};
  if (top < 0x7f800000u) {
    const int k = e8m0_exponent(__uint_as_float(top));
    code = (uint32_t)(k + 127);
    const float inv = pow2f(-k);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
      q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, lo, true);
    }
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    const int k = e8m0_exponent(max16(amax));
    code = (uint32_t)(k + 127);
    const float inv = pow2f(-k);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i / 4] |= f32_to_e4m3(f[i] * inv) << (8 * (i & 3));
  }
  return q;
}

// 4 E4M3 codes -> their values times 2^(code - 127): the hardware's scaled conversion, exact for
// every code and every scale code 0..254 (a scale code of 255 is NaN).
__device__ __forceinline__ void ckpt_decode4(uint32_t q, uint32_t code, float f[4]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(code << 23);
  const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, false);
  const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, true);
  f[0] = lo[0];
  f[1] = lo[1];
  f[2] = hi[0];
  f[3] = hi[1];
}
__device__ __forceinline__ void ckpt_decode8(const u32x2& q, uint32_t code, float f[8]) {
  ckpt_decode4(q[0], code, f);
  ckpt_decode4(q[1], code, f + 4);
}

// Lanes of one launch: they are counted in 32 bits, and the last workgroup may be short.
constexpr int64_t kMaxLanes = ((int64_t)1 << 32) - 1024;

// Position of a lane's chunk when rows of `per_row` chunks are dealt out to workgroups of 256
// lanes: the workgroup's first chunk is split once (uniform), the lane's offset with a
// multiply-high (exact: offset < per_row + 256 and per_row < 2^15) or, where a row is longer than
// that, by one comparison.
struct RowSplit {
  uint32_t per_row;
  uint32_t magic;  // ceil(2^32 / per_row)
};
inline RowSplit make_row_split(uint32_t per_row) {
  return RowSplit{per_row, (uint32_t)((((uint64_t)1 << 32) + per_row - 1) / per_row)};
}
__device__ __forceinline__ void split_chunk(const RowSplit& sp, int64_t& row, int& chunk) {
  const int64_t base = (int64_t)blockIdx.x * 256;
  const int64_t r0 = base / sp.per_row;
  const uint32_t n = (uint32_t)(base - r0 * sp.per_row) + threadIdx.x;
  uint32_t k = 0;
  if (sp.per_row == 1) k = n;  // the multiplier of 1 does not fit 32 bits
  else if (sp.per_row < 32768) k = __umulhi(n, sp.magic);
  else k = n >= sp.per_row ? 1u : 0u;
  row = r0 + k;
  chunk = (int)(n - k * sp.per_row);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

}  // namespace moe
