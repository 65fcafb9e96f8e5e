// Shared pieces of the token-matrix operators (8-bit quantization, norm,
// distillation loss, 8-bit product): argument checks that admit empty
// matrices, typed loads and stores of 8 elements, block reductions and the
// rounding to 8 bits.
#pragma once

#include "internal.h"

namespace ouo {

// Checks one matrix whose elements have `es` bytes.  Unlike the optimizer's
// batches, a token matrix may be empty (no tokens in this batch): its pointer
// is then not looked at.
inline int validate_tokens(const ouo_mat& m, size_t es, const char* name, int i) {
  if (m.rows < 0 || m.cols < 0)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: negative shape %lld x %lld", name, i,
                     (long long)m.rows, (long long)m.cols);
  if (m.rows >= (int64_t)1 << 31 || m.cols >= (int64_t)1 << 31)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: shape too large", name, i);
  if (m.rows == 0 || m.cols == 0) return OUO_OK;
  if (!m.ptr) return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: NULL pointer", name, i);
  if (m.ld < m.cols)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: ld %lld < cols %lld", name, i,
                     (long long)m.ld, (long long)m.cols);
  if ((uintptr_t)m.ptr % es != 0)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: pointer not aligned to its element size",
                     name, i);
  return OUO_OK;
}

inline int validate_shape(const ouo_mat& m, int64_t rows, int64_t cols, const char* name, int i) {
  if (m.rows != rows || m.cols != cols)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d] is %lld x %lld, needs %lld x %lld", name, i,
                     (long long)m.rows, (long long)m.cols, (long long)rows, (long long)cols);
  return OUO_OK;
}

// A device vector of `n` elements of `es` bytes.
inline int validate_vec(const void* p, int64_t n, size_t es, const char* name) {
  if (n > 0 && !p) return set_error(OUO_ERR_INVALID_ARG, "%s: NULL pointer", name);
  if ((uintptr_t)p % es != 0)
    return set_error(OUO_ERR_INVALID_ARG, "%s: not aligned to its element size", name);
  return OUO_OK;
}

inline bool rows16(const ouo_mat& m, size_t es) {
  return (uintptr_t)m.ptr % 16 == 0 && (m.rows <= 1 || (size_t)m.ld * es % 16 == 0);
}

// -------------------------------------------------------------- device side

__device__ __forceinline__ float ld1(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i])
              : reinterpret_cast<const float*>(p)[i];
}

__device__ __forceinline__ void st1(void* p, int64_t i, float v, int bf16) {
  if (bf16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else reinterpret_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float v[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Elements i .. i+7 (p + i on a 16-byte boundary).
__device__ __forceinline__ void ld8(const void* p, int64_t i, int bf16, float v[8]) {
  if (bf16) {
    unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i), v);
  } else {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ void st8(void* p, int64_t i, int bf16, const float v[8]) {
  if (bf16) {
    uint4 u;
    u.x = pack_bf16x2(v[0], v[1]);
    u.y = pack_bf16x2(v[2], v[3]);
    u.z = pack_bf16x2(v[4], v[5]);
    u.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = u;
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float round_to(float v, int bf16) {
  return bf16 ? bf16_to_f32(f32_to_bf16(v)) : v;
}

// The larger of two magnitudes, NaN if either is: the bit patterns of
// non-negative floats order as integers, with NaN above infinity.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Sum / maximum over a block of at most 1024 threads; every thread gets the
// result.  `red` holds 32 words of shared memory and is free again on return.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0u;
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  return v;
}

// 8-bit rounding of a row with the largest magnitude `amax`:
//   scale = amax / 127,  q = rint(x * (127 / amax)).
// The quotient 127 / amax is rounded once, so x * inv is within 1.5 ulp of
// x / scale and q differs from the exact quotient's rounding only where that
// lies within 1e-5 of a half.  Below 2^-96 the reciprocal could overflow:
// there x and amax are multiplied by 2^96 (exact) first.  A zero row has scale
// 0 and zeros; a row with a NaN or an infinity has scale NaN and zeros, so
// that what is computed from it is NaN.
struct Quant {
  float scale, inv, pre;
};

__device__ __forceinline__ Quant quant_of(uint32_t amax_bits) {
  Quant q;
  const float amax = __uint_as_float(amax_bits);
  if (amax_bits >= 0x7f800000u) {
    q.scale = __uint_as_float(0x7fc00000u);
    q.inv = 0.f;
    q.pre = 0.f;
    return q;
  }
  q.scale = __fdiv_rn(amax, 127.f);
  q.pre = amax < 0x1p-96f ? 0x1p96f : 1.f;
  q.inv = amax > 0.f ? __fdiv_rn(127.f, amax * q.pre) : 0.f;
  return q;
}

__device__ __forceinline__ int quant1(float x, const Quant& q) {
  // inv is 0 for rows that are not finite; NaN * 0 converts to 0
  const int i = __float2int_rn(x * q.pre * q.inv);
  return max(-127, min(127, i));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | ((uint32_t)(b & 255) << 8) | ((uint32_t)(c & 255) << 16) |
         ((uint32_t)d << 24);
}

}  // namespace ouo
