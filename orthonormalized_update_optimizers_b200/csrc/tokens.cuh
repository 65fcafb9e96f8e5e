// Shared pieces of the token-matrix operators (8-bit quantization, norm,
// distillation loss, 8-bit product): argument checks that admit empty
// matrices, typed loads and stores of 8 elements, block reductions and the
// rounding to 8 bits.
#pragma once

#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "overlap.h"

namespace ouo {

// Checks one matrix whose elements have `es` bytes.  Unlike the optimizer's
// batches, a token matrix may be empty (no tokens in this batch): its pointer
// is then not looked at.
inline int validate_tokens(const ouo_mat& m, size_t es, const char* name, int i) {
  if (m.rows < 0 || m.cols < 0)
    return set_error(OUO_ERR_INVALID_ARG, "%s[%d]: negative shape %lld x %lld", name, i,
                     (long long)m.rows, (long long)m.cols);
  if (m.rows > (int64_t)1 << 30 || m.cols > (int64_t)1 << 30)
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

// An output in place of an input has to be that input, element for element.
inline int validate_in_place(const ouo_mat& out, int out_dtype, const ouo_mat& in, int in_dtype,
                             const char* names) {
  if (out.ptr == in.ptr && out.rows > 0 && out.cols > 0 &&
      (out_dtype != in_dtype || (out.rows > 1 && out.ld != in.ld)))
    return set_error(OUO_ERR_INVALID_ARG, "%s: in place needs the same type and row pitch", names);
  return OUO_OK;
}

// A device vector of `n` elements of `es` bytes.
inline int validate_vec(const void* p, int64_t n, size_t es, const char* name) {
  if (n > 0 && !p) return set_error(OUO_ERR_INVALID_ARG, "%s: NULL pointer", name);
  if ((uintptr_t)p % es != 0)
    return set_error(OUO_ERR_INVALID_ARG, "%s: not aligned to its element size", name);
  return OUO_OK;
}

// What a call reads or writes, for the check that outputs are apart from
// everything else.  `in_place`: the input that this output may be, if it starts
// where that does (validate_in_place has looked at the rest).
struct Operand {
  Span span;
  const char* name;
  const void* in_place = nullptr;
  const void* in_place2 = nullptr;
};

inline Operand operand(const ouo_mat& m, int64_t es, const char* name,
                       const void* in_place = nullptr, const void* in_place2 = nullptr) {
  return Operand{Span{(uintptr_t)m.ptr, m.rows, m.cols * es, m.ld * es}, name, in_place, in_place2};
}
inline Operand operand(const void* p, int64_t n, int64_t es, const char* name) {
  return Operand{Span{(uintptr_t)p, p ? 1 : 0, n * es, n * es}, name};
}

inline int validate_apart(std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (const Operand* o = outs.begin(); o != outs.end(); ++o) {
    for (const Operand& i : ins) {
      const void* p = (const void*)i.span.p;
      if (p == (const void*)o->span.p && p && (p == o->in_place || p == o->in_place2)) continue;
      if (overlap(o->span, i.span))
        return set_error(OUO_ERR_INVALID_ARG, "%s and %s overlap", o->name, i.name);
    }
    for (const Operand* q = o + 1; q != outs.end(); ++q)
      if (overlap(o->span, q->span))
        return set_error(OUO_ERR_INVALID_ARG, "%s and %s overlap", o->name, q->name);
  }
  return OUO_OK;
}

// Raises a kernel's shared-memory limit once per device.
struct Once {
  std::mutex mu;
  bool ready[64] = {false};
  template <class K>
  int smem(K kern, size_t bytes) {
    int dev = 0;
    OUO_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64)
      return set_error(OUO_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      OUO_CHECK_CUDA(
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
      ready[dev] = true;
    }
    return OUO_OK;
  }
};

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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float v[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
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
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = pack8(v);
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float round_to(float v, int bf16) {
  return bf16 ? bf16_to_f32(f32_to_bf16(v)) : v;
}

// The larger of m and |v|, NaN if either is NaN.
__device__ __forceinline__ float max_mag(float m, float v) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v)));
  return m;
}

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

// ------------------------------------------------------------------ teams
// A team of TPR threads (32, 128 or 512) holds one row of a matrix in
// registers: chunk c of thread t is elements 8 (t + c TPR) .. + 7, NV chunks a
// thread.  One read of the row then serves its norm, its largest magnitude
// and its rounding.  A block is one team, or four of one warp each.
template <int TPR>
constexpr int kTeamThreads = TPR < 128 ? 128 : TPR;

// Sum / maximum over a team.  `red` holds kTeamThreads / 32 words of shared
// memory, one set per reduction in flight (two reductions in a row use two
// sets, so that one barrier each is enough).
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) v += red[i];
  return v;
}

template <int TPR>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (TPR == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) v = max(v, red[i]);
  return v;
}

// Chunk of 8 elements starting at j of a row of n; vec: 16-byte loads allowed.
__device__ __forceinline__ void row_ld8(const void* p, int j, int n, int bf16, int vec,
                                        float v[8]) {
  if (vec && j + 8 <= n) {
    ld8(p, j, bf16, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j + i < n ? ld1(p, j + i, bf16) : 0.f;
  }
}

__device__ __forceinline__ void row_st8(void* p, int j, int n, int bf16, int vec,
                                        const float v[8]) {
  if (vec && j + 8 <= n) {
    st8(p, j, bf16, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < n) st1(p, j + i, v[i], bf16);
  }
}

// A thread's share of one row: NV chunks of 8 elements.  Loading and converting
// are separate, so that every load of the row is in flight before the first
// one is waited for.  The mode says, when the kernel is compiled, what the
// matrices are:
//   1, 2: all bf16 / fp32, 16-byte accesses, n a multiple of 8: chunk c of
//         thread t is elements 8 (t + c TPR) .. + 7;
//   3, 4: all bf16 / fp32, any alignment and n: element i of chunk c is
//         (8 c + i) TPR + t, so that a warp's accesses lie next to each other;
//   5:    a bf16 layer on an fp32 residual stream (norm only): 1 and 2;
//   0:    other mixtures: as 1 and 2, element by element where need be.
template <int TPR, int NV, int MODE>
struct RowRaw {
  uint4 a[MODE <= 2 ? NV : 1], b[MODE == 0 || MODE == 2 ? NV : 1];  // b: second half of fp32
  float f[MODE >= 3 ? NV : 1][8];

  __device__ __forceinline__ void load(const void* p, int t, int n, int bf16, int vec) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int i = t + c * TPR;
      if constexpr (MODE == 1) {
        a[c] = 8 * i < n ? q[i] : zero;
      } else if constexpr (MODE == 2) {
        a[c] = 8 * i < n ? q[2 * i] : zero;
        b[c] = 8 * i < n ? q[2 * i + 1] : zero;
      } else if constexpr (MODE >= 3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = (8 * c + e) * TPR + t;
          f[c][e] = j < n ? ld1(p, j, MODE == 3) : 0.f;
        }
      } else {
        float v[8];
        row_ld8(p, 8 * i, n, bf16, vec, v);
        a[c] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
        b[c] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                          __float_as_uint(v[7]));
      }
    }
  }

  __device__ __forceinline__ void get(float v[NV][8]) const {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if constexpr (MODE == 1) {
        unpack8(a[c], v[c]);
      } else if constexpr (MODE >= 3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = f[c][e];
      } else {
        const uint4 x = a[c], y = b[c];
        v[c][0] = __uint_as_float(x.x); v[c][1] = __uint_as_float(x.y);
        v[c][2] = __uint_as_float(x.z); v[c][3] = __uint_as_float(x.w);
        v[c][4] = __uint_as_float(y.x); v[c][5] = __uint_as_float(y.y);
        v[c][6] = __uint_as_float(y.z); v[c][7] = __uint_as_float(y.w);
      }
    }
  }
};

// The mode of the same accesses to the other type.
template <int MODE>
constexpr int kOtherType = MODE == 1 ? 2 : MODE == 2 ? 1 : MODE == 3 ? 4 : MODE == 4 ? 3 : 0;

template <int TPR, int NV, int MODE>
__device__ __forceinline__ void store_row(void* p, int t, int n, int bf16, int vec,
                                          const float v[NV][8]) {
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int j = 8 * (t + c * TPR);
    if (MODE >= 3) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = (8 * c + e) * TPR + t;
        if (k < n) st1(p, k, v[c][e], MODE == 3);
      }
    } else if (MODE == 0) {
      row_st8(p, j, n, bf16, vec, v[c]);
    } else if (j < n) {
      st8(p, j, MODE == 1, v[c]);
    }
  }
}

constexpr int64_t kTeamMost = 512 * 4 * 8;  // elements that a block's registers take

// How a matrix of rows x cols is given to teams: enough threads per row that
// a thread holds at most 8 chunks, and whole blocks per row where there are
// too few rows to fill the GPU with warps (a row's latency counts then), or
// where a row is read element by element (modes 3 and 4: then every element
// costs registers, and fewer a thread leave more threads to wait with).
// cols above kTeamMost do not fit: TPR 0.
struct Team {
  int tpr, nv;
};

inline Team team_for(int64_t rows, int64_t cols, int mode) {
  const int64_t chunks = ceil_div(cols, (int64_t)8);
  int tpr = chunks <= 32 * 8 ? 32 : chunks <= 128 * 8 ? 128 : 512;
  if (cols > kTeamMost) return Team{0, 0};
  if (rows < 4 * num_sms() || mode == 3 || mode == 4) tpr = chunks <= 128 ? (chunks <= 32 ? 32 : 128) : 512;
  int nv = 1;
  while ((int64_t)tpr * nv < chunks) nv *= 2;
  return Team{tpr, nv};
}

template <int I>
using C = std::integral_constant<int, I>;

// f(C<TPR>, C<NV>) for the team's instance.
template <class F>
int with_team_of(Team t, F&& f) {
  switch (t.tpr * 16 + t.nv) {
    case 32 * 16 + 1: return f(C<32>{}, C<1>{});
    case 32 * 16 + 2: return f(C<32>{}, C<2>{});
    case 32 * 16 + 4: return f(C<32>{}, C<4>{});
    case 32 * 16 + 8: return f(C<32>{}, C<8>{});
    case 128 * 16 + 1: return f(C<128>{}, C<1>{});
    case 128 * 16 + 4: return f(C<128>{}, C<4>{});
    case 128 * 16 + 8: return f(C<128>{}, C<8>{});
    case 512 * 16 + 1: return f(C<512>{}, C<1>{});
    case 512 * 16 + 2: return f(C<512>{}, C<2>{});
    default: return f(C<512>{}, C<4>{});
  }
}

// f(C<TPR>, C<NV>, C<MODE>): see RowRaw for the modes.
template <class F>
int with_team(Team t, int mode, F&& f) {
  return with_team_of(t, [&](auto tpr, auto nv) -> int {
    switch (mode) {
      case 1: return f(tpr, nv, C<1>{});
      case 2: return f(tpr, nv, C<2>{});
      case 3:
      case 4:  // of the teams that team_for gives these
        if constexpr (decltype(nv)::value == 1 || decltype(tpr)::value == 512)
          return mode == 3 ? f(tpr, nv, C<3>{}) : f(tpr, nv, C<4>{});
        return set_error(OUO_ERR_UNSUPPORTED, "no team of %d x %d takes single elements",
                         decltype(tpr)::value, decltype(nv)::value);
      case 5: return f(tpr, nv, C<5>{});
      default: return f(tpr, nv, C<0>{});
    }
  });
}

// 8-bit rounding of a row with the largest magnitude `amax`:
//   scale = amax / 127,  q = rint(x * (127 / amax)),  ties to even.
// An fp32 product with a rounded quotient can land on either side of a half
// that the exact value hits, and bf16 rows hit one often: x = amax / 2 is 63.5.
// With amax = a 2^i and x = m 2^j (a, m odd) the quotient is (127 m / a) 2^(j-i),
// a half-integer only if
//   * a divides m: then it is 63.5, the only odd multiple of 127 / 2 up to 127,
//     and 127 / amax rounded up keeps the product at or above it: 64;
//   * or a = 127 b: then amax / 127 is an fp32 number.  If 127 / amax is one
//     too (b = 1, the only such bf16 rows), products are exact.  Else (fp32
//     rows only, one in 127) the division's remainder corrects the product.
// So bf16 rows get the exact quotient's rounding; an fp32 quotient within
// 1e-5 of a half, but not on it, may go either way.  Below 2^-96 the quotient
// could overflow: there x and amax are multiplied by 2^96 (exact) first.  A
// zero row has scale 0 and zeros; a row with a NaN or an infinity has scale NaN
// and zeros, so that what is computed from it is NaN.
struct Quant {
  float scale, inv, pre;
  float unit;  // amax pre / 127 where products need the correction, else 0
};

// BF: the row is bf16, which no correction is needed for (and compiled into).
template <int BF>
__device__ __forceinline__ Quant quant_of(uint32_t amax_bits) {
  Quant q;
  const float amax = __uint_as_float(amax_bits);
  q.unit = 0.f;
  if (amax_bits >= 0x7f800000u) {
    q.scale = __uint_as_float(0x7fc00000u);
    q.inv = 0.f;
    q.pre = 0.f;
    return q;
  }
  q.scale = __fdiv_rn(amax, 127.f);
  q.pre = amax < 0x1p-96f ? 0x1p96f : 1.f;
  const float a = amax * q.pre;
  if (a > 0.f) {
    q.inv = __fdiv_rn(127.f, a);
    const float over = fmaf(q.inv, a, -127.f);  // of the rounded quotient, exact
    if (over < 0.f) q.inv = __uint_as_float(__float_as_uint(q.inv) + 1u);
    if (!BF) {
      const float unit = q.pre == 1.f ? q.scale : __fdiv_rn(a, 127.f);
      if (over != 0.f && fmaf(unit, 127.f, -a) == 0.f) q.unit = unit;
    }
  } else {
    q.inv = 0.f;
  }
  return q;
}

// The integer nearest to a value is in the low byte of its sum with 1.5 * 2^23,
// an fp32 sum whose last place is 1 (to nearest even; |x * inv| is at most 127
// up to rounding, so nothing needs clamping).
constexpr float kMagic = 12582912.f;

__device__ __forceinline__ int quant1(float x, const Quant& q) {
  if (q.pre == 0.f) return 0;
  const float v = x * q.pre;
  float s = fmaf(v, q.inv, kMagic);
  if (q.unit != 0.f) {
    const float p = v * q.inv;
    s = fmaf(fmaf(-p, q.unit, v), q.inv, p) + kMagic;
  }
  return (int8_t)(__float_as_uint(s) & 255u);
}

// Eight of them as 8 bytes; the rare rows that are not finite, tiny or
// corrected take the second branch together.
__device__ __forceinline__ uint2 quant8(const float v[8], const Quant& q) {
  uint32_t b[8];
  if (q.pre == 1.f && q.unit == 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(v[i], q.inv, kMagic));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (uint32_t)quant1(v[i], q);
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return o;
}

// Bytes j .. j+7 of a row of n; vec: the row starts on an 8-byte boundary.
__device__ __forceinline__ void row_stq(int8_t* p, int j, int n, int vec, uint2 v) {
  if (vec && j + 8 <= n) {
    *reinterpret_cast<uint2*>(p + j) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < n) p[j + i] = (int8_t)((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))) & 255u);
  }
}

// A thread's share of a row in 8 bits.
template <int TPR, int NV, int MODE>
__device__ __forceinline__ void store_q(int8_t* p, int t, int n, int vec, const float v[NV][8],
                                        const Quant& q) {
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const uint2 o = quant8(v[c], q);
    if (MODE >= 3) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = (8 * c + e) * TPR + t;
        if (k < n) p[k] = (int8_t)((e < 4 ? o.x >> (8 * e) : o.y >> (8 * (e - 4))) & 255u);
      }
    } else {
      row_stq(p, 8 * (t + c * TPR), n, vec, o);
    }
  }
}

}  // namespace ouo
