// int8_matmul: D = diag(a_scale) (A B^T) diag(b_scale), A (M x K) and B
// (N x K) 8-bit integers, the products summed exactly in 32 bits.
//
// Tensor cores (tcgen05.mma kind::i8, 32-bit integer accumulators in TMEM),
// operands staged by TMA, 128 bytes of K per stage in the 128-byte swizzle:
//   * pair kernel: clusters of two CTAs share a 256 x 256 tile (each stages its
//     128 rows of A and half of B's rows); persistent, two accumulators in
//     TMEM, so that a tile's epilogue (scales, rounding, store) runs under the
//     next tile's products.  Bound by the tensor pipe: 8192 x 14336 x 4096 in
//     333 us, 2.89 POP/s, the pipe 78% active (390 us under a long load, at the
//     1.33 GHz that the power limit leaves).
//   * split kernel: for few tokens, or outputs of few tiles.  128 rows of one
//     operand x BN rows of the other per cluster; the cluster's CTAs split K,
//     and join their 32-bit sums through distributed shared memory (integer
//     sums: the same bits in any order).  Bound by reading the larger operand,
//     and by some 4 us of set-up and join: 16 x 14336 x 4096 in 14.2 us.
// Matrices whose rows do not start on 16-byte boundaries cannot be read by the
// TMA; they take a CUDA-core kernel (dp4a).
// int8_matmul_deep, for depths whose sums leave 32 bits, cuts K into pieces that
// do not and adds those in 64 bits: the split kernel's eight CTAs, where it
// joins them, or in registers.
#include <cuda.h>

#include <cstring>
#include <mutex>

#include "tokens.cuh"
#include "umma.cuh"

namespace ouo {
namespace {

// CUDA cores: 64 x 64 tile per block, 32 bytes of K per step, 4 x 4 outputs
// per thread, four products per dp4a.  Takes any row pitch and alignment, byte
// by byte: 333 x 1024 x 4096 in 181 us (8.3 on the tensor cores), 1 x 14336 x
// 4096 in 209.
// DEEP: 32-bit sums of kSimtPiece elements are added in 64 bits.
constexpr int64_t kSimtPiece = OUO_INT8_MAX_DEPTH / 32 * 32;

template <int DEEP>
__global__ void __launch_bounds__(256)
s8_simt_kernel(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* as,
               const float* bs, void* D, int64_t ldd, int bf16, int64_t M, int64_t N, int64_t K,
               int64_t tiles_n) {
  __shared__ int sa[64][9], sb[64][9];
  const int64_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  long long wide[4][4] = {};
  int64_t next = kSimtPiece;
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    if (DEEP && k0 == next) {
      next += kSimtPiece;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          wide[i][j] += acc[i][j];
          acc[i][j] = 0;
        }
    }
    for (int e = threadIdx.x; e < 512; e += 256) {
      const int r = e >> 3, w = e & 7;
      int va = 0, vb = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t k = k0 + 4 * w + b;
        if (k < K && m0 + r < M) va |= (int)(uint8_t)A[(m0 + r) * lda + k] << (8 * b);
        if (k < K && n0 + r < N) vb |= (int)(uint8_t)B[(n0 + r) * ldb + k] << (8 * b);
      }
      sa[r][w] = va;
      sb[r][w] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      int x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = sa[ty * 4 + i][w];
        y[i] = sb[tx + 16 * i][w];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx + 16 * j;
      const float sum = DEEP ? (float)(wide[i][j] + acc[i][j]) : (float)acc[i][j];
      if (n < N) st1(D, m * ldd + n, sum * as[m] * bs[n], bf16);
    }
  }
}


// MT tokens, one or two: a warp per row of B (per 4 for two tokens), 16 bytes a
// lane and load, dp4a.  Bound by reading B; the tensor-core kernels' set-up (TMEM, barriers,
// a pipeline to fill) costs more than these few products.  A lane's share of K,
// a 32nd, fits in 32 bits at any depth; the lanes' sum is taken in two halves.
constexpr int kVecThreads = 128;
template <int MT>
constexpr int kVecRows = MT == 1 ? 1 : 4;

template <int MT>
__global__ void __launch_bounds__(kVecThreads)
s8_vec_kernel(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* as,
              const float* bs, void* D, int64_t ldd, int bf16, int N, int K) {
  constexpr int kR = kVecRows<MT>;
  const int lane = threadIdx.x & 31;
  const int64_t n0 = ((int64_t)blockIdx.x * (kVecThreads / 32) + (threadIdx.x >> 5)) * kR;
  if (n0 >= N) return;
  const int8_t* b[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) b[r] = B + (n0 + r < N ? n0 + r : N - 1) * ldb;
  int acc[kR][MT] = {};
  const int k16 = K & ~15;
  constexpr int kU = MT == 1 ? 4 : 2;
  for (int k = 16 * lane; k < k16; k += 512 * kU) {
    int4 x[kU][kR];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < kR; ++r)
        x[u][r] = k + 512 * u < k16 ? __ldcs(reinterpret_cast<const int4*>(b[r] + k + 512 * u))
                                    : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (k + 512 * u >= k16) break;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int4 y = *reinterpret_cast<const int4*>(A + m * lda + k + 512 * u);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          acc[r][m] = __dp4a(x[u][r].x, y.x, acc[r][m]);
          acc[r][m] = __dp4a(x[u][r].y, y.y, acc[r][m]);
          acc[r][m] = __dp4a(x[u][r].z, y.z, acc[r][m]);
          acc[r][m] = __dp4a(x[u][r].w, y.w, acc[r][m]);
        }
      }
    }
  }
  if (k16 + lane < K) {  // the last K % 16 bytes
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int y = A[m * lda + k16 + lane];
#pragma unroll
      for (int r = 0; r < kR; ++r) acc[r][m] += y * (int)b[r][k16 + lane];
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float s;
      if (K <= OUO_INT8_MAX_DEPTH) {
        s = (float)__reduce_add_sync(0xffffffffu, acc[r][m]);
      } else {
        const int hi = __reduce_add_sync(0xffffffffu, acc[r][m] >> 16);
        const int lo = __reduce_add_sync(0xffffffffu, acc[r][m] & 0xffff);
        s = (float)((long long)hi * 65536 + lo);
      }
      if (lane == r * MT + m && n0 + r < N)
        st1(D, m * ldd + n0 + r, s * as[m] * bs[n0 + r], bf16);
    }
}

// ------------------------------------------------------------ tensor cores

constexpr uint32_t kRowB = 128;                // bytes of K per stage
constexpr uint32_t kABytes = 128 * kRowB;      // 128 operand rows
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpiWarps;
constexpr int kGroupM = 8;  // row tiles that share B's columns in L2

struct S8Args {
  CUtensorMap tmA, tmB, tmD;
  const float* as;
  const float* bs;
  void* D;
  int64_t ldd;
  int bf16, tma_out, ragged;
  int M, N, nk;          // nk: K in stages
  int tiles_m, tiles_n;
  int64_t total;
  int* status;
};

// 128-byte swizzle position of a 4-byte column of a 32-row staging buffer: what
// the TMA store expects, and free of bank conflicts.
__device__ __forceinline__ int stg32(int row, int col) {
  return row * 32 + ((((col >> 2) ^ row) & 7) << 2) + (col & 3);
}
constexpr int kPairN = 256;  // columns of a pair's tile

struct PairCfg {
  static constexpr uint32_t kBBytes = (kPairN / 2) * kRowB;  // this CTA's half of B
  static constexpr uint32_t kStage = kABytes + kBBytes;
  static constexpr int kStages = 5;
  static constexpr uint32_t kTmemCols = 2 * kPairN;
  static constexpr uint32_t kEpi = kEpiWarps * 2 * 4096;  // two 4 KB buffers a warp
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpi + 512;
};

__device__ __forceinline__ void decode(const S8Args& a, int64_t t, int* ti, int* tj) {
  const int64_t width = (int64_t)kGroupM * a.tiles_n;
  const int g = (int)(t / width);
  const int64_t r = t - g * width;
  const int first = g * kGroupM;
  const int rows = min(a.tiles_m - first, kGroupM);
  *tj = (int)(r / rows);
  *ti = first + (int)(r - (int64_t)*tj * rows);
}

__global__ void __launch_bounds__(kPairThreads, 1)
s8_pair_kernel(const __grid_constant__ S8Args a) {
  using C = PairCfg;
  constexpr uint32_t kIdesc = ptx::instr_desc_s8(kPairN, 256);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* epi = smem + C::kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + C::kEpi);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int64_t tile0 = blockIdx.x / 2, step = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&tfull[s], 1);
      ptx::mbar_init(&tempty[s], kEpiWarps * 2);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&a.tmA);
    ptx::prefetch_tmap(&a.tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc2(holder, C::kTmemCols);
    ptx::tmem_relinquish2();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0 && lane == 0) {
    // producer: both CTAs' loads complete on the even CTA's stage barrier
    uint32_t stage = 0, phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t t = tile0; ok && t < a.total; t += step) {
      int ti, tj;
      decode(a, t, &ti, &tj);
      const int32_t arow = ti * 256 + (int32_t)rank * 128;
      const int32_t brow = tj * kPairN + (int32_t)rank * (kPairN / 2);
      for (int kb = 0; kb < a.nk; ++kb) {
        if (!ptx::mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * C::kStage);
        const uint32_t fb = ptx::mapa(ptx::smem_u32(&full[stage]), 0);
        uint8_t* sa = smem + stage * C::kStage;
        ptx::tma_load_2d_pair(sa, &a.tmA, fb, kb * (int)kRowB, arow);
        ptx::tma_load_2d_pair(sa + kABytes, &a.tmB, fb, kb * (int)kRowB, brow);
        ++issued;
        if (++stage == (uint32_t)C::kStages) { stage = 0; phase ^= 1; }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      report_status(a.status, OUO_STATUS_TIMEOUT);
      // loads in flight land before the CTA exits: the even CTA waits for
      // its barriers' last fill, the odd one (whose loads signal the even
      // CTA) a fixed 2 ms, far longer than a load takes
      if (rank != 0) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
        issued = 0;
      }
      for (int s = 0; s < C::kStages; ++s) {
        const int64_t fills = issued / C::kStages + (s < issued % C::kStages ? 1 : 0);
        if (fills > 0)
          ptx::mbar_wait_timed(&full[s], (uint32_t)((fills - 1) & 1), 100000000ull);
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // MMA issuer
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    int64_t local = 0;
    for (int64_t t = tile0; ok && t < a.total; t += step, ++local) {
      const uint32_t buf = (uint32_t)(local & 1);
      if (!ptx::mbar_wait(&tempty[buf], (uint32_t)((local >> 1) & 1) ^ 1, abort_flag)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t d = tmem + buf * kPairN;
      for (int kb = 0; kb < a.nk; ++kb) {
        if (!ptx::mbar_wait(&full[stage], phase, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sa = ptx::smem_u32(smem + stage * C::kStage);
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk)
          ptx::mma2_i8(d, ptx::smem_desc_sw128(sa + kk * 32, 16, 1024),
                       ptx::smem_desc_sw128(sa + kABytes + kk * 32, 16, 1024), kIdesc,
                       (kb > 0 || kk > 0) ? 1u : 0u);
        ptx::mma2_commit(&empty[stage], 0x3);
        if (++stage == (uint32_t)C::kStages) { stage = 0; phase ^= 1; }
      }
      if (!ok) break;
      ptx::mma2_commit(&tfull[buf], 0x3);
    }
    if (!ok) {
      *abort_flag = 1;
      report_status(a.status, OUO_STATUS_TIMEOUT);
    }
    ptx::mma2_commit(drain, 0x1);
    if (!ptx::mbar_wait_timed(drain, 0, kWaitLimitNs)) report_status(a.status, OUO_STATUS_TIMEOUT);
  } else if (warp >= 2) {
    // epilogue: one TMEM lane quarter and half of the columns per warp
    const uint32_t q = (uint32_t)(warp & 3), half = (uint32_t)((warp - 2) >> 2);
    constexpr int kCh = kPairN / 64;  // 32-column chunks per warp
    const uint32_t tempty_lead = ptx::mapa(ptx::smem_u32(tempty), 0);
    float* const stg0 = reinterpret_cast<float*>(epi + (warp - 2) * 8192);
    uint32_t nst = 0;
    int64_t local = 0;
    for (int64_t t = tile0; t < a.total; t += step, ++local) {
      int ti, tj;
      decode(a, t, &ti, &tj);
      const uint32_t buf = (uint32_t)(local & 1);
      const int row0 = ti * 256 + (int)rank * 128 + (int)q * 32;
      const int col0 = tj * kPairN + (int)half * (kPairN / 2);
      const float as = row0 + lane < a.M ? a.as[row0 + lane] : 0.f;
      float bs[kCh];  // lane's column of each chunk
#pragma unroll
      for (int c = 0; c < kCh; ++c)
        bs[c] = col0 + c * 32 + lane < a.N ? a.bs[col0 + c * 32 + lane] : 0.f;
      int ok = 1;
      if (lane == 0) ok = ptx::mbar_wait(&tfull[buf], (uint32_t)((local >> 1) & 1), abort_flag) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          report_status(a.status, OUO_STATUS_TIMEOUT);
        }
        break;
      }
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const int gj0 = col0 + c * 32;
        if (row0 >= a.M || gj0 >= a.N) continue;
        float v[32];
        ptx::tmem_ld32(tmem + ((q * 32u) << 16) + buf * kPairN + half * (kPairN / 2) + c * 32, v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j] = (float)__float_as_int(v[j]) * as * __shfl_sync(0xffffffffu, bs[c], j);
        float* stg = stg0 + (nst & 1u) * 1024;
        // The TMA store clips a box at 16 bytes, not at the element: a box over
        // D's last column goes by TMA only if the row ends on that boundary.
        const int box = a.bf16 ? gj0 - (c & 1) * 32 : gj0;
        if (a.tma_out && (!a.ragged || box + (a.bf16 ? 64 : 32) <= a.N)) {
          // a staging buffer is 32 rows of 128 bytes: 32 fp32 columns, or 64
          // bf16 ones, the second chunk filling the rows' second half
          const bool lo = !a.bf16 || (c & 1) == 0;
          const bool last = !a.bf16 || (c & 1) == 1 || gj0 + 32 >= a.N;
          if (lo) {  // the store before last has finished reading the buffer
            if (lane == 0) ptx::bulk_wait_read1();
            __syncwarp();
          }
          if (!a.bf16) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(stg + stg32(lane, j)) =
                  make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4*>(stg + stg32(lane, (c & 1) * 16 + j / 2)) = pack8(v + j);
          }
          if (last) {
            ptx::fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_2d(&a.tmD, stg, lo ? gj0 : gj0 - 32, row0);
              ptx::bulk_commit();
            }
            ++nst;
          }
        } else {
          if (lane == 0) ptx::bulk_wait_read0();  // stores by TMA have read the buffers
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(stg + stg32(lane, j)) =
                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          __syncwarp();
          if (gj0 + lane < a.N) {
            const int rows = min(32, a.M - row0);
            const int64_t o = (int64_t)row0 * a.ldd + gj0 + lane;
            if (a.bf16) {
              __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(a.D) + o;
#pragma unroll 8
              for (int r = 0; r < rows; ++r) d[r * a.ldd] = __float2bfloat16_rn(stg[stg32(r, lane)]);
            } else {
              float* d = reinterpret_cast<float*>(a.D) + o;
#pragma unroll 8
              for (int r = 0; r < rows; ++r) d[r * a.ldd] = stg[stg32(r, lane)];
            }
          }
          __syncwarp();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(tempty_lead + buf * 8u);
    }
    if (lane == 0) ptx::bulk_wait0();
    __syncwarp();
  }
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc2(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------ split kernel

constexpr int kSplitThreads = 192;
using C0 = std::integral_constant<int, 0>;
using C1 = std::integral_constant<int, 1>;

struct SplitArgs {
  CUtensorMap tmR, tmT;  // R: 128 rows a tile; T: BN rows a tile
  const float* rs;
  const float* ts;
  void* D;
  int64_t ldd;
  int bf16;
  int t_rows;   // D's rows are T's rows (else R's)
  int R, T, nk, nk_cta;
  int tiles_t;
  int vec;      // D rows on 16-byte boundaries
  int* status;
};

template <int BN>
struct SplitCfg {
  static constexpr uint32_t kTBytes = BN * kRowB;
  static constexpr uint32_t kStage = kABytes + kTBytes;
  // two CTAs a SM
  static constexpr int kStages = BN == 16 ? 6 : BN == 32 ? 5 : BN == 64 ? 4 : 3;
  static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 256;
  static_assert((size_t)BN * 512 <= (size_t)kStages * kStage, "partial sums reuse the stages");
};

// NS: CTAs of the cluster, which divide K.  DEEP: each one's sums fit in 32
// bits, all together in 64.
template <int BN, int NS, int DEEP>
__global__ void __launch_bounds__(kSplitThreads)
s8_split_kernel(const __grid_constant__ SplitArgs a) {
  using C = SplitCfg<BN>;
  constexpr uint32_t kIdesc = ptx::instr_desc_s8(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
  __shared__ __align__(16) float rs[128];
  __shared__ float ts[BN / NS];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = NS > 1 ? ptx::cluster_ctarank() : 0u;
  const int tile = (int)(blockIdx.x / NS);
  const int r0 = tile / a.tiles_t * 128, t0 = tile % a.tiles_t * BN;
  const int kb0 = (int)rank * a.nk_cta, kb1 = min(a.nk, kb0 + a.nk_cta);

  auto load = [&](int stage, int kb) {
    ptx::mbar_arrive_expect_tx(&full[stage], C::kStage);
    uint8_t* s = smem + stage * C::kStage;
    ptx::tma_load_2d(s, &a.tmR, &full[stage], kb * (int)kRowB, r0);
    ptx::tma_load_2d(s + kABytes, &a.tmT, &full[stage], kb * (int)kRowB, t0);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(done, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::fence_async_shared();  // the barriers, for the TMA
    // the first stages' loads need nobody else: they run under the set-up
    for (int i = 0; i < C::kStages && kb0 + i < kb1; ++i) load(i, kb0 + i);
  }
  if (warp == 1) {
    ptx::tmem_alloc(holder, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *holder;

  constexpr int kPer = BN / NS;            // T rows that this CTA writes
  const int first = t0 + (int)rank * kPer;  // its first one
  // the scales arrive under the products
  for (int i = threadIdx.x; i < kPer; i += kSplitThreads)
    ts[i] = first + i < a.T ? a.ts[first + i] : 0.f;
  if (threadIdx.x < 128) rs[threadIdx.x] = r0 + threadIdx.x < a.R ? a.rs[r0 + threadIdx.x] : 0.f;
  __syncwarp();

  if (warp == 0 && lane == 0) {
    // stages are refilled in order, as their products finish
    uint32_t stage = 0, phase = 0;
    int issued = min(C::kStages, max(0, kb1 - kb0));
    bool ok = true;
    for (int kb = kb0 + C::kStages; kb < kb1; ++kb) {
      if (!ptx::mbar_wait(&empty[stage], phase, abort_flag)) {
        ok = false;
        break;
      }
      load((int)stage, kb);
      ++issued;
      if (++stage == (uint32_t)C::kStages) { stage = 0; phase ^= 1; }
    }
    if (!ok) {
      *abort_flag = 1;
      report_status(a.status, OUO_STATUS_TIMEOUT);
      for (int s = 0; s < C::kStages; ++s) {
        const int fills = issued / C::kStages + (s < issued % C::kStages ? 1 : 0);
        if (fills > 0)
          ptx::mbar_wait_timed(&full[s], (uint32_t)((fills - 1) & 1), 100000000ull);
      }
    }
  } else if (warp == 1 && lane == 0) {
    uint32_t stage = 0, phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!ptx::mbar_wait(&full[stage], phase, abort_flag)) {
        *abort_flag = 1;
        report_status(a.status, OUO_STATUS_TIMEOUT);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t s = ptx::smem_u32(smem + stage * C::kStage);
#pragma unroll
      for (uint32_t kk = 0; kk < 4; ++kk)
        ptx::mma_i8(tmem, ptx::smem_desc_sw128(s + kk * 32, 16, 1024),
                    ptx::smem_desc_sw128(s + kABytes + kk * 32, 16, 1024), kIdesc,
                    (kb > kb0 || kk > 0) ? 1u : 0u);
      ptx::mma_commit(&empty[stage]);
      if (++stage == (uint32_t)C::kStages) { stage = 0; phase ^= 1; }
    }
    ptx::mma_commit(done);
    // after an aborted loop too: TMEM is released only when this is over
    if (!ptx::mbar_wait_timed(done, 0, kWaitLimitNs)) report_status(a.status, OUO_STATUS_TIMEOUT);
  }
  __syncwarp();
  // The products are done and the stages free, in every CTA of the cluster.
  if (NS > 1) ptx::cluster_sync();
  else __syncthreads();
  const uint32_t q = (uint32_t)(warp & 3);  // TMEM lanes 32 q .. + 31
  constexpr int kStep = BN < 32 ? 16 : 32;
  if (warp >= 2) ptx::tc_fence_after();
  auto sums = [&](int c, float v[kStep]) {  // columns c .. of the lane's row
    if (kb1 > kb0) {
      if (kStep == 16) ptx::tmem_ld16(tmem + ((q * 32u) << 16) + c, v);
      else ptx::tmem_ld32(tmem + ((q * 32u) << 16) + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < kStep; ++j) v[j] = 0.f;
    }
  };
  // Each CTA owns kPer of the T rows: it gets every CTA's sums for them (remote
  // stores, which nobody waits for), adds and writes them.
  int* part = reinterpret_cast<int*>(smem);  // [NS][kPer][128]
  if (warp >= 2) {
    uint32_t to[NS];
#pragma unroll
    for (int o = 0; o < NS; ++o) {
      const uint32_t at = ptx::smem_u32(part + (int)rank * kPer * 128 + q * 32 + lane);
      to[o] = NS > 1 ? ptx::mapa(at, o) : at;
    }
#pragma unroll
    for (int c = 0; c < BN; c += kStep) {
      float v[kStep];
      sums(c, v);
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const uint32_t at = to[(c + j) / kPer] + (uint32_t)((c + j) % kPer) * 512u;
        if (NS > 1) ptx::st_cluster_int(at, __float_as_int(v[j]));
        else part[(c + j) * 128 + q * 32 + lane] = __float_as_int(v[j]);
      }
    }
  }
  __syncwarp();
  if (NS > 1) ptx::cluster_sync();
  else __syncthreads();
  using Sum = std::conditional_t<DEEP, long long, int>;
  // Branched on the output's type once: a branch per element costs more than
  // the element (a 128 x 128 tile took 12,000 cycles to write).
  {
    const int n = min(kPer, a.T - first);
    auto write = [&](auto bf) {
      constexpr int BF = decltype(bf)::value;
      using E = std::conditional_t<BF, __nv_bfloat16, float>;
      if (a.t_rows) {
        const int r = r0 + 4 * lane;
        const bool wide = a.vec && r + 3 < a.R;
        const float4 s4 = *reinterpret_cast<const float4*>(rs + 4 * lane);
        E* d = reinterpret_cast<E*>(a.D) + (int64_t)first * a.ldd + r;
#pragma unroll 4
        for (int j = warp; j < n; j += kSplitThreads / 32) {
          Sum x[4] = {0, 0, 0, 0};
#pragma unroll
          for (int p = 0; p < NS; ++p) {
            const int4 y = *reinterpret_cast<const int4*>(part + (p * kPer + j) * 128 + 4 * lane);
            x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
          }
          const float t = ts[j];
          const float v[4] = {(float)x[0] * t * s4.x, (float)x[1] * t * s4.y,
                              (float)x[2] * t * s4.z, (float)x[3] * t * s4.w};
          E* o = d + (int64_t)j * a.ldd;
          if (wide) {
            if (BF) *reinterpret_cast<uint2*>(o) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
            else *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (r + k < a.R) o[k] = (E)v[k];
          }
        }
      } else if (threadIdx.x < 128 && r0 + threadIdx.x < a.R) {
        const int row = threadIdx.x;
        const float s = rs[row];
        E* d = reinterpret_cast<E*>(a.D) + (int64_t)(r0 + row) * a.ldd + first;
        auto value = [&](int j) {
          Sum x = 0;
#pragma unroll
          for (int p = 0; p < NS; ++p) x += part[(p * kPer + j) * 128 + row];
          return (float)x * s * ts[j];
        };
        if (kPer % 8 == 0 && a.vec && n == kPer) {
#pragma unroll 2
          for (int j = 0; j < kPer; j += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = value(j + k);
            st8(d, j, BF, v);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (j < n) d[j] = (E)value(j);
        }
      }
    };
    if (a.bf16) write(C1{});
    else write(C0{});
  }
  if (warp >= 2) ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------- host

int make_map(CUtensorMap* map, const ouo_mat& m, CUtensorMapDataType type, size_t es,
             uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swz) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return set_error(OUO_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows};
  // the pitch of a single row is not used, but has to be a valid one
  cuuint64_t strides[1] = {m.rows > 1 ? (cuuint64_t)m.ld * es
                                      : (cuuint64_t)align_up((size_t)m.cols * es, 16)};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, type, 2, m.ptr, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(OUO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return OUO_OK;
}

int map_s8(CUtensorMap* map, const ouo_mat& m, uint32_t box_rows) {
  return make_map(map, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kRowB, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaLaunchConfig_t config(unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                          unsigned cluster, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// What a kernel needs set once per device.
struct Setup {
  std::mutex mu;
  int slots[64] = {0};  // 0: not yet set up; else resident clusters
};

template <class K>
int setup(Setup& st, K kern, unsigned threads, size_t smem, unsigned cluster, int* slots) {
  int dev = 0;
  OUO_CHECK_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64)
    return set_error(OUO_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(st.mu);
  if (!st.slots[dev]) {
    OUO_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)smem));
    int n = 0;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(cluster * (unsigned)num_sms(), threads, smem, nullptr, cluster, attr);
    OUO_CHECK_CUDA(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
    if (n < 1) return set_error(OUO_ERR_UNSUPPORTED, "no cluster of the 8-bit product fits");
    st.slots[dev] = n;
  }
  *slots = st.slots[dev];
  return OUO_OK;
}

struct Product {
  ouo_mat A, B, D;
  const float* as;
  const float* bs;
  int bf16;
  int* status;
};

int run_pair(const Product& p, cudaStream_t s) {
  using C = PairCfg;
  static Setup st;
  int slots = 0;
  OUO_TRY(setup(st, s8_pair_kernel, kPairThreads, C::kSmem, 2, &slots));
  S8Args a;
  memset(&a, 0, sizeof(a));
  OUO_TRY(map_s8(&a.tmA, p.A, 128));
  OUO_TRY(map_s8(&a.tmB, p.B, kPairN / 2));
  const size_t es = p.bf16 ? 2 : 4;
  a.tma_out = rows16(p.D, es) ? 1 : 0;
  a.ragged = p.D.cols * es % 16 != 0;
  if (a.tma_out)
    OUO_TRY(make_map(&a.tmD, p.D,
                     p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                     es, p.bf16 ? 64 : 32, 32, CU_TENSOR_MAP_SWIZZLE_128B));
  a.as = p.as; a.bs = p.bs;
  a.D = p.D.ptr; a.ldd = p.D.ld; a.bf16 = p.bf16;
  a.M = (int)p.D.rows; a.N = (int)p.D.cols;
  a.nk = (int)ceil_div(p.A.cols, (int64_t)kRowB);
  a.tiles_m = (int)ceil_div(p.D.rows, 256);
  a.tiles_n = (int)ceil_div(p.D.cols, kPairN);
  a.total = (int64_t)a.tiles_m * a.tiles_n;
  a.status = p.status;
  const int64_t n = a.total < slots ? a.total : slots;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config((unsigned)(2 * n), kPairThreads, C::kSmem, s, 2, attr);
  OUO_CHECK_CUDA(cudaLaunchKernelEx(&cfg, s8_pair_kernel, a));
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

// t_rows: T is A (D's rows), R is B; else the other way round.
template <int BN, int NS, int DEEP>
int run_split(const Product& p, bool t_rows, cudaStream_t s) {
  using C = SplitCfg<BN>;
  static Once once;
  OUO_TRY(once.smem((s8_split_kernel<BN, NS, DEEP>), C::kSmem));
  SplitArgs a;
  memset(&a, 0, sizeof(a));
  const ouo_mat& R = t_rows ? p.B : p.A;
  const ouo_mat& T = t_rows ? p.A : p.B;
  OUO_TRY(map_s8(&a.tmR, R, 128));
  OUO_TRY(map_s8(&a.tmT, T, BN));
  a.rs = t_rows ? p.bs : p.as;
  a.ts = t_rows ? p.as : p.bs;
  a.D = p.D.ptr; a.ldd = p.D.ld; a.bf16 = p.bf16;
  a.t_rows = t_rows ? 1 : 0;
  a.R = (int)R.rows; a.T = (int)T.rows;
  a.nk = (int)ceil_div(R.cols, (int64_t)kRowB);
  a.nk_cta = (int)ceil_div(a.nk, (int64_t)NS);
  a.tiles_t = (int)ceil_div(T.rows, BN);
  a.vec = rows16(p.D, p.bf16 ? 2 : 4);
  a.status = p.status;
  const int64_t tiles = ceil_div(R.rows, 128) * (int64_t)a.tiles_t;
  if (tiles * NS > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "D: too many tiles");
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config((unsigned)(tiles * NS), kSplitThreads, C::kSmem, s, NS, attr);
  OUO_CHECK_CUDA(cudaLaunchKernelEx(&cfg, s8_split_kernel<BN, NS, DEEP>, a));
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

template <int BN>
int run_split(const Product& p, bool t_rows, int nsplit, cudaStream_t s) {
  if (p.A.cols > OUO_INT8_MAX_DEPTH) return run_split<BN, 8, 1>(p, t_rows, s);
  switch (nsplit) {
    case 1: return run_split<BN, 1, 0>(p, t_rows, s);
    case 2: return run_split<BN, 2, 0>(p, t_rows, s);
    case 4: return run_split<BN, 4, 0>(p, t_rows, s);
    default: return run_split<BN, 8, 0>(p, t_rows, s);
  }
}

int run_simt(const Product& p, cudaStream_t s) {
  const int64_t tn = ceil_div(p.D.cols, 64), tiles = ceil_div(p.D.rows, 64) * tn;
  if (tiles > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "D: too many tiles");
  auto kern = p.A.cols > OUO_INT8_MAX_DEPTH ? s8_simt_kernel<1> : s8_simt_kernel<0>;
  kern<<<(unsigned)tiles, 256, 0, s>>>(
      (const int8_t*)p.A.ptr, p.A.ld, (const int8_t*)p.B.ptr, p.B.ld, p.as, p.bs, p.D.ptr, p.D.ld,
      p.bf16, p.D.rows, p.D.cols, p.A.cols, tn);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

template <int MT>
int run_vec(const Product& p, cudaStream_t s) {
  const int64_t blocks = ceil_div(p.D.cols, (int64_t)(kVecThreads / 32) * kVecRows<MT>);
  if (blocks > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "D: too many columns");
  s8_vec_kernel<MT><<<(unsigned)blocks, kVecThreads, 0, s>>>(
      (const int8_t*)p.A.ptr, p.A.ld, (const int8_t*)p.B.ptr, p.B.ld, p.as, p.bs, p.D.ptr, p.D.ld,
      p.bf16, (int)p.D.cols, (int)p.A.cols);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

int product(const Product& p, cudaStream_t s) {
  const int64_t M = p.D.rows, N = p.D.cols, K = p.A.cols;
  if (M == 0 || N == 0) return OUO_OK;
  if (K == 0 || !rows16(p.A, 1) || !rows16(p.B, 1)) return run_simt(p, s);
  // One or two tokens: 10.9 / 12.2 us at 14336 x 4096 against 13.9 / 14.1 in the
  // split kernel.
  if (M == 1) return run_vec<1>(p, s);
  if (M == 2) return run_vec<2>(p, s);
  // Pair tiles once they occupy two thirds of the SMs: 18.1 us at 1024 x 4096 x
  // 4096 (64 tiles) against 20.1 in the split kernel, 17.1 against 15.8 at half
  // the rows (32 tiles).
  const int64_t sms = num_sms();
  if (K <= OUO_INT8_MAX_DEPTH && M > 128 && N > 128 && 3 * ceil_div(M, 256) * ceil_div(N, 256) >= sms) return run_pair(p, s);
  // T is the side with fewer rows, A unless B's rows are few.
  const bool t_rows = M <= N || N > 128;
  const int64_t T = t_rows ? M : N, R = t_rows ? N : M;
  const int bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  // K is divided while the CTAs fit one to an SM and keep enough of it: the
  // join grows with the tile (128 x 4096 x 4096, 32 tiles: 18.0 / 12.8 / 10.9 /
  // 14.8 us in 1 / 2 / 4 / 8; 4 x 1024 x 4096, 8 tiles: 12.5 / 8.1 / 5.9 / 4.9).  In
  // two as long as both halves fit two to an SM (512 x 4096 x 4096: 18.2 / 15.4 / 24.5).
  const int64_t st = ceil_div(R, 128) * ceil_div(T, bn), nk = ceil_div(K, (int64_t)kRowB);
  const int64_t least = bn <= 32 ? 2 : 8;
  int split = 1;
  while (split < 8 && st * 2 * split <= sms && nk / (2 * split) >= (split == 1 ? 2 : least)) split *= 2;
  if (split == 1 && st <= sms && nk >= 4) split = 2;
  switch (bn) {
    case 16: return run_split<16>(p, t_rows, split, s);
    case 32: return run_split<32>(p, t_rows, split, s);
    case 64: return run_split<64>(p, t_rows, split, s);
    default: return run_split<128>(p, t_rows, split, s);
  }
}

// Deepest product: eight CTAs' shares of whole stages, each with 32-bit sums.
static_assert(OUO_INT8_MAX_DEEP == 8 * (OUO_INT8_MAX_DEPTH / 128 * 128), "eight CTAs' depth");

int matmul(int64_t deepest, const ouo_mat* A, const float* const* a_scale, const ouo_mat* B,
           const float* const* b_scale, const ouo_mat* D, int d_dtype, int nmat, int* dev_status,
           void* stream) {
  clear_error();
  if (nmat < 0 || nmat > OUO_MAX_BATCH)
    return set_error(OUO_ERR_INVALID_ARG, "nmat %d out of range", nmat);
  if (nmat == 0) return OUO_OK;
  if (!A || !B || !D || !a_scale || !b_scale)
    return set_error(OUO_ERR_INVALID_ARG, "NULL batch array");
  OUO_TRY(validate_dtype(d_dtype, "D"));
  if ((uintptr_t)dev_status % 4 != 0)
    return set_error(OUO_ERR_INVALID_ARG, "dev_status: not 4-byte aligned");
  for (int i = 0; i < nmat; ++i) {
    OUO_TRY(validate_tokens(A[i], 1, "A", i));
    OUO_TRY(validate_tokens(B[i], 1, "B", i));
    OUO_TRY(validate_tokens(D[i], elem_size(d_dtype), "D", i));
    if (A[i].cols != B[i].cols)
      return set_error(OUO_ERR_INVALID_ARG, "A[%d] has %lld columns, B[%d] has %lld", i,
                       (long long)A[i].cols, i, (long long)B[i].cols);
    if (A[i].cols > deepest)
      return set_error(OUO_ERR_UNSUPPORTED,
                       "A[%d]: depth %lld above %lld (the sums would leave 32 bits)", i,
                       (long long)A[i].cols, (long long)deepest);
    OUO_TRY(validate_shape(D[i], A[i].rows, B[i].rows, "D", i));
    OUO_TRY(validate_vec(a_scale[i], A[i].rows, 4, "a_scale"));
    OUO_TRY(validate_vec(b_scale[i], B[i].rows, 4, "b_scale"));
  }
  OUO_TRY(require_sm100());
  for (int i = 0; i < nmat; ++i)
    OUO_TRY(validate_apart({operand(D[i], (int64_t)elem_size(d_dtype), "D")},
                           {operand(A[i], 1, "A"), operand(B[i], 1, "B"),
                            operand(a_scale[i], A[i].rows, 4, "a_scale"),
                            operand(b_scale[i], B[i].rows, 4, "b_scale")}));
  cudaStream_t s = (cudaStream_t)stream;
  for (int i = 0; i < nmat; ++i) {
    OUO_TRY(product(Product{A[i], B[i], D[i], a_scale[i], b_scale[i], d_dtype == OUO_BF16,
                            dev_status}, s));
  }
  return OUO_OK;
}

}  // namespace
}  // namespace ouo

extern "C" {

int int8_matmul(const ouo_mat* A, const float* const* a_scale, const ouo_mat* B,
                const float* const* b_scale, const ouo_mat* D, int d_dtype, int nmat,
                int* dev_status, void* stream) {
  return ouo::matmul(OUO_INT8_MAX_DEPTH, A, a_scale, B, b_scale, D, d_dtype, nmat, dev_status,
                     stream);
}

int int8_matmul_deep(const ouo_mat* A, const float* const* a_scale, const ouo_mat* B,
                     const float* const* b_scale, const ouo_mat* D, int d_dtype, int nmat,
                     int* dev_status, void* stream) {
  return ouo::matmul(OUO_INT8_MAX_DEEP, A, a_scale, B, b_scale, D, d_dtype, nmat, dev_status,
                     stream);
}

}  // extern "C"
