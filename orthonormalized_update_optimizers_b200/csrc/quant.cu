// quantize_int8: matrices to 8-bit integers with one scale per row, or
// transposed with one scale per column.
//
//   scale_i = max_j |x_ij| / 127,  q_ij = rint(x_ij / scale_i)
//
// HBM-bound: each element is read once and leaves as one byte.
#include <cstring>

#include "tokens.cuh"
#include "umma.cuh"

namespace ouo {
namespace {

struct QuantArgs {
  int nmat, bf16;
  int64_t row_start[kChunk + 1];
  int64_t cols[kChunk];
  const void* X[kChunk];
  int64_t ldx[kChunk];
  int8_t* Q[kChunk];
  int64_t ldq[kChunk];
  float* scale[kChunk];
  uint8_t vecx[kChunk], vecq[kChunk];
};

// Matrix of a launch-wide row.
__device__ __forceinline__ int matrix_of(const QuantArgs& a, int64_t row) {
  int lo = 0, hi = a.nmat - 1;
  while (lo < hi) {
    int mid = (lo + hi + 1) >> 1;
    if (a.row_start[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A team per row, the row in registers: one read, one write.  Bound by HBM:
// 14336 x 4096 bf16 in 27.8 us, 6.3 TB/s.
template <int TPR, int NV, int MODE>
__global__ void __launch_bounds__(kTeamThreads<TPR>)
quant_rows_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t red[kTeamThreads<TPR> / 32];
  constexpr int kTeams = kTeamThreads<TPR> / TPR;
  const int64_t row = (int64_t)blockIdx.x * kTeams + (kTeams > 1 ? threadIdx.x / TPR : 0);
  if (kTeams > 1 && row >= a.row_start[a.nmat]) return;
  const int t = threadIdx.x % TPR;
  const int g = matrix_of(a, row);
  const int64_t r = row - a.row_start[g];
  const int n = (int)a.cols[g];
  if (n == 0) {  // rows without columns: nothing to read (the team's row, so no
                 // thread waits for it)
    if (t == 0) a.scale[g][r] = 0.f;
    return;
  }
  constexpr int kBf = MODE == 1 || MODE == 3;
  const char* x = reinterpret_cast<const char*>(a.X[g]) + r * a.ldx[g] * (kBf ? 2 : 4);
  RowRaw<TPR, NV, MODE> raw;
  float v[NV][8];
  raw.load(x, t, n, kBf, MODE <= 2);
  raw.get(v);
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_mag(m, v[c][i]);
  const Quant q = quant_of<kBf>(team_max<TPR>(__float_as_uint(m), red));
  if (t == 0) a.scale[g][r] = q.scale;
  int8_t* o = a.Q[g] + r * a.ldq[g];
  store_q<TPR, NV, MODE>(o, t, n, a.vecq[g], v, q);
}

// Rows too long for registers: one block per row, read twice (the second
// time from the caches).  Bound by one load in flight a thread: 1024 x 131072
// bf16 in 140 us, 2.9 TB/s of what it has to move.
__global__ void __launch_bounds__(512) quant_long_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t red[32];
  const int64_t row = blockIdx.x;
  const int g = matrix_of(a, row);
  const int64_t r = row - a.row_start[g];
  const int64_t n = a.cols[g];
  const char* x = reinterpret_cast<const char*>(a.X[g]) + r * a.ldx[g] * (a.bf16 ? 2 : 4);
  int8_t* o = a.Q[g] + r * a.ldq[g];
  float m = 0.f;
  for (int64_t j = 8 * threadIdx.x; j < n; j += 8 * 512) {
    float v[8];
    row_ld8(x, (int)j, (int)n, a.bf16, a.vecx[g], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_mag(m, v[i]);
  }
  const Quant q = quant_of<0>(block_max(__float_as_uint(m), red));
  if (threadIdx.x == 0) a.scale[g][r] = q.scale;
  for (int64_t j = 8 * threadIdx.x; j < n; j += 8 * 512) {
    float v[8];
    row_ld8(x, (int)j, (int)n, a.bf16, a.vecx[g], v);
    row_stq(o, (int)j, (int)n, a.vecq[g], quant8(v, q));
  }
}

// Transposed.  A cluster of CTAs takes a strip of 64 bytes of columns and
// divides its rows; every CTA keeps its rows in shared memory (as many as
// fit) while it looks for the columns' largest magnitudes, the cluster joins
// those through distributed shared memory, and the CTA writes its rows' share
// of the strip's transpose.  So X is read once (rows past what fits, twice),
// in one launch and without a workspace.
constexpr int kTThreads = 256;
constexpr int kSegBytes = 64;  // of a row in one strip: 32 bf16 or 16 fp32 columns
constexpr int kMaxCluster = 8;

struct QuantTArgs {
  const void* X;
  int64_t rows, cols, ldx;
  int8_t* Q;
  int64_t ldq;
  float* scale;
  int vecx, vecq;
  int64_t rows_cta;  // a multiple of 32
  int cached;        // rows of a CTA that stay in shared memory, a multiple of 32
};

// 16 bytes of row r from column c, zero outside the matrix, element by element.
template <int BF>
__device__ __forceinline__ uint4 seg_ld(const QuantTArgs& a, int64_t r, int64_t c) {
  constexpr int kE = BF ? 8 : 4;
  const char* p = reinterpret_cast<const char*>(a.X) + (r * a.ldx + c) * (BF ? 2 : 4);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    if (c + i >= a.cols) break;
    if (BF) w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    else w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int BF>
__global__ void __launch_bounds__(kTThreads, 3)
quant_cols_kernel(const __grid_constant__ QuantTArgs a) {
  constexpr int kCols = BF ? 32 : 16;  // of the strip
  extern __shared__ __align__(16) uint32_t cache[];  // [cached][16 words]
  __shared__ uint32_t wmax[kTThreads / 32][kCols];
  __shared__ uint32_t cmax[kCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t nct;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nct));
  const uint32_t rank = ptx::cluster_ctarank();
  const int64_t strip = blockIdx.x / nct;
  const int64_t c0 = strip * kCols;
  const int64_t ra = rank * a.rows_cta;
  const int64_t rb = ra + a.rows_cta < a.rows ? ra + a.rows_cta : a.rows;
  // columns' largest magnitudes: four threads per row, 16 bytes each
  const int seg = threadIdx.x & 3;
  uint32_t m[BF ? 8 : 4];
#pragma unroll
  for (int i = 0; i < (BF ? 8 : 4); ++i) m[i] = 0;
  auto take = [&](const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF) {
        m[2 * i] = max(m[2 * i], (w[i] << 16) & 0x7fffffffu);
        m[2 * i + 1] = max(m[2 * i + 1], w[i] & 0x7fff0000u);
      } else {
        m[i] = max(m[i], w[i] & 0x7fffffffu);
      }
    }
  };
  constexpr int kRowsPass = kTThreads / 4;
  const int64_t cs = c0 + seg * (BF ? 8 : 4);
  auto keep = [&](int64_t l, const uint4& u) {
    take(u);
    if (l < a.cached) reinterpret_cast<uint4*>(cache)[l * 4 + seg] = u;
  };
  if (a.vecx && c0 + kCols <= a.cols) {
    // every row that stays is requested at once; the thread that copied a
    // piece is the one that looks at it
    const char* p = reinterpret_cast<const char*>(a.X) + cs * (BF ? 2 : 4);
    const int64_t pitch = a.ldx * (BF ? 2 : 4);
    const int lt = threadIdx.x >> 2;
    const int ln = rb > ra ? (int)(rb - ra < a.cached ? rb - ra : a.cached) : 0;
    for (int l = lt; l < ln; l += kRowsPass)
      ptx::copy16(cache + l * 16 + seg * 4, p + (ra + l) * pitch);
    ptx::copy16_wait_all();
#pragma unroll 4
    for (int l = lt; l < ln; l += kRowsPass) take(reinterpret_cast<const uint4*>(cache)[l * 4 + seg]);
    constexpr int kU = 4;
    for (int64_t r = ra + ln + lt; r < rb; r += kRowsPass * kU) {
      uint4 u[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        u[k] = make_uint4(0, 0, 0, 0);
        if (r + k * kRowsPass < rb)
          u[k] = *reinterpret_cast<const uint4*>(p + (r + k * kRowsPass) * pitch);
      }
#pragma unroll
      for (int k = 0; k < kU; ++k) take(u[k]);
    }
  } else {
    for (int64_t r = ra + (threadIdx.x >> 2); r < rb; r += kRowsPass) keep(r - ra, seg_ld<BF>(a, r, cs));
  }
#pragma unroll
  for (int i = 0; i < (BF ? 8 : 4); ++i) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    if (lane < 4) wmax[warp][seg * (BF ? 8 : 4) + i] = m[i];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kTThreads / 32; ++w) v = max(v, wmax[w][threadIdx.x]);
    cmax[threadIdx.x] = v;
  }
  __syncwarp();
  ptx::cluster_sync();
  // every thread's one or two columns: word `wd` of a row
  const int wd = lane & 15, half = lane >> 4;
  uint32_t x0 = 0, x1 = 0;
#pragma unroll
  for (uint32_t p = 0; p < kMaxCluster; ++p) {
    if (p >= nct) break;
    x0 = max(x0, (uint32_t)ptx::ld_cluster_int(
                     ptx::mapa(ptx::smem_u32(&cmax[BF ? 2 * wd : wd]), p)));
    if (BF)
      x1 = max(x1, (uint32_t)ptx::ld_cluster_int(ptx::mapa(ptx::smem_u32(&cmax[2 * wd + 1]), p)));
  }
  __syncwarp();
  ptx::cluster_sync();  // everyone has read everyone's (nothing is read from afar below)
  const Quant q0 = quant_of<BF>(x0), q1 = quant_of<BF>(x1);
  const int64_t col = c0 + (BF ? 2 * wd : wd);
  if (rank == 0 && warp == 0 && half == 0) {
    if (col < a.cols) a.scale[col] = q0.scale;
    if (BF && col + 1 < a.cols) a.scale[col + 1] = q1.scale;
  }
  // 32 rows per warp and pass; a half warp takes 16 of them, each lane a word
  // of every row.  The halves read rows of opposite parity, so that their 16
  // words lie in different banks.
  for (int64_t base = ra + warp * 32; base < rb; base += kTThreads) {
    const int64_t r0 = base + 16 * half;
    uint32_t w[16];
    if (base + 32 - ra <= a.cached) {
      const uint32_t* q = cache + (r0 - ra) * 16 + wd;
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = q[(i ^ half) * 16];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + (i ^ half);
        w[i] = 0;
        if (r >= rb) continue;
        if (BF) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(a.X) + r * a.ldx + col;
          if (col < a.cols) w[i] = p[0];
          if (col + 1 < a.cols) w[i] |= (uint32_t)p[1] << 16;
        } else if (col < a.cols) {
          w[i] = reinterpret_cast<const uint32_t*>(a.X)[r * a.ldx + col];
        }
      }
    }
    if (half) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint32_t s = w[i];
        w[i] = w[i + 1];
        w[i + 1] = s;
      }
    }
#pragma unroll
    for (int e = 0; e < (BF ? 2 : 1); ++e) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(!BF ? w[i] : e ? w[i] & 0xffff0000u : w[i] << 16);
      const Quant& q = e ? q1 : q0;
      const uint2 lo = quant8(v, q), hi = quant8(v + 8, q);
      if (col + e >= a.cols || r0 >= rb) continue;
      int8_t* o = a.Q + (col + e) * a.ldq;
      if (a.vecq && r0 + 16 <= rb) {
        *reinterpret_cast<uint4*>(o + r0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        const uint32_t b[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (r0 + i < rb) o[r0 + i] = (int8_t)((b[i >> 2] >> (8 * (i & 3))) & 255u);
      }
    }
  }
}

template <int BF>
int quant_cols(const ouo_mat& X, const ouo_mat& Q, float* scale, cudaStream_t s) {
  // shared memory for two CTAs a SM; a CTA keeps 128 rows at least
  constexpr int kCached = 1600;
  constexpr size_t kSmem = (size_t)kCached * kSegBytes;
  static Once once;
  OUO_TRY(once.smem(quant_cols_kernel<BF>, kSmem));
  unsigned cluster = 1;
  while (cluster < kMaxCluster && ceil_div(X.rows, (int64_t)2 * cluster) >= 128) cluster *= 2;
  QuantTArgs a;
  a.X = X.ptr; a.rows = X.rows; a.cols = X.cols; a.ldx = X.ld;
  a.Q = (int8_t*)Q.ptr; a.ldq = Q.ld;
  a.scale = scale;
  a.vecx = rows16(X, BF ? 2 : 4);
  a.vecq = rows16(Q, 1);
  a.rows_cta = ceil_div(ceil_div(X.rows, (int64_t)cluster), 32) * 32;
  a.cached = (int)(a.rows_cta < kCached ? a.rows_cta : kCached);
  const int64_t strips = ceil_div(X.cols, (int64_t)(BF ? 32 : 16));
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(strips * cluster), 1, 1);
  cfg.blockDim = dim3(kTThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.cached * kSegBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  OUO_CHECK_CUDA(cudaLaunchKernelEx(&cfg, quant_cols_kernel<BF>, a));
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

// ---- Transposed, in two launches: the columns' largest magnitudes in
// `splits` row ranges, then the rounding, tile by tile.  X is read twice (the second
// time from L2 as far as it fits), but both passes stream: 14336 x 4096 bf16 in
// 61.0 us, 4.8 TB/s of what they move.

struct QuantT2Args {
  const void* X;
  int64_t rows, cols, ldx;
  int8_t* Q;
  int64_t ldq;
  float* scale;
  uint32_t* part;  // [splits][cols]
  int splits;
  int64_t rows_split;
  int vecx, vecq;
  int64_t tiles_c;
};

template <int BF>
__global__ void __launch_bounds__(256) col_amax_kernel(const __grid_constant__ QuantT2Args a) {
  constexpr int kE = BF ? 8 : 4, kU = 16;
  __shared__ float red[8][32][kE + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t strips = (a.cols + 32 * kE - 1) / (32 * kE);
  const int64_t split = blockIdx.x / strips, strip = blockIdx.x - split * strips;
  const int64_t c = strip * 32 * kE + lane * kE;
  const int64_t ra = split * a.rows_split;
  const int64_t rb = ra + a.rows_split < a.rows ? ra + a.rows_split : a.rows;
  float m[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) m[i] = 0.f;
  const bool wide = a.vecx && (strip + 1) * 32 * kE <= a.cols;
  if (wide) {
    const char* p = reinterpret_cast<const char*>(a.X) + c * (BF ? 2 : 4);
    const int64_t pitch = a.ldx * (BF ? 2 : 4);
    for (int64_t r = ra + warp; r < rb; r += 8 * kU) {
      uint4 u[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        u[k] = make_uint4(0, 0, 0, 0);
        if (r + 8 * k < rb) u[k] = *reinterpret_cast<const uint4*>(p + (r + 8 * k) * pitch);
      }
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        if (BF) {
          float v[8];
          unpack8(u[k], v);
#pragma unroll
          for (int i = 0; i < kE; ++i) m[i] = max_mag(m[i], v[i]);
        } else {
          const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
          for (int i = 0; i < kE; ++i) m[i] = max_mag(m[i], __uint_as_float(w[i & 3]));
        }
      }
    }
  } else {
    // element by element: a lane's columns 32 apart, four rows in flight.  What
    // is past the end reads the last one again: a maximum does not mind, and
    // loads without conditions are issued together.
    using E = std::conditional_t<BF, uint16_t, uint32_t>;
    const int64_t ce = strip * 32 * kE + lane;
    int at[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i)
      at[i] = (int)(ce + 32 * i < a.cols ? ce + 32 * i : a.cols - 1);
    for (int64_t r = ra + warp; r < rb; r += 8 * 4) {
      uint32_t v[4][kE];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const E* x = reinterpret_cast<const E*>(a.X) + (r + 8 * k < rb ? r + 8 * k : rb - 1) * a.ldx;
#pragma unroll
        for (int i = 0; i < kE; ++i) v[k][i] = x[at[i]];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < kE; ++i)
          m[i] = max_mag(m[i], __uint_as_float(BF ? v[k][i] << 16 : v[k][i]));
    }
  }
  // red[warp][column of the strip / kE][% kE], whichever way they were read
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const int e = wide ? lane * kE + i : 32 * i + lane;
    red[warp][e / kE][e % kE] = m[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * kE; e += 256) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v = max_mag(v, red[w][e / kE][e % kE]);
    if (strip * 32 * kE + e < a.cols)
      a.part[split * a.cols + strip * 32 * kE + e] = __float_as_uint(v);
  }
}

constexpr int kMaxSplits = 32;

// A tile of 128 bytes of columns x kTileRows rows goes through shared memory.
constexpr int kTileRows = 256;
constexpr int kOutPitch = kTileRows + 16;

template <int BF>
__global__ void __launch_bounds__(256, 4)
quant_tile_kernel(const __grid_constant__ QuantT2Args a) {
  constexpr int kCols = BF ? 64 : 32;
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t(*tile)[32] = reinterpret_cast<uint32_t(*)[32]>(dyn);
  // the tile's transpose: row e * 32 + l for column 2 l + e (fp32: l), pitch
  // padded so that the 16-byte writes of a quarter warp lie in different banks
  uint8_t(*out)[kOutPitch] = reinterpret_cast<uint8_t(*)[kOutPitch]>(dyn + kTileRows * 32);
  __shared__ uint32_t cm[8][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
  const int64_t r0 = tr * kTileRows, c0 = tc * kCols;
  const int nr = (int)(a.rows - r0 < kTileRows ? a.rows - r0 : kTileRows);
  const int piece = threadIdx.x & 7;
  if (a.vecx && c0 + kCols <= a.cols) {
    const char* p = reinterpret_cast<const char*>(a.X) + (r0 * a.ldx + c0) * (BF ? 2 : 4) + piece * 16;
    const int64_t pitch = a.ldx * (BF ? 2 : 4);
#pragma unroll
    for (int k = 0; k < kTileRows / 32; ++k) {
      const int l = (threadIdx.x >> 3) + 32 * k;
      if (l < nr) ptx::copy16(&tile[l][piece * 4], p + l * pitch);
    }
  } else {
    // element by element, a warp per row, eight rows in flight; what is past the
    // end reads the last one again and is not used
    using E = std::conditional_t<BF, uint16_t, uint32_t>;
    int at[kCols / 32];
#pragma unroll
    for (int i = 0; i < kCols / 32; ++i)
      at[i] = (int)(c0 + lane + 32 * i < a.cols ? c0 + lane + 32 * i : a.cols - 1);
    for (int l0 = warp; l0 < nr; l0 += 64) {
      uint32_t v[8][kCols / 32];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const E* x = reinterpret_cast<const E*>(a.X) + (r0 + min(l0 + 8 * k, nr - 1)) * a.ldx;
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i) v[k][i] = x[at[i]];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i)
          if (l0 + 8 * k < nr) reinterpret_cast<E*>(tile[l0 + 8 * k])[lane + 32 * i] = (E)v[k][i];
    }
  }
  // the columns' magnitudes, a group of threads per range of splits
  {
    constexpr int kG = 256 / kCols;
    const int col = threadIdx.x % kCols, g = threadIdx.x / kCols;
    uint32_t m = 0;
    if (c0 + col < a.cols) {
      const uint32_t* p = a.part + c0 + col;
#pragma unroll
      for (int k = 0; k < kMaxSplits / kG; ++k)  // all in flight together
        if (g + k * kG < a.splits) m = max(m, p[(g + k * kG) * a.cols]);
    }
    cm[g][col] = m;
  }
  ptx::copy16_wait_all();
  __syncthreads();
  if (threadIdx.x < kCols) {
    constexpr int kG = 256 / kCols;
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < kG; ++g) m = max(m, cm[g][threadIdx.x]);
    cm[0][threadIdx.x] = m;
    if (tr == 0 && c0 + threadIdx.x < a.cols) a.scale[c0 + threadIdx.x] = quant_of<BF>(m).scale;
  }
  __syncthreads();
  const Quant q0 = quant_of<BF>(cm[0][BF ? 2 * lane : lane]);
  const Quant q1 = BF ? quant_of<BF>(cm[0][2 * lane + 1]) : q0;
  for (int b = warp * 16; b < nr; b += 128) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = tile[b + i][lane];
#pragma unroll
    for (int e = 0; e < (BF ? 2 : 1); ++e) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(!BF ? w[i] : e ? w[i] & 0xffff0000u : w[i] << 16);
      const Quant& q = e ? q1 : q0;
      const uint2 lo = quant8(v, q), hi = quant8(v + 8, q);
      *reinterpret_cast<uint4*>(&out[e * 32 + lane][b]) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  __syncthreads();
  // whole rows of the transpose leave in order: 256 bytes each
  for (int r = threadIdx.x >> 4; r < kCols; r += 16) {
    const int64_t col = c0 + (BF ? 2 * (r & 31) + (r >> 5) : r);
    if (col >= a.cols) continue;
    int8_t* o = a.Q + col * a.ldq + r0;
    const int l = threadIdx.x & 15;
    if (a.vecq && 16 * l + 16 <= nr) {
      *reinterpret_cast<uint4*>(o + 16 * l) = *reinterpret_cast<const uint4*>(&out[r][16 * l]);
    } else if (a.vecq) {
      for (int i = 16 * l; i < nr && i < 16 * l + 16; ++i) o[i] = (int8_t)out[r][i];
    } else {
      for (int i = l; i < nr; i += 16) o[i] = (int8_t)out[r][i];
    }
  }
}

// Row ranges of the first pass: about three blocks a SM, a function of the
// shape alone (the workspace query needs no device).
int amax_splits(int64_t rows, int64_t cols, int bf16) {
  const int64_t strips = ceil_div(cols, (int64_t)(bf16 ? 256 : 128));
  int64_t n = ceil_div((int64_t)3 * 148, strips);
  if (n > kMaxSplits) n = kMaxSplits;
  if (n > ceil_div(rows, (int64_t)64)) n = ceil_div(rows, (int64_t)64);
  return (int)(n < 1 ? 1 : n);
}

// Which of the two: the clusters while the matrix is small and launches count
// (us, clusters / two passes, bf16: 64 x 4096 3.3 / 5.0, 256 x 1024 3.4 / 5.7),
// two passes above 3 MB, where the clusters' waits for one another do
// (512 x 4096 8.3 / 6.4, 2048 x 4096 21.6 / 13.5, 14336 x 4096 76.4 / 61.6).
bool two_passes(int64_t rows, int64_t cols, int bf16) {
  return rows * cols * (bf16 ? 2 : 4) > (int64_t)3 << 20;
}

template <int BF>
int quant_cols2(const ouo_mat& X, const ouo_mat& Q, float* scale, void* ws, cudaStream_t s) {
  QuantT2Args a;
  a.X = X.ptr; a.rows = X.rows; a.cols = X.cols; a.ldx = X.ld;
  a.Q = (int8_t*)Q.ptr; a.ldq = Q.ld;
  a.scale = scale;
  a.part = (uint32_t*)ws;
  a.vecx = rows16(X, BF ? 2 : 4);
  a.vecq = rows16(Q, 1);
  a.splits = amax_splits(X.rows, X.cols, BF);
  a.rows_split = ceil_div(X.rows, (int64_t)a.splits);
  a.tiles_c = ceil_div(X.cols, (int64_t)(BF ? 64 : 32));
  const int64_t strips = ceil_div(X.cols, (int64_t)(BF ? 256 : 128));
  const int64_t tiles = a.tiles_c * ceil_div(X.rows, (int64_t)kTileRows);
  if (tiles > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "X: too many tiles");
  col_amax_kernel<BF><<<(unsigned)(strips * a.splits), 256, 0, s>>>(a);
  OUO_CHECK_LAUNCH();
  constexpr size_t kSmem = (size_t)kTileRows * 128 + (size_t)(BF ? 64 : 32) * kOutPitch;
  static Once once;
  OUO_TRY(once.smem(quant_tile_kernel<BF>, kSmem));
  quant_tile_kernel<BF><<<(unsigned)tiles, 256, kSmem, s>>>(a);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

// The kinds of a batch's matrices, each with launches of its own, so that one
// that cannot take 16-byte accesses, or whose rows do not fit in registers,
// does not slow the others down.
enum { kRowsVec, kRowsElem, kRowsLong };

int rows_kind(const ouo_mat& x, size_t es) {
  if (x.cols == 0) return kRowsVec;
  if (x.cols > kTeamMost) return kRowsLong;
  return rows16(x, es) && x.cols % 8 == 0 ? kRowsVec : kRowsElem;
}

// One launch; the longest rows choose its teams.
int quant_rows(QuantArgs& a, int64_t rows, int64_t longest, int kind, cudaStream_t s) {
  if (rows == 0) return OUO_OK;
  a.row_start[a.nmat] = rows;
  if (kind == kRowsLong) {
    quant_long_kernel<<<(unsigned)rows, 512, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
    return OUO_OK;
  }
  // (element by element too, a quantized row is one load and one store: the
  // smaller teams of the vector modes do better)
  const Team t = team_for(rows, longest, a.bf16 ? 1 : 2);
  return with_team_of(t, [&](auto tpr, auto nv) -> int {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int kTeams = kTeamThreads<TPR> / TPR;
    auto kern = kind == kRowsElem
                    ? (a.bf16 ? quant_rows_kernel<TPR, NV, 3> : quant_rows_kernel<TPR, NV, 4>)
                    : (a.bf16 ? quant_rows_kernel<TPR, NV, 1> : quant_rows_kernel<TPR, NV, 2>);
    kern<<<(unsigned)ceil_div(rows, (int64_t)kTeams), kTeamThreads<TPR>, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
    return OUO_OK;
  });
}

}  // namespace
}  // namespace ouo

extern "C" size_t quantize_int8_workspace_bytes(const ouo_mat* X, int x_dtype, int nmat,
                                                int transpose) {
  using namespace ouo;
  if (!X || !transpose || (x_dtype != OUO_F32 && x_dtype != OUO_BF16)) return 0;
  const int bf16 = x_dtype == OUO_BF16;
  size_t most = 0;  // the matrices of a batch follow one another
  for (int i = 0; i < nmat; ++i)
    if (X[i].rows > 0 && X[i].cols > 0 && two_passes(X[i].rows, X[i].cols, bf16)) {
      const size_t b = (size_t)amax_splits(X[i].rows, X[i].cols, bf16) * (size_t)X[i].cols * 4;
      if (b > most) most = b;
    }
  return most;
}

extern "C" int quantize_int8(const ouo_mat* X, int x_dtype, const ouo_mat* Q, float* const* scale,
                             int nmat, int transpose, void* ws, size_t ws_bytes, void* stream) {
  using namespace ouo;
  clear_error();
  if (nmat < 0 || nmat > OUO_MAX_BATCH)
    return set_error(OUO_ERR_INVALID_ARG, "nmat %d out of range", nmat);
  if (nmat == 0) return OUO_OK;
  if (!X || !Q || !scale) return set_error(OUO_ERR_INVALID_ARG, "NULL batch array");
  if (transpose != 0 && transpose != 1)
    return set_error(OUO_ERR_INVALID_ARG, "transpose must be 0 or 1");
  OUO_TRY(validate_dtype(x_dtype, "X"));
  for (int i = 0; i < nmat; ++i) {
    OUO_TRY(validate_tokens(X[i], elem_size(x_dtype), "X", i));
    OUO_TRY(validate_tokens(Q[i], 1, "Q", i));
    OUO_TRY(validate_shape(Q[i], transpose ? X[i].cols : X[i].rows,
                           transpose ? X[i].rows : X[i].cols, "Q", i));
    OUO_TRY(validate_vec(scale[i], Q[i].rows, 4, "scale"));
  }
  const size_t need = quantize_int8_workspace_bytes(X, x_dtype, nmat, transpose);
  if (need > 0 && (!ws || ws_bytes < need || (uintptr_t)ws % 16 != 0))
    return set_error(OUO_ERR_WORKSPACE, "workspace: %zu bytes needed (16-byte aligned), %zu given",
                     need, ws ? ws_bytes : (size_t)0);
  OUO_TRY(require_sm100());
  for (int i = 0; i < nmat; ++i)
    OUO_TRY(validate_apart({operand(Q[i], 1, "Q"), operand(scale[i], Q[i].rows, 4, "scale")},
                           {operand(X[i], (int64_t)elem_size(x_dtype), "X")}));
  cudaStream_t s = (cudaStream_t)stream;
  const int bf16 = x_dtype == OUO_BF16;
  if (transpose) {
    for (int i = 0; i < nmat; ++i) {
      if (X[i].cols == 0) continue;
      if (two_passes(X[i].rows, X[i].cols, bf16)) {
        OUO_TRY(bf16 ? quant_cols2<1>(X[i], Q[i], scale[i], ws, s)
                     : quant_cols2<0>(X[i], Q[i], scale[i], ws, s));
        continue;
      }
      OUO_TRY(bf16 ? quant_cols<1>(X[i], Q[i], scale[i], s) : quant_cols<0>(X[i], Q[i], scale[i], s));
    }
    return OUO_OK;
  }
  for (int kind = 0; kind < 3; ++kind) {
    QuantArgs a;
    a.bf16 = bf16;
    a.nmat = 0;
    int64_t rows = 0, longest = 0;
    for (int i = 0; i < nmat; ++i) {
      const ouo_mat &x = X[i], &q = Q[i];
      if (x.rows == 0 || rows_kind(x, elem_size(x_dtype)) != kind) continue;
      if (a.nmat == kChunk || rows + x.rows > 0x7fffffff) {
        OUO_TRY(quant_rows(a, rows, longest, kind, s));
        a.nmat = 0;
        rows = longest = 0;
      }
      const int g = a.nmat++;
      a.row_start[g] = rows;
      a.cols[g] = x.cols;
      a.X[g] = x.ptr;
      a.ldx[g] = x.ld;
      a.Q[g] = (int8_t*)q.ptr;
      a.ldq[g] = q.ld;
      a.scale[g] = scale[i];
      a.vecx[g] = rows16(x, elem_size(x_dtype));
      a.vecq[g] = (uintptr_t)q.ptr % 8 == 0 && (x.rows <= 1 || q.ld % 8 == 0);
      rows += x.rows;
      if (x.cols > longest) longest = x.cols;
    }
    OUO_TRY(quant_rows(a, rows, longest, kind, s));
  }
  return OUO_OK;
}
