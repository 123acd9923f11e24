// MXFP4 x MXFP4 products on the matrix cores:
//   y[m, n] = epi( sum_b 2^(sx[m,b] + sw[n,b] - 254) sum_{k in b} qx[m,k] qw[n,k] )
// for one weight matrix, or for the experts of a bank over rows in expert
// order (rows offsets[e] .. offsets[e+1] - 1 against expert e's matrix).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as E2M1 codes with an
// E8M0 scale per 32 values: lane l carries row l % 16 and the 32 values (16
// bytes) and the scale of block l / 16, so the scales cost no vector work.
#include "pq_mxfp4_dev.h"

extern "C" int pq_quantize_mxfp4(const void* in, int in_is_f32, int rows, int K, uint8_t* codes, uint8_t* scales,
                                 void* stream);

namespace {

typedef int int32x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int BM = 64, BN = 64;        // tile: 4 waves, 2 x 2, 32 x 32 each

struct GArgs {
  const uint8_t* xq;        // [xrows][K/2]
  const uint8_t* xs;        // [xrows][K/32]
  const uint8_t* w;         // [E][N][K/2]
  const uint8_t* ws;        // [E][N][K/32]
  uint16_t* y;              // [P][R]
  const int32_t* offsets;   // [E+1], or null: one matrix for all P rows
  const int32_t* order;     // [P] pairs, or null: row r reads x row r
  int xrows, P, K, N, R, E, top_k, silu;
  int tn;                   // tiles along the output columns
};

__device__ __forceinline__ floatx4 mfma_fp4(uint4 a, uint4 b, floatx4 c, uint32_t sa, uint32_t sb) {
  const int32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const int32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// First rows and row-tile counts of the experts: start[e] = number of row
// tiles before expert e (start[E] = all of them).  Offsets are clamped to
// [0, P] and a falling pair counts as no rows, so a tile never leaves x or y.
__device__ __forceinline__ int rows_of(const GArgs& a, int e, int* first) {
  if (!a.offsets) {
    *first = 0;
    return a.P;
  }
  const int lo = min(max(a.offsets[e], 0), a.P), hi = min(max(a.offsets[e + 1], 0), a.P);
  *first = lo;
  return max(hi - lo, 0);
}

template <int TILE>
__device__ __forceinline__ void tile_starts(const GArgs& a, int* start) {
  if (threadIdx.x == 0) {
    int at = 0;
    for (int e = 0; e < a.E; ++e) {
      int f;
      start[e] = at;
      at += (rows_of(a, e, &f) + TILE - 1) / TILE;
    }
    start[a.E] = at;
  }
  __syncthreads();
}

// output column of the tile's B row r: plain, or under SiLU*up runs of 16 as
// gate, up, gate, up; -1 past the matrix
__device__ __forceinline__ int b_row(const GArgs& a, int tile_n, int r) {
  if (!a.silu) {
    const int n = tile_n * BN + r;
    return n < a.N ? n : -1;
  }
  const int c = tile_n * (BN / 2) + (r >> 5) * 16 + (r & 15);
  if (c >= a.R) return -1;
  return (r & 16) ? c + a.R : c;
}

__global__ __launch_bounds__(kThreads) void gemm_mxfp4_kernel(GArgs a) {
  __shared__ int start[kMaxExperts + 1];
  tile_starts<BM>(a, start);
  const int lane = pq::lane_id(), wv = pq::wave_id();
  const int wm = wv >> 1, wn = wv & 1, rl = lane & 15, g = lane >> 4;
  const int total = start[a.E] * a.tn;
  const int nb = a.K / pq::kMxBlock;
  const uint32_t rowb = (uint32_t)(a.K / 2);
  const pq::rsrc_t xr = pq::make_rsrc(a.xq, (uint32_t)((size_t)a.xrows * rowb));
  const pq::rsrc_t xsr = pq::make_rsrc(a.xs, (uint32_t)((size_t)a.xrows * nb));
  for (int t = (int)blockIdx.x; t < total; t += (int)gridDim.x) {
    const int mt = t / a.tn, tile_n = t - mt * a.tn;
    int lo = 0, hi = a.E;                    // the expert whose row tiles hold mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= mt) lo = mid;
      else hi = mid;
    }
    int first;
    const int n_rows = rows_of(a, lo, &first);
    const int m0 = (mt - start[lo]) * BM;
    const pq::rsrc_t wr = pq::make_rsrc(a.w + (size_t)lo * a.N * rowb, (uint32_t)((size_t)a.N * rowb));
    const pq::rsrc_t wsr = pq::make_rsrc(a.ws + (size_t)lo * a.N * nb, (uint32_t)((size_t)a.N * nb));
    int arow[2], brow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = m0 + 32 * wm + 16 * i + rl;
      arow[i] = -1;
      if (r < n_rows) {
        if (a.order) {
          const int p = a.order[first + r];
          if (p >= 0 && p / a.top_k < a.xrows) arow[i] = p / a.top_k;
        } else {
          arow[i] = first + r;
        }
      }
      brow[i] = b_row(a, tile_n, 32 * wn + 16 * i + rl);
    }
    floatx4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = 0; b0 < nb; b0 += 4) {
      const int blk = b0 + g;
      uint4 av[2], bv[2];
      uint32_t sa[2], sb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool oa = arow[i] >= 0 && blk < nb, ob = brow[i] >= 0 && blk < nb;
        av[i] = pq::buf_load16(xr, oa ? (uint32_t)arow[i] * rowb + 16u * blk : pq::kOOB);
        bv[i] = pq::buf_load16(wr, ob ? (uint32_t)brow[i] * rowb + 16u * blk : pq::kOOB);
        sa[i] = __builtin_amdgcn_raw_buffer_load_b8(xsr, (int)(oa ? (uint32_t)arow[i] * nb + blk : pq::kOOB), 0, 0);
        sb[i] = __builtin_amdgcn_raw_buffer_load_b8(wsr, (int)(ob ? (uint32_t)brow[i] * nb + blk : pq::kOOB), 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_fp4(av[i], bv[j], acc[i][j], sa[i], sb[j]);
    }
    // lane (g, c) of sub-tile (i, j) holds rows 4g .. 4g+3 of i and column c of j
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m0 + 32 * wm + 16 * i + 4 * g + r;
        if (row >= n_rows) continue;
        uint16_t* yr = a.y + (size_t)(first + row) * a.R;
        if (a.silu) {
          const int c = tile_n * (BN / 2) + wn * 16 + rl;
          if (c < a.R) yr[c] = pq::bf16_rne(pq::silu_mul_f32(acc[i][0][r], acc[i][1][r]));
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int n = tile_n * BN + 32 * wn + 16 * j + rl;
            if (n < a.N) yr[n] = pq::bf16_rne(acc[i][j][r]);
          }
        }
      }
  }
  // rows behind the last expert's: zeros
  if (a.offsets) {
    const int end = min(max(a.offsets[a.E], 0), a.P);
    for (long i = (long)end * a.R + (long)blockIdx.x * kThreads + threadIdx.x; i < (long)a.P * a.R;
         i += (long)gridDim.x * kThreads)
      a.y[i] = 0;
  }
}

// Shapes shared by the entry points; E and N, K of one expert's matrix.
int check_shape(int xrows, int P, int K, int N, int E, int epi) {
  if (xrows < 1 || P < 1 || N < 1 || E < 1 || E > kMaxExperts || K < pq::kMxBlock || K % pq::kMxBlock != 0)
    return PQ_ERR_SHAPE;
  if (epi != PQ_EPI_NONE && epi != PQ_EPI_SILU_MUL) return PQ_ERR_SHAPE;
  if (epi == PQ_EPI_SILU_MUL && N % 2 != 0) return PQ_ERR_SHAPE;
  if ((size_t)N * (K / 2) > pq::kMaxBufferBytes || (size_t)xrows * (K / 2) > pq::kMaxBufferBytes) return PQ_ERR_SHAPE;
  return PQ_OK;
}

int run(GArgs& a, int epi, hipStream_t stream) {
  pqhost::DeviceInfo dev;
  const int st = pqhost::current_device_info(&dev);
  if (st != PQ_OK) return st;
  a.silu = epi == PQ_EPI_SILU_MUL;
  a.R = a.silu ? a.N / 2 : a.N;
  a.tn = a.silu ? (a.R + BN / 2 - 1) / (BN / 2) : (a.N + BN - 1) / BN;
  const long most = ((long)a.P / BM + (a.E < a.P ? a.E : a.P)) * a.tn;   // tiles, whatever the offsets
  const long grid = most < 8L * dev.num_cus ? most : 8L * dev.num_cus;
  hipLaunchKernelGGL(gemm_mxfp4_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
  PQ_HIP_CHECK(hipGetLastError());
  return PQ_OK;
}

// codes, then scales, of `rows` quantised rows in a workspace's data region
size_t scratch_bytes(int rows, int K) {
  return pq::kWsDataOff + pqhost::align_up((size_t)rows * (K / 2), 256) +
         pqhost::align_up((size_t)rows * (K / pq::kMxBlock), 256);
}
uint8_t* scratch_codes(void* ws) { return reinterpret_cast<uint8_t*>(ws) + pq::kWsDataOff; }
uint8_t* scratch_scales(void* ws, int rows, int K) {
  return scratch_codes(ws) + pqhost::align_up((size_t)rows * (K / 2), 256);
}

}  // namespace

extern "C" {

size_t pq_gemm_mxfp4_workspace(int M, int K, int N, int epi) {
  return check_shape(M, M, K, N, 1, epi) == PQ_OK ? scratch_bytes(M, K) : 0;
}

int pq_gemm_mxfp4_prequant(const uint8_t* xq, const uint8_t* xs, int M, int K, const uint8_t* w,
                           const uint8_t* w_scale, int N, int epi, uint16_t* y, void* stream) {
  if (!xq || !xs || !w || !w_scale || !y) return PQ_ERR_NULL;
  const int st = check_shape(M, M, K, N, 1, epi);
  if (st != PQ_OK) return st;
  if (!pqhost::aligned16(xq) || !pqhost::aligned16(xs) || !pqhost::aligned16(w) || !pqhost::aligned16(w_scale) ||
      !pqhost::aligned16(y))
    return PQ_ERR_ALIGN;
  GArgs a = {};
  a.xq = xq; a.xs = xs; a.w = w; a.ws = w_scale; a.y = y;
  a.xrows = a.P = M;
  a.K = K; a.N = N; a.E = 1; a.top_k = 1;
  return run(a, epi, (hipStream_t)stream);
}

int pq_gemm_mxfp4(const uint16_t* x, int M, int K, const uint8_t* w, const uint8_t* w_scale, int N, int epi,
                  uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !w || !w_scale || !y) return PQ_ERR_NULL;
  int st = check_shape(M, M, K, N, 1, epi);
  if (st != PQ_OK) return st;
  if (!pqhost::aligned16(x) || !pqhost::aligned16(w) || !pqhost::aligned16(w_scale) || !pqhost::aligned16(y))
    return PQ_ERR_ALIGN;
  if (!ws || ws_bytes < scratch_bytes(M, K)) return PQ_ERR_WORKSPACE;
  if (!pqhost::aligned16(ws)) return PQ_ERR_ALIGN;
  st = pq_quantize_mxfp4(x, 0, M, K, scratch_codes(ws), scratch_scales(ws, M, K), stream);
  if (st != PQ_OK) return st;
  return pq_gemm_mxfp4_prequant(scratch_codes(ws), scratch_scales(ws, M, K), M, K, w, w_scale, N, epi, y, stream);
}

size_t pq_gemm_mxfp4_grouped_workspace(int rows, int K, int N, int epi) {
  return pq_gemm_mxfp4_workspace(rows, K, N, epi);
}

int pq_gemm_mxfp4_grouped_prequant(const uint8_t* xq, const uint8_t* xs, int rows, int K, const int32_t* order,
                                   int top_k, const int32_t* offsets, int P, int E, const uint8_t* w,
                                   const uint8_t* w_scale, int N, int epi, uint16_t* y, void* stream) {
  if (!xq || !xs || !offsets || !w || !w_scale || !y) return PQ_ERR_NULL;
  const int st = check_shape(rows, P, K, N, E, epi);
  if (st != PQ_OK) return st;
  if (top_k < 1 || (order ? (long)rows * top_k != P : rows != P)) return PQ_ERR_SHAPE;
  if (!pqhost::aligned16(xq) || !pqhost::aligned16(xs) || !pqhost::aligned16(offsets) || !pqhost::aligned16(w) ||
      !pqhost::aligned16(w_scale) || !pqhost::aligned16(y) || (order && !pqhost::aligned16(order)))
    return PQ_ERR_ALIGN;
  GArgs a = {};
  a.xq = xq; a.xs = xs; a.w = w; a.ws = w_scale; a.y = y;
  a.offsets = offsets;
  a.order = order;
  a.xrows = rows; a.P = P;
  a.K = K; a.N = N; a.E = E; a.top_k = top_k;
  return run(a, epi, (hipStream_t)stream);
}

int pq_gemm_mxfp4_grouped(const uint16_t* x, int rows, int K, const int32_t* order, int top_k,
                          const int32_t* offsets, int P, int E, const uint8_t* w, const uint8_t* w_scale, int N,
                          int epi, uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !offsets || !w || !w_scale || !y) return PQ_ERR_NULL;
  int st = check_shape(rows, P, K, N, E, epi);
  if (st != PQ_OK) return st;
  if (top_k < 1 || (order ? (long)rows * top_k != P : rows != P)) return PQ_ERR_SHAPE;
  if (!pqhost::aligned16(x) || !pqhost::aligned16(offsets) || !pqhost::aligned16(w) ||
      !pqhost::aligned16(w_scale) || !pqhost::aligned16(y) || (order && !pqhost::aligned16(order)))
    return PQ_ERR_ALIGN;
  if (!ws || ws_bytes < scratch_bytes(rows, K)) return PQ_ERR_WORKSPACE;
  if (!pqhost::aligned16(ws)) return PQ_ERR_ALIGN;
  uint8_t *xq = scratch_codes(ws), *xs = scratch_scales(ws, rows, K);
  st = pq_quantize_mxfp4(x, 0, rows, K, xq, xs, stream);
  if (st != PQ_OK) return st;
  return pq_gemm_mxfp4_grouped_prequant(xq, xs, rows, K, order, top_k, offsets, P, E, w, w_scale, N, epi, y, stream);
}

}  // extern "C"
