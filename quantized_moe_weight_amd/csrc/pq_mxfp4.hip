// MXFP4 encoding and decoding of rows: one E8M0 scale byte per 32 values, E2M1
// codes.
//
// Bound by memory: the encoder reads 2 or 4 bytes a value and writes 17/32 of
// one, the decoder the reverse.  A thread owns 8 consecutive values (one or
// two 16-byte accesses); 4 lanes share a block, whose largest magnitude is the
// maximum of the values' absolute bits as integers (the order of non-negative
// floats, with infinities and NaN above every finite value), by lane swaps.
#include "pq_mxfp4_dev.h"
#include "pq_quant_dev.h"

namespace {

constexpr int kThreads = 256;
constexpr long kMaxBlocks = 1 << 20;   // threads of a launch stay below 2^32; larger inputs loop

// maximum over the 4 lanes of a block, in every lane
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = pq::umax(v, (uint32_t)pq::dpp_i32<0xB1>((int)v));    // quad_perm [1,0,3,2]
  return pq::umax(v, (uint32_t)pq::dpp_i32<0x4E>((int)v)); // quad_perm [2,3,0,1]
}

// Groups of 8 values that a thread has in flight, kThreads groups apart, and
// whether they are read past the caches (bf16 32768 x 2048: 27.8 us at 4 and
// past them, 30.8 at 1; fp32 17408 x 5120, whose group is two loads: 81.7 and
// 69.7).
template <bool F32_IN>
constexpr int kInFlight = F32_IN ? 1 : 4;

template <bool F32_IN>
__device__ __forceinline__ uint4 load16(const uint4* p) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  if constexpr (F32_IN) return *p;
  else return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}

template <bool F32_IN>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(const void* in, long total8, uint8_t* codes,
                                                                   uint8_t* scales) {
  constexpr int U = kInFlight<F32_IN>;
  constexpr int W = F32_IN ? 2 : 1;                 // 16-byte loads per group
  // total8 is a multiple of 4, so the 4 lanes of a block go together
  for (long t0 = (long)blockIdx.x * kThreads * U + threadIdx.x; t0 < total8; t0 += (long)gridDim.x * kThreads * U) {
    uint4 raw[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long t = t0 + u * kThreads;
#pragma unroll
      for (int i = 0; i < W; ++i)
        raw[u][i] = t < total8 ? load16<F32_IN>(reinterpret_cast<const uint4*>(in) + W * t + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long t = t0 + u * kThreads;
      float v[8];
      if constexpr (F32_IN) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v[4 * i] = __uint_as_float(raw[u][i].x); v[4 * i + 1] = __uint_as_float(raw[u][i].y);
          v[4 * i + 2] = __uint_as_float(raw[u][i].z); v[4 * i + 3] = __uint_as_float(raw[u][i].w);
        }
      } else {
        pq::bf16x8_to_f32(raw[u][0], v);
      }
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = pq::umax(m, __float_as_uint(v[i]) & 0x7fffffffu);
      const uint32_t byte = pq::mx_scale_byte(quad_umax(m));
      const uint32_t w = pq::mx_codes8(v, pq::mx_scale_operand(byte));
      if (t < total8) {
        reinterpret_cast<uint32_t*>(codes)[t] = byte == pq::kMxNan ? 0u : w;
        if ((threadIdx.x & 3) == 0) scales[t >> 2] = (uint8_t)byte;
      }
    }
  }
}

template <bool F32_OUT>
__global__ __launch_bounds__(kThreads) void dequantize_mxfp4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                     long total8, void* out) {
  for (long t = (long)blockIdx.x * kThreads + threadIdx.x; t < total8; t += (long)gridDim.x * kThreads) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[t];
    const float s = pq::mx_scale_operand(scales[t >> 2]);
    if (F32_OUT) {
      float4* p = reinterpret_cast<float4*>(out) + 2 * t;
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
      const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
      const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
      p[0] = make_float4(a[0], a[1], b[0], b[1]);
      p[1] = make_float4(c[0], c[1], d[0], d[1]);
    } else {
      reinterpret_cast<uint4*>(out)[t] = pq::mx_bf16x8(w, s);
    }
  }
}

unsigned grid_for(long total8) {
  const long blocks = (total8 + kThreads - 1) / kThreads;
  return (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

}  // namespace

extern "C" {

int pq_quantize_mxfp4(const void* in, int in_is_f32, int rows, int K, uint8_t* codes, uint8_t* scales,
                      void* stream) {
  if (!in || !codes || !scales) return PQ_ERR_NULL;
  if (rows < 1 || K < pq::kMxBlock || K % pq::kMxBlock != 0) return PQ_ERR_SHAPE;
  if (!pqhost::aligned16(in) || !pqhost::aligned16(codes) || !pqhost::aligned16(scales)) return PQ_ERR_ALIGN;
  pqhost::DeviceInfo dev;
  const int st = pqhost::current_device_info(&dev);
  if (st != PQ_OK) return st;
  const long total8 = (long)rows * K / 8;
  const int u = in_is_f32 ? kInFlight<true> : kInFlight<false>;
  auto kern = in_is_f32 ? quantize_mxfp4_kernel<true> : quantize_mxfp4_kernel<false>;
  hipLaunchKernelGGL(kern, dim3(grid_for((total8 + u - 1) / u)), dim3(kThreads), 0, (hipStream_t)stream, in, total8,
                     codes, scales);
  PQ_HIP_CHECK(hipGetLastError());
  return PQ_OK;
}

int pq_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int rows, int K, int out_is_f32, void* out,
                        void* stream) {
  if (!codes || !scales || !out) return PQ_ERR_NULL;
  if (rows < 1 || K < pq::kMxBlock || K % pq::kMxBlock != 0) return PQ_ERR_SHAPE;
  if (!pqhost::aligned16(codes) || !pqhost::aligned16(scales) || !pqhost::aligned16(out)) return PQ_ERR_ALIGN;
  pqhost::DeviceInfo dev;
  const int st = pqhost::current_device_info(&dev);
  if (st != PQ_OK) return st;
  const long total8 = (long)rows * K / 8;
  if (out_is_f32)
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<true>, dim3(grid_for(total8)), dim3(kThreads), 0, (hipStream_t)stream,
                       codes, scales, total8, out);
  else
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<false>, dim3(grid_for(total8)), dim3(kThreads), 0,
                       (hipStream_t)stream, codes, scales, total8, out);
  PQ_HIP_CHECK(hipGetLastError());
  return PQ_OK;
}

}  // extern "C"
