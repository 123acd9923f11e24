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

template <bool F32_IN>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(const void* in, long total8, uint8_t* codes,
                                                                   uint8_t* scales) {
  // total8 is a multiple of 4, so the 4 lanes of a block loop together
  for (long t = (long)blockIdx.x * kThreads + threadIdx.x; t < total8; t += (long)gridDim.x * kThreads) {
    float v[8];
    if (F32_IN) {
      const float4* p = reinterpret_cast<const float4*>(in) + 2 * t;
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      pq::bf16x8_to_f32(reinterpret_cast<const uint4*>(in)[t], v);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = pq::umax(m, __float_as_uint(v[i]) & 0x7fffffffu);
    const uint32_t byte = pq::mx_scale_byte(quad_umax(m));
    const uint32_t w = pq::mx_codes8(v, pq::mx_scale_operand(byte));
    reinterpret_cast<uint32_t*>(codes)[t] = byte == pq::kMxNan ? 0u : w;
    if ((threadIdx.x & 3) == 0) scales[t >> 2] = (uint8_t)byte;
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
  if (in_is_f32)
    hipLaunchKernelGGL(quantize_mxfp4_kernel<true>, dim3(grid_for(total8)), dim3(kThreads), 0, (hipStream_t)stream,
                       in, total8, codes, scales);
  else
    hipLaunchKernelGGL(quantize_mxfp4_kernel<false>, dim3(grid_for(total8)), dim3(kThreads), 0, (hipStream_t)stream,
                       in, total8, codes, scales);
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
