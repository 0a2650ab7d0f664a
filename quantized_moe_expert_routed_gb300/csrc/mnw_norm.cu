// mnw_norm.cu -- root-mean-square norm with the residual's addition, output
// in BF16 and, on request, as INT8 codes with an FP32 scale per 128 values.
//
//   r' = bf16(x + r)                         (r' = x without a residual)
//   y  = bf16(r' * (mean(r'^2) + eps)^-1/2 * w)
//   per 128 values of y: s = max|y| / 127, code = clamp(rne(y / s), -127, 127)
//
// The norm is taken of the rounded r', the value that the next layer's
// residual stream holds, and the codes are those mnw_moe_quantize_act() gives
// for the rounded y, so the fused call equals the separate steps bit for bit.
// The sum of squares is FP32.
//
// Every element is read and written once, the row staying in registers
// between the sum and the product, so memory bounds it: 8192 rows of 4096 with
// residual and codes (303 MB) in 46.9 us, 6.5 TB/s and 97 % of the copy rate.
// Few rows are bound by one row's chain of load, two reductions and store:
// 1.4 us for one row of 2048, 2.2 us for 32 with codes.
#include <cuda_bf16.h>

#include "mnw_convert.cuh"
#include "mnw_int8_code.cuh"
#include "mnw_internal.h"
#include "mnw_ptx.cuh"

namespace mnw {
namespace norm {

constexpr int kMaxH = 16384;

struct Args {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;
  const __nv_bfloat16* w;
  __nv_bfloat16* residual_out;
  __nv_bfloat16* y;
  int8_t* codes;
  float* scales;
  long long x_stride;
  int T, H;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// One CTA per row, the row kept in registers: thread t holds the 16-byte
// words t, t + blockDim, ... (NV of them).  blockDim is a multiple of 16 words
// = 128 values, so a quantisation group lies in one half-warp.
template <int NV>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const Args a) {
  __shared__ float sums[32];
  pdl_launch_dependents();
  pdl_wait();
  const int words = a.H / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.x_stride);
  const size_t row = static_cast<size_t>(t) * a.H;
  // everything a thread reads is requested before the first use
  uint4 raw[NV], rr[NV], rw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    raw[i] = rr[i] = rw[i] = make_uint4(0, 0, 0, 0);
    if (c < words) {
      raw[i] = xr[c];
      if (a.residual) rr[i] = reinterpret_cast<const uint4*>(a.residual + row)[c];
      rw[i] = __ldg(reinterpret_cast<const uint4*>(a.w) + c);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    float v[8];
    unpack8(raw[i], v);
    if (a.residual) {
      float q[8];
      unpack8(rr[i], q);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += q[j];
      raw[i] = pack8(v);
      if (a.residual_out && c < words) reinterpret_cast<uint4*>(a.residual_out + row)[c] = raw[i];
      unpack8(raw[i], v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  sum = lane < static_cast<int>(blockDim.x >> 5) ? sums[lane] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = rsqrtf(sum / static_cast<float>(a.H) + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    float v[8], w[8];
    unpack8(raw[i], v);
    unpack8(rw[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * w[j];
    const uint4 out = pack8(v);
    if (a.y && c < words) reinterpret_cast<uint4*>(a.y + row)[c] = out;
    if (a.codes) {  // uniform over the CTA; the groups' maxima are half-warp reductions
      unpack8(out, v);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      uint32_t packed[2] = {0, 0};
      float scale = 0.f;
      if (amax > 0.f) {
        scale = __fdiv_rn(amax, 127.0f);
        const float rs = __frcp_rn(scale);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          packed[j >> 2] |= (static_cast<uint32_t>(int8_code(v[j], scale, rs)) & 0xFFu) << (8 * (j & 3));
      }
      if (c < words) {
        reinterpret_cast<uint2*>(a.codes + row)[c] = make_uint2(packed[0], packed[1]);
        if ((c & 15) == 0) a.scales[row / 128 + (c >> 4)] = scale;
      }
    }
  }
}

}  // namespace norm
}  // namespace mnw

using namespace mnw;

extern "C" {

int mnw_rmsnorm(const void* x, long long x_stride, const void* residual, const void* w, int T, int H, float eps,
                void* residual_out, void* y, int8_t* codes, float* scales, mnw_stream stream) {
  MNW_RANGE("mnw_rmsnorm");
  if (T < 0 || H <= 0 || H % 8 || !(eps >= 0.f) || !(eps < 3.0e38f)) return MNW_E_INVALID_ARG;
  if (x_stride < H || x_stride % 8) return MNW_E_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (!y && !codes)) return MNW_E_INVALID_ARG;
  if (residual_out && !residual) return MNW_E_INVALID_ARG;
  if (H > norm::kMaxH || (codes && H % 128)) return MNW_E_UNSUPPORTED;
  if (T == 0) return MNW_OK;
  if (!x || !w || !aligned(x, 16) || !aligned(w, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return MNW_E_INVALID_ARG;
  norm::Args a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.residual = static_cast<const __nv_bfloat16*>(residual);
  a.w = static_cast<const __nv_bfloat16*>(w);
  a.residual_out = static_cast<__nv_bfloat16*>(residual_out);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.codes = codes;
  a.scales = scales;
  a.x_stride = x_stride;
  a.T = T;
  a.H = H;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int words = H / 8;
  // Two words a thread where the rows fill the GPU many times over: half the threads of a row, twice the loads of each
  // under way and fewer warps at the row's barrier (8192 x 4096 with codes: 54 us with one, 46.7 with two, 48.7 with
  // four).  One where they do not and a row's own time counts (32 x 2048: 2.1 us, 2.6 with two; 1027 x 2176: 2.5, 2.7).
  const int per = words > 1024 || T >= 16 * current_sm_count() ? 2 : 1;
  const int threads = ((words + per - 1) / per + 31) / 32 * 32;
  const dim3 grid(T), block(threads);
  const cudaError_t e = per == 1 ? launch_pdl(norm::rmsnorm_kernel<1>, grid, block, 0, st, a)
                                 : launch_pdl(norm::rmsnorm_kernel<2>, grid, block, 0, st, a);
  return e == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}

}  // extern "C"
