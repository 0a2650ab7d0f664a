// mnw_kv_values.cu -- the BF16 values of a quantised cache's pages.
//
// INT8: code * scale; INT4: code * (m * S) (mnw_int4_row.cuh).  Each is a
// product in FP32 (m * S exact where S has at most 16 bits, as the append's
// have) rounded to BF16: off by half a step and a 2^-16 of one.
//
// Every byte is read and written once, so memory bounds it.  A thread makes 8
// elements, one 16-byte store.  129 pages of 4 x 64 rows of 128 (10.8 MB): 3.4 us
// in a graph.  Alone and cold 4.8; with the page by a 64-bit division a thread 6.5.
#include <cuda_bf16.h>

#include "mnw_convert.cuh"
#include "mnw_int4_row.cuh"
#include "mnw_internal.h"
#include "mnw_paged.cuh"

namespace mnw {
namespace kvval {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // chunks of 8 elements of a thread under way

struct Args {
  const uint8_t* cache;
  const void* scale;
  __nv_bfloat16* out;
  long long page_bytes;     // between pages of the cache
  long long chunks;         // of all pages
  int page_chunks;
  paged::FastDiv page_div;  // by page_chunks
};

// BIG: more than 2^31 chunks, whose places take 64 bits.
template <int D, bool INT4, bool BIG>
__global__ void __launch_bounds__(kThreads) kv_values_kernel(const Args a) {
  constexpr int kBytes = INT4 ? 4 : 8;  // of a chunk's codes
  constexpr int kPerRow = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const long long at0 = static_cast<long long>(blockIdx.x) * (kThreads * kBatch) + threadIdx.x;
  uint2 raw[kBatch], rec[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const long long at = at0 + i * kThreads;
    raw[i] = rec[i] = make_uint2(0, 0);
    if (at < a.chunks) {
      const long long page = BIG ? at / a.page_chunks : static_cast<int>(paged::quotient(static_cast<uint32_t>(at), a.page_div));
      const uint8_t* src = a.cache + page * a.page_bytes + (at - page * a.page_chunks) * kBytes;
      const long long row = at / kPerRow;
      if constexpr (INT4) {
        raw[i].x = *reinterpret_cast<const uint32_t*>(src);
        rec[i] = static_cast<const uint2*>(a.scale)[row];
      } else {
        raw[i] = *reinterpret_cast<const uint2*>(src);
        rec[i].x = static_cast<const uint32_t*>(a.scale)[row];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const long long at = at0 + i * kThreads;
    if (at >= a.chunks) break;
    float f = __uint_as_float(rec[i].x);
    float v[8];
    if constexpr (INT4) {
      const int g = static_cast<int>(at % kPerRow) / (kPerRow / 4);
      f *= static_cast<float>((rec[i].y >> (8 * g)) & 0xFFu);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = static_cast<float>(static_cast<int>((raw[i].x >> (4 * (e / 2) + 16 * (e % 2))) & 15u) - 8) * f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = static_cast<float>(static_cast<int8_t>(((e < 4 ? raw[i].x : raw[i].y) >> (8 * (e & 3))) & 0xFFu)) * f;
    }
    *reinterpret_cast<uint4*>(a.out + at * 8) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

template <int D, bool INT4>
cudaError_t launch(const Args& a, cudaStream_t st) {
  constexpr int kPer = kThreads * kBatch;
  const dim3 grid(static_cast<unsigned>((a.chunks + kPer - 1) / kPer));
  return a.chunks > 0x7fffffffll ? launch_pdl(kv_values_kernel<D, INT4, true>, grid, dim3(kThreads), 0, st, a)
                                 : launch_pdl(kv_values_kernel<D, INT4, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace kvval
}  // namespace mnw

using namespace mnw;

extern "C" {

int mnw_kv_values(const void* cache, const void* scale, int fmt, int n_pages, int page_size, int Hkv, int d,
                  long long page_stride, void* out, mnw_stream stream) {
  MNW_RANGE("mnw_kv_values");
  if (fmt != MNW_KV_INT8 && fmt != MNW_KV_INT4) return MNW_E_INVALID_ARG;
  const float* sc = static_cast<const float*>(scale);
  const int rc = paged::check_cache(cache, cache, sc, sc, fmt, n_pages, page_size, Hkv, d, page_stride);
  if (rc != MNW_OK) return rc;
  if (!out || !aligned(out, 16)) return MNW_E_INVALID_ARG;
  kvval::Args a{};
  a.cache = static_cast<const uint8_t*>(cache);
  a.scale = scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.page_bytes = fmt == MNW_KV_INT4 ? page_stride / 2 : page_stride;
  const long long page_chunks = static_cast<long long>(Hkv) * page_size * (d / 8);
  if (page_chunks > 0x7fffffffll) return MNW_E_UNSUPPORTED;
  a.page_chunks = static_cast<int>(page_chunks);
  a.chunks = page_chunks * n_pages;
  a.page_div = paged::fast_div(static_cast<uint32_t>(page_chunks));
  if (a.chunks > 0x7fffffffll * 256) return MNW_E_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (fmt == MNW_KV_INT4)
    e = d == 128 ? kvval::launch<128, true>(a, st) : kvval::launch<64, true>(a, st);
  else
    e = d == 128 ? kvval::launch<128, false>(a, st) : kvval::launch<64, false>(a, st);
  return e == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}

}  // extern "C"
