// mnw_kv_append.cu -- new tokens' keys and values into a paged cache, with the
// position rotation of q and k applied on the way.
//
// Rotation of pair i of a head at position p, angle a = p * inv_freq[i]:
//   (u, w) -> m * (u cos a - w sin a, w cos a + u sin a)
// where (u, w) are elements (i, i + rot/2) of the head (half layout) or
// (2i, 2i + 1) (interleaved); elements past rot are copied.  FP32 arithmetic,
// one rounding to BF16.  INT8 caches quantise the rounded row: s = max|x| /
// 127, code = clamp(rne(x / s), -127, 127), as mnw_moe_quantize_act() does.
//
// The angle: at position 10^5 a radian's fraction lies 17 bits down, so a
// plain FP32 product would leave 7 bits of it.  It is taken in turns and in
// fixed point: inv_freq / (2 pi) as a 64-bit fraction, times the position
// modulo 2^64, loses whole turns and nothing else (2^-32 of a turn).  The upper
// 32 bits, rounded to FP32's 24, go to sincospif: 2^-25 turns at any position.
//
// Every element is read and written once, so memory bounds it.  Measured on
// one GB300 with 16 query, 4 key and 4 value heads of 128: 8192 BF16 tokens
// (101 MB) in 16.0 us, 6.3 TB/s, 94 % of the copy rate; 512 tokens into INT8
// pages in 3.9 us and four tokens in 2.7 us, bound by the chain of loads length
// -> page -> store.  One 16-byte chunk a thread, with the other element of a
// pair by shuffles, took 21.0 us for the 8192 (issue slots).
#include <cuda_bf16.h>

#include <cmath>

#include "mnw_convert.cuh"
#include "mnw_int8_code.cuh"
#include "mnw_internal.h"
#include "mnw_paged.cuh"
#include "mnw_ptx.cuh"

namespace mnw {
namespace kvapp {

using paged::Batch;
using paged::FastDiv;
using paged::Seq;

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;  // rot <= d <= 128
constexpr int kMaxTokens = 4;  // of a CTA
constexpr int kBatch = 3;      // pieces of a thread under way

struct Args {
  Batch bt;
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  __nv_bfloat16* q_out;
  uint8_t *kc, *vc;
  float *ks, *vs;
  long long page_stride;  // elements
  FastDiv page_div, row_div;  // row_div: by the head rows of a token
  int n_pages, page_size, Hq, Hkv, rot, tokens;
  const float* inv_freq;
  float mscale;
  uint32_t* err;
};

// Fraction of a turn, in [-1/2, 1/2], of position p >= 0 at frequency f (NaN and
// infinite frequencies give NaN).
__device__ __forceinline__ float turn_fraction(uint32_t p, float f) {
  constexpr uint32_t kHi = 0x28BE60DBu, kLo = 0x9391054Au;  // 2^64 / (2 pi)
  const uint32_t bits = __float_as_uint(f), m = bits << 8 | 0x80000000u;  // |f| = m 2^(e - 158)
  const int e = static_cast<int>(bits >> 23 & 0xFFu);
  const uint64_t mt = static_cast<uint64_t>(m) * kHi + __umulhi(m, kLo);  // m 2^32 / (2 pi)
  // |f| / (2 pi) in units of 2^-64, whole turns lost
  const uint64_t g = e <= 126 ? mt >> min(126 - e, 63) : mt << min(e - 126, 63);
  const float r = static_cast<float>(static_cast<int>((g * p) >> 32)) * 0x1p-32f;
  return fmaf(f, 0.f, f < 0.f ? -r : r);
}

// One CTA per `tokens` tokens.  A head row is D/16 pieces of two 16-byte
// chunks, one thread each: the two that hold both elements of 8 rotation pairs
// (half layout: chunks p and p + rot/16; elsewhere, and past rot, neighbours),
// so a rotation stays in a thread.  kBatch pieces of a thread are under way at
// a time, and the first batch is requested before the tokens' positions, pages
// and angles are worked out.
template <int D, bool INT8, bool HALF>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const Args a) {
  constexpr int P = D / 16;  // pieces (threads) of a row
  // sine and cosine, two pairs a word: pairs 8 p + 2 j, 8 p + 2 j + 1 at [j][p], so that a row's lanes read neighbours
  __shared__ float4 cs[kMaxTokens][4][kMaxPairs / 8];
  __shared__ int page_of[kMaxTokens], slot_of[kMaxTokens];  // the token's page (-1: none) and its slot there
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.bt.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.rot / 2;
  const int q_rows = a.q ? a.Hq : 0;
  const int rows = q_rows + 2 * a.Hkv;  // q heads, k heads, v heads of a token
  const int total = nt * rows * P;
  const int p = threadIdx.x % P;  // (kThreads is a multiple of P)
  const bool in_rot = 16 * p < a.rot;
  const int c0 = HALF && in_rot ? p : 2 * p, c1 = HALF && in_rot ? p + a.rot / 16 : 2 * p + 1;  // chunks

  struct Row {
    int tk, row;  // token of the CTA, head row of the token
  };
  auto row_at = [&](int idx) {
    const int rw = idx / P;
    Row x;
    x.tk = static_cast<int>(paged::quotient(rw, a.row_div));
    x.row = rw - x.tk * rows;
    return x;
  };
  uint4 raw[kBatch][2];
  auto load_batch = [&](int base) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int idx = base + i * kThreads + threadIdx.x;
      raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
      if (idx < total) {  // a row's lanes are all live or all not
        const Row x = row_at(idx);
        const long long t = t0 + x.tk;
        const __nv_bfloat16* src = x.row < q_rows           ? a.q + t * a.q_stride + x.row * D
                                   : x.row < q_rows + a.Hkv ? a.k + t * a.k_stride + (x.row - q_rows) * D
                                                            : a.v + t * a.v_stride + (x.row - q_rows - a.Hkv) * D;
        raw[i][0] = *reinterpret_cast<const uint4*>(src + c0 * 8);
        raw[i][1] = *reinterpret_cast<const uint4*>(src + c1 * 8);
      }
    }
  };
  load_batch(0);

  // a warp per token: its sequence, position, slot and angles
  if (warp < nt) {
    const int t = t0 + warp;
    int b;
    if (a.bt.q_start) {
      int cnt = 0;  // sequences that end at or before t
      for (int j = lane; j < a.bt.B; j += 32) cnt += __ldg(a.bt.q_start + j + 1) <= t ? 1 : 0;
      b = __reduce_add_sync(0xffffffffu, cnt);
    } else {
      b = t / a.bt.n_uniform;
    }
    bool bad = b >= a.bt.B;
    int pos = 0, page = -1, slot = 0;
    if (!bad) {
      const Seq s = paged::sequence(a.bt, b, a.page_size, &bad);
      pos = s.first + (t - s.start);
      const bool inside = t >= s.start && t < s.start + s.n && pos >= 0 && pos < s.len;
      if (inside) {
        const int pi = static_cast<int>(paged::quotient(pos, a.page_div));
        slot = pos - pi * a.page_size;
        page = __ldg(a.bt.block_table + static_cast<size_t>(b) * a.bt.max_pages + pi);
        if (page < 0 || page >= a.n_pages) {
          page = -1;
          if (lane == 0 && a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
        }
      } else {
        bad = true;
        if (pos >= s.len && lane == 0 && a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);  // past the table: no page
      }
    }
    if (bad && lane == 0 && a.err) atomicOr(a.err, MNW_DEVERR_BAD_LENGTH);
    if (lane == 0) {
      page_of[warp] = page;
      slot_of[warp] = slot;
    }
    for (int i = lane; i < pairs; i += 32) {
      float sn, co;
      sincospif(2.f * turn_fraction(static_cast<uint32_t>(pos), __ldg(a.inv_freq + i)), &sn, &co);
      reinterpret_cast<float2*>(&cs[warp][(i & 7) >> 1][i >> 3])[i & 1] = make_float2(co * a.mscale, sn * a.mscale);
    }
  }
  __syncthreads();

#pragma unroll 1
  for (int base = 0; base < total; base += kBatch * kThreads) {
    if (base > 0) load_batch(base);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int idx = base + i * kThreads + threadIdx.x;
      if (base + i * kThreads >= total) break;  // uniform
      const bool live = idx < total;
      const Row at = live ? row_at(idx) : Row{0, 0};
      const int tk = at.tk, row = at.row;
      const bool is_q = row < q_rows, is_k = !is_q && row < q_rows + a.Hkv;
      const int h = is_q ? row : (is_k ? row - q_rows : row - q_rows - a.Hkv);
      uint32_t u[2][4] = {{raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w}, {raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w}};
      if (in_rot && (is_q || is_k)) {
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // pairs 8 p + 2 j, 8 p + 2 j + 1
          const float4 f = cs[tk][j][p];
          if constexpr (HALF) {
            const float x0 = lo(u[0][j]), x1 = hi(u[0][j]), w0 = lo(u[1][j]), w1 = hi(u[1][j]);
            u[0][j] = pack_bf16x2(x0 * f.x - w0 * f.y, x1 * f.z - w1 * f.w);
            u[1][j] = pack_bf16x2(w0 * f.x + x0 * f.y, w1 * f.z + x1 * f.w);
          } else {
            uint32_t &a0 = u[j >> 1][2 * (j & 1)], &a1 = u[j >> 1][2 * (j & 1) + 1];
            const float x0 = lo(a0), w0 = hi(a0), x1 = lo(a1), w1 = hi(a1);
            a0 = pack_bf16x2(x0 * f.x - w0 * f.y, w0 * f.x + x0 * f.y);
            a1 = pack_bf16x2(x1 * f.z - w1 * f.w, w1 * f.z + x1 * f.w);
          }
        }
      }
      const uint4 out0 = make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]), out1 = make_uint4(u[1][0], u[1][1], u[1][2], u[1][3]);
      const int page = page_of[tk];
      const size_t head_row = static_cast<size_t>(h) * a.page_size + slot_of[tk];  // within the page
      if (is_q && live) {
        __nv_bfloat16* dst = a.q_out + (static_cast<size_t>(t0 + tk) * a.Hq + h) * D;
        *reinterpret_cast<uint4*>(dst + c0 * 8) = out0;
        *reinterpret_cast<uint4*>(dst + c1 * 8) = out1;
      }
      if constexpr (!INT8) {
        if (live && !is_q && page >= 0) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_k ? a.kc : a.vc) + page * a.page_stride + head_row * D;
          *reinterpret_cast<uint4*>(dst + c0 * 8) = out0;
          *reinterpret_cast<uint4*>(dst + c1 * 8) = out1;
        }
      } else {
        float y[2][8];
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[e][2 * j] = __uint_as_float(u[e][j] << 16);
            y[e][2 * j + 1] = __uint_as_float(u[e][j] & 0xFFFF0000u);
            amax = fmaxf(amax, fmaxf(fabsf(y[e][2 * j]), fabsf(y[e][2 * j + 1])));
          }
#pragma unroll
        for (int d = P / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (live && !is_q && page >= 0) {
          uint32_t packed[2][2] = {{0, 0}, {0, 0}};
          float scale = 0.f;
          if (amax > 0.f) {
            scale = __fdiv_rn(amax, 127.0f);
            const float rs = __frcp_rn(scale);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                packed[e][j >> 2] |= (static_cast<uint32_t>(int8_code(y[e][j], scale, rs)) & 0xFFu) << (8 * (j & 3));
          }
          uint8_t* dst = (is_k ? a.kc : a.vc) + page * a.page_stride + head_row * D;
          *reinterpret_cast<uint2*>(dst + c0 * 8) = make_uint2(packed[0][0], packed[0][1]);
          *reinterpret_cast<uint2*>(dst + c1 * 8) = make_uint2(packed[1][0], packed[1][1]);
          if (p == 0) (is_k ? a.ks : a.vs)[static_cast<size_t>(page) * a.Hkv * a.page_size + head_row] = scale;
        }
      }
    }
  }
}

template <int D, bool INT8>
cudaError_t launch(const Args& a, bool half, cudaStream_t st) {
  const dim3 grid((a.bt.T + a.tokens - 1) / a.tokens), block(kThreads);
  return half ? launch_pdl(kv_append_kernel<D, INT8, true>, grid, block, 0, st, a)
              : launch_pdl(kv_append_kernel<D, INT8, false>, grid, block, 0, st, a);
}

}  // namespace kvapp
}  // namespace mnw

using namespace mnw;

extern "C" {

int mnw_rope_frequencies(int rot, double base, int scale, double factor, double original_len, double beta_fast,
                         double beta_slow, float* inv_freq_host, float* mscale) {
  if (rot <= 0 || rot % 2 || !(base > 1.0) || !std::isfinite(base) || !inv_freq_host) return MNW_E_INVALID_ARG;
  if (scale < MNW_ROPE_SCALE_NONE || scale > MNW_ROPE_SCALE_BY_PARTS) return MNW_E_INVALID_ARG;
  if (scale != MNW_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MNW_E_INVALID_ARG;
  const bool parts = scale == MNW_ROPE_SCALE_BY_PARTS;
  if (parts && (!(original_len > 0.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return MNW_E_INVALID_ARG;
  if (scale == MNW_ROPE_SCALE_NTK) {
    if (rot < 4) return MNW_E_INVALID_ARG;
    base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  }
  const double two_pi = 6.283185307179586476925;
  // pair (as a real number) that turns beta times within original_len
  auto pair_of = [&](double beta) { return rot * std::log(original_len / (beta * two_pi)) / (2.0 * std::log(base)); };
  double lo = 0.0, hi = 1.0;
  if (parts) {
    lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.0);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scale == MNW_ROPE_SCALE_LINEAR) f /= factor;
    if (parts) {
      const double slow = std::fmin(1.0, std::fmax(0.0, (i - lo) / (hi - lo)));
      f = f / factor * slow + f * (1.0 - slow);
    }
    inv_freq_host[i] = static_cast<float>(f);
  }
  if (mscale) *mscale = parts ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return MNW_OK;
}

int mnw_kv_append(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                  long long v_stride, int B, int T, int Hq, int Hkv, int d, const float* inv_freq, int rot, int layout,
                  float mscale, void* k_cache, void* v_cache, float* k_scale, float* v_scale, int fmt, int n_pages,
                  int page_size, long long page_stride, const int32_t* block_table, int max_pages,
                  const int32_t* cache_lens, const int32_t* q_start, void* q_out, uint32_t* err, mnw_stream stream) {
  MNW_RANGE("mnw_kv_append");
  if (B < 0 || T < 0) return MNW_E_INVALID_ARG;
  if (B == 0 || T == 0) return T == 0 ? MNW_OK : MNW_E_INVALID_ARG;
  int rc = paged::check_cache(k_cache, v_cache, k_scale, v_scale, fmt, n_pages, page_size, Hkv, d, page_stride);
  if (rc != MNW_OK) return rc;
  rc = paged::check_batch(block_table, cache_lens, q_start, B, T, max_pages, page_size);
  if (rc != MNW_OK) return rc;
  if (rot < 0 || rot > d || (rot > 0 && !inv_freq) || !aligned(inv_freq, 4)) return MNW_E_INVALID_ARG;
  if (layout != MNW_ROPE_HALF && layout != MNW_ROPE_INTERLEAVED) return MNW_E_INVALID_ARG;
  if (rot % 16) return MNW_E_UNSUPPORTED;
  if (!(mscale > 0.f) || !(mscale < 3.0e38f)) return MNW_E_INVALID_ARG;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8 ||
      k_stride < static_cast<long long>(Hkv) * d || v_stride < static_cast<long long>(Hkv) * d)
    return MNW_E_INVALID_ARG;
  if (q) {
    if (Hq <= 0 || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 ||
        q_stride < static_cast<long long>(Hq) * d)
      return MNW_E_INVALID_ARG;
    if (Hq > 1024) return MNW_E_UNSUPPORTED;
  }
  kvapp::Args a{};
  a.bt = paged::Batch{block_table, cache_lens, q_start, B, T, max_pages, q_start ? 0 : T / B};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.ks = k_scale;
  a.vs = v_scale;
  a.page_stride = page_stride;
  a.page_div = paged::fast_div(page_size);
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.rot = rot;
  // One token a CTA while the batch does not fill the GPU several times over (512 INT8 tokens: 3.8 us), four from there
  // on, whose loads are under way together (8192 tokens: 24.4 us with one, 19.6 two, 15.7 four, 15.5 eight).
  a.tokens = T >= 8 * current_sm_count() ? kvapp::kMaxTokens : 1;
  a.row_div = paged::fast_div((q ? Hq : 0) + 2 * Hkv);
  a.inv_freq = inv_freq;
  a.mscale = mscale;
  a.err = err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool half = layout == MNW_ROPE_HALF, int8 = fmt == MNW_KV_INT8;
  cudaError_t e;
  if (d == 128)
    e = int8 ? kvapp::launch<128, true>(a, half, st) : kvapp::launch<128, false>(a, half, st);
  else
    e = int8 ? kvapp::launch<64, true>(a, half, st) : kvapp::launch<64, false>(a, half, st);
  return e == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}

}  // extern "C"
