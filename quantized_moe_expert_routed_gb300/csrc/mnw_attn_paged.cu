// mnw_attn_paged.cu -- attention of new tokens (one each, a refinement block,
// several) over a paged key/value cache, split over the cache's length.
//
// For new token i of sequence b (position p = len - n + i) and query head h
// (kv head g = h / (Hq / Hkv)), over the allowed positions j < min(len,
// (p / blk + 1) * blk):
//   s_j = scale * q . k_j,   out = sum_j e^{s_j} v_j / sum_j e^{s_j},
//   lse = log sum_j e^{s_j}
// One pass with a running maximum and sum per row.
//
// Bound: every cached key and value is read once for all rows of its kv head
// (n * Hq / Hkv query rows), so up to ~100 rows the reads of the cache are the
// floor.  Measured on one GB300: 2 single tokens over 200,000 BF16 positions, 32
// query and 8 key heads of 128 (1.64 GB): 243 us, 6.7 TB/s, 94 % of the rate of
// reads alone; 32 over 2048 to 8192 positions in pages of 16, 16 and 4 heads
// (336 MB): 65 us, 5.2 TB/s, of which ~10 us are the head (split, first page
// lookups) and the join; one over 777 positions: 7.9 us, the chain split -> page
// -> tile -> products -> join.  INT8, 2 over 200,000 (0.84 GB): 210 us, 4.0 TB/s,
// bound by the conversion of codes and by latency at 8 warps an SM (issue slots
// 50 %); three CTAs of two stages instead of two of three: 230 us.
//
// The work's split over CTAs and the joining of its parts: mnw_attn_split.cuh.
//
// Up to 16 query rows (INT8: 32) go here, more to the block kernel.  A CTA is
// WR x WK warps: WR row blocks of 16 query rows, each tile's keys cut over WK
// warps.  Tiles arrive by 16-byte cp.async through a ring of kStages stages,
// one page lookup per key, so pages of any size may end inside a tile; rows
// past the length are filled with zeros (a masked probability of 0 then meets
// a finite value, whatever the page holds there).  Both products are mma.sync
// with FP32 accumulation.
//
// BF16 caches: probabilities enter the second product rounded to BF16 (2^-8
// relative each, independent, so the sum's error stays near the output's own
// rounding); the sum of probabilities is taken before that rounding.
// INT8 caches: the first product runs on FP16 operands: codes are exact there,
// and q is re-encoded per row as FP16 times a power of two (exact for values
// within 2^28 of the row's largest); the keys' scales multiply the FP32 scores.
// The second runs on TF32: codes are exact, and the probabilities times the
// values' scales, rounded to 11 bits (2^-11), keep FP32's exponents, so value
// scales of any spread keep the sum's accuracy (FP16 would lose weights 2^-24
// below the largest).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <ctime>

#include "mnw_attn_split.cuh"

namespace mnw {
namespace pattn {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Code `B` of four biased ones as FP32: the byte under the exponent of 2^23 is
// the value 2^23 + byte.
template <int B>
__device__ __forceinline__ uint32_t code_f32(uint32_t w) {
  return __float_as_uint(__uint_as_float(prmt(w, 0x4B000000u, 0x7440 + B)) - 8388736.f);
}
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool INT8, int WR, int WK>
struct Cfg {
  static constexpr int kWarps = WR * WK, kThreads = kWarps * 32, kRT = WR * 16;
  static constexpr int kTK = INT8 ? 128 : 64;  // keys per tile: 16 KB of keys either way (d = 128)
  static constexpr int kRowBytes = INT8 ? D : 2 * D;
  static constexpr int kTileBytes = kTK * kRowBytes;
  static constexpr int kScaleBytes = INT8 ? 2 * kTK * 4 : 0;
  static constexpr int kStageBytes = 2 * kTileBytes + kScaleBytes;
  static constexpr int kStages = 3;
  static constexpr int kSmem = kStages * kStageBytes;
  // at an item's end the warps' outputs meet in the stage just read
  static_assert(kWarps * 16 * D * 4 <= kStageBytes && kTK <= kThreads && WK > 1);
  static_assert(kThreads / (D / 4) * 2 * kJoinBatch * 4 <= kStageBytes);
};

// Byte offset of 16-byte chunk c of row r in a tile: chunks are exchanged by
// the row so that the eight rows of a matrix load fall into different banks.
template <int D, bool INT8>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (!INT8) return static_cast<uint32_t>(r * D * 2 + ((c ^ (r & 7)) << 4));
  else if constexpr (D == 128)  // key reads take rows 2h, 2h+1 x 4 chunks, value reads rows 0,2,4,6 x 2 chunks
    return static_cast<uint32_t>(r * D + ((c ^ ((r & 6) ^ ((r & 1) << 2))) << 4));
  else
    return static_cast<uint32_t>(r * D + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, bool INT8, int WR, int WK>
__global__ void __launch_bounds__(WR* WK * 32) paged_attn_kernel(const Args a) {
  using C = Cfg<D, INT8, WR, WK>;
  constexpr int kRT = C::kRT, kThreads = C::kThreads, kStages = C::kStages, kTK = C::kTK;
  constexpr int kKS = D / 16;        // k steps of the first product
  constexpr int kNO = D / 8;         // output column tiles
  constexpr int kKW = kTK / WK;      // keys of a tile per warp
  constexpr int kNB = kKW / 16;      // 16-key blocks per warp
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SplitShared split;
  __shared__ float2 ml[C::kWarps * 16];
  __shared__ long long row_at[kStages][kTK];                // byte offset of a tile's keys' cached rows, -1: none
  __shared__ long long scale_at[INT8 ? kStages : 1][kTK];   // INT8: and of their scales
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wr = warp / WK, wk = warp % WK;
  const int g8 = lane >> 2, t4 = lane & 3;
  const uint32_t sbase = smem_u32(smem);

  pdl_launch_dependents();
  pdl_wait();

  const Run run = find_run<kRT, kTK, kThreads, 0>(a, &split);
  if (run.seq < 0) return;  // no units left for this run
  Cursor<kRT, kTK> cc;  // the tile computed
  cc.set(a, run);
  int item_first = run.u0 - cc.kt;  // first unit of its item
  const int tiles = run.pad == 1 ? run.u1 - run.u0 : min(run.u1 - run.u0, cc.sh.kt - cc.kt);
  if (tiles <= 0) return;

  // ---- tile loads: page lookups run one tile ahead of the copies, those kStages - 1 ahead of the products ----
  Cursor<kRT, kTK> lc = cc;  // the tile looked up next
  auto look = [&](int2& at) {  // raw page entry and head row of key tid of tile lc; then on to the next tile
    const int p = lc.kt * kTK + tid;
    at = make_int2(0, -1);
    if (tid < kTK && p < lc.s.len) {
      const int pi = static_cast<int>(paged::quotient(p, a.page_div));
      at.x = __ldg(a.bt.block_table + static_cast<size_t>(lc.b) * a.bt.max_pages + pi);
      at.y = lc.g * a.page_size + (p - pi * a.page_size);
    }
    if (++lc.kt == lc.sh.kt) lc.next_item(a, run.pad);
  };
  auto keep = [&](int2 at, int slot) {
    if (tid >= kTK) return;
    bool has = at.y >= 0;
    if (has && static_cast<unsigned>(at.x) >= static_cast<unsigned>(a.n_pages)) {
      has = false;
      if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
    }
    row_at[slot][tid] = has ? at.x * a.page_bytes + static_cast<long long>(at.y) * C::kRowBytes : -1;
    if constexpr (INT8) scale_at[slot][tid] = (static_cast<long long>(at.x) * a.Hkv * a.page_size + at.y) * 4;
  };
  auto load_tile = [&](int slot) {
    const uint32_t st = sbase + slot * C::kStageBytes;
    constexpr int kCh = C::kRowBytes / 16;  // chunks per row
    constexpr int kRP = kThreads / kCh;     // rows per pass
    const int c = tid % kCh;
#pragma unroll
    for (int i = 0; i < kTK / kRP; ++i) {
      const int r = i * kRP + tid / kCh;
      const long long at = row_at[slot][r];
      const uint32_t n = at >= 0 ? 16u : 0u;
      const long long off = n ? at + c * 16 : 0;
      const uint32_t to = st + chunk_at<D, INT8>(r, c);
      cp_async16(to, a.kc + off, n);
      cp_async16(to + C::kTileBytes, a.vc + off, n);
    }
    if constexpr (INT8) {
      for (int r2 = tid; r2 < 2 * kTK; r2 += kThreads) {
        const uint32_t n = row_at[slot][r2 % kTK] >= 0 ? 4u : 0u;
        const long long off = n ? scale_at[slot][r2 % kTK] : 0;
        cp_async4(st + 2 * C::kTileBytes + r2 * 4, reinterpret_cast<const char*>(r2 < kTK ? a.ks : a.vs) + off, n);
      }
    }
  };
  {
    int2 at[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (i < tiles) look(at[i]);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (i < tiles) keep(at[i], i);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < tiles) load_tile(i);
      cp_commit();
    }
  }

  // ---- state of the item in hand ----
  uint32_t qf[kKS][4];
  float qfac0 = a.scale_log2, qfac1 = a.scale_log2;  // score factor of rows r0, r1
  const int r0 = wr * 16 + g8, r1 = r0 + 8;
  int rows = 0, lim_lo = 0, lim_hi = 0, lim0 = 0, lim1 = 0;
  float o[kNO][4];
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
  int kt_begin = 0;
  auto begin_item = [&]() {
    kt_begin = cc.kt;
    rows = min(kRT, cc.s.n * a.G - cc.rt * kRT);
    // limits ascend with the rows, but for tokens past the table at the end, which have none
    const int ri = cc.rt * kRT, first = row_limit(a, cc.s, ri), last = row_limit(a, cc.s, ri + rows - 1);
    lim_lo = min(first, last);
    lim_hi = last;
    if (last == 0 && cc.s.first + static_cast<int>(paged::quotient(ri + rows - 1, a.g_div)) >= cc.s.len &&
        cc.s.first + static_cast<int>(paged::quotient(ri, a.g_div)) < cc.s.len)
      lim_hi = cc.s.len;  // the row of the last position is between
    lim0 = r0 < rows ? row_limit(a, cc.s, cc.rt * kRT + r0) : lim_hi;
    lim1 = r1 < rows ? row_limit(a, cc.s, cc.rt * kRT + r1) : lim_hi;
#pragma unroll
    for (int i = 0; i < kNO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    // ---- query fragments ----
    {
      auto row_ptr = [&](int r) -> const __nv_bfloat16* {
        const int ri = cc.rt * kRT + r;
        const int i = static_cast<int>(paged::quotient(ri, a.g_div)), hh = ri - i * a.G;
        return a.q + static_cast<long long>(cc.s.start + i) * a.q_stride + static_cast<long long>(cc.g * a.G + hh) * D;
      };
      const bool ok0 = r0 < rows, ok1 = r1 < rows;
      const __nv_bfloat16 *p0 = row_ptr(ok0 ? r0 : 0), *p1 = row_ptr(ok1 ? r1 : 0);
      if constexpr (!INT8) {
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          qf[ks][0] = ok0 ? *reinterpret_cast<const uint32_t*>(p0 + 16 * ks + 2 * t4) : 0u;
          qf[ks][1] = ok1 ? *reinterpret_cast<const uint32_t*>(p1 + 16 * ks + 2 * t4) : 0u;
          qf[ks][2] = ok0 ? *reinterpret_cast<const uint32_t*>(p0 + 16 * ks + 2 * t4 + 8) : 0u;
          qf[ks][3] = ok1 ? *reinterpret_cast<const uint32_t*>(p1 + 16 * ks + 2 * t4 + 8) : 0u;
        }
      } else {
        // k step 4j + s4 of the products takes elements 16 (t4 + 4j) + 4 s4 .. + 3 of lane t4: the order in
        // which a lane's 16-byte word of codes holds them
        uint32_t m0 = 0, m1 = 0;  // magnitudes' largest bit patterns
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int s4 = 0; s4 < 4; ++s4) {
            const int e = 16 * (t4 + 4 * j) + 4 * s4;
            const uint2 x0 = ok0 ? *reinterpret_cast<const uint2*>(p0 + e) : make_uint2(0, 0);
            const uint2 x1 = ok1 ? *reinterpret_cast<const uint2*>(p1 + e) : make_uint2(0, 0);
            qf[4 * j + s4][0] = x0.x;
            qf[4 * j + s4][2] = x0.y;
            qf[4 * j + s4][1] = x1.x;
            qf[4 * j + s4][3] = x1.y;
            m0 = max(max(m0, x0.x & 0x7FFFu), max((x0.x >> 16) & 0x7FFFu, max(x0.y & 0x7FFFu, (x0.y >> 16) & 0x7FFFu)));
            m1 = max(max(m1, x1.x & 0x7FFFu), max((x1.x >> 16) & 0x7FFFu, max(x1.y & 0x7FFFu, (x1.y >> 16) & 0x7FFFu)));
          }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, d));
          m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, d));
        }
        const int e0 = row_exponent(m0), e1 = row_exponent(m1);
        const float i0 = two_to(-e0), i1 = two_to(-e1);
        qfac0 = a.scale_log2 * two_to(e0);
        qfac1 = a.scale_log2 * two_to(e1);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float f = (w & 1) ? i1 : i0;
            const uint32_t x = qf[ks][w];
            const __half2 hv = __floats2half2_rn(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
            qf[ks][w] = *reinterpret_cast<const uint32_t*>(&hv);
          }
      }
    }
  };

  for (int t = 0, slot = 0; t < tiles; ++t) {
    cp_wait<kStages - 2>();
    __syncthreads();
    {
      int ns = slot + kStages - 1;
      if (ns >= kStages) ns -= kStages;
      if (t + kStages - 1 < tiles) load_tile(ns);
      cp_commit();
    }
    int2 ahead;
    const bool more = t + kStages < tiles;
    if (more) look(ahead);
    if (t == 0 || cc.kt == 0) begin_item();
    const uint32_t kst = sbase + slot * C::kStageBytes, vst = kst + C::kTileBytes;
    uint8_t* stage = smem + slot * C::kStageBytes;

    if (cc.kt * kTK < lim_hi) {  // a tile past every row's limit adds nothing
      // scores of the warp's keys
      float sc[2 * kNB][4];
#pragma unroll
      for (int i = 0; i < 2 * kNB; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
      if constexpr (!INT8) {
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
          const int row = wk * kKW + nb * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks) {
            uint32_t kf[4];
            ldsm4(kst + chunk_at<D, INT8>(row, 2 * ks + ((lane >> 3) & 1)), kf);
            mma16816<false>(sc[2 * nb], qf[ks], kf[0], kf[1]);
            mma16816<false>(sc[2 * nb + 1], qf[ks], kf[2], kf[3]);
          }
        }
      } else {
        // the accumulators' chains in turn: one after the other they are kKS products' latencies each
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 w[2 * kNB];
#pragma unroll
          for (int i = 0; i < 2 * kNB; ++i)
            w[i] = *reinterpret_cast<const uint4*>(stage + chunk_at<D, INT8>(wk * kKW + 8 * i + g8, t4 + 4 * j));
#pragma unroll
          for (int s4 = 0; s4 < 4; ++s4) {
#pragma unroll
            for (int i = 0; i < 2 * kNB; ++i) {
              const uint32_t x = (s4 == 0 ? w[i].x : s4 == 1 ? w[i].y : s4 == 2 ? w[i].z : w[i].w) ^ 0x80808080u;
              mma16816<true>(sc[i], qf[4 * j + s4], codes_lo(x), codes_hi(x));
            }
          }
        }
      }
      if constexpr (INT8) {
        const float* ksc = reinterpret_cast<const float*>(stage + 2 * C::kTileBytes);
#pragma unroll
        for (int i = 0; i < 2 * kNB; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(ksc + wk * kKW + 8 * i + 2 * t4);
          sc[i][0] *= f.x;
          sc[i][1] *= f.y;
          sc[i][2] *= f.x;
          sc[i][3] *= f.y;
        }
      }
      const int key_base = cc.kt * kTK + wk * kKW + 2 * t4;
      if ((cc.kt + 1) * kTK > lim_lo) {  // some row's limit lies in this tile
#pragma unroll
        for (int i = 0; i < 2 * kNB; ++i) {
          const int k = key_base + 8 * i;
          if (k >= lim0) sc[i][0] = -INFINITY;
          if (k + 1 >= lim0) sc[i][1] = -INFINITY;
          if (k >= lim1) sc[i][2] = -INFINITY;
          if (k + 1 >= lim1) sc[i][3] = -INFINITY;
        }
      }
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2 * kNB; ++i) {
        x0 = fmaxf(x0, fmaxf(sc[i][0], sc[i][1]));
        x1 = fmaxf(x1, fmaxf(sc[i][2], sc[i][3]));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      const float n0 = fmaxf(m0, x0 * qfac0), n1 = fmaxf(m1, x1 * qfac1);
      const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
      float c0 = ex2(m0 - b0), c1 = ex2(m1 - b1);
      m0 = n0;
      m1 = n1;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int i = 0; i < 2 * kNB; ++i) {
        sc[i][0] = ex2(fmaf(sc[i][0], qfac0, -b0));
        sc[i][1] = ex2(fmaf(sc[i][1], qfac0, -b0));
        sc[i][2] = ex2(fmaf(sc[i][2], qfac1, -b1));
        sc[i][3] = ex2(fmaf(sc[i][3], qfac1, -b1));
        l0 += sc[i][0] + sc[i][1];
        l1 += sc[i][2] + sc[i][3];
      }
      if constexpr (INT8) {
        const float* vsc = reinterpret_cast<const float*>(stage + 2 * C::kTileBytes) + kTK;
#pragma unroll
        for (int i = 0; i < 2 * kNB; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(vsc + wk * kKW + 8 * i + 2 * t4);
          sc[i][0] *= f.x;
          sc[i][1] *= f.y;
          sc[i][2] *= f.x;
          sc[i][3] *= f.y;
        }
      }
      if (__any_sync(0xffffffffu, c0 != 1.f || c1 != 1.f)) {  // (rare along a long cache)
#pragma unroll
        for (int i = 0; i < kNO; ++i) {
          o[i][0] *= c0;
          o[i][1] *= c0;
          o[i][2] *= c1;
          o[i][3] *= c1;
        }
      }
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        const int key0 = wk * kKW + nb * 16;
        if constexpr (!INT8) {
          uint32_t pf[4];
          pf[0] = pack_bf16x2(sc[2 * nb][0], sc[2 * nb][1]);
          pf[1] = pack_bf16x2(sc[2 * nb][2], sc[2 * nb][3]);
          pf[2] = pack_bf16x2(sc[2 * nb + 1][0], sc[2 * nb + 1][1]);
          pf[3] = pack_bf16x2(sc[2 * nb + 1][2], sc[2 * nb + 1][3]);
          const int row = key0 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
          for (int db = 0; db < kNO / 2; ++db) {
            uint32_t vf[4];
            ldsm4t(vst + chunk_at<D, INT8>(row, 2 * db + (lane >> 4)), vf);
            mma16816<false>(o[2 * db], pf, vf[0], vf[1]);
            mma16816<false>(o[2 * db + 1], pf, vf[2], vf[3]);
          }
        } else {
          // k slot t4 (t4 + 4) of an 8-key step is key 2 t4 (2 t4 + 1), as the scores lie; a lane holds elements
          // kNO g8 .. kNO g8 + kNO - 1 of its two keys, output tile i takes element kNO g8 + i
          constexpr int kWords = kNO / 4;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float(&p)[4] = sc[2 * nb + h];
            const uint32_t pf[4] = {tf32(p[0]), tf32(p[2]), tf32(p[1]), tf32(p[3])};
            uint32_t cw[2][kWords];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = key0 + 8 * h + 2 * t4 + x;
              const uint8_t* at = stage + C::kTileBytes + chunk_at<D, INT8>(row, D == 128 ? g8 : g8 >> 1);
              if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(at);
                cw[x][0] = w.x; cw[x][1] = w.y; cw[x][2] = w.z; cw[x][3] = w.w;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(at + 8 * (g8 & 1));
                cw[x][0] = w.x; cw[x][1] = w.y;
              }
#pragma unroll
              for (int y = 0; y < kWords; ++y) cw[x][y] ^= 0x80808080u;
            }
#pragma unroll
            for (int y = 0; y < kWords; ++y) {
              mma1688(o[4 * y], pf, code_f32<0>(cw[0][y]), code_f32<0>(cw[1][y]));
              mma1688(o[4 * y + 1], pf, code_f32<1>(cw[0][y]), code_f32<1>(cw[1][y]));
              mma1688(o[4 * y + 2], pf, code_f32<2>(cw[0][y]), code_f32<2>(cw[1][y]));
              mma1688(o[4 * y + 3], pf, code_f32<3>(cw[0][y]), code_f32<3>(cw[1][y]));
            }
          }
        }
      }
    }

    if (more) keep(ahead, slot);  // this tile's entries are read

    if (cc.kt + 1 == cc.sh.kt || t + 1 == tiles) {
      // ---- the item's end, or the run's: join the warps' key slices ----
      const bool whole = kt_begin == 0 && cc.kt + 1 == cc.sh.kt;
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      __syncthreads();  // the stage is read; copies into it begin behind the next barrier of the loop
      float* mo = reinterpret_cast<float*>(stage);  // [warp][16][D]
      // element column of accumulator (i, j): j = 0, 1
      auto col = [&](int i, int j) { return INT8 ? kNO * (2 * t4 + j) + i : 8 * i + 2 * t4 + j; };
#pragma unroll
      for (int i = 0; i < kNO; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mo[(warp * 16 + g8) * D + col(i, j)] = o[i][j];
          mo[(warp * 16 + g8 + 8) * D + col(i, j)] = o[i][2 + j];
        }
      if (t4 == 0) {
        ml[warp * 16 + g8] = make_float2(m0, l0);
        ml[warp * 16 + g8 + 8] = make_float2(m1, l1);
      }
      __syncthreads();
      const long long pslot = 2ll * blockIdx.x + (kt_begin > 0 ? 0 : 1);
      for (int e = tid * 4; e < rows * D; e += kThreads * 4) {
        const int r = e / D, c = e % D;
        const int w0 = (r >> 4) * WK, rr = r & 15;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WK; ++w) M = fmaxf(M, ml[(w0 + w) * 16 + rr].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const float2 q = ml[(w0 + w) * 16 + rr];
          const float f = ex2(q.x - base);
          const float4 v = *reinterpret_cast<const float4*>(mo + ((w0 + w) * 16 + rr) * D + c);
          L += f * q.y;
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        if (whole) {
          const size_t row = out_row<kRT>(a, cc.s, cc.g, cc.rt, r);
          const float inv = L == 0.f ? 0.f : 1.f / L;
          *reinterpret_cast<uint2*>(a.out + row * D + c) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          if (a.lse && c == 0) a.lse[row] = (M + log2f(L)) * kLn2;
        } else {
          __stcg(reinterpret_cast<float4*>(a.part_o + (pslot * kRT + r) * D + c), acc);
          if (c == 0) __stcg(a.part_ml + pslot * kRT + r, make_float2(M, L));
        }
      }
      if (!whole && a.fused) {
        const Span sp = span_of(item_first, cc.sh.ku, run.per);
        if (all_arrived(a, sp, run.per, pslot)) {
          join_item<D, kRT, kThreads>(a, cc.s, sp, run.per, cc.g, cc.rt, rows, reinterpret_cast<float*>(stage), tid);
          clear_arrivals(a, sp, run.per);
        }
      }
      item_first += cc.sh.ku;
    }
    if (++cc.kt == cc.sh.kt) cc.next_item(a, run.pad);
    if (++slot == kStages) slot = 0;
  }
}

// ---- host ----

// Row tile for `rows` query rows per (sequence, kv head) on average: the block
// kernel where a warp-level tile would have to read the cache's tiles again for
// each 16 rows.  BF16, 32 rows: 2 sequences of 200,000 positions 275 us
// warp-level, 247 block; 16 of up to 4000 27 and 22; at 16 rows 250 and 246, 23
// and 22, with 64-wide heads 42 and 44.  INT8, where the block kernel has to
// convert the codes: 32 rows 335 and 537, 34 and 40; 64 rows 54 and 40.
inline int row_tile(long long rows, bool int8) { return rows <= 16 ? 16 : (int8 && rows <= 32 ? 32 : kBlockRows); }
// CTAs resident on an SM
inline int runs_per_sm(int rt) { return rt == kBlockRows ? 1 : 2; }
// The last arrival joins items of at most this many rows (on average over the
// sequences), which its threads take in one pass: no slower on the GPU (one token over 777 positions 7.7 us
// either way, 2 over 200,000 246.5 and 247.3) and a launch (2 us of the
// host's time) less.  With more rows the joining kernel is faster: 8 rows 249.4
// and 248.1 us, 16 rows of 16 sequences 27.2 and 23.3 us, 32 rows 34.1 and 26.8.
constexpr int kFusedRows = 4;

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline int max_runs(int rt) { return runs_per_sm(rt) * current_sm_count(); }
struct Workspace {
  size_t arrivals, starts, ml, o, bytes;
};
inline Workspace workspace_of(int B, int rt, int d) {
  Workspace w;
  const size_t slots = static_cast<size_t>(2) * max_runs(rt);
  w.arrivals = 0;
  w.starts = up256(slots * 8);
  w.ml = w.starts + up256((static_cast<size_t>(B) + 2) * 4);
  w.o = w.ml + up256(slots * rt * 8);
  w.bytes = w.o + up256(slots * rt * d * 4);
  return w;
}

// The call's number in the parts' marks: never the same twice in a process,
// and begun anywhere, so that a word left by anything else does not match.
inline unsigned long long next_tag() {
  static std::atomic<unsigned long long> n{[] {
    timespec ts;
    clock_gettime(CLOCK_REALTIME, &ts);
    return (static_cast<unsigned long long>(ts.tv_sec) * 1000000007ull + ts.tv_nsec) * 0x9E3779B97F4A7C15ull;
  }()};
  const unsigned long long v = n.fetch_add(1, std::memory_order_relaxed);
  return v ? v : next_tag();
}

// The launch's grid and workspace for row tiles of `rt` and key tiles of `tk`;
// false where the units pass 32 bits.
inline bool plan(Args& a, int rt, int tk, int d, uint8_t* ws, int* runs, bool* shared) {
  const Workspace w = workspace_of(a.bt.B, rt, d);
  a.arrivals = reinterpret_cast<unsigned long long*>(ws + w.arrivals);
  a.starts = reinterpret_cast<int*>(ws + w.starts);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  // most units that the batch can have: every row tile over a full block table
  const long long kt = (static_cast<long long>(a.bt.max_pages) * a.page_size + tk - 1) / tk;
  const long long items = (static_cast<long long>(a.bt.T) * a.G / rt + a.bt.B) * a.Hkv, units = items * kt;
  const int most = max_runs(rt);
  if (units > 0x7fffffffll - most) return false;
  *runs = static_cast<int>(std::min<long long>(most, units));
  *shared = kt > 1;  // items of one tile are never shared
  a.fused = rt != kBlockRows && (a.bt.T + a.bt.B - 1) / a.bt.B * a.G <= kFusedRows;
  a.tag = next_tag();
  return true;
}

template <int D, int RT, int TK>
int launch_join(const Args& a, cudaStream_t st) {
  constexpr int kRows = kJoinThreads / (D / 4);
  const dim3 grid(static_cast<unsigned>((a.bt.T * a.Hq + kRows - 1) / kRows));
  return launch_pdl(paged_join_kernel<D, RT, TK>, grid, dim3(kJoinThreads), 0, st, a) == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}

template <int D, bool INT8, int WR, int WK>
int launch(Args& a, uint8_t* ws, cudaStream_t st) {
  using C = Cfg<D, INT8, WR, WK>;
  auto kern = paged_attn_kernel<D, INT8, WR, WK>;
  static std::atomic<uint64_t> attr{0};
  uint64_t bit;
  if (attrs_needed(attr, &bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return MNW_E_CUDA;
    attrs_done(attr, bit);
  }
  int runs;
  bool shared;
  if (!plan(a, C::kRT, C::kTK, D, ws, &runs, &shared)) return MNW_E_UNSUPPORTED;
  if (launch_pdl(kern, dim3(runs), dim3(C::kThreads), C::kSmem, st, a) != cudaSuccess) return MNW_E_CUDA;
  return a.fused || !shared ? MNW_OK : launch_join<D, C::kRT, C::kTK>(a, st);
}

template <int D, bool INT8>
int launch_rows(Args& a, uint8_t* ws, int rt, cudaStream_t st) {
  if (rt == 16) return launch<D, INT8, 1, 4>(a, ws, st);
  if constexpr (INT8) {
    if (rt == 32) return launch<D, INT8, 2, 2>(a, ws, st);
  }
  int runs;
  bool shared;
  if (!plan(a, kBlockRows, kBlockKeys, D, ws, &runs, &shared)) return MNW_E_UNSUPPORTED;
  const int rc = launch_block(a, D, INT8, runs, st);
  return rc != MNW_OK || !shared ? rc : launch_join<D, kBlockRows, kBlockKeys>(a, st);
}

}  // namespace pattn
}  // namespace mnw

using namespace mnw;

extern "C" {

size_t mnw_attn_paged_workspace_size(int B, int T, int Hq, int Hkv, int d) {
  if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv) return 0;
  const long long rows = (static_cast<long long>(T) + B - 1) / B * (Hq / Hkv);
  return std::max(pattn::workspace_of(B, pattn::row_tile(rows, false), d).bytes,
                  pattn::workspace_of(B, pattn::row_tile(rows, true), d).bytes);
}

int mnw_attn_paged(const void* q, long long q_stride, int B, int T, int Hq, int Hkv, int d, const void* k_cache,
                   const void* v_cache, const float* k_scale, const float* v_scale, int fmt, int n_pages,
                   int page_size, long long page_stride, const int32_t* block_table, int max_pages,
                   const int32_t* cache_lens, const int32_t* q_start, int blk, float scale, void* out, float* lse,
                   void* ws, size_t ws_bytes, uint32_t* err, mnw_stream stream) {
  MNW_RANGE("mnw_attn_paged");
  using namespace pattn;
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || blk < 1) return MNW_E_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < 3.0e38f)) return MNW_E_INVALID_ARG;
  if (B == 0 || T == 0) return T == 0 ? MNW_OK : MNW_E_INVALID_ARG;
  int rc = paged::check_cache(k_cache, v_cache, k_scale, v_scale, fmt, n_pages, page_size, Hkv, d, page_stride);
  if (rc != MNW_OK) return rc;
  rc = paged::check_batch(block_table, cache_lens, q_start, B, T, max_pages, page_size);
  if (rc != MNW_OK) return rc;
  if (!q || !out || !ws || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 256) ||
      q_stride % 8 || q_stride < static_cast<long long>(Hq) * d)
    return MNW_E_INVALID_ARG;
  if (static_cast<long long>(T) * Hq > 0x7fffffffll / 8) return MNW_E_UNSUPPORTED;
  if (ws_bytes < mnw_attn_paged_workspace_size(B, T, Hq, Hkv, d)) return MNW_E_WORKSPACE_TOO_SMALL;
  Args a{};
  a.bt = paged::Batch{block_table, cache_lens, q_start, B, T, max_pages, q_start ? 0 : T / B};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = k_scale;
  a.vs = v_scale;
  const bool int8 = fmt == MNW_KV_INT8;
  a.page_bytes = page_stride * (int8 ? 1 : 2);
  a.page_div = paged::fast_div(page_size);
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.g_div = paged::fast_div(a.G);
  a.blk = blk;
  a.blk_div = paged::fast_div(blk);
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = err;
  const int rt = row_tile((static_cast<long long>(T) + B - 1) / B * a.G, int8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto* w = static_cast<uint8_t*>(ws);
  if (d == 128) return int8 ? launch_rows<128, true>(a, w, rt, st) : launch_rows<128, false>(a, w, rt, st);
  return int8 ? launch_rows<64, true>(a, w, rt, st) : launch_rows<64, false>(a, w, rt, st);
}

}  // extern "C"
