// mnw_attn_paged_int4.cu -- attention of new tokens over a paged cache held in
// 4 bits.  Formulas: mnw_attn_paged.cu; the cached rows: mnw_int4_row.cuh; the
// work's split and the joining of its parts: mnw_attn_split.cuh.
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with the
// cache as the left operand: a code is converted once for all query rows of a
// warp, and 8 query rows (the few that a single token has) fill an instruction
// whose other form takes 16.  S^T comes out with keys in the accumulator's
// rows; P^T goes in with keys along k, which is that tile transposed
// (movmatrix).
//
// A CTA is four warps, each with 32 keys of a tile of 128 and all 8 NT query
// rows.  Tiles arrive by cp.async through a ring, one page lookup a key, so
// pages of any size may end inside a tile; rows past the length are zeros.
//
// Operands are FP16 and exact but for the probabilities: codes times the
// group's multiplier (as multiples of 2^-24), q as FP16 times a power of two a
// row; the keys' scales multiply the FP32 scores.  A probability times its
// value's scale is rounded to FP16 (2^-11 relative) relative to the row's
// largest such product so far, lifted by 2^6, so one 2^-30 of the largest is
// still held.  Maximum and unit of a row move only when a score passes them by
// more than 2^8, so that most tiles need no reduction over the warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mnw_attn_split.cuh"
#include "mnw_int4_row.cuh"

namespace mnw {
namespace pattn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kTK = kInt4Keys;
constexpr int kStages = 3;
constexpr float kLow = -1e30f;   // a maximum of nothing: finite, so that -inf minus it is -inf
constexpr float kStep = 8.f;     // log2 by which scores may pass a row's maximum and unit
constexpr float kHalfUnit = 4096.f;  // the operands' 2^-24 is taken back half with the keys' scales, half with the queries' factors
constexpr float kLift = 6.f;     // log2: the largest FP16 value is 2^(kStep + kLift) = 2^14

template <int D, int NT>
struct Cfg4 {
  static constexpr int kRT = 8 * NT;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kTileBytes = kTK * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kTK * int4row::kRecord;
  static constexpr int kQBytes = NT > 2 ? (D / 16) * NT * 32 * 8 : 0;  // query fragments, where registers cannot hold them
  static constexpr int kSmem = kStages * kStageBytes + kQBytes;
  static constexpr int kPad = D + 4;  // of a row where the warps' outputs meet, in the stage just read
  static_assert(kWarps * 8 * kPad * 4 <= kStageBytes);
  static_assert(kThreads / (D / 4) * 2 * kJoinBatch * 4 <= kStageBytes);
};

// Values lie with neighbouring keys' rows apart, so that the lanes of a load (keys 2 t, pieces g of a row) fall into
// different banks.
template <int D>
__device__ __forceinline__ uint32_t v_at(int r, int byte) {
  if constexpr (D == 128) {
    const int p = r ^ ((r >> 1) & 1);
    return static_cast<uint32_t>(p * 64 + (byte ^ ((p & 4) << 3)));
  } else {
    return static_cast<uint32_t>((r ^ ((r >> 2) & 1)) * 32 + byte);
  }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, int4_runs_per_sm(8 * NT)) paged_int4_kernel(const Args a) {
  using C = Cfg4<D, NT>;
  constexpr int kRT = C::kRT;
  constexpr int kKS = D / 16;   // k steps of the first product
  constexpr int kNO = D / 16;   // row tiles of the second
  constexpr int kMT = kTK / kWarps / 16;  // 16-key tiles of a warp
  constexpr int kW = D / 64;    // words of a lane's piece of a value row; half of those of a key's
  constexpr bool kQRegs = NT <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SplitShared split;
  __shared__ float2 ml[kWarps][kRT];
  __shared__ long long row_at[kStages][kTK];  // byte offset of a tile's keys' cached rows, -1: none
  __shared__ long long rec_at[kStages][kTK];  // and of their records
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  uint2* const qs = reinterpret_cast<uint2*>(smem + kStages * C::kStageBytes);  // [k step][n tile][lane]

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
    if (p < lc.s.len) {
      const int pi = static_cast<int>(paged::quotient(p, a.page_div));
      at.x = __ldg(a.bt.block_table + static_cast<size_t>(lc.b) * a.bt.max_pages + pi);
      at.y = lc.g * a.page_size + (p - pi * a.page_size);
    }
    if (++lc.kt == lc.sh.kt) lc.next_item(a, run.pad);
  };
  auto keep = [&](int2 at, int slot) {
    bool has = at.y >= 0;
    if (has && static_cast<unsigned>(at.x) >= static_cast<unsigned>(a.n_pages)) {
      has = false;
      if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
    }
    row_at[slot][tid] = has ? at.x * a.page_bytes + static_cast<long long>(at.y) * C::kRowBytes : -1;
    rec_at[slot][tid] = (static_cast<long long>(at.x) * a.Hkv * a.page_size + at.y) * int4row::kRecord;
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
      cp_async16(st + r * C::kRowBytes + c * 16, a.kc + off, n);
      cp_async16(st + C::kTileBytes + v_at<D>(r, c * 16), a.vc + off, n);
    }
    const uint32_t n = row_at[slot][tid] >= 0 ? 8u : 0u;
    const long long off = n ? rec_at[slot][tid] : 0;
    const uint32_t to = st + 2 * C::kTileBytes + tid * int4row::kRecord;
    cp_async8(to, reinterpret_cast<const char*>(a.ks) + off, n);
    cp_async8(to + kTK * int4row::kRecord, reinterpret_cast<const char*>(a.vs) + off, n);
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

  // ---- state of the item in hand; of rows 8 nt + 2 t4 + x ----
  uint32_t qf[kQRegs ? kKS : 1][kQRegs ? NT : 1][2];
  float qfac[NT][2];                      // score factor
  float m[NT][2], l[NT][2], unit[NT][2];  // log2 of the weights' reference, sum, log2 of the products' reference
  float lift[NT][2];
  int lim[NT][2];                         // first key that is not seen
  float o[kNO][NT][4];
  int rows = 0, lim_lo = 0, lim_hi = 0, kt_begin = 0;
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
#pragma unroll
    for (int i = 0; i < kNO; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * nt + 2 * t4 + x;
        lim[nt][x] = r < rows ? row_limit(a, cc.s, ri + r) : lim_hi;
        m[nt][x] = unit[nt][x] = kLow;
        l[nt][x] = 0.f;
        lift[nt][x] = 0.f;
      }
      // Row 8 nt + g8 as the right operand: k step s takes elements (D / 4) t4 + 4 s .. + 3 of lane t4, the order in
      // which a lane's words of codes hold them.
      const int r = 8 * nt + g8, rr = ri + (r < rows ? r : 0);
      const int tok = static_cast<int>(paged::quotient(rr, a.g_div)), hh = rr - tok * a.G;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(cc.s.start + tok) * a.q_stride +
                                                        static_cast<long long>(cc.g * a.G + hh) * D + (D / 4) * t4);
      uint4 w[D / 32];
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        w[i] = r < rows ? src[i] : make_uint4(0, 0, 0, 0);
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu), __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
      }
      uint32_t top = max(big >> 16, big & 0xFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = row_exponent(top);
      const float f = two_to(-e);
      auto half = [&](uint32_t y) { return half2_of(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xFFFF0000u) * f); };
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t h[4] = {half(w[i].x), half(w[i].y), half(w[i].z), half(w[i].w)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (kQRegs) {
            qf[2 * i + j][nt][0] = h[2 * j];
            qf[2 * i + j][nt][1] = h[2 * j + 1];
          } else {
            if (warp == nt % kWarps) qs[((2 * i + j) * NT + nt) * 32 + lane] = make_uint2(h[2 * j], h[2 * j + 1]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        qfac[nt][x] = a.scale_log2 * kHalfUnit * two_to(__shfl_sync(0xffffffffu, e, 4 * (2 * t4 + x)));
    }
    if constexpr (!kQRegs) __syncthreads();
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
    uint8_t* stage = smem + slot * C::kStageBytes;

    if (cc.kt * kTK < lim_hi) {  // a tile past every row's limit adds nothing
      const uint8_t *krec = stage + 2 * C::kTileBytes, *vrec = krec + kTK * int4row::kRecord;
      const int k0 = warp * (kTK / kWarps);  // the warp's first key of the tile
      // ---- scores: keys 16 mt + g8 (+ 8) in rows, query rows 8 nt + 2 t4 (+ 1) in columns ----
      float sc[kMT][NT][4];
      {
        uint32_t kw[kMT][2][2 * kW];
        int4row::Mul km[kMT][2];
        float ks[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = k0 + 16 * mt + 8 * h + g8;
            const uint8_t* at = stage + key * C::kRowBytes + t4 * (D / 8);
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(at);
              kw[mt][h][0] = w.x; kw[mt][h][1] = w.y; kw[mt][h][2] = w.z; kw[mt][h][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(at);
              kw[mt][h][0] = w.x; kw[mt][h][1] = w.y;
            }
            const uint2 rec = *reinterpret_cast<const uint2*>(krec + key * int4row::kRecord);
            ks[mt][h] = __uint_as_float(rec.x) * kHalfUnit;
            km[mt][h] = int4row::multipliers(prmt(rec.y, 0u, t4 * 0x101u));  // the lane's codes are of group t4
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2 * kW; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int s = 2 * i + j;
            uint32_t ka[kMT][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                ka[mt][h] = j ? int4row::pair<2>(kw[mt][h][i], km[mt][h]) : int4row::pair<0>(kw[mt][h][i], km[mt][h]);
                ka[mt][2 + h] = j ? int4row::pair<3>(kw[mt][h][i], km[mt][h]) : int4row::pair<1>(kw[mt][h][i], km[mt][h]);
              }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 b;
              if constexpr (kQRegs)
                b = make_uint2(qf[s][nt][0], qf[s][nt][1]);
              else
                b = qs[(s * NT + nt) * 32 + lane];
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt) mma_f16(sc[mt][nt], ka[mt][0], ka[mt][1], ka[mt][2], ka[mt][3], b.x, b.y);
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] *= ks[mt][e >> 1] * qfac[nt][e & 1];
      }
      if ((cc.kt + 1) * kTK > lim_lo) {  // some row's limit lies in this tile
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cc.kt * kTK + k0 + 16 * mt + 8 * (e >> 1) + g8 >= lim[nt][e & 1]) sc[mt][nt][e] = -INFINITY;
      }
      // ---- maximum and unit, where a score passes them ----
      float vs[kMT][2], lv[kMT][2];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          vs[mt][h] = *reinterpret_cast<const float*>(vrec + (k0 + 16 * mt + 8 * h + g8) * int4row::kRecord);
          lv[mt][h] = __log2f(fabsf(vs[mt][h]));
        }
      bool over = false;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            over = over || sc[mt][nt][e] > m[nt][e & 1] + kStep || sc[mt][nt][e] + lv[mt][e >> 1] > unit[nt][e & 1] + kStep;
      if (__any_sync(0xffffffffu, over)) {
        float alpha[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = kLow, topv = kLow;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                top = fmaxf(top, sc[mt][nt][2 * h + x]);
                topv = fmaxf(topv, sc[mt][nt][2 * h + x] + lv[mt][h]);
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
            }
            const float n = fmaxf(m[nt][x], top);
            // held within 2^100 of the maximum so that the lift stays finite
            const float u = fmaxf(fmaxf(unit[nt][x], topv), n - 100.f);
            l[nt][x] *= ex2(m[nt][x] - n);
            alpha[nt][x] = ex2(unit[nt][x] - u);
            lift[nt][x] = ex2(n - u + kLift);
            m[nt][x] = n;
            unit[nt][x] = u;
          }
#pragma unroll
        for (int i = 0; i < kNO; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][nt][e] *= alpha[nt][e & 1];
      }
      // ---- probabilities, and the second product, 16 keys at a time ----
      const uint32_t vsel = static_cast<uint32_t>(g8 >> 1) * 0x101u + 0x400u;  // the lane's elements are of group g8 / 2
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(sc[mt][nt][e] - m[nt][e & 1]);
            l[nt][e & 1] += p[e];
            p[e] *= vs[mt][e >> 1] * lift[nt][e & 1];
          }
          pb[nt][0] = transposed(half2_of(p[0], p[1]));
          pb[nt][1] = transposed(half2_of(p[2], p[3]));
        }
        // keys 2 t4, 2 t4 + 1 (h = 0) and 8 further (h = 1), in the halves of a register
        uint32_t vl[2][kW], vh[2][kW];  // even and odd elements of the lane's words
        int4row::Mul vm[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = k0 + 16 * mt + 8 * h + 2 * t4;
          uint32_t w0[kW], w1[kW];
          const uint8_t *at0 = stage + C::kTileBytes + v_at<D>(key, g8 * (D / 16)), *at1 = stage + C::kTileBytes + v_at<D>(key + 1, g8 * (D / 16));
          if constexpr (D == 128) {
            const uint2 y0 = *reinterpret_cast<const uint2*>(at0), y1 = *reinterpret_cast<const uint2*>(at1);
            w0[0] = y0.x; w0[1] = y0.y;
            w1[0] = y1.x; w1[1] = y1.y;
          } else {
            w0[0] = *reinterpret_cast<const uint32_t*>(at0);
            w1[0] = *reinterpret_cast<const uint32_t*>(at1);
          }
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            vl[h][i] = prmt(w0[i], w1[i], 0x5410u);
            vh[h][i] = prmt(w0[i], w1[i], 0x7632u);
          }
          const uint32_t m0 = *reinterpret_cast<const uint32_t*>(vrec + key * int4row::kRecord + 4);
          const uint32_t m1 = *reinterpret_cast<const uint32_t*>(vrec + (key + 1) * int4row::kRecord + 4);
          vm[h] = int4row::multipliers(prmt(m0, m1, vsel));
        }
        auto tile = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[i][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        };
        using int4row::pair;
#pragma unroll
        for (int i = 0; i < kW; ++i) {  // row tile 4 i + j: elements 8 i + 2 j (rows g8) and 8 i + 2 j + 1 (rows g8 + 8)
          tile(4 * i, pair<0>(vl[0][i], vm[0]), pair<0>(vh[0][i], vm[0]), pair<0>(vl[1][i], vm[1]), pair<0>(vh[1][i], vm[1]));
          tile(4 * i + 1, pair<1>(vl[0][i], vm[0]), pair<1>(vh[0][i], vm[0]), pair<1>(vl[1][i], vm[1]), pair<1>(vh[1][i], vm[1]));
          tile(4 * i + 2, pair<2>(vl[0][i], vm[0]), pair<2>(vh[0][i], vm[0]), pair<2>(vl[1][i], vm[1]), pair<2>(vh[1][i], vm[1]));
          tile(4 * i + 3, pair<3>(vl[0][i], vm[0]), pair<3>(vh[0][i], vm[0]), pair<3>(vl[1][i], vm[1]), pair<3>(vh[1][i], vm[1]));
        }
      }
    }

    if (more) keep(ahead, slot);  // this tile's entries are read

    if (cc.kt + 1 == cc.sh.kt || t + 1 == tiles) {
      // ---- the item's end, or the run's: join the warps' key slices, 8 rows at a time ----
      const bool whole = kt_begin == 0 && cc.kt + 1 == cc.sh.kt;
      const long long pslot = 2ll * blockIdx.x + (kt_begin > 0 ? 0 : 1);
      float* mo = reinterpret_cast<float*>(stage);  // [warp][8][kPad]
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float fac[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum = l[nt][x];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          // sums relative to the maximum again
          fac[x] = ex2(unit[nt][x] - m[nt][x] - kLift) * int4row::kUnit;
          if (g8 == 0) ml[warp][8 * nt + 2 * t4 + x] = make_float2(m[nt][x] == kLow ? -INFINITY : m[nt][x], sum);
        }
        __syncthreads();  // the stage is read (copies into it begin behind the next barrier of the loop), or the rows before are
#pragma unroll
        for (int i = 0; i < kNO; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *reinterpret_cast<float2*>(mo + (warp * 8 + 2 * t4 + x) * C::kPad + (D / 8) * g8 + 2 * i) =
                make_float2(o[i][nt][x] * fac[x], o[i][nt][2 + x] * fac[x]);
        __syncthreads();
        const int here = min(8, rows - 8 * nt);
        for (int e = tid * 4; e < here * D; e += kThreads * 4) {
          const int rr = e / D, c = e % D, r = 8 * nt + rr;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][r].x);
          const float base = M == -INFINITY ? 0.f : M;
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 q = ml[w][r];
            const float f = ex2(q.x - base);
            const float4 v = *reinterpret_cast<const float4*>(mo + (w * 8 + rr) * C::kPad + c);
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

template <int D, int NT>
int launch(const Args& a, int runs, cudaStream_t st) {
  using C = Cfg4<D, NT>;
  auto kern = paged_int4_kernel<D, NT>;
  static std::atomic<uint64_t> attr{0};
  uint64_t bit;
  if (attrs_needed(attr, &bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return MNW_E_CUDA;
    attrs_done(attr, bit);
  }
  return launch_pdl(kern, dim3(runs), dim3(kThreads), C::kSmem, st, a) == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}
template <int D>
int launch_rt(const Args& a, int rt, int runs, cudaStream_t st) {
  return rt == 8 ? launch<D, 1>(a, runs, st) : (rt == 16 ? launch<D, 2>(a, runs, st) : launch<D, 4>(a, runs, st));
}

}  // namespace

int launch_int4(const Args& a, int d, int rt, int runs, cudaStream_t st) {
  return d == 128 ? launch_rt<128>(a, rt, runs, st) : launch_rt<64>(a, rt, runs, st);
}

}  // namespace pattn
}  // namespace mnw
