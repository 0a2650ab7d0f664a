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
// A CTA is four warps, each with 64 keys of a tile of 256 and all 8 NT query
// rows.  The warps meet only at an item's end: each loads its own keys through
// a ring of its own, as bulk copies (a lane per page, waited for on a barrier
// of the ring's slot) where its keys lie inside the length in whole pieces of
// pages, and else by 16-byte cp.async with a page lookup per key, so pages of
// any size may end inside a tile; rows past the length are zeros.
//
// Bound: one pass over the cache, 144 bytes a position and kv head (d = 128).
// Measured on one GB300: 2 single tokens over 200,000 positions, 32 query and 8
// key heads of 128 (461 MB): 105 us, 4.4 TB/s; 32 over 2048 to 8192 positions in
// pages of 16, 16 and 4 heads (95 MB): 33 us; one over 777: 8.4 us.  Latency
// bounds it: 16 keys take about 360 instructions, 160 of them the conversion
// (mask, and product with the multiplier, two codes each), and 12 warps an SM of
// 167 registers each issue 2.0 a clock, half of what it could (50 % of the slots;
// memory 38 %, tensor pipe 18 %).  With all slots the same instructions would
// take some 53 us, less than the bytes' 68.  A CTA's warps meeting at every tile,
// with 16-byte copies by all threads, took 123 us; two CTAs with more registers
// for a wider group of keys 110 to 115.
//
// Operands are FP16 and exact but for the probabilities: codes times the
// group's multiplier (as multiples of 2^-24), q as FP16 times a power of two a
// row; the keys' scales multiply the FP32 scores.  A probability times its
// value's scale is rounded to FP16 (2^-11 relative) relative to the row's
// largest such product so far, lifted by 2^6, so one 2^-30 of the largest is
// still held.  Maximum and unit of a row move only when a probability passes
// 2^8 or a product 2^14; that is looked for in what was computed, and the tile's
// probabilities are then computed again, so most tiles need no reduction over
// the warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "mnw_attn_split.cuh"
#include "mnw_int4_row.cuh"

namespace mnw {
namespace pattn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kTK = kInt4Keys;
constexpr int kWK = kTK / kWarps;  // keys of a warp
constexpr float kLow = -3e38f;   // a maximum of nothing: finite, so that -inf minus it is -inf
constexpr float kLift = 6.f;     // log2 of the unit's own product as FP16
constexpr float kMostP = 256.f, kMostW = 16384.f;  // probabilities and products that a row's maximum and unit allow

template <int D, int NT>
struct Cfg4 {
  static constexpr int kRT = 8 * NT;
  // 16-key operand tiles computed together, and such groups: one where 32 rows' sums leave registers for no more
  static constexpr int kMT = NT <= 2 ? 2 : 1, kSubs = kWK / (16 * kMT);
  static constexpr int kStages = NT == 2 ? 3 : 2;  // what the CTAs of an SM have room for
  static constexpr int kRowBytes = D / 2;
  static constexpr int kTileBytes = kWK * kRowBytes, kRecBytes = kWK * int4row::kRecord;  // of a warp's keys
  static constexpr int kSlotBytes = 2 * (kTileBytes + kRecBytes);  // keys, values, their records
  static constexpr int kQBytes = NT > 2 ? (D / 16) * NT * 32 * 8 : 0;  // query fragments, where registers cannot hold them
  static constexpr int kSmem = kWarps * kStages * kSlotBytes + kQBytes;
  static constexpr int kPad = D + 4;  // floats of a row where the warps' outputs meet, in the slots just read
  static_assert(8 * kPad * 4 <= kSlotBytes && kThreads / (D / 4) * 2 * kJoinBatch * 4 <= kSlotBytes);
};

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
// Two FP32 values in a 64-bit register.
__device__ __forceinline__ uint64_t two(float lo, float hi) { return f32x2_pack(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float lo32(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi32(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }

// The largest of magnitudes; NaN where one is.
__device__ __forceinline__ float most_nan(float most, float a, float b) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(most), "f"(a), "f"(b));
  return y;
}

// Row i of a warp's 16-key operand tiles is key i ^ (i / 2 % 2): the keys that a load's lanes read then lie in rows of
// both parities, whose 64 bytes are the two halves of the banks.
__device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 1) & 1); }

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, int4_runs_per_sm(8 * NT)) paged_int4_kernel(const Args a, const int whole_pages) {
  using C = Cfg4<D, NT>;
  constexpr int kRT = C::kRT, kMT = C::kMT, kSubs = C::kSubs, kStages = C::kStages;
  constexpr int kKS = D / 16;   // k steps of the first product
  constexpr int kNO = D / 16;   // row tiles of the second
  constexpr int kW = D / 64;    // words of a lane's piece of a value row; half of those of a key's
  constexpr bool kQRegs = NT <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SplitShared split;
  __shared__ float2 ml[kWarps][kRT];
  __shared__ uint64_t full[kWarps][kStages];  // a slot's bulk copies have landed
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint8_t* const mine = smem + warp * (kStages * C::kSlotBytes);  // the warp's ring
  uint2* const qs = reinterpret_cast<uint2*>(smem + kWarps * kStages * C::kSlotBytes);  // [k step][n tile][lane]

  pdl_launch_dependents();
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&full[w][i], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();

  const Run run = find_run<kRT, kTK, kThreads, 0>(a, &split);  // (with barriers, behind which full[] is set up)
  if (run.seq < 0) return;  // no units left for this run
  Cursor<kRT, kTK> cc;  // the tile computed
  cc.set(a, run);
  int item_first = run.u0 - cc.kt;  // first unit of its item
  const int tiles = run.pad == 1 ? run.u1 - run.u0 : min(run.u1 - run.u0, cc.sh.kt - cc.kt);
  if (tiles <= 0) return;

  // ---- loads of the warp's keys: whole pieces of pages are looked up a tile before they are copied ----
  Cursor<kRT, kTK> lc = cc;  // the tile looked up next
  const int span = min(a.page_size, kWK);  // keys of a piece
  auto row_of = [&](int p, int& entry, int& row) {  // page table entry of position p, and its row in the page
    const int pi = static_cast<int>(paged::quotient(p, a.page_div));
    entry = __ldg(a.bt.block_table + static_cast<size_t>(lc.b) * a.bt.max_pages + pi);
    row = lc.g * a.page_size + (p - pi * a.page_size);
  };
  int entry = 0, row = 0;  // of lane i's piece
  bool bulk;
  auto look = [&]() {
    const int p0 = lc.kt * kTK + warp * kWK;
    bulk = whole_pages && p0 + kWK <= lc.s.len;
    if (bulk && lane * span < kWK) row_of(p0 + lane * span, entry, row);
  };
  uint32_t phases = 0, bulks = 0;  // per slot: parity of its barrier's next phase; whether bulk copies are under way to it
  bool gave_up = false;            // a wait ran out: reported, and the result is void
  auto fill = [&](int slot) {  // what look() found, into a slot that the whole warp has read; then on to the next tile
    uint8_t* to = mine + slot * C::kSlotBytes;
    const bool piece = lane * span < kWK;
    if (bulk && !__any_sync(0xffffffffu, piece && static_cast<unsigned>(entry) >= static_cast<unsigned>(a.n_pages))) {
      bulks |= 1u << slot;
      uint64_t* bar = &full[warp][slot];
      if (lane == 0) mbar_arrive_expect_tx(bar, C::kSlotBytes);
      __syncwarp();
      if (piece) {
        const long long at = entry * a.page_bytes + static_cast<long long>(row) * C::kRowBytes;
        const long long rec = (static_cast<long long>(entry) * (a.Hkv * a.page_size) + row) * int4row::kRecord;
        const uint32_t nrow = span * C::kRowBytes, nrec = span * int4row::kRecord;
        bulk_load(to + lane * nrow, a.kc + at, nrow, bar);
        bulk_load(to + C::kTileBytes + lane * nrow, a.vc + at, nrow, bar);
        bulk_load(to + 2 * C::kTileBytes + lane * nrec, reinterpret_cast<const uint8_t*>(a.ks) + rec, nrec, bar);
        bulk_load(to + 2 * C::kTileBytes + C::kRecBytes + lane * nrec, reinterpret_cast<const uint8_t*>(a.vs) + rec, nrec, bar);
      }
    } else {
      constexpr int kCh = C::kRowBytes / 16, kRows = 32 / kCh;
      const int c = lane % kCh;
      const uint32_t st = smem_u32(to);
#pragma unroll 1
      for (int k0 = 0; k0 < kWK; k0 += 32) {  // a key a lane
        const int p = lc.kt * kTK + warp * kWK + k0 + lane;
        int e = -1, r = 0;
        if (p < lc.s.len) {
          row_of(p, e, r);
          if (static_cast<unsigned>(e) >= static_cast<unsigned>(a.n_pages)) {
            e = -1;
            if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
          }
        }
        const bool has = e >= 0;
        const long long at = has ? e * a.page_bytes + static_cast<long long>(r) * C::kRowBytes : -1;
#pragma unroll 1
        for (int i = 0; i < 32 / kRows; ++i) {
          const int key = i * kRows + lane / kCh;
          const long long from = __shfl_sync(0xffffffffu, at, key);
          const uint32_t n = from >= 0 ? 16u : 0u, dst = st + (k0 + key) * C::kRowBytes + c * 16;
          const long long off = n ? from + c * 16 : 0;
          cp_async16(dst, a.kc + off, n);
          cp_async16(dst + C::kTileBytes, a.vc + off, n);
        }
        const long long rec = has ? (static_cast<long long>(e) * (a.Hkv * a.page_size) + r) * int4row::kRecord : 0;
        const uint32_t dst = st + 2 * C::kTileBytes + (k0 + lane) * int4row::kRecord;
        cp_async8(dst, reinterpret_cast<const uint8_t*>(a.ks) + rec, has ? 8u : 0u);
        cp_async8(dst + C::kRecBytes, reinterpret_cast<const uint8_t*>(a.vs) + rec, has ? 8u : 0u);
      }
    }
    cp_commit();
    if (++lc.kt == lc.sh.kt) lc.next_item(a, run.pad);
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) {
    if (i < tiles) {
      look();
      fill(i);
    } else {
      cp_commit();
    }
  }

  // ---- state of the item in hand; of rows 8 nt + 2 t4 and + 1, packed ----
  uint32_t qf[kQRegs ? kKS : 1][kQRegs ? NT : 1][2];
  uint64_t qfac[NT];                    // score factors
  uint64_t neg[NT], sum[NT], lift[NT];  // minus the maximum (log2), sum, 2^(maximum - unit + kLift)
  float unit[NT][2];                    // log2 of the products' reference, from the maximum
  int lim[NT][2];                       // first key that is not seen
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
        unit[nt][x] = 0.f;
      }
      neg[nt] = two(-kLow, -kLow);
      sum[nt] = lift[nt] = 0ull;
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
      const float f0 = two_to(__shfl_sync(0xffffffffu, e, 4 * (2 * t4))), f1 = two_to(__shfl_sync(0xffffffffu, e, 4 * (2 * t4 + 1)));
      qfac[nt] = two(a.scale_log2 * kHalfUnit * f0, a.scale_log2 * kHalfUnit * f1);
    }
    if constexpr (!kQRegs) __syncthreads();
  };

  const uint64_t one2 = ones(a);
  // byte offsets of what a lane reads: keys' and values' rows and records
  const int k_row = key_of(g8) * C::kRowBytes + t4 * (D / 8), k_rec = key_of(g8) * int4row::kRecord;
  const int v_key0 = key_of(2 * t4), v_key1 = key_of(2 * t4 + 1);
  const uint32_t ksel = t4 * 0x101u;                      // the lane's codes of a key are of group t4,
  const uint32_t vsel = (g8 >> 1) * 0x101u + 0x400u;      // its elements of a value of group g8 / 2

#pragma unroll 1
  for (int t = 0, slot = 0; t < tiles; ++t) {
    const bool more = t + kStages < tiles;
    if (more) look();
    if (t == 0 || cc.kt == 0) begin_item();
    cp_wait<kStages - 1>();
    const bool by_rows = !(bulks >> slot & 1);
    if (!by_rows && !gave_up) {
      bool there = mbar_try_wait(&full[warp][slot], phases >> slot & 1);
      if (!there) there = polled_wait(&full[warp][slot], phases >> slot & 1, &abort_flag, a.err);
      gave_up = !__all_sync(0xffffffffu, there);
      if (!gave_up) {
        phases ^= 1u << slot;
        bulks ^= 1u << slot;
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int sub = 0; sub < kSubs; ++sub) {
      const int p0 = cc.kt * kTK + warp * kWK + sub * (16 * kMT);  // the first position
      if (p0 >= lim_hi) break;                                     // keys past every row's limit add nothing
      const uint8_t* const st = mine + slot * C::kSlotBytes + sub * (16 * kMT) * C::kRowBytes;
      const uint8_t* const krec = mine + slot * C::kSlotBytes + 2 * C::kTileBytes + sub * (16 * kMT) * int4row::kRecord;
      const uint8_t* const vrec = krec + C::kRecBytes;
      // ---- scores: keys 16 mt + 8 h + g8 in rows, query rows 8 nt + 2 t4 (+ 1) in columns ----
      float sc[kMT][NT][4];
      uint64_t fac[kMT][NT][2];
      {
        uint32_t kw[kMT][2][2 * kW];
        int4row::Mul km[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* at = st + k_row + (16 * mt + 8 * h) * C::kRowBytes;
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(at);
              kw[mt][h][0] = w.x; kw[mt][h][1] = w.y; kw[mt][h][2] = w.z; kw[mt][h][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(at);
              kw[mt][h][0] = w.x; kw[mt][h][1] = w.y;
            }
            const uint2 rec = *reinterpret_cast<const uint2*>(krec + k_rec + (16 * mt + 8 * h) * int4row::kRecord);
            const float ks = __uint_as_float(rec.x) * kHalfUnit;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) fac[mt][nt][h] = two(ks * lo32(qfac[nt]), ks * hi32(qfac[nt]));
            km[mt][h] = int4row::multipliers(prmt(rec.y, 0u, ksel));
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
      }
      if (p0 + 16 * kMT > lim_lo) {  // some row's limit lies among these keys
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int p = p0 + 16 * mt + 8 * h + key_of(g8);
              sc[mt][nt][2 * h] = p >= lim[nt][0] ? -INFINITY : sc[mt][nt][2 * h] * lo32(fac[mt][nt][h]);
              sc[mt][nt][2 * h + 1] = p >= lim[nt][1] ? -INFINITY : sc[mt][nt][2 * h + 1] * hi32(fac[mt][nt][h]);
              fac[mt][nt][h] = two(1.f, 1.f);
            }
          }
      }
      // ---- probabilities, and their products with the values' scales as FP16 ----
      float vs[kMT][2];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) vs[mt][h] = *reinterpret_cast<const float*>(vrec + k_rec + (16 * mt + 8 * h) * int4row::kRecord);
      uint32_t pw[kMT][NT][2];
      uint64_t now[NT];
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        float most_p = 0.f, most_w = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          now[nt] = sum[nt];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // the score is rounded before the maximum goes off, as it was for the maximum: of huge ones a fused product
              // would leave its rounding
              const uint64_t s2 = f32x2_mul(two(sc[mt][nt][2 * h], sc[mt][nt][2 * h + 1]), fac[mt][nt][h]);
              const uint64_t e2 = f32x2_fma(s2, one2, neg[nt]);
              const uint64_t p2 = two(ex2(lo32(e2)), ex2(hi32(e2)));
              now[nt] = f32x2_add(now[nt], p2);
              const uint64_t w2 = f32x2_mul(p2, two(vs[mt][h] * lo32(lift[nt]), vs[mt][h] * hi32(lift[nt])));
              most_p = fmaxf(fmaxf(most_p, lo32(p2)), hi32(p2));
              most_w = most_nan(most_w, lo32(w2), hi32(w2));
              pw[mt][nt][h] = half2_of(lo32(w2), hi32(w2));
            }
        }
        if (!__any_sync(0xffffffffu, most_p > kMostP || !(most_w <= kMostW))) break;
        // a value that is not finite counts nothing (0 * NaN would, in rows that do not see it) and makes the rows that see it
        // NaN by what they hold
        int odd = INT_MAX;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (!(fabsf(vs[mt][h]) < INFINITY)) {
              odd = min(odd, p0 + 16 * mt + 8 * h + key_of(g8));
              vs[mt][h] = 0.f;
            }
        odd = __reduce_min_sync(0xffffffffu, odd);
        float alpha[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[2], n[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = kLow, topv = kLow;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                sc[mt][nt][2 * h + x] = __fmul_rn(sc[mt][nt][2 * h + x], x ? hi32(fac[mt][nt][h]) : lo32(fac[mt][nt][h]));
                top = fmaxf(top, sc[mt][nt][2 * h + x]);
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m = x ? -hi32(neg[nt]) : -lo32(neg[nt]);
            n[x] = fmaxf(m, top);
            // relative to the maximum: next to a huge score the logarithm of a value's scale would be lost
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                topv = fmaxf(topv, sc[mt][nt][2 * h + x] - n[x] + __log2f(fabsf(vs[mt][h])));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
            // held within 2^100 of the maximum so that the lift stays finite
            const float now_at = unit[nt][x] + (m - n[x]), u = fmaxf(fmaxf(now_at, topv), -100.f);
            c[x] = ex2(m - n[x]);
            alpha[nt][x] = odd < lim[nt][x] ? __uint_as_float(0x7FC00000u) : ex2(now_at - u);
            unit[nt][x] = u;
          }
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) fac[mt][nt][0] = fac[mt][nt][1] = two(1.f, 1.f);
          neg[nt] = two(-n[0], -n[1]);
          sum[nt] = f32x2_mul(sum[nt], two(c[0], c[1]));
          lift[nt] = two(ex2(kLift - unit[nt][0]), ex2(kLift - unit[nt][1]));
        }
#pragma unroll
        for (int i = 0; i < kNO; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][nt][e] *= alpha[nt][e & 1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sum[nt] = now[nt];
      // ---- the second product, 16 keys at a time ----
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = transposed(pw[mt][nt][0]);
          pb[nt][1] = transposed(pw[mt][nt][1]);
        }
        // rows 2 t4 and 2 t4 + 1 (h = 0) and 8 further (h = 1), in the halves of a register
        uint32_t vl[2][kW], vh[2][kW];  // even and odd elements of the lane's words
        int4row::Mul vm[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* at = st + C::kTileBytes + g8 * (D / 16) + (16 * mt + 8 * h) * C::kRowBytes;
          uint32_t w0[kW], w1[kW];
          if constexpr (D == 128) {
            const uint2 y0 = *reinterpret_cast<const uint2*>(at + v_key0 * C::kRowBytes), y1 = *reinterpret_cast<const uint2*>(at + v_key1 * C::kRowBytes);
            w0[0] = y0.x; w0[1] = y0.y;
            w1[0] = y1.x; w1[1] = y1.y;
          } else {
            w0[0] = *reinterpret_cast<const uint32_t*>(at + v_key0 * C::kRowBytes);
            w1[0] = *reinterpret_cast<const uint32_t*>(at + v_key1 * C::kRowBytes);
          }
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            vl[h][i] = prmt(w0[i], w1[i], 0x5410u);
            vh[h][i] = prmt(w0[i], w1[i], 0x7632u);
          }
          const uint8_t* rec = vrec + (16 * mt + 8 * h) * int4row::kRecord + 4;
          const uint32_t m0 = *reinterpret_cast<const uint32_t*>(rec + v_key0 * int4row::kRecord);
          const uint32_t m1 = *reinterpret_cast<const uint32_t*>(rec + v_key1 * int4row::kRecord);
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

    if (cc.kt + 1 == cc.sh.kt || t + 1 == tiles) {
      // ---- the item's end, or the run's: join the warps' key slices, 8 rows at a time ----
      const bool whole = kt_begin == 0 && cc.kt + 1 == cc.sh.kt;
      const long long pslot = 2ll * blockIdx.x + (kt_begin > 0 ? 0 : 1);
      // the warps' outputs meet in the slots just read: [8][kPad] of each warp
      auto meet = [&](int w) { return reinterpret_cast<float*>(smem + (w * kStages + slot) * C::kSlotBytes); };
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0) __syncthreads();  // the rows before are read
        float back[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float all = x ? hi32(sum[nt]) : lo32(sum[nt]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
          const float m = x ? -hi32(neg[nt]) : -lo32(neg[nt]);
          // sums relative to the maximum again (and of the operands' unit: one after the other, their product may pass FP32)
          back[x] = ex2(unit[nt][x] - kLift);
          if (g8 == 0) ml[warp][8 * nt + 2 * t4 + x] = make_float2(m == kLow ? -INFINITY : m, all);
        }
        float* const mo = meet(warp);
#pragma unroll
        for (int i = 0; i < kNO; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *reinterpret_cast<float2*>(mo + (2 * t4 + x) * C::kPad + (D / 8) * g8 + 2 * i) =
                make_float2(o[i][nt][x] * int4row::kUnit * back[x], o[i][nt][2 + x] * int4row::kUnit * back[x]);
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
            const float4 v = *reinterpret_cast<const float4*>(meet(w) + rr * C::kPad + c);
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
          join_item<D, kRT, kThreads>(a, cc.s, sp, run.per, cc.g, cc.rt, rows, meet(0), tid);
          clear_arrivals(a, sp, run.per);
        }
      }
      item_first += cc.sh.ku;
      // what was written here comes before the slot's next copies
      fence_proxy_async_smem();
      __syncthreads();
    }
    __syncwarp();  // the slot is read
    if (more && !gave_up) {
      if (by_rows) fence_proxy_async_smem();
      __syncwarp();
      fill(slot);
    } else {
      cp_commit();
    }
    if (++cc.kt == cc.sh.kt) cc.next_item(a, run.pad);
    if (++slot == kStages) slot = 0;
  }
  for (int i = 0; i < kStages; ++i)  // (a wait that ran out) copies under way land before the CTA exits
    if (bulks >> i & 1) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&full[warp][i], phases >> i & 1) && globaltimer() - t0 <= kWaitLimitNs) {
      }
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
  // bulk copies: pages that divide a warp's keys, in pieces of 4 keys at least, or hold them; records on 16 bytes
  const int ps = a.page_size;
  const int whole = (ps & (ps - 1)) == 0 && ps >= 4 && aligned(a.ks, 16) && aligned(a.vs, 16) ? 1 : 0;
  return launch_pdl(kern, dim3(runs), dim3(kThreads), C::kSmem, st, a, whole) == cudaSuccess ? MNW_OK : MNW_E_CUDA;
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
