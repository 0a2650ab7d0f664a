// mnw_attn_paged_block.cu -- paged attention for blocks of new tokens: 128
// query rows (tokens x the query heads of a kv head) on tcgen05, scores and
// probabilities in tensor memory.  Formulas: mnw_attn_paged.cu; the work's
// split and the joining of its parts: mnw_attn_split.cuh.
//
// A refinement block of 32 tokens with 4 query heads per kv head is 128 rows:
// 128 flops per byte of a BF16 cache, 256 of an INT8 one, which the warp-level
// tensor instructions cannot feed (2046 of tcgen05's ~3800 multiply-adds a
// clock, and every 16 rows would read the tile from shared memory again).
//
// Roles (512 threads):
//   warps 0-1   key loaders, warps 2-3 value loaders.  A tile that lies whole
//               inside the length, of pages that divide it (or that it
//               divides), comes by TMA, a lane per page, straight into operand
//               tiles of the 128-byte-swizzle layout.  Other tiles (the last of
//               a sequence, whose rows past the length must read as zeros; odd
//               page sizes) come by 16-byte cp.async, 64 keys a warp, fenced to
//               the tensor cores' proxy.  INT8: codes land in a raw buffer
//               (bulk copies), are taken into registers, and leave them as FP16
//               operand tiles (exact) while the next codes land.
//   warp 4      issues S_t = Q K_t^T, warp 5 O += P_t V_t, with P_t from
//               tensor memory and V as it lies in the cache, [key][d], an
//               operand whose N dimension is contiguous.  Two warps, because
//               one accumulator's products follow each other at ~96 cycles
//               and the two chains fill each other's gaps.
//   warps 6-7   the query tile of each segment (a run's part of an item) but
//               the first, and the segment's description for the other roles.
//   warps 8-15  softmax, 16 rows a warp, a thread 32 keys of two rows (so a
//               key's scales serve two rows), kept in registers from the
//               maximum to P; the next tiles' scores are computed meanwhile.
// S of a tile goes into its score buffer once P V of the tile there before is
// complete.
//
// Measured on one GB300: 16 sequences of 32 tokens over up to 4000 INT8
// positions, 16 query and 4 key heads of 128 (42 MB of cache): 43.2 us; 8 of 32
// over up to 16384 BF16 positions, 32 and 8 heads of 64 (170 MB): 45.1 us,
// 3.8 TB/s.  About 10 us of each are a run's head (split, first tiles) and
// tail and the joining kernel.  In between BF16 is bound by the softmax (about
// 1700 clocks a tile), INT8 by the loaders' step (about 4500): the conversion,
// the wait for the next codes, which are asked for only when the one raw
// buffer's last quarter is in registers, and instruction fetches, not told
// apart.  Tried: two softmax groups of 4 warps on alternate tiles, an accumulator
// each (48 and 51 us), twice the loader warps with fewer registers for the rest
// (44 and 51, when this form took 45 and 47: the conversion alone does not bound
// it), 64 keys at a time in the softmax (5 us more).
//
// BF16 caches: P is rounded to BF16 relative to a running maximum that moves
// only when it grows by more than 2^8.  INT8 caches: scores times the key's
// scale; P times the value's scale is rounded to FP16 (2^-11 relative)
// relative to the row's largest such product so far, lifted by 2^14, so one
// 2^-38 of the largest is still held.  The FP16 form costs half of what the TF32
// one does here, where the products are the bound, not the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "mnw_attn_split.cuh"

namespace mnw {
namespace pattn {
namespace {

constexpr int kRT = kBlockRows, kTK = kBlockKeys;
constexpr int kThreads = 512;
constexpr int kLoadWarps = 4, kWarpS = 4, kWarpPv = 5, kWarpQ = 6, kWarpSm0 = 8;
constexpr int kTmemCols = 512;
constexpr int kMaxSegs = 8;      // segment descriptions held; at most four segments are under way
constexpr int kMaxSlots = 4;
constexpr int kMaxKScales = 9, kMaxVScales = 6;
constexpr int kMaxBufs = 3;
constexpr float kRescaleLog2 = 8.f;

template <int D, bool INT8>
struct BCfg {
  static constexpr int kHalves = D / 64;                   // 64 elements = 128 bytes per operand row piece
  static constexpr uint32_t kPiece = kTK * 128;            // 128 rows of 128 bytes
  static constexpr uint32_t kTile = kHalves * kPiece;      // operand tile
  static constexpr int kSlotsK = D == 64 ? 4 : (INT8 ? 2 : 3), kSlotsV = D == 64 ? 4 : 2;
  static constexpr uint32_t kRaw = INT8 ? kTK * D : 0;     // raw codes of a tile
  // Tensor memory: score buffers (tile t in buffer t % kBufs, its P over the first half), then O.  Three: one in the
  // softmax, one whose P is being consumed, one being computed.
  static constexpr int kBufs = 3;
  static constexpr uint32_t kColO = kBufs * kTK;
  static_assert(kColO + D <= kTmemCols && kBufs <= kMaxBufs);
  // Scales are copied with a tile's codes, which are issued once the tile two before went into its operand slot, that
  // is, once the product with the tile that held the slot before is complete (S waits for P V of kBufs tiles before);
  // the softmax of a tile reads them last before P V of the tile is issued.
  static constexpr int kScalesK = 2 + kSlotsK + kBufs, kScalesV = 2 + kSlotsV;
  static_assert(kScalesK <= kMaxKScales && kScalesV <= kMaxVScales && kSlotsK <= kMaxSlots && kSlotsV <= kMaxSlots);
  static constexpr uint32_t kOffK = kTile;                 // Q first
  static constexpr uint32_t kOffV = kOffK + kSlotsK * kTile;
  static constexpr uint32_t kOffRaw = kOffV + kSlotsV * kTile;            // keys' codes, values' codes
  static constexpr uint32_t kOffKS = kOffRaw + 2 * kRaw;                  // [kScalesK][kTK] scales of keys
  static constexpr uint32_t kOffVS = kOffKS + (INT8 ? kScalesK * kTK * 4 : 0);  // [kScalesV][2][kTK] of values, and their log2
  static constexpr uint32_t kOffBars = kOffVS + (INT8 ? kScalesV * 2 * kTK * 4 : 0);
};

// A run's part of one item.
struct Seg {
  int tiles, kt0;       // tiles of the run, from key tile kt0
  int g, rt, whole;     // kv head, row tile; whether it is the item whole
  Seq s;
};

struct Bars {
  uint64_t full[2][kMaxSlots], empty[2][kMaxSlots];  // operand rings: keys, values
  uint64_t raw_full[2], raw_empty[2];
  uint64_t q0_full, q_full, q_empty;                 // the first query tile is there, a later one; consumed
  uint64_t s_full[kMaxBufs], p_full[kMaxBufs], s_free[kMaxBufs];  // per score buffer: scores complete, P written, P consumed
  uint64_t o_full, epi;                 // a segment's output complete; read
  uint64_t ks_full[kMaxKScales], vs_full[kMaxVScales];
  uint64_t seg_full[kMaxSegs];
  uint64_t drain[2];
  float qfac[4][kRT];                   // [segment % 4] INT8: the query rows' powers of two
  Seg seg[kMaxSegs];
  uint32_t tmem_base;
  int abort;
};

// The warpgroup's registers a thread from here on: more (N > 0, waits until
// they are free) or fewer (N < 0).  The kernel is built for kRegsBuilt, and the
// split must not pass that in sum.  Once a role: a second change would have to
// meet the whole warpgroup first, and may wait for a contiguous range for ever.
constexpr int kRegsBuilt = 128, kRegsLoad = 88, kRegsMma = 72, kRegsSoftmax = 176;
static_assert(kRegsLoad + kRegsMma + 2 * kRegsSoftmax == 4 * kRegsBuilt);
template <int N>
__device__ __forceinline__ void registers() {
  if constexpr (N > 0)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(-N));
}

struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void advance(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// The roles' waits are polled_wait()s, short in code: the kernel's has to stay
// below the instruction cache's size (at 142 KB the INT8 form stalled for
// thousands of cycles at a time).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = polled_wait(bar, parity, abort, err) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) return;
  }
}
// Operand whose N dimension is contiguous (128-byte swizzle): 64 elements of N
// per 128-byte row, rows along K; 8-row groups 1024 bytes apart (stride), the
// next 64 elements of N one piece further (leading).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t piece) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(piece >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kBMajorN = 1u << 16;  // instruction descriptor: B's N dimension contiguous

// Both of two barriers, polled by different lanes.  A vote orders no memory accesses: what the polling lanes saw is
// before what the others do only behind the next __syncwarp().
__device__ __forceinline__ bool warp_poll2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* abort, uint32_t* err) {
  int ok = 1;
  const int lane = threadIdx.x & 31;
  if (lane < 2) ok = polled_wait(lane ? b : a, lane ? pb : pa, abort, err) ? 1 : 0;
  return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* abort, uint32_t* err) {
  const bool both = warp_poll2(a, pa, b, pb, abort, err);
  __syncwarp();
  return both;
}
// Tensor memory, 16 lanes from the address's: thread (g, t) = (lane / 4, lane % 4) gets of every 8 columns 2t and 2t + 1
// of row g, then of row g + 8 (registers 4j .. 4j + 3 of columns 8j ..).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// As above with one register per row and 4 columns: column t of row g, of row g + 8 (registers 2j, 2j + 1 of columns 4j ..).
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float lo32(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi32(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1)
    paged_block_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a,
                       const int whole_pages) {
  using C = BCfg<D, INT8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset: the pointer stays a shared-memory one)
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBars);
  volatile int* abort = &bars->abort;
  __shared__ SplitShared split;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      for (int i = 0; i < kMaxSlots; ++i) {
        mbar_init(&bars->full[x][i], 2);
        mbar_init(&bars->empty[x][i], 1);
      }
      mbar_init(&bars->raw_full[x], 1);
      mbar_init(&bars->raw_empty[x], 2);
      mbar_init(&bars->drain[x], 1);
    }
    mbar_init(&bars->q0_full, 8);
    mbar_init(&bars->q_full, 2);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->epi, 8);
    for (int i = 0; i < kMaxKScales; ++i) mbar_init(&bars->ks_full[i], 2);
    for (int i = 0; i < kMaxVScales; ++i) mbar_init(&bars->vs_full[i], 2);
    for (int i = 0; i < kMaxSegs; ++i) mbar_init(&bars->seg_full[i], 1);
    for (int i = 0; i < kMaxBufs; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 8);
      mbar_init(&bars->s_free[i], 1);
    }
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpS) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  const Run run = find_run<kRT, kTK, kThreads, kMaxSlack>(a, &split);
  Cursor<kRT, kTK> kc{};
  int tiles = 0;
  if (run.seq >= 0) {
    kc.set(a, run);
    tiles = run.pad == 1 ? run.u1 - run.u0 : min(run.u1 - run.u0, kc.sh.kt - kc.kt);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // A warp's part of segment `seg`'s query tile, the item at kc: rows r0 .. r0 + n, n a multiple of 16.
  auto query_rows = [&](int seg, int r0, int n) {
    constexpr int kQC = D / 8, kQR = 32 / kQC;  // lanes of a row, rows at a time
    constexpr int kQB = 16 / kQR;               // rows of a lane at once; one by one is a chain of latencies
    const int rows = min(kRT, kc.s.n * a.G - kc.rt * kRT);
    const int c = lane % kQC;
    auto chunk = [&](int r) { return (c >> 3) * C::kPiece + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
#pragma unroll 2
    for (int i = 0; i < n / kQR; ++i) {
      const int r = r0 + lane / kQC + i * kQR;
      const int ri = kc.rt * kRT + (r < rows ? r : 0);
      const int tok = static_cast<int>(paged::quotient(ri, a.g_div)), hh = ri - tok * a.G;
      cp_async16(sbase + chunk(r), a.q + static_cast<long long>(kc.s.start + tok) * a.q_stride +
                                 static_cast<long long>(kc.g * a.G + hh) * D + c * 8,
           r < rows ? 16u : 0u);
    }
    cp_commit();
    cp_wait<0>();
    if constexpr (INT8) {  // in place: FP16 times a power of two
#pragma unroll 1
      for (int rb = r0 + lane / kQC; rb < r0 + n; rb += 16) {
        uint4 w[kQB];
        uint32_t mag[kQB];
#pragma unroll
        for (int i = 0; i < kQB; ++i) w[i] = *reinterpret_cast<const uint4*>(smem + chunk(rb + i * kQR));
#pragma unroll
        for (int i = 0; i < kQB; ++i) {
          const uint32_t m = __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                      __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
          mag[i] = max(m >> 16, m & 0xFFFFu);
        }
#pragma unroll
        for (int d = kQC / 2; d > 0; d >>= 1)
#pragma unroll
          for (int i = 0; i < kQB; ++i) mag[i] = max(mag[i], __shfl_xor_sync(0xffffffffu, mag[i], d));
#pragma unroll
        for (int i = 0; i < kQB; ++i) {
          const int e = row_exponent(mag[i]);
          const float f = two_to(-e);
          auto half = [&](uint32_t y) { return half2_bits(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xFFFF0000u) * f); };
          const int r = rb + i * kQR;
          *reinterpret_cast<uint4*>(smem + chunk(r)) = make_uint4(half(w[i].x), half(w[i].y), half(w[i].z), half(w[i].w));
          if (c == 0) bars->qfac[seg & 3][r] = two_to(e);
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp < kLoadWarps) {
    // ======================= loaders =======================
    registers<-kRegsLoad>();
    const bool values = warp >= 2;   // (uniform in the warp)
    const int lw = warp & 1;         // which 64 keys of a tile
    const int ring_slots = values ? C::kSlotsV : C::kSlotsK;
    const uint32_t ring_at = values ? C::kOffV : C::kOffK;
    uint64_t* const full = bars->full[values ? 1 : 0];
    uint64_t* const empty = bars->empty[values ? 1 : 0];
    const uint8_t* const base = values ? a.vc : a.kc;
    constexpr int kCh = (INT8 ? D : 2 * D) / 16;  // chunks of a cached row
    constexpr int kRows = 32 / kCh;               // rows per pass of the warp
    // whole pages: page `lane` of a tile, `span` keys each
    const int span = min(a.page_size, kTK), pieces = kTK / span;
    bool ok = tiles > 0;
    RingPos ring;
    auto table_at = [&](int seq, int p) {
      return __ldg(a.bt.block_table + static_cast<size_t>(seq) * a.bt.max_pages + paged::quotient(p, a.page_div));
    };
    // What is issued: the tile at kc; its pieces' pages are looked up a tile early.
    bool whole;
    int page;
    auto peek = [&]() {
      whole = whole_pages && (kc.kt + 1) * kTK <= kc.s.len;
      page = whole && lane < pieces ? table_at(kc.b, kc.kt * kTK + lane * span) : 0;
    };
    // row by row: this warp's 64 keys of the tile, to `to` (operand tile, or raw codes) and its scales to `sc`
    auto copy_rows = [&](uint32_t to, uint32_t sc) {
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const int r0 = lw * 64 + part * 32;
        const int p = kc.kt * kTK + r0 + lane;
        int pg = -1, at = 0;
        if (p < kc.s.len) {
          pg = table_at(kc.b, p);
          at = kc.g * a.page_size + (p - static_cast<int>(paged::quotient(p, a.page_div)) * a.page_size);
          if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) {
            pg = -1;
            if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
          }
        }
        const long long mine = pg >= 0 ? pg * a.page_bytes + static_cast<long long>(at) * (kCh * 16) : -1;
        const int c = lane % kCh;
#pragma unroll 2
        for (int i = 0; i < 32 / kRows; ++i) {
          const int r = i * kRows + lane / kCh;
          const long long off = __shfl_sync(0xffffffffu, mine, r);
          const int row = r0 + r;
          const uint32_t dst = INT8 ? to + row * D + c * 16
                                    : to + (c >> 3) * C::kPiece + row * 128 + (((c & 7) ^ (row & 7)) << 4);
          cp_async16(dst, base + (off >= 0 ? off + c * 16 : 0), off >= 0 ? 16u : 0u);
        }
        if constexpr (INT8)
          cp_async4(sc + (r0 + lane) * 4, (values ? a.vs : a.ks) + (pg >= 0 ? static_cast<long long>(pg) * a.Hkv * a.page_size + at : 0),
              pg >= 0 ? 4u : 0u);
      }
      cp_commit();
    };
    auto step = [&]() {
      if (++kc.kt == kc.sh.kt) kc.next_item(a, run.pad);
    };
    if (ok) peek();
    if constexpr (!INT8) {
      uint64_t* pending = nullptr;  // the barrier of a tile copied row by row and not yet given on
      auto give = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(pending);
        pending = nullptr;
      };
      for (int t = 0; ok && t < tiles; ++t) {
        if (!warp_wait(&empty[ring.slot], ring.phase ^ 1, abort, a.err)) { ok = false; break; }
        uint64_t* bar = &full[ring.slot];
        const uint32_t at = ring_at + ring.slot * C::kTile;
        const bool rows = !whole || __any_sync(0xffffffffu, static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages));
        if (rows) {
          copy_rows(sbase + at, 0);
        } else {
          if (lw == 0) {
            if (lane == 0) mbar_arrive_expect_tx(bar, C::kTile);
            __syncwarp();
            if (lane < pieces) {
              const int in_page = a.page_size > kTK ? (kc.kt * kTK) & (a.page_size - 1) : 0;
              uint8_t* dst = smem + at + lane * span * 128;
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
                tma_load_4d(dst + h * C::kPiece, values ? &tm_v : &tm_k, bar, 64 * h, in_page, kc.g, page);
            }
            __syncwarp();
          } else if (lane == 0) {
            mbar_arrive(bar);
          }
        }
        if (pending) {
          if (rows)
            cp_wait<1>();
          else
            cp_wait<0>();
          give();
        }
        if (rows) pending = bar;
        ring.advance(ring_slots);
        step();
        if (t + 1 < tiles) peek();
      }
      cp_wait<0>();
      if (pending) give();
      if (*abort && lw == 0) {
        // let every bulk copy already issued land before the CTA exits
        for (int i = 0; i < ring_slots; ++i) drain_wait(&full[i], i < static_cast<int>(ring.slot) ? ring.phase : ring.phase ^ 1);
      }
    } else {
      uint64_t *const raw_full = &bars->raw_full[values ? 1 : 0], *const raw_empty = &bars->raw_empty[values ? 1 : 0];
      const uint32_t raw_at = C::kOffRaw + (values ? C::kRaw : 0);
      uint32_t raw_phase = 0;  // parity of the next bulk landing
      int sc_issue = 0, sc_now = 0;  // scale slots of the tile issued next, of the tile that lands next
      auto scales_at = [&](int slot) { return values ? C::kOffVS + slot * (2 * kTK * 4) : C::kOffKS + slot * (kTK * 4); };
      const int sc_slots = values ? C::kScalesV : C::kScalesK;
      bool landing_rows = false;
      // codes of the tile at kc into the raw buffer, whose last codes both warps have taken (uses counted by `uses`); rows
      // into the warp's own half, whose last codes it has taken itself
      auto issue = [&](int uses) -> bool {
        landing_rows = !whole || __any_sync(0xffffffffu, static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages));
        if (landing_rows) {
          copy_rows(sbase + raw_at, sbase + scales_at(sc_issue));
        } else if (lw == 0) {
          if (!warp_wait(raw_empty, (uses & 1) ^ 1, abort, a.err)) return false;
          if (lane == 0) mbar_arrive_expect_tx(raw_full, C::kRaw + kTK * 4);
          __syncwarp();
          if (lane < pieces) {
            const int at = kc.g * a.page_size + (a.page_size > kTK ? (kc.kt * kTK) & (a.page_size - 1) : 0);
            bulk_load(smem + raw_at + lane * span * D, base + page * a.page_bytes + static_cast<long long>(at) * D, span * D,
                      raw_full);
            bulk_load(smem + scales_at(sc_issue) + lane * span * 4,
                      (values ? a.vs : a.ks) + static_cast<long long>(page) * a.Hkv * a.page_size + at, span * 4, raw_full);
          }
          __syncwarp();
        }
        if (++sc_issue == sc_slots) sc_issue = 0;
        return true;
      };
      bool bulk_out = false;  // a bulk copy is under way
      constexpr int kW = 4 * kCh, kOC = D / 8;  // 64 rows, 8 codes a lane: one 16-byte chunk of the operand row
      // step t: tile t lands and is converted in parts, each by way of registers; the copies of tile t + 1 go out as soon
      // as the last is there
      constexpr int kParts = 4, kPW = kW / kParts, kPR = 64 / kParts;
      for (int t = -1; ok && t < tiles; ++t) {
        if (t >= 0) {
          if (landing_rows) {
            cp_wait<0>();
            fence_proxy_async_smem();  // rows came by this proxy, the next codes may come by the other
            __syncwarp();
          } else {
            if (!(values ? warp_wait(raw_full, raw_phase, abort, a.err)
                         : warp_wait2(raw_full, raw_phase, &empty[ring.slot], ring.phase ^ 1, abort, a.err))) { ok = false; break; }
            raw_phase ^= 1;
            bulk_out = false;
          }
          // the values' scales are given on at once: the softmax of a tile runs while its values still wait for their slot
          if (values) {
            float* sc = reinterpret_cast<float*>(smem + scales_at(sc_now)) + lw * 64 + lane;
            sc[kTK] = __log2f(sc[0]);
            sc[kTK + 32] = __log2f(sc[32]);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(values ? &bars->vs_full[sc_now] : &bars->ks_full[sc_now]);
          if (++sc_now == sc_slots) sc_now = 0;
          // The slot; for rows also that both warps have taken the codes before (raw_full implies it for bulk copies).  A
          // warp that went ahead alone through tiles of rows would complete raw_empty's phases in the other's place, and
          // the parity that a later bulk copy waits for would stand for another phase.
          if ((values || landing_rows) &&
              !warp_wait2(&empty[ring.slot], ring.phase ^ 1, landing_rows ? raw_empty : &empty[ring.slot],
                          (landing_rows ? t & 1 : ring.phase) ^ 1, abort, a.err)) { ok = false; break; }
        }
        uint8_t* op = smem + ring_at + ring.slot * C::kTile + lw * 64 * 128;
        const uint8_t* raw = smem + raw_at + lw * 64 * D + lane * 8;
#pragma unroll 1
        for (int part = t < 0 ? kParts - 1 : 0; part < kParts; ++part) {
          uint2 w[kPW];
          if (t >= 0) {
#pragma unroll
            for (int i = 0; i < kPW; ++i) w[i] = *reinterpret_cast<const uint2*>(raw + part * (kPR * D) + i * 256);
          }
          if (part == kParts - 1) {
            if (t >= 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive(raw_empty);
              step();
              if (t + 1 < tiles) peek();
            }
            if (t + 1 < tiles) {
              if (!issue(t + 1)) { ok = false; break; }
              bulk_out = !landing_rows;
            }
          }
          if (t >= 0) {
#pragma unroll
            for (int i = 0; i < kPW; ++i) {
              const int row = part * kPR + i * (32 / kOC) + lane / kOC, c = lane % kOC;  // of the warp's 64
              const uint32_t x = w[i].x ^ 0x80808080u, y = w[i].y ^ 0x80808080u;
              *reinterpret_cast<uint4*>(op + (c >> 3) * C::kPiece + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                  make_uint4(codes_lo(x), codes_hi(x), codes_lo(y), codes_hi(y));
            }
          }
        }
        if (!ok) break;
        if (t >= 0) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[ring.slot]);
          ring.advance(ring_slots);
        }
      }
      cp_wait<0>();
      if (bulk_out && lw == 0) drain_wait(raw_full, raw_phase);  // (an abort) the copy lands before the CTA exits
    }
  } else if (warp < kWarpSm0) {
    registers<-kRegsMma>();
    // ======================= MMA issuers =======================
    // The warps stay together and their first lanes issue.
    constexpr int kUnrollMma = INT8 ? 1 : 8;  // (the INT8 form is bound by its instruction cache)
    const bool lead = lane == 0;
    if (warp == kWarpS && tiles > 0) {
      const uint32_t idesc = idesc_f16(kRT, kTK, !INT8);
      RingPos kr, buf;
      int seg = 0, left = 0;  // segment of the next scores, its tiles to go
      for (int t = 0; t < tiles; ++t) {
        if (left == 0) {
          if (!warp_wait(&bars->seg_full[seg % kMaxSegs], (seg / kMaxSegs) & 1, abort, a.err)) break;
          left = bars->seg[seg % kMaxSegs].tiles;
          if (!warp_wait(seg ? &bars->q_full : &bars->q0_full, seg ? (seg - 1) & 1 : 0, abort, a.err)) break;
        }
        if (!warp_wait2(&bars->full[0][kr.slot], kr.phase, &bars->s_free[buf.slot], buf.phase ^ 1, abort, a.err)) break;
        tc_fence_after();
        --left;
        if (lead) {
          const uint32_t k_s = sbase + C::kOffK + kr.slot * C::kTile;
          const uint32_t d = tmem + buf.slot * kTK;
          // (descriptors count 16 bytes)
          uint64_t da = sdesc_sw128(sbase), db = sdesc_sw128(k_s);
#pragma unroll kUnrollMma
          for (int kk = 0; kk < D / 16; ++kk) {
            mma_ss(d, da, db, idesc, kk > 0);
            const uint32_t next = (kk & 3) == 3 ? (C::kPiece - 96) >> 4 : 2;
            da += next;
            db += next;
          }
          mma_commit(&bars->s_full[buf.slot]);
          mma_commit(&bars->empty[0][kr.slot]);
          if (left == 0) mma_commit(&bars->q_empty);
        }
        __syncwarp();
        kr.advance(C::kSlotsK);
        buf.advance(C::kBufs);
        if (left == 0) ++seg;
      }
    }
    if (warp == kWarpPv && tiles > 0) {
      const uint32_t idesc = idesc_f16(kRT, D, !INT8) | kBMajorN;
      RingPos vr, buf;
      int seg = 0, left = 0, begin = 0;  // segment of the next product, its tiles to go, its first tile
      for (int t = 0; t < tiles; ++t) {
        if (left == 0) {
          if (!warp_wait(&bars->seg_full[seg % kMaxSegs], (seg / kMaxSegs) & 1, abort, a.err)) break;
          left = bars->seg[seg % kMaxSegs].tiles;
          // the segment before has been read out of O
          if (seg > 0 && !warp_wait(&bars->epi, (seg - 1) & 1, abort, a.err)) break;
        }
        if (!warp_wait2(&bars->full[1][vr.slot], vr.phase, &bars->p_full[buf.slot], buf.phase, abort, a.err)) break;
        tc_fence_after();
        --left;
        if (lead) {
          const uint32_t v_s = sbase + C::kOffV + vr.slot * C::kTile;
          const uint32_t p = tmem + buf.slot * kTK;  // two keys per column
          const uint32_t o = tmem + C::kColO;
          const bool fresh = t == begin;
          uint64_t db = sdesc_mn_sw128(v_s, C::kPiece);
#pragma unroll kUnrollMma
          for (int kk = 0; kk < kTK / 16; ++kk, db += 2048 >> 4) mma_ts(o, p + kk * 8, db, idesc, !(fresh && kk == 0));
          mma_commit(&bars->s_free[buf.slot]);
          mma_commit(&bars->empty[1][vr.slot]);
          if (left == 0) mma_commit(&bars->o_full);
        }
        __syncwarp();
        vr.advance(C::kSlotsV);
        buf.advance(C::kBufs);
        if (left == 0) {
          ++seg;
          begin = t + 1;
        }
      }
    }
    if (warp >= kWarpQ) {
      // ======================= queries =======================
      const int qw = warp - kWarpQ;  // which 64 rows
      int t = 0;
      for (int seg = 0; t < tiles; ++seg) {
        const int n = min(kc.sh.kt - kc.kt, tiles - t);
        if (qw == 0 && lane == 0) {
          Seg d;
          d.tiles = n;
          d.kt0 = kc.kt;
          d.g = kc.g;
          d.rt = kc.rt;
          d.whole = kc.kt == 0 && n == kc.sh.kt;
          d.s = kc.s;
          bars->seg[seg % kMaxSegs] = d;
          mbar_arrive(&bars->seg_full[seg % kMaxSegs]);
        }
        if (seg > 0) {  // (the first segment's: the softmax warps)
          if (!warp_wait(&bars->q_empty, (seg - 1) & 1, abort, a.err)) break;
          query_rows(seg, qw * 64, 64);
          if (lane == 0) mbar_arrive(&bars->q_full);
        }
        t += n;
        if (t < tiles) kc.next_item(a, run.pad);
      }
    }
    if ((warp == kWarpS || warp == kWarpPv) && lead) {
      // every MMA has finished with shared and tensor memory before the CTA tears down
      mma_commit(&bars->drain[warp - kWarpS]);
      drain_wait(&bars->drain[warp - kWarpS], 0);
    }
    __syncwarp();
  } else {
    // ======================= softmax =======================
    registers<kRegsSoftmax>();
    // nothing to do yet: the first segment's queries, 16 rows each (by the two query warps alone they were the last thing
    // the first scores waited for)
    if (tiles > 0) {
      query_rows(0, (warp - kWarpSm0) * 16, 16);
      if (lane == 0) mbar_arrive(&bars->q0_full);
    }
    const int grp = (warp - kWarpSm0) >> 2;  // rows 16 grp .. of the lane quarter's 32
    const int quarter = warp & 3;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int r16 = quarter * 32 + 16 * grp + g8;  // this thread's rows: r16, r16 + 8
    const uint32_t at16 = tmem + (static_cast<uint32_t>(quarter * 32 + 16 * grp) << 16);
    bool ok = true;
    int t = 0, ks_slot = 0, vs_slot = 0;
    uint32_t ks_phase = 0, vs_phase = 0;
    RingPos buf;  // tile t's score buffer
    for (int seg = 0; ok && t < tiles; ++seg) {
      if (!warp_wait(&bars->seg_full[seg % kMaxSegs], (seg / kMaxSegs) & 1, abort, a.err)) break;
      const Seg& sg = bars->seg[seg % kMaxSegs];
      const int rows = min(kRT, sg.s.n * a.G - sg.rt * kRT);
      const int end = t + sg.tiles;
      // of rows r16 + 8 x: first key (of the tile at hand) not seen, maximum, sum of this thread's keys, log2 of O's unit
      struct RowState {
        int left;
        float m, l, unit;
      } st[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        st[x] = RowState{row_limit(a, sg.s, sg.rt * kRT + min(r16 + 8 * x, rows - 1)) - sg.kt0 * kTK, -INFINITY, 0.f, -INFINITY};
      const int begin = t;
      for (; t < end; ++t) {
        if constexpr (INT8) {
          if (!warp_poll2(&bars->ks_full[ks_slot], ks_phase, &bars->vs_full[vs_slot], vs_phase, abort, a.err)) { ok = false; break; }
        }
        if (!warp_wait(&bars->s_full[buf.slot], buf.phase, abort, a.err)) { ok = false; break; }
        const uint32_t s_at = at16 + buf.slot * kTK;
        const float *ks = nullptr, *vs = nullptr;
        if constexpr (INT8) {
          ks = reinterpret_cast<const float*>(smem + C::kOffKS) + ks_slot * kTK + 2 * t4;
          vs = reinterpret_cast<const float*>(smem + C::kOffVS) + vs_slot * 2 * kTK + 2 * t4;
        }
        tc_fence_after();
        float fac[2] = {a.scale_log2, a.scale_log2};
        if constexpr (INT8) {
          // the query rows' factors were written before q_full, which the scores waited for
          const float* qf = &bars->qfac[seg & 3][r16];
          fac[0] *= qf[0];
          fac[1] *= qf[8];
        }
        const uint64_t fac2[2] = {f32x2_pack(__float_as_uint(fac[0]), __float_as_uint(fac[0])),
                                  f32x2_pack(__float_as_uint(fac[1]), __float_as_uint(fac[1]))};
        // scales are loaded in one go ahead of their use: a load before each use waited for it 48 times a half
        uint64_t f[16];
        if constexpr (INT8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = *reinterpret_cast<const uint64_t*>(ks + 8 * i);
        }
        // the rows' scores, scaled (INT8) and masked: register 4 i + 2 x + e is key 8 i + 2 t4 + e of row g8 + 8 x
        uint32_t sv[64];
        tmem_ld_frag(s_at, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld_frag(s_at + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_wait_ld();
        if constexpr (INT8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint64_t y = f32x2_mul(f32x2_pack(sv[4 * i + 2 * x], sv[4 * i + 2 * x + 1]), f[i]);
              sv[4 * i + 2 * x] = static_cast<uint32_t>(y);
              sv[4 * i + 2 * x + 1] = static_cast<uint32_t>(y >> 32);
            }
          }
        }
        if (__any_sync(0xffffffffu, min(st[0].left, st[1].left) < kTK)) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (8 * (e >> 2) + 2 * t4 + (e & 1) >= st[(e >> 1) & 1].left) sv[e] = 0xff800000u;  // -inf
        }
        // the rows' maxima; INT8: also log2 of their largest e^score times value scale
        float top[2] = {-INFINITY, -INFINITY}, topv[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float other = -INFINITY;  // two chains
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            top[x] = fmaxf(fmaxf(top[x], __uint_as_float(sv[4 * i + 2 * x])), __uint_as_float(sv[4 * i + 2 * x + 1]));
            other = fmaxf(fmaxf(other, __uint_as_float(sv[4 * i + 4 + 2 * x])), __uint_as_float(sv[4 * i + 4 + 2 * x + 1]));
          }
          top[x] = fmaxf(top[x], other);
        }
        if constexpr (INT8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = *reinterpret_cast<const uint64_t*>(vs + kTK + 8 * i);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint64_t y = f32x2_fma(f32x2_pack(sv[4 * i + 2 * x], sv[4 * i + 2 * x + 1]), fac2[x], f[i]);
              topv[x] = fmaxf(fmaxf(topv[x], lo32(y)), hi32(y));
            }
          }
        }
        float alpha[2] = {1.f, 1.f}, lift[2] = {1.f, 1.f};
        uint64_t neg2[2], l2[2] = {0ull, 0ull};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], d));
            if constexpr (INT8) topv[x] = fmaxf(topv[x], __shfl_xor_sync(0xffffffffu, topv[x], d));
          }
          top[x] *= fac[x];
          RowState& rs = st[x];
          if constexpr (!INT8) {
            if (top[x] > rs.m + kRescaleLog2 || rs.m == -INFINITY) {
              const float n = fmaxf(rs.m, top[x]);
              alpha[x] = n == -INFINITY ? 1.f : ex2(rs.m - n);  // 0 where nothing was seen before
              rs.l *= alpha[x];
              rs.m = n;
            }
          } else {
            const float n = fmaxf(rs.m, top[x]);
            rs.l *= n == -INFINITY ? 1.f : ex2(rs.m - n);
            rs.m = n;
            // held within 2^100 of e^m so that the lift stays finite
            const float at = fmaxf(topv[x], n - 100.f);
            if (n != -INFINITY && at > rs.unit + 1.f) {
              alpha[x] = ex2(rs.unit - at);  // 0 from -inf
              rs.unit = at;
            }
            lift[x] = rs.unit == -INFINITY ? 0.f : ex2(n - rs.unit + 14.f);
          }
          const float base = rs.m == -INFINITY ? 0.f : rs.m;
          neg2[x] = f32x2_pack(__float_as_uint(-base), __float_as_uint(-base));
        }
        if (t > begin && __any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
          // the product before has to be complete
          if (!warp_wait(&bars->s_free[(t - 1) % C::kBufs], ((t - 1) / C::kBufs) & 1, abort, a.err)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < D; i += 64) {
            uint32_t o[32];
            tmem_ld_frag(at16 + C::kColO + i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[(e >> 1) & 1]);
            tmem_st_frag(at16 + C::kColO + i, o);
          }
        }
        if constexpr (INT8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = *reinterpret_cast<const uint64_t*>(vs + 8 * i);
        }
        // p = 2^(s fac - m), two keys per packed operation, its sum, and P, two keys a column, over the first half of
        // the rows' S columns
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint64_t e2 = f32x2_fma(f32x2_pack(sv[4 * i + 2 * x], sv[4 * i + 2 * x + 1]), fac2[x], neg2[x]);
            uint64_t p2 = f32x2_pack(__float_as_uint(ex2(lo32(e2))), __float_as_uint(ex2(hi32(e2))));
            l2[x] = f32x2_add(l2[x], p2);
            if constexpr (INT8)
              p2 = f32x2_mul(f32x2_mul(p2, f[i]), f32x2_pack(__float_as_uint(lift[x]), __float_as_uint(lift[x])));
            sv[2 * i + x] = INT8 ? half2_bits(lo32(p2), hi32(p2)) : pack_bf16x2(lo32(p2), hi32(p2));
          }
        }
        tmem_st_pairs(s_at, *reinterpret_cast<uint32_t(*)[16]>(&sv[0]));
        tmem_st_pairs(s_at + 32, *reinterpret_cast<uint32_t(*)[16]>(&sv[16]));
#pragma unroll
        for (int x = 0; x < 2; ++x) st[x].l += lo32(l2[x]) + hi32(l2[x]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[buf.slot]);
        buf.advance(C::kBufs);
#pragma unroll
        for (int x = 0; x < 2; ++x) st[x].left -= kTK;
        if constexpr (INT8) {
          if (++ks_slot == C::kScalesK) {
            ks_slot = 0;
            ks_phase ^= 1;
          }
          if (++vs_slot == C::kScalesV) {
            vs_slot = 0;
            vs_phase ^= 1;
          }
        }
      }
      if (!ok) break;
      // ---- the segment's end ----
      const bool whole = sg.whole != 0;
      const long long pslot = 2ll * blockIdx.x + (sg.kt0 > 0 ? 0 : 1);
      float f[2];
      size_t row[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const RowState& rs = st[x];
        float sum = rs.l;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        f[x] = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        if (INT8 && rs.unit != -INFINITY) f[x] *= ex2(rs.unit - rs.m - 14.f);
        const int r = r16 + 8 * x;
        row[x] = out_row<kRT>(a, sg.s, sg.g, sg.rt, min(r, rows - 1));
        if (r < rows && t4 == 0) {
          if (!whole)
            __stcg(a.part_ml + pslot * kRT + r, make_float2(rs.m, sum));
          else if (a.lse)
            a.lse[row[x]] = (rs.m + log2f(sum)) * kLn2;
        }
      }
      if (!warp_wait(&bars->o_full, seg & 1, abort, a.err)) break;
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < D; i += 64) {
        uint32_t o[32];
        tmem_ld_frag(at16 + C::kColO + i, o);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (r16 + 8 * x < rows) {
            if (whole) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row[x] * D + i + 2 * t4);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                dst[4 * j] = pack_bf16x2(__uint_as_float(o[4 * j + 2 * x]) * f[x], __uint_as_float(o[4 * j + 2 * x + 1]) * f[x]);
            } else {
              float2* dst = reinterpret_cast<float2*>(a.part_o + (pslot * kRT + r16 + 8 * x) * D + i + 2 * t4);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                __stcg(dst + 4 * j, make_float2(__uint_as_float(o[4 * j + 2 * x]) * f[x], __uint_as_float(o[4 * j + 2 * x + 1]) * f[x]));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->epi);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool INT8>
int launch(const Args& a, int runs, cudaStream_t st) {
  constexpr size_t kSmem = BCfg<D, INT8>::kOffBars + sizeof(Bars) + 1024;
  static_assert(kSmem <= 232448 - 512, "shared memory of a CTA");
  auto kern = paged_block_kernel<D, INT8>;
  static std::atomic<uint64_t> attr{0};
  uint64_t bit;
  if (attrs_needed(attr, &bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
      return MNW_E_CUDA;
    // the roles' register split waits forever if the kernel was built for fewer
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != kRegsBuilt) return MNW_E_CUDA;
    attrs_done(attr, bit);
  }
  // tiles of whole pages: the page divides the tile in pieces of 8 rows at least (a swizzle atom), or holds tiles
  const int ps = a.page_size;
  bool whole = (ps & (ps - 1)) == 0 && ps >= 8;
  CUtensorMap maps[2];
  memset(maps, 0, sizeof(maps));
  if constexpr (INT8) {
    whole = whole && aligned(a.ks, 16) && aligned(a.vs, 16);
  } else if (whole) {
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(ps), static_cast<uint64_t>(a.Hkv),
                              static_cast<uint64_t>(a.n_pages)};
    const uint64_t strides[3] = {D * 2, static_cast<uint64_t>(ps) * D * 2, static_cast<uint64_t>(a.page_bytes)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(ps < kTK ? ps : kTK), 1, 1};
    whole = encode_map(&maps[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.kc, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
            encode_map(&maps[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.vc, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  return launch_pdl(kern, dim3(runs), dim3(kThreads), kSmem, st, maps[0], maps[1], a, whole ? 1 : 0) == cudaSuccess
             ? MNW_OK
             : MNW_E_CUDA;
}

}  // namespace

int launch_block(const Args& a, int d, bool int8, int runs, cudaStream_t st) {
  if (d == 128) return int8 ? launch<128, true>(a, runs, st) : launch<128, false>(a, runs, st);
  return int8 ? launch<64, true>(a, runs, st) : launch<64, false>(a, runs, st);
}

}  // namespace pattn
}  // namespace mnw
