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
//   warps 0-3   loaders.  A tile that lies whole inside the length, of pages
//               that divide it (or that it divides), comes by TMA, a lane per
//               page, straight into operand tiles of the 128-byte-swizzle
//               layout.  Other tiles (the last of a sequence, whose rows past
//               the length must read as zeros; odd page sizes) come by 16-byte
//               cp.async, each warp 32 keys, fenced to the tensor cores' proxy.
//               INT8: codes land in a raw ring (bulk copies) and the four
//               warps rewrite them as FP16 operand tiles (exact).  They also
//               bring the query tile of each segment (a run's part of an item)
//               and describe the segment to the other roles.
//   warp 4      issues the MMAs (one thread): S_t = Q K_t^T, O_g += P_t V_t
//               with P_t from tensor memory and V as it lies in the cache,
//               [key][d], an operand whose N dimension is contiguous.
//   warps 8-15  softmax, two groups of 4 warps: group t % 2 takes tile t, one
//               row per thread, with its own O accumulator, maximum and sum,
//               so that one group computes while the other's products run.
// Order of the products: S_0, S_1, then O += P_t V_t, S_{t+2}; a tile's
// scores being complete therefore means that its group's earlier product into
// O is complete too (one issuing thread, in order).
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
constexpr int kLoadWarps = 4, kWarpMma = 4, kWarpSm0 = 8;
constexpr int kTmemCols = 512;
constexpr uint32_t kColO = 256;  // O_g at kColO + 128 g; S_g at 128 g
constexpr int kMaxScaleSlots = 8, kMaxRawSlots = 3;
constexpr int kMaxSegs = 8;      // segment descriptions held; at most four segments are under way
constexpr float kRescaleLog2 = 8.f;

template <int D, bool INT8>
struct BCfg {
  static constexpr int kHalves = D / 64;                   // 64 elements = 128 bytes per operand row piece
  static constexpr uint32_t kPiece = kTK * 128;            // 128 rows of 128 bytes
  static constexpr uint32_t kTile = kHalves * kPiece;      // operand tile
  static constexpr int kSlots = D == 64 ? 8 : (INT8 ? 4 : 5);
  static constexpr int kAhead = 2;                         // items in flight behind the one being issued
  static constexpr int kRawSlots = kAhead + 1;
  // the scales of tile t + kScaleSlots are copied once P V of tile t was issued: the copy of keys t + n (item 2 (t + n) - 1)
  // follows the release of the operand slot kAhead + 1 + kSlots items before it, and values of tile j are item 2 j + 2
  static constexpr int kScaleSlots = kSlots == 8 ? 8 : 5;
  static_assert(!INT8 || 2 * kScaleSlots - 1 - (kAhead + 1) - kSlots >= 2);
  static constexpr uint32_t kRaw = INT8 ? kTK * D : 0;     // raw codes of a tile
  static constexpr uint32_t kScaleSlot = 3 * kTK * 4;      // scales of a tile's keys, of its values, log2 of the latter
  static constexpr uint32_t kOffRing = kTile;              // Q first
  static constexpr uint32_t kOffRaw = kOffRing + kSlots * kTile;
  static constexpr uint32_t kOffScale = kOffRaw + kRawSlots * kRaw;
  static constexpr uint32_t kOffBars = kOffScale + (INT8 ? kScaleSlots * kScaleSlot : 0);
};

// A run's part of one item.
struct Seg {
  int tiles, kt0;       // tiles of the run, from key tile kt0
  int g, rt, whole;     // kv head, row tile; whether it is the item whole
  int us, ku;           // the item's units
  Seq s;
};

struct Bars {
  uint64_t full[8], empty[8];           // operand ring
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2];        // per softmax group
  uint64_t o_full, epi;                 // a segment's output complete; read
  uint64_t sc_full[kMaxScaleSlots];
  uint64_t raw_full[kMaxRawSlots], raw_empty[kMaxRawSlots];
  uint64_t seg_full[kMaxSegs];
  uint64_t fin[4];                      // per lane quarter: both groups' maxima and sums written
  uint64_t drain;
  float st_m[2][2][kRT], st_l[2][2][kRT], st_u[2][2][kRT];  // [segment parity][group][row]: maximum, sum, log2 of O's unit over 2^maximum
  float qfac[4][kRT];                   // [segment % 4] INT8: the query rows' powers of two
  int st_any[2][2];                     // [segment parity][group]: whether the group had a tile
  Seg seg[kMaxSegs];
  Seg part[2];                          // the run's parts of shared items: the one that continues an item, that begins one
  int has_part[2];
  uint32_t tmem_base;
  int abort;
};

struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void advance(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The wait's slow side is a call: inlined at every wait of the roles it would
// be a good part of the kernel's code, whose size shows (instruction fetches).
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  return bounded_wait(bar, parity, abort, err);
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  return mbar_try_wait(bar, parity) || slow_wait(bar, parity, abort, err);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_for(bar, parity, abort, err) ? 1 : 0;
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
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBars);
  volatile int* abort = &bars->abort;
  __shared__ SplitShared split;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bars->full[i], kLoadWarps);
      mbar_init(&bars->empty[i], 1);
    }
    mbar_init(&bars->q_full, kLoadWarps);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
      bars->has_part[i] = 0;
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->epi, 8);
    for (int i = 0; i < kMaxScaleSlots; ++i) mbar_init(&bars->sc_full[i], kLoadWarps);
    for (int i = 0; i < kMaxRawSlots; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], kLoadWarps);
    }
    for (int i = 0; i < kMaxSegs; ++i) mbar_init(&bars->seg_full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bars->fin[i], 2);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  const Run run = find_run<kRT, kTK, kThreads>(a, &split);
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

  if (warp < kLoadWarps) {
    // ======================= loaders =======================
    // One loop with one place for each step: the code of the roles together
    // should stay near the instruction cache's size.
    bool ok = true;
    const int key = warp * 32 + lane;  // this lane's key of a tile copied row by row
    // whole pages: page `lane` of a tile, `span` keys each
    const int span = min(a.page_size, kTK), pieces = kTK / span;
    struct Tile {
      int b, g, kt, len;
      int page;    // of this lane's piece
      bool whole;  // by whole pages
    } now{}, prev{}, next{};
    int seg = -1, t_now = -1;
    int us = run.u0 - kc.kt;  // first unit of kc's item
    const uint32_t all = 2u * tiles;
    uint32_t n_items = 0, sent = 0;  // items issued; given to the tensor cores
    uint32_t by_rows = 0;            // bit i: item n_items - 1 - i was copied row by row
    uint32_t raw_phase = 0;          // bit s: parity of raw slot s's next bulk landing
    constexpr int kCh = (INT8 ? D : 2 * D) / 16;  // chunks of a cached row
    constexpr int kRows = 32 / kCh;               // rows per pass of the warp
    auto table_at = [&](int seq, int p) {
      return __ldg(a.bt.block_table + static_cast<size_t>(seq) * a.bt.max_pages + paged::quotient(p, a.page_div));
    };
    // the tile at kc, its page looked up early
    auto peek = [&](Tile& x) {
      x.b = kc.b;
      x.g = kc.g;
      x.kt = kc.kt;
      x.len = kc.s.len;
      x.whole = whole_pages && (kc.kt + 1) * kTK <= kc.s.len;
      x.page = x.whole && lane < pieces ? table_at(kc.b, kc.kt * kTK + lane * span) : 0;
    };
    if (tiles > 0) peek(next);
    while (ok) {
      // item i: keys of tile 0, then keys of tile (i + 1) / 2 where i is odd, values of tile i / 2 - 1 where it is even;
      // the values of the last tile end the order
      const bool issue = n_items < all;
      const bool values = n_items > 0 && ((n_items & 1) == 0 || n_items + 1 == all);
      const bool seg_begin = issue && !values && (n_items == 0 || next.kt == 0);
      // what is in flight lands and is given on: all of it before a segment's queries, which wait for its products
      const uint32_t keep = !issue || seg_begin ? 0u : static_cast<uint32_t>(C::kAhead);
      while (ok && n_items - sent > keep) {
        const bool rows = (by_rows >> (n_items - 1 - sent)) & 1;
        if (rows) {
          if (keep == 0)
            wait_copies<0>();
          else
            wait_copies<C::kAhead>();
          __syncwarp();
        }
        const uint32_t it = sent++, slot = it % C::kSlots;
        if constexpr (INT8) {
          const uint32_t rs = it % C::kRawSlots;
          if (!rows) {
            if (!warp_wait(&bars->raw_full[rs], (raw_phase >> rs) & 1, abort, a.err)) { ok = false; break; }
            raw_phase ^= 1u << rs;
          }
          if (!warp_wait(&bars->empty[slot], ((it / C::kSlots) & 1) ^ 1, abort, a.err)) { ok = false; break; }
          const uint8_t* raw = smem + C::kOffRaw + rs * C::kRaw;
          uint8_t* op = smem + C::kOffRing + slot * C::kTile;
          uint4 w[kCh];
#pragma unroll
          for (int i = 0; i < kCh; ++i) w[i] = *reinterpret_cast<const uint4*>(raw + warp * 32 * D + (i * 32 + lane) * 16);
#pragma unroll
          for (int i = 0; i < kCh; ++i) {
            const int row = warp * 32 + i * kRows + lane / kCh, c = lane % kCh;
            const uint32_t ww[4] = {w[i].x ^ 0x80808080u, w[i].y ^ 0x80808080u, w[i].z ^ 0x80808080u, w[i].w ^ 0x80808080u};
            const uint4 h0 = make_uint4(codes_lo(ww[0]), codes_hi(ww[0]), codes_lo(ww[1]), codes_hi(ww[1]));
            const uint4 h1 = make_uint4(codes_lo(ww[2]), codes_hi(ww[2]), codes_lo(ww[3]), codes_hi(ww[3]));
            uint8_t* piece = op + (c >> 2) * C::kPiece + row * 128;
            const int o = (2 * c) & 7, first = (c >> 2) & 1;  // the two pieces' lanes start on different banks
            *reinterpret_cast<uint4*>(piece + (((o + first) ^ (row & 7)) << 4)) = first ? h1 : h0;
            *reinterpret_cast<uint4*>(piece + (((o + (first ^ 1)) ^ (row & 7)) << 4)) = first ? h0 : h1;
          }
          const bool keys = it == 0 || ((it & 1) && it + 1 < all);  // these came with their tile's scales
          const uint32_t ss = (it + 1) / 2 % C::kScaleSlots;
          if (keys) {
            float* sc = reinterpret_cast<float*>(smem + C::kOffScale + ss * C::kScaleSlot);
            sc[2 * kTK + key] = __log2f(sc[kTK + key]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->full[slot]);
            mbar_arrive(&bars->raw_empty[rs]);
            if (keys) mbar_arrive(&bars->sc_full[ss]);
          }
        } else if (rows) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->full[slot]);
        }
      }
      if (!ok || !issue) break;

      if (seg_begin) {
        // ---- the segment's description and its queries, one row per lane ----
        ++seg;
        if (threadIdx.x == 0) {
          Seg d;
          d.tiles = min(kc.sh.kt - kc.kt, tiles - (t_now + 1));
          d.kt0 = kc.kt;
          d.g = kc.g;
          d.rt = kc.rt;
          d.whole = kc.kt == 0 && d.tiles == kc.sh.kt;
          d.us = us;
          d.ku = kc.sh.ku;
          d.s = kc.s;
          bars->seg[seg % kMaxSegs] = d;
          mbar_arrive(&bars->seg_full[seg % kMaxSegs]);
        }
        if (seg > 0 && !warp_wait(&bars->q_empty, (seg - 1) & 1, abort, a.err)) { ok = false; break; }
        const int rows = min(kRT, kc.s.n * a.G - kc.rt * kRT);
        const int r = key;
        const bool live = r < rows;
        const int ri = kc.rt * kRT + (live ? r : 0);
        const int i = static_cast<int>(paged::quotient(ri, a.g_div)), hh = ri - i * a.G;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(kc.s.start + i) * a.q_stride +
                                                          static_cast<long long>(kc.g * a.G + hh) * D);
        float f = 1.f;
        if constexpr (INT8) {
          uint32_t mag = 0;
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) {
            const uint4 w = live ? src[c] : make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) mag = max(mag, max(u[x] & 0x7FFFu, (u[x] >> 16) & 0x7FFFu));
          }
          // 2^e with the row's largest magnitude in [2^14, 2^15) after x * 2^-e
          const int e = mag == 0 ? 0 : max(-110, min(113, static_cast<int>(mag >> 7) - 127 - 14));
          f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          bars->qfac[seg & 3][r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        }
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = live ? src[c] : make_uint4(0, 0, 0, 0);
          if constexpr (INT8) {
            auto half = [&](uint32_t u) { return half2_bits(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f); };
            w = make_uint4(half(w.x), half(w.y), half(w.z), half(w.w));
          }
          *reinterpret_cast<uint4*>(smem + (c >> 3) * C::kPiece + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
      }
      if (!values) {
        prev = now;
        now = next;
        ++t_now;
        if (++kc.kt == kc.sh.kt) {
          us += kc.sh.ku;
          kc.next_item(a, run.pad);
        }
        if (t_now + 1 < tiles) peek(next);
      }

      // ---- issue item n_items ----
      const bool back = values && n_items + 1 != all;  // values of the tile before
      const Tile x{back ? prev.b : now.b,     back ? prev.g : now.g,       back ? prev.kt : now.kt,
                   back ? prev.len : now.len, back ? prev.page : now.page, back ? prev.whole : now.whole};
      const uint32_t it = n_items++;
      const uint32_t slot = it % C::kSlots, rs = it % C::kRawSlots;
      const bool rows = !x.whole || __any_sync(0xffffffffu, static_cast<unsigned>(x.page) >= static_cast<unsigned>(a.n_pages));
      by_rows = by_rows << 1 | (rows ? 1u : 0u);
      if constexpr (!INT8) {
        if (!warp_wait(&bars->empty[slot], ((it / C::kSlots) & 1) ^ 1, abort, a.err)) { ok = false; break; }
      } else if (warp == 0) {  // all four warps have read the raw slot's last codes
        if (!warp_wait(&bars->raw_empty[rs], ((it / C::kRawSlots) & 1) ^ 1, abort, a.err)) { ok = false; break; }
      }
      const uint8_t* base = values ? a.vc : a.kc;
      const uint32_t scale_at = C::kOffScale + (t_now % C::kScaleSlots) * C::kScaleSlot;
      if (rows) {
        const int p = x.kt * kTK + key;
        int page = -1, at = 0;
        if (p < x.len) {
          page = table_at(x.b, p);
          at = x.g * a.page_size + (p - static_cast<int>(paged::quotient(p, a.page_div)) * a.page_size);
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
            page = -1;
            if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
          }
        }
        const uint32_t to = INT8 ? sbase + C::kOffRaw + rs * C::kRaw : sbase + C::kOffRing + slot * C::kTile;
        const long long mine = page >= 0 ? page * a.page_bytes + static_cast<long long>(at) * (kCh * 16) : -1;
        const int c = lane % kCh;
#pragma unroll 4
        for (int i = 0; i < 32 / kRows; ++i) {
          const int r = i * kRows + lane / kCh;  // of the warp's 32
          const long long off = __shfl_sync(0xffffffffu, mine, r);
          const int row = warp * 32 + r;
          const uint32_t dst = INT8 ? to + row * D + c * 16
                                    : to + (c >> 3) * C::kPiece + row * 128 + (((c & 7) ^ (row & 7)) << 4);
          cp16(dst, base + (off >= 0 ? off + c * 16 : 0), off >= 0 ? 16u : 0u);
        }
        if (INT8 && !values) {  // both scales of the tile, with its keys
          const long long so = page >= 0 ? static_cast<long long>(page) * a.Hkv * a.page_size + at : 0;
          const uint32_t n = page >= 0 ? 4u : 0u;
          cp4(sbase + scale_at + key * 4, a.ks + so, n);
          cp4(sbase + scale_at + kTK * 4 + key * 4, a.vs + so, n);
        }
      } else {
        const int slot_in_page = a.page_size > kTK ? (x.kt * kTK) & (a.page_size - 1) : 0;
        if constexpr (!INT8) {
          if (lane == 0) {
            if (warp == 0)
              mbar_arrive_expect_tx(&bars->full[slot], C::kTile);
            else
              mbar_arrive(&bars->full[slot]);
          }
          __syncwarp();
          if (warp == 0 && lane < pieces) {
            uint8_t* dst = smem + C::kOffRing + slot * C::kTile + lane * span * 128;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(dst + h * C::kPiece, values ? &tm_v : &tm_k, &bars->full[slot], 64 * h, slot_in_page, x.g, x.page);
          }
        } else if (warp == 0) {
          if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[rs], C::kRaw + (values ? 0 : 2 * kTK * 4));
          __syncwarp();
          if (lane < pieces) {
            const int at = x.g * a.page_size + slot_in_page;
            bulk_load(smem + C::kOffRaw + rs * C::kRaw + lane * span * D,
                      base + x.page * a.page_bytes + static_cast<long long>(at) * D, span * D, &bars->raw_full[rs]);
            if (!values) {
              const long long so = static_cast<long long>(x.page) * a.Hkv * a.page_size + at;
              bulk_load(smem + scale_at + lane * span * 4, a.ks + so, span * 4, &bars->raw_full[rs]);
              bulk_load(smem + scale_at + kTK * 4 + lane * span * 4, a.vs + so, span * 4, &bars->raw_full[rs]);
            }
          }
        }
      }
      commit_copies();
    }
    wait_copies<0>();
    if (*abort && warp == 0) {
      // let every bulk copy already issued land before the CTA exits
      for (uint32_t it = n_items > C::kSlots ? n_items - C::kSlots : 0; it < n_items; ++it) {
        if ((by_rows >> (n_items - 1 - it)) & 1) continue;
        if constexpr (INT8) {
          if (it >= sent) drain_wait(&bars->raw_full[it % C::kRawSlots], (raw_phase >> (it % C::kRawSlots)) & 1);
        } else {
          drain_wait(&bars->full[it % C::kSlots], (it / C::kSlots) & 1);
        }
      }
    }
  } else if (warp < kWarpSm0) {
    if (warp == kWarpMma && lane == 0 && tiles > 0) {
      // ======================= MMA issuer =======================
      const uint32_t idesc = idesc_f16(kRT, kTK, !INT8);
      const uint32_t idesc_pv = idesc_f16(kRT, D, !INT8) | kBMajorN;
      bool ok = true;
      RingPos ring;
      int s_seg = 0, s_left = 0;               // segment of the next scores, its tiles to go
      int p_seg = 0, p_left = 0, p_begin = 0;  // of the next product
      // step x: scores of tile x, then the product of tile x - 1 (so S_0, S_1, P V_0, S_2, P V_1, ...)
      for (int x = 0; ok && x <= tiles; ++x) {
        if (x < tiles) {
          if (s_left == 0) {
            if (!wait_for(&bars->seg_full[s_seg % kMaxSegs], (s_seg / kMaxSegs) & 1, abort, a.err)) break;
            s_left = bars->seg[s_seg % kMaxSegs].tiles;
            if (!wait_for(&bars->q_full, s_seg & 1, abort, a.err)) break;
          }
          if (!wait_for(&bars->full[ring.slot], ring.phase, abort, a.err)) break;
          tc_fence_after();
          const uint32_t k_s = sbase + C::kOffRing + ring.slot * C::kTile;
          const uint32_t d = tmem + static_cast<uint32_t>(x & 1) * kTK;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::kPiece + (kk & 3) * 32;
            mma_ss(d, sdesc_sw128(sbase + off), sdesc_sw128(k_s + off), idesc, kk > 0);
          }
          mma_commit(&bars->s_full[x & 1]);
          mma_commit(&bars->empty[ring.slot]);
          ring.advance(C::kSlots);
          if (--s_left == 0) {
            mma_commit(&bars->q_empty);
            ++s_seg;
          }
        }
        if (x == 0) continue;
        const int t = x - 1;
        if (p_left == 0) {
          p_left = bars->seg[p_seg % kMaxSegs].tiles;
          // the segment before has been read out of O
          if (p_seg > 0 && !wait_for(&bars->epi, (p_seg - 1) & 1, abort, a.err)) break;
        }
        if (!wait_for(&bars->full[ring.slot], ring.phase, abort, a.err)) break;
        if (!wait_for(&bars->p_full[t & 1], (t >> 1) & 1, abort, a.err)) break;
        tc_fence_after();
        const uint32_t v_s = sbase + C::kOffRing + ring.slot * C::kTile;
        const uint32_t p = tmem + static_cast<uint32_t>(t & 1) * kTK;  // two keys per column
        const uint32_t o = tmem + kColO + static_cast<uint32_t>(t & 1) * 128;
        const bool fresh = t - p_begin < 2;  // the group's first tile of the segment
#pragma unroll
        for (int kk = 0; kk < kTK / 16; ++kk)
          mma_ts(o, p + kk * 8, sdesc_mn_sw128(v_s + kk * 2048, C::kPiece), idesc_pv, !(fresh && kk == 0));
        mma_commit(&bars->empty[ring.slot]);
        ring.advance(C::kSlots);
        if (--p_left == 0) {
          mma_commit(&bars->o_full);
          ++p_seg;
          p_begin = t + 1;
        }
      }
      // every MMA has finished with shared and tensor memory before the CTA tears down
      mma_commit(&bars->drain);
      drain_wait(&bars->drain, 0);
    }
  } else {
    // ======================= softmax =======================
    const int grp = (warp - kWarpSm0) >> 2;  // tiles grp, grp + 2, ... of the run
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tmem + lane_bits + static_cast<uint32_t>(grp) * kTK;
    const uint32_t o_at = tmem + lane_bits + kColO + static_cast<uint32_t>(grp) * 128;
    bool ok = true;
    int t = 0;
    for (int seg = 0; ok && t < tiles; ++seg) {
      if (!warp_wait(&bars->seg_full[seg % kMaxSegs], (seg / kMaxSegs) & 1, abort, a.err)) break;
      const Seg& sg = bars->seg[seg % kMaxSegs];
      const int rows = min(kRT, sg.s.n * a.G - sg.rt * kRT);
      const int lim = row_limit(a, sg.s, sg.rt * kRT + min(r, rows - 1));
      const int end = t + sg.tiles;
      int left = lim - sg.kt0 * kTK;  // keys of the tile below it are seen
      float m = -INFINITY, l = 0.f, unit = -INFINITY, fac = a.scale_log2;
      bool any = false;
      for (; t < end; ++t, left -= kTK) {
        if ((t & 1) != grp) continue;
        if (!warp_wait(&bars->s_full[grp], (t >> 1) & 1, abort, a.err)) { ok = false; break; }
        const float* scales = nullptr;
        if constexpr (INT8) {
          if (!warp_wait(&bars->sc_full[t % C::kScaleSlots], (t / C::kScaleSlots) & 1, abort, a.err)) { ok = false; break; }
          scales = reinterpret_cast<const float*>(smem + C::kOffScale + (t % C::kScaleSlots) * C::kScaleSlot);
          // the query rows' factors were written before q_full, which the scores waited for
          fac = a.scale_log2 * bars->qfac[seg & 3][r];
        }
        tc_fence_after();
        const uint64_t fac2 = f32x2_pack(__float_as_uint(fac), __float_as_uint(fac));
        // 64 scores of the row, scaled (INT8) and masked.  Scores are read twice from tensor memory: all 128 at once
        // would not fit the registers.
        auto load_scores = [&](int h, uint32_t (&sv)[64]) {
          tmem_ld32(s_at + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld32(s_at + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_wait_ld();
          if constexpr (INT8) {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scales + 64 * h + i);
              const uint64_t x0 = f32x2_mul(f32x2_pack(sv[i], sv[i + 1]), f.x), x1 = f32x2_mul(f32x2_pack(sv[i + 2], sv[i + 3]), f.y);
              sv[i] = static_cast<uint32_t>(x0);
              sv[i + 1] = static_cast<uint32_t>(x0 >> 32);
              sv[i + 2] = static_cast<uint32_t>(x1);
              sv[i + 3] = static_cast<uint32_t>(x1 >> 32);
            }
          }
          const int lh = left - 64 * h;
          if (__any_sync(0xffffffffu, lh < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= lh) sv[i] = 0xff800000u;  // -inf
          }
        };
        // the row's maximum; INT8: also log2 of its largest e^score times value scale
        float top = -INFINITY, topv = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[64];
          load_scores(h, sv);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const int x = (i >> 1) & 2;
            mx[x] = fmaxf(fmaxf(mx[x], __uint_as_float(sv[i])), __uint_as_float(sv[i + 1]));
            mx[x + 1] = fmaxf(fmaxf(mx[x + 1], __uint_as_float(sv[i + 2])), __uint_as_float(sv[i + 3]));
            if constexpr (INT8) {
              const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(scales + 2 * kTK + 64 * h + i);
              const uint64_t y0 = f32x2_fma(f32x2_pack(sv[i], sv[i + 1]), fac2, g.x);
              const uint64_t y1 = f32x2_fma(f32x2_pack(sv[i + 2], sv[i + 3]), fac2, g.y);
              mv[0] = fmaxf(fmaxf(mv[0], lo32(y0)), hi32(y0));
              mv[1] = fmaxf(fmaxf(mv[1], lo32(y1)), hi32(y1));
            }
          }
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          topv = fmaxf(topv, fmaxf(mv[0], mv[1]));
        }
        top *= fac;
        float alpha = 1.f;  // what O is multiplied by
        float lift = 1.f;
        if constexpr (!INT8) {
          if (top > m + kRescaleLog2 || m == -INFINITY) {
            const float n = fmaxf(m, top);
            alpha = n == -INFINITY ? 1.f : ex2(m - n);  // 0 where nothing was seen before
            l *= alpha;
            m = n;
          }
        } else {
          const float n = fmaxf(m, top);
          l *= n == -INFINITY ? 1.f : ex2(m - n);
          m = n;
          // held within 2^100 of e^m so that the lift stays finite
          const float at = fmaxf(topv, m - 100.f);
          if (m != -INFINITY && at > unit + 1.f) {
            alpha = ex2(unit - at);  // 0 from -inf
            unit = at;
          }
          lift = unit == -INFINITY ? 0.f : ex2(m - unit + 14.f);
        }
        const float base = m == -INFINITY ? 0.f : m;
        if (any && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_grp holds this group's earlier products, all complete (see above)
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_ld32(o_at + i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(o_at + i, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
            tmem_st16(o_at + i + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
          }
        }
        any = true;
        // p = 2^(s fac - m), two keys per packed operation, its sum, and P over the first half of the group's S columns,
        // two keys a column
        const uint64_t neg2 = f32x2_pack(__float_as_uint(-base), __float_as_uint(-base));
        const uint64_t lift2 = f32x2_pack(__float_as_uint(lift), __float_as_uint(lift));
        uint64_t l2[2] = {0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[64];
          load_scores(h, sv);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            ulonglong2 w{};
            if constexpr (INT8) w = *reinterpret_cast<const ulonglong2*>(scales + kTK + 64 * h + i);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint64_t e2 = f32x2_fma(f32x2_pack(sv[i + 2 * x], sv[i + 2 * x + 1]), fac2, neg2);
              uint64_t p2 = f32x2_pack(__float_as_uint(ex2(lo32(e2))), __float_as_uint(ex2(hi32(e2))));
              l2[x] = f32x2_add(l2[x], p2);
              if constexpr (INT8) p2 = f32x2_mul(f32x2_mul(p2, x ? w.y : w.x), lift2);
              sv[i / 2 + x] = INT8 ? half2_bits(lo32(p2), hi32(p2)) : pack_bf16x2(lo32(p2), hi32(p2));
            }
          }
          tmem_st16(s_at + 32 * h, *reinterpret_cast<uint32_t(*)[16]>(&sv[0]));
          tmem_st16(s_at + 32 * h + 16, *reinterpret_cast<uint32_t(*)[16]>(&sv[16]));
        }
        const uint64_t ls = f32x2_add(l2[0], l2[1]);
        l += lo32(ls) + hi32(ls);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[grp]);
      }
      if (!ok) break;
      // ---- the segment's end: both groups' parts of a row meet ----
      const int par = seg & 1;
      bars->st_m[par][grp][r] = m;
      bars->st_l[par][grp][r] = l;
      bars->st_u[par][grp][r] = INT8 && unit != -INFINITY ? unit - m - 14.f : 0.f;
      bars->st_any[par][grp] = any;  // the same for all rows
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->fin[quarter]);
      if (!warp_wait(&bars->fin[quarter], par, abort, a.err)) break;
      if (!warp_wait(&bars->o_full, par, abort, a.err)) break;
      tc_fence_after();
      const float m0 = bars->st_m[par][0][r], m1 = bars->st_m[par][1][r];
      const float M = fmaxf(m0, m1);  // a group without tiles has -inf
      const float bs = M == -INFINITY ? 0.f : M;
      const float L = ex2(m0 - bs) * bars->st_l[par][0][r] + ex2(m1 - bs) * bars->st_l[par][1][r];
      const bool whole = sg.whole != 0;
      const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
      const float f0 = ex2(m0 - bs + bars->st_u[par][0][r]) * inv, f1 = ex2(m1 - bs + bars->st_u[par][1][r]) * inv;
      const bool has0 = bars->st_any[par][0] != 0, has1 = bars->st_any[par][1] != 0;
      const size_t row = out_row<kRT>(a, sg.s, sg.g, sg.rt, min(r, rows - 1));
      const int which = sg.kt0 > 0 ? 0 : 1;
      const long long pslot = 2ll * blockIdx.x + which;
      // group g writes columns g D/2 ... of its quarter's rows, 16 at a time
#pragma unroll 1
      for (int i = 0; i < D / 2; i += 16) {
        const int col = grp * (D / 2) + i;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        uint32_t o[16];
        if (has0) {
          tmem_ld16(tmem + lane_bits + kColO + col, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * f0;
        }
        if (has1) {
          tmem_ld16(tmem + lane_bits + kColO + 128 + col, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = fmaf(__uint_as_float(o[e]), f1, v[e]);
        }
        if (r < rows) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + col);
            dst[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                pack_bf16x2(v[6], v[7]));
            dst[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                                pack_bf16x2(v[14], v[15]));
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (pslot * kRT + r) * D + col);
#pragma unroll
            for (int e = 0; e < 4; ++e) __stcg(dst + e, make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
          }
        }
      }
      if (r < rows && grp == 0) {
        if (!whole)
          __stcg(a.part_ml + pslot * kRT + r, make_float2(M, L));
        else if (a.lse)
          a.lse[row] = (M + log2f(L)) * kLn2;
      }
      if (!whole && warp == kWarpSm0 && lane == 0) {
        bars->part[which] = sg;
        bars->has_part[which] = 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->epi);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (a.fused && !*abort) {
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      if (!bars->has_part[x]) continue;
      const Seg sg = bars->part[x];
      const Span sp = span_of(sg.us, sg.ku, run.per);
      if (!all_arrived(a, sp, run.per, 2ll * blockIdx.x + x)) continue;
      const int rows = min(kRT, sg.s.n * a.G - sg.rt * kRT);
      float* scratch = reinterpret_cast<float*>(smem) + threadIdx.x / (D / 4) * 2 * kJoinBatch;
      for (int r = threadIdx.x / (D / 4); r < rows; r += kThreads / (D / 4))
        join_row<D, kRT>(a, sg.s, sp, run.per, sg.g, sg.rt, r, scratch);
      clear_arrivals(a, sp, run.per);
    }
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
