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
//   warps 0-3   loaders.  Each owns 32 keys of every 128-key tile: looks up
//               their pages, copies their rows (16-byte cp.async) into operand
//               tiles of the 128-byte-swizzle layout, and fences them to the
//               tensor cores' proxy.  INT8: rows land in a raw ring first and
//               are rewritten as FP16 codes (exact).  Also the query tile.
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

#include "mnw_attn_split.cuh"

namespace mnw {
namespace pattn {
namespace {

constexpr int kRT = kBlockRows, kTK = kBlockKeys;
constexpr int kThreads = 512;
// registers a thread of the four warpgroups: the kernel is built for 128 each, and 88 + 56 + 2 * 184 = 4 * 128
constexpr int kLoadWarps = 4, kWarpMma = 4, kWarpSm0 = 8;
constexpr int kTmemCols = 512;
constexpr uint32_t kColO = 256;  // O_g at kColO + 128 g; S_g at 128 g
constexpr int kSegs = 2;         // parity slots of per-segment exchanges
constexpr int kMaxScaleSlots = 8;
constexpr float kRescaleLog2 = 8.f;

template <int D, bool INT8>
struct BCfg {
  static constexpr int kHalves = D / 64;                   // 64 elements = 128 bytes per operand row piece
  static constexpr uint32_t kPiece = kTK * 128;            // 128 rows of 128 bytes
  static constexpr uint32_t kTile = kHalves * kPiece;      // operand tile
  static constexpr int kSlots = D == 64 ? 8 : (INT8 ? 4 : 5);
  static constexpr int kAhead = 2;                         // copies in flight behind the one being issued
  // the scales of tile t + kScaleSlots are copied once P V of tile t was issued: the copy of keys t + n (item 2 (t + n) - 1)
  // follows the release of the operand slot kAhead + 1 + kSlots items before it, and values of tile j are item 2 j + 2
  static constexpr int kScaleSlots = kSlots == 8 ? 8 : 6;
  static_assert(2 * kScaleSlots - 1 - (kAhead + 1) - kSlots >= 2 && kScaleSlots <= kMaxScaleSlots);
  static constexpr uint32_t kRaw = INT8 ? kTK * D : 0;     // raw codes of a tile
  static constexpr int kRawSlots = kAhead + 1;
  static constexpr uint32_t kOffRing = kTile;              // Q first
  static constexpr uint32_t kOffRaw = kOffRing + kSlots * kTile;
  static constexpr uint32_t kOffScale = kOffRaw + kRawSlots * kRaw;
  static constexpr uint32_t kOffBars = kOffScale + (INT8 ? kScaleSlots * 2 * kTK * 4 : 0);
};

struct Bars {
  uint64_t full[8], empty[8];           // operand ring
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2];        // per softmax group
  uint64_t o_full, epi;                 // a segment's output complete; read
  uint64_t sc_full[kMaxScaleSlots];
  uint64_t fin[4];                      // per lane quarter: both groups' maxima and sums written
  uint64_t drain;
  float4 st[kSegs][2][kRT];             // [segment parity][group][row]: maximum, sum, unit of O, any tiles
  float qfac[4][kRT];                   // [segment % 4] INT8: the query rows' powers of two (up to three segments are live)
  uint32_t tmem_base;
  int abort;
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
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = bounded_wait(bar, parity, abort, err) ? 1 : 0;
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

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1) paged_block_kernel(const Args a) {
  using C = BCfg<D, INT8>;
  using Cur = Cursor<kRT, kTK>;
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
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->epi, 8);
    for (int i = 0; i < kMaxScaleSlots; ++i) mbar_init(&bars->sc_full[i], kLoadWarps);
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
  Cur cur{};
  int tiles = 0;
  if (run.seq >= 0) {
    cur.set(a, run);
    tiles = run.pad == 1 ? run.u1 - run.u0 : min(run.u1 - run.u0, cur.sh.kt - cur.kt);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < kLoadWarps) {
    // ======================= loaders =======================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    bool ok = true;
    const int key = warp * 32 + lane;  // this lane's key of a tile
    Cur kc = cur, vc = cur;            // tiles whose keys, values come next
    int n_items = 0, seg = -1;
    uint32_t sent = 0;                 // items whose arrival was given
    // a warp's page offsets: (page, head row) of its lane's key
    auto look = [&](const Cur& c, int& page, int& at) {
      const int p = c.kt * kTK + key;
      page = -1;
      at = 0;
      if (p < c.s.len) {
        const int pi = static_cast<int>(paged::quotient(p, a.page_div));
        page = __ldg(a.bt.block_table + static_cast<size_t>(c.b) * a.bt.max_pages + pi);
        at = c.g * a.page_size + (p - pi * a.page_size);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
          page = -1;
          if (a.err) atomicOr(a.err, MNW_DEVERR_BAD_PAGE);
        }
      }
    };
    constexpr int kCh = (INT8 ? D : 2 * D) / 16;  // chunks of a cached row
    constexpr int kRows = 32 / kCh;               // rows per pass of the warp
    auto copy_rows = [&](const uint8_t* base, uint32_t to, int page, int at) {
      const long long mine = page >= 0 ? page * a.page_bytes + static_cast<long long>(at) * (kCh * 16) : -1;
      const int c = lane % kCh;
#pragma unroll 8
      for (int i = 0; i < 32 / kRows; ++i) {
        const int r = i * kRows + lane / kCh;  // of the warp's 32
        const long long off = __shfl_sync(0xffffffffu, mine, r);
        const int row = warp * 32 + r;
        uint32_t dst;
        if constexpr (INT8)
          dst = to + row * D + c * 16;
        else
          dst = to + (c >> 3) * C::kPiece + row * 128 + (((c & 7) ^ (row & 7)) << 4);
        cp16(dst, base + (off >= 0 ? off + c * 16 : 0), off >= 0 ? 16u : 0u);
      }
    };
    // gives item `it` to the tensor cores: its copies have landed
    auto send = [&](uint32_t it) -> bool {
      const uint32_t slot = it % C::kSlots;
      if constexpr (INT8) {
        if (!warp_wait(&bars->empty[slot], ((it / C::kSlots) & 1) ^ 1, abort, a.err)) return false;
        const uint8_t* raw = smem + C::kOffRaw + (it % C::kRawSlots) * C::kRaw;
        uint8_t* op = smem + C::kOffRing + slot * C::kTile;
        __syncwarp();  // the warp's copies are visible to its lanes
#pragma unroll 2
        for (int i = 0; i < kCh; ++i) {
          const int x = i * 32 + lane, row = warp * 32 + x / kCh, c = x % kCh;
          const uint4 w = *reinterpret_cast<const uint4*>(raw + row * D + c * 16);
          const uint32_t ww[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
          uint4 h[2];
          h[0] = make_uint4(codes_lo(ww[0]), codes_hi(ww[0]), codes_lo(ww[1]), codes_hi(ww[1]));
          h[1] = make_uint4(codes_lo(ww[2]), codes_hi(ww[2]), codes_lo(ww[3]), codes_hi(ww[3]));
          uint8_t* piece = op + (c >> 2) * C::kPiece + row * 128;
          const int o = (2 * c) & 7, first = (c >> 2) & 1;  // the two pieces' lanes start on different banks
          *reinterpret_cast<uint4*>(piece + (((o + first) ^ (row & 7)) << 4)) = first ? h[1] : h[0];
          *reinterpret_cast<uint4*>(piece + (((o + (first ^ 1)) ^ (row & 7)) << 4)) = first ? h[0] : h[1];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->full[slot]);
      return true;
    };
    // all copies issued so far are given on
    auto flush = [&]() -> bool {
      wait_copies<0>();
      bool good = true;
      while (good && sent < static_cast<uint32_t>(n_items)) good = send(sent++);
      return good;
    };
    auto load_q = [&]() -> bool {
      ++seg;
      if (seg > 0) {
        if (!flush()) return false;  // the scores before this segment's wait for them
        if (!warp_wait(&bars->q_empty, (seg - 1) & 1, abort, a.err)) return false;
      }
      const int rows = min(kRT, kc.s.n * a.G - kc.rt * kRT);
      // one query row per lane: row 32 warp + lane
      const int r = key;
      const bool live = r < rows;
      const int ri = kc.rt * kRT + (live ? r : 0);
      const int i = static_cast<int>(paged::quotient(ri, a.g_div)), hh = ri - i * a.G;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(kc.s.start + i) * a.q_stride +
                                                        static_cast<long long>(kc.g * a.G + hh) * D);
      float f = 1.f;
      if constexpr (INT8) {
        uint32_t mag = 0;
#pragma unroll 4
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
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        uint4 w = live ? src[c] : make_uint4(0, 0, 0, 0);
        if constexpr (INT8) {
          uint32_t* u = &w.x;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            u[x] = half2_bits(__uint_as_float(u[x] << 16) * f, __uint_as_float(u[x] & 0xFFFF0000u) * f);
        }
        *reinterpret_cast<uint4*>(smem + (c >> 3) * C::kPiece + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_full);
      return true;
    };
    // items in the order of their products: K_0, K_1, V_0, K_2, V_1, ...
    auto load_item = [&](bool values, int t) -> bool {
      Cur& c = values ? vc : kc;
      int page, at;
      look(c, page, at);
      const uint32_t it = n_items++;
      if constexpr (!INT8) {
        if (!warp_wait(&bars->empty[it % C::kSlots], ((it / C::kSlots) & 1) ^ 1, abort, a.err)) return false;
        copy_rows(values ? a.vc : a.kc, sbase + C::kOffRing + (it % C::kSlots) * C::kTile, page, at);
      } else {
        copy_rows(values ? a.vc : a.kc, sbase + C::kOffRaw + (it % C::kRawSlots) * C::kRaw, page, at);
        if (!values) {  // both scales of the tile, with its keys
          const long long so = page >= 0 ? static_cast<long long>(page) * a.Hkv * a.page_size + at : 0;
          const uint32_t n = page >= 0 ? 4u : 0u;
          const uint32_t to = sbase + C::kOffScale + (t % C::kScaleSlots) * (2 * kTK * 4) + key * 4;
          cp4(to, a.ks + so, n);
          cp4(to + kTK * 4, a.vs + so, n);
        }
      }
      commit_copies();
      if (++c.kt == c.sh.kt) c.next_item(a, run.pad);
      if (n_items - static_cast<int>(sent) > C::kAhead) {
        wait_copies<C::kAhead>();
        return send(sent++);
      }
      return true;
    };
    // the scales of tile t are in shared memory once its keys' item was sent
    int keys_sent = 0;
    auto tell_scales = [&]() {
      if constexpr (INT8) {
        // items 0, 1 are keys, then values and keys alternate: item i >= 2 is keys if odd
        while (keys_sent < tiles) {
          const uint32_t it = keys_sent < 2 ? keys_sent : 2 * keys_sent - 1;
          if (it >= sent) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->sc_full[keys_sent % C::kScaleSlots]);
          ++keys_sent;
        }
      }
    };
    for (int t = 0; ok && t < tiles + 1; ++t) {
      if (t < tiles) {
        if (t == 0 || kc.kt == 0) ok = load_q();
        if (ok) ok = load_item(false, t);
        tell_scales();
      }
      if (ok && t >= 1) {
        ok = load_item(true, t - 1);
        tell_scales();
      }
    }
    if (ok) {
      flush();
      tell_scales();
    }
    wait_copies<0>();
  } else if (warp < kWarpSm0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kWarpMma && lane == 0 && tiles > 0) {
      // ======================= MMA issuer =======================
      const uint32_t idesc = idesc_f16(kRT, kTK, !INT8);
      const uint32_t idesc_pv = idesc_f16(kRT, D, !INT8) | kBMajorN;
      bool ok = true;
      uint32_t item = 0;
      // place of tile ts (scores) and tp (products) in their segments
      Cur sc = cur, pc = cur;
      int s_seg = 0, p_seg = 0, p_begin = 0, q_seen = -1;
      auto issue_s = [&](int t) -> bool {
        if (q_seen != s_seg) {
          if (!bounded_wait(&bars->q_full, s_seg & 1, abort, a.err)) return false;
          q_seen = s_seg;
        }
        const uint32_t slot = item % C::kSlots;
        if (!bounded_wait(&bars->full[slot], (item / C::kSlots) & 1, abort, a.err)) return false;
        tc_fence_after();
        const uint32_t k_s = sbase + C::kOffRing + slot * C::kTile;
        const uint32_t d = tmem + static_cast<uint32_t>(t & 1) * kTK;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kPiece + (kk & 3) * 32;
          mma_ss(d, sdesc_sw128(sbase + off), sdesc_sw128(k_s + off), idesc, kk > 0);
        }
        mma_commit(&bars->empty[slot]);
        mma_commit(&bars->s_full[t & 1]);
        ++item;
        const bool last = sc.kt + 1 == sc.sh.kt;
        if (last) {
          mma_commit(&bars->q_empty);
          ++s_seg;
        }
        if (++sc.kt == sc.sh.kt) sc.next_item(a, run.pad);
        return true;
      };
      auto issue_pv = [&](int t) -> bool {
        if (t == p_begin && p_seg > 0) {  // the segment before has been read out of O
          if (!bounded_wait(&bars->epi, (p_seg - 1) & 1, abort, a.err)) return false;
        }
        if (!bounded_wait(&bars->p_full[t & 1], (t >> 1) & 1, abort, a.err)) return false;
        const uint32_t slot = item % C::kSlots;
        if (!bounded_wait(&bars->full[slot], (item / C::kSlots) & 1, abort, a.err)) return false;
        tc_fence_after();
        const uint32_t v_s = sbase + C::kOffRing + slot * C::kTile;
        const uint32_t p = tmem + static_cast<uint32_t>(t & 1) * kTK;  // two keys per column
        const uint32_t o = tmem + kColO + static_cast<uint32_t>(t & 1) * 128;
        const bool fresh = t - p_begin < 2;
#pragma unroll
        for (int kk = 0; kk < kTK / 16; ++kk)
          mma_ts(o, p + kk * 8, sdesc_mn_sw128(v_s + kk * 2048, C::kPiece), idesc_pv, !(fresh && kk == 0));
        mma_commit(&bars->empty[slot]);
        ++item;
        if (pc.kt + 1 == pc.sh.kt || t + 1 == tiles) {
          mma_commit(&bars->o_full);
          ++p_seg;
          p_begin = t + 1;
        }
        if (++pc.kt == pc.sh.kt) pc.next_item(a, run.pad);
        return true;
      };
      ok = issue_s(0);
      if (ok && tiles > 1) ok = issue_s(1);
      for (int t = 0; ok && t < tiles; ++t) {
        ok = issue_pv(t);
        if (ok && t + 2 < tiles) ok = issue_s(t + 2);
      }
      // every MMA has finished with shared and tensor memory before the CTA tears down
      mma_commit(&bars->drain);
      drain_wait(&bars->drain, 0);
    }
  } else {
    // ======================= softmax =======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int grp = (warp - kWarpSm0) >> 2;  // tiles grp, grp + 2, ... of the run
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tmem + lane_bits + static_cast<uint32_t>(grp) * kTK;
    const uint32_t o_at = tmem + lane_bits + kColO + static_cast<uint32_t>(grp) * 128;
    Cur c = cur;
    bool ok = true;
    int seg = 0, begin = 0;  // segment and its first tile (of the run)
    int kt_begin = c.kt, lim = 0, rows = 0;
    float m = -INFINITY, l = 0.f, unit = -INFINITY, fac = a.scale_log2;
    bool any = false;
    for (int t = 0; ok && t < tiles; ++t) {
      if (t == begin) {
        kt_begin = c.kt;
        rows = min(kRT, c.s.n * a.G - c.rt * kRT);
        lim = row_limit(a, c.s, c.rt * kRT + min(r, rows - 1));
        m = unit = -INFINITY;
        l = 0.f;
        any = false;
      }
      const bool last = c.kt + 1 == c.sh.kt || t + 1 == tiles;
      if ((t & 1) == grp) {
        const int k = t >> 1;
        if (!warp_wait(&bars->s_full[grp], k & 1, abort, a.err)) { ok = false; break; }
        const float* scales = nullptr;
        if constexpr (INT8) {
          if (!warp_wait(&bars->sc_full[t % C::kScaleSlots], (t / C::kScaleSlots) & 1, abort, a.err)) { ok = false; break; }
          scales = reinterpret_cast<const float*>(smem + C::kOffScale + (t % C::kScaleSlots) * (2 * kTK * 4));
          // the query rows' factors were written before q_full, which the scores waited for
          fac = a.scale_log2 * bars->qfac[seg & 3][r];
        }
        tc_fence_after();
        uint32_t sv[kTK];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * i]));
        tmem_wait_ld();
        if constexpr (INT8) {
#pragma unroll
          for (int i = 0; i < kTK; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + i);
            sv[i] = __float_as_uint(__uint_as_float(sv[i]) * f.x);
            sv[i + 1] = __float_as_uint(__uint_as_float(sv[i + 1]) * f.y);
            sv[i + 2] = __float_as_uint(__uint_as_float(sv[i + 2]) * f.z);
            sv[i + 3] = __float_as_uint(__uint_as_float(sv[i + 3]) * f.w);
          }
        }
        const int left = lim - c.kt * kTK;  // keys below it are seen
        if (__any_sync(0xffffffffu, left < kTK)) {
#pragma unroll
          for (int i = 0; i < kTK; ++i)
            if (i >= left) sv[i] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kTK; i += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mx[x] = fmaxf(fmaxf(mx[x], __uint_as_float(sv[i + 2 * x])), __uint_as_float(sv[i + 2 * x + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * fac;
        float alpha = 1.f;  // what O is multiplied by
        if constexpr (!INT8) {
          if (!any || top > m + kRescaleLog2 || m == -INFINITY) {
            const float n = fmaxf(m, top);
            const float d = n == -INFINITY ? 1.f : ex2(m - n);  // 0 where nothing was seen before
            alpha = d;
            l *= d;
            m = n;
          }
        } else {
          const float n = fmaxf(m, top);
          l *= n == -INFINITY ? 1.f : ex2(m - n);
          m = n;
        }
        const float base = m == -INFINITY ? 0.f : m;
        // p = 2^(s fac - m), two keys per packed operation, and its sum
        const uint64_t fac2 = f32x2_pack(__float_as_uint(fac), __float_as_uint(fac));
        const uint64_t neg2 = f32x2_pack(__float_as_uint(-base), __float_as_uint(-base));
        uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < kTK; i += 2) {
          const uint64_t e2 = f32x2_fma(f32x2_pack(sv[i], sv[i + 1]), fac2, neg2);
          sv[i] = __float_as_uint(ex2(__uint_as_float(static_cast<uint32_t>(e2))));
          sv[i + 1] = __float_as_uint(ex2(__uint_as_float(static_cast<uint32_t>(e2 >> 32))));
          l2[(i >> 1) & 1] = f32x2_add(l2[(i >> 1) & 1], f32x2_pack(sv[i], sv[i + 1]));
        }
        const uint64_t ls = f32x2_add(l2[0], l2[1]);
        l += __uint_as_float(static_cast<uint32_t>(ls)) + __uint_as_float(static_cast<uint32_t>(ls >> 32));
        float lift = 1.f;
        if constexpr (INT8) {
          float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kTK; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + kTK + i);
            const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float p = __uint_as_float(sv[i + x]) * w[x];
              sv[i + x] = __float_as_uint(p);
              y[x] = fmaxf(y[x], p);
            }
          }
          const float big = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
          // log2 of the row's largest product, held within 2^100 of e^m so that the lift stays finite
          const float at = fmaxf(base + __log2f(big), base - 100.f);
          if (m != -INFINITY && at > unit + 1.f) {
            alpha = ex2(unit - at);  // 0 from -inf
            unit = at;
          }
          lift = unit == -INFINITY ? 0.f : ex2(base - unit + 14.f);
        }
        if (any && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_grp holds this group's earlier products, all complete (see above)
#pragma unroll
          for (int i = 0; i < D; i += 16) {
            uint32_t o[16];
            tmem_ld16(o_at + i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(o_at + i, o);
          }
        }
        any = true;
        // P over the first half of the group's S columns, two keys a column
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = __uint_as_float(sv[32 * i + 2 * e]), p1 = __uint_as_float(sv[32 * i + 2 * e + 1]);
            pk[e] = INT8 ? half2_bits(p0 * lift, p1 * lift) : pack_bf16x2(p0, p1);
          }
          tmem_st16(s_at + 16 * i, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[grp]);
      }
      if (last) {
        // ---- the segment's end: both groups' parts of a row meet ----
        const float to_m = INT8 ? (unit == -INFINITY ? 0.f : unit - m - 14.f) : 0.f;  // log2 of O's unit over 2^m
        bars->st[seg & 1][grp][r] = make_float4(m, l, to_m, any ? 1.f : 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->fin[quarter]);
        if (!warp_wait(&bars->fin[quarter], seg & 1, abort, a.err)) { ok = false; break; }
        if (!warp_wait(&bars->o_full, seg & 1, abort, a.err)) { ok = false; break; }
        tc_fence_after();
        const float4 s0 = bars->st[seg & 1][0][r], s1 = bars->st[seg & 1][1][r];
        const float M = fmaxf(s0.x, s1.x);  // a group without tiles has -inf
        const float bs = M == -INFINITY ? 0.f : M;
        const float w0 = ex2(s0.x - bs), w1 = ex2(s1.x - bs);
        const float L = w0 * s0.y + w1 * s1.y;
        const bool whole = kt_begin == 0 && c.kt + 1 == c.sh.kt;
        const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
        const float f0 = ex2(s0.x - bs + s0.z) * inv, f1 = ex2(s1.x - bs + s1.z) * inv;
        const bool has0 = s0.w != 0.f, has1 = s1.w != 0.f;  // the same for all rows
        const size_t row = out_row<kRT>(a, c.s, c.g, c.rt, min(r, rows - 1));
        const long long pslot = 2ll * blockIdx.x + (kt_begin > 0 ? 0 : 1);
        // group g writes columns g D/2 ... of its quarter's rows, 16 at a time
#pragma unroll
        for (int i = 0; i < D / 2; i += 16) {
          const int col = grp * (D / 2) + i;
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.f;
          if (has0) {
            uint32_t o[16];
            tmem_ld16(tmem + lane_bits + kColO + col, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * f0;
          }
          if (has1) {
            uint32_t o[16];
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->epi);
        ++seg;
        begin = t + 1;
      }
      if (++c.kt == c.sh.kt) c.next_item(a, run.pad);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
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
    attrs_done(attr, bit);
  }
  return launch_pdl(kern, dim3(runs), dim3(kThreads), kSmem, st, a) == cudaSuccess ? MNW_OK : MNW_E_CUDA;
}

}  // namespace

int launch_block(const Args& a, int d, bool int8, int runs, cudaStream_t st) {
  if (d == 128) return int8 ? launch<128, true>(a, runs, st) : launch<128, false>(a, runs, st);
  return int8 ? launch<64, true>(a, runs, st) : launch<64, false>(a, runs, st);
}

}  // namespace pattn
}  // namespace mnw
