// mnw_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = bf16(y[t] + s_i B_i (A_i x[t])),   i = adapter[t]
// y is the shared projection's output; a token of adapter -1 keeps y.
//
// The inner product v = A_i x is summed in FP32 and enters the second product
// as two BF16 terms (v to 2^-16), so the output's rounding is the only one that
// counts.
//
// Bound: x, y and the adapters in use are read once and out is written once, 2 R
// flops a byte at most, so memory is the floor for many tokens; for few it is
// the chain adapter -> tokens -> x and A -> v -> out.  Two forms:
//  - for few tokens (few_tokens() below) one kernel, a cluster of eight CTAs per
//    tile of 32 or 16 tokens of one adapter, each of which finds its tile by itself;
//  - above, three: tokens are listed by adapter, v = A x and out = y + s B v on
//    tcgen05 with 128 tokens a tile.
// Each token's result depends on its own row alone, so it is the same however
// tokens are arranged.
//
// Measured on one GB300 (device time in a replayed graph; one kernel and three):
// 64 tokens of 24 adapters, H = 4096, N = 5120, R = 16: 6.0 us by one.  9000 tokens
// of 4 adapters, R = 64 (262 MB): 65 us by three, 4.0 TB/s; alone and cold the first
// product takes 22, the second 45; with warp-level products they took 28 and 68.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "mnw_convert.cuh"
#include "mnw_internal.h"
#include "mnw_ptx.cuh"

namespace mnw {
namespace lora {

struct Args {
  const __nv_bfloat16 *x, *a, *b, *y;
  __nv_bfloat16* out;
  long long x_stride, y_stride, out_stride;
  const float* scale;      // [n] or null: 1
  const int32_t* ranks;    // [n] or null: R
  const int32_t* adapter;  // [T]
  int n, R, T, H, N;
  int splits;              // of H in the first product
  int spans;               // shares of N in the second
  // workspace
  int32_t* starts;   // [n + 2] first place of each adapter's tokens in `order`, of those without one, and T
  int32_t* order;    // [T] tokens grouped by adapter
  float* v;          // [splits][T][padded R], by place
  uint32_t* err;
};

__device__ __forceinline__ int bin_of(const Args& a, int t) {
  const int id = __ldg(a.adapter + t);
  return static_cast<unsigned>(id) < static_cast<unsigned>(a.n) ? id : a.n;
}
__device__ __forceinline__ int checked_rank(const Args& a, int r) {
  if (static_cast<unsigned>(r) > static_cast<unsigned>(a.R)) {
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, MNW_DEVERR_BAD_ADAPTER);
    return r < 0 ? 0 : a.R;
  }
  return r;
}
__device__ __forceinline__ int rank_of(const Args& a, int i) { return checked_rank(a, a.ranks ? __ldcg(a.ranks + i) : a.R); }

// ---- grouping: CTA e lists the tokens of adapter e (e = n: of none) ----
constexpr int kGroupThreads = 1024, kRun = 16;  // tokens of a thread at a time
__global__ void __launch_bounds__(kGroupThreads) lora_group_kernel(const Args a) {
  constexpr int kWarps = kGroupThreads / 32;
  static_assert(kWarps == 32);
  __shared__ int sums[kRun][kWarps + 1], befores[kWarps], totals[kRun];
  pdl_wait();
  pdl_launch_dependents();
  const int e = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Adapters of lower numbers come first; with more tokens than the threads take at a time, theirs are counted beforehand.
  const bool once = a.T <= kGroupThreads * kRun;
  int start = 0, done = 0;
  if (!once) {
    int before = 0;
#pragma unroll 8
    for (int t = tid; t < a.T; t += kGroupThreads) before += bin_of(a, t) < e ? 1 : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) befores[warp] = before;
    __syncthreads();
    start = __reduce_add_sync(0xffffffffu, befores[lane]);
  }
  for (int t0 = 0; t0 < a.T; t0 += kGroupThreads * kRun) {
    int id[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int t = t0 + i * kGroupThreads + tid;
      id[i] = t < a.T ? __ldg(a.adapter + t) : INT_MAX;
    }
    uint32_t bits = 0;  // which of this thread's tokens are the adapter's
    int before = 0, warp_sum = 0;
    __syncthreads();  // the sums before are read
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (t0 + i * kGroupThreads >= a.T) break;
      const bool on = t0 + i * kGroupThreads + tid < a.T;
      const int bin = static_cast<unsigned>(id[i]) < static_cast<unsigned>(a.n) ? id[i] : a.n;
      const bool is = on && bin == e;
      bits |= (is ? 1u : 0u) << i;
      before += on && bin < e ? 1 : 0;
      if (is && e == a.n && id[i] != -1 && a.err) atomicOr(a.err, MNW_DEVERR_BAD_ADAPTER);
      const int c = __popc(__ballot_sync(0xffffffffu, is));
      if (lane == i) warp_sum = c;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane < kRun) sums[lane][warp] = warp_sum;
    if (lane == 0) befores[warp] = before;
    __syncthreads();
    if (warp < kRun && t0 + warp * kGroupThreads < a.T) {  // a warp per row of sums
      const int m = sums[warp][lane];
      int incl = m;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      sums[warp][lane] = incl - m;
      if (lane == 31) totals[warp] = incl;
    }
    __syncthreads();
    if (once) start = __reduce_add_sync(0xffffffffu, befores[lane]);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (t0 + i * kGroupThreads >= a.T) break;
      const bool is = bits >> i & 1;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      if (is) a.order[start + done + sums[i][warp] + __popc(m & ((1u << lane) - 1u))] = t0 + i * kGroupThreads + tid;
      done += totals[i];
    }
  }
  if (tid == 0) {
    a.starts[e] = start;
    if (e == a.n) a.starts[e + 1] = a.T;
  }
}

// ---- tiles of kTT tokens of one adapter ----
// Adapter e's tiles are numbered from starts[e] / kTT + e on, which leaves room for each (a few numbers stay unused).
constexpr int kTT = 128, kThreads = 256;
struct Tile {
  int bin, first, count;  // adapter (n: none), place of the first token, tokens (0: no such tile)
};
__device__ __forceinline__ Tile find_tile(const Args& a, int q, Tile* sh) {
  if (threadIdx.x == 0) sh->count = 0;
  __syncthreads();
  for (int e = threadIdx.x; e <= a.n; e += blockDim.x) {
    const int lo = __ldcg(a.starts + e), hi = __ldcg(a.starts + e + 1);
    const int j = q - (lo / kTT + e);
    if (j >= 0 && j * kTT < hi - lo) *sh = Tile{e, lo + j * kTT, min(kTT, hi - lo - j * kTT)};
  }
  __syncthreads();
  return *sh;
}
inline int tile_numbers(int T, int n) { return T / kTT + n + 1; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// v as two BF16 terms: the nearest (no further than BF16's largest, for finite ones that lie past it), and what that leaves,
// nothing of an infinite one.
__device__ __forceinline__ float first_of(float v) {
  constexpr float kMost = 0x1.FEp127f;
  return fabsf(v) < INFINITY ? fminf(fmaxf(v, -kMost), kMost) : v;
}
__device__ __forceinline__ float rest_of(float v, uint32_t first) {
  const float r = v - __uint_as_float(first);
  return fabsf(r) < INFINITY ? r : 0.f;
}
__device__ __forceinline__ void terms_of(float4 v, uint2& first, uint2& rest) {
  first = make_uint2(pack_bf16x2(first_of(v.x), first_of(v.y)), pack_bf16x2(first_of(v.z), first_of(v.w)));
  rest = make_uint2(pack_bf16x2(rest_of(v.x, first.x << 16), rest_of(v.y, first.x & 0xFFFF0000u)),
                    pack_bf16x2(rest_of(v.z, first.y << 16), rest_of(v.w, first.y & 0xFFFF0000u)));
}
// The ranks that count, of the 4 from e on (an infinite x times the zeros of the others would be NaN).
__device__ __forceinline__ float4 ranks_of(float4 v, int e, int rank) {
  return make_float4(e < rank ? v.x : 0.f, e + 1 < rank ? v.y : 0.f, e + 2 < rank ? v.z : 0.f, e + 3 < rank ? v.w : 0.f);
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- v = A x on tcgen05: a tile of tokens and a share of H ----
// Tokens are the rows of the product, ranks its columns.  Steps of 64 elements of H arrive by cp.async in the operands'
// 128-byte swizzle; one thread issues the instructions, and the sums lie in tensor memory until the end.  The warps do
// nothing but copy.
template <int NR>
struct ShrinkCfg {
  static constexpr int kStages = 4;
  static constexpr int kXBytes = kTT * 128, kABytes = NR * 8 * 128, kStageBytes = kXBytes + kABytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr int kTmemCols = NR * 8 < 32 ? 32 : NR * 8;
};
template <int NR>
__global__ void __launch_bounds__(kThreads, NR <= 8 ? 2 : 1) lora_shrink_kernel(const Args a) {
  using C = ShrinkCfg<NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Tile tile_sh;
  __shared__ int tokens[kTT];
  __shared__ uint64_t empty[C::kStages], done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // The kernel behind this one begins with inputs that are complete by now, the grouping among them; only v it waits for.
  pdl_launch_dependents();
  const Tile tl = find_tile(a, blockIdx.x, &tile_sh);
  if (tl.count == 0 || tl.bin == a.n) return;
  if (tid < kTT) tokens[tid] = tid < tl.count ? a.order[tl.first + tid] : -1;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&empty[i], 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  const int rank = rank_of(a, tl.bin);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int steps_all = (a.H + 63) / 64;
  const int s0 = static_cast<int>(static_cast<long long>(steps_all) * blockIdx.y / a.splits);
  const int s1 = static_cast<int>(static_cast<long long>(steps_all) * (blockIdx.y + 1) / a.splits);
  const __nv_bfloat16* wa = a.a + static_cast<long long>(tl.bin) * a.R * a.H;
  const int lr = tid >> 3, lc = tid & 7;  // row (of 32) and chunk that this thread copies
  const __nv_bfloat16* xp[kTT / 32];
#pragma unroll
  for (int i = 0; i < kTT / 32; ++i) {
    const int t = tokens[i * 32 + lr];
    xp[i] = t >= 0 ? a.x + t * a.x_stride + lc * 8 : nullptr;
  }
  auto load = [&](int s, int slot) {
    const uint32_t st = sbase + slot * C::kStageBytes;
    const int k = s * 64;
    const bool in = k + lc * 8 < a.H;
#pragma unroll
    for (int i = 0; i < kTT / 32; ++i) {
      const bool on = in && xp[i];
      cp_async16(sw128(st, i * 32 + lr, lc), on ? xp[i] + k : a.x, on ? 16u : 0u);
    }
#pragma unroll
    for (int i = 0; i < (NR * 8 + 31) / 32; ++i) {
      const int r = i * 32 + lr;
      const bool on = in && r < rank;
      if (NR * 8 >= 32 || r < NR * 8)
        cp_async16(sw128(st + C::kXBytes, r, lc), on ? wa + static_cast<long long>(r) * a.H + k + lc * 8 : wa, on ? 16u : 0u);
    }
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (s0 + i < s1) load(s0 + i, i);
    cp_commit();
  }
  constexpr uint32_t idesc = idesc_f16(kTT, NR * 8, true);
  int slot = 0, use = 0;  // slot of step s, and how often the ring has gone round
  for (int s = s0; s < s1; ++s) {
    cp_wait<C::kStages - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t st = sbase + slot * C::kStageBytes;
      uint64_t da = sdesc_sw128(st), db = sdesc_sw128(st + C::kXBytes);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk, da += 2, db += 2) mma_ss(tmem, da, db, idesc, s > s0 || kk > 0);
      mma_commit(&empty[slot]);
    }
    // the slot of the step before, once its product is complete
    const int ns = slot == 0 ? C::kStages - 1 : slot - 1;
    if (s + C::kStages - 1 < s1) {
      if (s > s0) bounded_wait(&empty[ns], (slot == 0 ? use - 1 : use) & 1, &abort_flag, a.err);
      load(s + C::kStages - 1, ns);
    }
    cp_commit();
    if (++slot == C::kStages) {
      slot = 0;
      ++use;
    }
  }
  if (tid == 0) mma_commit(&done);
  bounded_wait(&done, 0, &abort_flag, a.err);
  __syncwarp();
  tc_fence_after();
  // a thread: one token, its share of the ranks
  float* v = a.v + (static_cast<long long>(blockIdx.y) * a.T + tl.first) * (NR * 8);
  const int r = (warp & 3) * 32 + lane;
  constexpr int kShare = NR >= 4 ? NR * 4 : 16;  // columns of a warp
  if (NR >= 4 || warp < 4) {
#pragma unroll
    for (int c = 0; c < kShare; c += 16) {
      const int col = (NR >= 4 ? (warp >> 2) * kShare : 0) + c;
      uint32_t o[16];
      tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + col, o);
      tmem_wait_ld();
      if (r < tl.count) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          __stcg(reinterpret_cast<uint4*>(v + static_cast<long long>(r) * (NR * 8) + col + e), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
      }
    }
  }
  cp_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---- out = y + s B v on tcgen05: a tile of tokens and some columns, a block of kCols at a time ----
// y comes by cp.async, whole rows of a block, into shared memory, where the product is added, and leaves from there in
// rows; v lies there as two operands, its two terms.  While one block is worked on, the next one's y and B are under way.
// (9000 tokens, N = 5120, in a graph with all before it: 65 us, with the copies alone 61.  This kernel by itself and cold:
// 45, with rows of y and out as bulk copies of 384 bytes 59, two a token and block being more than the copy unit takes;
// with 8 warps 6 more; in three stages of 128 columns, or two CTAs an SM, 0 to 3 more.)
constexpr int kExpandThreads = 512;
template <int NR>
struct ExpandCfg {
  static constexpr int kPieces = NR <= 8 ? 1 : 2;         // of 64 ranks: 128-byte rows of an operand
  static constexpr int kCols = kPieces == 1 ? 192 : 128;  // what shared memory holds
  static constexpr uint32_t kPieceA = kTT * 128, kPieceB = kCols * 128;
  static constexpr uint32_t kOffB = 2 * kPieces * kPieceA, kBytesB = kPieces * kPieceB;
  static constexpr uint32_t kRowY = kCols * 2 + 16;       // so that a column's rows fall into different banks
  static constexpr uint32_t kOffY = kOffB + 2 * kBytesB, kBytesY = kTT * kRowY;
  static constexpr uint32_t kSmem = kOffY + 2 * kBytesY + 1024;
};
template <int NR>
__global__ void __launch_bounds__(kExpandThreads, 1) lora_expand_kernel(const Args a) {
  using C = ExpandCfg<NR>;
  constexpr int kCols = C::kCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Tile tile_sh;
  __shared__ uint64_t d_full[2];
  __shared__ long long y_row[kTT], out_row[kTT];  // first elements of the tokens' rows
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Everything but v was complete before the kernel ahead let this one start; it is read past L1, which may hold lines of
  // before.
  const Tile tl = find_tile(a, blockIdx.x, &tile_sh);
  const bool none = tl.bin == a.n;
  if (tl.count == 0 || (none && a.out == a.y)) {
    pdl_wait();  // (the kernels behind this one count on the ones ahead of it)
    return;
  }
  const int blocks_all = (a.N + kCols - 1) / kCols;
  // every spans-th block is this CTA's, so that the CTAs of a tile go along its rows together
  const int blocks = (blocks_all - static_cast<int>(blockIdx.y) + a.spans - 1) / a.spans;
  auto column = [&](int b) { return (b * a.spans + static_cast<int>(blockIdx.y)) * kCols; };
  if (tid < kTT) {
    const int t = tid < tl.count ? __ldcg(a.order + tl.first + tid) : 0;
    y_row[tid] = t * a.y_stride;
    out_row[tid] = t * a.out_stride;
  }
  if (none) {  // y as it is
    pdl_wait();
    __syncthreads();
    const int chunks = a.N / 8, c0 = static_cast<int>(static_cast<long long>(chunks) * blockIdx.y / a.spans);
    const int w = static_cast<int>(static_cast<long long>(chunks) * (blockIdx.y + 1) / a.spans) - c0;
    for (long long i = tid; i < static_cast<long long>(tl.count) * w; i += kExpandThreads) {
      const int r = static_cast<int>(i / w), c = (c0 + static_cast<int>(i % w)) * 8;
      *reinterpret_cast<uint4*>(a.out + out_row[r] + c) = __ldcg(reinterpret_cast<const uint4*>(a.y + y_row[r] + c));
    }
    return;
  }
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int rank = rank_of(a, tl.bin);
  const __nv_bfloat16* const wb = a.b + static_cast<long long>(tl.bin) * a.N * a.R;
  // y's rows into shared memory (in), or out's from there: a warp a row or two, a chunk of 8 columns a lane
  constexpr int kChunks = kCols / 8, kAtOnce = 32 / kChunks;
  const int rc = lane % kChunks, rr = lane / kChunks * (kExpandThreads / 32) + warp;
  const uint32_t r_at = C::kOffY + rr * C::kRowY + rc * 16;
  auto rows = [&](int b, bool in) {
    const int col = column(b) + rc * 8;
    if (lane >= kAtOnce * kChunks || col >= a.N) return;
    const uint32_t at = r_at + (b & 1) * C::kBytesY;
    constexpr int kStep = kAtOnce * (kExpandThreads / 32);
#pragma unroll
    for (int i = 0; i < kTT / kStep; ++i) {
      const int r = rr + i * kStep;
      if (r >= tl.count) break;
      if (in)
        cp_async16(sbase + at + i * (kStep * C::kRowY), a.y + y_row[r] + col, 16);
      else
        *reinterpret_cast<uint4*>(a.out + out_row[r] + col) = *reinterpret_cast<const uint4*>(smem + at + i * (kStep * C::kRowY));
    }
  };
  auto load_b = [&](int b) {
    const uint32_t to = sbase + C::kOffB + (b & 1) * C::kBytesB;
    for (int i = tid; i < kCols * NR; i += kExpandThreads) {
      const int n = i / NR, c = i % NR, col = column(b) + n, left = min(16, 2 * (rank - c * 8));  // (a rank need not be a multiple of 8)
      const bool on = col < a.N && left > 0;
      cp_async16(sw128(to + (c >> 3) * C::kPieceB, n, c & 7), on ? wb + static_cast<long long>(col) * a.R + c * 8 : wb, on ? left : 0);
    }
  };
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&d_full[i], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  load_b(0);
  __syncthreads();
  rows(0, true);
  cp_commit();
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {  // (not before the wait: the kernel ahead may still have to allocate)
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  {  // v's two terms: 4 ranks a thread and step, rows without a token are zeros
    constexpr int kQ = NR * 2;  // quads of a row
    for (int i = tid; i < kTT * kQ; i += kExpandThreads) {
      const int r = i / kQ, e = i % kQ * 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < tl.count) {
        for (int p = 0; p < a.splits; ++p) {
          const float4 z = __ldcg(reinterpret_cast<const float4*>(a.v + (static_cast<long long>(p) * a.T + tl.first + r) * (NR * 8) + e));
          f.x += z.x;
          f.y += z.y;
          f.z += z.z;
          f.w += z.w;
        }
      }
      f = ranks_of(f, e, rank);
      uint2 first, rest;
      terms_of(f, first, rest);
      uint8_t* to = smem + (e >> 6) * C::kPieceA + r * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + (e & 4) * 2;
      *reinterpret_cast<uint2*>(to) = first;
      *reinterpret_cast<uint2*>(to + C::kPieces * C::kPieceA) = rest;
    }
  }
  const float scale = a.scale ? __ldcg(a.scale + tl.bin) : 1.f;
  constexpr uint32_t idesc = idesc_f16(kTT, kCols, true);
  const int row = (warp & 3) * 32 + lane;  // of the product, in the end, and kShare columns of it
  constexpr int kShare = kCols * 4 / (kExpandThreads / 32);
  for (int b = 0; b < blocks; ++b) {
    const int at = b & 1;
    const uint32_t phase = b >> 1 & 1;
    cp_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    const uint32_t tmem = tmem_base;
    if (tid == 0) {
      tc_fence_after();
      const uint32_t bs = sbase + C::kOffB + at * C::kBytesB;
#pragma unroll 1
      for (int term = 0; term < 2; ++term)
#pragma unroll
        for (int kk = 0; kk < NR / 2; ++kk)
          mma_ss(tmem + at * kCols, sdesc_sw128(sbase + (term * C::kPieces + kk / 4) * C::kPieceA + (kk & 3) * 32),
                 sdesc_sw128(bs + kk / 4 * C::kPieceB + (kk & 3) * 32), idesc, term > 0 || kk > 0);
      mma_commit(&d_full[at]);
    }
    if (b + 1 < blocks) {
      rows(b + 1, true);
      load_b(b + 1);
    }
    cp_commit();
    bounded_wait(&d_full[at], phase, &abort_flag, a.err);
    __syncwarp();
    tc_fence_after();
    uint8_t* const mine = smem + C::kOffY + at * C::kBytesY + row * C::kRowY + (warp >> 2) * (kShare * 2);
#pragma unroll
    for (int c = 0; c < kShare; c += 16) {
      uint32_t d[16];
      tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + at * kCols + (warp >> 2) * kShare + c, d);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        uint4* const p = reinterpret_cast<uint4*>(mine + (c + e) * 2);
        uint4 u = *p;
        auto add = [&](uint32_t w, uint32_t lo, uint32_t hi) {
          return pack_bf16x2(fmaf(scale, __uint_as_float(lo), __uint_as_float(w << 16)),
                             fmaf(scale, __uint_as_float(hi), __uint_as_float(w & 0xFFFF0000u)));
        };
        u.x = add(u.x, d[e], d[e + 1]);
        u.y = add(u.y, d[e + 2], d[e + 3]);
        u.z = add(u.z, d[e + 4], d[e + 5]);
        u.w = add(u.w, d[e + 6], d[e + 7]);
        *p = u;
      }
    }
    tc_fence_before();
    __syncthreads();
    rows(b, false);
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---- a batch of few tokens: all in one kernel ----
// A cluster of kCluster CTAs takes a tile of kTF tokens of one adapter.  Every CTA works out by itself which (the list is
// short), takes a share of H in the first product, reads the others' shares of v from their shared memory, and takes a
// share of N in the second.  Operands go from global memory to the instructions' registers, in an order of k that gives a
// lane 16 neighbouring bytes; what the second product reads is asked for before the exchange.
constexpr int kFewTokens = 1024, kCluster = 8;
template <int NR, int MT>
struct FewCfg {
  static constexpr int kMT = MT;                    // 16-token operand tiles
  static constexpr int kDeep = MT == 1 && NR <= 4 ? 2 : 1;  // groups of columns of a warp asked for ahead
  static constexpr int kTF = 16 * kMT;
  static constexpr int kRp = NR * 8, kWarps = kThreads / 32;
  static constexpr int kOffOwn = kWarps * kTF * kRp * 4;       // [kTF][kRp] the CTA's share of v, behind its warps' shares
  static constexpr int kOffV = kOffOwn + kTF * kRp * 4;        // [2][kTF][kRp + 8] v's two terms
  static constexpr int kRowV = kRp + 8;
  static constexpr int kSmem = kOffV + 2 * kTF * kRowV * 2;
};
inline int few_tiles(int T, int n, int tf) { return T / tf + std::min(n + 1, T); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, int cta) {
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(cta));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(there) : "memory");
  return v;
}
// Elements of a chunk of 8 that lie below `left`.
__device__ __forceinline__ uint4 elements_below(uint4 w, int left) {
  auto keep = [&](uint32_t x, int e) { return left >= e + 2 ? x : (left == e + 1 ? x & 0xFFFFu : 0u); };
  return make_uint4(keep(w.x, 0), keep(w.y, 2), keep(w.z, 4), keep(w.w, 6));
}

template <int NR, int MT>
__global__ void __launch_bounds__(kThreads, NR <= 8 ? 2 : 1) lora_few_kernel(const Args a) {
  using C = FewCfg<NR, MT>;
  constexpr int kMT = C::kMT, kTF = C::kTF, kRp = C::kRp, kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ short counts[kWarps][1026];
  __shared__ int warp_heads[kWarps];
  __shared__ int tokens[kTF];
  __shared__ int tile_bin, tile_base, tile_count, tile_rank;
  __shared__ float tile_scale;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  const int cta = blockIdx.x % kCluster, q = blockIdx.x / kCluster;
  pdl_launch_dependents();
  for (int e = lane; e <= a.n; e += 32) counts[warp][e] = 0;
  if (tid < kTF) tokens[tid] = -1;
  if (tid == 0) {
    tile_bin = -1;
    tile_count = 0;
  }
  __syncthreads();
  pdl_wait();

  // ---- the tile: tokens are numbered within their adapter; every kTF-th begins one ----
  // A warp numbers its share of the tokens by counts of its own, to which those of the warps before are added.
  const int share = (a.T + kThreads - 1) / kThreads * 32;
  constexpr int kMost = kFewTokens / kThreads;  // tokens of a lane
  int bin_t[kMost], place_t[kMost], rank_t[kMost];  // with the adapters' ranks and scales, on their way while tokens are numbered
  float scale_t[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int t = warp * share + i * 32 + lane;
    const bool on = i * 32 < share && t < a.T;
    bin_t[i] = on ? bin_of(a, t) : -1;
    if (on && bin_t[i] == a.n && blockIdx.x == 0 && a.err && __ldg(a.adapter + t) != -1) atomicOr(a.err, MNW_DEVERR_BAD_ADAPTER);
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const bool one = bin_t[i] >= 0 && bin_t[i] < a.n;
    rank_t[i] = one && a.ranks ? __ldcg(a.ranks + bin_t[i]) : a.R;
    scale_t[i] = one && a.scale ? __ldcg(a.scale + bin_t[i]) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const bool on = bin_t[i] >= 0;
    place_t[i] = 1;
    if (i * 32 >= share) continue;
    const uint32_t same = __match_any_sync(0xffffffffu, bin_t[i]), below = same & ((1u << lane) - 1u);
    if (on) place_t[i] = counts[warp][bin_t[i]] + __popc(below);
    __syncwarp();
    if (on && below == 0) counts[warp][bin_t[i]] = static_cast<short>(place_t[i] + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  int heads = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (bin_t[i] >= 0)
      for (int w = 0; w < warp; ++w) place_t[i] += counts[w][bin_t[i]];
    heads += __popc(__ballot_sync(0xffffffffu, bin_t[i] >= 0 && place_t[i] % kTF == 0));
  }
  if (lane == 0) warp_heads[warp] = heads;
  __syncthreads();
  heads = 0;
  for (int w = 0; w < warp; ++w) heads += warp_heads[w];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const bool head = bin_t[i] >= 0 && place_t[i] % kTF == 0;
    const uint32_t hm = __ballot_sync(0xffffffffu, head);
    if (head && heads + __popc(hm & ((1u << lane) - 1u)) == q) {
      tile_bin = bin_t[i];
      tile_base = place_t[i];
      tile_rank = rank_t[i];
      tile_scale = scale_t[i];
    }
    heads += __popc(hm);
  }
  __syncthreads();
  const int bin = tile_bin;
  if (bin < 0) return;  // (the whole cluster)
  const bool none = bin == a.n;
  if (none && a.out == a.y) return;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int r = place_t[i] - tile_base;
    if (bin_t[i] == bin && static_cast<unsigned>(r) < static_cast<unsigned>(kTF)) {
      tokens[r] = warp * share + i * 32 + lane;
      atomicAdd(&tile_count, 1);
    }
  }
  const int rank = none ? 0 : checked_rank(a, tile_rank);
  const float scale = none ? 0.f : tile_scale;
  __syncthreads();
  const int count = tile_count;

  // ---- the second product's operands, asked for ahead: 32 columns at a time, as in the kernel for many tokens ----
  const int groups = (a.N + 31) / 32;
  const int g0 = groups * cta / kCluster + warp, g1 = groups * (cta + 1) / kCluster;
  const __nv_bfloat16* wb = a.b + static_cast<long long>(none ? 0 : bin) * a.N * a.R;
  constexpr int kB = NR == 2 ? 1 : NR / 4;  // chunks of a lane in a row of B
  struct Group {
    uint4 b[4][kB], y[kMT][2];
  } ahead[C::kDeep];
  auto fetch = [&](int g, Group& f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = g * 32 + 8 * (g8 >> 1) + 2 * j + (g8 & 1);
#pragma unroll
      for (int c = 0; c < kB; ++c) {
        const int r = NR == 2 ? 4 * t4 : 32 * c + 8 * t4;
        f.b[j][c] = make_uint4(0, 0, 0, 0);
        if (n < a.N && r < rank) {
          const __nv_bfloat16* src = wb + static_cast<long long>(n) * a.R + r;
          if constexpr (NR == 2) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
            f.b[j][c].x = w.x;
            f.b[j][c].y = w.y;
          } else {
            f.b[j][c] = __ldg(reinterpret_cast<const uint4*>(src));
          }
        }
      }
    }
    const int col = g * 32 + 8 * t4;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = tokens[16 * mt + 8 * x + g8];
        f.y[mt][x] = make_uint4(0, 0, 0, 0);
        if (t >= 0 && col < a.N) f.y[mt][x] = *reinterpret_cast<const uint4*>(a.y + t * a.y_stride + col);
      }
  };
#pragma unroll
  for (int i = 0; i < C::kDeep; ++i)
    if (g0 + i * kWarps < g1) fetch(g0 + i * kWarps, ahead[i]);

  // ---- v: this CTA's share of H ----
  const uint32_t sbase = smem_u32(smem);
  if (!none) {
    const __nv_bfloat16* wa = a.a + static_cast<long long>(bin) * a.R * a.H;
    const int blocks = (a.H + 31) / 32;
    const int b1 = blocks * (cta + 1) / kCluster;
    float acc[kMT][NR][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[mt][i][0] = acc[mt][i][1] = acc[mt][i][2] = acc[mt][i][3] = 0.f;
#pragma unroll(NR <= 4 ? 2 : 1)
    for (int b = blocks * cta / kCluster + warp; b < b1; b += kWarps) {
      const int k = b * 32 + 8 * t4;
      uint4 xw[kMT][2], w[NR];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = tokens[16 * mt + 8 * x + g8];
          xw[mt][x] = make_uint4(0, 0, 0, 0);
          if (t >= 0 && k < a.H) xw[mt][x] = *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + k);
        }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int r = 8 * i + g8;
        w[i] = make_uint4(0, 0, 0, 0);
        if (r < rank && k < a.H) w[i] = __ldg(reinterpret_cast<const uint4*>(wa + static_cast<long long>(r) * a.H + k));
      }
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          mma_bf16(acc[mt][i], xw[mt][0].x, xw[mt][1].x, xw[mt][0].y, xw[mt][1].y, w[i].x, w[i].y);
          mma_bf16(acc[mt][i], xw[mt][0].z, xw[mt][1].z, xw[mt][0].w, xw[mt][1].w, w[i].z, w[i].w);
        }
    }
    float* part = reinterpret_cast<float*>(smem) + warp * (kTF * kRp);
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 16 * mt + 8 * x + g8;
#pragma unroll
        for (int i = 0; i < NR; ++i)
          *reinterpret_cast<float2*>(part + r * kRp + 8 * i + 2 * t4) = make_float2(acc[mt][i][2 * x], acc[mt][i][2 * x + 1]);
      }
    __syncthreads();
    const int used = count * kRp;  // rows of other tokens are not looked at
    for (int e = tid * 4; e < used; e += kThreads * 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(smem + (w * (kTF * kRp) + e) * 4);
        s.x += z.x;
        s.y += z.y;
        s.z += z.z;
        s.w += z.w;
      }
      *reinterpret_cast<float4*>(smem + C::kOffOwn + e * 4) = s;
    }
    cluster_arrive();
    cluster_wait();
    for (int e = tid * 4; e < kTF * kRp; e += kThreads * 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < used) {
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
          const float4 z = ld_cluster(sbase + C::kOffOwn + e * 4, c);
          s.x += z.x;
          s.y += z.y;
          s.z += z.z;
          s.w += z.w;
        }
      }
      s = ranks_of(s, e % kRp, rank);
      uint2 first, rest;
      terms_of(s, first, rest);
      uint8_t* to = smem + C::kOffV + (e / kRp * C::kRowV + e % kRp) * 2;
      *reinterpret_cast<uint2*>(to) = first;
      *reinterpret_cast<uint2*>(to + kTF * C::kRowV * 2) = rest;
    }
    cluster_arrive();  // the others' shares are read
    __syncthreads();
  }

  // ---- out = y + s B v ----
  auto finish = [&](int g, Group& f) {
    float acc[kMT][4][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[mt][j][0] = acc[mt][j][1] = acc[mt][j][2] = acc[mt][j][3] = 0.f;
    if (!none) {
#pragma unroll
      for (int c = 0; c < kB; ++c) {
        const int e = NR == 2 ? 4 * t4 : 32 * c + 8 * t4;  // the lane's elements of v and B
        if (rank & 7) {
#pragma unroll
          for (int j = 0; j < 4; ++j) f.b[j][c] = elements_below(f.b[j][c], rank - e);
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint8_t* at = smem + C::kOffV + ((term * kTF + 16 * mt + g8) * C::kRowV + e) * 2;
            if constexpr (NR == 2) {
              const uint2 v0 = *reinterpret_cast<const uint2*>(at), v1 = *reinterpret_cast<const uint2*>(at + 8 * C::kRowV * 2);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_bf16(acc[mt][j], v0.x, v1.x, v0.y, v1.y, f.b[j][c].x, f.b[j][c].y);
            } else {
              const uint4 v0 = *reinterpret_cast<const uint4*>(at), v1 = *reinterpret_cast<const uint4*>(at + 8 * C::kRowV * 2);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                mma_bf16(acc[mt][j], v0.x, v1.x, v0.y, v1.y, f.b[j][c].x, f.b[j][c].y);
                mma_bf16(acc[mt][j], v0.z, v1.z, v0.w, v1.w, f.b[j][c].z, f.b[j][c].w);
              }
            }
          }
      }
    }
    const int col = g * 32 + 8 * t4;
    auto add = [&](uint32_t u, float p, float r) {
      return pack_bf16x2(fmaf(scale, p, __uint_as_float(u << 16)), fmaf(scale, r, __uint_as_float(u & 0xFFFF0000u)));
    };
    uint4 ow[kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 u = f.y[mt][x];
        ow[mt][x] = none ? u : make_uint4(add(u.x, acc[mt][0][2 * x], acc[mt][0][2 * x + 1]), add(u.y, acc[mt][1][2 * x], acc[mt][1][2 * x + 1]),
                                          add(u.z, acc[mt][2][2 * x], acc[mt][2][2 * x + 1]), add(u.w, acc[mt][3][2 * x], acc[mt][3][2 * x + 1]));
      }
    if (g + C::kDeep * kWarps < g1) fetch(g + C::kDeep * kWarps, f);
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = tokens[16 * mt + 8 * x + g8];
        if (t >= 0 && col < a.N) *reinterpret_cast<uint4*>(a.out + t * a.out_stride + col) = ow[mt][x];
      }
  };
  for (int g = g0; g < g1; g += C::kDeep * kWarps) {
#pragma unroll
    for (int i = 0; i < C::kDeep; ++i)
      if (g + i * kWarps < g1) finish(g + i * kWarps, ahead[i]);
  }
  if (!none) cluster_wait();  // a CTA's memory stays until the others have read it
}

// ---- host ----

// About the clusters that run at a time, by the SMs; the last form has one CTA an SM.  (A cluster lies in one part of the
// GPU, whose SMs are not a multiple of 8: on 152 SMs the occupancy query says 36 and 15 where this says 38 and 19.  The
// rules below were measured with these numbers: at R = 128 256 tokens, more than 15 tiles, are still faster by one kernel.)
inline int clusters_at_once(int R) { return (R <= 64 ? 2 : 1) * current_sm_count() / kCluster; }
// Tokens up to which one kernel takes a batch: as many as its counters hold for up to 32 ranks, and with more, whose tiles
// are of 16 tokens, about one round of tiles.  One kernel and three, H = 4096, N = 5120, 8 adapters unless given:
// R = 16: 512 tokens 10.3 and 13.6 us, 1024 of one 11.1 and 13.5, of eight 15.7 and 16.8, of 64 24.2 and 37.2;
// R = 64: 256 tokens 13.1 and 17.5, 512 of one 13.9 and 16.5, of eight 20.7 and 17.3, 768 26.7 and 19.9, 1024 28.5 and 23.9;
// R = 128: 256 tokens 23.6 and 26.9, 512 37.0 and 27.7, 1024 66.4 and 33.2 (but 512 of 64 adapters 74.5 and 98.5: how many
// adapters a batch has is known on the device only.)
inline int few_tokens(int R) { return R <= 32 ? kFewTokens : std::min(kFewTokens, 16 * clusters_at_once(R)); }

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline int padded(int R) { return R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128)); }
// Shares of H in the first product: as many as fill the GPU, 256 elements each at least.
inline int splits_of(int T, int H) {
  const int tiles = (T + kTT - 1) / kTT;
  return std::max(1, std::min({2 * current_sm_count() / tiles, H / 256, 16}));
}
// Shares of N in the second product, each some of its blocks, for about `tiles` tiles and one CTA an SM: fewest rounds of blocks, where a CTA's
// beginning and end cost about one more.
inline int spans_of(int tiles, int blocks) {
  const int sms = current_sm_count();
  int best = 1;
  long long least = 0;
  for (int s = 1; s <= blocks && s <= 64; ++s) {
    const long long cost = static_cast<long long>((tiles * static_cast<long long>(s) + sms - 1) / sms) * ((blocks + s - 1) / s + 1);
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}
struct Workspace {
  size_t starts, order, v, bytes;
};
inline Workspace workspace_of(int T, int H, int R, int n) {
  Workspace w{};
  if (T <= few_tokens(R)) return w;
  w.starts = 0;
  w.order = up256((static_cast<size_t>(n) + 2) * 4);
  w.v = w.order + up256(static_cast<size_t>(T) * 4);
  w.bytes = w.v + up256(static_cast<size_t>(splits_of(T, H)) * T * padded(R) * 4);
  return w;
}

template <int NR, int MT>
int launch_few(const Args& a, cudaStream_t st) {
  using C = FewCfg<NR, MT>;
  auto kern = lora_few_kernel<NR, MT>;
  static std::atomic<uint64_t> attr{0};
  uint64_t bit;
  if (attrs_needed(attr, &bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return MNW_E_CUDA;
    attrs_done(attr, bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(few_tiles(a.T, a.n, C::kTF) * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kCluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return MNW_E_CUDA;
  note_launch();
  return MNW_OK;
}

template <int NR>
int launch(Args& a, uint8_t* ws, cudaStream_t st) {
  if (a.T <= few_tokens(a.R)) {
    // Tiles of 16 tokens, whose registers hold two groups of columns ahead, up to about one round of tiles, and of 32
    // above.  H = 4096, N = 5120, R = 16 and 32: 64 tokens of one adapter 5.6 and 6.9 us (tiles of 32: 7.1 and 9.4),
    // 512 of four 7.8 and 10.2 (10.1 and 13.5), 1024 of one 15.2 and 18.9 (11.1 and 14.8).
    if constexpr (NR <= 4)
      if (a.T > 16 * clusters_at_once(a.R)) return launch_few<NR, 2>(a, st);
    return launch_few<NR, 1>(a, st);
  }
  const Workspace w = workspace_of(a.T, a.H, a.R, a.n);
  a.starts = reinterpret_cast<int32_t*>(ws + w.starts);
  a.order = reinterpret_cast<int32_t*>(ws + w.order);
  a.v = reinterpret_cast<float*>(ws + w.v);
  a.splits = splits_of(a.T, a.H);
  auto shrink = lora_shrink_kernel<NR>;
  auto expand = lora_expand_kernel<NR>;
  static std::atomic<uint64_t> attr{0};
  uint64_t bit;
  if (attrs_needed(attr, &bit)) {
    if (cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, ShrinkCfg<NR>::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize, ExpandCfg<NR>::kSmem) != cudaSuccess)
      return MNW_E_CUDA;
    attrs_done(attr, bit);
  }
  const unsigned tiles = tile_numbers(a.T, a.n);
  a.spans = spans_of((a.T + kTT - 1) / kTT + std::min(a.n, a.T / kTT) / 2, (a.N + ExpandCfg<NR>::kCols - 1) / ExpandCfg<NR>::kCols);
  if (launch_pdl(lora_group_kernel, dim3(a.n + 1), dim3(kGroupThreads), 0, st, a) != cudaSuccess ||
      launch_pdl(shrink, dim3(tiles, a.splits), dim3(kThreads), ShrinkCfg<NR>::kSmem, st, a) != cudaSuccess ||
      launch_pdl(expand, dim3(tiles, a.spans), dim3(kExpandThreads), ExpandCfg<NR>::kSmem, st, a) != cudaSuccess)
    return MNW_E_CUDA;
  return MNW_OK;
}

}  // namespace lora
}  // namespace mnw

using namespace mnw;

extern "C" {

size_t mnw_lora_workspace_size(int T, int H, int R, int n_adapters) {
  if (T <= 0 || H <= 0 || R <= 0 || R > 128 || n_adapters <= 0) return 0;
  return lora::workspace_of(T, H, R, n_adapters).bytes;
}

int mnw_lora_add(const void* x, long long x_stride, const void* a, const void* b, const float* scale,
                 const int32_t* ranks, int n_adapters, int R, const int32_t* adapter, int T, int H, int N,
                 const void* y, long long y_stride, void* out, long long out_stride, void* ws, size_t ws_bytes,
                 uint32_t* err, mnw_stream stream) {
  MNW_RANGE("mnw_lora_add");
  if (T < 0 || H <= 0 || N <= 0 || R <= 0 || n_adapters <= 0) return MNW_E_INVALID_ARG;
  if (T == 0) return MNW_OK;
  if (H % 8 || N % 8 || R % 8 || R > 128 || n_adapters > 1024 || T > (1 << 24) || N > (1 << 20)) return MNW_E_UNSUPPORTED;
  const size_t need = mnw_lora_workspace_size(T, H, R, n_adapters);
  if (!x || !a || !b || !adapter || !y || !out || (need > 0 && !ws) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(y, 16) || !aligned(out, 16) || !aligned(ws, 256) || !aligned(adapter, 4) || !aligned(ranks, 4) ||
      !aligned(scale, 4) || !aligned(err, 4) || x_stride % 8 || y_stride % 8 || out_stride % 8 || x_stride < H || y_stride < N || out_stride < N)
    return MNW_E_INVALID_ARG;
  // rows of one over others of the other, or over x, which is still read
  if ((y == out && y_stride != out_stride && T > 1) || x == out) return MNW_E_INVALID_ARG;
  if (ws_bytes < need) return MNW_E_WORKSPACE_TOO_SMALL;
  lora::Args p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.a = static_cast<const __nv_bfloat16*>(a);
  p.b = static_cast<const __nv_bfloat16*>(b);
  p.y = static_cast<const __nv_bfloat16*>(y);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.x_stride = x_stride;
  p.y_stride = y_stride;
  p.out_stride = out_stride;
  p.scale = scale;
  p.ranks = ranks;
  p.adapter = adapter;
  p.n = n_adapters;
  p.R = R;
  p.T = T;
  p.H = H;
  p.N = N;
  p.err = err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto* w = static_cast<uint8_t*>(ws);
  switch (lora::padded(R)) {
    case 16: return lora::launch<2>(p, w, st);
    case 32: return lora::launch<4>(p, w, st);
    case 64: return lora::launch<8>(p, w, st);
    default: return lora::launch<16>(p, w, st);
  }
}

}  // extern "C"
