// mnw_attn_split.cuh -- the split of paged attention's work over CTAs and the
// joining of its parts.
//
// The unit is one tile of kTK keys of one item (sequence, kv head, tile of RT
// query rows).  All units in order are cut into equal runs, one per CTA, so
// ragged lengths load the CTAs evenly and one long sequence spreads over the
// whole GPU.  A run that covers an item whole writes its output; otherwise it
// leaves a part (maximum, sum, unnormalised output) in the workspace.  A run
// can end inside one item and begin inside one, so it has two slots: 2c for a part that
// continues an item, 2c + 1 for one that begins it.
//
// Joining: parts are added in run order, so the result does not depend on
// timing.  Items of a few rows: the CTA that arrives last at an item joins it
// (a launch less).  Otherwise a second kernel does, over the whole GPU.  A part that is written is
// marked with the call's number, so the workspace needs no clearing: a mark of
// another call, or anything else, is none; the joining CTA clears the item's
// marks (a replayed graph brings the same number).
#pragma once
#include <cuda_bf16.h>

#include <atomic>

#include "mnw_convert.cuh"
#include "mnw_internal.h"
#include "mnw_paged.cuh"
#include "mnw_ptx.cuh"

namespace mnw {
namespace pattn {

using paged::Batch;
using paged::FastDiv;
using paged::Seq;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBlockRows = 128, kBlockKeys = 128;  // the block kernel's tiles (mnw_attn_paged_block.cu)
constexpr int kInt4Keys = 256;                     // the INT4 kernel's (mnw_attn_paged_int4.cu), and its CTAs on an SM
// INT4: the operands' 2^-24 is taken back half with the keys' scales, half with the queries' factors.
constexpr float kHalfUnit = 4096.f;
constexpr int int4_runs_per_sm(int rt) { return rt <= 8 ? 3 : 2; }

struct Args {
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  long long page_bytes;  // bytes between pages of kc and vc
  FastDiv page_div;
  FastDiv g_div, blk_div;
  int n_pages, page_size, Hq, Hkv, G, blk;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  // workspace
  unsigned long long* arrivals;  // [2 * runs] marks of the parts
  int* starts;                   // [B + 2] first unit of each sequence, then units per run and their padding
  float* part_o;                 // [2 * runs][RT][D]
  float2* part_ml;               // [2 * runs][RT]
  unsigned long long tag;        // the call's number
  int fused;                     // the last arrival joins
  uint32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two FP32 ones that the compiler does not know for such (Hq > 0): a packed sum written as x * 1 + y cannot be joined with
// the product that x is, which a packed addition was.
__device__ __forceinline__ uint64_t ones(const Args& a) {
  const uint32_t one = 0x3F800000u | static_cast<uint32_t>(a.Hq >> 31);
  return f32x2_pack(one, one);
}

// 16-, 8- and 4-byte asynchronous copies; bytes 0: zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// INT8: q enters the first product as FP16 times a power of two a row: e with the
// row's largest magnitude (given as BF16 bits) in [2^14, 2^15) after x * 2^-e.
__device__ __forceinline__ int row_exponent(uint32_t largest) {
  return largest == 0 ? 0 : max(-110, min(113, static_cast<int>(largest >> 7) - 127 - 14));
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Four unsigned-biased codes (code + 128 per byte) -> FP16 pairs: byte b under
// the exponent byte 0x64 is the FP16 value 1024 + b.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return f16x2_sub(prmt(w, 0x64646464u, 0x4140), 0x64806480u); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return f16x2_sub(prmt(w, 0x64646464u, 0x4342), 0x64806480u); }
// Units of a sequence (the host bounds their sum below 2^31 for ranges of rows
// in order; others are not computed at all, see find_run).  An item counts
// as a multiple of `pad` units, so that with runs of `pad` none begins inside
// one item and goes on in the next.
struct Shape {
  int units, rt, kt, ku;  // row tiles; key tiles of an item (one at least, so that empty caches still write their rows); its units
};
template <int RT, int TK>
__device__ __forceinline__ Shape shape_of(const Seq& s, int G, int Hkv, int pad) {
  Shape h;
  h.rt = (s.n * G + RT - 1) / RT;
  h.kt = max(1, (s.len + TK - 1) / TK);
  h.ku = pad == 1 ? h.kt : (h.kt + pad - 1) / pad * pad;
  h.units = Hkv * h.rt * h.ku;
  return h;
}

constexpr int kMaxSlack = 4;
struct SplitShared {
  int scan[32], pads[kMaxSlack][32];
  int seq, first;  // sequence of the run's first unit and its first unit
};

struct Run {
  int u0, u1, per, pad;  // units [u0, u1) of runs of `per`
  int seq, first;        // sequence that holds u0 (-1: none) and its first unit
};

// Where run blockIdx.x begins.  All threads call; ends with a barrier.  Runs
// are equal shares of the units.  With SLACK > 0, for a kernel that pays more
// for a second item in a run than for a few more tiles, the SLACK lengths from
// the equal share on are tried, and the first at which runs that do not cross
// items fit the grid is taken (block kernel, 16 sequences of up to 4000 INT8
// positions, 64 items on 152 CTAs: 65 us with equal shares, 56 with SLACK 4).
template <int RT, int TK, int THREADS, int SLACK>
__device__ __forceinline__ Run find_run(const Args& a, SplitShared* sh) {
  constexpr int kWarps = THREADS / 32;
  static_assert(SLACK <= kMaxSlack);
  const Batch& bt = a.bt;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool scribe = blockIdx.x == 0;  // run 0 reports bad lengths and writes the sequences' first units
  if (tid == 0) sh->seq = -1;
  const int runs = gridDim.x;
  // runs that the items of a sequence make at p units each (clipped: they are added up)
  auto runs_of = [&](const Shape& one, int p) { return min(a.Hkv * one.rt * ((one.kt + p - 1) / p), 1 << 20); };
  int total = 0;
  bool back = false;
  Seq s{};
  for (int b = tid; b < bt.B; b += THREADS) {
    bool bad;
    s = paged::sequence(bt, b, a.page_size, &bad);
    if (bad && scribe && a.err) atomicOr(a.err, MNW_DEVERR_BAD_LENGTH);
    back = back || paged::backwards(bt, b);
    total += shape_of<RT, TK>(s, a.G, a.Hkv, 1).units;
  }
  // Rows counted by several sequences could pass the 32-bit units, and every run's and join's place with them: then no
  // run has anything to do, and the joining kernel is told by a share of 0.
  const int tw = __reduce_add_sync(0xffffffffu, total);
  back = __any_sync(0xffffffffu, back);
  if (lane == 0) sh->scan[warp] = back ? -1 : tw;
  __syncthreads();
  total = 0;
  int least = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    total += sh->scan[w];
    least = min(least, sh->scan[w]);
  }
  if (least < 0) total = 0;
  Run r;
  r.per = max(1, (total + runs - 1) / runs);
  r.pad = 1;
  int limit = total;
  if (SLACK > 0 && total > runs) {
    int sums[SLACK > 0 ? SLACK : 1];
#pragma unroll
    for (int k = 0; k < SLACK; ++k) sums[k] = 0;
    for (int b = tid; b < bt.B; b += THREADS) {
      bool bad;
      if (bt.B > THREADS) s = paged::sequence(bt, b, a.page_size, &bad);
      const Shape one = shape_of<RT, TK>(s, a.G, a.Hkv, 1);
#pragma unroll
      for (int k = 0; k < SLACK; ++k) sums[k] = min(sums[k] + runs_of(one, r.per + k), 1 << 20);
    }
#pragma unroll
    for (int k = 0; k < SLACK; ++k) {
      const int v = __reduce_add_sync(0xffffffffu, sums[k]);
      if (lane == 0) sh->pads[k][warp] = v;
    }
    __syncthreads();
    const int share = r.per;
#pragma unroll
    for (int k = SLACK - 1; k >= 0; --k) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sh->pads[k][w];
      if (v <= runs) {
        r.pad = r.per = share + k;
        limit = v * (share + k);
      }
    }
  }
  r.u0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * r.per, static_cast<long long>(limit)));
  r.u1 = min(limit, r.u0 + r.per);
  int carry = 0;
  for (int b0 = 0; b0 < bt.B; b0 += THREADS) {
    const int b = b0 + tid;
    int mine = 0;
    if (b < bt.B) {
      bool bad;
      if (bt.B > THREADS) s = paged::sequence(bt, b, a.page_size, &bad);
      mine = shape_of<RT, TK>(s, a.G, a.Hkv, r.pad).units;
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    __syncthreads();  // the sums above are read
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = sh->scan[w];
      if (w < warp) before += v;
      carry += v;
    }
    const int first = before + incl - mine;
    if (b < bt.B) {
      if (scribe) a.starts[b] = first;
      if (mine > 0 && first <= r.u0 && r.u0 < first + mine) {
        sh->seq = b;
        sh->first = first;
      }
    }
  }
  if (scribe && tid == 0) {
    a.starts[bt.B] = r.u1 > 0 ? r.per : 0;
    a.starts[bt.B + 1] = r.pad;
  }
  __syncthreads();
  r.seq = r.u0 < r.u1 ? sh->seq : -1;
  r.first = sh->first;
  return r;
}

// A place in the order of units.
template <int RT, int TK>
struct Cursor {
  Seq s;
  Shape sh;
  int b, g, rt, kt;  // sequence, kv head, row tile, key tile

  __device__ __forceinline__ void set(const Args& a, const Run& r) {
    bool bad;
    b = r.seq;
    s = paged::sequence(a.bt, b, a.page_size, &bad);
    sh = shape_of<RT, TK>(s, a.G, a.Hkv, r.pad);
    const int in = r.u0 - r.first, item = in / sh.ku;
    kt = in - item * sh.ku;
    g = sh.rt == 1 ? item : item / sh.rt;
    rt = item - g * sh.rt;
  }
  // First tile of the next item; false past the last.
  __device__ __forceinline__ bool next_item(const Args& a, int pad) {
    kt = 0;
    if (++rt < sh.rt) return true;
    rt = 0;
    if (++g < a.Hkv) return true;
    g = 0;
    do {
      if (++b >= a.bt.B) return false;
      bool bad;
      s = paged::sequence(a.bt, b, a.page_size, &bad);
      sh = shape_of<RT, TK>(s, a.G, a.Hkv, pad);
    } while (sh.units == 0);
    return true;
  }
};

// First position that query row ri (token ri / G of the sequence) may not see;
// 0 for a token without a cached position.
__device__ __forceinline__ int row_limit(const Args& a, const Seq& s, int ri) {
  const int p = s.first + static_cast<int>(paged::quotient(ri, a.g_div));
  if (p < 0 || p >= s.len) return 0;
  const long long e = (static_cast<long long>(paged::quotient(p, a.blk_div)) + 1) * a.blk;
  return e < s.len ? static_cast<int>(e) : s.len;
}

// An item's extent: units [us, us + ku), runs c0 .. c1.
struct Span {
  int us, c0, c1;
};
__device__ __forceinline__ Span span_of(int us, int ku, int per) { return Span{us, us / per, (us + ku - 1) / per}; }
__device__ __forceinline__ long long slot_of(const Span& sp, int c, int per) {
  return 2ll * c + (static_cast<long long>(c) * per > sp.us ? 0 : 1);
}

// Row of the output that row r of row tile rt, kv head g, holds.
template <int RT>
__device__ __forceinline__ size_t out_row(const Args& a, const Seq& s, int g, int rt, int r) {
  const int ri = rt * RT + r, i = static_cast<int>(paged::quotient(ri, a.g_div));
  return static_cast<size_t>(s.start + i) * a.Hq + g * a.G + (ri - i * a.G);
}

// Marks this CTA's part of an item as written; true where every part of the
// item is.  All threads call, after writing the part.  The mark is a release
// for the whole CTA: the barrier orders the other threads' writes before the
// fence of the thread that stores it.  The mark is stored before the others are
// read, with a sequentially consistent fence between, so the last CTA to mark
// sees all marks; CTAs that mark at the same time may all see them, and then
// write the same result.  A thread that reads marks fences before the barrier
// that lets the others read the parts.  No CTA waits.
__device__ __forceinline__ bool all_arrived(const Args& a, const Span& sp, int per, long long mine) {
  __syncthreads();
  if (threadIdx.x == 0) {
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(a.arrivals + mine), "l"(a.tag) : "memory");
    asm volatile("fence.sc.gpu;" ::: "memory");
  }
  __syncthreads();
  bool all = true;
  const int first = sp.c0 + static_cast<int>(threadIdx.x);
  for (int c = first; c <= sp.c1; c += blockDim.x) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(a.arrivals + slot_of(sp, c, per)) : "memory");
    all = all && v == a.tag;
  }
  if (first <= sp.c1) asm volatile("fence.acq_rel.gpu;" ::: "memory");
  return __syncthreads_and(all) != 0;
}
// After joining: a replayed graph brings the same number again.
__device__ __forceinline__ void clear_arrivals(const Args& a, const Span& sp, int per) {
  for (int c = sp.c0 + static_cast<int>(threadIdx.x); c <= sp.c1; c += blockDim.x)
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(a.arrivals + slot_of(sp, c, per)), "l"(0ull) : "memory");
}

// Adds the parts of one row and writes it.  D / 4 neighbouring lanes work on a
// row, 4 columns each; `scratch` is theirs, 2 * kJoinBatch floats of shared
// memory.  Loads go past L1: the parts are other CTAs' writes.
constexpr int kJoinBatch = 64;  // parts whose weights are held at a time
template <int D, int RT>
__device__ __forceinline__ void join_row(const Args& a, const Seq& s, const Span& sp, int per, int g, int rt, int r,
                                         float* scratch) {
  constexpr int kCols = D / 4;
  const int j = threadIdx.x % kCols, col = j * 4;
  const uint32_t mask = kCols == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  const int parts = sp.c1 - sp.c0 + 1;
  auto load_o = [&](int c) {
    return __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot_of(sp, sp.c0 + c, per) * RT + r) * D + col));
  };
  // the first parts' loads go out together with those of the maxima
  constexpr int kAhead = 8;
  float4 v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) v[i] = i < parts ? load_o(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kMine = kJoinBatch / kCols;
  float2 ml[kMine];  // of parts j, j + kCols, ... of the first batch
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int c = j + i * kCols;
    ml[i] = c < parts ? __ldcg(a.part_ml + slot_of(sp, sp.c0 + c, per) * RT + r) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, ml[i].x);
  }
  for (int c = j + kJoinBatch; c < parts; c += kCols) M = fmaxf(M, __ldcg(a.part_ml + slot_of(sp, sp.c0 + c, per) * RT + r).x);
#pragma unroll
  for (int d = kCols / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(mask, M, d));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cb = 0; cb < parts; cb += kJoinBatch) {
    const int nb = min(kJoinBatch, parts - cb);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int c = j + i * kCols;
      if (cb > 0) ml[i] = c < nb ? __ldcg(a.part_ml + slot_of(sp, sp.c0 + cb + c, per) * RT + r) : make_float2(-INFINITY, 0.f);
      const float f = ex2(ml[i].x - base);
      scratch[2 * c] = f;
      scratch[2 * c + 1] = f * ml[i].y;
    }
    __syncwarp(mask);
    for (int c0 = 0; c0 < nb; c0 += kAhead) {
      if (cb + c0 > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = c0 + i < nb ? load_o(cb + c0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float f = scratch[2 * (c0 + i)];
        L += scratch[2 * (c0 + i) + 1];
        acc.x = fmaf(f, v[i].x, acc.x);
        acc.y = fmaf(f, v[i].y, acc.y);
        acc.z = fmaf(f, v[i].z, acc.z);
        acc.w = fmaf(f, v[i].w, acc.w);
      }
    }
    __syncwarp(mask);
  }
  const size_t row = out_row<RT>(a, s, g, rt, r);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + row * D + col) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && j == 0) a.lse[row] = (M + log2f(L)) * kLn2;
}

// As join_row for at most kFewParts parts, the usual case where runs are about
// as long as items: all loads go out at once, without a maximum first.
constexpr int kFewParts = 4;
template <int D, int RT>
__device__ __forceinline__ void join_few(const Args& a, const Seq& s, const Span& sp, int per, int g, int rt, int r, int col) {
  float2 ml[kFewParts];
  float4 v[kFewParts];
#pragma unroll
  for (int p = 0; p < kFewParts; ++p) {
    ml[p] = make_float2(-INFINITY, 0.f);
    v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sp.c0 + p <= sp.c1) {
      const long long at = slot_of(sp, sp.c0 + p, per) * RT + r;
      ml[p] = __ldcg(a.part_ml + at);
      v[p] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + col));
    }
  }
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int p = 0; p < kFewParts; ++p) M = fmaxf(M, ml[p].x);
  const float base = M == -INFINITY ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int p = 0; p < kFewParts; ++p) {
    const float f = ex2(ml[p].x - base);
    L += f * ml[p].y;
    acc.x = fmaf(f, v[p].x, acc.x);
    acc.y = fmaf(f, v[p].y, acc.y);
    acc.z = fmaf(f, v[p].z, acc.z);
    acc.w = fmaf(f, v[p].w, acc.w);
  }
  const size_t row = out_row<RT>(a, s, g, rt, r);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + row * D + col) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && col == 0) a.lse[row] = (M + log2f(L)) * kLn2;
}

// The rows [0, rows) of an item by THREADS threads (`tid` their index).
template <int D, int RT, int THREADS>
__device__ __forceinline__ void join_item(const Args& a, const Seq& s, const Span& sp, int per, int g, int rt, int rows,
                                          float* scratch, int tid) {
  constexpr int kCols = D / 4;
  const bool few = sp.c1 - sp.c0 < kFewParts;
#pragma unroll 1
  for (int r = tid / kCols; r < rows; r += THREADS / kCols) {
    if (few)
      join_few<D, RT>(a, s, sp, per, g, rt, r, (tid % kCols) * 4);
    else
      join_row<D, RT>(a, s, sp, per, g, rt, r, scratch + tid / kCols * 2 * kJoinBatch);
  }
}

// The block kernel over `runs` runs (mnw_attn_paged_block.cu).
int launch_block(const Args& a, int d, int fmt, int runs, cudaStream_t st);
// The INT4 kernel for row tiles of rt = 8, 16 or 32 (mnw_attn_paged_int4.cu).
int launch_int4(const Args& a, int d, int rt, int runs, cudaStream_t st);

// The joining kernel: D / 4 lanes per (token, query head) row; rows of items
// that one run covered are done already.
constexpr int kJoinThreads = 128;
template <int D, int RT, int TK>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const Args a) {
  constexpr int kRows = kJoinThreads / (D / 4);
  __shared__ float scratch[kRows][2 * kJoinBatch];
  pdl_launch_dependents();
  pdl_wait();
  const int rr = threadIdx.x / (D / 4);
  const int row = blockIdx.x * kRows + rr;
  if (row >= a.bt.T * a.Hq) return;
  const int t = row / a.Hq, h = row - t * a.Hq;
  int b;
  if (a.bt.q_start) {  // sequences that end at or before t
    b = 0;
    for (int j = 0; j < a.bt.B; ++j) b += __ldg(a.bt.q_start + j + 1) <= t ? 1 : 0;
  } else {
    b = t / a.bt.n_uniform;
  }
  if (b >= a.bt.B) return;
  bool bad;
  const Seq s = paged::sequence(a.bt, b, a.page_size, &bad);
  if (t < s.start || t >= s.start + s.n) return;
  const int per = a.starts[a.bt.B];
  if (per == 0) return;
  const Shape sh = shape_of<RT, TK>(s, a.G, a.Hkv, a.starts[a.bt.B + 1]);
  const int g = h / a.G, ri = (t - s.start) * a.G + (h - g * a.G);
  const int rt = ri / RT;
  const Span sp = span_of(a.starts[b] + (g * sh.rt + rt) * sh.ku, sh.ku, per);
  if (sp.c0 == sp.c1) return;
  if (sp.c1 - sp.c0 < kFewParts)
    join_few<D, RT>(a, s, sp, per, g, rt, ri - rt * RT, threadIdx.x % (D / 4) * 4);
  else
    join_row<D, RT>(a, s, sp, per, g, rt, ri - rt * RT, scratch[rr]);
}

}  // namespace pattn
}  // namespace mnw
