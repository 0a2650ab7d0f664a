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
// timing.  Few parts and rows: the CTA that arrives last at an item joins it
// (a launch less).  Otherwise a second kernel does, a CTA per few rows.
// Arrivals are counted in a workspace word tagged with the call's number, so
// the workspace needs no clearing: a word of another call or of anything else
// counts as zero, and the last arrival leaves zero (a replayed graph has the
// same number).
#pragma once
#include <cuda_bf16.h>

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

struct Args {
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  long long page_bytes;  // bytes between pages of kc and vc
  FastDiv page_div;
  int n_pages, page_size, Hq, Hkv, G, blk;
  int min_units;  // units of a run at least, where there are few
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  // workspace
  unsigned long long* arrivals;  // [runs] of the item that begins in run c and goes on in the next
  int* starts;                   // [B] first unit of each sequence, [B] = units per run (for the joining kernel)
  float* part_o;                 // [2 * runs][RT][D]
  float2* part_ml;               // [2 * runs][RT]
  unsigned long long tag;        // the call's number << 16
  int fused;                     // the last arrival joins
  uint32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Units of a sequence (the host bounds their sum below 2^31).
struct Shape {
  int units, rt, kt;  // row tiles, key tiles (one at least, so that empty caches still write their rows)
};
template <int RT, int TK>
__device__ __forceinline__ Shape shape_of(const Seq& s, int G, int Hkv) {
  Shape h;
  h.rt = (s.n * G + RT - 1) / RT;
  h.kt = max(1, (s.len + TK - 1) / TK);
  h.units = Hkv * h.rt * h.kt;
  return h;
}

struct SplitShared {
  int scan[32];
  int seq, first;  // sequence of the run's first unit and its first unit
};

struct Run {
  int u0, u1, per;   // units [u0, u1) of runs of `per`
  int seq, first;    // sequence that holds u0 (-1: none) and its first unit
};

// Where run blockIdx.x begins.  All threads call; ends with a barrier.
template <int RT, int TK, int THREADS>
__device__ __forceinline__ Run find_run(const Args& a, SplitShared* sh) {
  constexpr int kWarps = THREADS / 32;
  const Batch& bt = a.bt;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool scribe = blockIdx.x == 0;  // run 0 reports bad lengths and writes the sequences' first units
  if (tid == 0) sh->seq = -1;
  Run r;
  int carry = 0, first = 0, mine = 0, total = 0;
  // up to THREADS sequences a pass; beyond one pass, the total first
  const int passes = (bt.B + THREADS - 1) / THREADS;
  if (passes > 1) {
    for (int b = tid; b < bt.B; b += THREADS) {
      bool bad;
      total += shape_of<RT, TK>(paged::sequence(bt, b, a.page_size, &bad), a.G, a.Hkv).units;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) sh->scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sh->scan[w];
    __syncthreads();
  }
  for (int p = 0; p < passes; ++p) {
    const int b = p * THREADS + tid;
    mine = 0;
    if (b < bt.B) {
      bool bad;
      mine = shape_of<RT, TK>(paged::sequence(bt, b, a.page_size, &bad), a.G, a.Hkv).units;
      if (bad && scribe && a.err) atomicOr(a.err, MNW_DEVERR_BAD_LENGTH);
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = sh->scan[w];
      if (w < warp) before += v;
      carry += v;
    }
    first = before + incl - mine;
    if (passes == 1) total = carry;
    r.per = max(a.min_units, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
    r.u0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * r.per, static_cast<long long>(total)));
    r.u1 = min(total, r.u0 + r.per);
    if (b < bt.B) {
      if (scribe) a.starts[b] = first;
      if (mine > 0 && first <= r.u0 && r.u0 < first + mine) {
        sh->seq = b;
        sh->first = first;
      }
    }
    __syncthreads();
  }
  if (scribe && tid == 0) a.starts[bt.B] = r.per;
  r.seq = sh->seq;
  r.first = sh->first;
  return r;
}

// An item's extent: units [us, us + kt), runs c0 .. c1.
struct Span {
  int us, c0, c1;
};
__device__ __forceinline__ Span span_of(int us, int kt, int per) { return Span{us, us / per, (us + kt - 1) / per}; }
__device__ __forceinline__ long long slot_of(const Span& sp, int c, int per) {
  return 2ll * c + (static_cast<long long>(c) * per > sp.us ? 0 : 1);
}

// Row of the output that row r of row tile rt, kv head g, holds.
template <int RT>
__device__ __forceinline__ size_t out_row(const Args& a, const Seq& s, int g, int rt, int r) {
  const int ri = rt * RT + r, i = ri / a.G;
  return static_cast<size_t>(s.start + i) * a.Hq + g * a.G + (ri - i * a.G);
}

// Counts this CTA's part of an item; true for the last of `need`.  All threads
// call after writing the part.
__device__ __forceinline__ bool arrive_last(const Args& a, const Span& sp, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long* w = a.arrivals + sp.c0;
    const unsigned need = sp.c1 - sp.c0 + 1;
    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(w);
    bool last;
    for (;;) {  // an exchange fails only when another part arrived: at most `need` times
      const unsigned n = ((old ^ a.tag) >> 16) == 0 ? static_cast<unsigned>(old & 0xFFFFu) : 0u;
      last = n + 1 >= need;
      const unsigned long long seen = atomicCAS(w, old, last ? 0ull : (a.tag | (n + 1)));
      if (seen == old) break;
      old = seen;
    }
    *flag = last;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
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
  float M = -INFINITY;
  for (int c = j; c < parts; c += kCols) M = fmaxf(M, __ldcg(&a.part_ml[slot_of(sp, sp.c0 + c, per) * RT + r].x));
#pragma unroll
  for (int d = kCols / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(mask, M, d));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cb = 0; cb < parts; cb += kJoinBatch) {
    const int nb = min(kJoinBatch, parts - cb);
    for (int c = j; c < nb; c += kCols) {
      const float2 ml = __ldcg(&a.part_ml[slot_of(sp, sp.c0 + cb + c, per) * RT + r]);
      const float f = ex2(ml.x - base);
      scratch[2 * c] = f;
      scratch[2 * c + 1] = f * ml.y;
    }
    __syncwarp(mask);
#pragma unroll 8
    for (int c = 0; c < nb; ++c) {
      const float4 v =
          __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot_of(sp, sp.c0 + cb + c, per) * RT + r) * D + col));
      const float f = scratch[2 * c];
      L += scratch[2 * c + 1];
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    __syncwarp(mask);
  }
  const size_t row = out_row<RT>(a, s, g, rt, r);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + row * D + col) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && j == 0) a.lse[row] = (M + log2f(L)) * kLn2;
}

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
  const Shape sh = shape_of<RT, TK>(s, a.G, a.Hkv);
  const int g = h / a.G, ri = (t - s.start) * a.G + (h - g * a.G);
  const int rt = ri / RT, per = a.starts[a.bt.B];
  const Span sp = span_of(a.starts[b] + (g * sh.rt + rt) * sh.kt, sh.kt, per);
  if (sp.c0 == sp.c1) return;
  join_row<D, RT>(a, s, sp, per, g, rt, ri - rt * RT, scratch[rr]);
}

}  // namespace pattn
}  // namespace mnw
