// mnw_paged.cuh -- what the paged key/value cache's kernels share: the cache's
// description, a sequence's new tokens and length, and the page of a position.
//
// Cache: k and v [n_pages][Hkv][page_size][d] (a page of one head is
// contiguous), consecutive pages page_stride elements apart; INT8 caches hold
// codes and k_scale, v_scale [n_pages][Hkv][page_size] f32, one scale per
// cached head row.  Position p of sequence b lives in page
// block_table[b][p / page_size], slot p % page_size.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mnw_moe.h"

namespace mnw {
namespace paged {

// x / d for 0 <= x < 2^31 by a multiplication (round-up method): with
// s = ceil(log2 d) and mul = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (mulhi(x, mul) + x) >> s.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ uint32_t quotient(uint32_t x, const FastDiv& f) {
  return (__umulhi(x, f.mul) + x) >> f.shift;
}

struct Batch {
  const int32_t* block_table;  // [B][max_pages]
  const int32_t* cache_lens;   // [B], the new tokens included
  const int32_t* q_start;      // [B + 1] or null: n_uniform tokens a sequence
  int B, T, max_pages, n_uniform;
};

struct Seq {
  int start, n, len;  // first token row, new tokens, cached positions (those that the block table holds)
  int first;          // position of the first new token
};

// Sequence b, with values that would lead out of the token rows or of the
// block table brought back inside (*bad tells).  Positions come from the values
// as they are given: a length past the table, or rows past the last, must not
// move the other tokens to slots that hold earlier ones.  So positions below 0
// or from `len` on can occur; their tokens have no slot.
__device__ __forceinline__ Seq sequence(const Batch& bt, int b, int page_size, bool* bad) {
  Seq s;
  int given;  // new tokens from row `start` on
  if (bt.q_start) {
    const int lo = __ldg(bt.q_start + b), hi = __ldg(bt.q_start + b + 1);
    s.start = max(0, min(lo, bt.T));
    s.n = max(0, min(hi, bt.T) - s.start);
    *bad = lo != s.start || hi != s.start + s.n;
    given = s.n > 0 ? hi - s.start : 0;
  } else {
    s.start = b * bt.n_uniform;
    s.n = given = bt.n_uniform;
    *bad = false;
  }
  const int len = __ldg(bt.cache_lens + b);
  const long long room = static_cast<long long>(bt.max_pages) * page_size;
  s.len = len < 0 ? 0 : (len > room ? static_cast<int>(room) : len);
  s.first = max(len, 0) - given;
  *bad = *bad || s.len != len || len < given;
  return s;
}

// Whether sequence b's range of rows runs backwards.  Where none does, the
// ranges are disjoint and hold at most T rows together, which bounds the work
// that the host planned for.
__device__ __forceinline__ bool backwards(const Batch& bt, int b) {
  return bt.q_start && __ldg(bt.q_start + b) > __ldg(bt.q_start + b + 1);
}

// Argument checks shared by the calls on a cache.
inline int check_cache(const void* k, const void* v, const float* ks, const float* vs, int fmt, int n_pages,
                       int page_size, int Hkv, int d, long long page_stride) {
  if (fmt != MNW_KV_BF16 && fmt != MNW_KV_INT8) return MNW_E_INVALID_ARG;
  if (n_pages <= 0 || page_size <= 0 || Hkv <= 0 || d <= 0) return MNW_E_INVALID_ARG;
  if (d != 64 && d != 128) return MNW_E_UNSUPPORTED;
  if (page_size > 65536 || Hkv > 1024) return MNW_E_UNSUPPORTED;
  const int unit = fmt == MNW_KV_BF16 ? 8 : 16;  // 16 bytes
  if (page_stride < static_cast<long long>(Hkv) * page_size * d || page_stride % unit) return MNW_E_INVALID_ARG;
  if (!k || !v || (reinterpret_cast<uintptr_t>(k) & 15) || (reinterpret_cast<uintptr_t>(v) & 15))
    return MNW_E_INVALID_ARG;
  if (fmt == MNW_KV_INT8 &&
      (!ks || !vs || (reinterpret_cast<uintptr_t>(ks) & 3) || (reinterpret_cast<uintptr_t>(vs) & 3)))
    return MNW_E_INVALID_ARG;
  return MNW_OK;
}
inline int check_batch(const int32_t* table, const int32_t* lens, const int32_t* q_start, int B, int T,
                       int max_pages, int page_size) {
  if (!table || !lens || (reinterpret_cast<uintptr_t>(table) & 3) || (reinterpret_cast<uintptr_t>(lens) & 3) ||
      (reinterpret_cast<uintptr_t>(q_start) & 3))
    return MNW_E_INVALID_ARG;
  if (max_pages <= 0 || (!q_start && T % B)) return MNW_E_INVALID_ARG;
  // positions are 32-bit
  if (static_cast<long long>(max_pages) * page_size > 0x7fffffffll - 65536) return MNW_E_UNSUPPORTED;
  return MNW_OK;
}

}  // namespace paged
}  // namespace mnw
