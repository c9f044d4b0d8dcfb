// The quantised KV cache (sm_103a): record layout, e4m3 conversions, and the
// page lists of the attention kernels that read it.
//
// A record holds one (page, KV head): the e4m3 codes of 16 key rows, of 16
// value rows, and one power-of-two scale per row (include/locks.h).  It is
// one contiguous, 16-byte aligned run of 4128 bytes = 129 memory sectors, so
// one bulk copy brings a page's keys, values and scales on chip.  A scale
// that is a power of two makes x / 2^e exact: the codes do not depend on how
// the division is carried out, and a number read back is exact in bf16.
#pragma once

#include "common.cuh"

namespace locks {

constexpr int kQRec = LOCKS_KV_RECORD_BYTES;  // 4128
constexpr int kQCodes = kPage * kDim;         // codes of keys or of values
constexpr int kQOffV = kQCodes;
constexpr int kQOffKE = 2 * kQCodes;          // key scale exponents
constexpr int kQOffVE = kQOffKE + kPage;      // value scale exponents
constexpr int kQExpLo = -32, kQExpHi = 31;    // limits of a scale exponent

static_assert(kQOffVE + kPage == kQRec, "record size");

// attention: scores in base 2; weights are 2^(score - m + 8), their reference m
// trails the largest score by at most 7
constexpr float kQScale = 0.12751743074602467f;  // log2(e) / sqrt(128)
constexpr float kQLift = 8.f, kQSlack = 7.f;
// value scales further apart than 2^8 leave fp16 weights too few bits
constexpr uint32_t kQSpread = 8;

// Where the 16-byte group c (dims 16c .. 16c + 15) of the row in slot s sits
// in the row.  Both readings of a record from shared memory are then free of
// bank conflicts: eight lanes that read key rows 2i, 2i + 1, groups 4j .. 4j
// + 3 (slots that differ in bit 0 use different halves of the row), and
// eight lanes that read groups 2i, 2i + 1 of value rows 0, 2, 4, 6 or
// 1, 3, 5, 7.
__host__ __device__ __forceinline__ int q_group(int c, int s) {
  return c ^ (s & 6) ^ ((s & 1) * 5);
}

// Exponent of a row's scale: the least e with absmax <= 448 * 2^e, limited.
// 448 = 1.75 * 2^8, so e = E - 8 for absmax = 1.m * 2^E with 1.m <= 1.75 and
// E - 7 above; zero and subnormal maxima fall to the lower limit, infinity
// to the upper.
__device__ __forceinline__ int q_exponent(float absmax) {
  const uint32_t b = __float_as_uint(absmax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
  return max(kQExpLo, min(kQExpHi, e));
}

// A value scale's byte as the attention takes it.  Zeroed records, which no row
// has been written to, hold 0 there: codes of zero, so that any scale stands
// for the same values, and the format's least keeps 2^-127 out of the factors.
__device__ __forceinline__ uint32_t q_scale_byte(uint32_t b) {
  return max(b, (uint32_t)(kQExpLo + 127));
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// two numbers -> two e4m3 codes (low byte: lo), round to nearest even,
// clamped to +-448, NaN kept
__device__ __forceinline__ uint32_t e4m3x2_from(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 codes (low 16 bits of x, or high) -> half2, exact
__device__ __forceinline__ uint32_t e4m3x2_lo(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n"
      " cvt.rn.f16x2.e4m3x2 %0, l;\n}\n"
      : "=r"(r)
      : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n"
      " cvt.rn.f16x2.e4m3x2 %0, h;\n}\n"
      : "=r"(r)
      : "r"(x));
  return r;
}

// Waits are bounded in time (about a second), not in tries: a try may itself
// wait on the barrier for as long as the hardware likes.
constexpr long long kQWaitCycles = 1LL << 31;

// false when the barrier did not complete in time
__device__ __forceinline__ bool q_wait(uint64_t *bar, uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const long long t0 = clock64();
  do {
    if (mbar_try_wait(bar, phase)) return true;
  } while (clock64() - t0 < kQWaitCycles);
  return false;
}

// ---------------------------------------------------------------------------
// page lists
// ---------------------------------------------------------------------------
// The list entries ("positions") of all (sequence, KV head) units laid end to
// end: sequence b's h_kv units are consecutive, each as long as b's list, and
// start at first(b): b * h_kv * k where every list has k entries (per_seq =
// h_kv * k), pre[b] where a list is the sequence's own pages (per_seq = 0).
struct PageLists {
  const int *pre;
  int batch, h_kv, per_seq;

  __device__ __forceinline__ int first(int b) const {
    return per_seq ? b * per_seq : pre[b];
  }
  __device__ __forceinline__ int length(int b) const {
    return (first(b + 1) - first(b)) / h_kv;
  }
  __device__ __forceinline__ int sequence(int p) const {  // p below the total
    if (per_seq) return p / per_seq;
    int lo = 0, hi = batch;  // the last b with pre[b] <= p
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= p) lo = mid; else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ int unit(int p) const {
    const int b = sequence(p);
    return b * h_kv + (p - first(b)) / length(b);
  }
  __device__ __forceinline__ int2 span(int u) const {  // positions of unit u
    const int b = u / h_kv, n = length(b);
    const int f = first(b) + (u - b * h_kv) * n;
    return make_int2(f, f + n);
  }
};

// This thread's accesses to shared memory so far come before what the copy
// engine and the tensor core do there for it later: reads of a buffer before
// the next copy into it (without the fence, a loop that had only __syncwarp
// between them was seen to read the next tile's values), writes before the
// product that reads them.
__device__ __forceinline__ void fence_to_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

__device__ __forceinline__ int checked_len(const int32_t *seq_lens, int b,
                                           int max_pages, int32_t *status) {
  const int L = __ldcg(seq_lens + b);  // not by L1: see QdArgs::beside
  const int top = max_pages * kPage;
  if (L < 0 || L > top) {
    set_status(status, LOCKS_DEV_BAD_SEQ_LEN);
    return L < 0 ? 0 : top;
  }
  return L;
}

}  // namespace locks
