// The K largest of n keys by one block: a radix select on 11-bit digits, then the
// places of the chosen ones in rising order; of equal keys the earlier places.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace coli {

// Tokens of sequence b: within the table, else latched and cut.
COLI_DEV int context_len(const int32_t* seq_lens, int b, int max_pages, int page_size, int* status,
                         bool latch) {
  int len = __ldg(seq_lens + b);
  const int most = max_pages * page_size;
  if (len < 0 || len > most) {
    if (latch) latch_error(status, kErrDevice);
    len = len < 0 ? 0 : most;
  }
  return len;
}

// Unsigned keys in the numbers' order; NaN counts as -infinity, -0 as 0.
COLI_DEV uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x != x ? -INFINITY : x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
COLI_DEV uint64_t order_key(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x != x ? -INFINITY : x + 0.));
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

constexpr int kDigit = 11, kBins = 1 << kDigit;

struct PickShared {
  int bins[kBins];
  int warp[2][32];
  unsigned long long low[32], top[32];
  int bin, above, in_bin;
};

// What is chosen: keys above `from`, and of those equal to it the first `equal`.
template <class Key>
struct Cut {
  Key from;
  int equal;
};

// Sum of the first w of kW <= 32 numbers (a warp; w the same for its lanes).
template <int kW>
COLI_DEV int before(const int* v, int w) {
  const int lane = lane_id();
  int x = lane < kW && lane < w ? v[lane] : 0;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
  return x;
}

// The K-th largest of n keys, 1 <= K <= n; key(i) for i < n. Every thread of the block calls it.
// The largest key of all, ~0, stands for what is chosen in any case. Digits are taken from the
// highest bit in which the other keys differ: numbers of a few octaves spread over the bins
// (by their own highest bits they meet in ten of them, and wait for each other). EARLY: a bin
// that is chosen whole ends the search (`from` is then below the bin's keys, none of the n).
template <int THREADS, bool EARLY, class Key, class F>
COLI_DEV Cut<Key> radix_cut(int n, int K, F key, PickShared& s) {
  constexpr int kBits = sizeof(Key) * 8, kW = THREADS / 32;
  constexpr Key kAll = static_cast<Key>(~0ull);
  const int lane = lane_id(), w = threadIdx.x / 32;
  Key low = kAll, top = 0;
  int sure = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const Key k = key(i);
    sure += k == kAll;
    low = k < low ? k : low;  // (kAll, the largest, changes nothing here)
    top = k > top && k != kAll ? k : top;
  }
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const Key a = __shfl_xor_sync(0xffffffffu, low, i), b = __shfl_xor_sync(0xffffffffu, top, i);
    low = a < low ? a : low;
    top = b > top ? b : top;
    sure += __shfl_xor_sync(0xffffffffu, sure, i);
  }
  if (lane == 0) s.low[w] = low, s.top[w] = top, s.warp[0][w] = sure;
  __syncthreads();
  low = lane < kW ? static_cast<Key>(s.low[lane]) : kAll;
  top = lane < kW ? static_cast<Key>(s.top[lane]) : 0;
  sure = lane < kW ? s.warp[0][lane] : 0;
#pragma unroll
  for (int i = 1; i < kW; i <<= 1) {
    const Key a = __shfl_xor_sync(0xffffffffu, low, i), b = __shfl_xor_sync(0xffffffffu, top, i);
    low = a < low ? a : low;
    top = b > top ? b : top;
    sure += __shfl_xor_sync(0xffffffffu, sure, i);
  }
  low = __shfl_sync(0xffffffffu, low, 0);
  top = __shfl_sync(0xffffffffu, top, 0);
  sure = __shfl_sync(0xffffffffu, sure, 0);
  __syncthreads();
  int need = K - sure;
  if (need <= 0) return {kAll, K};
  int high = low == top ? 0 : 64 - __clzll(static_cast<unsigned long long>(low ^ top));
  Key prefix = high >= kBits ? 0 : low >> high;
#pragma unroll 1
  while (high > 0) {
    const int width = high < kDigit ? high : kDigit, shift = high - width;
    for (int i = threadIdx.x; i < kBins; i += THREADS) s.bins[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const Key k = key(i);
      if (k != kAll && (high >= kBits || (k >> (high & (kBits - 1))) == prefix))
        atomicAdd(&s.bins[static_cast<int>(k >> shift) & ((1 << width) - 1)], 1);
    }
    __syncthreads();
    // thread t: the bins from kBins - (t + 1) * kEach up; counts of the bins above
    constexpr int kEach = kBins / THREADS;
    const int at = kBins - (threadIdx.x + 1) * kEach;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += s.bins[at + i];
    int upto = sum;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, i);
      if (lane >= i) upto += o;
    }
    if (lane == 31) s.warp[0][w] = upto;
    __syncthreads();
    upto += before<kW>(s.warp[0], w);
    if (upto >= need && upto - sum < need) {
      int above = upto - sum;
      for (int i = kEach - 1; i >= 0; --i) {
        const int c = s.bins[at + i];
        if (above + c >= need) {
          s.bin = at + i;
          s.above = above;
          s.in_bin = c;
          break;
        }
        above += c;
      }
    }
    __syncthreads();
    prefix = static_cast<Key>(prefix << width) | static_cast<Key>(s.bin);
    need -= s.above;
    high = shift;
    const int in_bin = s.in_bin;
    __syncthreads();
    if (EARLY && in_bin == need) {  // the whole bin
      const Key least = static_cast<Key>(prefix << shift);
      if (least > 0) return {static_cast<Key>(least - 1), 0};
      return {0, n};
    }
  }
  return {prefix, need};
}

// put(rank, i) for the chosen places i in rising order.
template <int THREADS, class Key, class F, class P>
COLI_DEV void chosen(int n, const Cut<Key>& cut, F key, P put, PickShared& s) {
  constexpr int kW = THREADS / 32;
  const int lane = lane_id(), w = threadIdx.x / 32;
  const int each = ((n + kW - 1) / kW + 31) / 32 * 32;  // places of a warp
  const int i0 = w * each, i1 = min(n, i0 + each);
  int over = 0, same = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const Key k = key(i);
    over += k > cut.from;
    same += k == cut.from;
  }
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    over += __shfl_xor_sync(0xffffffffu, over, i);
    same += __shfl_xor_sync(0xffffffffu, same, i);
  }
  if (lane == 0) s.warp[0][w] = over, s.warp[1][w] = same;
  __syncthreads();
  // chosen above and equal ones before this warp's places
  int a = before<kW>(s.warp[0], w), b = before<kW>(s.warp[1], w);
  if (over == 0 && (same == 0 || b >= cut.equal)) return;
#pragma unroll 2
  for (int i = i0; i < i1; i += 32) {
    const Key k = i + lane < i1 ? key(i + lane) : 0;
    const bool in = i + lane < i1;
    const uint32_t hi = __ballot_sync(0xffffffffu, in && k > cut.from);
    const uint32_t eq = __ballot_sync(0xffffffffu, in && k == cut.from);
    if ((hi | eq) == 0) continue;
    const uint32_t below = (1u << lane) - 1;
    const int ra = a + __popc(hi & below), rb = b + __popc(eq & below);
    if (in && (k > cut.from || (k == cut.from && rb < cut.equal)))
      put(ra + min(rb, cut.equal), i + lane);
    a += __popc(hi);
    b += __popc(eq);
  }
}

}  // namespace coli
