// How a decode cuts the slots of all sequences into units, and its CTAs' shares of
// them (see fa2_paged_decode.cu).
#pragma once
#include "fa2_cache.cuh"

namespace fa2 {

// Slots per unit: 32 KiB of K and V. A warp has 16 (d = 128) or 32 (d = 64) of
// them, so that its fixed cost per unit (maximum, ring, cursor) is spread over
// the same bytes at both head sizes.
template <int D>
constexpr int kUnit = decode_unit(D);
constexpr int kDecWarps = 4;  // of a CTA of the decode
constexpr float kLn2f = 0.6931471805599453f;
constexpr float kLog2ef = 1.4426950408889634f;

// ---- Units ---------------------------------------------------------------
// HH = Hkv * HG items per sequence: item hh is head tile hh % HG of key head hh / HG.
// SHARED: a sequence that reaches the prefix has the slots behind it only; before all
// sequences may come items of the prefix itself (b = -1, hh their number).
// Its workers are CTAs, or warps with units of a warp's share of the others'.
enum : int { kNotShared = 0, kSharedCta = 1, kSharedWarp = 2 };
template <int D, int SHARED = kNotShared>
__device__ __forceinline__ int tiles_of(int n) {
  constexpr int U = SHARED == kSharedWarp ? kUnit<D> / kDecWarps : kUnit<D>;
  return (n + U - 1) / U;
}

// Quotient of 0 <= a and b > 0; 32 bits when they do, which is nearly always.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

struct UnitCursor {
  int b, hh, tile;  // sequence, item of the sequence, unit of the item
  int n, ntiles;    // slots of the sequence, units of the item
  int start;        // SHARED: slots of the prefix before them
};

// Slots of the prefix that a sequence of n slots leaves to it.
__device__ __forceinline__ int prefix_of(int n, const PrefixLen& p) { return n >= p.len ? p.cut : 0; }

// The units of all sequences, by a whole warp: T, and where a unit lies. Up to
// 32 sequences are read once and their running sums stay with the lanes.
template <int D, int SHARED = kNotShared>
struct UnitMap {
  const CacheView& c;
  int HH, lane;
  PrefixLen P;
  int n;
  long long incl, T;

  __device__ UnitMap(const CacheView& view, int hh, int l, PrefixLen prefix = {}) : c(view), HH(hh), lane(l), P(prefix) {
    n = length(lane);
    incl = scan(n);
    T = __shfl_sync(0xffffffffu, incl, 31);
    for (int b0 = 32; b0 < c.B; b0 += 32) T += __shfl_sync(0xffffffffu, scan(length(b0 + lane)), 31);
  }
  __device__ int length(int b) const {
    if (b >= c.B) return 0;
    const int x = seq_len(c, b);
    return SHARED != kNotShared ? x - prefix_of(x, P) : x;
  }
  // out[b]: units before those of sequence b, `base` before all; out[B] = base + T.
  __device__ void write_starts(long long* out, long long base) const {
    if (lane == 0) out[c.B] = base + T;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
      const int len = b0 == 0 ? n : length(b0 + lane);
      const long long sum = scan(len);
      if (b0 + lane < c.B) out[b0 + lane] = base + sum - static_cast<long long>(tiles_of<D, SHARED>(len)) * HH;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __device__ long long scan(int slots) const {
    long long t = static_cast<long long>(tiles_of<D, SHARED>(slots)) * HH;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    return t;
  }
  // Cursor of unit u < T.
  __device__ UnitCursor at(long long u) const {
    long long base = 0, sum = incl;
    int len = n;
    for (int b0 = 0;; b0 += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, u < base + sum);
      if (hit != 0u) {
        const int src = __ffs(hit) - 1;
        UnitCursor k;
        k.b = b0 + src;
        k.n = __shfl_sync(0xffffffffu, len, src);
        k.ntiles = tiles_of<D, SHARED>(k.n);
        k.start = SHARED != kNotShared ? prefix_of(seq_len(c, k.b), P) : 0;
        const long long r = u - (base + __shfl_sync(0xffffffffu, sum, src) - static_cast<long long>(k.ntiles) * HH);
        k.hh = static_cast<int>(div_pos(r, k.ntiles));
        k.tile = static_cast<int>(r - static_cast<long long>(k.hh) * k.ntiles);
        return k;
      }
      if (b0 + 32 >= c.B) return UnitCursor{};
      base += __shfl_sync(0xffffffffu, sum, 31);
      len = length(b0 + 32 + lane);
      sum = scan(len);
    }
  }
};

template <int D, int SHARED = kNotShared>
__device__ __forceinline__ void unit_advance(const CacheView& c, int HH, UnitCursor& k, PrefixLen P = {}, int prefix_items = 0) {
  if (++k.tile < k.ntiles) return;
  k.tile = 0;
  if (++k.hh < (SHARED != kNotShared && k.b < 0 ? prefix_items : HH)) return;
  k.hh = 0;
  do {
    if (++k.b >= c.B) {
      k.n = k.ntiles = 0;
      return;
    }
    k.n = seq_len(c, k.b);
    if constexpr (SHARED != kNotShared) {
      k.start = prefix_of(k.n, P);
      k.n -= k.start;
    }
  } while (k.n == 0);
  k.ntiles = tiles_of<D, SHARED>(k.n);
}

// Units [u0, u1) of CTA x of G over T units, and the CTA of unit u. With fewer
// units than CTAs, T CTAs take one each.
__device__ __forceinline__ long long unit_begin(long long x, long long G, long long T) { return div_pos(x * T, G); }
__device__ __forceinline__ int unit_cta(long long u, long long G, long long T) {
  return static_cast<int>(div_pos((u + 1) * G - 1, T));
}

// The same where the first `early` workers begin beside the prefix's kernel and the others
// when it ends: kShares + k parts for kShares - k of a later one. k = 0: all alike.
constexpr int kShares = 8, kMaxUneven = 4;
struct UnitDeal {
  long long T;  // units
  int S, early, more, less;  // parts of them
  __device__ __forceinline__ UnitDeal(int G, int first, long long units, int k) : T(units) {
    early = k == 0 ? 0 : first;
    more = k == 0 ? 1 : kShares + k;
    less = k == 0 ? 1 : kShares - k;
    S = more * early + less * (G - early);
  }
  __device__ __forceinline__ long long begin(int x) const {
    return unit_begin(less * x + (more - less) * min(x, early), S, T);
  }
  __device__ __forceinline__ int worker(long long u) const {
    const int s = unit_cta(u, S, T), e = more * early;
    const bool late = s >= e;
    // s / more: below 2^14, so that half of 1 / more is far above the error.
    const float q = __fdividef(static_cast<float>(late ? s - e : s) + 0.5f, static_cast<float>(late ? less : more));
    return early == 0 ? s : (late ? early : 0) + static_cast<int>(q);
  }
};

// k of a call whose workers are warps and whose prefix has a kernel of its own: five times the time that the early
// workers have alone (about 4 us of its start and end, and 4.8, or 3.4 at d = 64, per slot
// tile of two row tiles) by the time that all units take, as far as every worker then has a
// unit. 64 sequences behind 8192 slots, 32/8 heads, d = 128, up to 1024 own slots: 50.1 us
// and 53.4 with equal shares; up to 4000: 118.3 and 121.4; up to 300: 37.0 and 36.9; d = 64,
// fp16, up to 1024: 37.2 and 42.0. The other way round: d = 128 in fp16, whose own slots'
// products take longer than the rule's time for them, 61.6 and 56.6; and 16 sequences of
// 128/4 heads behind 16384 slots, 52.9 and 49.3.
template <int D>
__device__ __forceinline__ int uneven_shares(const DecodeArgs& a, int cut, int G, int first, long long T) {
  if (a.early == 0 || G < 2 * first || cut == 0) return 0;
  const float tiles = static_cast<float>(a.prefix_items) * static_cast<float>((cut + 127) / 128);
  const float alone = 4000.f + __fdividef(tiles * (D == 128 ? 4800.f : 3400.f), static_cast<float>(a.early));  // ns
  const int k = static_cast<int>(fminf(__fdividef(5.f * alone, static_cast<float>(T) * 2.f) + 0.5f, kMaxUneven));
  return (kShares - k) * T >= (kShares + k) * first + (kShares - k) * (G - first) ? k : 0;
}

// 2^(from - to) for a reference that rises to `to`. 1 at -inf, where all that
// there is are zeros, or NaN that has to stay.
__device__ __forceinline__ float step_down(float from, float to) { return from == to ? 1.f : ex2_approx(from - to); }

}  // namespace fa2
