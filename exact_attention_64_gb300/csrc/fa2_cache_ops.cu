// Writes to the paged cache: appending new tokens, and eviction.
#include "fa2_cache.cuh"

namespace fa2 {

// ---- Append ----------------------------------------------------------------
// New token i of sequence b and key head h goes to slot lens[b] + i. A copy:
// bound by HBM for prompts (521 MB in 84 us, 6.17 TB/s, at B = 4, 32 heads of up
// to 8192 tokens, d = 128) and by three dependent reads for single tokens (256
// heads in 3.0 us). One thread moves 16 bytes of K and of V; consecutive threads
// walk a row. One row per thread: two, four and eight per thread, their loads in
// flight together, took 90, 128 and 207 us and 3.4, 4.4 and 6.5 us.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) fa2_cache_append_kernel(const AppendArgs a) {
  constexpr int CH = D / 8;                 // 16-byte chunks of a row
  constexpr int ROWS = kAppendThreads / CH;  // rows per CTA
  grid_dependency_wait();
  const CacheView& c = a.c;
  const int ch = threadIdx.x % CH;
  const long long r = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / CH;
  // New lengths, by the first CTA. A length or a count outside its range is
  // cut and reported.
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < c.B; b += kAppendThreads) {
      const int n = seq_len(c, b);
      const int want = a.num_new != nullptr ? ld_global(a.num_new + b) : a.T;
      const int cnt = cut_len(want, a.T);
      if (n != ld_global(c.lens + b) || cnt != want || n > c.L - cnt) report_page(c.status);
      a.lens_out[b] = n > c.L - cnt ? c.L : n + cnt;
    }
  }
  if (r >= a.rows) return;
  const int rr = static_cast<int>(r), bh = div_by(rr, a.fT), i = rr - bh * a.T;
  const int b = div_by(bh, a.fH), h = bh - b * c.Hkv;
  const int cnt = a.num_new != nullptr ? ld_global(a.num_new + b) : a.T;
  const int n = seq_len(c, b);
  if (i >= cnt || i >= c.L - n) return;  // padding, or no room in the table (n + i may not fit in 31 bits)
  const int slot = n + i;
  const uint4 kx = ld_once(reinterpret_cast<const uint4*>(a.k + static_cast<size_t>(rr) * D) + ch);
  const uint4 vx = ld_once(reinterpret_cast<const uint4*>(a.v + static_cast<size_t>(rr) * D) + ch);
  const int row = slot_row(c, b, h, slot);
  if (row < 0) {
    report_page(c.status);
    return;
  }
  reinterpret_cast<uint4*>(a.kc + static_cast<size_t>(row) * D)[ch] = kx;
  reinterpret_cast<uint4*>(a.vc + static_cast<size_t>(row) * D)[ch] = vx;
  if (ch != 0) return;
  const size_t at = static_cast<size_t>(bh) * c.L + slot;
  if (a.weights != nullptr) a.weights[at] = a.new_weights != nullptr ? ld_global(a.new_weights + rr) : 0.f;
  if (a.positions != nullptr) a.positions[at] = ld_global(a.next_pos + b) + i;
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  const int per = kAppendThreads / (a.d / 8);
  const long long grid = (a.rows + per - 1) / per;
  return launch_dependent(a.d == 64 ? fa2_cache_append_kernel<64> : fa2_cache_append_kernel<128>,
                          dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0, stream, a);
}

// ---- Eviction --------------------------------------------------------------
// Of a sequence and key head with more than `budget` slots the budget slots
// with the largest keys stay. A key orders the slots: recent tokens first
// (position >= next_pos - recent), then by weight, NaN last; equal keys by the
// lower slot. Attention does not depend on the order of the slots, so the kept
// slots below budget stay where they are, and the i-th evicted slot below
// budget takes the i-th kept slot at or past budget: no row moves that does not
// have to, and sources and destinations are disjoint.
//
// Selection: the key becomes a 32-bit integer of the same order, and the
// budget-th largest is found digit by digit, 8 bits a pass, from histograms,
// until all keys that share the digits so far stay: after the third pass as a
// rule (2 heads of 16384 slots 13.1 us back to back, 14.5 with a fourth pass always).
// (The first digit counted in 4 to 16 copies, against collisions: 0.3 us slower.
// Three passes of 11 bits and fewer collisions, before the early launches: no
// faster in one CTA, and 17 against 12 us in a cluster of 8, whose CTAs read each
// other's counters.) A
// (sequence, key head) is the work of one cluster, a warp has a run of its
// slots, and the keys stay in registers, so that weights and positions are
// read once; the histograms of a pass are added up through distributed shared
// memory. Integer counts: the result does not depend on any order. Rows too
// long for the registers of a cluster keep their keys in its shared memory
// (keys in shared memory throughout: 56.0 us for 128 heads of 8192 slots cut to
// 2048, against 51.4; 2 heads of 16384 15.1 and 13.1), and past that make them again
// from global memory. One slot too many, the steady state of a bounded cache, needs
// no histogram: the smallest key goes, of equal ones the highest slot (4.4 us for
// 256 heads of 2049 slots in a table of 2064, against 8.4).
//
// Moves: a warp takes 8 at a time, so that 4 KiB per warp are in flight. A few
// moves per row (a cache that is one token over) are made by the cluster that
// found them; many are left as lists to a second launch whose grid is cut by
// moves, because the clusters of a wave find theirs at the same time and would
// leave the memory idle until then. (32 moves per warp, looked up at once and
// copied four rows at a time with four more on their way: no faster for 128
// heads of 8192 slots, 14.0 us against 13.0 for 2 of 16384.) What "many" is goes by
// the list's capacity, min(budget, L - budget), and so by the table: the 256 heads
// of 2049 slots take 11.3 us in a table of 4096 and 17.4 in one of 8192, for a second
// launch that finds one move each, and for clusters of two.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictRegs = 8;      // keys a thread can hold: 4096 slots per CTA
constexpr int kEvictKeys = 49152;  // keys a CTA's shared memory can hold: 192 KiB
constexpr int kMoveThreads = 256;
constexpr int kMovesPerWarp = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// By all threads of the cluster, each warp converged.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Words of shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long cluster_load64(const unsigned long long* p, uint32_t rank) {
  uint32_t a;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Integer of the same order as a weight: NaN 0, then -inf ... +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  __align__(16) uint32_t hist[4][256];
  __align__(16) uint32_t total[256];
  unsigned long long least[kEvictWarps], cta_least;
  int one[2];  // source and destination of a single move
  uint32_t warp_gt[kEvictWarps], warp_tie[kEvictWarps];  // per warp, then exclusive
  uint32_t cta_gt, cta_tie, cta_gt_lo, cta_tie_lo;       // this CTA's counts
};

// Moves m0 .. m0 + 7 of an item with `moves` of them, by a whole warp: lanes 0 ..
// 7 look up the sources, 8 .. 15 the destinations, then all copy, 16 bytes of K
// and of V per lane and row.
template <int D>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int item, const int* movers, const int* holes, int m0,
                                          int moves, int lane) {
  const CacheView& c = a.c;
  const int b = item / c.Hkv, h = item - b * c.Hkv;
  const size_t base = static_cast<size_t>(item) * c.L;
  const int m = m0 + (lane & 7);
  int slot = 0, row = -1;
  if (lane < 16 && m < moves) {
    slot = (lane < 8 ? movers : holes)[m];
    row = slot_row(c, b, h, slot);
    if (row < 0) report_page(c.status);
  }
  const int to = __shfl_down_sync(0xffffffffu, slot, 8);
  if (lane < 8 && m < moves) {
    a.w_out[base + to] = a.w_in[base + slot];
    if (a.p_in != nullptr) a.p_out[base + to] = a.p_in[base + slot];
  }
  constexpr int CH = D / 8, RPI = 32 / CH, IT = kMovesPerWarp / RPI;
  const int ch = lane % CH, sub = lane / CH;
  uint4 kx[IT], vx[IT];
  int dst[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int s = __shfl_sync(0xffffffffu, row, i * RPI + sub);
    dst[i] = __shfl_sync(0xffffffffu, row, 8 + i * RPI + sub);
    if (s < 0) dst[i] = -1;
    if (dst[i] >= 0) {
      kx[i] = reinterpret_cast<const uint4*>(a.kc + static_cast<size_t>(s) * D)[ch];
      vx[i] = reinterpret_cast<const uint4*>(a.vc + static_cast<size_t>(s) * D)[ch];
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    if (dst[i] < 0) continue;
    reinterpret_cast<uint4*>(a.kc + static_cast<size_t>(dst[i]) * D)[ch] = kx[i];
    reinterpret_cast<uint4*>(a.vc + static_cast<size_t>(dst[i]) * D)[ch] = vx[i];
  }
}

template <int D, bool REG>
__global__ void __launch_bounds__(kEvictThreads) fa2_cache_evict_kernel(const EvictArgs a, int C) {
  extern __shared__ uint32_t s_keys[];
  __shared__ EvictShared sh;
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / C;
  const int rank = static_cast<int>(C > 1 ? cluster_rank() : 0u);
  const int b = item / c.Hkv, h = item - b * c.Hkv;
  const int n = seq_len(c, b);
  const int k = min(n, a.budget);
  const size_t base = static_cast<size_t>(item) * c.L;
  const float* w_in = a.w_in + base;
  float* w_out = a.w_out + base;
  const int* p_in = a.p_in != nullptr ? a.p_in + base : nullptr;
  int* p_out = a.p_in != nullptr ? a.p_out + base : nullptr;
  const bool copy_w = a.w_out != a.w_in, copy_p = p_in != nullptr && a.p_out != a.p_in;
  if (rank == 0 && tid == 0) {
    if (h == 0) {
      if (n != ld_global(c.lens + b)) report_page(c.status);
      a.lens_out[b] = k;
    }
    if (n <= a.budget) a.counts[item] = 0;
  }
  if (n <= a.budget) {  // nothing to evict
    for (int j = rank * kEvictThreads + tid; j < n; j += C * kEvictThreads) {
      if (copy_w) w_out[j] = w_in[j];
      if (copy_p) p_out[j] = p_in[j];
    }
    return;  // the whole cluster
  }
  // This CTA's slots are kEvictWarps runs of whole 32s, one per warp; this
  // warp's are [w0, w1), of which a lane has w0 + lane, w0 + 32 + lane, ...
  const int run = (((n + C - 1) / C + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int j0 = min(n, rank * run * kEvictWarps), j1 = min(n, j0 + run * kEvictWarps);
  const int w0 = min(j1, j0 + warp * run), w1 = min(j1, w0 + run);
  const long long first_recent =
      p_in != nullptr ? static_cast<long long>(ld_global(a.next_pos + b)) - a.recent : 0;
  auto key_of = [&](int j, float w, int pos) -> uint32_t {
    // Without positions the slots are in the order of their tokens.
    const bool is_recent = p_in != nullptr ? pos >= first_recent : j >= n - a.recent;
    return is_recent && a.recent > 0 ? 0xffffffffu : weight_key(w);
  };
  // Each of the warp's slots in order of i, `f(i, j)`: i-th 32 of the run.
  uint32_t key[REG ? kEvictRegs : 1];
  auto each = [&](auto f) {
    if constexpr (REG) {
#pragma unroll
      for (int i = 0; i < kEvictRegs; ++i) f(i, w0 + 32 * i + lane);
    } else {
      for (int i = 0; w0 + 32 * i < w1; ++i) f(i, w0 + 32 * i + lane);
    }
  };
  // Keys, and the copies of the slots below budget: evicted ones are written
  // again when a kept slot takes their place.
  auto load_key = [&](int j) -> uint32_t {
    const float w = w_in[j];
    const int pos = p_in != nullptr ? p_in[j] : 0;
    return key_of(j, w, pos);
  };
  if constexpr (REG) {
    float w[kEvictRegs];
    int pos[kEvictRegs];
    each([&](int i, int j) {
      w[i] = j < w1 ? w_in[j] : 0.f;
      pos[i] = j < w1 && p_in != nullptr ? p_in[j] : 0;
    });
    each([&](int i, int j) {
      key[i] = key_of(j, w[i], pos[i]);
      if (j < w1 && j < k) {
        if (copy_w) w_out[j] = w[i];
        if (copy_p) p_out[j] = pos[i];
      }
    });
  } else {
    each([&](int, int j) {
      if (j >= w1) return;
      if (a.cached) s_keys[j - j0] = load_key(j);
      if (j < k) {
        if (copy_w) w_out[j] = w_in[j];
        if (copy_p) p_out[j] = p_in[j];
      }
    });
  }
  auto key_at = [&](int i, int j) -> uint32_t {
    if constexpr (REG) return key[i];
    else return a.cached ? s_keys[j - j0] : load_key(j);
  };
  if (n - k == 1) {
    // The smallest key, of equal ones the highest slot, as one number to
    // minimise: key, then the slot's complement.
    unsigned long long least = ~0ull;
    each([&](int i, int j) {
      if (j >= w1) return;
      const unsigned long long x = (static_cast<unsigned long long>(key_at(i, j)) << 32) | ~static_cast<uint32_t>(j);
      least = x < least ? x : least;
    });
    auto warp_least = [&](unsigned long long x) {
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, x, o);
        x = y < x ? y : x;
      }
      return x;
    };
    least = warp_least(least);
    if (lane == 0) sh.least[warp] = least;
    __syncthreads();
    if (C > 1) {
      if (warp == 0) {
        least = warp_least(lane < kEvictWarps ? sh.least[lane] : ~0ull);
        if (lane == 0) sh.cta_least = least;
      }
      cluster_sync();
    }
    if (rank == 0 && warp == 0) {
      unsigned long long x = ~0ull;
      if (C > 1) {
        if (lane < C) x = cluster_load64(&sh.cta_least, lane);
      } else if (lane < kEvictWarps) {
        x = sh.least[lane];
      }
      const int gone = static_cast<int>(~static_cast<uint32_t>(warp_least(x)));
      if (lane == 0) {
        a.counts[item] = 0;
        sh.one[0] = k;
        sh.one[1] = gone;
      }
      __syncwarp();
      if (gone < k) move_rows<D>(a, item, &sh.one[0], &sh.one[1], 0, 1, lane);
    }
    if (C > 1) cluster_sync();  // the others' shared memory has been read
    return;
  }
  for (int i = tid; i < 4 * 256; i += kEvictThreads) (&sh.hist[0][0])[i] = 0u;
  if (tid == 0) sh.cta_gt = sh.cta_tie = sh.cta_gt_lo = sh.cta_tie_lo = 0u;
  __syncthreads();
  uint32_t prefix = 0, want = k;  // the want-th largest among the keys that start with prefix
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    shift -= 8;
    each([&](int i, int j) {
      if (j >= w1) return;
      const uint32_t x = key_at(i, j);
      if (pass == 0 || (x >> (shift + 8)) == prefix) atomicAdd(&sh.hist[pass][(x >> shift) & 255u], 1u);
    });
    const uint32_t* total = sh.hist[pass];
    if (C > 1) {
      cluster_sync();
      if (tid < 256) {
        uint32_t t = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x < C) t += cluster_load(&sh.hist[pass][tid], x);
        sh.total[tid] = t;
      }
      total = sh.total;
    }
    __syncthreads();
    // Every warp finds the digit for itself: lane l has digits 255 - 8 l ...
    // 248 - 8 l, the largest first.
    uint32_t v[8], sum = 0;
    *reinterpret_cast<uint4*>(&v[0]) = *reinterpret_cast<const uint4*>(total + 248 - 8 * lane);
    *reinterpret_cast<uint4*>(&v[4]) = *reinterpret_cast<const uint4*>(total + 252 - 8 * lane);
#pragma unroll
    for (int x = 0; x < 8; ++x) sum += v[x];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    uint32_t above = incl - sum, digit = 0, left = 0, all = 0;
    const unsigned hit = __ballot_sync(0xffffffffu, above < want && want <= incl);
#pragma unroll
    for (int x = 7; x >= 0; --x) {
      if (above < want && want <= above + v[x]) {
        digit = 248 - 8 * lane + x;
        left = want - above;
        all = v[x];
      }
      above += v[x];
    }
    const int src = __ffs(hit) - 1;
    prefix = (prefix << 8) | __shfl_sync(0xffffffffu, digit, src);
    want = __shfl_sync(0xffffffffu, left, src);
    // All keys that start with prefix stay, so every key from the least such one
    // on does. (That one is above 0, or all n keys would stay.)
    if (want == __shfl_sync(0xffffffffu, all, src)) {
      prefix = (prefix << shift) - 1u;
      want = 0u;
      break;
    }
    if (C > 1) __syncthreads();  // sh.total is rewritten by the next pass
  }
  // Slots with a key above `prefix` stay, and the first `want` of those equal to
  // it. Counts before each warp's run, over the cluster in slot order.
  uint32_t gt = 0, tie = 0, gt_lo = 0, tie_lo = 0;
  each([&](int i, int j) {
    if (j >= w1) return;
    const uint32_t x = key_at(i, j);
    const uint32_t g1 = x > prefix, t1 = x == prefix;
    gt += g1;
    tie += t1;
    if (j < k) {
      gt_lo += g1;
      tie_lo += t1;
    }
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  tie = __reduce_add_sync(0xffffffffu, tie);
  gt_lo = __reduce_add_sync(0xffffffffu, gt_lo);
  tie_lo = __reduce_add_sync(0xffffffffu, tie_lo);
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_tie[warp] = tie;
    atomicAdd(&sh.cta_gt, gt);
    atomicAdd(&sh.cta_tie, tie);
    atomicAdd(&sh.cta_gt_lo, gt_lo);
    atomicAdd(&sh.cta_tie_lo, tie_lo);
  }
  if (C > 1) cluster_sync(); else __syncthreads();
  uint32_t gt_before = 0, tie_before = 0, lo_gt = 0, lo_tie = 0;
  if (C == 1) {
    lo_gt = sh.cta_gt_lo;
    lo_tie = sh.cta_tie_lo;
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (x >= C) break;
      const uint32_t g1 = cluster_load(&sh.cta_gt, x), t1 = cluster_load(&sh.cta_tie, x);
      gt_before += x < rank ? g1 : 0u;
      tie_before += x < rank ? t1 : 0u;
      lo_gt += cluster_load(&sh.cta_gt_lo, x);
      lo_tie += cluster_load(&sh.cta_tie_lo, x);
    }
  }
  for (int x = 0; x < warp; ++x) {
    gt_before += sh.warp_gt[x];
    tie_before += sh.warp_tie[x];
  }
  const uint32_t kept_lo = lo_gt + min(lo_tie, want);  // kept slots below k
  const int moves = k - static_cast<int>(kept_lo);
  int* holes = a.holes + static_cast<size_t>(item) * a.list;
  int* movers = a.movers + static_cast<size_t>(item) * a.list;
  each([&](int i, int j) {
    const uint32_t x = j < w1 ? key_at(i, j) : 0u;
    const bool g1 = j < w1 && x > prefix, t1 = j < w1 && x == prefix;
    const uint32_t gm = __ballot_sync(0xffffffffu, g1), tm = __ballot_sync(0xffffffffu, t1);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t tb = tie_before + __popc(tm & below);
    const uint32_t kept = gt_before + __popc(gm & below) + min(tb, want);  // kept slots before j
    const bool keep = g1 || (t1 && tb < want);
    if (j < w1) {
      if (j < k && !keep) holes[j - kept] = j;
      if (j >= k && keep) movers[kept - kept_lo] = j;
    }
    gt_before += __popc(gm);
    tie_before += __popc(tm);
  });
  if (rank == 0 && tid == 0) a.counts[item] = moves;
  // No CTA leaves while another may still read its counts, and the lists are
  // complete after this.
  if (C > 1) cluster_sync(); else __syncthreads();
  if (a.list <= kInlineMoves)
    for (int m0 = (rank * kEvictWarps + warp) * kMovesPerWarp; m0 < moves; m0 += C * kEvictWarps * kMovesPerWarp)
      move_rows<D>(a, item, movers, holes, m0, moves, lane);
}

// The moves of all items, kMoveThreads / 32 * 8 per CTA.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) fa2_cache_move_kernel(const EvictArgs a, int chunks) {
  const int item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int moves = a.counts[item];
  const int m0 = (chunk * (kMoveThreads / 32) + warp) * kMovesPerWarp;
  const size_t list = static_cast<size_t>(item) * a.list;
  if (m0 < moves) move_rows<D>(a, item, a.movers + list, a.holes + list, m0, moves, lane);
}

cudaError_t launch_cache_evict(const EvictArgs& a0, cudaStream_t stream) {
  EvictArgs a = a0;
  const long long items = static_cast<long long>(a.c.B) * a.c.Hkv;
  // CTAs per (sequence, key head): doubled from 1 to 8 while a CTA has more
  // slots than its registers take. More CTAs than that cost more in cluster
  // barriers than they save: 2 heads of 16384 slots 13.1 us with 4, 14.0 with 8; 128
  // of 8192 51.4 with 2, 60.9 with 4.
  constexpr int kReg = kEvictThreads * kEvictRegs;
  const auto share = [&](int C) {  // slots of a CTA
    const int run = (((a.c.L + C - 1) / C + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
    return static_cast<long long>(run) * kEvictWarps;
  };
  int C = 1;
  while (C < 8 && share(C) > kReg) C *= 2;
  const bool reg = share(C) <= kReg;
  a.cached = !reg && share(C) <= kEvictKeys;
  const size_t smem = a.cached ? static_cast<size_t>(share(C)) * 4 : 0;
  auto kern = a.d == 64 ? (reg ? fa2_cache_evict_kernel<64, true> : fa2_cache_evict_kernel<64, false>)
                        : (reg ? fa2_cache_evict_kernel<128, true> : fa2_cache_evict_kernel<128, false>);
  cudaError_t e = cudaSuccess;
  if (!reg) {
    static std::atomic<unsigned long long> done[2];
    e = allow_smem(kern, kEvictKeys * 4, done[a.d == 64]);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * C));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, C);
  if (e != cudaSuccess || a.list <= kInlineMoves) return e;
  static_assert(kMoveThreads / 32 * kMovesPerWarp == kMovesPerCta, "move_ctas counts these");
  const int chunks = static_cast<int>(move_ctas(1, a.list));
  return launch_dependent(a.d == 64 ? fa2_cache_move_kernel<64> : fa2_cache_move_kernel<128>,
                          dim3(static_cast<unsigned>(items * chunks)), dim3(kMoveThreads), 0, stream, a, chunks);
}

}  // namespace fa2
