// Accumulated attention weight of a prompt's keys.
//
//   w[j] = sum over the query heads of key head h and the queries i that see
//   key j (i >= j when causal, i < q_lens[b]) of P_ij = e^(scale q_i . k_j - L_i)
//
// with L the forward's logsumexp: the column sums of the attention matrix,
// which the forward cannot form itself, L being known only after its last tile.
//
// What bounds it: one product, S = Q K^T, 2 d flop per (query, key), and one
// exponential for it. A unit of 128 queries x 256 keys takes 1024 clocks of
// tensor core at d = 128 (512 at d = 64) and 1220 of the exponentials: a loop of
// the same arithmetic alone reaches 26.8 per clock and SM. The kernel takes
// about 1800: with the products taken out 1710, with the arithmetic taken out
// 1780, so neither alone holds it up. Each warp also waits for its product, for
// TMEM (slow to answer while the tensor core accumulates there) and at each 16
// columns for the tail of its own arithmetic, and four warps per scheduler hide
// two thirds of that.
//
// Layout: TMEM lane = query, column = key, and a thread keeps the running sums
// of its 64 columns in registers over all query tiles of an item. So L is one
// scalar per thread and tile, nothing is read from shared memory between the
// product and the sums (its bandwidth belongs to the product's operands), and
// the sum over lanes happens once per item. The transposed form (lane = key)
// needs no such sum but a broadcast read of L per column: 290 us against 236 at
// B = 2, H = 16, N = 8192, d = 128, causal.
//
// A work item is 256 keys, tiles A and B, so that a Q tile fetched from L2
// feeds two products; two groups of four compute warps own 64 columns of each.
// All of TMEM is two S buffers per tile. Not kept: two groups of 128 columns
// (254 us, two warps per scheduler); one product 256 wide with one barrier for
// both tiles (231 us there, but 56 against 51 on B = 8, 16/4 heads, N = 2048,
// where more tiles are masked); a part of the exponentials as a polynomial on the
// FMA pipes (248 with one pair of eight, 265 with two); four units in a row
// without a break at d = 128 (279: spills).
//
// Split: the (item, query head, query tile) units of all items, in that order,
// are cut into one run per SM of equal length. An item inside one run is
// stored; one that is cut leaves its 256 sums in the workspace, two per CTA at
// most, and a second launch adds its parts in their order, so the result does
// not depend on timing.
#include "fa2_bwd_parts.cuh"
#include "fa2_cache.cuh"

namespace fa2 {

constexpr int kKwKeys = 256;  // keys per item
constexpr int kKwThreads = 640;  // 4 control warps, 4 groups of 4 compute warps
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));


// Query tiles [i0, nq) of item kb; none: no query sees its keys.
struct KwShape {
  int causal, nkb, g;
  // Units of one (sequence, key head) with nq query tiles, and of its first m items.
  __host__ __device__ long long before(int m, int nq) const {
    if (!causal) return static_cast<long long>(m) * nq * g;
    const long long mm = m < (nq + 1) / 2 ? m : (nq + 1) / 2;
    return (mm * nq - mm * (mm - 1)) * g;
  }
  __device__ int i0(int kb) const { return causal ? 2 * kb : 0; }
};

__device__ __forceinline__ int kw_qlen(const KeyWeightArgs& a, int b) {
  if (a.q_lens == nullptr) return a.N;
  return min(max(__ldg(a.q_lens + b), 0), a.N);
}
__device__ __forceinline__ int kw_tiles(int n) { return (n + kTileRows - 1) / kTileRows; }

__device__ __forceinline__ long long kw_total(const KeyWeightArgs& a, const KwShape& s, int lane) {
  long long t = 0;
  if (a.q_lens == nullptr) return s.before(s.nkb, kw_tiles(a.N)) * a.Hkv * a.B;
  for (int b = lane; b < a.B; b += 32) t += s.before(s.nkb, kw_tiles(kw_qlen(a, b))) * a.Hkv;
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}
// Units of the sequences before b, by a whole warp.
__device__ __forceinline__ long long kw_before(const KeyWeightArgs& a, const KwShape& s, int b, int lane) {
  if (a.q_lens == nullptr) return s.before(s.nkb, kw_tiles(a.N)) * a.Hkv * b;
  long long t = 0;
  for (int x = lane; x < b; x += 32) t += s.before(s.nkb, kw_tiles(kw_qlen(a, x))) * a.Hkv;
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

struct KwCursor {
  int b, h, kb, gh, i;  // sequence, key head, item, query head of the group, query tile
  int qlen, nq;
  long long to_end;     // units left in the item, this one included
};

// Cursor of unit u < T, by a whole warp.
__device__ __forceinline__ KwCursor kw_cursor(const KeyWeightArgs& a, const KwShape& s, long long u, int lane) {
  KwCursor k{};
  long long r = u, per = 0;
  if (a.q_lens == nullptr) {
    k.qlen = a.N;
    k.nq = kw_tiles(k.qlen);
    per = s.before(s.nkb, k.nq);
    k.b = static_cast<int>(r / (per * a.Hkv));
    r -= per * a.Hkv * k.b;
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int ql = b < a.B ? kw_qlen(a, b) : 0;
      const long long mine = s.before(s.nkb, kw_tiles(ql)) * a.Hkv;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, u < base + incl);
      if (hit != 0u) {
        const int src = __ffs(hit) - 1;
        r = u - (base + __shfl_sync(0xffffffffu, incl - mine, src));
        k.b = b0 + src;
        k.qlen = __shfl_sync(0xffffffffu, ql, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    k.nq = kw_tiles(k.qlen);
    per = s.before(s.nkb, k.nq);
  }
  k.h = static_cast<int>(r / per);
  r -= per * k.h;
  int lo = 0, hi = s.nkb - 1;  // last item that begins at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (s.before(mid, k.nq) <= r) lo = mid; else hi = mid - 1;
  }
  k.kb = lo;
  r -= s.before(lo, k.nq);
  const int w = k.nq - s.i0(lo);
  k.gh = static_cast<int>(r / w);
  k.i = s.i0(lo) + static_cast<int>(r - static_cast<long long>(k.gh) * w);
  k.to_end = static_cast<long long>(w) * s.g - r;
  return k;
}

// Next unit; true when it begins an item.
__device__ __forceinline__ bool kw_advance(const KeyWeightArgs& a, const KwShape& s, KwCursor& k) {
  --k.to_end;
  if (++k.i < k.nq) return false;
  k.i = s.i0(k.kb);
  if (++k.gh < s.g) return false;
  k.gh = 0;
  ++k.kb;
  if (k.kb >= s.nkb || s.i0(k.kb) >= k.nq) {
    k.kb = 0;
    if (++k.h >= a.Hkv) {
      k.h = 0;
      do {
        if (++k.b >= a.B) {
          k.nq = 0;
          return true;
        }
        k.qlen = kw_qlen(a, k.b);
      } while (k.qlen == 0);
      k.nq = kw_tiles(k.qlen);
    }
  }
  k.i = s.i0(k.kb);
  k.to_end = static_cast<long long>(k.nq - k.i) * s.g;
  return true;
}

// Whether tile t (128 keys) of the unit has a visible key: B of the first
// diagonal tile has none, nor has one past the keys.
__device__ __forceinline__ bool kw_active(const KeyWeightArgs& a, const KwShape& s, const KwCursor& k, int t) {
  const int kt = 2 * k.kb + t;
  return kt * kTileRows < a.Nk && (!s.causal || k.i >= kt);
}

// Shared memory: two K buffers of 256 rows (the next item's keys arrive while
// this one's are in use) and a ring of Q tiles.
template <int D>
struct KwCfg {
  static constexpr int TILE = kTileRows * D * 2;
  static constexpr int NQ = D == 128 ? 2 : 8;  // Q tiles in flight: 64 KiB, 128 KiB
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = 4 * TILE;
  static constexpr int SMEM = OFF_Q + NQ * TILE + 1024;
};

// What the compute warps need to know of a unit, written by a warp of its own:
// it keeps the unit arithmetic out of registers that hold sums. One slot per S
// buffer.
struct KwInfo {
  float2 row[kTileRows];  // (nl, f) of each query, see kw_chunk
  float* dst;             // where the 256 sums go when the unit ends a run of its item
  int keys;               // how many of them there are
  int flags;              // 1, 2: tile A, B active; 4, 8: masked; 16: ends the run
  int d0;                 // first query minus first key (not causal: past every key)
  int rows;               // queries of the tile below the sequence's end
};

template <int D>
struct KwShared {
  uint64_t k_full[2], k_free[2];
  uint64_t q_full[KwCfg<D>::NQ], q_free[KwCfg<D>::NQ];
  uint64_t s_full[2][2], s_free[2][2];  // [tile][buffer]
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  uint64_t sum_full[4], sum_free[4];  // per group
  float2 sums[4][3][32];  // per group: the sums of 64 keys of its warps 1 .. 3
  KwInfo info[2];
};

// 16 columns (keys) of one query row: acc += e^(score - L), as
// 2^(s c + nl) f with nl an integer and f in 2^-0.5 .. 2^0.5. With MASK only
// keys below lim count.
template <bool MASK>
__device__ __forceinline__ void kw_chunk(const uint32_t (&v)[16], float2* acc, float c, float nl, float f,
                                         int lim) {
  const float2 c2 = make_float2(c, c), n2 = make_float2(nl, nl), f2 = make_float2(f, f);
#pragma unroll
  for (int x = 0; x < 16; x += 2) {
    const float2 e = f2_fma(make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), c2, n2);
    float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
    if constexpr (MASK) {
      p.x = x < lim ? p.x : 0.f;
      p.y = x + 1 < lim ? p.y : 0.f;
    }
    acc[x / 2] = f2_fma(p, f2, acc[x / 2]);
  }
}

// The compute warps: group cg has columns 64 cg .. 64 cg + 63 (half of tile
// cg / 2), a thread one query row (TMEM lane), with the sums of its 64 keys in
// registers.
template <int D>
__device__ __forceinline__ void kw_compute(KwShared<D>& sh, uint32_t tmem, float c, long long units, int warp,
                                           int lane, const WaitCtx& wc) {
  const int cg = (warp - 4) >> 2, t = cg >> 1, quad = warp & 3, r = quad * 32 + lane;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 2 * t * kTileRows + (cg & 1) * 64;
  float2 acc[32];
#pragma unroll
  for (int x = 0; x < 32; ++x) acc[x] = make_float2(0.f, 0.f);
  auto release = [&](int buf) {  // the buffer and its unit's facts have been read
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.s_free[t][buf]);
  };
  int n = 0, flushes = 0;
  while (units > 0) {
    const int buf = n & 1;
    const uint32_t ts = t_lane + buf * kTileRows;
    if (!mbar_wait_warp(&sh.s_full[t][buf], (n >> 1) & 1, wc)) return;
    tc_fence_after();
    int flags = sh.info[buf].flags;
    float* dst = sh.info[buf].dst;
    int keys = sh.info[buf].keys;
    const float2 row = sh.info[buf].row[r];
    const int plain = 1 << t, kind = 5 << t;  // active, not masked
    if ((flags & kind) == plain) {
      uint32_t va[16], vb[16];
      tmem_ld_32x32b_x16(ts, va);
      tmem_wait_ld();
      reg_fence(va);
      tmem_ld_32x32b_x16(ts + 16, vb);
      kw_chunk<false>(va, acc, c, row.x, row.y, 0);
      tmem_wait_ld();
      reg_fence(vb);
      tmem_ld_32x32b_x16(ts + 32, va);
      kw_chunk<false>(vb, acc + 8, c, row.x, row.y, 0);
      tmem_wait_ld();
      reg_fence(va);
      tmem_ld_32x32b_x16(ts + 48, vb);
      kw_chunk<false>(va, acc + 16, c, row.x, row.y, 0);
      tmem_wait_ld();
      reg_fence(vb);
      release(buf);
      ++n;
      --units;
      if (D == 64 && !(flags & 16)) {
        // The same item goes on: its next unit's first columns are asked for
        // before this one's last are worked on, so that every other wait for a
        // product and for TMEM is hidden. (Always doing so carries loads across
        // the loop's back edge, which costs spills: twice the time.) Worth it
        // where the products are short: 214 against 227 us at d = 64, 239
        // against 237 at d = 128 (B = 2, H = 16, N = 8192, causal).
        if (!mbar_wait_warp(&sh.s_full[t][buf ^ 1], (n >> 1) & 1, wc)) return;
        tc_fence_after();
        const int f1 = sh.info[buf ^ 1].flags;
        if ((f1 & kind) == plain) {
          const float2 row1 = sh.info[buf ^ 1].row[r];
          const uint32_t t1 = t_lane + (buf ^ 1) * kTileRows;
          tmem_ld_32x32b_x16(t1, va);
          kw_chunk<false>(vb, acc + 24, c, row.x, row.y, 0);
          tmem_wait_ld();
          reg_fence(va);
          tmem_ld_32x32b_x16(t1 + 16, vb);
          kw_chunk<false>(va, acc, c, row1.x, row1.y, 0);
          tmem_wait_ld();
          reg_fence(vb);
          tmem_ld_32x32b_x16(t1 + 32, va);
          kw_chunk<false>(vb, acc + 8, c, row1.x, row1.y, 0);
          tmem_wait_ld();
          reg_fence(va);
          tmem_ld_32x32b_x16(t1 + 48, vb);
          kw_chunk<false>(va, acc + 16, c, row1.x, row1.y, 0);
          tmem_wait_ld();
          reg_fence(vb);
          flags = f1;
          dst = sh.info[buf ^ 1].dst;
          keys = sh.info[buf ^ 1].keys;
          release(buf ^ 1);
          kw_chunk<false>(vb, acc + 24, c, row1.x, row1.y, 0);
          ++n;
          --units;
        } else {
          kw_chunk<false>(vb, acc + 24, c, row.x, row.y, 0);
        }
      } else {
        kw_chunk<false>(vb, acc + 24, c, row.x, row.y, 0);
      }
    } else {
      if (flags & plain) {
        // Visible keys of this row, from the group's first one.
        const int lim = r < sh.info[buf].rows ? sh.info[buf].d0 + r - cg * 64 + 1 : 0;
#pragma unroll
        for (int x = 0; x < 64; x += 16) {
          if (__all_sync(0xffffffffu, lim <= x)) break;  // the warp's rows see none of the rest
          uint32_t va[16];
          tmem_ld_32x32b_x16(ts + x, va);
          tmem_wait_ld();
          reg_fence(va);
          kw_chunk<true>(va, acc + x / 2, c, row.x, row.y, lim - x);
        }
      }
      release(buf);
      ++n;
      --units;
    }
    if (flags & 16) {
      // Sums over the warp's 32 rows by halving: lane l ends with keys 2 l and
      // 2 l + 1; the group's first warp adds the four warps' in order.
#pragma unroll
      for (int o = 16, m = 16; o > 0; o >>= 1, m >>= 1) {
#pragma unroll
        for (int x = 0; x < m; ++x) {
          const bool up = lane & o;
          const float2 keep = up ? acc[x + m] : acc[x], give = up ? acc[x] : acc[x + m];
          acc[x] = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, give.x, o),
                               keep.y + __shfl_xor_sync(0xffffffffu, give.y, o));
        }
      }
      if (quad > 0) {
        if (flushes > 0 && !mbar_wait_warp(&sh.sum_free[cg], (flushes - 1) & 1, wc)) return;
        sh.sums[cg][quad - 1][lane] = acc[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_full[cg]);
      } else {
        if (!mbar_wait_warp(&sh.sum_full[cg], flushes & 1, wc)) return;
        float2 sum = acc[0];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const float2 y = sh.sums[cg][x][lane];
          sum = make_float2(sum.x + y.x, sum.y + y.y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_free[cg]);
        const int key = cg * 64 + 2 * lane;
        if (key < keys) dst[key] = sum.x;
        if (key + 1 < keys) dst[key + 1] = sum.y;
      }
      ++flushes;
#pragma unroll
      for (int x = 0; x < 32; ++x) acc[x] = make_float2(0.f, 0.f);
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kKwThreads, 1)
    fa2_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const KeyWeightArgs a, const KwShape s) {
  using C = KwCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ KwShared<D> sh;
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Barriers are set up by one lane of three warps, TMEM by a fourth, while the
  // others already look for their first unit.
  if (lane == 0) {
    if (warp == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      for (int i = 0; i < C::NQ; ++i) {
        mbar_init(&sh.q_full[i], 1);
        mbar_init(&sh.q_free[i], 1);
      }
      sh.abort_flag = 0;
      fence_mbar_init();
    } else if (warp == 2) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.k_full[i], 1);
        mbar_init(&sh.k_free[i], 1);
        for (int t = 0; t < 2; ++t) {
          mbar_init(&sh.s_full[t][i], 2);  // the product and the unit's facts
          mbar_init(&sh.s_free[t][i], 8);  // one arrival per compute warp of the tile
        }
      }
      mbar_init(&sh.mma_done, 1);
      fence_mbar_init();
    } else if (warp == 3) {
      for (int i = 0; i < 4; ++i) {
        mbar_init(&sh.sum_full[i], 3);
        mbar_init(&sh.sum_free[i], 1);
      }
      fence_mbar_init();
    }
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  const long long T = kw_total(a, s, lane);
  const long long G = T < gridDim.x ? T : gridDim.x;
  const int cta = blockIdx.x;
  const long long u0 = cta < G ? cta * T / G : 0, u1 = cta < G ? (cta + 1) * T / G : 0;
  KwCursor cu{};
  if (u0 < u1 && warp < 4) cu = kw_cursor(a, s, u0, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const WaitCtx wc{a.status, &sh.abort_flag, a.timeout_ns};

  if (warp < 4) {
    // 4 x 32 x 64 + 16 x 32 x 104 = 61,440 = the launch's 640 x 96 registers.
    setmaxnreg_dec<64>();
    if (warp == 0 && lane == 0 && u0 < u1) {
      // Producer: the Q tiles of the units, K of each item before its first.
      int items = 0, qs = 0, qph = 0, used = 0;
      bool ok = true, fresh = true;
      for (long long u = u0; u < u1 && ok; ++u) {
        if (fresh) {
          const int kb = items & 1;
          if (items > 1) ok = mbar_wait(&sh.k_free[kb], ((items >> 1) - 1) & 1, wc);
          if (!ok) break;
          mbar_arrive_expect_tx(&sh.k_full[kb], 2 * C::TILE);
#pragma unroll
          for (int t = 0; t < 2; ++t)
            load_tile<D>(smem + C::OFF_K + (2 * kb + t) * C::TILE, &tm_k, &sh.k_full[kb],
                         cu.kb * kKwKeys + t * kTileRows, cu.b * a.Hkv + cu.h);
          ++items;
        }
        if (used >= C::NQ) ok = mbar_wait(&sh.q_free[qs], qph ^ 1, wc);
        if (!ok) break;
        if (a.fault == 0 || u > u0) {
          mbar_arrive_expect_tx(&sh.q_full[qs], C::TILE);
          load_tile<D>(smem + C::OFF_Q + qs * C::TILE, &tm_q, &sh.q_full[qs], cu.i * kTileRows,
                       cu.b * a.Hq + cu.h * a.g + cu.gh);
        }
        ++used;
        if (++qs == C::NQ) {
          qs = 0;
          qph ^= 1;
        }
        fresh = kw_advance(a, s, cu);
      }
      if (!ok) {  // copies in flight land before the CTA ends
        for (int x = 0; x < 2; ++x) {
          const int uses = (items + 1 - x) / 2;
          if (uses > 0) mbar_wait_drain(&sh.k_full[x], (uses - 1) & 1, a.timeout_ns);
        }
        for (int x = 0; x < C::NQ; ++x) {
          const int uses = used / C::NQ + (x < used % C::NQ ? 1 : 0);
          if (uses > 0) mbar_wait_drain(&sh.q_full[x], (uses - 1) & 1, a.timeout_ns);
        }
      }
    } else if (warp == 1 && u0 < u1) {
      // Issuer: S of unit n into buffer n % 2.
      int items = 0, qs = 0, qph = 0, n = 0;
      bool ok = true, fresh = true;
      const uint32_t k_base = smem_u32(smem + C::OFF_K), q_base = smem_u32(smem + C::OFF_Q);
      for (long long u = u0; u < u1; ++u, ++n) {
        if (fresh) {
          ok = mbar_wait_warp(&sh.k_full[items & 1], (items >> 1) & 1, wc);
          if (!ok) break;
          ++items;
        }
        const int buf = n & 1, kb = (items - 1) & 1;
        ok = mbar_wait_warp(&sh.q_full[qs], qph, wc);
        const bool act_b = kw_active(a, s, cu, 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && n > 1) ok = mbar_wait_warp(&sh.s_free[t][buf], ((n >> 1) - 1) & 1, wc);
          if (!ok) break;
          if (t == 0 || act_b) {
            tc_fence_after();
            mma_rows_x_rows<D, BF16>(tmem + (2 * t + buf) * kTileRows, q_base + qs * C::TILE,
                                     k_base + (2 * kb + t) * C::TILE);
            umma_commit_warp(&sh.s_full[t][buf]);
          } else if (lane == 0) {
            mbar_arrive(&sh.s_full[t][buf]);
          }
        }
        if (!ok) break;
        umma_commit_warp(&sh.q_free[qs]);
        if (++qs == C::NQ) {
          qs = 0;
          qph ^= 1;
        }
        fresh = kw_advance(a, s, cu);
        if (fresh) umma_commit_warp(&sh.k_free[kb]);
      }
      umma_commit_warp(&sh.mma_done);
      mbar_wait_drain(&sh.mma_done, 0, a.timeout_ns);
    } else if (warp == 2 && u0 < u1) {
      int n = 0;
      bool from_start = cu.to_end == static_cast<long long>(cu.nq - s.i0(cu.kb)) * s.g;
      for (long long u = u0; u < u1; ++u, ++n) {
        const float* lse = a.lse + (static_cast<size_t>(cu.b) * a.Hq + static_cast<size_t>(cu.h) * a.g + cu.gh) * a.N;
        const int q0 = cu.i * kTileRows;
        float2 row[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int q = q0 + x * 32 + lane;
          const float l = q < cu.qlen ? __ldg(lse + q) : 0.f;
          // 2^(s c - L log2 e) with the integer part of L log2 e in the exponent
          // and the rest as a factor: neither is rounded against the large
          // exponents of s and L.
          const float hi = l * kLog2e;
          const float lo = fmaf(l, kLog2e, -hi) + l * kLog2eRest;
          const float whole = rintf(hi);
          // L = +inf: no weight (2^-inf), as in e^(s - L).
          row[x] = make_float2(-whole, isinf(hi) ? 1.f : ex2_approx(-((hi - whole) + lo)));
        }
        const int buf = n & 1, par = ((n >> 1) - 1) & 1;
        if (n > 1 && !mbar_wait2_warp(&sh.s_free[0][buf], par, &sh.s_free[1][buf], par, wc)) break;
        KwInfo& w = sh.info[buf];
#pragma unroll
        for (int x = 0; x < 4; ++x) w.row[x * 32 + lane] = row[x];
        if (lane == 0) {
          const bool item_end = cu.to_end == 1, flush = item_end || u + 1 == u1;
          const bool tail = q0 + kTileRows > cu.qlen;
          w.flags = 1 | (kw_active(a, s, cu, 1) ? 2 : 0) | (tail || (s.causal && cu.i == 2 * cu.kb) ? 4 : 0) |
                    (tail || (s.causal && cu.i == 2 * cu.kb + 1) ? 8 : 0) | (flush ? 16 : 0);
          w.d0 = s.causal ? q0 - cu.kb * kKwKeys : 2 * kKwKeys;
          w.rows = cu.qlen - q0;
          if (from_start && item_end) {
            w.dst = a.out + (static_cast<size_t>(cu.b) * a.Hkv + cu.h) * a.Nk + cu.kb * kKwKeys;
            w.keys = a.Nk - cu.kb * kKwKeys;
          } else {
            w.dst = a.part + (static_cast<size_t>(2) * cta + (from_start ? 1 : 0)) * kKwKeys;
            w.keys = kKwKeys;
          }
        }
        __syncwarp();
        if (lane < 2) mbar_arrive(&sh.s_full[lane][buf]);
        if (kw_advance(a, s, cu)) from_start = true;
      }
    }
  } else if (u0 < u1) {
    setmaxnreg_inc<104>();
    kw_compute<D>(sh, tmem, a.scale_log2, u1 - u0, warp, lane, wc);
  } else {
    setmaxnreg_inc<104>();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of cut items, in order, and writes the zeros of keys that no
// query sees. One CTA per item.
__global__ void __launch_bounds__(kKwKeys) fa2_key_weights_join_kernel(const KeyWeightArgs a, const KwShape s,
                                                                       int ctas) {
  const int lane = threadIdx.x & 31;
  const int kb = blockIdx.x % a.nkb, bh = blockIdx.x / a.nkb;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int nq = kw_tiles(kw_qlen(a, b));
  const long long T = kw_total(a, s, lane);
  const long long G = T < ctas ? T : ctas;
  const long long before = kw_before(a, s, b, lane);
  grid_dependency_wait();
  const int key = kb * kKwKeys + threadIdx.x;
  float* dst = a.out + static_cast<size_t>(bh) * a.Nk + key;
  const long long n = s.before(kb + 1, nq) - s.before(kb, nq);
  if (n == 0) {
    if (key < a.Nk) *dst = 0.f;
    return;
  }
  const long long ub = before + s.before(s.nkb, nq) * h + s.before(kb, nq);
  const int c0 = static_cast<int>(((ub + 1) * G - 1) / T), c1 = static_cast<int>(((ub + n) * G - 1) / T);
  if (c0 == c1) return;
  float w = 0.f;
  for (int x = c0; x <= c1; ++x)
    w += a.part[(static_cast<size_t>(2) * x + (x == c0 ? 1 : 0)) * kKwKeys + threadIdx.x];
  if (key < a.Nk) *dst = w;
}

template <int D, bool BF16>
static cudaError_t launch_key_weights_t(const CUtensorMap& tq, const CUtensorMap& tk, const KeyWeightArgs& a,
                                        const KwShape& s, int ctas, cudaStream_t stream) {
  auto kern = fa2_key_weights_kernel<D, BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, KwCfg<D>::SMEM, done);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kKwThreads, KwCfg<D>::SMEM, stream>>>(tq, tk, a, s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(fa2_key_weights_join_kernel, dim3(static_cast<unsigned>(a.B * a.Hkv) * a.nkb),
                          dim3(kKwKeys), 0, stream, a, s, ctas);
}

cudaError_t launch_key_weights(int d, bool bf16, bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                               const KeyWeightArgs& a, int ctas, cudaStream_t stream) {
  const KwShape s{causal ? 1 : 0, a.nkb, a.g};
  if (d == 64) return bf16 ? launch_key_weights_t<64, true>(tq, tk, a, s, ctas, stream)
                           : launch_key_weights_t<64, false>(tq, tk, a, s, ctas, stream);
  return bf16 ? launch_key_weights_t<128, true>(tq, tk, a, s, ctas, stream)
              : launch_key_weights_t<128, false>(tq, tk, a, s, ctas, stream);
}

}  // namespace fa2
