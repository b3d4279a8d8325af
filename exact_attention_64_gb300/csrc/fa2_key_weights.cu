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
// about 1630 at B = 2, H = 16, N = 8192, not causal: with the products taken out
// 1340, with the arithmetic taken out 1320. The rest is the wait for a product
// that cannot begin before its S has been read.
//
// Layout: S^T = K Q^T, TMEM lane = key, column = query, so that a thread's sums
// are one key's and need no other lane, and a key that the causal mask hides
// takes out whole columns of a warp. -L log2(e) is read from shared memory, four
// queries at a time. A product is 128 keys x 256 queries (two query tiles of one
// head, when there are two): per flop it reads three quarters of the shared
// memory of one that is 128 wide, which runs at shared memory's limit. TMEM
// holds one S for each of the item's two tiles, A and B; the eight warps of one
// tile work while the tensor core forms the other's. Each tile has an issuer of
// its own: at a diagonal B has less to do, and runs ahead (B = 8, 16/4 heads,
// N = 2048: 50 us against 56 with one issuer in fixed order; with a lock that
// keeps the two from issuing at once 85).
//
// At B = 2, H = 16, N = 8192, d = 128 it takes 211 to 223 us causal and 371 to 390
// not causal, by the clock that the power limit leaves; d = 64: 179 and 336.
// The other orientation, lane = query with a thread's 64 sums in registers, takes
// 236 and 431 there, and 51 at the N = 2048 above. Also not kept: eight compute warps with 64 columns in
// flight (272 us, two warps per scheduler), S in halves of 128 queries with a
// barrier each (296), one issuer that polls both tiles (239).
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
  return min(max(ld_global(a.q_lens + b), 0), a.N);
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
  long long at;         // the unit's place among all
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
  k.at = u;
  return k;
}

// Next unit; true when it begins an item.
__device__ __forceinline__ bool kw_advance(const KeyWeightArgs& a, const KwShape& s, KwCursor& k) {
  --k.to_end;
  ++k.at;
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

// A step: one unit, or two that follow each other in one query head, whose query
// tiles then form one product 256 wide.
__device__ __forceinline__ int kw_step(const KwCursor& k, long long left) {
  return left > 1 && k.i + 1 < k.nq ? 2 : 1;
}
// Advances past a step; true when the next unit begins an item.
__device__ __forceinline__ bool kw_advance_step(const KeyWeightArgs& a, const KwShape& s, KwCursor& k, int cnt) {
  bool fresh = kw_advance(a, s, k);
  if (cnt == 2) fresh = kw_advance(a, s, k);
  return fresh;
}
// Whether tile t (128 keys) has a visible key in a step.
__device__ __forceinline__ bool kw_active(const KeyWeightArgs& a, const KwShape& s, const KwCursor& k, int cnt, int t) {
  const int kt = 2 * k.kb + t;
  return kt * kTileRows < a.Nk && (!s.causal || k.i + cnt - 1 >= kt);
}

// Shared memory: the item's two K tiles, and a ring of Q steps.
template <int D>
struct KwCfg {
  static constexpr int TILE = kTileRows * D * 2;
  static constexpr int NQ = D == 128 ? 2 : 4;  // steps in flight: 128 KiB
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int SMEM = OFF_Q + NQ * 2 * TILE + 1024;
};

// What the compute warps need to know of a step, written ahead by a warp of its
// own.
constexpr int kKwInfos = 4;
struct KwInfo {
  float4 nl[2 * kTileRows / 4];  // -L log2(e) of each query
  float* dst;                    // where the 256 sums go when the step ends a run of its item
  int keys;                      // how many of them there are
  int flags;                     // 1, 2: tile A, B active; 4, 8: masked; 16: the sums go out; 32: two units;
                                 // 64: the last step
  int d0;                        // first query minus first key (not causal: past every key)
  int rows;                      // queries of the step below the sequence's end
};

template <int D>
struct KwShared {
  uint64_t k_full[2], k_free[2];  // per tile
  uint64_t q_full[KwCfg<D>::NQ], q_free[KwCfg<D>::NQ];
  uint64_t i_full[kKwInfos], i_free[kKwInfos];
  uint64_t s_full[2], s_free[2];  // per tile
  uint64_t sum_full[2], sum_free[2];
  uint64_t mma_done[2];
  uint32_t tmem_base;
  int abort_flag;
  float sum[2][kTileRows];
  alignas(16) KwInfo info[kKwInfos];
};

// S^T = K Q^T of one tile and step: M = 128 keys, N = 128 or 256 queries. The
// step's query rows lie in one slab of 256 rows per 64 columns.
template <int D, bool BF16, int N>
__device__ __forceinline__ void kw_issue(uint32_t d_tmem, uint32_t k_smem, uint32_t q_smem) {
  constexpr uint32_t idesc = make_idesc_f16(128, N, BF16, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t ad = make_sdesc_sw128(k_smem + (kk / 4) * (kTileRows * 128) + (kk % 4) * 32, 16, 1024);
    const uint64_t bd = make_sdesc_sw128(q_smem + (kk / 4) * (2 * kTileRows * 128) + (kk % 4) * 32, 16, 1024);
    umma_ss_warp(d_tmem, ad, bd, idesc, kk > 0 ? 1u : 0u);
  }
}

// 32 queries (columns) of one key: acc += 2^(s c - L log2 e). With MASK only
// columns whose bit is set count.
template <bool MASK>
__device__ __forceinline__ void kw_chunk(const uint32_t (&v)[32], const float4* nl, float2 (&acc)[2], float c,
                                         uint32_t bits = 0) {
  const float2 c2 = make_float2(c, c);
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    const float4 n = nl[x / 4];
    const float2 s0 = make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1]));
    const float2 s1 = make_float2(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
    const float2 e0 = f2_fma(s0, c2, make_float2(n.x, n.y));
    const float2 e1 = f2_fma(s1, c2, make_float2(n.z, n.w));
    float2 p0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
    float2 p1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
    if constexpr (MASK) {
      p0.x = bits & (1u << x) ? p0.x : 0.f;
      p0.y = bits & (1u << (x + 1)) ? p0.y : 0.f;
      p1.x = bits & (1u << (x + 2)) ? p1.x : 0.f;
      p1.y = bits & (1u << (x + 3)) ? p1.y : 0.f;
    }
    acc[0] = f2_add(acc[0], p0);
    acc[1] = f2_add(acc[1], p1);
  }
}

// The compute warps: group (t, j) = tile t, half j of its columns; a thread =
// one key (TMEM lane).
template <int D>
__device__ __forceinline__ void kw_compute(const KeyWeightArgs& a, KwShared<D>& sh, uint32_t tmem, int warp,
                                           int lane, const WaitCtx& wc) {
  const int t = ((warp - 4) >> 2) & 1, j = (warp - 4) >> 3, quad = warp & 3, r = quad * 32 + lane;
  const uint32_t ts = tmem + (static_cast<uint32_t>(quad * 32) << 16) + t * 2 * kTileRows + j * 32;
  const float c = a.scale_log2;
  float2 acc[2];
  acc[0] = acc[1] = make_float2(0.f, 0.f);
  int done = 0, sums = 0;  // S of this tile, and its sums, so far
  for (int n = 0, flags = 0; !(flags & 64); ++n) {
    const int st = n % kKwInfos;
    if (!mbar_wait_warp(&sh.i_full[st], (n / kKwInfos) & 1, wc)) return;
    const KwInfo& w = sh.info[st];
    flags = w.flags;
    if (flags & (1 << t)) {
      if (!mbar_wait_warp(&sh.s_full[t], done & 1, wc)) return;
      ++done;
      tc_fence_after();
      auto release = [&]() {  // S has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_free[t]);
      };
      uint32_t v[2][32];
      if ((flags & (32 | 4 << t)) == 32) {
        tmem_ld_32x32b_x32(ts, v[0]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          tmem_wait_ld();
          reg_fence(v[m & 1]);
          if (m < 3) tmem_ld_32x32b_x32(ts + (m + 1) * 64, v[(m + 1) & 1]);
          else release();
          kw_chunk<false>(v[m & 1], w.nl + (2 * m + j) * 8, acc, c);
        }
      } else {
        // Columns that this key's sum takes: queries from the key on (causal)
        // and below the sequence's end. A warp's diagonal lies in one chunk.
        const int first = t * kTileRows + quad * 32 - w.d0, hi = min(w.rows, flags & 32 ? 256 : 128);
        const int m0 = first <= 0 ? 0 : (first / 32 - j + 1) >> 1, m1 = ((hi + 31) / 32 - j + 1) >> 1;
        if (m0 >= m1) release();
#pragma unroll 1
        for (int m = m0; m < m1; ++m) {
          const int x = (2 * m + j) * 32;
          tmem_ld_32x32b_x32(ts + m * 64, v[0]);
          tmem_wait_ld();
          reg_fence(v[0]);
          if (m + 1 == m1) release();
          const uint32_t bits = (x > first ? ~0u : ~0u << lane) & (x + 32 <= hi ? ~0u : ~(~0u << (hi - x)));
          if (x > first && x + 32 <= hi) kw_chunk<false>(v[0], w.nl + x / 4, acc, c);
          else kw_chunk<true>(v[0], w.nl + x / 4, acc, c, bits);
        }
      }
    }
    if (flags & 16) {
      const int key = t * kTileRows + r;
      const float2 x = f2_add(acc[0], acc[1]);
      if (j == 1) {
        if (sums > 0 && !mbar_wait_warp(&sh.sum_free[t], (sums - 1) & 1, wc)) return;
        sh.sum[t][r] = x.x + x.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_full[t]);
      } else {
        if (!mbar_wait_warp(&sh.sum_full[t], sums & 1, wc)) return;
        if (key < w.keys) w.dst[key] = x.x + x.y + sh.sum[t][r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_free[t]);
      }
      ++sums;
      acc[0] = acc[1] = make_float2(0.f, 0.f);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.i_free[st]);
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Barriers are set up by one lane of three warps, TMEM by a fourth, while all
  // of the control warps look for their first unit.
  if (lane == 0) {
    if (warp == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&sh.k_full[t], 1);
        mbar_init(&sh.k_free[t], 1);
      }
      for (int i = 0; i < C::NQ; ++i) {
        mbar_init(&sh.q_full[i], 1);
        mbar_init(&sh.q_free[i], 2);
      }
      sh.abort_flag = 0;
      fence_mbar_init();
    } else if (warp == 2) {
      for (int i = 0; i < kKwInfos; ++i) {
        mbar_init(&sh.i_full[i], 1);
        mbar_init(&sh.i_free[i], 16);  // one arrival per compute warp
      }
      fence_mbar_init();
    } else if (warp == 3) {
      for (int t = 0; t < 2; ++t) {
        mbar_init(&sh.s_full[t], 1);
        mbar_init(&sh.mma_done[t], 1);
        mbar_init(&sh.s_free[t], 8);  // one arrival per compute warp of the tile
        mbar_init(&sh.sum_full[t], 4);
        mbar_init(&sh.sum_free[t], 4);
      }
      fence_mbar_init();
    }
  }
  __syncwarp();
  grid_dependency_wait();
  grid_launch_dependents();
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
    if (warp == 0 && lane == 0 && u0 < u1) {
      // Producer: the query tiles of the steps, K of each item before its first.
      int items = 0, qs = 0, qph = 0, used = 0, loads[2] = {0, 0};
      bool ok = true, fresh = true;
      while (cu.at < u1 && ok) {
        const int cnt = kw_step(cu, u1 - cu.at);
        if (used >= C::NQ) ok = mbar_wait(&sh.q_free[qs], qph ^ 1, wc);
        if (!ok) break;
        if (a.fault == 0 || used > 0) {
          mbar_arrive_expect_tx(&sh.q_full[qs], cnt * C::TILE);
          for (int j = 0; j < cnt; ++j)
#pragma unroll
            for (int sl = 0; sl < D / 64; ++sl)
              tma_load_3d(smem + C::OFF_Q + qs * 2 * C::TILE + (2 * sl + j) * (kTileRows * 128), &tm_q, &sh.q_full[qs],
                          sl * 64, (cu.i + j) * kTileRows, cu.b * a.Hq + cu.h * a.g + cu.gh);
        }
        ++used;
        if (++qs == C::NQ) {
          qs = 0;
          qph ^= 1;
        }
        if (fresh) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (items > 0 && ok) ok = mbar_wait(&sh.k_free[t], (items - 1) & 1, wc);
            if (!ok) continue;
            mbar_arrive_expect_tx(&sh.k_full[t], C::TILE);
            load_tile<D>(smem + C::OFF_K + t * C::TILE, &tm_k, &sh.k_full[t], cu.kb * kKwKeys + t * kTileRows,
                         cu.b * a.Hkv + cu.h);
            ++loads[t];
          }
          ++items;
        }
        fresh = kw_advance_step(a, s, cu, cnt);
      }
      // Copies in flight land before the CTA ends, whoever has given up. (If nobody
      // has, they are landing anyway.)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (loads[t] > 0) mbar_wait_drain(&sh.k_full[t], (loads[t] - 1) & 1, a.timeout_ns);
      for (int x = 0; x < C::NQ; ++x) {
        const int uses = used / C::NQ + (x < used % C::NQ ? 1 : 0);
        if (uses > 0) mbar_wait_drain(&sh.q_full[x], (uses - 1) & 1, a.timeout_ns);
      }
    } else if ((warp & 1) && u0 < u1) {
      // Issuers: S^T of tile A by warp 1, of tile B by warp 3. While the groups
      // of one tile work the tensor core forms the other's.
      const int t = warp >> 1;
      int items = 0, qs = 0, qph = 0, done = 0;
      bool fresh = true;
      const uint32_t k = smem_u32(smem + C::OFF_K) + t * C::TILE, acc = tmem + t * 2 * kTileRows;
      while (cu.at < u1) {
        const int cnt = kw_step(cu, u1 - cu.at);
        if (!mbar_wait_warp(&sh.q_full[qs], qph, wc)) break;
        if (fresh && !mbar_wait_warp(&sh.k_full[t], items++ & 1, wc)) break;
        const uint32_t q = smem_u32(smem + C::OFF_Q) + qs * 2 * C::TILE;
        if (kw_active(a, s, cu, cnt, t)) {
          if (done > 0 && !mbar_wait_warp(&sh.s_free[t], (done - 1) & 1, wc)) break;
          tc_fence_after();
          if (cnt == 1) kw_issue<D, BF16, 128>(acc, k, q);
          else if (!kw_active(a, s, cu, 1, t)) kw_issue<D, BF16, 128>(acc + kTileRows, k, q + kTileRows * 128);
          else kw_issue<D, BF16, 256>(acc, k, q);
          umma_commit_warp(&sh.s_full[t]);
          ++done;
        }
        umma_commit_warp(&sh.q_free[qs]);
        if (cu.to_end == cnt) umma_commit_warp(&sh.k_free[t]);
        if (++qs == C::NQ) {
          qs = 0;
          qph ^= 1;
        }
        fresh = kw_advance_step(a, s, cu, cnt);
      }
      umma_commit_warp(&sh.mma_done[t]);
      mbar_wait_drain(&sh.mma_done[t], 0, a.timeout_ns);
    } else if (warp == 2 && u0 < u1) {
      int n = 0;
      bool from_start = cu.to_end == static_cast<long long>(cu.nq - s.i0(cu.kb)) * s.g;
      for (; cu.at < u1; ++n) {
        const int cnt = kw_step(cu, u1 - cu.at);
        const float* lse = a.lse + (static_cast<size_t>(cu.b) * a.Hq + static_cast<size_t>(cu.h) * a.g + cu.gh) * a.N;
        const int q0 = cu.i * kTileRows;
        float4 nl[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float l[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int q = q0 + x * kTileRows + lane * 4 + y;
            l[y] = x < cnt && q < cu.qlen ? ld_global(lse + q) : 0.f;
          }
          nl[x] = make_float4(-l[0] * kLog2e, -l[1] * kLog2e, -l[2] * kLog2e, -l[3] * kLog2e);
        }
        const int st = n % kKwInfos;
        if (n >= kKwInfos && !mbar_wait_warp(&sh.i_free[st], (n / kKwInfos - 1) & 1, wc)) break;
        KwInfo& w = sh.info[st];
        w.nl[lane] = nl[0];
        w.nl[32 + lane] = nl[1];
        if (lane == 0) {
          const bool item_end = cu.to_end == cnt, last = cu.at + cnt == u1;
          const bool tail = q0 + cnt * kTileRows > cu.qlen;
          int flags = (item_end || last ? 16 : 0) | (cnt == 2 ? 32 : 0) | (last ? 64 : 0);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (kw_active(a, s, cu, cnt, t)) flags |= 1 << t;
            if (tail || (s.causal && cu.i <= 2 * cu.kb + t)) flags |= 4 << t;
          }
          w.flags = flags;
          w.d0 = s.causal ? q0 - cu.kb * kKwKeys : 2 * kKwKeys;  // a multiple of 32
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
        if (lane == 0) mbar_arrive(&sh.i_full[st]);
        if (kw_advance_step(a, s, cu, cnt)) from_start = true;
      }
    }
  } else {
    if (u0 < u1) kw_compute<D>(a, sh, tmem, warp, lane, wc);
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
  grid_launch_dependents();
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
  e = launch_dependent(kern, dim3(ctas), dim3(kKwThreads), KwCfg<D>::SMEM, stream, tq, tk, a, s);
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
