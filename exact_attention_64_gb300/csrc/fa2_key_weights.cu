// Accumulated attention weight of a prompt's keys.
//
//   w[j] = sum over the query heads of key head h and the queries i that see
//   key j (i >= j when causal, i < q_lens[b]) of P_ij = e^(scale q_i . k_j - L_i)
//
// with L the forward's logsumexp: the column sums of the attention matrix,
// which the forward cannot form itself, L being known only after its last tile.
//
// What bounds it: one product, S^T = K Q^T, 2 d flop per (key, query), and one
// exponential for it. A 128 x 128 tile takes 512 clocks of tensor core at
// d = 128 (256 at d = 64) and 512 clocks of the SM's 32 exponentials per clock.
//
// S^T and not S: TMEM lane = key, so a thread owns a key and its sum over the
// queries is a chain of additions in a register, without shuffles or atomics;
// what varies along the columns, L, is one broadcast shared-memory load for
// four columns. A work item is 256 keys (tiles A and B, a warpgroup each), so
// that a Q tile fetched from L2 feeds two products; each tile has two S^T
// buffers, all of TMEM, so the tensor core fills one while the warpgroup
// reads the other.
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

struct BoolTrue { static constexpr bool value = true; };
struct BoolFalse { static constexpr bool value = false; };

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

template <int D>
struct KwCfg {
  static constexpr int TILE = kTileRows * D * 2;
  static constexpr int NQ = D == 128 ? 4 : 8;  // Q tiles in flight: 128 KiB
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_L = OFF_Q + NQ * TILE;
  static constexpr int SMEM = OFF_L + NQ * kTileRows * 4 + 1024;
};

template <int D>
struct KwShared {
  uint64_t k_full, k_free;
  uint64_t q_full[KwCfg<D>::NQ], q_free[KwCfg<D>::NQ];
  uint64_t l_full[KwCfg<D>::NQ], l_free[KwCfg<D>::NQ];
  uint64_t s_full[2][2], s_free[2][2];  // [tile][buffer]
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(384, 1)
    fa2_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const KeyWeightArgs a, const KwShape s) {
  using C = KwCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ KwShared<D> sh;
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sh.k_full, 1);
    mbar_init(&sh.k_free, 1);
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_free[i], 1);
      mbar_init(&sh.l_full[i], 1);
      mbar_init(&sh.l_free[i], 8);
    }
    for (int t = 0; t < 2; ++t)
      for (int x = 0; x < 2; ++x) {
        mbar_init(&sh.s_full[t][x], 1);
        mbar_init(&sh.s_free[t][x], 4);
      }
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const WaitCtx wc{a.status, &sh.abort_flag, a.timeout_ns};
  const long long T = kw_total(a, s, lane);
  const long long G = T < gridDim.x ? T : gridDim.x;
  const int cta = blockIdx.x;
  const long long u0 = cta < G ? cta * T / G : 0, u1 = cta < G ? (cta + 1) * T / G : 0;
  KwCursor cu{};
  if (u0 < u1) cu = kw_cursor(a, s, u0, lane);
  float* lsm = reinterpret_cast<float*>(smem + C::OFF_L);

  if (warp == 0 && lane == 0 && u0 < u1) {
    // Producer: K of each item, then its Q tiles.
    int items = 0, qs = 0, qph = 0, last_k = -1;
    int used = 0;  // Q stages issued
    bool ok = true, fresh = true;
    for (long long u = u0; u < u1 && ok; ++u) {
      if (fresh) {
        if (items > 0) ok = mbar_wait(&sh.k_free, (items - 1) & 1, wc);
        if (!ok) break;
        const int bk = cu.b * a.Hkv + cu.h;
        mbar_arrive_expect_tx(&sh.k_full, 2 * C::TILE);
        load_tile<D>(smem + C::OFF_K, &tm_k, &sh.k_full, cu.kb * kKwKeys, bk);
        load_tile<D>(smem + C::OFF_K + C::TILE, &tm_k, &sh.k_full, cu.kb * kKwKeys + kTileRows, bk);
        last_k = items++;
      }
      if (used >= C::NQ) ok = mbar_wait(&sh.q_free[qs], qph ^ 1, wc);
      if (!ok) break;
      mbar_arrive_expect_tx(&sh.q_full[qs], C::TILE);
      load_tile<D>(smem + C::OFF_Q + qs * C::TILE, &tm_q, &sh.q_full[qs], cu.i * kTileRows,
                   cu.b * a.Hq + cu.h * a.g + cu.gh);
      ++used;
      if (++qs == C::NQ) {
        qs = 0;
        qph ^= 1;
      }
      fresh = kw_advance(a, s, cu);
    }
    if (!ok) {  // copies in flight land before the CTA ends
      if (last_k >= 0) mbar_wait_drain(&sh.k_full, last_k & 1, a.timeout_ns);
      for (int x = 0; x < C::NQ; ++x) {
        const int uses = used / C::NQ + (x < used % C::NQ ? 1 : 0);
        if (uses > 0) mbar_wait_drain(&sh.q_full[x], (uses - 1) & 1, a.timeout_ns);
      }
    }
  } else if (warp == 2 && u0 < u1) {
    // -L log2(e) of each query tile.
    int st = 0, ph = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok; ++u) {
      const float* src = a.lse + (static_cast<size_t>(cu.b) * a.Hq + static_cast<size_t>(cu.h) * a.g + cu.gh) * a.N;
      float v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int q = cu.i * kTileRows + x * 32 + lane;
        v[x] = q < cu.qlen ? -__ldg(src + q) * kLog2e : 0.f;
      }
      if (u - u0 >= C::NQ) ok = mbar_wait_warp(&sh.l_free[st], ph ^ 1, wc);
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < 4; ++x) lsm[st * kTileRows + x * 32 + lane] = v[x];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.l_full[st]);
      if (++st == C::NQ) {
        st = 0;
        ph ^= 1;
      }
      kw_advance(a, s, cu);
    }
  } else if (warp == 1 && u0 < u1) {
    // Issuer: S^T of tiles A and B into buffer (use of the tile) % 2.
    int items = 0, qs = 0, qph = 0, cnt[2] = {0, 0};
    bool ok = true, fresh = true;
    const uint32_t k_base = smem_u32(smem + C::OFF_K), q_base = smem_u32(smem + C::OFF_Q);
    for (long long u = u0; u < u1 && ok; ++u) {
      if (fresh) {
        ok = mbar_wait_warp(&sh.k_full, items & 1, wc);
        if (!ok) break;
        ++items;
      }
      ok = mbar_wait_warp(&sh.q_full[qs], qph, wc);
      if (!ok) break;
      const bool act0 = kw_active(a, s, cu, 0), act1 = kw_active(a, s, cu, 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!(t == 0 ? act0 : act1)) continue;
        const int buf = cnt[t] & 1, use = cnt[t] >> 1;
        if (use > 0) ok = ok && mbar_wait_warp(&sh.s_free[t][buf], (use - 1) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        mma_rows_x_rows<D, BF16>(tmem + (t * 2 + buf) * 128, k_base + t * C::TILE, q_base + qs * C::TILE);
        umma_commit_warp(&sh.s_full[t][buf]);
        ++cnt[t];
      }
      if (!ok) break;
      umma_commit_warp(&sh.q_free[qs]);
      if (++qs == C::NQ) {
        qs = 0;
        qph ^= 1;
      }
      fresh = kw_advance(a, s, cu);
      if (fresh) umma_commit_warp(&sh.k_free);
    }
    umma_commit_warp(&sh.mma_done);
    mbar_wait_drain(&sh.mma_done, 0, a.timeout_ns);
  } else if (warp >= 4 && u0 < u1) {
    const int t = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + t * 256;
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    int st = 0, ph = 0, cnt = 0;
    bool ok = true;
    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
    bool from_start = cu.to_end == static_cast<long long>(cu.nq - s.i0(cu.kb)) * s.g;
    for (long long u = u0; u < u1; ++u) {
      ok = mbar_wait_warp(&sh.l_full[st], ph, wc);
      if (!ok) break;
      const int key = cu.kb * kKwKeys + t * kTileRows + r;
      if (kw_active(a, s, cu, t)) {
        const int buf = cnt & 1;
        ok = mbar_wait_warp(&sh.s_full[t][buf], (cnt >> 1) & 1, wc);
        if (!ok) break;
        ++cnt;
        tc_fence_after();
        const float4* nl = reinterpret_cast<const float4*>(lsm + st * kTileRows);
        const int q0 = cu.i * kTileRows;
        const bool mask = (s.causal && cu.i == 2 * cu.kb + t) || q0 + kTileRows > cu.qlen;
        const uint32_t ts = t_lane + buf * 128;
#pragma unroll
        for (int cb = 0; cb < 128; cb += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(ts + cb, v);
          tmem_wait_ld();
          reg_fence(v);
          if (cb == 96) {  // the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_free[t][buf]);
          }
          auto body = [&](auto masked) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 n4 = nl[(cb + x) / 4];
              const float2 x0 = f2_fma(make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sl2,
                                       make_float2(n4.x, n4.y));
              const float2 x1 = f2_fma(make_float2(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), sl2,
                                       make_float2(n4.z, n4.w));
              float2 p0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
              float2 p1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
              if constexpr (decltype(masked)::value) {
                const int q = q0 + cb + x;
                auto seen = [&](int qq) { return qq < cu.qlen && (!s.causal || qq >= key); };
                p0.x = seen(q) ? p0.x : 0.f;
                p0.y = seen(q + 1) ? p0.y : 0.f;
                p1.x = seen(q + 2) ? p1.x : 0.f;
                p1.y = seen(q + 3) ? p1.y : 0.f;
              }
              acc0 = f2_add(acc0, p0);
              acc1 = f2_add(acc1, p1);
            }
          };
          if (mask) body(BoolTrue{}); else body(BoolFalse{});
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.l_free[st]);
      if (++st == C::NQ) {
        st = 0;
        ph ^= 1;
      }
      const bool item_end = cu.to_end == 1;
      if (item_end || u + 1 == u1) {
        const float w = (acc0.x + acc0.y) + (acc1.x + acc1.y);
        if (from_start && item_end) {
          if (key < a.Nk) a.out[(static_cast<size_t>(cu.b) * a.Hkv + cu.h) * a.Nk + key] = w;
        } else {
          a.part[(static_cast<size_t>(2) * cta + (from_start ? 1 : 0)) * kKwKeys + t * kTileRows + r] = w;
        }
        acc0 = acc1 = make_float2(0.f, 0.f);
      }
      if (kw_advance(a, s, cu)) from_start = true;
    }
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
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KwCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<ctas, 384, KwCfg<D>::SMEM, stream>>>(tq, tk, a, s);
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
