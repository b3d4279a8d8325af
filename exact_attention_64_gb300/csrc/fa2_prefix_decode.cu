// Attention of one new token per sequence over a paged cache, for sequences that
// begin with the same slots.
//
//   s_j = scale q . k_j, o = sum_j e^(s_j - L) v_j, L = ln sum_j e^(s_j)
//
// over the P shared slots and a sequence's own behind them. The sum splits: with (m, l,
// O) = (reference, sum of 2^(s - m), sum of 2^(s - m) v) of any set of slots, those of a
// union are l = sum 2^(m_i - m) l_i and so on. So the prefix is attended to once, by the
// queries of all sequences together; each sequence's own slots as in fa2_paged_decode;
// and a last launch joins the parts.
//
// What bounds it: for R = B g query rows of a key head the prefix costs 4 R flop per
// cached element of 2 bytes, so up to about 128 rows it is bound by HBM, and past that by
// the products and their exponentials. fa2_paged_decode would read the prefix B times.
//
// Prefix: the forward's shape with paged keys. Query rows are the TMEM lanes, 128 to a
// tile; an item is up to two tiles (256 rows) of one key head and all tiles of 128
// slots, and CTA c of G has the units [c T / G, (c + 1) T / G) of the T = items x slot
// tiles, so that every SM has the same share whatever the sizes. A segment (an item's
// part in a CTA) leaves (m, l, O) in the workspace.
//   warp 0       copies of K and of V: one TMA box of up to 16 slots x 64 columns per
//                lane and page piece, into 128-slot tiles with the 128-byte swizzle.
//   warp 1       the products: S = Q K^T, then O += P V with P read from TMEM.
//   warps 4-11   two groups of 128 threads, a thread per row, each with an S and an O in
//                TMEM: one per row tile, or, when the item has one tile only, both on it
//                with every other slot tile each, joined at the segment's end.
// P enters its product as two 16-bit numbers, rounded and remainder: bf16 to 2^-16 of p;
// fp16, which has no exponents for small p, with the largest at up to 2^15 and 2^-24 as
// the last place, 2^-36 of a row's reference or less. (64 sequences behind 8192 slots,
// Q ~ N(0, 2^2): 0.23 % of the bf16 outputs one step from the rounded exact value, 0.15 %
// of a plain fp32 form's; a first piece that is cut instead of rounded 0.39 %, no faster.)
// The third bf16 piece that would make P exact has no room in TMEM (S and O of two tiles
// fill it), and would be half a product more.
//
// Per CTA and slot tile of two row tiles about 4300 clocks at d = 128, of which the 48
// products are about 3070 at the tensor core's best. B = 256, 32/8 heads, 16384 slots and up to
// 200 own ones: 106 us, of which the prefix's kernel takes about 80.
#include "fa2_common.cuh"
#include "fa2_decode_units.cuh"

namespace fa2 {

// Shared memory and registers leave room for a CTA of the own slots' kernel beside each
// of these: its loads and the prefix's products run at the same time.
template <int D>
struct PfxCfg {
  static constexpr int SLAB = kTileRows * 128;  // 128 rows x 64 columns
  static constexpr int TILE = kTileRows * D * 2;
  static constexpr int NS = D == 128 ? 3 : 6;   // ring of K and V tiles in turn
  static constexpr int OFF_RING = 2 * TILE;     // after the two Q tiles
  // In a Q tile, once its products have completed: 4 KiB for each of its warps' rows on
  // their way out. With one row tile also both streams' references and the second's sums:
  // at d = 128 behind those in the second tile, which has no queries then; at d = 64 they
  // fill the tile.
  static constexpr int STAGE = 4096;
  static constexpr int ML_BYTES = 3 * kTileRows * 4;
  static constexpr int OFF_ML = D == 128 ? TILE + 4 * STAGE : OFF_RING + NS * TILE;
  static constexpr int SMEM = OFF_RING + NS * TILE + (D == 128 ? 0 : ML_BYTES) + 1024;
  static_assert(4 * STAGE <= TILE && (D != 128 || OFF_ML + ML_BYTES <= 2 * TILE), "inside the tiles");
  static constexpr int THREADS = 384;
  // Registers a thread at the launch, and of the control and the row warps from then on.
  // A split of more than the launch has would wait for ever: the launch checks what the
  // compiler gave.
  static constexpr int REGS = 104, REGS_CONTROL = 72, REGS_ROWS = 120;
  static_assert(4 * 32 * REGS_CONTROL + 8 * 32 * REGS_ROWS <= THREADS * REGS, "the split comes out of the launch's");
  static constexpr uint32_t TMEM_COLS = 512;
  // P overwrites S, 32 slots in 32 columns: 16 of the first pieces, 16 of the second.
  __host__ __device__ static constexpr uint32_t TM_S(int t) { return t * 128u; }
  __host__ __device__ static constexpr uint32_t TM_O(int t) { return 256u + t * D; }
};

template <int D>
struct PfxShared {
  uint64_t q_full, stored;
  uint64_t full[PfxCfg<D>::NS], empty[PfxCfg<D>::NS];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t ml_full;
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

// A CTA's units, from tile0 of an item on.
struct PfxWork {
  int P, tiles;    // slots in whole boxes, tiles of 128 of them
  int item, tile0;
  long long left;
};
// A segment: the units of one item.
struct PfxSeg {
  int h, row0, rows;  // key head, first query row, rows (up to 256)
  int tile0, cnt;     // slot tiles
  bool two;
};

// CTAs of T units: as few as finish at the same time, so that the own slots' kernel finds
// room beside them, and fewer parts are to be joined.
__device__ __forceinline__ long long pfx_ctas(const PrefixArgs& a, long long T) {
  if (T <= a.ctas) return T;
  const long long longest = div_pos(T + a.ctas - 1, a.ctas);
  return div_pos(T + longest - 1, longest);
}

__device__ __forceinline__ PfxWork pfx_work(const PrefixArgs& a, int cta, long long* ctas) {
  PfxWork w;
  w.P = prefix_slots(a.d).cut;
  w.tiles = (w.P + kTileRows - 1) / kTileRows;
  const long long T = static_cast<long long>(a.items) * w.tiles, G = pfx_ctas(a, T);
  *ctas = G;
  w.left = 0;
  w.item = w.tile0 = 0;
  if (cta < G) {
    const long long u0 = unit_begin(cta, G, T);
    w.left = unit_begin(cta + 1, G, T) - u0;
    w.item = static_cast<int>(div_pos(u0, w.tiles));
    w.tile0 = static_cast<int>(u0 - static_cast<long long>(w.item) * w.tiles);
  }
  return w;
}
__device__ __forceinline__ PfxSeg pfx_seg(const PrefixArgs& a, const PfxWork& w) {
  PfxSeg s;
  s.tile0 = w.tile0;
  s.cnt = static_cast<int>(min(static_cast<long long>(w.tiles - w.tile0), w.left));
  s.h = div_by(w.item, a.fblocks);
  s.row0 = (w.item - s.h * a.fblocks.d) * 2 * kTileRows;
  s.rows = min(2 * kTileRows, a.d.rows - s.row0);
  s.two = s.rows > kTileRows;
  return s;
}
__device__ __forceinline__ void pfx_next(PfxWork& w, int cnt) {
  w.left -= cnt;
  w.tile0 = 0;
  ++w.item;
}

// Cache row of box i of a slot tile, or -1: past the prefix, or a page that the cache
// does not have.
__device__ __forceinline__ int pfx_row(const PrefixArgs& a, int P, int h, int tile, int i) {
  const CacheView& c = a.d.c;
  const int slot = tile * kTileRows + i * a.d.box;
  if (slot >= P) return -1;
  const int p = div_by(slot, c.ps);
  return page_row(c, ld_global(a.d.prefix + p), h, slot - p * c.ps.d);
}

// ---- Copies: one warp ---------------------------------------------------------
// Tile number 2 g (K) and 2 g + 1 (V) of a CTA go through one ring. One warp fills all of
// it: it has then waited for every phase of a slot's barrier in turn, which a wait by
// parity needs. (Two warps, for K and for V, would each see every other phase only, and
// take a slot that has not been read for one that was read twice.)
template <int D>
__device__ bool pfx_producer(const PrefixArgs& a, PfxWork w, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             PfxShared<D>& sh, uint8_t* ring, int lane, const WaitCtx& wc) {
  using C = PfxCfg<D>;
  const int boxes = kTileRows / a.d.box, bytes = a.d.box * 128;
  const int nowhere = a.d.c.num_pages * a.d.c.Hkv * a.d.c.ps.d;  // past the cache: reads as zeros
  int x = 0;
  bool ok = true;
  while (w.left > 0 && ok) {
    const PfxSeg s = pfx_seg(a, w);
    for (int j = 0; j < s.cnt && ok; ++j) {
      const int tile = s.tile0 + j;
      int row = lane < boxes ? pfx_row(a, w.P, s.h, tile, lane) : -1;
      for (int kv = 0; kv < 2; ++kv, ++x) {
        const int st = x % C::NS;
        ok = mbar_wait_warp(&sh.empty[st], ((x / C::NS) & 1) ^ 1, wc);
        if (!ok) break;
        if (a.fault != 0 && x == 1) continue;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], C::TILE);
        __syncwarp();
        const CUtensorMap* map = kv ? &tm_v : &tm_k;
        for (int i = lane; i < boxes; i += 32) {
          const int rr = i < 32 ? row : pfx_row(a, w.P, s.h, tile, i);
          if (kv == 0 && rr < 0 && tile * kTileRows + i * a.d.box < w.P) report_page(a.d.c.status);
          const int at = rr < 0 ? nowhere : rr;
          uint8_t* dst = ring + st * C::TILE + i * bytes;
#pragma unroll
          for (int y = 0; y < D / 64; ++y) tma_load_3d(dst + y * C::SLAB, map, &sh.full[st], y * 64, at, 0);
        }
        __syncwarp();
      }
    }
    pfx_next(w, s.cnt);
  }
  // Whoever gave up, this warp's copies land before the CTA ends.
  if (lane == 0)
    for (int y = max(0, x - C::NS); y < x; ++y)
      if (!(a.fault != 0 && y == 1)) mbar_wait_drain(&sh.full[y % C::NS], (y / C::NS) & 1, a.timeout_ns);
  return ok;
}

// ---- Products -----------------------------------------------------------------
// Task i of a segment: row tile i & 1 with slot tile i / 2 (two row tiles), or the one
// row tile with slot tile i for stream i & 1. S(i) and S(i + 1) are in flight; S(i + 2)
// follows O += P(i) V, which reads the P that it overwrites. A task's 24 products take
// about 1850 clocks (B = 256, 32/8 heads, d = 128), the next one's begin 400 later. Not
// kept: a warp for each stream, whose products interleave (65 clocks each instead of 77
// to 90) but whose rows are then all at work at once, 6200 clocks a slot tile of both
// streams instead of 4600; O in two halves of d in turn, 4900.
template <int D, bool BF16>
__device__ bool pfx_issuer(const PrefixArgs& a, PfxWork w, PfxShared<D>& sh, uint8_t* smem, uint32_t tmem,
                           const WaitCtx& wc) {
  using C = PfxCfg<D>;
  constexpr uint32_t id_s = make_idesc_f16(kTileRows, kTileRows, BF16, false, false);
  constexpr uint32_t id_o = make_idesc_f16(kTileRows, D, BF16, false, true);
  const uint32_t q = smem_u32(smem), ring = q + C::OFF_RING;
  int g0 = 0, segs = 0, tasks[2] = {0, 0};
  bool ok = true;
  for (; w.left > 0 && ok; ++segs) {
    const PfxSeg s = pfx_seg(a, w);
    const int n = s.two ? 2 * s.cnt : s.cnt, sh2 = s.two ? 1 : 0;
    auto issue_s = [&](int i) {
      const int x = 2 * (g0 + (i >> sh2)), st = x % C::NS, t = i & 1;
      if (!s.two || t == 0) {
        if (!mbar_wait_warp(&sh.full[st], (x / C::NS) & 1, wc)) return false;
        tc_fence_after();
      }
      const uint32_t qt = q + (s.two ? t : 0) * C::TILE, kt = ring + st * C::TILE;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * C::SLAB + (kk % 4) * 32;
        umma_ss_warp(tmem + C::TM_S(t), make_sdesc_sw128(qt + off, 16, 1024), make_sdesc_sw128(kt + off, 16, 1024), id_s,
                     kk > 0 ? 1u : 0u);
      }
      umma_commit_warp(&sh.s_full[t]);
      if (!s.two || t == 1) umma_commit_warp(&sh.empty[st]);
      return true;
    };
    ok = mbar_wait_warp(&sh.q_full, segs & 1, wc);
    if (!ok) break;
    tc_fence_after();
    ok = issue_s(0) && (n < 2 || issue_s(1));
    for (int i = 0; i < n && ok; ++i) {
      const int x = 2 * (g0 + (i >> sh2)) + 1, st = x % C::NS, t = i & 1;
      ok = mbar_wait2_warp(&sh.full[st], (x / C::NS) & 1, &sh.p_full[t], tasks[t] & 1, wc);
      if (!ok) break;
      ++tasks[t];
      tc_fence_after();
      const uint32_t vt = ring + st * C::TILE;
#pragma unroll
      for (int piece = 0; piece < 2; ++piece)
#pragma unroll
        for (int kk = 0; kk < kTileRows / 16; ++kk)
          umma_ts_warp(tmem + C::TM_O(t), tmem + C::TM_S(t) + (kk / 2) * 32 + piece * 16 + (kk % 2) * 8,
                       make_sdesc_sw128(vt + kk * 2048, C::SLAB, 1024), id_o, (i >= 2 || piece > 0 || kk > 0) ? 1u : 0u);
      umma_commit_warp(&sh.o_full[t]);
      if (!s.two || t == 1) umma_commit_warp(&sh.empty[st]);
      if (i + 2 < n) ok = issue_s(i + 2);
    }
    g0 += s.cnt;
    pfx_next(w, s.cnt);
  }
  // Every product that was issued completes before TMEM is released.
  umma_commit_warp(&sh.mma_done);
  mbar_wait_drain(&sh.mma_done, 0, a.timeout_ns);
  return ok;
}

// ---- Rows -----------------------------------------------------------------------
template <bool BF16>
constexpr float kPfxBias = BF16 ? 0.f : 12.f;     // log2 of the largest p after a reference is set
template <bool BF16>
constexpr float kPfxRescale = BF16 ? 8.f : 3.f;   // how far a row's maximum may pass its reference (log2 units)

// Which columns of a slot tile count: a bit per box.
struct PfxMask {
  uint32_t w[4];
  bool all;
};
__device__ __forceinline__ PfxMask pfx_mask(const PrefixArgs& a, int P, int h, int tile, int lane) {
  const int boxes = kTileRows / a.d.box;
  PfxMask m;
  m.all = true;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    m.w[x] = 0u;
    if (32 * x >= boxes) break;
    const bool in = lane + 32 * x < boxes;
    m.w[x] = __ballot_sync(0xffffffffu, in && pfx_row(a, P, h, tile, lane + 32 * x) >= 0);
    m.all = m.all && m.w[x] == __ballot_sync(0xffffffffu, in);
  }
  return m;
}

// -inf into the columns of S that do not count.
__device__ __noinline__ void pfx_hide(uint32_t t_s, const PfxMask& mask, int box) {
  const int lb = __ffs(box) - 1;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t s[32];
    tmem_ld_32x32b_x32(t_s + 32 * x, s);
    tmem_wait_ld();
    reg_fence(s);
    // Column c's box is c / box; 32 columns' boxes are bits of one word.
    const uint32_t word = box >= 4 ? mask.w[0] : box == 2 ? mask.w[x / 2] : mask.w[x];
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((word >> (((32 * x + c) >> lb) & 31)) & 1u)) s[c] = __float_as_uint(-INFINITY);
    tmem_st_32x32b_x32(t_s + 32 * x, s);
  }
  tmem_wait_st();
}

// One slot tile of a thread's row: P from S, the row's sum, and O's rescale when the
// reference moves (only when the maximum passes it by kPfxRescale: exact, O and l share
// it).
template <int D, bool BF16>
__device__ __forceinline__ bool pfx_step(PfxShared<D>& sh, int t, uint32_t t_s, uint32_t t_o, const PfxMask& mask,
                                         int box, float sl2, bool first, int done, float& m_ref, float& l, int lane,
                                         const WaitCtx& wc) {
  if (!mbar_wait_warp(&sh.s_full[t], done & 1, wc)) return false;
  __syncwarp();
  tc_fence_after();
  if (!mask.all) pfx_hide(t_s, mask, box);
  // Short loops over 32 columns: S is read twice, which costs less than keeping it, and
  // the kernel's first steps wait for few instructions to arrive.
  float mx = -INFINITY;
#pragma unroll 1
  for (int x = 0; x < 4; ++x) {
    uint32_t s[32];
    tmem_ld_32x32b_x32(t_s + 32 * x, s);
    tmem_wait_ld();
    reg_fence(s);
    float m8[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) m8[c] = fmax3(__uint_as_float(s[c]), __uint_as_float(s[8 + c]), __uint_as_float(s[16 + c]));
#pragma unroll
    for (int c = 0; c < 8; c += 2) m8[c] = fmax3(m8[c], __uint_as_float(s[24 + c]), m8[c + 1]);
    mx = fmax3(mx, fmax3(m8[0], m8[2], m8[4]), m8[6]);
#pragma unroll
    for (int c = 1; c < 8; c += 2) mx = fmaxf(mx, __uint_as_float(s[24 + c]));
  }
  const float m_new = fmaxf(m_ref, mx);
  const bool rescale = (m_new - m_ref) * sl2 > kPfxRescale<BF16>;  // also from -inf
  float alpha = 1.f;
  if (rescale) {
    alpha = ex2_approx((m_ref - m_new) * sl2);
    m_ref = m_new;
  }
  const float neg = m_ref == -INFINITY ? 0.f : kPfxBias<BF16> - m_ref * sl2;
  float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 sl = make_float2(sl2, sl2), ng = make_float2(neg, neg);
#pragma unroll 1
  for (int x = 0; x < 4; ++x) {
    uint32_t s[32], pp[32];  // 32 slots: 16 columns of first pieces, 16 of second ones
    tmem_ld_32x32b_x32(t_s + 32 * x, s);
    tmem_wait_ld();
    reg_fence(s);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float2 y = f2_fma(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl, ng);
      const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
      rs[c & 1] = f2_add(rs[c & 1], p);
      pp[c] = pack_x2<BF16>(p.x, p.y);
      const float2 r = f2_sub(p, unpack_x2<BF16>(pp[c]));
      pp[16 + c] = pack_x2<BF16>(r.x, r.y);
    }
    tmem_st_32x32b_x32(t_s + 32 * x, pp);
  }
  l = l * alpha + ((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y));
  tmem_wait_st();
  if (!first && __any_sync(0xffffffffu, rescale)) {
    if (!mbar_wait_warp(&sh.o_full[t], (done - 1) & 1, wc)) return false;
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      tmem_ld_32x32b_x32(t_o + c, o);
      tmem_wait_ld();
      reg_fence(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
      tmem_st_32x32b_x32(t_o + c, o);
    }
    tmem_wait_st();
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.p_full[t]);
  return true;
}

// Rows [r0, r0 + n) of a tile of query rows, by a warp, 8 loads in flight.
template <int D>
__device__ __forceinline__ void pfx_load_q(const PrefixArgs& a, int h, int row0, int r0, int n, uint8_t* tile, int lane) {
  constexpr int CH = D / 8, PER = 32 / CH;
  const DecodeArgs& d = a.d;
  const int ch = lane % CH, sub = lane / CH;
#pragma unroll 1
  for (int x = 0; x < n; x += 8 * PER) {
    uint4 v[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const int in = x + y * PER + sub, R = row0 + r0 + in;
      v[y] = make_uint4(0u, 0u, 0u, 0u);
      if (in < n && R < d.rows) {
        const int b = div_by(R, d.fg), gx = R - b * d.g;
        v[y] = ld_global(reinterpret_cast<const uint4*>(
                             d.q + (static_cast<size_t>(b) * d.Hq + static_cast<size_t>(h) * d.g + gx) * D) + ch);
      }
    }
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const int in = x + y * PER + sub, r = r0 + in;
      if (in >= n) continue;
      *reinterpret_cast<uint4*>(tile + (ch / 8) * PfxCfg<D>::SLAB + r * 128 + (((ch % 8) ^ (r & 7)) * 16)) = v[y];
    }
  }
}

// Columns [c0, c1) of a warp's 32 rows, x f0 + y f1, to rows of a part. y only with
// JOIN, and then only if it has been written (any).
template <int D, bool JOIN>
__device__ __forceinline__ void pfx_store(uint32_t tx, uint32_t ty, float f0, float f1, bool any, int c0, int c1,
                                          float* dst, int rows, int lane, float4* slice) {
  const int sub = lane >> 3, seg = lane & 7;
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint32_t x[32], y[32];
    tmem_ld_32x32b_x32(tx + c, x);
    if (JOIN && any) tmem_ld_32x32b_x32(ty + c, y);
    tmem_wait_ld();
    reg_fence(x);
    if (JOIN && any) {
      reg_fence(y);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        x[i] = __float_as_uint(__uint_as_float(x[i]) * f0 + __uint_as_float(y[i]) * f1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      slice[lane * 8 + (i ^ (lane & 7))] = make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                                                       __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + sub;
      const float4 v = slice[r * 8 + (seg ^ (r & 7))];
      if (r < rows) reinterpret_cast<float4*>(dst + static_cast<size_t>(r) * D + c)[seg] = v;
    }
    __syncwarp();
  }
}

template <int D, bool BF16>
__device__ bool pfx_rows(const PrefixArgs& a, PfxWork w, PfxShared<D>& sh, uint8_t* smem, uint32_t tmem, int cta,
                         int warp, int lane, const WaitCtx& wc) {
  using C = PfxCfg<D>;
  const int t = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t t_s = lanes + C::TM_S(t), t_o = lanes + C::TM_O(t);
  float4* slice = reinterpret_cast<float4*>(smem + t * C::TILE + quad * C::STAGE);
  float* sh_m = reinterpret_cast<float*>(smem + C::OFF_ML);  // [2][128], then the second stream's sums [128]
  const float sl2 = a.d.scale_log2;
  int done = 0;          // tasks of this stream so far
  int joined = 0;        // segments of one row tile
  for (int seg = 0; w.left > 0; ++seg) {
    const PfxSeg s = pfx_seg(a, w);
    if (seg > 0 && !mbar_wait_warp(&sh.stored, (seg - 1) & 1, wc)) return false;  // nobody uses the tiles any more
    // Queries: tile t, or half a warp's rows of the one tile each.
    if (s.two) pfx_load_q<D>(a, s.h, s.row0 + t * kTileRows, quad * 32, 32, smem + t * C::TILE, lane);
    else pfx_load_q<D>(a, s.h, s.row0, quad * 32 + t * 16, 16, smem, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_full);
    const int n1 = s.two ? s.cnt : s.cnt / 2, n = t ? n1 : s.cnt - (s.two ? 0 : n1);  // tasks of the second, of this stream
    float m_ref = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) {
      const PfxMask mask = pfx_mask(a, w.P, s.h, s.tile0 + (s.two ? i : 2 * i + t), lane);
      if (!pfx_step<D, BF16>(sh, t, t_s, t_o, mask, a.d.box, sl2, i == 0, done + i, m_ref, l, lane, wc)) return false;
    }
    done += n;
    if (n > 0 && !mbar_wait_warp(&sh.o_full[t], (done - 1) & 1, wc)) return false;
    __syncwarp();
    tc_fence_after();
    const float M = m_ref == -INFINITY ? -INFINITY : m_ref * sl2 - kPfxBias<BF16>;
    const size_t part = static_cast<size_t>(shared_part(w.item, cta)) * 2 * kTileRows;
    if (s.two) {
      const int rows = min(32, s.rows - t * kTileRows - quad * 32);
      pfx_store<D, false>(t_o, 0u, 1.f, 0.f, false, 0, D, a.part_o + (part + t * kTileRows + quad * 32) * D, rows, lane,
                          slice);
      if (lane < rows) a.part_ml[part + t * kTileRows + r] = make_float2(M, l);
    } else {
      // Both streams' sums of the same rows, half of the columns each, when both are
      // complete.
      tc_fence_before();
      sh_m[t * kTileRows + r] = M;
      if (t == 1) sh_m[2 * kTileRows + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ml_full);
      if (!mbar_wait_warp(&sh.ml_full, joined & 1, wc)) return false;
      ++joined;
      __syncwarp();
      tc_fence_after();
      const float m0 = sh_m[r], m1 = sh_m[kTileRows + r];
      const float top = fmaxf(m0, m1), f0 = step_down(m0, top), f1 = step_down(m1, top);
      const int rows = min(32, s.rows - quad * 32);
      pfx_store<D, true>(lanes + C::TM_O(0), lanes + C::TM_O(1), n1 > 0 ? f0 : 1.f, f1, n1 > 0, t * (D / 2),
                         (t + 1) * (D / 2), a.part_o + (part + quad * 32) * D, rows, lane, slice);
      if (t == 0 && lane < rows)
        a.part_ml[part + r] = n1 > 0 ? make_float2(top, l * f0 + sh_m[2 * kTileRows + r] * f1) : make_float2(M, l);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.stored);
    pfx_next(w, s.cnt);
  }
  return true;
}

// With a CTA of the own slots' kernel, 64 KiB of ring, and what the system takes of each
// CTA, at most the 228 KiB of an SM.
static_assert(PfxCfg<128>::SMEM + sizeof(PfxShared<128>) + 65536 + 512 + 2048 <= 233472, "room for both");

template <int D, bool BF16>
__global__ void __maxnreg__(PfxCfg<D>::REGS)
    fa2_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const PrefixArgs a) {
  using C = PfxCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ PfxShared<D> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 8);
    mbar_init(&sh.ml_full, 8);
    mbar_init(&sh.stored, 8);
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], 4);
      mbar_init(&sh.o_full[t], 1);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  grid_dependency_wait();
  grid_launch_dependents();  // the kernel of the own slots relies on the wait above
  const int cta = blockIdx.x;
  long long G;
  const PfxWork w = pfx_work(a, cta, &G);
  if (cta == 0 && threadIdx.x == 0) a.d.starts[a.d.c.B + 1] = G;  // for the join
  if (cta == 0 && threadIdx.x == 0 && ld_global(a.d.prefix_len) != prefix_slots(a.d).len) report_page(a.d.c.status);
  const WaitCtx wc{a.d.c.status, &sh.abort_flag, a.timeout_ns};
  if (warp < 4) {
    setmaxnreg_dec<C::REGS_CONTROL>();
    if (warp == 0)
      pfx_producer<D>(a, w, tm_k, tm_v, sh, smem + C::OFF_RING, lane, wc);
    else if (warp == 1)
      pfx_issuer<D, BF16>(a, w, sh, smem, tmem, wc);
  } else {
    setmaxnreg_inc<C::REGS_ROWS>();
    pfx_rows<D, BF16>(a, w, sh, smem, tmem, cta, warp, lane, wc);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---- Join -----------------------------------------------------------------------
// A query row's parts, of the prefix and of its own slots, by `per_row` warps (a power of
// two, so that each has about four to read at once). A warp takes 1 (d = 128) or 2 parts
// at a time, (m, l) and O read together.
constexpr int kPjThreads = 256, kPjWarps = kPjThreads / 32;
constexpr int kPjResident = 152 * 32;  // warps of the join that run at once

// Infinite entries of V. A remainder of p may be negative or 0, and -1 * inf or 0 * inf
// beside the first piece's product makes NaN in the prefix's kernel of what is infinite.
// So where a row's sum is NaN and its l is a number, V's columns are looked through: an
// infinite entry of a slot that weighs more than 0 makes the output infinite; both signs,
// a NaN, or an infinite entry of a slot that weighs nothing make NaN. By one warp, 4 columns
// a lane, once the row of o stands there. Its time, a row's latency for each 8 slots, counts
// for such rows only: 0.13 us a slot, 2 ms for 64 sequences of 16384 slots with one such
// entry. The others pay for the test of their sums 0.1 us a call, 0.4 at d = 64 (64
// sequences, 32/8 heads, 8192 slots: 49.8 -> 50.0 and 35.6 -> 36.0; as a function that is
// called, in the same registers, 50.1 and 36.2, and 1.2 more in fp16).
template <int D, bool BF16>
__device__ __forceinline__ void pfx_infinite(const DecodeArgs& d, long long row, float M, int lane) {
  constexpr uint32_t EXP = BF16 ? 0x7f80u : 0x7c00u, MAN = BF16 ? 0x7fu : 0x3ffu;
  constexpr int U = 8;  // slots in flight (with 16 the join has too many registers: 1 us a call)
  const CacheView& c = d.c;
  const int b = static_cast<int>(div_pos(row, d.Hq)), x = static_cast<int>(row - static_cast<long long>(b) * d.Hq);
  const int h = div_by(x, d.fg), len = seq_len(c, b), first = prefix_of(len, prefix_slots(d)), e = lane * 4;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(d.q + row * D);
  auto halves = [](const uint2& v, uint32_t (&w)[4]) {
    w[0] = v.x & 0xffffu, w[1] = v.x >> 16, w[2] = v.y & 0xffffu, w[3] = v.y >> 16;
  };
  auto is_nan = [](uint32_t w) { return (w & EXP) == EXP && (w & MAN) != 0u; };
  uint32_t o[4] = {0u, 0u, 0u, 0u}, seen[4] = {0u, 0u, 0u, 0u};  // seen: 1: inf, 2: -inf, 4: NaN
  if (e < D) halves(ld_global(reinterpret_cast<const uint2*>(d.o + row * D + e)), o);
  // A lane looks up the page of one of 32 slots; then all read their columns of each.
  auto look_up = [&](int j) {
    if (j >= len) return -1;
    const int p = div_by(j, c.ps);
    const int page = ld_global(j < first ? d.prefix + p : c.table + static_cast<size_t>(b) * c.max_pages + p);
    return page_row(c, page, h, j - p * c.ps.d);
  };
  int next = look_up(lane);
#pragma unroll 1
  for (int j0 = 0; j0 < len; j0 += 32) {
    bool open = false;  // a column that may still change
#pragma unroll
    for (int i = 0; i < 4; ++i) open |= is_nan(o[i]) && seen[i] < 3u;
    if (!__any_sync(0xffffffffu, open)) break;
    const int rows = next;
    next = look_up(j0 + 32 + lane);
#pragma unroll 1
    for (int u0 = 0; u0 < 32; u0 += U) {
      uint2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = __shfl_sync(0xffffffffu, rows, u0 + u);
        v[u] = make_uint2(0u, 0u);
        if (open && at >= 0) v[u] = ld_global(reinterpret_cast<const uint2*>(d.v + static_cast<size_t>(at) * D + e));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = __shfl_sync(0xffffffffu, rows, u0 + u);
        uint32_t w[4];
        halves(v[u], w);
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= is_nan(o[i]) && (w[i] & EXP) == EXP;
        if (!any) continue;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(d.k + static_cast<size_t>(at) * D);
        float s = 0.f;
#pragma unroll 1
        for (int i = 0; i < D / 2; ++i) {
          const float2 y = unpack_x2<BF16>(ld_global(q + i)), z = unpack_x2<BF16>(ld_global(k + i));
          s = fmaf(y.x, z.x, fmaf(y.y, z.y, s));
        }
        const bool weighs = ex2_approx(s * d.scale_log2 - M) > 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((w[i] & EXP) == EXP) seen[i] |= !weighs || is_nan(w[i]) ? 4u : w[i] >> 15 ? 2u : 1u;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (is_nan(o[i]) && (seen[i] == 1u || seen[i] == 2u)) d.o[row * D + e + i] = static_cast<uint16_t>(EXP | (seen[i] == 2u ? 0x8000u : 0u));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPjThreads)
    fa2_prefix_join_kernel(const PrefixArgs a, int per_row) {
  constexpr int LPR = D / 4, PPW = 32 / LPR, U = 4;
  __shared__ float2 s_ml[kPjWarps];
  __shared__ float4 s_acc[kPjWarps][LPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (per_row - 1);
  const DecodeArgs& d = a.d;
  const CacheView& c = d.c;
  const long long first_row = static_cast<long long>(blockIdx.x) * (kPjWarps / per_row);
  const long long row = first_row + warp / per_row;
  const bool on = row < static_cast<long long>(c.B) * d.Hq;
  const int b = on ? static_cast<int>(div_pos(row, d.Hq)) : 0, x = on ? static_cast<int>(row - static_cast<long long>(b) * d.Hq) : 0;
  const int h = div_by(x, d.fg), gx = x - h * d.g;
  const bool inside = d.row_tiles > 0;  // the prefix was attended to by the kernel of the own slots
  grid_dependency_wait();
  const PrefixLen P = prefix_slots(d);
  const int len = seq_len(c, b);
  const long long T = ld_global(d.starts + c.B), start = ld_global(d.starts + b);
  const long long PG = inside ? 0 : ld_global(d.starts + c.B + 1);
  const int uneven = inside ? 0 : static_cast<int>(ld_global(d.starts + c.B + 2));
  // Parts of the prefix, then own ones: from the first to the last CTA (worker) of an
  // item. Lanes 0 and 1 find those of the prefix, 2 and 3 those of the own slots.
  const int first = prefix_of(len, P), own = len - first;
  auto own_tiles = [&](int n) { return a.tail_warps ? tiles_of<D, kSharedWarp>(n) : tiles_of<D>(n); };
  const int W = a.tail_warps ? kDecWarps : 1;  // workers of a CTA
  const UnitDeal deal(static_cast<int>(min(static_cast<long long>(a.tail_ctas) * W, T)), d.early * W, T, uneven);
  const int R = b * d.g + gx, p_step = inside ? a.head_tile : 2 * kTileRows;
  const int p_tile = inside ? (a.head_tile == 8 ? R >> 3 : R >> 4) : R / (2 * kTileRows);
  const int p_item = h * (inside ? d.row_tiles : a.fblocks.d) + p_tile;
  const int tiles_p = inside ? own_tiles(P.cut) : (P.cut + kTileRows - 1) / kTileRows, tiles_o = own_tiles(own);
  const int o_tile = a.head_tile == 8 ? gx >> 3 : gx >> 4, hh = h * d.HG + o_tile;
  const int o_item = (inside && P.cut > 0 ? d.row_tiles * c.Hkv : 0) + b * c.Hkv * d.HG + hh;
  int cta = 0;
  {
    const bool pre = lane < 2;
    const int tiles = pre ? tiles_p : tiles_o;
    const long long u0 = pre ? static_cast<long long>(p_item) * tiles : start + static_cast<long long>(hh) * tiles;
    if (lane < 4 && (pre ? first : own) > 0) {
      const long long u = u0 + (lane & 1 ? tiles - 1 : 0);
      cta = pre && !inside ? unit_cta(u, PG, static_cast<long long>(a.items) * tiles) : deal.worker(u);
    }
  }
  const int pc = __shfl_sync(0xffffffffu, cta, 0), oc = __shfl_sync(0xffffffffu, cta, 2);
  int np = __shfl_sync(0xffffffffu, cta, 1) - pc + 1, ns = __shfl_sync(0xffffffffu, cta, 3) - oc + 1;
  if (first == 0) np = 0;
  if (own == 0) ns = 0;
  // Their first rows in the workspace.
  const size_t p0 = static_cast<size_t>(shared_part(p_item, pc)) * p_step + (R - p_tile * p_step);
  const size_t o0 = static_cast<size_t>(shared_part(o_item, oc)) * a.head_tile + (gx - o_tile * a.head_tile);
  const float2* p_ml = inside ? d.part_ml : a.part_ml;
  const float* p_o = inside ? d.part_o : a.part_o;
  if (!on) np = ns = 0;
  float M = -INFINITY, S = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m, float l, const float4& v) {
    const float n = fmaxf(M, m), f = step_down(M, n), e = step_down(m, n);
    M = n;
    S = S * f + l * e;
    acc = make_float4(acc.x * f + v.x * e, acc.y * f + v.y * e, acc.z * f + v.z * e, acc.w * f + v.w * e);
  };
  const int e = (lane % LPR) * 4, stride = per_row * PPW;
#pragma unroll 1
  for (int i0 = sub * PPW + lane / LPR; i0 < np + ns; i0 += U * stride) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * stride;
      ml[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np + ns) {
        const bool pre = i < np;
        const size_t at = pre ? p0 + static_cast<size_t>(i) * p_step : o0 + static_cast<size_t>(i - np) * a.head_tile;
        ml[u] = ld_global((pre ? p_ml : d.part_ml) + at);
        v[u] = ld_global(reinterpret_cast<const float4*>((pre ? p_o : d.part_o) + at * D + e));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) add(ml[u].x, ml[u].y, v[u]);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, S, o);
    const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                                 __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
    add(m, l, v);
  }
  if (per_row > 1) {
    if (lane < LPR) s_acc[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(M, S);
    __syncthreads();
    if (sub == 0 && lane < LPR)
      for (int y = 1; y < per_row; ++y) add(s_ml[warp + y].x, s_ml[warp + y].y, s_acc[warp + y][lane]);
  }
  if (!on || sub != 0) return;
  bool nan = false;
  if (lane < LPR) {
    const float inv = S == 0.f ? 0.f : 1.f / S;
    *reinterpret_cast<uint2*>(d.o + row * D + lane * 4) =
        make_uint2(pack_x2<BF16>(acc.x * inv, acc.y * inv), pack_x2<BF16>(acc.z * inv, acc.w * inv));
    if (lane == 0) d.lse[row] = S == 0.f ? -INFINITY : (M + log2f(S)) * kLn2f;
    const float all = (acc.x + acc.y) + (acc.z + acc.w);
    nan = all != all && S > 0.f && S < INFINITY;
  }
  if (__any_sync(0xffffffffu, nan)) pfx_infinite<D, BF16>(d, row, M, lane);
}

cudaError_t launch_decode_suffix(int d, bool bf16, int head_tile, const DecodeArgs& a, bool warps, int ctas,
                                 cudaStream_t stream);

template <int D, bool BF16>
static cudaError_t launch_prefix_t(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.items > 0) {
    auto kern = fa2_prefix_kernel<D, BF16>;
    static std::atomic<unsigned long long> done{0};
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_acquire) == 0) {
      cudaFuncAttributes at;
      e = cudaFuncGetAttributes(&at, kern);
      if (e != cudaSuccess) return e;
      regs.store(at.numRegs, std::memory_order_release);
    }
    if (regs.load(std::memory_order_acquire) < PfxCfg<D>::REGS) return cudaErrorInvalidKernelImage;
    e = allow_smem(kern, PfxCfg<D>::SMEM, done, true);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(a.ctas), dim3(PfxCfg<D>::THREADS), PfxCfg<D>::SMEM, stream, tk, tv, a);
    if (e != cudaSuccess) return e;
  }
  e = launch_decode_suffix(D, BF16, a.head_tile, a.d, a.tail_warps != 0, a.tail_ctas, stream);
  if (e != cudaSuccess) return e;
  // Warps per row: four parts each at a time, about (the CTAs that share an item, and own
  // ones), but no more warps than run at once.
  const int items = a.items > 0 ? a.items : a.d.row_tiles * a.d.c.Hkv, ctas = a.items > 0 ? a.ctas : a.tail_ctas * (a.tail_warps ? kDecWarps : 1);
  const int parts = (ctas + items - 1) / items + 3;
  const long long rows = static_cast<long long>(a.d.c.B) * a.d.Hq;
  int per_row = 1;
  while (per_row < kPjWarps && per_row * 4 * (128 / D) < parts && rows * per_row * 2 <= kPjResident) per_row *= 2;
  return launch_dependent(fa2_prefix_join_kernel<D, BF16>,
                          dim3(static_cast<unsigned>((rows * per_row + kPjWarps - 1) / kPjWarps)), dim3(kPjThreads), 0,
                          stream, a, per_row);
}

cudaError_t launch_prefix_decode(int d, bool bf16, const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                                 cudaStream_t stream) {
  if (d == 64) return bf16 ? launch_prefix_t<64, true>(tk, tv, a, stream) : launch_prefix_t<64, false>(tk, tv, a, stream);
  return bf16 ? launch_prefix_t<128, true>(tk, tv, a, stream) : launch_prefix_t<128, false>(tk, tv, a, stream);
}

}  // namespace fa2
