// Attention of one new token over a paged key-value cache.
//
//   s_j = scale q . k_j, L = ln sum_j e^(s_j), o = sum_j e^(s_j - L) v_j over the
//   lens[b] slots of a sequence; with weights also
//   w_out[j] = w_in[j] + sum over the query heads of a key head of e^(s_j - L).
//
// What bounds it: every cached K and V byte is read once for up to 16 query heads
// of a key head (once more for each further 16) and 4 flop per element and head,
// so HBM. What a design has to give is bytes in flight and an even share of the
// cache for every SM whatever the lengths; the arithmetic only has to stay out of
// the way.
//
// Short tables (see the rule at the launch): a CTA has one item, the slots of one
// (sequence, key head), and there is nothing to join and no second launch.
//
// Split, for all others. The cache's slots are cut into units of 64 (sequence, then key head,
// then slot) and CTA c of G takes units [c T / G, (c+1) T / G) of the T units
// that the lengths in device memory amount to: every CTA reads the same share
// of the cache, with one long sequence or many uneven ones, and the same launch
// serves a captured graph whose lengths change. A (sequence, key head) inside
// one CTA's range is finished there; one that is cut leaves its unnormalised
// O, m and l in the workspace, two per CTA at most, and a second launch joins them.
//
// A CTA has 4 warps; warp w owns slots 16 w .. 16 w + 15 of every unit and
// feeds itself: cp.async copies of 16 bytes into its own ring of shared memory
// (rows XOR-swizzled by 16-byte chunk), no CTA-wide barrier until a segment
// ends. 16-byte copies follow any page size, a page per slot included, which a
// bulk copy of a page's run cannot.
//
// Products. S^T = K Q^T with m16n8k16 matrix instructions: the 16 slots are the
// long side and 8 query heads the short one; O^T += V^T P^T with the same, 16
// columns of V the long side. At 8 heads a slot costs 512 bytes (d = 128) and 2 x
// 16/16 to 3 x 16/16 of these instructions, far below what they can do at the
// memory's pace, so tcgen05 (M = 128 rows of which g would be used) would gain
// nothing here. P enters its product in pieces (see "P" below), so that the output
// carries the one rounding at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa2_cache.cuh"

namespace fa2 {

constexpr int kDecWarps = 4;
// Slots per unit: 32 KiB of K and V. A warp has 16 (d = 128) or 32 (d = 64) of
// them, so that its fixed cost per unit (maximum, ring, cursor) is spread over
// the same bytes at both head sizes.
template <int D>
constexpr int kUnit = decode_unit(D);
constexpr float kLn2f = 0.6931471805599453f;
constexpr float kLog2ef = 1.4426950408889634f;

// `pol`: the cache is read once (by a group of up to 16 heads), so its lines leave
// L2 first; what the join reads again (logits, partial results) stays.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full, uint64_t pol) {
  const int n = full ? 16 : 0;  // 0: the 16 bytes are filled with zeros, src is not read
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
               "l"(pol)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// Transpose of an 8 x 8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D (16 x 8, fp32) += A (16 x 8) B (8 x 8), both read to 11 significant bits and
// with the exponents of fp32.
__device__ __forceinline__ void mma1688_tf32(float (&d)[4], const float (&a)[4], float b0, float b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                 "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// ---- P -------------------------------------------------------------------
// P of 16 slots and 8 heads, transposed from the accumulator's layout (slots r8
// and r8 + 8, heads 2t and 2t + 1) into that of a second operand (slots 2t, 2t + 1,
// 2t + 8 and 2t + 9, head r8), and its product with V.
constexpr uint32_t kLow16 = 0x5410u, kHigh16 = 0x7632u;  // both low, both high halves

// bf16: fp32's 24 bits are three pieces of 8, each a bf16 number, so that P enters
// the product as it is. (Two pieces rounded to nearest leave up to 2^-17 of p out,
// and are 1 to 4 % faster where memory is not the bound: 17.2 us against 17.6 for
// B = 8, 32/8 heads of 2000 slots, 30.6 and 31.8 for B = 16, 64/4 heads of 4000; the
// tf32 form below took 18.0 and 33.7.)
//
// A piece after the first is positive where p is: 0 would make 0 * inf = NaN of an
// infinite V. At least 2^-40 of p, it adds nothing that shows; a slot that weighs
// nothing adds nothing.
constexpr float kLeastPiece = 9.094947e-13f;

__device__ __forceinline__ float high_bf16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_high(float x, float y) {
  return __byte_perm(__float_as_uint(x), __float_as_uint(y), kHigh16);
}

template <bool BF16>
struct ProbT;

template <>
struct ProbT<true> {
  uint32_t b[3][2];
  __device__ __forceinline__ void set(const float (&p)[4]) {
    float r[4] = {p[0], p[1], p[2], p[3]};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      b[i][0] = transpose8(pack_high(r[0], r[1]));
      b[i][1] = transpose8(pack_high(r[2], r[3]));
#pragma unroll
      for (int y = 0; y < 4; ++y) r[y] = fmaxf(r[y] - high_bf16(r[y]), p[y] * kLeastPiece);
    }
  }
  __device__ __forceinline__ void add(float (&o)[4], const uint32_t (&va)[4]) const {
#pragma unroll
    for (int i = 0; i < 3; ++i) mma16816<true>(o, va, b[i][0], b[i][1]);
  }
};

// fp16 has no exponents for small p: in two fp16 numbers a slot 2^-25 below the
// largest of its warp would be lost, and such slots together can be what o is made
// of. So V, exact in 11 bits, is multiplied in tf32 by two pieces of p, 11 bits each
// (cut: 2^-21 of p at most). Two fp16 numbers took 13.5 us where this takes 14.6
// (B = 32, 8 heads of 500 slots, d = 128), 30.7 and 33.3 (B = 16, 64/4 heads of 4000
// slots), 27.0 and 28.2 (B = H = 16, 2047 slots, d = 64); large batches are at
// memory's pace either way.
__device__ __forceinline__ float high_tf32(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

template <>
struct ProbT<false> {
  float hi[4], lo[4];
  __device__ __forceinline__ void set(const float (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = __float_as_uint(p[2 * i]), y = __float_as_uint(p[2 * i + 1]);
      const uint32_t u = transpose8(__byte_perm(x, y, kLow16)), v = transpose8(__byte_perm(x, y, kHigh16));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t z = __byte_perm(u, v, j == 0 ? kLow16 : kHigh16);
        hi[2 * i + j] = high_tf32(__uint_as_float(z));
        lo[2 * i + j] = high_tf32(fmaxf(__uint_as_float(z) - hi[2 * i + j], __uint_as_float(z) * kLeastPiece));
      }
    }
  }
  // The order of the 8 slots of an instruction is free: its k = t and t + 4 are
  // slots 2t and 2t + 1, the two halves of a register of V.
  __device__ __forceinline__ void add(float (&o)[4], const uint32_t (&va)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = unpack_x2<false>(va[2 * i]), y = unpack_x2<false>(va[2 * i + 1]);
      const float v[4] = {x.x, y.x, x.y, y.y};
      mma1688_tf32(o, v, hi[2 * i], hi[2 * i + 1]);
      mma1688_tf32(o, v, lo[2 * i], lo[2 * i + 1]);
    }
  }
};

// ---- Units ---------------------------------------------------------------
// HH = Hkv * HG items per sequence: item hh is head tile hh % HG of key head hh / HG.
template <int D>
__device__ __forceinline__ int tiles_of(int n) { return (n + kUnit<D> - 1) / kUnit<D>; }

// Quotient of 0 <= a and b > 0; 32 bits when they do, which is nearly always.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

struct UnitCursor {
  int b, hh, tile;  // sequence, item of the sequence, unit of the item
  int n, ntiles;    // slots of the sequence, units of the item
};

// The units of all sequences, by a whole warp: T, and where a unit lies. Up to
// 32 sequences are read once and their running sums stay with the lanes.
template <int D>
struct UnitMap {
  const CacheView& c;
  int HH, lane, n;
  long long incl, T;

  __device__ UnitMap(const CacheView& view, int hh, int l) : c(view), HH(hh), lane(l) {
    n = length(lane);
    incl = scan(n);
    T = __shfl_sync(0xffffffffu, incl, 31);
    for (int b0 = 32; b0 < c.B; b0 += 32) T += __shfl_sync(0xffffffffu, scan(length(b0 + lane)), 31);
  }
  __device__ int length(int b) const { return b < c.B ? seq_len(c, b) : 0; }
  __device__ long long scan(int slots) const {
    long long t = static_cast<long long>(tiles_of<D>(slots)) * HH;
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
        k.ntiles = tiles_of<D>(k.n);
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

template <int D>
__device__ __forceinline__ void unit_advance(const CacheView& c, int HH, UnitCursor& k) {
  if (++k.tile < k.ntiles) return;
  k.tile = 0;
  if (++k.hh < HH) return;
  k.hh = 0;
  do {
    if (++k.b >= c.B) {
      k.n = k.ntiles = 0;
      return;
    }
    k.n = seq_len(c, k.b);
  } while (k.n == 0);
  k.ntiles = tiles_of<D>(k.n);
}

// Units [u0, u1) of CTA x of G over T units, and the CTA of unit u. With fewer
// units than CTAs, T CTAs take one each.
__device__ __forceinline__ long long unit_begin(long long x, long long G, long long T) { return div_pos(x * T, G); }
__device__ __forceinline__ int unit_cta(long long u, long long G, long long T) {
  return static_cast<int>(div_pos((u + 1) * G - 1, T));
}

// w_out += e^(s - L) over the group's heads for slots [j0, j1). VEC logits of a
// slot are read at a time.
template <int THREADS, int VEC>
__device__ __forceinline__ void add_weights(const DecodeArgs& a, size_t base, int j0, int j1, const float* s_lse) {
  constexpr int U = 4;  // slots per thread in flight
  const int g = a.g;
  for (int j = j0 + threadIdx.x; j < j1; j += U * THREADS) {
    float w[U], add[U];
#pragma unroll
    for (int y = 0; y < U; ++y) {
      const int jj = j + y * THREADS;
      w[y] = jj < j1 ? a.w_in[base + jj] : 0.f;
      add[y] = 0.f;
    }
    for (int hd = 0; hd < g; hd += VEC) {
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const int jj = j + y * THREADS;
        if (jj >= j1) continue;
        const float* lg = a.logits + (base + jj) * g + hd;
        float x[VEC];
        if constexpr (VEC == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(lg);
        else if constexpr (VEC == 2) *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(lg);
        else x[0] = *lg;
#pragma unroll
        for (int e = 0; e < VEC; ++e) add[y] += x[e] == -INFINITY ? 0.f : ex2_approx(x[e] - s_lse[hd + e]);
      }
    }
#pragma unroll
    for (int y = 0; y < U; ++y) {
      const int jj = j + y * THREADS;
      if (jj < j1) a.w_out[base + jj] = w[y] + add[y];
    }
  }
}

template <int THREADS>
__device__ __forceinline__ void add_weights(const DecodeArgs& a, size_t base, int j0, int j1, const float* s_lse) {
  if (a.g % 4 == 0) add_weights<THREADS, 4>(a, base, j0, j1, s_lse);
  else if (a.g % 2 == 0) add_weights<THREADS, 2>(a, base, j0, j1, s_lse);
  else add_weights<THREADS, 1>(a, base, j0, j1, s_lse);
}

template <int D, int NT>
struct DecCfg {
  static constexpr int ROW = D * 2;                        // bytes of a row
  static constexpr int RB = 128 / D;                       // blocks of 16 slots per warp and unit
  static constexpr int ROWS = 16 * RB;                     // slots per warp and unit
  static constexpr int STAGE = 2 * ROWS * ROW;             // a warp's K and V of one unit: 8 KiB
  static constexpr int STAGES = 3;
  static constexpr int RING = kDecWarps * STAGES * STAGE;  // 96 KiB per CTA
  static constexpr int HS = D + 4;                         // merge: floats per head (4: no bank conflicts)
  static constexpr int SMEM = RING + kDecWarps * 8 * HS * 4;
  static constexpr int HEADS = 8 * NT;                     // query heads of a tile
};

template <int D, bool BF16, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(kDecWarps * 32, 2) fa2_paged_decode_kernel(const DecodeArgs a) {
  using C = DecCfg<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[kDecWarps][8];
  __shared__ uint32_t s_mask[kDecWarps][C::STAGES];
  __shared__ float s_lse[C::HEADS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheView& c = a.c;
  const int HH = c.Hkv * a.HG;
  const int cta = blockIdx.x;
  long long u0 = 0, u1 = 0;
  UnitCursor cc{};
  if (a.whole) {
    cc.b = cta / HH;
    cc.hh = cta - cc.b * HH;
    cc.n = seq_len(c, cc.b);
    u1 = cc.ntiles = tiles_of<D>(cc.n);
    if (cc.hh == 0 && threadIdx.x == 0 && ld_global(c.lens + cc.b) != cc.n) report_page(c.status);
    if (cc.n == 0) {  // no token: o = 0, L = -inf
      const int h = cc.hh / a.HG, head0 = (cc.hh - h * a.HG) * C::HEADS;
      const size_t row = static_cast<size_t>(cc.b) * a.Hq + static_cast<size_t>(h) * a.g + head0;
      const int heads = min(C::HEADS, a.g - head0);
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + row * D);
      for (int x = threadIdx.x; x < heads * D / 2; x += kDecWarps * 32) dst[x] = 0u;
      if (threadIdx.x < heads) a.lse[row + threadIdx.x] = -INFINITY;
      return;
    }
  } else {
    const UnitMap<D> map(c, HH, lane);
    const long long T = map.T, G = min(static_cast<long long>(gridDim.x), T);
    if (cta == 0 && warp == 0)
      for (int b = lane; b < c.B; b += 32)
        if (ld_global(c.lens + b) != seq_len(c, b)) report_page(c.status);
    if (cta >= G) return;
    u0 = unit_begin(cta, G, T);
    u1 = unit_begin(cta + 1, G, T);
    cc = map.at(u0);
  }
  UnitCursor ic = cc;  // next unit to copy
  const uint64_t pol = read_once_policy();
  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
  float* merge = reinterpret_cast<float*>(smem + C::RING);

  // Page of this lane's slot (lane mod the warp's slots) in the next unit to
  // copy, looked up one unit ahead of its use.
  long long left = u1 - u0;  // units not yet copied
  int pg = 0, off = 0, hk = 0;
  bool in = false;
  auto look_up = [&]() {
    const int slot = ic.tile * kUnit<D> + warp * C::ROWS + (lane & (C::ROWS - 1));
    in = left > 0 && slot < ic.n;
    hk = a.HG == 1 ? ic.hh : ic.hh / a.HG;
    if (in) {
      const int p = div_by(slot, c.ps);
      off = slot - p * c.ps.d;
      pg = ld_global(c.table + static_cast<size_t>(ic.b) * c.max_pages + p);
    }
  };
  auto copy_next = [&](int st) {
    if (left > 0) {
      const int row = in ? page_row(c, pg, hk, off) : -1;
      if (in && row < 0) report_page(c.status);
      const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) s_mask[warp][st] = mask;
      if (__any_sync(0xffffffffu, in)) {
        constexpr int CH = D / 8;            // 16-byte chunks per row
        constexpr int RPI = 32 / CH;         // rows per warp-wide copy
        const uint32_t base = ring + st * C::STAGE;
        const int ch = lane % CH;
#pragma unroll
        for (int i = 0; i < C::ROWS / RPI; ++i) {
          const int r = i * RPI + lane / CH;
          const int rr = __shfl_sync(0xffffffffu, row, r);
          const size_t e = static_cast<size_t>(max(rr, 0)) * D + ch * 8;
          const uint32_t dst = base + r * C::ROW + ((ch ^ (r & 7)) * 16);
          cp_async16(dst, a.k + e, rr >= 0, pol);
          cp_async16(dst + C::ROWS * C::ROW, a.v + e, rr >= 0, pol);
        }
      }
      unit_advance<D>(c, HH, ic);
      --left;
      look_up();
    }
    cp_async_commit();
  };
  look_up();
#pragma unroll 1
  for (int s = 0; s < C::STAGES; ++s) copy_next(s);

  uint32_t qf[NT][D / 16][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  int st = 0;
  const int t = lane & 3, r8 = lane >> 2;
  auto load_q = [&](const UnitCursor& k) {
    const int h = a.HG == 1 ? k.hh : k.hh / a.HG;
    const int head0 = (k.hh - h * a.HG) * C::HEADS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hd = head0 + nt * 8 + r8;
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(
          a.q + (static_cast<size_t>(k.b) * a.Hq + static_cast<size_t>(h) * a.g + (hd < a.g ? hd : 0)) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[nt][kk][0] = hd < a.g ? ld_global(qp + kk * 8 + t) : 0u;
        qf[nt][kk][1] = hd < a.g ? ld_global(qp + kk * 8 + 4 + t) : 0u;
      }
    }
  };
  load_q(cc);
#pragma unroll 1
  for (long long u = u0; u < u1; ++u) {
    const bool first = u == u0 || cc.tile == 0;
    const int h = a.HG == 1 ? cc.hh : cc.hh / a.HG;
    const int head0 = (cc.hh - h * a.HG) * C::HEADS;  // first head of the tile inside its group
    if (first) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[nt][x][y] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
      }
    }
    cp_async_wait<C::STAGES - 1>();
    __syncwarp();
    const int slot0 = cc.tile * kUnit<D> + warp * C::ROWS;
    if (slot0 < cc.n) {
      const uint32_t mask = s_mask[warp][st];
      const uint32_t kb = ring + st * C::STAGE, vb = kb + C::ROWS * C::ROW;
      const int lr = lane & 15, lc = lane >> 4;  // ldmatrix row and chunk of this lane
      float s[C::RB][NT][4];
#pragma unroll
      for (int rb = 0; rb < C::RB; ++rb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[rb][nt][0] = s[rb][nt][1] = s[rb][nt][2] = s[rb][nt][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int rb = 0; rb < C::RB; ++rb) {
          uint32_t ka[4];
          ldsm4(ka, kb + (rb * 16 + lr) * C::ROW + (((2 * kk + lc) ^ (lr & 7)) * 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(s[rb][nt], ka, qf[nt][kk][0], qf[nt][kk][1]);
        }
      }
      ProbT<BF16> pt[C::RB][NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[C::RB][4];
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int rb = 0; rb < C::RB; ++rb) {
          const bool ok0 = (mask >> (rb * 16 + r8)) & 1u, ok1 = (mask >> (rb * 16 + r8 + 8)) & 1u;
#pragma unroll
          for (int y = 0; y < 4; ++y) x[rb][y] = (y < 2 ? ok0 : ok1) ? s[rb][nt][y] * a.scale_log2 : -INFINITY;
          if constexpr (WEIGHTS) {
            // Logits of slots r8 and r8 + 8, heads 2t and 2t + 1 of the tile.
            const int hd = head0 + nt * 8 + 2 * t, j = slot0 + rb * 16 + r8;
            float* lg = a.logits + ((static_cast<size_t>(cc.b) * c.Hkv + h) * c.L + j) * a.g + hd;
            const bool in0 = j < cc.n, in1 = j + 8 < cc.n;
            if (a.g % 2 == 0) {
              if (hd < a.g && in0) *reinterpret_cast<float2*>(lg) = make_float2(x[rb][0], x[rb][1]);
              if (hd < a.g && in1)
                *reinterpret_cast<float2*>(lg + 8 * static_cast<size_t>(a.g)) = make_float2(x[rb][2], x[rb][3]);
            } else {
              if (hd < a.g && in0) lg[0] = x[rb][0];
              if (hd + 1 < a.g && in0) lg[1] = x[rb][1];
              if (hd < a.g && in1) lg[8 * static_cast<size_t>(a.g)] = x[rb][2];
              if (hd + 1 < a.g && in1) lg[8 * static_cast<size_t>(a.g) + 1] = x[rb][3];
            }
          }
          mx0 = fmaxf(mx0, fmaxf(x[rb][0], x[rb][2]));
          mx1 = fmaxf(mx1, fmaxf(x[rb][1], x[rb][3]));
        }
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, of));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, of));
        }
        // The reference moves only when the maximum grows by more than 8 (log2
        // units): exact, since O and l share it, and p stays below 2^8.
        if (__any_sync(0xffffffffu, mx0 > m[nt][0] + 8.f || mx1 > m[nt][1] + 8.f)) {
          const float n0 = fmaxf(m[nt][0], mx0), n1 = fmaxf(m[nt][1], mx1);
          const float f0 = m[nt][0] == n0 ? 1.f : ex2_approx(m[nt][0] - n0);
          const float f1 = m[nt][1] == n1 ? 1.f : ex2_approx(m[nt][1] - n1);
          m[nt][0] = n0;
          m[nt][1] = n1;
          l[nt][0] *= f0;
          l[nt][1] *= f1;
#pragma unroll
          for (int y = 0; y < D / 16; ++y) {
            o[nt][y][0] *= f0;
            o[nt][y][1] *= f1;
            o[nt][y][2] *= f0;
            o[nt][y][3] *= f1;
          }
        }
        const float z0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], z1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int rb = 0; rb < C::RB; ++rb) {
          float p[4];
          p[0] = ex2_approx(x[rb][0] - z0);
          p[1] = ex2_approx(x[rb][1] - z1);
          p[2] = ex2_approx(x[rb][2] - z0);
          p[3] = ex2_approx(x[rb][3] - z1);
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pt[rb][nt].set(p);
        }
      }
      const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
#pragma unroll
        for (int rb = 0; rb < C::RB; ++rb) {
          uint32_t va[4];
          ldsm4_t(va, vb + (rb * 16 + vr) * C::ROW + (((2 * dt + vc) ^ (vr & 7)) * 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) pt[rb][nt].add(o[nt][dt], va);
        }
      }
    }
    __syncwarp();
    copy_next(st);
    st = st + 1 == C::STAGES ? 0 : st + 1;

    if (u + 1 == u1 || cc.tile + 1 == cc.ntiles) {
      // End of a segment: the four warps' (m, l, O) are merged, while the next
      // one's queries are on their way.
      UnitCursor next = cc;
      unit_advance<D>(c, HH, next);
      if (u + 1 < u1) load_q(next);
      const bool from_start = cc.tile - (u - u0) <= 0;  // the segment begins with its item
      const bool whole = from_start && cc.tile + 1 == cc.ntiles;
      const int slot = 2 * cta + (from_start ? 1 : 0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float x = l[nt][y];
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) x += __shfl_xor_sync(0xffffffffu, x, of);
          if (r8 == 0) s_ml[warp][2 * t + y] = make_float2(m[nt][y], x);
        }
        float* mg = merge + warp * 8 * C::HS;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          mg[(2 * t) * C::HS + x * 16 + r8] = o[nt][x][0];
          mg[(2 * t + 1) * C::HS + x * 16 + r8] = o[nt][x][1];
          mg[(2 * t) * C::HS + x * 16 + r8 + 8] = o[nt][x][2];
          mg[(2 * t + 1) * C::HS + x * 16 + r8 + 8] = o[nt][x][3];
        }
        __syncthreads();
        const int hd = threadIdx.x >> 4;              // head of the tile of 8
        const int e0 = (threadIdx.x & 15) * (D / 16); // its first element here
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, s_ml[w][hd].x);
        float S = 0.f, acc[D / 16];
#pragma unroll
        for (int x = 0; x < D / 16; ++x) acc[x] = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float2 ml = s_ml[w][hd];
          const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
          S += ml.y * f;
          const float4* src = reinterpret_cast<const float4*>(merge + (w * 8 + hd) * C::HS + e0);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const float4 y = src[x];
            acc[4 * x] += y.x * f;
            acc[4 * x + 1] += y.y * f;
            acc[4 * x + 2] += y.z * f;
            acc[4 * x + 3] += y.w * f;
          }
        }
        const int gh = head0 + nt * 8 + hd;
        if (gh < a.g) {
          if (whole) {
            const size_t row = static_cast<size_t>(cc.b) * a.Hq + static_cast<size_t>(h) * a.g + gh;
            const float inv = S == 0.f ? 0.f : 1.f / S;
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + row * D + e0);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) dst[x] = pack_x2<BF16>(acc[2 * x] * inv, acc[2 * x + 1] * inv);
            if (e0 == 0) {
              const float lse = S == 0.f ? -INFINITY : M + log2f(S);
              a.lse[row] = lse * kLn2f;
              if constexpr (WEIGHTS) s_lse[nt * 8 + hd] = lse;
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(
                a.part_o + (static_cast<size_t>(slot) * C::HEADS + nt * 8 + hd) * D + e0);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              dst[x] = make_float4(acc[4 * x], acc[4 * x + 1], acc[4 * x + 2], acc[4 * x + 3]);
            if (e0 == 0) a.part_ml[static_cast<size_t>(slot) * C::HEADS + nt * 8 + hd] = make_float2(M, S);
          }
        }
        __syncthreads();
      }
    }
    unit_advance<D>(c, HH, cc);
  }
  if constexpr (WEIGHTS) {
    if (a.whole) {  // a key head is one item: its weights from the logits that this CTA wrote
      const int hh = cta % HH, b = cta / HH;
      add_weights<kDecWarps * 32>(a, (static_cast<size_t>(b) * c.Hkv + hh) * c.L, 0, seq_len(c, b), s_lse);
    }
  }
}

// ---- Join ------------------------------------------------------------------
// The same CTAs over the same units. The P parts of a cut item are joined by the
// CTAs that hold them, each taking every P-th piece of 32 elements of a head;
// then, with weights, every CTA adds its own slots' weights, e^(s - L) summed over
// the group's heads, from the logits that it wrote.

// Parts [c0, c1] of the item of units [ub, ub + ntiles).
struct ItemParts {
  int c0, c1;
};
__device__ __forceinline__ ItemParts item_parts(long long ub, int ntiles, long long G, long long T) {
  return ItemParts{unit_cta(ub, G, T), unit_cta(ub + ntiles - 1, G, T)};
}
// Workspace slot of CTA x's part of an item whose first part is CTA c0's.
__device__ __forceinline__ int part_slot(int x, int c0) { return 2 * x + (x == c0 ? 1 : 0); }

// 2^(from - to) for a reference that rises to `to`. 1 at -inf, where all that
// there is are zeros, or NaN that has to stay.
__device__ __forceinline__ float step_down(float from, float to) { return from == to ? 1.f : ex2_approx(from - to); }

// (M, S) of one head over an item's parts, by a whole warp.
__device__ __forceinline__ float2 join_ml(const float2* part_ml, int heads, int hd, ItemParts p, int lane) {
  float M = -INFINITY, S = 0.f;
#pragma unroll 4
  for (int x = p.c0 + lane; x <= p.c1; x += 32) {
    const float2 ml = part_ml[static_cast<size_t>(part_slot(x, p.c0)) * heads + hd];
    const float n = fmaxf(M, ml.x);
    S = S * step_down(M, n) + ml.y * step_down(ml.x, n);
    M = n;
  }
  float top = M;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  S *= step_down(M, top);
#pragma unroll
  for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
  return make_float2(top, S);
}

// What bounds the join: the latency of a few dependent reads, and with weights
// the logits, which come from L2. Without weights (m, l) and O are read together
// and a CTA's two cut items at once (8 heads of 512 slots 5.8 us with the decode,
// 6.5 with (m, l) first and one item after the other; of 2048 slots 7.6 and 10.2).
// With weights a thread has several loads in flight, and a CTA's range is shared
// by up to kJoinSplit blocks, one per kJoinUnits units. All blocks have to be
// resident at once: 2 x 304 blocks of 256 threads with 64 registers fill the SMs;
// with 4 x 304 those waiting for the decode to end kept the rest out (118 us
// against 110 for the decode of 32 sequences, 613 MB, with weights).
constexpr int kJoinThreads = 256;
constexpr int kJoinSplit = 2;
constexpr int kJoinUnits = 8;

// Elements e0 .. e0 + 3 of a head's output, and its L.
template <int D, bool BF16>
__device__ __forceinline__ void store_piece(const DecodeArgs& a, size_t row, int e0, float M, float S,
                                            const float4& acc) {
  const float inv = S == 0.f ? 0.f : 1.f / S;
  *reinterpret_cast<uint2*>(a.o + row * D + e0) =
      make_uint2(pack_x2<BF16>(acc.x * inv, acc.y * inv), pack_x2<BF16>(acc.z * inv, acc.w * inv));
  if (e0 == 0) a.lse[row] = S == 0.f ? -INFINITY : (M + log2f(S)) * kLn2f;
}

// With weights: O and L of the heads of one cut item, by block `sub` of `subs` of
// CTA `cta`, and (M, S) of its heads. (The forms below without weights, with the
// heads' (M, S) formed apart: up to 1 us slower.)
// Pieces of 32 elements of a head are dealt to the blocks of all its parts.
template <int D, bool BF16, int NT>
__device__ __forceinline__ void join_item(const DecodeArgs& a, const UnitCursor& k, ItemParts p, int cta, int sub,
                                          int subs, int warp, int lane, bool need_ml, float2* s_ml, float4 (*s_acc)[8]) {
  constexpr int HEADS = 8 * NT, WARPS = kJoinThreads / 32, PC = D / 32;
  const int P = p.c1 - p.c0 + 1;
  const int h = k.hh / a.HG, hg = k.hh - h * a.HG;
  const int heads = min(HEADS, a.g - hg * HEADS);
  const size_t row0 = static_cast<size_t>(k.b) * a.Hq + static_cast<size_t>(h) * a.g + hg * HEADS;
  if (!need_ml && (cta - p.c0) * subs + sub >= heads * PC) return;  // nothing dealt to this block
  for (int hd = warp; hd < heads; hd += WARPS) {
    const float2 x = join_ml(a.part_ml, HEADS, hd, p, lane);
    if (lane == 0) s_ml[hd] = x;
  }
  __syncthreads();
  // Few parts: a warp per piece, four parts at a time. Many: the block.
  const bool wide = P > 32;
  const int rank = (cta - p.c0) * subs + sub, ranks = P * subs;
  const int step = wide ? kJoinThreads / 8 : 4, first = wide ? threadIdx.x >> 3 : lane >> 3;
  for (int y = wide ? rank : rank + ranks * warp; y < heads * PC; y += wide ? ranks : ranks * WARPS) {
    const int hd = y / PC, e0 = (y - hd * PC) * 32 + (lane & 7) * 4;
    const float2 ml = s_ml[hd];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = p.c0 + first; x <= p.c1; x += step) {
      const size_t at = static_cast<size_t>(part_slot(x, p.c0)) * HEADS + hd;
      const float px = a.part_ml[at].x;
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * D + e0);
      const float f = step_down(px, ml.x);
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (wide) {
      if (lane < 8) s_acc[warp][lane] = acc;
      __syncthreads();
      if (warp == 0 && lane < 8) {
#pragma unroll
        for (int x = 1; x < WARPS; ++x) {
          const float4 v = s_acc[x][lane];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
      }
      __syncthreads();
    }
    if (lane < 8 && (!wide || warp == 0)) {
      store_piece<D, BF16>(a, row0 + hd, e0, ml.x, ml.y, acc);
    }
  }
  __syncthreads();
}

// A piece of 32 elements of one head of an item with few parts, by a warp: four
// groups of 8 lanes have two parts each, whose (m, l) and O are read together.
// Block x of the P that hold the parts has the pieces x, x + P, ...
constexpr int kFewParts = 8;
template <int D, bool BF16, int NT>
struct FewParts {
  float2 ml[2];
  float4 v[2];
  size_t row;
  int e0;
  bool on;

  __device__ __forceinline__ void load(const DecodeArgs& a, const UnitCursor& k, ItemParts p, int y, int lane) {
    constexpr int HEADS = 8 * NT, PC = D / 32;
    const int h = k.hh / a.HG, hg = k.hh - h * a.HG;
    on = p.c1 > p.c0 && p.c1 - p.c0 < kFewParts && y < min(HEADS, a.g - hg * HEADS) * PC;
    const int hd = y / PC;
    e0 = (y - hd * PC) * 32 + (lane & 7) * 4;
    row = static_cast<size_t>(k.b) * a.Hq + static_cast<size_t>(h) * a.g + hg * HEADS + hd;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = p.c0 + (lane >> 3) + 4 * u;
      ml[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on && x <= p.c1) {
        const size_t at = static_cast<size_t>(part_slot(x, p.c0)) * HEADS + hd;
        ml[u] = a.part_ml[at];
        v[u] = *reinterpret_cast<const float4*>(a.part_o + at * D + e0);
      }
    }
  }
  __device__ __forceinline__ void finish(const DecodeArgs& a, int lane) const {
    if (!on) return;
    float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float f[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) f[u] = step_down(ml[u].x, M);
    float S = f[0] * ml[0].y + f[1] * ml[1].y;
    float4 acc = make_float4(f[0] * v[0].x + f[1] * v[1].x, f[0] * v[0].y + f[1] * v[1].y,
                             f[0] * v[0].z + f[1] * v[1].z, f[0] * v[0].w + f[1] * v[1].w);
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (lane < 8) store_piece<D, BF16>(a, row, e0, M, S, acc);
  }
};

// The same of an item with many parts, by the block: 32 groups of 8 threads.
template <int D, bool BF16, int NT>
struct ManyParts {
  float M, S;
  float4 acc;
  size_t row;
  int e0;
  bool on;

  __device__ __forceinline__ void add(float m, float l, const float4& v) {
    const float n = fmaxf(M, m), f = step_down(M, n), g = step_down(m, n);
    M = n;
    S = S * f + l * g;
    acc = make_float4(acc.x * f + v.x * g, acc.y * f + v.y * g, acc.z * f + v.z * g, acc.w * f + v.w * g);
  }
  __device__ __forceinline__ void load(const DecodeArgs& a, const UnitCursor& k, ItemParts p, int y) {
    constexpr int HEADS = 8 * NT, PC = D / 32;
    const int h = k.hh / a.HG, hg = k.hh - h * a.HG;
    on = p.c1 - p.c0 >= kFewParts && y < min(HEADS, a.g - hg * HEADS) * PC;
    const int hd = y / PC;
    e0 = (y - hd * PC) * 32 + (threadIdx.x & 7) * 4;
    row = static_cast<size_t>(k.b) * a.Hq + static_cast<size_t>(h) * a.g + hg * HEADS + hd;
    M = -INFINITY;
    S = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!on) return;
#pragma unroll 4
    for (int x = p.c0 + (threadIdx.x >> 3); x <= p.c1; x += kJoinThreads / 8) {
      const size_t at = static_cast<size_t>(part_slot(x, p.c0)) * HEADS + hd;
      const float2 ml = a.part_ml[at];
      add(ml.x, ml.y, *reinterpret_cast<const float4*>(a.part_o + at * D + e0));
    }
  }
  __device__ __forceinline__ void finish(const DecodeArgs& a, float4 (*s_acc)[8], float2* s_part) {
    if (!on) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, S, o);
      const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                                   __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
      add(m, l, v);
    }
    if (lane < 8) s_acc[warp][lane] = acc;
    if (lane == 0) s_part[warp] = make_float2(M, S);
    __syncthreads();
    if (warp == 0 && lane < 8) {
#pragma unroll
      for (int x = 1; x < kJoinThreads / 32; ++x) add(s_part[x].x, s_part[x].y, s_acc[x][lane]);
      store_piece<D, BF16>(a, row, e0, M, S, acc);
    }
    __syncthreads();
  }
};

template <int D, bool BF16, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(kJoinThreads, 4) fa2_paged_join_kernel(const DecodeArgs a) {
  constexpr int HEADS = 8 * NT, WARPS = kJoinThreads / 32;
  const int split = a.join_split;
  __shared__ float2 s_ml[2][HEADS];  // of the CTA's first and last item, if cut
  __shared__ float4 s_acc[WARPS][8];
  __shared__ float2 s_part[WARPS];
  __shared__ float s_lse[kMaxGroup];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheView& c = a.c;
  const int HH = c.Hkv * a.HG;
  const UnitMap<D> map(c, HH, lane);
  const long long T = map.T;
  const long long G = min(static_cast<long long>(gridDim.x / split), T);
  const int cta = blockIdx.x / split, sub = blockIdx.x - cta * split;
  long long u0 = 0, u1 = 0, v0 = 0, v1 = 0;  // units of the CTA, and this block's share of them
  int subs = 1;
  UnitCursor first{}, last{}, cc{};
  if (cta < G) {
    u0 = unit_begin(cta, G, T);
    u1 = unit_begin(cta + 1, G, T);
    // The same for every CTA, whose shares may differ by one unit: the pieces of
    // an item are dealt to the blocks of all its parts.
    subs = static_cast<int>(max(1LL, min(static_cast<long long>(split), div_pos(div_pos(T, G), kJoinUnits))));
    if (sub < subs) {
      v0 = u0 + div_pos((u1 - u0) * sub, subs);
      v1 = u0 + div_pos((u1 - u0) * (sub + 1), subs);
      first = last = cc = map.at(u0);
      last.tile += static_cast<int>(u1 - 1 - u0);
      if (first.tile + (u1 - 1 - u0) >= first.ntiles) last = map.at(u1 - 1);
      if (sub > 0) cc = map.at(v0);
    }
  }
  // Sequences without a token: o = 0, L = -inf. (All before the decode has ended
  // once this kernel runs, and the decode itself leaves their rows alone.)
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    if (seq_len(c, b) > 0) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + static_cast<size_t>(b) * a.Hq * D);
    for (int x = threadIdx.x; x < a.Hq * D / 2; x += kJoinThreads) dst[x] = 0u;
    for (int x = threadIdx.x; x < a.Hq; x += kJoinThreads) a.lse[static_cast<size_t>(b) * a.Hq + x] = -INFINITY;
  }
  grid_dependency_wait();
  if (cta >= G || sub >= subs) return;
  // Only the first and the last item of a CTA can be cut.
  const long long b_first = u0 - first.tile, b_last = u1 - 1 - last.tile;  // their first units
  const ItemParts pf = item_parts(b_first, first.ntiles, G, T);
  const ItemParts pl = b_last > b_first ? item_parts(b_last, last.ntiles, G, T) : ItemParts{0, 0};
  const bool cut_first = pf.c0 != pf.c1, cut_last = pl.c0 != pl.c1;
  if constexpr (!WEIGHTS) {
    const int at_f = cta - pf.c0, at_l = cta - pl.c0, P = pf.c1 - pf.c0 + 1, Q = pl.c1 - pl.c0 + 1;
    if ((cut_first && P <= kFewParts) || (cut_last && Q <= kFewParts)) {
      for (int i = warp;; i += WARPS) {
        FewParts<D, BF16, NT> x, y;
        x.load(a, first, pf, at_f + P * i, lane);
        y.load(a, last, pl, at_l + Q * i, lane);
        if (!x.on && !y.on) break;
        x.finish(a, lane);
        y.finish(a, lane);
      }
    }
    if (P > kFewParts || Q > kFewParts) {
      for (int i = 0;; ++i) {
        ManyParts<D, BF16, NT> x, y;
        x.load(a, first, pf, at_f + P * i);
        y.load(a, last, pl, at_l + Q * i);
        if (!x.on && !y.on) break;
        x.finish(a, s_acc, s_part);
        y.finish(a, s_acc, s_part);
      }
    }
  } else {
    if (cut_first)
      join_item<D, BF16, NT>(a, first, pf, cta, sub, subs, warp, lane, v0 < b_first + first.ntiles, s_ml[0], s_acc);
    if (cut_last) join_item<D, BF16, NT>(a, last, pl, cta, sub, subs, warp, lane, v1 > b_last, s_ml[1], s_acc);
  }
  if constexpr (WEIGHTS) {
    for (long long u = v0; u < v1;) {
      const int cnt = static_cast<int>(min(static_cast<long long>(cc.ntiles - cc.tile), v1 - u));
      const int h = cc.hh / a.HG;
      if (cc.hh == h * a.HG) {  // one head tile of a group adds for all
        const long long ub = u - cc.tile;
        // L of every head of the group, whatever its tile's parts are.
        for (int hd = warp; hd < a.g; hd += WARPS) {
          const int x = hd / HEADS;
          float2 ml;
          bool whole = false;
          if (x == 0 && ub == b_first && cut_first) {
            ml = s_ml[0][hd];
          } else if (x == 0 && ub == b_last && cut_last) {
            ml = s_ml[1][hd];
          } else {
            const ItemParts p = item_parts(ub + static_cast<long long>(x) * cc.ntiles, cc.ntiles, G, T);
            whole = p.c0 == p.c1;
            if (!whole) ml = join_ml(a.part_ml, HEADS, hd - x * HEADS, p, lane);
          }
          float v;
          if (whole) v = a.lse[static_cast<size_t>(cc.b) * a.Hq + static_cast<size_t>(h) * a.g + hd] * kLog2ef;
          else v = ml.y == 0.f ? -INFINITY : ml.x + log2f(ml.y);
          if (lane == 0) s_lse[hd] = v;
        }
        __syncthreads();
        const size_t base = (static_cast<size_t>(cc.b) * c.Hkv + h) * c.L;
        const int j0 = cc.tile * kUnit<D>, j1 = min((cc.tile + cnt) * kUnit<D>, cc.n);
        add_weights<kJoinThreads>(a, base, j0, j1, s_lse);
        __syncthreads();  // s_lse is rewritten by the next item
      }
      cc.tile += cnt - 1;
      unit_advance<D>(c, HH, cc);
      u += cnt;
    }
  }
}

template <int D, bool BF16, int NT, bool WEIGHTS>
static cudaError_t launch_decode_t(DecodeArgs a, int ctas, cudaStream_t stream) {
  // A full table gives each CTA this many units; the lengths may give fewer.
  const long long per = static_cast<long long>(a.c.B) * a.c.Hkv * a.HG * ((a.c.L + kUnit<D> - 1) / kUnit<D>) / ctas;
  a.join_split = WEIGHTS && per >= 2 * kJoinUnits ? kJoinSplit : 1;
  using C = DecCfg<D, NT>;
  auto kern = fa2_paged_decode_kernel<D, BF16, NT, WEIGHTS>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  if (a.whole)
    return launch_dependent(kern, dim3(static_cast<unsigned>(a.c.B) * a.c.Hkv * a.HG), dim3(kDecWarps * 32), C::SMEM,
                            stream, a);
  e = launch_dependent(kern, dim3(ctas), dim3(kDecWarps * 32), C::SMEM, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa2_paged_join_kernel<D, BF16, NT, WEIGHTS>, dim3(ctas * a.join_split),
                          dim3(kJoinThreads), 0, stream, a);
}

cudaError_t launch_paged_decode(int d, bool bf16, int head_tile, const DecodeArgs& a, int ctas,
                                cudaStream_t stream) {
  const bool w = a.w_out != nullptr;
#define FA2_DEC_CASE(DD, BB, NN, WW) \
  if (d == DD && bf16 == BB && head_tile == 8 * NN && w == WW) \
    return launch_decode_t<DD, BB, NN, WW>(a, ctas, stream);
#define FA2_DEC_CASES(DD, BB) \
  FA2_DEC_CASE(DD, BB, 1, false) FA2_DEC_CASE(DD, BB, 1, true) \
  FA2_DEC_CASE(DD, BB, 2, false) FA2_DEC_CASE(DD, BB, 2, true)
  FA2_DEC_CASES(64, true)
  FA2_DEC_CASES(64, false)
  FA2_DEC_CASES(128, true)
  FA2_DEC_CASES(128, false)
#undef FA2_DEC_CASES
#undef FA2_DEC_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa2
