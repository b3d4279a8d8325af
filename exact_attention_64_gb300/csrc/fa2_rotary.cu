// Rotary positions of queries and keys, with an optional norm per head in the
// same pass, and the backward pass.
//
//   n = (mean_i x_i^2 + eps)^(-1/2), u_i = x_i n w_i   (with weights; else u = x)
//   (y_a, y_b) = A (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = position f_j
// for the pairs j of the first r elements of a head: (a, b) = (2j, 2j + 1), or
// (j, j + r / 2); the other elements are y = u. Backward, with g the gradient dy
// turned back (A, -t):
//   dw_i = sum over rows of g_i x_i n,
//   dx_i = n (w_i g_i - x_i n mean_k(w_k g_k x_k n)).
//
// What bounds it: every element is read and written once, so HBM. A lane has 16
// elements of a row, two runs of 8 that hold both ends of its 8 pairs, so that no
// element changes lanes; 8 (d = 128) or 4 (d = 64) lanes have a row, and keep its
// token's sines for a run of heads, four of which are in flight at once. 1.07 GB (B = 4, 32
// and 32 heads, N = 8192, d = 128) take 157 us, 6.84 TB/s, and with a norm 167; one token
// of 40 heads 3.5. (Two heads in flight and three CTAs per SM 159 and 174; scalar instead
// of paired fp32 instructions 162 and 184.)
// Inputs and outputs may have any strides: a projection's token-major rows become
// the head-major ones of attention without a pass of their own.
//
// Angles: f / 2 pi is formed in two pieces and kept as a 64-bit fraction of a turn, and
// its product with the position modulo 2^64 is exact, so that an angle is right to 2^-31
// turns at any position (|f| up to 2^40): two integer multiplications instead of a
// reduction in 64-bit floating point. Its sine and cosine are taken of 24 bits of it, half
// a turn or less: 2^-26 turns.
#include "fa2_rotary.cuh"

namespace fa2 {

constexpr int kRotUnroll = 4;     // heads in flight per lane

template <int D>
struct RotCfg {
  static constexpr int LANES = D / 16;                    // of a row
  static constexpr int GROUPS = kRotThreads / LANES;      // rows in work per CTA
};

// A lane's 16 elements of a row: two runs of 8, one from each half of the turned part
// (or of the rest), so that neighbouring lanes' runs fill whole sectors. A run holds
// the first or the second elements of 8 pairs, or 4 pairs if they are interleaved.
struct RotLane {
  int e0, e1;  // first elements of its two runs
  int p0, p1;  // pairs of its turns 0 .. 3 and 4 .. 7
  bool turned;
};
__device__ __forceinline__ RotLane rot_lane(int l, int d, int r, int interleaved) {
  RotLane x;
  x.turned = 16 * l < r;
  x.e0 = x.turned ? 8 * l : r + 8 * (l - r / 16);
  x.e1 = x.e0 + (x.turned ? r : d - r) / 2;
  x.p0 = interleaved ? 4 * l : 8 * l;
  x.p1 = interleaved ? r / 4 + 4 * l : 8 * l + 4;
  return x;
}

// A lane's 16 elements as 8 neighbouring pairs: fp32 pairs take one instruction where
// two numbers take two.
template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float2 (&x)[8]) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = unpack_x2<BF16>(w[i]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_x2<BF16>(x[0].x, x[0].y), pack_x2<BF16>(x[1].x, x[1].y), pack_x2<BF16>(x[2].x, x[2].y),
                    pack_x2<BF16>(x[3].x, x[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Weights of a lane's elements.
template <bool BF16>
__device__ __forceinline__ void load_weight(const void* w, int fp32, const RotLane& ln, float2 (&out)[8]) {
  if (fp32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + (h ? ln.e1 : ln.e0));
      const float4 a = ld_global(p), b = ld_global(p + 1);
      out[4 * h] = make_float2(a.x, a.y);
      out[4 * h + 1] = make_float2(a.z, a.w);
      out[4 * h + 2] = make_float2(b.x, b.y);
      out[4 * h + 3] = make_float2(b.z, b.w);
    }
  } else {
    const uint4* p = static_cast<const uint4*>(w);
    const uint4 v[2] = {ld_global(p + ln.e0 / 8), ld_global(p + ln.e1 / 8)};
    unpack16<BF16>(v, out);
  }
}

// The pairs' turns per position as 64-bit fractions, one pair per thread. (In
// 64-bit floating point, which this GPU has little of: once per CTA.) 1 / 2 pi is kInv2Pi +
// kInv2PiLow to 2^-110; what the product with the first rounds off is in the second.
constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLow = -9.839338337591243e-18;
__device__ __forceinline__ void rot_turns(const RotaryArgs& a, unsigned long long* s_turn) {
  for (int i = threadIdx.x; i < a.r / 2; i += kRotThreads) {
    const double f = ld_global(a.freqs + i), t = f * kInv2Pi, low = fma(f, kInv2PiLow, fma(f, kInv2Pi, -t));
    s_turn[i] = __double2ull_rz((t - floor(t)) * 18446744073709551616.0) +
                static_cast<unsigned long long>(__double2ll_rn((low - rint(low)) * 18446744073709551616.0));
  }
}

// A cos t and A sin t of a lane's pairs at a position.
struct RotTurn {
  float2 c[4], s[4];
  __device__ __forceinline__ void set(const unsigned long long* s_turn, const RotLane& ln, int pos, float amp,
                                      float sign) {
    float cv[8], sv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned long long f = ln.turned ? s_turn[i < 4 ? ln.p0 + i : ln.p1 + i - 4] : 0ull;
      // High word of position * f modulo 2^64: the angle in 2^-32 turns.
      const uint32_t lo = static_cast<uint32_t>(f), hi = static_cast<uint32_t>(f >> 32), p = static_cast<uint32_t>(pos);
      const uint32_t w = __umulhi(p, lo) + p * hi - (pos < 0 ? lo : 0u);
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int>(w)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
      cv[i] = cs * amp;
      sv[i] = sn * amp * sign;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(cv[2 * i], cv[2 * i + 1]);
      s[i] = make_float2(sv[2 * i], sv[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void apply(float2 (&x)[8], const RotLane& ln, int interleaved) const {
    if (!ln.turned) return;
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float cv = i & 1 ? c[i / 2].y : c[i / 2].x, sv = i & 1 ? s[i / 2].y : s[i / 2].x;
        x[i] = make_float2(x[i].x * cv - x[i].y * sv, x[i].y * cv + x[i].x * sv);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = x[i], b = x[4 + i];
        x[i] = f2_sub(f2_mul(a, c[i]), f2_mul(b, s[i]));
        x[4 + i] = f2_fma(b, c[i], f2_mul(a, s[i]));
      }
    }
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < RotCfg<D>::LANES; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int rot_position(const RotaryArgs& a, int t, int b, int n) {
  if (a.pos_mode == 0) return n;
  if (a.pos_mode == 1)
    return static_cast<int>(static_cast<uint32_t>(ld_global(a.positions + b)) + static_cast<uint32_t>(n));
  return ld_global(a.positions + t);
}

// Sum of the squares of a row, by its lanes.
template <int D>
__device__ __forceinline__ float row_squares(const float2 (&x)[8]) {
  float2 ss = f2_mul(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) ss = f2_fma(x[i], x[i], ss);
  return row_sum<D>(ss.x + ss.y);
}

// Row of head h of a token.
__device__ __forceinline__ uint4* row_at(const RowView& v, int b, int h, int n) {
  return reinterpret_cast<uint4*>(v.p + b * v.sb + h * v.sh + n * v.sn);
}

// Forward, and backward without a norm (the turn back). A work item is a run of
// heads of one token, queries or keys; tokens vary fastest, so that a warp's rows of
// one head are neighbours. Every lane makes the same number of steps, because the
// norm's sums cross lanes.
template <int D, bool BF16, bool NORM>
__global__ void __launch_bounds__(kRotThreads, 2) fa2_rotary_kernel(const RotaryArgs a) {
  using C = RotCfg<D>;
  constexpr int U = kRotUnroll;
  __shared__ unsigned long long s_turn[D / 2];
  grid_dependency_wait();
  rot_turns(a, s_turn);
  const RotLane ln = rot_lane(threadIdx.x % C::LANES, D, a.r, a.interleaved);
  const long long item = static_cast<long long>(blockIdx.x) * C::GROUPS + threadIdx.x / C::LANES;
  const bool on = item < a.tokens * a.chunks;
  const int it = on ? static_cast<int>(item) : 0;
  const int ck = div_by(it, a.fT), t = it - ck * a.fT.d, b = div_by(t, a.fN), n = t - b * a.N;
  const bool is_q = ck < a.chunks_q;
  const RotarySide& s = is_q ? a.q : a.k;
  const int h0 = (is_q ? ck : ck - a.chunks_q) * a.chunk, h1 = on ? s.H : 0;
  const int pos = rot_position(a, t, b, n);
  float2 w[8];
  if constexpr (NORM) load_weight<BF16>(s.weight, a.weight_fp32, ln, w);
  __syncthreads();
  RotTurn tn;
  tn.set(s_turn, ln, pos, a.amplitude, a.sign);
  const uint4* src = row_at(s.x, b, h0, n);
  uint4* dst = row_at(s.y, b, h0, n);
  const long long x_step = s.x.sh / 8, y_step = s.y.sh / 8;
#pragma unroll 1
  for (int i = 0; i < a.chunk; i += U, src += U * x_step, dst += U * y_step) {
    uint4 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u][0] = v[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h0 + i + u < h1) {
        v[u][0] = ld_global(src + u * x_step + ln.e0 / 8);
        v[u][1] = ld_global(src + u * x_step + ln.e1 / 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 x[8];
      unpack16<BF16>(v[u], x);
      if constexpr (NORM) {
        const float2 inv = both(rsqrtf(row_squares<D>(x) * (1.f / D) + a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = f2_mul(f2_mul(x[j], inv), w[j]);
      }
      tn.apply(x, ln, a.interleaved);
      if (h0 + i + u < h1) {
        const bool same = !NORM && !ln.turned;  // passed through, a NaN's bits too
        dst[u * y_step + ln.e0 / 8] = same ? v[u][0] : pack8<BF16>(x);
        dst[u * y_step + ln.e1 / 8] = same ? v[u][1] : pack8<BF16>(x + 4);
      }
    }
  }
}

constexpr int kRotAhead = 3;                    // heads of a lane in its ring
constexpr int kRotSlot = 4 * kRotThreads * 16;  // bytes of a head of every lane: two runs of x, two of g

// 16 bytes to a lane's own place, or zeros there.
__device__ __forceinline__ void rot_copy16(uint32_t to, const uint4* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}

// A CTA's units: heads of blocks of GROUPS tokens, in this order, all of queries or all
// of keys.
struct RotDeal {
  bool is_q;
  int cta, block, h, left;  // number among its tensor's CTAs; the first unit; their count
  __device__ __forceinline__ RotDeal(const RotaryArgs& a, const RotarySplit& sp, int groups) {
    const bool big = static_cast<int>(blockIdx.x) < sp.big_q + sp.big_k;
    const int x = big ? blockIdx.x : blockIdx.x - sp.big_q - sp.big_k, qs = big ? sp.big_q : sp.small_q;
    is_q = x < qs;
    const int bigs = is_q ? sp.big_q : sp.big_k, smalls = is_q ? sp.small_q : sp.small_k, H = is_q ? a.q.H : a.k.H;
    cta = (is_q ? x : x - qs) + (big ? 0 : bigs);
    auto before = [&](int c) { return min(c, bigs) * (kRotBig - 1) + c; };
    const long long units = (a.tokens + groups - 1) / groups * H, u0 = units * before(cta) / before(bigs + smalls);
    left = static_cast<int>(units * before(cta + 1) / before(bigs + smalls) - u0);
    block = static_cast<int>(u0 / H);
    h = static_cast<int>(u0 - static_cast<long long>(block) * H);
  }
};

// The same for calls of middle size, with a norm for large ones too: each lane copies its
// pieces of the next two heads' rows into its own places of shared memory while it works
// on one, and units are dealt evenly to two CTAs for each SM. Where units are many, six
// sevenths of them, and the last seventh to as many small CTAs, which go where a CTA
// ends first. Measured in us, and by runs of heads as above: B = 16, 8/1 heads, N = 4096, d
// = 64 with a norm 31 and 54, without 30 and 40; B = 8, 16/4 heads, N = 2048, d = 128 with a
// norm 29 and 37; 1.07 GB with a norm 165 and 167. The other way round: B = 1, 32/8 heads,
// N = 512, two units for a token's sines, 5.1 and 4.5; and without a norm, where runs of
// heads are at the copy rate, 537 MB 91 and 81, 1.07 GB 175 and 157. (Five heads ahead:
// 1.07 GB 175 with a norm. Three CTAs per SM: the same.)
template <int D, bool BF16, bool NORM>
__global__ void __launch_bounds__(kRotThreads, 2) fa2_rotary_ring_kernel(const RotaryArgs a, const RotarySplit sp) {
  using C = RotCfg<D>;
  constexpr int U = kRotAhead;
  extern __shared__ __align__(16) uint4 s_ring[];
  __shared__ unsigned long long s_turn[D / 2];
  grid_dependency_wait();
  rot_turns(a, s_turn);
  const RotLane ln = rot_lane(threadIdx.x % C::LANES, D, a.r, a.interleaved);
  const RotDeal deal(a, sp, C::GROUPS);
  const RotarySide& s = deal.is_q ? a.q : a.k;
  int left = deal.left, h = deal.h;
  const long long x_step = s.x.sh / 8, y_step = s.y.sh / 8;
  const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
  long long tt = static_cast<long long>(deal.block) * C::GROUPS + threadIdx.x / C::LANES, ct = tt;
  int ch = h, copies = left, put = 0, take = 0;  // token ct, head ch are copied next
  const uint4* xs = nullptr;
  auto token = [&](long long x, int* b, int* n) {
    const int t = x < a.tokens ? static_cast<int>(x) : 0;
    *b = div_by(t, a.fN);
    *n = t - *b * a.N;
    return t;
  };
  auto seek = [&]() {
    int b, n;
    (void)token(ct, &b, &n);
    xs = row_at(s.x, b, ch, n);
  };
  auto copy = [&]() {
    if (copies > 0) {
      const bool in = ct < a.tokens;
      const uint32_t to = ring + put * (kRotSlot / 2);
      rot_copy16(to, xs + ln.e0 / 8, in);
      rot_copy16(to + kRotThreads * 16, xs + ln.e1 / 8, in);
      put = put + 1 == U ? 0 : put + 1;
      xs += x_step;
      --copies;
      if (++ch == s.H) {
        ch = 0;
        ct += C::GROUPS;
        seek();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  seek();
#pragma unroll 1
  for (int i = 0; i < U - 1; ++i) copy();
  float2 w[8];
  if constexpr (NORM) load_weight<BF16>(s.weight, a.weight_fp32, ln, w);
  __syncthreads();
  RotTurn tn;
  for (; left > 0; tt += C::GROUPS, h = 0) {
    const bool on = tt < a.tokens;
    int b, n;
    const int t = token(tt, &b, &n);
    uint4* dst = row_at(s.y, b, h, n);
    tn.set(s_turn, ln, rot_position(a, t, b, n), a.amplitude, a.sign);
    const int heads = min(left, s.H - h);
    left -= heads;
#pragma unroll 1
    for (int i = 0; i < heads; ++i, dst += y_step) {
      copy();
      asm volatile("cp.async.wait_group %0;" ::"n"(U - 1) : "memory");
      const uint4* at = s_ring + take * (kRotSlot / 32) + threadIdx.x;
      take = take + 1 == U ? 0 : take + 1;
      const uint4 v[2] = {at[0], at[kRotThreads]};
      float2 x[8];
      unpack16<BF16>(v, x);
      if constexpr (NORM) {
        const float2 inv = both(rsqrtf(row_squares<D>(x) * (1.f / D) + a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = f2_mul(f2_mul(x[j], inv), w[j]);
      }
      tn.apply(x, ln, a.interleaved);
      if (on) {
        const bool same = !NORM && !ln.turned;  // passed through, a NaN's bits too
        dst[ln.e0 / 8] = same ? v[0] : pack8<BF16>(x);
        dst[ln.e1 / 8] = same ? v[1] : pack8<BF16>(x + 4);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Backward with a norm. A CTA's rows are all of queries or all of keys, so that a lane's
// 16 sums of the weights' gradients stay in registers; at its end the CTA adds up its
// rows' sums in a fixed order and leaves them in the workspace, so that the bits repeat.
// 127 registers leave 16 warps per SM, and a head that they read ahead in registers is 32
// KiB in flight, which took 50 us for 252 MB (B = 8, 16/4 heads, N = 2048, d = 128). So
// rows are copied to shared memory, two heads ahead of the one in work, where they need no
// registers: 44 us with the sum of the CTAs' parts, 5.7 TB/s (three heads ahead the same),
// and 239 for 1.61 GB (B = 4, 32 + 32 heads, N = 8192), the copy rate; 264 without the small
// CTAs at the end.
template <int D, bool BF16>
__global__ void __launch_bounds__(kRotThreads, 2) fa2_rotary_norm_bwd_kernel(const RotaryArgs a, const RotarySplit sp) {
  using C = RotCfg<D>;
  constexpr int WARPS = kRotThreads / 32;
  extern __shared__ __align__(16) uint4 s_ring[];
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ __align__(8) float s_dw[WARPS][D];
  grid_dependency_wait();
  grid_launch_dependents();
  rot_turns(a, s_turn);
  __syncthreads();
  const RotLane ln = rot_lane(threadIdx.x % C::LANES, D, a.r, a.interleaved);
  const RotDeal deal(a, sp, C::GROUPS);
  const RotarySide& s = deal.is_q ? a.q : a.k;
  int left = deal.left, h = deal.h;
  float2 w[8], dw[8];
  load_weight<BF16>(s.weight, a.weight_fp32, ln, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = make_float2(0.f, 0.f);
  const long long x_step = s.src.sh / 8, g_step = s.x.sh / 8, y_step = s.y.sh / 8;
  // Each lane copies its pieces of the next rows, from one token to the next, into its own
  // places of shared memory; it alone reads them.
  const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
  long long tt = static_cast<long long>(deal.block) * C::GROUPS + threadIdx.x / C::LANES, ct = tt;
  int ch = h, copies = left, put = 0, take = 0;  // token ct, head ch are copied next
  const uint4 *xs = nullptr, *gs = nullptr;
  auto token = [&](long long x, int* b, int* n) {
    const int t = x < a.tokens ? static_cast<int>(x) : 0;
    *b = div_by(t, a.fN);
    *n = t - *b * a.N;
    return t;
  };
  auto seek = [&]() {
    int b, n;
    (void)token(ct, &b, &n);
    xs = row_at(s.src, b, ch, n);
    gs = row_at(s.x, b, ch, n);
  };
  auto copy = [&]() {
    if (copies > 0) {
      const bool in = ct < a.tokens;
      const uint32_t to = ring + put * kRotSlot;
      rot_copy16(to, xs + ln.e0 / 8, in);
      rot_copy16(to + kRotThreads * 16, xs + ln.e1 / 8, in);
      rot_copy16(to + 2 * kRotThreads * 16, gs + ln.e0 / 8, in);
      rot_copy16(to + 3 * kRotThreads * 16, gs + ln.e1 / 8, in);
      put = put + 1 == kRotAhead ? 0 : put + 1;
      xs += x_step;
      gs += g_step;
      --copies;
      if (++ch == s.H) {
        ch = 0;
        ct += C::GROUPS;
        seek();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  seek();
#pragma unroll 1
  for (int i = 0; i < kRotAhead - 1; ++i) copy();
  RotTurn tn;
  for (; left > 0; tt += C::GROUPS, h = 0) {
    const bool on = tt < a.tokens;
    int b, n;
    const int t = token(tt, &b, &n);
    uint4* dst = row_at(s.y, b, h, n);
    tn.set(s_turn, ln, rot_position(a, t, b, n), a.amplitude, -1.f);
    const int heads = min(left, s.H - h);
    left -= heads;
#pragma unroll 1
    for (int i = 0; i < heads; ++i, dst += y_step) {
      copy();
      asm volatile("cp.async.wait_group %0;" ::"n"(kRotAhead - 1) : "memory");
      const uint4* at = s_ring + take * (kRotSlot / 16) + threadIdx.x;
      take = take + 1 == kRotAhead ? 0 : take + 1;
      float2 x[8], y[8];
      {
        const uint4 v[2] = {at[0], at[kRotThreads]}, g[2] = {at[2 * kRotThreads], at[3 * kRotThreads]};
        unpack16<BF16>(v, x);
        unpack16<BF16>(g, y);
      }
      tn.apply(y, ln, a.interleaved);
      const float inv = rsqrtf(row_squares<D>(x) * (1.f / D) + a.eps);
      // z = g n: dw += z x, dx = z w - x n^2 mean(z w x).
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = f2_mul(y[j], both(inv));
        if (on) dw[j] = f2_fma(y[j], x[j], dw[j]);
        y[j] = f2_mul(y[j], w[j]);
        dot = f2_fma(y[j], x[j], dot);
      }
      const float c = row_sum<D>(dot.x + dot.y) * (-1.f / D) * inv * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = f2_fma(x[j], both(c), y[j]);
      if (on) {
        dst[ln.e0 / 8] = pack8<BF16>(y);
        dst[ln.e1 / 8] = pack8<BF16>(y + 4);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = C::LANES; o < 32; o <<= 1) {
      dw[j].x += __shfl_xor_sync(0xffffffffu, dw[j].x, o);
      dw[j].y += __shfl_xor_sync(0xffffffffu, dw[j].y, o);
    }
    if (lane < C::LANES) *reinterpret_cast<float2*>(&s_dw[warp][(j < 4 ? ln.e0 : ln.e1 - 8) + 2 * j]) = dw[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f;
#pragma unroll
    for (int y = 0; y < WARPS; ++y) x += s_dw[y][threadIdx.x];
    a.part[static_cast<size_t>((deal.is_q ? 0 : sp.big_q + sp.small_q) + deal.cta) * D + threadIdx.x] = x;
  }
}

// The sums of the CTAs' parts, 32 elements of one weight per block (blockIdx.y: queries,
// keys), in a fixed order.
constexpr int kRotSumRows = 32;
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kRotSumRows) fa2_rotary_weight_kernel(const RotaryArgs a, int ctas_q, int ctas) {
  __shared__ float s_sum[kRotSumRows][33];
  const RotarySide& s = blockIdx.y == 0 ? a.q : a.k;
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32, e = blockIdx.x * 32 + lane;
  const int first = blockIdx.y == 0 ? 0 : ctas_q, last = blockIdx.y == 0 ? ctas_q : ctas;
  grid_dependency_wait();
  float x = 0.f;
  constexpr int U = 8;  // parts that are read at once
  for (int i = first + row; i < last; i += U * kRotSumRows) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = i + u * kRotSumRows < last ? a.part[static_cast<size_t>(i + u * kRotSumRows) * D + e] : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) x += v[u];
  }
  s_sum[row][lane] = x;
  __syncthreads();
  if (row != 0 || s.H == 0) return;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < kRotSumRows; ++i) y += s_sum[i][lane];
  if (a.weight_fp32) static_cast<float*>(s.weight_grad)[e] = y;
  else static_cast<uint16_t*>(s.weight_grad)[e] = static_cast<uint16_t>(pack_x2<BF16>(y, 0.f) & 0xffffu);
}

template <int D, bool BF16, bool NORM>
static cudaError_t launch_rotary_n(const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream) {
  if (sp.big_q == 0) {
    const long long items = a.tokens * a.chunks;
    const dim3 grid(static_cast<unsigned>((items + RotCfg<D>::GROUPS - 1) / RotCfg<D>::GROUPS));
    return launch_dependent(fa2_rotary_kernel<D, BF16, NORM>, grid, dim3(kRotThreads), 0, stream, a);
  }
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(fa2_rotary_ring_kernel<D, BF16, NORM>, kRotAhead * kRotSlot / 2, done, true);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa2_rotary_ring_kernel<D, BF16, NORM>, dim3(sp.big_q + sp.big_k + sp.small_q + sp.small_k),
                          dim3(kRotThreads), kRotAhead * kRotSlot / 2, stream, a, sp);
}
template <int D, bool BF16>
static cudaError_t launch_rotary_t(const RotaryArgs& a, bool norm, const RotarySplit& sp, cudaStream_t stream) {
  return norm ? launch_rotary_n<D, BF16, true>(a, sp, stream) : launch_rotary_n<D, BF16, false>(a, sp, stream);
}

template <int D, bool BF16>
static cudaError_t launch_rotary_bwd_t(const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream) {
  const int ctas_q = sp.big_q + sp.small_q, ctas = ctas_q + sp.big_k + sp.small_k;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(fa2_rotary_norm_bwd_kernel<D, BF16>, kRotAhead * kRotSlot, done, true);
  if (e != cudaSuccess) return e;
  e = launch_dependent(fa2_rotary_norm_bwd_kernel<D, BF16>, dim3(ctas), dim3(kRotThreads),
                       kRotAhead * kRotSlot, stream, a, sp);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa2_rotary_weight_kernel<D, BF16>, dim3(D / 32, a.k.H > 0 ? 2 : 1),
                          dim3(32 * kRotSumRows), 0, stream, a, ctas_q, ctas);
}

// By units if sp has CTAs, else by runs of heads.
cudaError_t launch_rotary(int d, bool bf16, bool norm, const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream) {
  if (d == 64) return bf16 ? launch_rotary_t<64, true>(a, norm, sp, stream) : launch_rotary_t<64, false>(a, norm, sp, stream);
  return bf16 ? launch_rotary_t<128, true>(a, norm, sp, stream) : launch_rotary_t<128, false>(a, norm, sp, stream);
}

cudaError_t launch_rotary_norm_bwd(int d, bool bf16, const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream) {
  if (d == 64) return bf16 ? launch_rotary_bwd_t<64, true>(a, sp, stream) : launch_rotary_bwd_t<64, false>(a, sp, stream);
  return bf16 ? launch_rotary_bwd_t<128, true>(a, sp, stream) : launch_rotary_bwd_t<128, false>(a, sp, stream);
}

}  // namespace fa2
