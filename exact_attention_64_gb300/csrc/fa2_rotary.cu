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
// token's sines for a run of heads, several of which are in flight at once.
// Inputs and outputs may have any strides: a projection's token-major rows become
// the head-major ones of attention without a pass of their own.
//
// Angles: f / 2 pi is kept as a 64-bit fraction of a turn, and its product with the
// position modulo 2^64 is exact, so that an angle is as exact at position 2^31 as at
// 1: two integer multiplications instead of a reduction in 64-bit floating point.
#include "fa2_rotary.cuh"

namespace fa2 {

constexpr int kRotUnroll = 4;     // heads in flight per lane
constexpr int kRotBwdUnroll = 2;

template <int D>
struct RotCfg {
  static constexpr int LANES = D / 16;                    // of a row
  static constexpr int GROUPS = kRotThreads / LANES;      // rows in work per CTA
};

// A lane's 16 elements of a row, and where they lie in it.
struct RotLane {
  int e0, e1;   // first elements of its two runs
  int pair;     // its first pair
  bool turned;  // its elements are pairs to turn
};
__device__ __forceinline__ RotLane rot_lane(int l, int r, int interleaved) {
  RotLane x;
  x.turned = 16 * l < r;
  x.pair = 8 * l;
  const bool halves = x.turned && !interleaved;
  x.e0 = halves ? 8 * l : 16 * l;
  x.e1 = halves ? r / 2 + 8 * l : 16 * l + 8;
  return x;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_x2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_x2<BF16>(x[0], x[1]), pack_x2<BF16>(x[2], x[3]), pack_x2<BF16>(x[4], x[5]),
                    pack_x2<BF16>(x[6], x[7]));
}

// Weights of a lane's elements.
template <bool BF16>
__device__ __forceinline__ void load_weight(const void* w, int fp32, const RotLane& ln, float (&out)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = h ? ln.e1 : ln.e0;
    if (fp32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + e);
      const float4 a = ld_global(p), b = ld_global(p + 1);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) out[8 * h + i] = v[i];
    } else {
      unpack8<BF16>(ld_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + e)), out + 8 * h);
    }
  }
}

// The pairs' turns per position as 64-bit fractions, one pair per thread. (In
// 64-bit floating point, which this GPU has little of: once per CTA.)
__device__ __forceinline__ void rot_turns(const RotaryArgs& a, unsigned long long* s_turn) {
  for (int i = threadIdx.x; i < a.r / 2; i += kRotThreads) {
    const double t = ld_global(a.freqs + i) * 0.15915494309189533577;
    s_turn[i] = __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
  }
}

// A cos t and A sin t of a lane's pairs at a position.
struct RotTurn {
  float c[8], s[8];
  __device__ __forceinline__ void set(const unsigned long long* s_turn, const RotLane& ln, int pos, float amp,
                                      float sign) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned long long f = ln.turned ? s_turn[ln.pair + i] : 0ull;
      // High word of position * f modulo 2^64: the angle in 2^-32 turns.
      const uint32_t lo = static_cast<uint32_t>(f), hi = static_cast<uint32_t>(f >> 32), p = static_cast<uint32_t>(pos);
      const uint32_t w = __umulhi(p, lo) + p * hi - (pos < 0 ? lo : 0u);
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int>(w)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
      c[i] = cs * amp;
      s[i] = sn * amp * sign;
    }
  }
  __device__ __forceinline__ void turn(float (&x)[16], int interleaved) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& a = interleaved ? x[2 * i] : x[i];
      float& b = interleaved ? x[2 * i + 1] : x[8 + i];
      const float u = a * c[i] - b * s[i], v = b * c[i] + a * s[i];
      a = u;
      b = v;
    }
  }
  __device__ __forceinline__ void apply(float (&x)[16], const RotLane& ln, int interleaved) const {
    if (!ln.turned) return;
    if (interleaved) turn(x, 1);
    else turn(x, 0);
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

__device__ __forceinline__ uint4* row_at(const RowView& v, int b, int h, int n) {
  return reinterpret_cast<uint4*>(v.p + b * v.sb + h * v.sh + n * v.sn);
}

// Forward, and backward without a norm (the turn back). A work item is a run of
// heads of one token, queries or keys; tokens vary fastest, so that a warp's rows of
// one head are neighbours. Every lane makes the same number of steps, because the
// norm's sums cross lanes.
template <int D, bool BF16, bool NORM>
__global__ void __launch_bounds__(kRotThreads) fa2_rotary_kernel(const RotaryArgs a) {
  using C = RotCfg<D>;
  constexpr int U = kRotUnroll;
  __shared__ unsigned long long s_turn[D / 2];
  grid_dependency_wait();
  rot_turns(a, s_turn);
  const RotLane ln = rot_lane(threadIdx.x % C::LANES, a.r, a.interleaved);
  const long long item = static_cast<long long>(blockIdx.x) * C::GROUPS + threadIdx.x / C::LANES;
  const bool on = item < a.tokens * a.chunks;
  const int it = on ? static_cast<int>(item) : 0;
  const int ck = div_by(it, a.fT), t = it - ck * a.fT.d, b = div_by(t, a.fN), n = t - b * a.N;
  const bool is_q = ck < a.chunks_q;
  const RotarySide& s = is_q ? a.q : a.k;
  const int h0 = (is_q ? ck : ck - a.chunks_q) * a.chunk, h1 = on ? s.H : 0;
  const int pos = rot_position(a, t, b, n);
  float w[16];
  if constexpr (NORM) load_weight<BF16>(s.weight, a.weight_fp32, ln, w);
  __syncthreads();
  RotTurn tn;
  tn.set(s_turn, ln, pos, a.amplitude, a.sign);
#pragma unroll 1
  for (int i = 0; i < a.chunk; i += U) {
    uint4 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u][0] = v[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h0 + i + u < h1) {
        const uint4* p = row_at(s.x, b, h0 + i + u, n);
        v[u][0] = ld_global(p + ln.e0 / 8);
        v[u][1] = ld_global(p + ln.e1 / 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[16];
      unpack8<BF16>(v[u][0], x);
      unpack8<BF16>(v[u][1], x + 8);
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
        const float inv = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = x[j] * inv * w[j];
      }
      tn.apply(x, ln, a.interleaved);
      if (h0 + i + u < h1) {
        uint4* p = row_at(s.y, b, h0 + i + u, n);
        const bool same = !NORM && !ln.turned;  // passed through, a NaN's bits too
        p[ln.e0 / 8] = same ? v[u][0] : pack8<BF16>(x);
        p[ln.e1 / 8] = same ? v[u][1] : pack8<BF16>(x + 8);
      }
    }
  }
}

// Backward with a norm. A CTA's items are all queries or all keys of the same run of
// heads (blockIdx.y), so that a lane's 16 sums of the weights' gradients stay in
// registers; at its end the CTA adds up its rows' sums in a fixed order and leaves
// them in the workspace. (Integer order of adds everywhere: the bits repeat.)
template <int D, bool BF16>
__global__ void __launch_bounds__(kRotThreads, 2) fa2_rotary_norm_bwd_kernel(const RotaryArgs a) {
  using C = RotCfg<D>;
  constexpr int U = kRotBwdUnroll, WARPS = kRotThreads / 32;
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ float s_dw[WARPS][D];
  grid_dependency_wait();
  grid_launch_dependents();
  rot_turns(a, s_turn);
  __syncthreads();
  const RotLane ln = rot_lane(threadIdx.x % C::LANES, a.r, a.interleaved);
  const int ck = blockIdx.y;
  const bool is_q = ck < a.chunks_q;
  const RotarySide& s = is_q ? a.q : a.k;
  const int h0 = (is_q ? ck : ck - a.chunks_q) * a.chunk;
  const int steps = min(a.chunk, s.H - h0);
  float w[16], dw[16];
  load_weight<BF16>(s.weight, a.weight_fp32, ln, w);
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[j] = 0.f;
  for (long long t0 = static_cast<long long>(blockIdx.x) * C::GROUPS; t0 < a.tokens;
       t0 += static_cast<long long>(gridDim.x) * C::GROUPS) {
    const long long tt = t0 + threadIdx.x / C::LANES;
    const bool on = tt < a.tokens;
    const int t = on ? static_cast<int>(tt) : 0, b = div_by(t, a.fN), n = t - b * a.N;
    RotTurn tn;
    tn.set(s_turn, ln, rot_position(a, t, b, n), a.amplitude, -1.f);
#pragma unroll 1
    for (int i = 0; i < steps; i += U) {
      uint4 v[U][2], g[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u][0] = v[u][1] = g[u][0] = g[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (on && i + u < steps) {
          const uint4* p = row_at(s.src, b, h0 + i + u, n);
          v[u][0] = ld_global(p + ln.e0 / 8);
          v[u][1] = ld_global(p + ln.e1 / 8);
          p = row_at(s.x, b, h0 + i + u, n);
          g[u][0] = ld_global(p + ln.e0 / 8);
          g[u][1] = ld_global(p + ln.e1 / 8);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u >= steps) break;
        float x[16], y[16];
        unpack8<BF16>(v[u][0], x);
        unpack8<BF16>(v[u][1], x + 8);
        unpack8<BF16>(g[u][0], y);
        unpack8<BF16>(g[u][1], y + 8);
        tn.apply(y, ln, a.interleaved);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
        const float inv = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[j] *= inv;
          if (on) dw[j] += y[j] * x[j];
          y[j] *= w[j];
          dot += y[j] * x[j];
        }
        dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = (y[j] - x[j] * dot) * inv;
        if (on) {
          uint4* p = row_at(s.y, b, h0 + i + u, n);
          p[ln.e0 / 8] = pack8<BF16>(y);
          p[ln.e1 / 8] = pack8<BF16>(y + 8);
        }
      }
    }
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = C::LANES; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
    if (lane < C::LANES) s_dw[warp][(j < 8 ? ln.e0 : ln.e1 - 8) + j] = dw[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f;
#pragma unroll
    for (int y = 0; y < WARPS; ++y) x += s_dw[y][threadIdx.x];
    a.part[(static_cast<size_t>(ck) * gridDim.x + blockIdx.x) * D + threadIdx.x] = x;
  }
}

// The sums of `rows` CTAs, 32 elements of one weight per block (blockIdx.y: queries,
// keys), in a fixed order.
constexpr int kRotSumRows = 32;
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kRotSumRows) fa2_rotary_weight_kernel(const RotaryArgs a, int per_chunk) {
  __shared__ float s_sum[kRotSumRows][33];
  const RotarySide& s = blockIdx.y == 0 ? a.q : a.k;
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32, e = blockIdx.x * 32 + lane;
  const int first = blockIdx.y == 0 ? 0 : a.chunks_q, last = blockIdx.y == 0 ? a.chunks_q : a.chunks;
  grid_dependency_wait();
  float x = 0.f;
#pragma unroll 4
  for (int i = first * per_chunk + row; i < last * per_chunk; i += kRotSumRows) x += a.part[static_cast<size_t>(i) * D + e];
  s_sum[row][lane] = x;
  __syncthreads();
  if (row != 0 || s.H == 0) return;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < kRotSumRows; ++i) y += s_sum[i][lane];
  if (a.weight_fp32) static_cast<float*>(s.weight_grad)[e] = y;
  else static_cast<uint16_t*>(s.weight_grad)[e] = static_cast<uint16_t>(pack_x2<BF16>(y, 0.f) & 0xffffu);
}

template <int D, bool BF16>
static cudaError_t launch_rotary_t(const RotaryArgs& a, bool norm, cudaStream_t stream) {
  const long long items = a.tokens * a.chunks;
  const dim3 grid(static_cast<unsigned>((items + RotCfg<D>::GROUPS - 1) / RotCfg<D>::GROUPS));
  return launch_dependent(norm ? fa2_rotary_kernel<D, BF16, true> : fa2_rotary_kernel<D, BF16, false>, grid,
                          dim3(kRotThreads), 0, stream, a);
}

template <int D, bool BF16>
static cudaError_t launch_rotary_bwd_t(const RotaryArgs& a, int per_chunk, cudaStream_t stream) {
  const cudaError_t e = launch_dependent(fa2_rotary_norm_bwd_kernel<D, BF16>, dim3(per_chunk, a.chunks),
                                         dim3(kRotThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa2_rotary_weight_kernel<D, BF16>, dim3(D / 32, a.k.H > 0 ? 2 : 1),
                          dim3(32 * kRotSumRows), 0, stream, a, per_chunk);
}

cudaError_t launch_rotary(int d, bool bf16, bool norm, const RotaryArgs& a, cudaStream_t stream) {
  if (d == 64) return bf16 ? launch_rotary_t<64, true>(a, norm, stream) : launch_rotary_t<64, false>(a, norm, stream);
  return bf16 ? launch_rotary_t<128, true>(a, norm, stream) : launch_rotary_t<128, false>(a, norm, stream);
}

// Backward with a norm, on a grid of per_chunk CTAs for each run of heads.
cudaError_t launch_rotary_norm_bwd(int d, bool bf16, const RotaryArgs& a, int per_chunk, cudaStream_t stream) {
  if (d == 64)
    return bf16 ? launch_rotary_bwd_t<64, true>(a, per_chunk, stream) : launch_rotary_bwd_t<64, false>(a, per_chunk, stream);
  return bf16 ? launch_rotary_bwd_t<128, true>(a, per_chunk, stream) : launch_rotary_bwd_t<128, false>(a, per_chunk, stream);
}

}  // namespace fa2
