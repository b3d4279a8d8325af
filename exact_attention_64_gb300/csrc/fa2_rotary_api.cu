// C ABI of the rotary positions: argument validation, work split and launches.
// Declarations and argument contracts live in include/fa2.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fa2.h"
#include "fa2_host.h"
#include "fa2_rotary.cuh"

namespace fa2 {
cudaError_t launch_rotary(int d, bool bf16, bool norm, const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream);
cudaError_t launch_rotary_norm_bwd(int d, bool bf16, const RotaryArgs& a, const RotarySplit& sp, cudaStream_t stream);
}  // namespace fa2

namespace {

constexpr long long kMaxItems = (1LL << 31) - 1;
constexpr int kRotCtas = 304;  // CTAs that run at once: two on each of 152 SMs
constexpr long long kRotSmall = 24 * kRotCtas;  // units from which as many small CTAs follow
// Units from which the turn is dealt by them, and, without a norm, up to which.
constexpr long long kRotUnits = 5 * kRotCtas, kRotMaxUnits = 64 * kRotCtas;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Sizes {
  int B, N, d;
};

// A strided tensor argument.
struct Rows {
  const void* p;
  const long long* st;  // strides of batch, head and token, in elements
  int H;
};

// Elements from the first to one past the last.
long long span(const Rows& r, const Sizes& z) {
  const int n[3] = {z.B, r.H, z.N};
  long long e = z.d;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1) e += (n[i] - 1) * r.st[i];
  return e;
}

int check_rows(const Rows& r, const Sizes& z) {
  if (!aligned(r.p, 16)) return FA2_ERR_ALIGNMENT;
  const int n[3] = {z.B, r.H, z.N};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (r.st[i] < 0 || r.st[i] > (1LL << 40)) return FA2_ERR_INVALID_ARG;
    if (r.st[i] % 8 != 0) return FA2_ERR_ALIGNMENT;
  }
  return FA2_OK;
}

// Whether rows of `d` elements at these (size, stride) dimensions are disjoint, by the
// sufficient rule that sorted by stride each step clears all that lies below it.
// *below: the elements that all of them span.
bool disjoint(const int* n, const long long* st, int dims, long long first, long long* below) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + dims, [&](int x, int y) { return st[x] < st[y]; });
  long long room = first;
  for (int i = 0; i < dims; ++i) {
    const int x = order[i];
    if (n[x] == 1) continue;
    if (st[x] < room) return false;
    room += (n[x] - 1) * st[x];
  }
  *below = room;
  return true;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Whether two outputs share an element. Two views of one buffer whose heads stand
// side by side, in a token's row (a packed projection) or head by head, do not.
bool outputs_clash(const Rows& x, const Rows& y, const Sizes& z) {
  if (!overlap(x.p, span(x, z) * 2, y.p, span(y, z) * 2)) return false;
  const Rows &lo = x.p < y.p ? x : y, &hi = x.p < y.p ? y : x;
  if ((z.B > 1 && x.st[0] != y.st[0]) || (z.N > 1 && x.st[2] != y.st[2])) return true;
  const long long bytes = static_cast<const char*>(hi.p) - static_cast<const char*>(lo.p);
  if (bytes % 2 != 0) return true;
  const long long off = bytes / 2;
  long long below = 0;
  // Together they are the heads of one tensor: the upper ones begin whole head strides on.
  const long long head = lo.H > 1 ? lo.st[1] : hi.H > 1 ? hi.st[1] : off;
  if (head > 0 && (hi.H == 1 || hi.st[1] == head) && off % head == 0 && off / head >= lo.H && off / head <= 65535) {
    const int all[3] = {z.B, static_cast<int>(off / head) + hi.H, z.N};
    const long long st[3] = {x.st[0], head, x.st[2]};
    if (disjoint(all, st, 3, z.d, &below)) return false;
  }
  // Or all heads of one token come before those of the next.
  if (off < (lo.H > 1 ? (lo.H - 1) * lo.st[1] : 0) + z.d) return true;
  const long long row = off + (hi.H > 1 ? (hi.H - 1) * hi.st[1] : 0) + z.d;
  const int n[2] = {z.B, z.N};
  const long long st[2] = {x.st[0], x.st[2]};
  return !disjoint(n, st, 2, row, &below);
}

struct Tensors {
  Rows in[6];  // inputs: gradients or x, then (backward) x
  int num_in;
  Rows out[2];
  int num_out;
};

int check_common(const Tensors& t, const Sizes& z, int Hq, int Hk, const double* freqs, const int* positions,
                 int rotary_dim, int pos_mode, int interleaved, float eps, float amplitude, int dtype,
                 int weight_dtype) {
  if (z.B < 1 || z.N < 1 || Hq < 1 || Hk < 0 || freqs == nullptr) return FA2_ERR_INVALID_ARG;
  if (dtype != FA2_FP16 && dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (weight_dtype != dtype && weight_dtype != FA2_FP32) return FA2_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA2_ERR_INVALID_ARG;
  if (pos_mode < 0 || pos_mode > 2 || (pos_mode != 0) != (positions != nullptr)) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(amplitude)) return FA2_ERR_INVALID_ARG;
  if (z.d != 64 && z.d != 128) return FA2_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > z.d || rotary_dim % 16 != 0) return FA2_ERR_UNSUPPORTED;
  if (z.B > 65535 || Hq > 65535 || Hk > 65535) return FA2_ERR_UNSUPPORTED;
  // Work items (at worst four heads of a token each) are numbered in 31 bits.
  const long long chunks = (Hq + 3) / 4 + (Hk + 3) / 4;
  if (static_cast<long long>(z.B) * z.N > kMaxItems / chunks) return FA2_ERR_UNSUPPORTED;
  if (!aligned(freqs, 8) || !aligned(positions, 4)) return FA2_ERR_ALIGNMENT;
  for (int i = 0; i < t.num_in + t.num_out; ++i) {
    const Rows& r = i < t.num_in ? t.in[i] : t.out[i - t.num_in];
    const int st = check_rows(r, z);
    if (st != FA2_OK) return st;
  }
  for (int i = 0; i < t.num_out; ++i) {
    const int n[3] = {z.B, t.out[i].H, z.N};
    long long below = 0;
    if (!disjoint(n, t.out[i].st, 3, z.d, &below)) return FA2_ERR_OVERLAP;
    for (int j = 0; j < t.num_in; ++j)
      if (overlap(t.out[i].p, span(t.out[i], z) * 2, t.in[j].p, span(t.in[j], z) * 2)) return FA2_ERR_OVERLAP;
  }
  if (t.num_out == 2 && outputs_clash(t.out[0], t.out[1], z)) return FA2_ERR_OVERLAP;
  return FA2_OK;
}

fa2::RowView view(const void* p, const long long* st) {
  return fa2::RowView{static_cast<uint16_t*>(const_cast<void*>(p)), st[0], st[1], st[2]};
}

int chunks_of(int H, int chunk) { return (H + chunk - 1) / chunk; }

// Heads per work item of the turn: enough of them to pay for a token's sines, few
// enough to give every SM work.
int turn_chunk(long long tokens, int H, int d) {
  const int groups = fa2::kRotThreads / (d / 16);
  for (int c = 16; c > 4; c /= 2)
    if (tokens * chunks_of(H, c) >= 608LL * groups) return c;
  return 4;
}

void fill(fa2::RotaryArgs& a, const Sizes& z, const double* freqs, const int* positions, int rotary_dim, int pos_mode,
          int interleaved, float eps, float amplitude, int weight_dtype) {
  a.freqs = freqs;
  a.positions = positions;
  a.pos_mode = pos_mode;
  a.B = z.B;
  a.N = z.N;
  a.r = rotary_dim;
  a.interleaved = interleaved;
  a.weight_fp32 = weight_dtype == FA2_FP32;
  a.eps = eps;
  a.amplitude = amplitude;
  a.tokens = static_cast<long long>(z.B) * z.N;
  a.fT = fa2::fast_div(static_cast<int>(a.tokens));
  a.fN = fa2::fast_div(z.N);
}

void set_chunks(fa2::RotaryArgs& a, int chunk) {
  a.chunk = chunk;
  a.chunks_q = chunks_of(a.q.H, chunk);
  a.chunks = a.chunks_q + chunks_of(a.k.H, chunk);
}

// The CTAs of a launch by units, heads of blocks of tokens: a tensor's share is as its heads,
// and each has at least a unit.
fa2::RotarySplit split(long long tokens, int Hq, int Hk, int d) {
  const int groups = fa2::kRotThreads / (d / 16);
  const long long blocks = (tokens + groups - 1) / groups;
  const int share = std::clamp((kRotCtas * Hq + (Hq + Hk) / 2) / (Hq + Hk), 1, Hk > 0 ? kRotCtas - 1 : kRotCtas);
  fa2::RotarySplit s{};
  s.big_q = static_cast<int>(std::min<long long>(share, blocks * Hq));
  s.big_k = static_cast<int>(std::min<long long>(kRotCtas - share, blocks * Hk));
  if (blocks * (Hq + Hk) >= kRotSmall) {
    s.small_q = s.big_q;
    s.small_k = s.big_k;
  }
  return s;
}

// The turn: by units, or by runs of heads (none in the split).
fa2::RotarySplit turn_split(fa2::RotaryArgs& a, int Hq, int Hk, int d, bool norm) {
  const int groups = fa2::kRotThreads / (d / 16);
  const long long units = (a.tokens + groups - 1) / groups * (Hq + Hk);
  if (units >= kRotUnits && (norm || units <= kRotMaxUnits)) return split(a.tokens, Hq, Hk, d);
  set_chunks(a, turn_chunk(a.tokens, Hq + Hk, d));
  return fa2::RotarySplit{};
}

int ctas_of(const fa2::RotarySplit& s) { return s.big_q + s.big_k + s.small_q + s.small_k; }

bool bwd_sizes_ok(int B, int Hq, int Hk, int N, int d) {
  return B >= 1 && N >= 1 && Hq >= 1 && Hk >= 0 && B <= 65535 && Hq <= 65535 && Hk <= 65535 && (d == 64 || d == 128);
}

}  // namespace

extern "C" {

int fa2_rotary_fwd(const void* q, const void* k, const double* freqs, const int* positions, const void* q_weight,
                   const void* k_weight, void* q_out, void* k_out, const long long* strides, int B, int Hq, int Hk,
                   int N, int d, int rotary_dim, int position_mode, int interleaved, float eps, float amplitude,
                   int dtype, int weight_dtype, void* stream) {
  if (!q || !q_out || !strides || (k == nullptr) != (Hk == 0) || (k == nullptr) != (k_out == nullptr))
    return FA2_ERR_INVALID_ARG;
  const bool norm = q_weight != nullptr;
  if ((k_weight != nullptr) != (norm && k != nullptr)) return FA2_ERR_INVALID_ARG;
  const Sizes z{B, N, d};
  Tensors t{};
  t.in[t.num_in++] = {q, strides, Hq};
  if (k) t.in[t.num_in++] = {k, strides + 3, Hk};
  t.out[t.num_out++] = {q_out, strides + 6, Hq};
  if (k) t.out[t.num_out++] = {k_out, strides + 9, Hk};
  int st = check_common(t, z, Hq, Hk, freqs, positions, rotary_dim, position_mode, interleaved, eps, amplitude, dtype,
                        weight_dtype);
  if (st != FA2_OK) return st;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return FA2_ERR_ALIGNMENT;
  const size_t wb = static_cast<size_t>(d) * (weight_dtype == FA2_FP32 ? 4 : 2);
  const size_t pb = static_cast<size_t>(B) * (position_mode == 2 ? N : 1) * 4;
  for (int i = 0; i < t.num_out; ++i) {
    const size_t ob = span(t.out[i], z) * 2;
    if (overlap(t.out[i].p, ob, freqs, static_cast<size_t>(rotary_dim) * 4) ||
        overlap(t.out[i].p, ob, positions, pb) || overlap(t.out[i].p, ob, q_weight, wb) ||
        overlap(t.out[i].p, ob, k_weight, wb))
      return FA2_ERR_OVERLAP;
  }
  int sms = 0, *status = nullptr;
  st = fa2::host_device_setup(&sms, &status);
  if (st != FA2_OK) return st;
  fa2::RotaryArgs a{};
  a.q.x = view(q, strides);
  a.q.y = view(q_out, strides + 6);
  a.q.weight = q_weight;
  a.q.H = Hq;
  if (k) {
    a.k.x = view(k, strides + 3);
    a.k.y = view(k_out, strides + 9);
    a.k.weight = k_weight;
    a.k.H = Hk;
  }
  fill(a, z, freqs, positions, rotary_dim, position_mode, interleaved, eps, amplitude, weight_dtype);
  a.sign = 1.f;
  const fa2::RotarySplit sp = turn_split(a, Hq, Hk, d, norm);
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_rotary(d, dtype == FA2_BF16, norm, a, sp, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

size_t fa2_rotary_bwd_workspace_size(int B, int Hq, int Hk, int N, int d, int norm) {
  if (!bwd_sizes_ok(B, Hq, Hk, N, d)) return 0;
  if (!norm) return 256;
  return static_cast<size_t>(ctas_of(split(static_cast<long long>(B) * N, Hq, Hk, d))) * d * 4;
}

int fa2_rotary_bwd(const void* dq, const void* dk, const void* q, const void* k, const double* freqs,
                   const int* positions, const void* q_weight, const void* k_weight, void* q_grad, void* k_grad,
                   void* q_weight_grad, void* k_weight_grad, const long long* strides, int B, int Hq, int Hk, int N,
                   int d, int rotary_dim, int position_mode, int interleaved, float eps, float amplitude, int dtype,
                   int weight_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dq || !q_grad || !strides || (dk == nullptr) != (Hk == 0) || (dk == nullptr) != (k_grad == nullptr))
    return FA2_ERR_INVALID_ARG;
  const bool norm = q_weight != nullptr, both = dk != nullptr;
  if ((q != nullptr) != norm || (q_weight_grad != nullptr) != norm) return FA2_ERR_INVALID_ARG;
  if ((k != nullptr) != (norm && both) || (k_weight != nullptr) != (norm && both) ||
      (k_weight_grad != nullptr) != (norm && both))
    return FA2_ERR_INVALID_ARG;
  const Sizes z{B, N, d};
  Tensors t{};
  t.in[t.num_in++] = {dq, strides, Hq};
  if (both) t.in[t.num_in++] = {dk, strides + 3, Hk};
  if (norm) t.in[t.num_in++] = {q, strides + 6, Hq};
  if (norm && both) t.in[t.num_in++] = {k, strides + 9, Hk};
  t.out[t.num_out++] = {q_grad, strides + 12, Hq};
  if (both) t.out[t.num_out++] = {k_grad, strides + 15, Hk};
  int st = check_common(t, z, Hq, Hk, freqs, positions, rotary_dim, position_mode, interleaved, eps, amplitude, dtype,
                        weight_dtype);
  if (st != FA2_OK) return st;
  const void* small[] = {q_weight, k_weight, q_weight_grad, k_weight_grad};
  for (const void* p : small)
    if (!aligned(p, 16)) return FA2_ERR_ALIGNMENT;
  const size_t need = norm ? fa2_rotary_bwd_workspace_size(B, Hq, Hk, N, d, 1) : 0;
  if (norm) {
    if (workspace == nullptr || workspace_bytes < need) return FA2_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  }
  const size_t wb = static_cast<size_t>(d) * (weight_dtype == FA2_FP32 ? 4 : 2);
  const size_t pb = static_cast<size_t>(B) * (position_mode == 2 ? N : 1) * 4;
  // Outputs other than the strided ones, against everything and each other.
  const struct {
    const void* p;
    size_t n;
  } outs[] = {{t.out[0].p, static_cast<size_t>(span(t.out[0], z)) * 2},
              {both ? t.out[1].p : nullptr, both ? static_cast<size_t>(span(t.out[1], z)) * 2 : 0},
              {q_weight_grad, wb},
              {k_weight_grad, wb},
              {norm ? workspace : nullptr, need}};
  for (int i = 0; i < 5; ++i) {
    if (overlap(outs[i].p, outs[i].n, freqs, static_cast<size_t>(rotary_dim) * 4) ||
        overlap(outs[i].p, outs[i].n, positions, pb) || overlap(outs[i].p, outs[i].n, q_weight, wb) ||
        overlap(outs[i].p, outs[i].n, k_weight, wb))
      return FA2_ERR_OVERLAP;
    if (i < 2) continue;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return FA2_ERR_OVERLAP;
    for (int j = 0; j < t.num_in; ++j)
      if (overlap(outs[i].p, outs[i].n, t.in[j].p, span(t.in[j], z) * 2)) return FA2_ERR_OVERLAP;
  }
  int sms = 0, *status = nullptr;
  st = fa2::host_device_setup(&sms, &status);
  if (st != FA2_OK) return st;
  fa2::RotaryArgs a{};
  a.q.x = view(dq, strides);
  a.q.y = view(q_grad, strides + 12);
  a.q.H = Hq;
  if (both) {
    a.k.x = view(dk, strides + 3);
    a.k.y = view(k_grad, strides + 15);
    a.k.H = Hk;
  }
  if (norm) {
    a.q.src = view(q, strides + 6);
    a.q.weight = q_weight;
    a.q.weight_grad = q_weight_grad;
    if (both) {
      a.k.src = view(k, strides + 9);
      a.k.weight = k_weight;
      a.k.weight_grad = k_weight_grad;
    }
  }
  fill(a, z, freqs, positions, rotary_dim, position_mode, interleaved, eps, amplitude, weight_dtype);
  a.sign = -1.f;
  (void)cudaGetLastError();
  cudaError_t e;
  if (norm) {
    a.part = static_cast<float*>(workspace);
    e = fa2::launch_rotary_norm_bwd(d, dtype == FA2_BF16, a, split(a.tokens, Hq, Hk, d), static_cast<cudaStream_t>(stream));
  } else {
    const fa2::RotarySplit sp = turn_split(a, Hq, Hk, d, false);
    e = fa2::launch_rotary(d, dtype == FA2_BF16, false, a, sp, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

}  // extern "C"
