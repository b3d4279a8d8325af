// C ABI of the paged key-value cache and of the key weights: argument
// validation, workspace layout and launches. Declarations and argument
// contracts live in include/fa2.h.
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa2.h"
#include "fa2_cache.cuh"
#include "fa2_host.h"

namespace fa2 {
cudaError_t launch_paged_decode(int d, bool bf16, int head_tile, const DecodeArgs& a, int ctas,
                                cudaStream_t stream);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream);
cudaError_t launch_key_weights(int d, bool bf16, bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                               const KeyWeightArgs& a, int ctas, cudaStream_t stream);
}  // namespace fa2

namespace {

constexpr int kDecodeCtas = 304;  // most CTAs of a decode: two on each of 152 SMs
constexpr int kKwCtas = 152;      // most CTAs of the key weights
constexpr long long kMaxRows = (1LL << 31) - 1;
constexpr long long kMaxSlots = 1LL << 30;  // slots that a table row can name

struct Buf {
  const void* p;
  size_t n;
};

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool overlap(const Buf& a, const Buf& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// No output may share bytes with an input or with another output.
template <int NO, int NI>
bool any_overlap(const Buf (&outs)[NO], const Buf (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

int check_cache(int B, int Hkv, int d, int num_pages, int page_size, int max_pages, int dtype) {
  if (B < 1 || Hkv < 1 || num_pages < 1 || page_size < 1 || max_pages < 1) return FA2_ERR_INVALID_ARG;
  if (dtype != FA2_FP16 && dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return FA2_ERR_UNSUPPORTED;
  // Rows of the cache are numbered in 31 bits; elements in 64.
  if (static_cast<long long>(num_pages) * Hkv > kMaxRows ||
      static_cast<long long>(num_pages) * Hkv * page_size > kMaxRows)
    return FA2_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > kMaxSlots) return FA2_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv > kMaxRows / 16) return FA2_ERR_UNSUPPORTED;
  return FA2_OK;
}

fa2::CacheView make_view(const int* table, const int* lens, int B, int Hkv, int num_pages, int page_size,
                         int max_pages) {
  fa2::CacheView c{};
  c.table = table;
  c.lens = lens;
  c.B = B;
  c.Hkv = Hkv;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  c.L = max_pages * page_size;
  c.ps = fa2::fast_div(page_size);
  return c;
}

size_t cache_bytes(int Hkv, int d, int num_pages, int page_size) {
  return static_cast<size_t>(num_pages) * Hkv * page_size * d * 2;
}
size_t slot_bytes(int B, int Hkv, int page_size, int max_pages) {
  return static_cast<size_t>(B) * Hkv * page_size * max_pages * 4;
}

// Query heads that one item of the decode carries: 8 fill the short side of
// its products; 16 read a group's keys half as often, and cost registers and
// products that a group of 8 would leave empty. B = 8, 8000 slots, d = 128, bf16:
// 16 heads to a key head 22.9 us with tiles of 16 and 32.2 with tiles of 8, 9 heads
// 29.0 and 35.6, 32 heads 22.5 and 29.7, 128 heads 51 and 71; at d = 64 15.9 and
// 19.0, 18.8 and 21.3, 14.9 and 17.7, 29.5 and 38.9. With weights the same, but for
// 128 heads at d = 64 (205 and 197).
int head_tile(int g) { return g <= 8 ? 8 : 16; }

// Most CTAs that a decode can use: one per unit of a full table.
int decode_ctas(int B, int Hq, int Hkv, int d, int page_size, int max_pages) {
  const int g = Hq / Hkv, unit = fa2::decode_unit(d);
  const long long L = static_cast<long long>(page_size) * max_pages;
  const long long items = static_cast<long long>(B) * Hkv * ((g + head_tile(g) - 1) / head_tile(g));
  const long long units = items * ((L + unit - 1) / unit);
  return units < kDecodeCtas ? static_cast<int>(units) : kDecodeCtas;
}

// Whether a decode gives each CTA a whole item instead of an equal share of all.
// It saves the join and the merges at cut ends, and costs where a CTA's one item
// takes longer than its share would: with few items, with a last wave of CTAs
// that leaves most of the `slots` CTAs that run at once idle, with uneven
// lengths. Four units (256 slots at d = 128, 512 at d = 64) take 6.1 us whole
// and 6.1 split for 8 items, 9.2 and 15.1 for 256; eight units 9.6 and 6.1 for 8
// items, 11.7 and 14.5 for 128, 14.0 and 19.3 for 256, 22.9 and 22.5 for 320 (d =
// 128). The table's width decides, lengths being known on the device only: the
// same 256 items of 256 slots in a table of 8192 are split, 14.9 us.
// With weights a CTA has to have all heads of its key head.
bool decode_whole(int B, int Hkv, int d, int page_size, int max_pages, int HG, int slots, bool weights) {
  const long long unit = fa2::decode_unit(d), units = (static_cast<long long>(page_size) * max_pages + unit - 1) / unit;
  const long long items = static_cast<long long>(B) * Hkv * HG, waves = (items + slots - 1) / slots;
  if (weights && HG > 1) return false;
  const bool filled = waves == 1 ? 5 * items >= 2 * slots : 5 * items >= 4 * waves * slots;
  return units <= (filled ? 8 : 4);
}

// Workspace of the decode: partial O and (m, l) of cut items, then the logits.
struct DecodeSpace {
  size_t o, ml, logits, total;
};
DecodeSpace decode_space(int B, int Hq, int Hkv, int d, int page_size, int max_pages, bool weights) {
  DecodeSpace s{};
  const size_t parts = static_cast<size_t>(2) * decode_ctas(B, Hq, Hkv, d, page_size, max_pages) * head_tile(Hq / Hkv);
  s.o = 0;
  s.ml = align_up(parts * d * 4, 256);
  s.logits = s.ml + align_up(parts * 8, 256);
  s.total = s.logits + (weights ? align_up(slot_bytes(B, Hq, page_size, max_pages), 256) : 0);
  return s;
}

// Longest list of moves of an eviction: slots below the budget, or past it.
long long evict_list(int page_size, int max_pages, int budget) {
  const long long past = static_cast<long long>(max_pages) * page_size - budget;
  return past <= 0 ? 0 : past < budget ? past : budget;
}

int check_heads(int Hq, int Hkv) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA2_ERR_INVALID_ARG;
  if (Hq > 65535 || Hq / Hkv > fa2::kMaxGroup) return FA2_ERR_UNSUPPORTED;
  return FA2_OK;
}

}  // namespace

extern "C" {

size_t fa2_paged_decode_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                                       int weights) {
  if (check_heads(Hq, Hkv) != FA2_OK) return 0;
  if (check_cache(B, Hkv, d, 1, page_size, max_pages, FA2_BF16) != FA2_OK) return 0;
  return decode_space(B, Hq, Hkv, d, page_size, max_pages, weights != 0).total;
}

int fa2_paged_decode(const void* q, const void* k_cache, const void* v_cache, const int* table,
                     const int* lens, const float* weights, float* weights_out, void* o, float* lse, int B,
                     int Hq, int Hkv, int d, int num_pages, int page_size, int max_pages, float scale,
                     int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !table || !lens || !o || !lse) return FA2_ERR_INVALID_ARG;
  if ((weights == nullptr) != (weights_out == nullptr)) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  int st = check_heads(Hq, Hkv);
  if (st != FA2_OK) return st;
  st = check_cache(B, Hkv, d, num_pages, page_size, max_pages, dtype);
  if (st != FA2_OK) return st;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4) || !aligned(weights, 4) ||
      !aligned(weights_out, 4))
    return FA2_ERR_ALIGNMENT;
  const DecodeSpace s = decode_space(B, Hq, Hkv, d, page_size, max_pages, weights != nullptr);
  if (workspace == nullptr || workspace_bytes < s.total) return FA2_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  const size_t qb = static_cast<size_t>(B) * Hq * d * 2, cb = cache_bytes(Hkv, d, num_pages, page_size);
  const size_t wb = slot_bytes(B, Hkv, page_size, max_pages);
  const Buf ins[] = {{q, qb}, {k_cache, cb}, {v_cache, cb},
                     {table, static_cast<size_t>(B) * max_pages * 4}, {lens, static_cast<size_t>(B) * 4},
                     {weights == weights_out ? nullptr : weights, wb}};
  const Buf outs[] = {{o, qb}, {lse, static_cast<size_t>(B) * Hq * 4}, {weights_out, wb}, {workspace, s.total}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::DecodeArgs a{};
  a.c = make_view(table, lens, B, Hkv, num_pages, page_size, max_pages);
  st = fa2::host_device_setup(&sms, &a.c.status);
  if (st != FA2_OK) return st;
  char* ws = static_cast<char*>(workspace);
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_cache);
  a.v = static_cast<const uint16_t*>(v_cache);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.w_in = weights;
  a.w_out = weights_out;
  a.part_o = reinterpret_cast<float*>(ws + s.o);
  a.part_ml = reinterpret_cast<float2*>(ws + s.ml);
  a.logits = reinterpret_cast<float*>(ws + s.logits);
  a.Hq = Hq;
  a.g = Hq / Hkv;
  const int ht = head_tile(a.g);
  a.HG = (a.g + ht - 1) / ht;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const int most = decode_ctas(B, Hq, Hkv, d, page_size, max_pages), ctas = 2 * sms < most ? 2 * sms : most;
  a.whole = decode_whole(B, Hkv, d, page_size, max_pages, a.HG, 2 * sms, weights != nullptr);
  (void)cudaGetLastError();  // a non-sticky error of another caller is not ours
  const cudaError_t e =
      fa2::launch_paged_decode(d, dtype == FA2_BF16, ht, a, ctas, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

int fa2_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, const int* table,
                     const int* lens, const int* num_new, float* weights, const float* new_weights,
                     int* positions, const int* next_pos, int* lens_out, int B, int Hkv, int T, int d,
                     int num_pages, int page_size, int max_pages, int dtype, void* stream) {
  if (!k || !v || !k_cache || !v_cache || !table || !lens || !lens_out) return FA2_ERR_INVALID_ARG;
  if (T < 1 || (weights == nullptr && new_weights != nullptr) || (positions == nullptr) != (next_pos == nullptr))
    return FA2_ERR_INVALID_ARG;
  int st = check_cache(B, Hkv, d, num_pages, page_size, max_pages, dtype);
  if (st != FA2_OK) return st;
  const long long rows = static_cast<long long>(B) * Hkv * T;
  if (rows > kMaxRows) return FA2_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(num_new, 4) || !aligned(weights, 4) ||
      !aligned(new_weights, 4) || !aligned(positions, 4) || !aligned(next_pos, 4) || !aligned(lens_out, 4))
    return FA2_ERR_ALIGNMENT;
  const size_t nb = static_cast<size_t>(rows) * d * 2, cb = cache_bytes(Hkv, d, num_pages, page_size);
  const size_t wb = slot_bytes(B, Hkv, page_size, max_pages), lb = static_cast<size_t>(B) * 4;
  const Buf ins[] = {{k, nb}, {v, nb}, {table, static_cast<size_t>(B) * max_pages * 4}, {lens, lb},
                     {num_new, lb}, {new_weights, static_cast<size_t>(rows) * 4}, {next_pos, lb}};
  const Buf outs[] = {{k_cache, cb}, {v_cache, cb}, {weights, wb}, {positions, wb}, {lens_out, lb}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::AppendArgs a{};
  a.c = make_view(table, lens, B, Hkv, num_pages, page_size, max_pages);
  st = fa2::host_device_setup(&sms, &a.c.status);
  if (st != FA2_OK) return st;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.kc = static_cast<uint16_t*>(k_cache);
  a.vc = static_cast<uint16_t*>(v_cache);
  a.num_new = num_new;
  a.weights = weights;
  a.new_weights = new_weights;
  a.positions = positions;
  a.next_pos = next_pos;
  a.lens_out = lens_out;
  a.T = T;
  a.d = d;
  a.fT = fa2::fast_div(T);
  a.fH = fa2::fast_div(Hkv);
  a.rows = rows;
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_cache_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

size_t fa2_cache_evict_workspace_size(int B, int Hkv, int page_size, int max_pages, int budget) {
  if (check_cache(B, Hkv, 64, 1, page_size, max_pages, FA2_BF16) != FA2_OK || budget < 1) return 0;
  const long long list = evict_list(page_size, max_pages, budget);
  if (fa2::move_ctas(static_cast<long long>(B) * Hkv, list) > kMaxRows) return 0;
  return 2 * align_up(static_cast<size_t>(B) * Hkv * list * 4, 256) + align_up(static_cast<size_t>(B) * Hkv * 4, 256);
}

int fa2_cache_evict(void* k_cache, void* v_cache, const int* table, const int* lens, const float* weights,
                    float* weights_out, const int* positions, int* positions_out, const int* next_pos,
                    int* lens_out, int B, int Hkv, int d, int num_pages, int page_size, int max_pages,
                    int budget, int recent, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!k_cache || !v_cache || !table || !lens || !weights || !weights_out || !lens_out)
    return FA2_ERR_INVALID_ARG;
  if ((positions == nullptr) != (positions_out == nullptr) || (positions == nullptr) != (next_pos == nullptr))
    return FA2_ERR_INVALID_ARG;
  if (budget < 1 || recent < 0 || recent > budget) return FA2_ERR_INVALID_ARG;
  int st = check_cache(B, Hkv, d, num_pages, page_size, max_pages, dtype);
  if (st != FA2_OK) return st;
  const long long list = evict_list(page_size, max_pages, budget);
  if (fa2::move_ctas(static_cast<long long>(B) * Hkv, list) > kMaxRows) return FA2_ERR_UNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(positions, 4) ||
      !aligned(positions_out, 4) || !aligned(next_pos, 4) || !aligned(lens_out, 4))
    return FA2_ERR_ALIGNMENT;
  const size_t need = fa2_cache_evict_workspace_size(B, Hkv, page_size, max_pages, budget);
  if (workspace == nullptr || workspace_bytes < need) return FA2_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  const size_t cb = cache_bytes(Hkv, d, num_pages, page_size), lb = static_cast<size_t>(B) * 4;
  const size_t wb = slot_bytes(B, Hkv, page_size, max_pages);
  const Buf ins[] = {{table, static_cast<size_t>(B) * max_pages * 4}, {lens, lb},
                     {weights == weights_out ? nullptr : weights, wb},
                     {positions == positions_out ? nullptr : positions, wb}, {next_pos, lb}};
  const Buf outs[] = {{k_cache, cb}, {v_cache, cb}, {weights_out, wb}, {positions_out, wb}, {lens_out, lb},
                      {workspace, need}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::EvictArgs a{};
  a.c = make_view(table, lens, B, Hkv, num_pages, page_size, max_pages);
  st = fa2::host_device_setup(&sms, &a.c.status);
  if (st != FA2_OK) return st;
  a.kc = static_cast<uint16_t*>(k_cache);
  a.vc = static_cast<uint16_t*>(v_cache);
  a.w_in = weights;
  a.w_out = weights_out;
  a.p_in = positions;
  a.p_out = positions_out;
  a.next_pos = next_pos;
  a.lens_out = lens_out;
  a.list = static_cast<int>(list);
  const size_t lists = align_up(static_cast<size_t>(B) * Hkv * a.list * 4, 256);
  a.holes = static_cast<int*>(workspace);
  a.movers = reinterpret_cast<int*>(static_cast<char*>(workspace) + lists);
  a.counts = reinterpret_cast<int*>(static_cast<char*>(workspace) + 2 * lists);
  a.budget = budget;
  a.recent = recent;
  a.d = d;
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_cache_evict(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

size_t fa2_key_weights_workspace_size(void) { return static_cast<size_t>(2) * kKwCtas * 256 * 4; }

int fa2_key_weights(const void* q, const void* k, const float* lse, const int* q_lens, float* out, int B,
                    int Hq, int Hkv, int N, int Nk, int d, int causal, float scale, int dtype, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!q || !k || !lse || !out) return FA2_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Nk < 1 || (causal != 0 && causal != 1)) return FA2_ERR_INVALID_ARG;
  if (dtype != FA2_FP16 && dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  int st = check_heads(Hq, Hkv);
  if (st != FA2_OK) return st;
  if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
  if (B > 65535) return FA2_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hq * (static_cast<long long>(N) + 127) > kMaxRows ||
      static_cast<long long>(B) * Hkv * (static_cast<long long>(Nk) + 255) > kMaxRows)
    return FA2_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 4) || !aligned(q_lens, 4) || !aligned(out, 4))
    return FA2_ERR_ALIGNMENT;
  const size_t need = fa2_key_weights_workspace_size();
  if (workspace == nullptr || workspace_bytes < need) return FA2_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  const Buf ins[] = {{q, static_cast<size_t>(B) * Hq * N * d * 2}, {k, static_cast<size_t>(B) * Hkv * Nk * d * 2},
                     {lse, static_cast<size_t>(B) * Hq * N * 4}, {q_lens, static_cast<size_t>(B) * 4}};
  const Buf outs[] = {{out, static_cast<size_t>(B) * Hkv * Nk * 4}, {workspace, need}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::KeyWeightArgs a{};
  st = fa2::host_device_setup(&sms, &a.status);
  if (st != FA2_OK) return st;
  CUtensorMap tq, tk;
  if (fa2::host_map_16bit(&tq, q, B * Hq, N, d, dtype) || fa2::host_map_16bit(&tk, k, B * Hkv, Nk, d, dtype))
    return FA2_ERR_CUDA;
  a.lse = lse;
  a.q_lens = q_lens;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.g = Hq / Hkv;
  a.N = N;
  a.Nk = Nk;
  a.nkb = (Nk + 255) / 256;
  // The forward's factor, rounded as it is there: with the L that the forward makes
  // of its scores the weights of a query sum to 1.
  a.scale_log2 = scale * 1.4426950408889634f;
  a.timeout_ns = fa2::kDefaultWaitTimeoutNs;
  a.fault = fa2::host_take_fault(6, &a.timeout_ns);
  const int ctas = sms < kKwCtas ? sms : kKwCtas;
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_key_weights(d, dtype == FA2_BF16, causal != 0, tq, tk, a, ctas,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA2_OK : fa2::host_cuda_fail(e);
}

}  // extern "C"
