// C ABI of the paged key-value cache and of the key weights: argument
// validation, workspace layout and launches. Declarations and argument
// contracts live in include/fa2.h.
#include <algorithm>
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
cudaError_t launch_prefix_decode(int d, bool bf16, const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                                 cudaStream_t stream);
cudaError_t launch_cache_resize(const ResizeArgs& a, cudaStream_t stream);
int resize_group(int B);
cudaError_t launch_key_weights(int d, bool bf16, bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                               const KeyWeightArgs& a, int ctas, cudaStream_t stream);
}  // namespace fa2

namespace {

constexpr int kDecodeCtas = 304;  // most CTAs of a decode: two on each of 152 SMs
constexpr int kDecodeWarps = 4;   // workers of a CTA, behind a shared prefix
constexpr int kPrefixCtas = 152;  // most CTAs of a shared prefix
constexpr int kKwCtas = 152;      // most CTAs of the key weights
constexpr long long kMaxRows = (1LL << 31) - 1;
constexpr long long kMaxSlots = 1LL << 30;  // slots that a table row can name
// Entries of a table that a resize can change: it numbers its releases and takes in 31
// bits, and a number may pass their count by a step of its loops, 16 CTAs x 512 threads.
constexpr long long kMaxEntries = (1LL << 31) - (1 << 14);

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

// Whether the prefix is attended to by the kernel of the own slots, in items of 8 or 16
// of the rows = B g query rows of a key head. That saves a launch and the other kernel's
// start, but reads and multiplies the prefix once for each 16 rows; one such tile is read
// once anyway. (32/8 heads, d = 128, inside and outside: 2000 slots, 48 rows 17.0 and 19.7
// us, 64 rows 17.6 and 19.7, 96 rows 22.0 and 21.3; 512 slots, 128 rows 15.3 and 16.3, 192
// rows 18.7 and 17.4; 8192 slots, 32 rows 23.6 and 24.0, 48 rows 28.2 and 22.7. Two heads
// of 16384 slots, d = 64, 32 rows 13.7 and 14.0, 128 rows 26.0 and 17.9.) The list's room
// decides, the prefix's length being known on the device only.
bool prefix_inside(int B, int Hq, int Hkv, int d, long long prefix_cap) {
  const long long rows = static_cast<long long>(B) * (Hq / Hkv), tiles = (rows + 15) / 16;
  return tiles == 1 || (tiles <= 8 && tiles * Hkv * prefix_cap <= 65536LL * 128 / d);
}
// Whether the workers of the own slots (and of a prefix inside) are warps: from 96 items
// on. By CTAs and by warps: 40 items (32/8 heads, 2000 slots and 300 own, d = 128) 12.4 and
// 16.4 us, 80 items 15.5 and 15.8, 120 items 19.1 and 17.1; 68 items (2 heads, 16384 slots,
// d = 64) 13.7 and 14.9; 384 items (32 heads, 4096 slots) 33.1 and 25.1.
bool prefix_by_warps(long long items) { return items >= 96; }
int prefix_head_tile(int B, int Hq, int Hkv, bool inside) {
  return inside && static_cast<long long>(B) * (Hq / Hkv) > 8 ? 16 : head_tile(Hq / Hkv);
}

// Items of a shared prefix: up to 256 of the B * g query rows of a key head.
long long prefix_items(int B, int Hq, int Hkv) {
  return static_cast<long long>(Hkv) * ((static_cast<long long>(B) * (Hq / Hkv) + 255) / 256);
}

// Workspace of a decode with a shared prefix: the parts of both kernels, and where
// each sequence's units begin.
struct PrefixSpace {
  size_t po, pml, so, sml, starts, total;
};
PrefixSpace prefix_space(int B, int Hq, int Hkv, int d) {
  PrefixSpace s{};
  const int g = Hq / Hkv;
  // Whichever kernel attends to the prefix.
  const size_t rows = B * g <= 16 ? 0 : static_cast<size_t>(prefix_items(B, Hq, Hkv) + kPrefixCtas) * 256;
  size_t own = 0;
  for (const bool inside : {false, true}) {
    const size_t ht = prefix_head_tile(B, Hq, Hkv, inside);
    const size_t items = static_cast<size_t>(B) * Hkv * ((g + ht - 1) / ht) +
                         (inside ? Hkv * ((static_cast<size_t>(B) * g + ht - 1) / ht) : 0);
    own = std::max(own, (items + kDecodeCtas * kDecodeWarps) * ht);
  }
  s.pml = s.po + align_up(rows * d * 4, 256);
  s.so = s.pml + align_up(rows * 8, 256);
  s.sml = s.so + align_up(own * d * 4, 256);
  s.starts = s.sml + align_up(own * 8, 256);
  s.total = s.starts + align_up(static_cast<size_t>(B + 3) * 8, 256);
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

size_t fa2_prefix_decode_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages) {
  if (check_heads(Hq, Hkv) != FA2_OK) return 0;
  if (check_cache(B, Hkv, d, 1, page_size, max_pages, FA2_BF16) != FA2_OK) return 0;
  return prefix_space(B, Hq, Hkv, d).total;
}

int fa2_prefix_decode(const void* q, const void* k_cache, const void* v_cache, const int* table, const int* lens,
                      const int* prefix, const int* prefix_len, void* o, float* lse, int B, int Hq, int Hkv, int d,
                      int num_pages, int page_size, int max_pages, int prefix_pages, float scale, int dtype,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !table || !lens || !prefix || !prefix_len || !o || !lse) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f) || prefix_pages < 1) return FA2_ERR_INVALID_ARG;
  int st = check_heads(Hq, Hkv);
  if (st != FA2_OK) return st;
  st = check_cache(B, Hkv, d, num_pages, page_size, max_pages, dtype);
  if (st != FA2_OK) return st;
  if (static_cast<long long>(prefix_pages) * page_size > kMaxSlots) return FA2_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(table, 4) ||
      !aligned(lens, 4) || !aligned(prefix, 4) || !aligned(prefix_len, 4) || !aligned(lse, 4))
    return FA2_ERR_ALIGNMENT;
  const PrefixSpace s = prefix_space(B, Hq, Hkv, d);
  if (workspace == nullptr || workspace_bytes < s.total) return FA2_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  const size_t qb = static_cast<size_t>(B) * Hq * d * 2, cb = cache_bytes(Hkv, d, num_pages, page_size);
  const Buf ins[] = {{q, qb}, {k_cache, cb}, {v_cache, cb}, {table, static_cast<size_t>(B) * max_pages * 4},
                     {lens, static_cast<size_t>(B) * 4}, {prefix, static_cast<size_t>(prefix_pages) * 4}, {prefix_len, 4}};
  const Buf outs[] = {{o, qb}, {lse, static_cast<size_t>(B) * Hq * 4}, {workspace, s.total}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::PrefixArgs a{};
  fa2::DecodeArgs& c = a.d;
  c.c = make_view(table, lens, B, Hkv, num_pages, page_size, max_pages);
  st = fa2::host_device_setup(&sms, &c.c.status);
  if (st != FA2_OK) return st;
  c.box = 1;
  while (c.box < 16 && page_size % (2 * c.box) == 0) c.box *= 2;
  c.prefix_cap = prefix_pages * page_size;
  const bool inside = prefix_inside(B, Hq, Hkv, d, c.prefix_cap);
  CUtensorMap tk{}, tv{};
  const int rows = num_pages * Hkv * page_size;
  if (!inside && (fa2::host_map_rows(&tk, k_cache, rows, d, dtype, c.box) ||
                  fa2::host_map_rows(&tv, v_cache, rows, d, dtype, c.box)))
    return FA2_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  c.q = static_cast<const uint16_t*>(q);
  c.k = static_cast<const uint16_t*>(k_cache);
  c.v = static_cast<const uint16_t*>(v_cache);
  c.o = static_cast<uint16_t*>(o);
  c.lse = lse;
  c.part_o = reinterpret_cast<float*>(ws + s.so);
  c.part_ml = reinterpret_cast<float2*>(ws + s.sml);
  c.starts = reinterpret_cast<long long*>(ws + s.starts);
  c.Hq = Hq;
  c.g = Hq / Hkv;
  a.head_tile = prefix_head_tile(B, Hq, Hkv, inside);
  c.HG = (c.g + a.head_tile - 1) / a.head_tile;
  c.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  c.prefix = prefix;
  c.prefix_len = prefix_len;
  c.rows = B * c.g;
  c.fg = fa2::fast_div(c.g);
  long long items = static_cast<long long>(B) * Hkv * c.HG;
  if (inside) {
    c.row_tiles = (c.rows + a.head_tile - 1) / a.head_tile;
    c.ft = fa2::fast_div(c.row_tiles);
    items += static_cast<long long>(Hkv) * c.row_tiles;
  } else {
    a.items = static_cast<int>(prefix_items(B, Hq, Hkv));
    a.fblocks = fa2::fast_div(a.items / Hkv);
    a.ctas = static_cast<int>(std::min<long long>(a.items * ((static_cast<long long>(c.prefix_cap) + 127) / 128),
                                                  std::min(sms, kPrefixCtas)));
  }
  a.tail_warps = prefix_by_warps(items);
  // At most one CTA per unit of full tables.
  const long long longest = std::max(static_cast<long long>(c.c.L), inside ? static_cast<long long>(c.prefix_cap) : 0LL);
  const long long units = items * ((longest + fa2::decode_unit(d) - 1) / fa2::decode_unit(d));
  a.tail_ctas = static_cast<int>(std::min<long long>(units, std::min(2 * sms, kDecodeCtas)));
  // By warps half of the CTAs begin beside the prefix's; by CTAs (115200 bytes of shared
  // memory at d = 128, where 68608 of an SM's are left) none has room there, and uneven
  // shares help or harm by chance: 64 sequences, 8/1 heads, 8192 slots and up to 1024 (4000)
  // own ones 26.7 us (35.3) even and 27.2 (36.8) uneven; 20 of 64/4 heads 40.2 and 42.1; 40
  // of 16/2 heads the other way, 29.6 and 28.2.
  if (!inside && a.tail_warps && a.tail_ctas == 2 * sms) {
    c.early = sms;
    c.prefix_items = a.items;
  }
  a.part_o = reinterpret_cast<float*>(ws + s.po);
  a.part_ml = reinterpret_cast<float2*>(ws + s.pml);
  a.timeout_ns = fa2::kDefaultWaitTimeoutNs;
  if (!inside) a.fault = fa2::host_take_fault(7, &a.timeout_ns);
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_prefix_decode(d, dtype == FA2_BF16, tk, tv, a, static_cast<cudaStream_t>(stream));
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

size_t fa2_cache_resize_workspace_size(int B, int num_pages, int page_size, int max_pages) {
  if (check_cache(B, 1, 64, 1, page_size, max_pages, FA2_BF16) != FA2_OK || num_pages < 1) return 0;
  if (static_cast<long long>(B) * max_pages > kMaxEntries) return 0;
  return align_up(static_cast<size_t>(num_pages) * 4, 256) + align_up(static_cast<size_t>(B) * max_pages * 4, 256);
}

int fa2_cache_resize(int* table, const int* lens, const int* new_lens, int* refs, int* free_pages, int* num_free,
                     int* lens_out, int B, int num_pages, int page_size, int max_pages, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!table || !lens || !new_lens || !refs || !free_pages || !num_free || !lens_out) return FA2_ERR_INVALID_ARG;
  if (num_pages < 1) return FA2_ERR_INVALID_ARG;
  int st = check_cache(B, 1, 64, 1, page_size, max_pages, FA2_BF16);
  if (st != FA2_OK) return st;
  if (static_cast<long long>(B) * max_pages > kMaxEntries) return FA2_ERR_UNSUPPORTED;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(new_lens, 4) || !aligned(refs, 4) ||
      !aligned(free_pages, 4) || !aligned(num_free, 4) || !aligned(lens_out, 4))
    return FA2_ERR_ALIGNMENT;
  const size_t need = fa2_cache_resize_workspace_size(B, num_pages, page_size, max_pages);
  if (workspace == nullptr || workspace_bytes < need) return FA2_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA2_ERR_ALIGNMENT;
  const size_t lb = static_cast<size_t>(B) * 4, pb = static_cast<size_t>(num_pages) * 4;
  const Buf ins[] = {{lens, lb}, {new_lens, lb}};
  const Buf outs[] = {{table, static_cast<size_t>(B) * max_pages * 4}, {refs, pb}, {free_pages, pb}, {num_free, 4},
                      {lens_out, lb}, {workspace, need}};
  if (any_overlap(outs, ins)) return FA2_ERR_OVERLAP;
  int sms = 0;
  fa2::ResizeArgs a{};
  st = fa2::host_device_setup(&sms, &a.status);
  if (st != FA2_OK) return st;
  a.table = table;
  a.lens = lens;
  a.new_lens = new_lens;
  a.refs = refs;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.lens_out = lens_out;
  a.owner = static_cast<int*>(workspace);
  a.gone = reinterpret_cast<int*>(static_cast<char*>(workspace) + align_up(pb, 256));
  a.B = B;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.L = max_pages * page_size;
  a.group = fa2::resize_group(B);
  a.ps = fa2::fast_div(page_size);
  (void)cudaGetLastError();
  const cudaError_t e = fa2::launch_cache_resize(a, static_cast<cudaStream_t>(stream));
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
