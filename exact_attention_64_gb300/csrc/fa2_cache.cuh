// The paged key-value cache: where a slot of a sequence lies, and small
// pieces that the cache's kernels share.
//
// A cache is [num_pages][Hkv][page_size][d] of 16-bit floats, one for K and one
// for V. Slot j of sequence b and key head h is row
//   (table[b][j / page_size] * Hkv + h) * page_size + j % page_size
// of the cache seen as rows of d elements. A page holds all heads of its slots,
// each head's slots contiguous, so a head of a page is one run of
// page_size * d * 2 bytes. A sequence has lens[b] slots in use, of at most
// L = max_pages * page_size.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>
#include "sm103_ptx.cuh"

namespace fa2 {

constexpr int kDevPage = 9;     // equals FA2_ERR_PAGE of the public header
constexpr int kMaxGroup = 128;  // query heads per key head

// Division of 0 <= n < 2^31 by a run-time d >= 1 as one multiplication: with
// s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1, n / d = (n m) >> (31 + s),
// since m d exceeds 2^(31+s) by at most d <= 2^s (division by invariant
// integers, Granlund and Montgomery 1994).
struct FastDiv {
  unsigned long long m;
  int s;
  int d;
};

inline FastDiv fast_div(int d) {
  FastDiv f;
  f.d = d;
  f.s = 0;
  while ((1LL << f.s) < d) ++f.s;
  f.m = (1ull << (31 + f.s)) / static_cast<unsigned long long>(d) + 1;
  f.s += 31;
  return f;
}

__device__ __forceinline__ int div_by(int n, const FastDiv& f) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(n)) * f.m) >> f.s);
}

// A plain load. `ld.global.nc` (__ldg) promises that nothing writes there while
// the kernel exists, and a kernel launched early exists before its inputs do.
template <class T>
__device__ __forceinline__ T ld_global(const T* p) {
  return *p;
}

struct CacheView {
  const int* table;  // [B][max_pages]
  const int* lens;   // [B]
  int B, Hkv;
  int num_pages, max_pages;
  int L;             // max_pages * page_size
  FastDiv ps;        // page size
  int* status;
};

// A length or a page that the cache does not have is never followed: the
// length is cut to what the table can hold, the page's slots are left out, and
// the status word says so, unless it holds a wait that ran out: bad lengths can be
// what that left behind.
__device__ __forceinline__ void report_page(int* status) { atomicCAS(status, kDevOk, kDevPage); }

__device__ __forceinline__ int cut_len(int n, int L) { return min(max(n, 0), L); }

__device__ __forceinline__ int seq_len(const CacheView& c, int b) { return cut_len(ld_global(c.lens + b), c.L); }

// Row of slot j (0 <= j < L) given its page number, or -1 for a bad page. Rows
// are below 2^31 (checked by the host).
__device__ __forceinline__ int page_row(const CacheView& c, int page, int h, int off) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages)
             ? (page * c.Hkv + h) * c.ps.d + off
             : -1;
}
__device__ __forceinline__ int slot_row(const CacheView& c, int b, int h, int j) {
  const int p = div_by(j, c.ps);
  const int page = ld_global(c.table + static_cast<size_t>(b) * c.max_pages + p);
  return page_row(c, page, h, j - p * c.ps.d);
}

// Programmatic dependent launch. Every kernel of the cache and of the key
// weights is launched with launch_dependent: its CTAs may be set up while the
// kernel before it in the stream ends, and they touch no memory that a call can
// share before grid_dependency_wait, after which everything before the kernel
// has completed and is visible. Back to back that takes 1 to 3 us off a call (one
// token appended 4.2 -> 3.2 us, a decode of 512 slots 8.3 -> 6.7).
// grid_launch_dependents lets the next kernel start before this one ends; it
// stands behind the wait, so that a second kernel of a call may rely on all that
// came before the first, and only in kernels of few CTAs: in the append's 65536
// it cost 10 % (85 against 96 us).
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Raises a kernel's shared-memory limit on the current device, once per device
// (`done`: a mask of devices, one per kernel). beside: all of an SM's memory becomes
// shared memory, so that another kernel's CTA may come beside this one's.
template <class K>
inline cudaError_t allow_smem(K kern, int bytes, std::atomic<unsigned long long>& done, bool beside = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && beside)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch of a kernel that calls grid_dependency_wait, in every CTA, before it
// reads or writes what another kernel may write or read.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Slots per unit of the decode: 32 KiB of K and V.
__host__ __device__ constexpr int decode_unit(int d) { return 64 * (128 / d); }

// The eviction's moves: a list of more than kInlineMoves is left to a second launch
// of this many CTAs.
constexpr int kInlineMoves = 256;
constexpr int kMovesPerCta = 64;
constexpr long long move_ctas(long long items, long long list) {
  return list > kInlineMoves ? items * ((list + kMovesPerCta - 1) / kMovesPerCta) : 0;
}

// ---- Arguments ------------------------------------------------------------
struct DecodeArgs {
  CacheView c;
  const uint16_t* q;      // [B][Hq][d]
  const uint16_t* k;      // cache
  const uint16_t* v;      // cache
  uint16_t* o;            // [B][Hq][d]
  float* lse;             // [B][Hq]
  const float* w_in;      // [B][Hkv][L] or nullptr
  float* w_out;
  float* logits;          // workspace, with weights: [B][Hkv][L][g], log2 units
  float* part_o;          // workspace [2 G][heads of a tile][d]: unnormalised O of a split segment
  float2* part_ml;        // workspace [2 G][heads of a tile]: its (m, l), m in log2 units
  int Hq, g;              // query heads; query heads per key head
  int HG;                 // head tiles per key head
  int join_split;         // blocks of the join per CTA of the decode
  int whole;              // a CTA has one whole item, and there is no join
  float scale_log2;       // scale * log2(e)
  const int* prefix;      // shared prefix: its pages [prefix_pages]
  const int* prefix_len;  // [1]
  int prefix_cap;         // slots that the prefix can have at most
  long long* starts;      // workspace [B + 3]: units before those of each sequence, the prefix's CTAs, uneven_shares
  int rows;               // query rows of a key head, B * g: row R is head R % g of sequence R / g
  FastDiv fg;
  int early;              // by warps: CTAs that begin beside the prefix's kernel; 0: all alike
  int prefix_items;       // with `early`: items of that kernel
  int row_tiles;          // tiles of query rows whose prefix this kernel attends to itself, per key head, or 0
  FastDiv ft;             // row_tiles
  int box;                // slots of one copy: a power of two, at most 16, that divides the page size
};

// The part of an item and a CTA: from one part to the next either number grows, or both.
__host__ __device__ constexpr int shared_part(int item, int cta) { return item + cta; }

// A shared prefix: its slots, and those of them in whole copies, which are attended to
// once for all sequences of at least `len` slots.
struct PrefixLen {
  int len, cut;
};
__device__ __forceinline__ PrefixLen prefix_slots(const DecodeArgs& a) {
  const int n = cut_len(ld_global(a.prefix_len), a.prefix_cap);
  return PrefixLen{n, n & ~(a.box - 1)};
}

// Attention to a prefix that sequences share.
struct PrefixArgs {
  DecodeArgs d;           // the slots behind the prefix: its view of the cache and its parts
  int head_tile;          // query heads of an item behind the prefix
  int tail_ctas;          // CTAs that work on them, as workers or each with four
  int tail_warps;         // 1: workers are warps
  int items;              // Hkv * ceil(rows / 256), or 0: d.row_tiles
  FastDiv fblocks;        // items per key head
  int ctas;               // of the prefix
  float* part_o;          // workspace [items + ctas][256][d]: unnormalised O of a segment
  float2* part_ml;        // workspace [items + ctas][256]: its (m, l)
  unsigned long long timeout_ns;
  int fault;              // 0 normally; failure-path test: the first V tile of each CTA never loads
};

struct AppendArgs {
  CacheView c;
  const uint16_t* k;      // [B][Hkv][T][d]
  const uint16_t* v;
  uint16_t* kc;
  uint16_t* vc;
  const int* num_new;     // [B] or nullptr (all T)
  float* weights;         // [B][Hkv][L] or nullptr
  const float* new_weights;  // [B][Hkv][T] or nullptr (0)
  int* positions;         // [B][Hkv][L] or nullptr
  const int* next_pos;    // [B]
  int* lens_out;          // [B]
  int T, d;
  FastDiv fT, fH;
  long long rows;         // B * Hkv * T
};

struct EvictArgs {
  CacheView c;
  uint16_t* kc;
  uint16_t* vc;
  const float* w_in;      // [B][Hkv][L]
  float* w_out;
  const int* p_in;        // [B][Hkv][L] or nullptr
  int* p_out;
  const int* next_pos;    // [B] (with p_in)
  int* lens_out;          // [B]
  int* holes;             // workspace [B*Hkv][list]
  int* movers;            // workspace [B*Hkv][list]
  int* counts;            // workspace [B*Hkv]: moves of each item
  int list;               // longest list of moves: min(budget, L - budget)
  int budget, recent, d;
  int cached;             // keys of a CTA's slots fit in its shared memory
};

struct ResizeArgs {
  int* table;             // [B][max_pages]
  const int* lens;        // [B]
  const int* new_lens;    // [B]
  int* refs;              // [num_pages]
  int* free_pages;        // [num_pages]
  int* num_free;          // [1]
  int* lens_out;          // [B]
  int* owner;             // workspace [num_pages]: a release of each page given back
  int* gone;              // workspace [B * max_pages]: the page of each release
  int B, num_pages, max_pages;
  int L;                  // max_pages * page_size
  int group;              // sequences per prefix sum
  FastDiv ps;
  int* status;
};

struct KeyWeightArgs {
  const float* lse;       // [B*Hq][N]
  const int* q_lens;      // [B] or nullptr
  float* out;             // [B*Hkv][Nk]
  float* part;            // workspace [2 G][256]
  int B, Hq, Hkv, g, N, Nk;
  int nkb;                // key blocks of 256
  float scale_log2;       // scale * log2(e)
  int* status;
  unsigned long long timeout_ns;
  int fault;              // 0 normally; failure-path test: the first Q tile of each CTA never loads
};

}  // namespace fa2
