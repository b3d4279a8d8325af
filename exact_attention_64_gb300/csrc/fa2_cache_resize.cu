// Page tables that follow lengths.
//
// Sequence b has ceil(lens[b] / page size) pages and is to have ceil(new_lens[b] /
// page size). Pages past the new length go back: their count of users falls by one,
// and a page that nobody names any more goes to the free list. Then sequences that
// grow take pages from the list's end, in their order, while they last.
//
// What bounds it: latency. A step of a served batch changes a few pages, and is the
// read of the lengths, a scan, and two dependent reads per page. One CTA does that. When
// many pages change it is the scattered accesses to counts and owners, five for each
// page given back, one sector each at about one a clock and SM: the CTAs of a cluster,
// 16 where the GPU allows it, share them.
//
// The result does not depend on timing. Releases and takes are numbered by (sequence,
// page of the sequence) through prefix sums of their counts; counts fall by atomic
// integer adds; of several releases that name a page the last in that order stands
// for it (a maximum), and the list receives the pages in reverse order, the first
// release at its end, so that a resize that is undone leaves the list as it was.
#include <atomic>

#include "fa2_cache.cuh"

namespace fa2 {

// A step of 256 sequences and back takes 7.7 us with 512 threads (8.0 to 8.2 on other
// boards), 10.8 with 1024 and 7.1 with 256; 512 sequences, three quarters of which change by up to 1024 pages, and back
// 77, 72 and 114.
constexpr int kRszThreads = 512;
constexpr int kRszWarps = kRszThreads / 32;
constexpr int kRszGroups = 4096;    // prefix sums kept in shared memory
constexpr int kRszAlone = 4096;     // releases and takes that one CTA makes by itself

struct RszShared {
  int rel[kRszGroups + 1], need[kRszGroups + 1];  // releases, takes before each group of sequences
  int2 warp[kRszWarps];
  int count[kRszWarps];
  uint32_t freed;                                 // pages that this CTA's releases free
  int taken;
};

__device__ __forceinline__ uint32_t rsz_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// By all threads of the cluster, each warp converged.
__device__ __forceinline__ void rsz_sync(int C) {
  __syncwarp();
  if (C > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else __syncthreads();
}
__device__ __forceinline__ uint32_t rsz_remote(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Pages before and after.
struct RszPages {
  int old_p, new_p;
  __device__ int rel() const { return max(old_p - new_p, 0); }
  __device__ int need() const { return max(new_p - old_p, 0); }
};
__device__ __forceinline__ RszPages rsz_pages(const ResizeArgs& a, int b) {
  const int ps = a.ps.d;
  return RszPages{div_by(cut_len(ld_global(a.lens + b), a.L) + ps - 1, a.ps),
                  div_by(cut_len(ld_global(a.new_lens + b), a.L) + ps - 1, a.ps)};
}

// Where release or take number i lies: its sequence, and its rank there.
template <bool TAKE>
__device__ __forceinline__ int rsz_find(const ResizeArgs& a, const RszShared& sh, int groups, int i, RszPages* pg,
                                        int* off) {
  const int* pre = TAKE ? sh.need : sh.rel;
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid - 1;
  }
  int r = i - pre[lo], b = lo * a.group;
  for (;; ++b) {
    *pg = rsz_pages(a, b);
    const int n = TAKE ? pg->need() : pg->rel();
    if (r < n) break;
    r -= n;
  }
  *off = r;
  return b;
}

__global__ void __launch_bounds__(kRszThreads, 1) fa2_cache_resize_kernel(const ResizeArgs a, int C) {
  __shared__ RszShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? static_cast<int>(rsz_rank()) : 0;
  grid_dependency_wait();
  grid_launch_dependents();

  const int listed = ld_global(a.num_free), nf = cut_len(listed, a.num_pages);
  // Prefix sums of the counts, by every CTA for itself.
  const int groups = (a.B + a.group - 1) / a.group, per = (groups + kRszThreads - 1) / kRszThreads;
  int2 mine = make_int2(0, 0);
  for (int g = tid * per; g < min((tid + 1) * per, groups); ++g) {
    sh.rel[g] = mine.x;
    sh.need[g] = mine.y;
    for (int b = g * a.group; b < min((g + 1) * a.group, a.B); ++b) {
      const RszPages p = rsz_pages(a, b);
      mine.x += p.rel();
      mine.y += p.need();
      if (rank == 0) {
        const int x = ld_global(a.lens + b), y = ld_global(a.new_lens + b);
        if (x != cut_len(x, a.L) || y != cut_len(y, a.L)) report_page(a.status);
      }
    }
  }
  int2 incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) sh.warp[warp] = incl;
  __syncthreads();
  int2 before = make_int2(incl.x - mine.x, incl.y - mine.y), total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kRszWarps; ++w) {
    const int2 x = sh.warp[w];
    if (w < warp) {
      before.x += x.x;
      before.y += x.y;
    }
    total.x += x.x;
    total.y += x.y;
  }
  for (int g = tid * per; g < min((tid + 1) * per, groups); ++g) {
    sh.rel[g] += before.x;
    sh.need[g] += before.y;
  }
  if (tid == 0) {
    sh.rel[groups] = total.x;
    sh.need[groups] = total.y;
  }
  __syncthreads();
  const int R = total.x;
  if (R <= kRszAlone && total.y <= kRszAlone) {
    if (rank > 0) return;
    C = 1;
  }
  if (rank == 0 && tid == 0 && nf != listed) report_page(a.status);

  int freed = 0;
  if (R > 0) {
    // A warp has a run of the releases, in their order.
    const int warps = C * kRszWarps, run = ((R + warps - 1) / warps + 31) / 32 * 32;
    const long long w0 = static_cast<long long>(rank * kRszWarps + warp) * run;
    const int i0 = static_cast<int>(min(w0, static_cast<long long>(R))), i1 = min(R - i0, run) + i0;
    constexpr int U = 4;  // releases of a lane whose reads are in flight together
    int first[U];         // pages of this lane's first U releases, -1: none
#pragma unroll
    for (int u = 0; u < U; ++u) first[u] = -1;
    for (int ib = i0 + lane; ib < i1; ib += 32 * U) {
      int page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = ib + 32 * u;
        page[u] = -1;
        if (i >= i1) continue;
        RszPages pg;
        int off;
        const int b = rsz_find<false>(a, sh, groups, i, &pg, &off);
        page[u] = ld_global(a.table + static_cast<size_t>(b) * a.max_pages + pg.new_p + off);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = ib + 32 * u;
        if (i >= i1) continue;
        if (static_cast<unsigned>(page[u]) < static_cast<unsigned>(a.num_pages)) {
          atomicSub(a.refs + page[u], 1);
          a.owner[page[u]] = i;  // any one of its releases
        } else {
          report_page(a.status);
          page[u] = -1;
        }
        a.gone[i] = page[u];
        if (ib == i0 + lane) first[u] = page[u];
      }
    }
    auto page_of = [&](int i, int k) {
      int p = -1;
      if (k >= U) return a.gone[i];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k == u) p = first[u];
      return p;
    };
    rsz_sync(C);
    // The last release of a page that nobody names any more stands for it. Where the
    // owner is another one, a maximum decides; one CTA knows when there is none.
    uint32_t mine = 0u;  // of this lane's first 32 releases, those that free a page
    bool clash = false;
    for (int ib = i0 + lane, kb = 0; ib < i1; ib += 32 * U, kb += U) {
      int page[U], refs[U], owner[U];
#pragma unroll
      for (int u = 0; u < U; ++u) page[u] = ib + 32 * u < i1 ? (kb == 0 ? first[u] : a.gone[ib + 32 * u]) : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        refs[u] = page[u] >= 0 ? __ldcg(a.refs + page[u]) : 1;
        owner[u] = page[u] >= 0 ? __ldcg(a.owner + page[u]) : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = ib + 32 * u;
        if (refs[u] < 0) report_page(a.status);  // given back more often than it was named
        if (refs[u] != 0) continue;
        if (kb < 32) mine |= 1u << (kb + u);
        if (owner[u] != i) clash = true;
        if (owner[u] < i) atomicMax(a.owner + page[u], i);
      }
    }
    auto owns = [&](int i, int k) { return __ldcg(a.owner + page_of(i, k)) == i; };
    auto frees = [&](int i, int k) {
      if (i >= i1) return false;
      if (k < 32) return (mine >> k & 1u) != 0u;
      return a.gone[i] >= 0 && __ldcg(a.refs + a.gone[i]) == 0 && owns(i, k);
    };
    if (C > 1 || __syncthreads_or(clash)) {
      rsz_sync(C);
      for (int i = i0 + lane, k = 0; i < i1 && k < 32; i += 32, ++k)
        if ((mine >> k & 1u) && !owns(i, k)) mine &= ~(1u << k);
    }
    int cnt = 0;
    for (int i = i0, k = 0; i < i1; i += 32, ++k) cnt += __popc(__ballot_sync(0xffffffffu, frees(i + lane, k)));
    if (lane == 0) sh.count[warp] = cnt;
    __syncthreads();
    int at = 0, sum = 0;
    for (int w = 0; w < kRszWarps; ++w) {
      if (w < warp) at += sh.count[w];
      sum += sh.count[w];
    }
    if (C > 1) {
      if (tid == 0) sh.freed = static_cast<uint32_t>(sum);
      rsz_sync(C);
    }
    for (int r = 0; r < C; ++r) {
      const int x = C > 1 ? static_cast<int>(rsz_remote(&sh.freed, r)) : sum;
      if (r < rank) at += x;
      freed += x;
    }
    for (int i = i0, k = 0; i < i1; i += 32, ++k) {
      const bool f = frees(i + lane, k);
      const unsigned m = __ballot_sync(0xffffffffu, f);
      const long long pos = static_cast<long long>(nf) + freed - 1 - at - __popc(m & ((1u << lane) - 1u));
      if (f) {
        if (pos < a.num_pages) a.free_pages[pos] = page_of(i + lane, k);
        else report_page(a.status);
      }
      at += __popc(m);
    }
    rsz_sync(C);  // the list is complete, and nobody reads another CTA's memory any more
  }

  const int have = static_cast<int>(min(static_cast<long long>(nf) + freed, static_cast<long long>(a.num_pages)));
  // Sequences take while the pages last: those whose takes end at or below `have`.
  if (tid == 0) {
    int taken = total.y;
    if (taken > have) {
      int lo = 0, hi = groups - 1;  // the last group that begins at or below `have`
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh.need[mid] <= have) lo = mid; else hi = mid - 1;
      }
      taken = sh.need[lo];
      for (int b = lo * a.group; b < a.B; ++b) {
        const int n = rsz_pages(a, b).need();
        if (n > have - taken) break;
        taken += n;
      }
    }
    sh.taken = taken;
  }
  __syncthreads();
  const int taken = sh.taken, step = C * kRszThreads;
  for (int i = rank * kRszThreads + tid; i < taken; i += step) {
    RszPages pg;
    int off;
    const int b = rsz_find<true>(a, sh, groups, i, &pg, &off);
    const int page = __ldcg(a.free_pages + have - 1 - i);
    a.table[static_cast<size_t>(b) * a.max_pages + pg.old_p + off] = page;
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages)) a.refs[page] = 1;
    else report_page(a.status);
  }
  for (int g = rank * kRszThreads + tid; g < groups; g += step) {
    int end = sh.need[g];
    for (int b = g * a.group; b < min((g + 1) * a.group, a.B); ++b) {
      const int n = rsz_pages(a, b).need();
      end += n;
      a.lens_out[b] = cut_len(ld_global((n == 0 || end <= taken ? a.new_lens : a.lens) + b), a.L);
    }
  }
  if (R == 0) rsz_sync(C);  // every CTA has read the count
  if (rank == 0 && tid == 0) *a.num_free = have - taken;
}

// CTAs of a cluster on the current device: 16 if it can run such a cluster, else 8, which
// every GPU can.
static cudaError_t rsz_cluster(cudaLaunchConfig_t& cfg, int* out) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>& k = known[dev & 63];
  if (k.load(std::memory_order_acquire) == 0) {
    int n = 8, clusters = 0;
    if (cudaFuncSetAttribute(fa2_cache_resize_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
      cfg.gridDim = dim3(16);
      cfg.attrs[1].val.clusterDim.x = 16;
      if (cudaOccupancyMaxActiveClusters(&clusters, fa2_cache_resize_kernel, &cfg) == cudaSuccess && clusters > 0) n = 16;
    }
    (void)cudaGetLastError();
    k.store(n, std::memory_order_release);
  }
  *out = k.load(std::memory_order_acquire);
  return cudaSuccess;
}

cudaError_t launch_cache_resize(const ResizeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRszThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  // A table that cannot change more pages than one CTA handles needs no more.
  int C = 1;
  if (static_cast<long long>(a.B) * a.max_pages > kRszAlone) {
    const cudaError_t e = rsz_cluster(cfg, &C);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(C);
  at[1].val.clusterDim.x = C;
  return cudaLaunchKernelEx(&cfg, fa2_cache_resize_kernel, a, C);
}

// Sequences per prefix sum.
int resize_group(int B) { return (B + kRszGroups - 1) / kRszGroups; }

}  // namespace fa2
