// pages.cu -- the page table and the slot map of a step, from the requests'
// lengths: pages for new tokens are taken from a stack of free ones, the new
// tokens' cache rows are written down, and ended requests give their pages back.
//
//   need[r]  = ceil((len[r] + n[r]) / 64) - ceil(len[r] / 64)
//   table[r][ceil(len[r] / 64) + j] = free[count - 1 - (sum of need[< r] + j)]
//   slot(token i of r) = table[r][(len[r] + i) / 64] * 64 + (len[r] + i) % 64
//
// Whole numbers only, and a few of them: what bounds it is the latency of one
// launch with two sums over all requests in it.  So one cluster does it all: its
// CTAs take a stretch of the requests each, exchange their sums through shared
// memory, hand out pages (a thread a page), and then share the tokens evenly (a
// thread four slots; whose they are is looked up in the offsets, in shared
// memory).  Barriers of the cluster stand between the phases, so that lengths,
// table and count may be updated in place: everything that another CTA reads
// before a barrier is written behind it.
#include <climits>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(pages)

namespace dsa {
namespace {

constexpr int kThreads = 1024;
constexpr int kOffsetsInSmem = 8192;      // offsets of up to so many requests (32 KB)

__device__ __forceinline__ int pages_of(int len) { return static_cast<int>((len + (kPage - 1LL)) / kPage); }

struct Sums {
  long long tokens, need, freed;
};

// Inclusive sums over the block's threads; every thread also gets the block's.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v.tokens, o), b = __shfl_up_sync(0xffffffffu, v.need, o),
                    c = __shfl_up_sync(0xffffffffu, v.freed, o);
    if (lane >= o) {
      v.tokens += a;
      v.need += b;
      v.freed += c;
    }
  }
  __syncthreads();      // the call before has read warp_sums
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Sums before = {0, 0, 0};
  total = before;
#pragma unroll 4
  for (int w = 0; w < kThreads / 32; ++w) {
    const Sums s = warp_sums[w];
    if (w < warp) {
      before.tokens += s.tokens;
      before.need += s.need;
      before.freed += s.freed;
    }
    total.tokens += s.tokens;
    total.need += s.need;
    total.freed += s.freed;
  }
  v.tokens += before.tokens;
  v.need += before.need;
  v.freed += before.freed;
  return v;
}

// One request as its thread sees it.
struct Request {
  int len;          // tokens before the call
  int add;          // new ones
  int need;         // pages it asks for
  bool fits;        // its row of the table holds them
  bool ended;
};

__device__ __forceinline__ Request load(const PagesLaunch& p, int r) {
  Request q = {0, 0, 0, true, false};
  if (r >= p.batch) return q;
  const int change = p.change[r];
  const long long cap = static_cast<long long>(p.max_pages) * kPage;
  q.len = p.seqlens[r];
  if (q.len < 0) q.len = 0;
  q.ended = change < 0;
  q.add = change > 0 ? change : 0;
  q.fits = q.ended || q.len + static_cast<long long>(q.add) <= cap;
  if (!q.fits) raise_error(kErrCheck);
  if (q.fits && q.add > 0) q.need = pages_of(q.len + q.add) - pages_of(q.len);
  return q;
}

// Pages that an ended request gives back: ids of its row inside the cache.  (One
// warp.  kPush: they go to the stack from `at` on, and the row is cleared.)
template <bool kPush>
__device__ __forceinline__ int give_back(const PagesLaunch& p, int r, int len, long long at) {
  const int lane = threadIdx.x & 31;
  const int n = min(pages_of(len), p.max_pages);
  int32_t* row = p.page_table + static_cast<long long>(r) * p.max_pages;
  int found = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int id = i < n ? row[i] : -1;
    const bool good = id >= 0 && id < p.num_pages;
    const uint32_t mask = __ballot_sync(0xffffffffu, good);
    if (kPush) {
      const long long to = at + found + __popc(mask & ((1u << lane) - 1u));
      if (good && to < p.num_pages) p.free_pages[to] = id;
      if (i < n && (!good || to >= p.num_pages)) raise_error(kErrCheck);
      if (i < n) row[i] = -1;
    }
    found += __popc(mask);
  }
  return found;
}

__global__ void __launch_bounds__(kThreads) pages_kernel(const PagesLaunch p) {
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ Sums cta_sums;             // of this CTA's requests
  __shared__ unsigned long long cta_taken;      // pages handed out, up to its last request that got some
  __shared__ int cta_refused, cta_ended;
  __shared__ int need_end[kThreads];    // of a tile of requests: pages asked for up to its end ...
  __shared__ int first_page[kThreads];  // ... and the table entry its new pages begin at (-1: refused)
  __shared__ int offsets[kOffsetsInSmem + 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x;
  const int per = (p.batch + ctas - 1) / ctas;
  const int r_lo = min(p.batch, rank * per), r_hi = min(p.batch, r_lo + per);
  int count = *p.free_count;
  if (count < 0 || count > p.num_pages) {
    raise_error(kErrCheck);
    count = min(max(count, 0), p.num_pages);
  }

  // Pages given back by the ended requests of a warp's lanes, each to its lane.
  auto freed_pages = [&](const Request& q, int r) {
    int mine = 0;
    uint32_t ended = __ballot_sync(0xffffffffu, q.ended && q.len > 0);
    while (ended) {
      const int l = __ffs(ended) - 1;
      ended &= ended - 1;
      const int n = give_back<false>(p, __shfl_sync(0xffffffffu, r, l), __shfl_sync(0xffffffffu, q.len, l), 0);
      if (lane == l) mine = n;
    }
    return mine;
  };

  // -------------------------------------------------- sums of the stretches
  Sums mine = {0, 0, 0};
  for (int r0 = r_lo; r0 < r_hi; r0 += kThreads) {
    const int r = r0 + tid < r_hi ? r0 + tid : p.batch;
    const Request q = load(p, r);
    Sums total;
    block_scan({q.add, q.need, freed_pages(q, r)}, warp_sums, total);
    mine.tokens += total.tokens;
    mine.need += total.need;
    mine.freed += total.freed;
  }
  if (tid == 0) {
    cta_sums = mine;
    cta_taken = 0;
    cta_refused = cta_ended = 0;
  }
  cluster_sync();
  auto remote64 = [&](const void* v, int c) {
    const uint32_t a = mapa_shared(smem_u32(v), c);
    return static_cast<long long>(static_cast<uint64_t>(ld_shared_cluster_u32(a)) |
                                  static_cast<uint64_t>(ld_shared_cluster_u32(a + 4)) << 32);
  };
  Sums before = {0, 0, 0};
  long long all_tokens = 0;
  for (int c = 0; c < ctas; ++c) {
    const long long t = remote64(&cta_sums.tokens, c);
    all_tokens += t;
    if (c < rank) {
      before.tokens += t;
      before.need += remote64(&cta_sums.need, c);
      before.freed += remote64(&cta_sums.freed, c);
    }
  }

  // ------------------------------------- offsets, lengths and the new pages
  const long long freed_before = before.freed;
  for (int r0 = r_lo; r0 < r_hi; r0 += kThreads) {
    const int r = r0 + tid < r_hi ? r0 + tid : p.batch;
    const Request q = load(p, r);
    Sums total, end = block_scan({q.add, q.need, 0}, warp_sums, total);
    const long long tok_end = before.tokens + end.tokens, need_all = before.need + end.need;
    // Pages in request order: a request that asks for more than are left gets
    // none, nor does any after it.  Nor one whose slots the map does not hold.
    const bool granted = q.fits && (q.need == 0 || need_all <= count) && (q.add == 0 || tok_end <= p.max_tokens);
    if (r < p.batch) {
      p.cu_new[r + 1] = static_cast<int>(min(tok_end, static_cast<long long>(p.max_tokens)));
      // (A refused request's length is written as ~length, until the slots are; an
      // ended one's is still needed.)
      if (q.ended) cta_ended = 1;
      else p.seqlens_out[r] = granted ? q.len + q.add : ~q.len;
      if (!granted) {
        raise_error(kErrCheck);
        cta_refused = 1;
      } else if (q.need > 0) {
        atomicMax(&cta_taken, static_cast<unsigned long long>(need_all));
      }
    }
    __syncthreads();
    need_end[tid] = static_cast<int>(min(end.need, static_cast<long long>(INT_MAX)));
    first_page[tid] = granted ? pages_of(q.len) : -1;
    __syncthreads();
    // A thread a page.
    const long long left = count - before.need;
    const int pages = static_cast<int>(max(0LL, min(total.need, left)));
    for (int e = tid; e < pages; e += kThreads) {
      int lo = 0, hi = kThreads - 1;      // the first thread whose request's pages end behind e
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (need_end[mid] > e) hi = mid;
        else lo = mid + 1;
      }
      if (first_page[lo] < 0) continue;
      int id = p.free_pages[count - 1 - (before.need + e)];
      if (id < 0 || id >= p.num_pages) {
        raise_error(kErrCheck);
        id = -1;
      }
      const int j = e - (lo > 0 ? need_end[lo - 1] : 0);
      p.page_table[static_cast<long long>(r0 + lo) * p.max_pages + first_page[lo] + j] = id;
    }
    before.tokens += total.tokens;
    before.need += total.need;
  }
  if (rank == 0 && tid == 0) p.cu_new[0] = 0;
  cluster_sync();      // table, offsets and lengths are written, free pages read
  long long taken = 0;
  bool refused = false;
  for (int c = 0; c < ctas; ++c) {
    taken = max(taken, remote64(&cta_taken, c));
    refused |= ld_shared_cluster_u32(mapa_shared(smem_u32(&cta_refused), c)) != 0;
  }

  // ------------------------------------------------------- pages given back
  if (cta_ended) {
    // A warp a request, their ids in the order of the requests.
    long long at = count - taken + freed_before;
    for (int r0 = r_lo; r0 < r_hi; r0 += kThreads / 32) {
      const int r = r0 + warp;
      const bool ended = r < r_hi && p.change[r] < 0;
      const int len = ended ? max(0, p.seqlens[r]) : 0;
      const int n = ended ? give_back<false>(p, r, len, 0) : 0;
      if (lane == 0) need_end[warp] = n;
      __syncthreads();
      long long to = at;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) to += need_end[w];
        at += need_end[w];
      }
      if (ended) {
        give_back<true>(p, r, len, to);
        if (lane == 0) p.seqlens_out[r] = 0;
      }
      __syncthreads();
    }
  }
  if (rank == 0 && tid == 0) {
    long long freed = 0;
    for (int c = 0; c < ctas; ++c) freed += remote64(&cta_sums.freed, c);
    p.free_count_out[0] = static_cast<int>(min(count - taken + freed, static_cast<long long>(p.num_pages)));
  }

  // ------------------------------------------------------------------ slots
  const bool near = p.batch <= kOffsetsInSmem;
  if (near)
    for (int i = tid; i <= p.batch; i += kThreads) offsets[i] = p.cu_new[i];
  __syncthreads();
  auto offset = [&](int i) { return near ? offsets[i] : p.cu_new[i]; };
  const int tokens = static_cast<int>(min(all_tokens, static_cast<long long>(p.max_tokens)));
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (long long t0 = 4LL * (rank * kThreads + tid); t0 < p.max_tokens; t0 += 4LL * kThreads * ctas) {
    int v[4] = {-1, -1, -1, -1};
    if (t0 < tokens) {
      int r = 0, hi = p.batch - 1;      // the first request that ends behind t0
      while (r < hi) {
        const int mid = (r + hi) >> 1;
        if (offset(mid + 1) > t0) hi = mid;
        else r = mid + 1;
      }
      int end = offset(r + 1), len = p.seqlens_out[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = static_cast<int>(t0) + e;
        if (t >= tokens) break;
        while (t >= end) {      // (requests without new tokens lie between)
          end = offset(++r + 1);
          len = p.seqlens_out[r];
        }
        if (len < 0) continue;
        const int pos = len - (end - t);
        const int id = p.page_table[static_cast<long long>(r) * p.max_pages + pos / kPage];
        if (id >= 0 && id < p.num_pages) v[e] = id * kPage + pos % kPage;
        else raise_error(kErrCheck);
      }
    }
    if (wide && t0 + 3 < p.max_tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t0 + e < p.max_tokens) p.slots[t0 + e] = v[e];
    }
  }
  cluster_sync();      // the others have read this CTA's sums, and the lengths
  if (refused)
    for (int r = r_lo + tid; r < r_hi; r += kThreads)
      if (p.seqlens_out[r] < 0) p.seqlens_out[r] = ~p.seqlens_out[r];
}

}  // namespace

// CTAs of the cluster: one where a block's threads have a request and a few
// slots each at most.
cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t s) {
  const int ctas = a.batch <= kThreads && a.max_tokens <= 8 * kThreads ? 1 : 16;
  if (ctas > 8) {
    cudaError_t e = cudaFuncSetAttribute(pages_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(pages_kernel, dim3(ctas), dim3(kThreads), 0, s, false, ctas, a);
}

}  // namespace dsa
