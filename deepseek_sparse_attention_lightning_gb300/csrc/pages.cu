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
// thread eight slots; whose they are is looked up in the offsets, in shared
// memory).  Barriers of the cluster stand between the phases, so that lengths,
// table and count may be updated in place: everything that another CTA reads
// before a barrier is written behind it.
#include <climits>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(pages)

namespace dsa {
namespace {

constexpr int kCluster = 16;
constexpr int kNear = 4096;      // offsets and lengths of up to so many requests in shared memory (32 KB)

__device__ __forceinline__ int pages_of(int len) { return static_cast<int>((len + (kPage - 1LL)) / kPage); }

// Sums of tokens and of pages asked for end at 2^32 - 1 (more than any slot map or
// stack holds): what lies behind is refused whatever its size.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? 0xffffffffu : s;
}

struct Sums {
  uint32_t tokens, need, freed;
};

// Inclusive sums over the block's threads (tokens and pages asked for); every
// thread also gets the block's.
template <int kThreads>
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  constexpr int kWarps = (kThreads / 32);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](uint32_t& x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = add_sat(x, y);
    }
  };
  scan(v.tokens);
  scan(v.need);
  __syncthreads();      // the call before has read warp_sums
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  // Each warp scans the warps' sums for itself.
  Sums w = lane < kWarps ? warp_sums[lane] : Sums{0u, 0u, 0u};
  scan(w.tokens);
  scan(w.need);
  total.tokens = __shfl_sync(0xffffffffu, w.tokens, 31);
  total.need = __shfl_sync(0xffffffffu, w.need, 31);
  const uint32_t bt = __shfl_sync(0xffffffffu, w.tokens, max(warp - 1, 0)), bn = __shfl_sync(0xffffffffu, w.need, max(warp - 1, 0));
  if (warp > 0) {
    v.tokens = add_sat(v.tokens, bt);
    v.need = add_sat(v.need, bn);
  }
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

// kCtas: of the cluster (the only one of the grid); kRun: slots of a thread in a row.
template <int kThreads, int kCtas, int kRun>
__global__ void __launch_bounds__(kThreads, 1) pages_kernel(const PagesLaunch p) {
  __shared__ Sums warp_sums[32];
  __shared__ Sums sums[kCtas];          // of each CTA's requests (every CTA writes its own to all)
  __shared__ int given[kCtas];          // pages handed out, up to a CTA's last request that got some (~: it refused one)
  __shared__ int cta_taken, cta_freed, cta_refused, cta_ended;
  __shared__ int need_end[kThreads];    // of a tile of requests: pages asked for up to its end ...
  __shared__ int first_page[kThreads];  // ... and the table entry its new pages begin at (-1: refused)
  __shared__ int offsets[kNear + 1], lengths[kNear];

  if (kCtas > 1) cluster_arrive();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kCtas > 1 ? static_cast<int>(cluster_ctarank()) : 0, per = (p.batch + kCtas - 1) / kCtas;
  const int r_lo = min(p.batch, rank * per), r_hi = min(p.batch, r_lo + per);
  int count = *p.free_count;
  if (count < 0 || count > p.num_pages) {
    raise_error(kErrCheck);
    count = min(max(count, 0), p.num_pages);
  }
  if (tid == 0) {
    cta_taken = cta_freed = 0;
    cta_refused = cta_ended = 0;
  }
  __syncthreads();
  // This CTA's value into element `rank` of an array of every CTA (one warp).
  auto publish = [&](const void* at, uint32_t v) {
    if (lane < kCtas) st_shared_cluster_u32(mapa_shared(smem_u32(at), lane), v);
  };

  Sums before = {0, 0, 0};      // of the CTAs before this one
  uint32_t all_tokens = 0;
  if constexpr (kCtas > 1) {
    // ------------------------------------------------ sums of the stretches
    Sums mine = {0, 0, 0};
    for (int r0 = r_lo; r0 < r_hi; r0 += kThreads) {
      const int r = r0 + tid < r_hi ? r0 + tid : p.batch;
      const Request q = load(p, r);
      Sums total;
      block_scan<kThreads>({static_cast<uint32_t>(q.add), static_cast<uint32_t>(q.need), 0u}, warp_sums, total);
      mine.tokens = add_sat(mine.tokens, total.tokens);
      mine.need = add_sat(mine.need, total.need);
      // Pages given back by the ended requests of a warp's lanes.
      uint32_t ended = __ballot_sync(0xffffffffu, q.ended);
      int freed = 0;
      while (ended) {
        const int l = __ffs(ended) - 1;
        ended &= ended - 1;
        freed += give_back<false>(p, __shfl_sync(0xffffffffu, r, l), __shfl_sync(0xffffffffu, q.len, l), 0);
      }
      if (lane == 0 && freed) atomicAdd(&cta_freed, freed);
    }
    cluster_wait();       // every CTA of the cluster has started
    __syncthreads();
    if (warp == 0) {
      publish(&sums[rank].tokens, mine.tokens);
      publish(&sums[rank].need, mine.need);
      publish(&sums[rank].freed, cta_freed);
    }
    cluster_sync();
    // (A lane a CTA.)
    const Sums of = lane < kCtas ? sums[lane] : Sums{0u, 0u, 0u};
    all_tokens = of.tokens;
    before = lane < rank ? of : Sums{0u, 0u, 0u};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all_tokens = add_sat(all_tokens, __shfl_xor_sync(0xffffffffu, all_tokens, o));
      before.tokens = add_sat(before.tokens, __shfl_xor_sync(0xffffffffu, before.tokens, o));
      before.need = add_sat(before.need, __shfl_xor_sync(0xffffffffu, before.need, o));
      before.freed += __shfl_xor_sync(0xffffffffu, before.freed, o);
    }
  }

  // ------------------------------------- offsets, lengths and the new pages
  const bool near = p.batch <= kNear;
  const long long freed_before = before.freed;
  for (int r0 = r_lo; r0 < r_hi; r0 += kThreads) {
    const int r = r0 + tid < r_hi ? r0 + tid : p.batch;
    const Request q = load(p, r);
    Sums total, end = block_scan<kThreads>({static_cast<uint32_t>(q.add), static_cast<uint32_t>(q.need), 0u}, warp_sums, total);
    const uint32_t tok_end = add_sat(before.tokens, end.tokens), need_all = add_sat(before.need, end.need);
    const uint32_t slots = p.max_tokens;
    // Pages in request order: a request that asks for more than are left gets
    // none, nor does any after it.  Nor one whose slots the map does not hold.
    const bool granted = q.fits && (q.need == 0 || need_all <= static_cast<uint32_t>(count)) && (q.add == 0 || tok_end <= slots);
    if (r < p.batch) {
      const int cut = static_cast<int>(min(tok_end, slots));
      p.cu_new[r + 1] = cut;
      // (A refused request's length is written as ~length, until the slots are; an
      // ended one's is still needed.)
      const int len = granted ? q.len + q.add : ~q.len;
      if (q.ended) cta_ended = 1;
      else p.seqlens_out[r] = len;
      if (kCtas == 1 && near) {
        offsets[r + 1] = cut;
        lengths[r] = len;
      }
      if (!granted) {
        raise_error(kErrCheck);
        cta_refused = 1;
      } else if (q.need > 0) {
        atomicMax(&cta_taken, static_cast<int>(need_all));
      }
    }
    __syncthreads();
    need_end[tid] = static_cast<int>(min(end.need, static_cast<uint32_t>(INT_MAX)));
    first_page[tid] = granted ? pages_of(q.len) : -1;
    __syncthreads();
    // A thread a page.
    const uint32_t left = before.need < static_cast<uint32_t>(count) ? count - before.need : 0u;
    const int pages = static_cast<int>(min(total.need, left));
    for (int e = tid; e < pages; e += kThreads) {
      int lo = 0, hi = kThreads - 1;      // the first thread whose request's pages end behind e
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (need_end[mid] > e) hi = mid;
        else lo = mid + 1;
      }
      if (first_page[lo] < 0) continue;
      int id = p.free_pages[count - 1 - (static_cast<int>(before.need) + e)];
      if (id < 0 || id >= p.num_pages) {
        raise_error(kErrCheck);
        id = -1;
      }
      const int j = e - (lo > 0 ? need_end[lo - 1] : 0);
      p.page_table[static_cast<long long>(r0 + lo) * p.max_pages + first_page[lo] + j] = id;
    }
    before.tokens = add_sat(before.tokens, total.tokens);
    before.need = add_sat(before.need, total.need);
  }
  if (rank == 0 && tid == 0) p.cu_new[0] = 0;
  __syncthreads();
  int taken = cta_taken;
  bool refused = cta_refused != 0;
  if constexpr (kCtas > 1) {
    if (warp == 0) publish(&given[rank], refused ? ~taken : taken);
    cluster_sync();      // table, offsets and lengths are written, free pages read
    const int v = lane < kCtas ? given[lane] : 0;
    refused = __any_sync(0xffffffffu, v < 0);
    taken = __reduce_max_sync(0xffffffffu, v < 0 ? ~v : v);
  } else {
    all_tokens = before.tokens;
  }

  // ------------------------------------------------------- pages given back
  long long at = static_cast<long long>(count) - taken + freed_before;      // where this CTA's go
  if (cta_ended) {
    // A warp a request, their ids in the order of the requests.
    for (int r0 = r_lo; r0 < r_hi; r0 += (kThreads / 32)) {
      const int r = r0 + warp;
      const bool ended = r < r_hi && p.change[r] < 0;
      const int len = ended ? max(0, p.seqlens[r]) : 0;
      const int n = ended ? give_back<false>(p, r, len, 0) : 0;
      if (lane == 0) need_end[warp] = n;
      __syncthreads();
      long long to = at;
      for (int w = 0; w < (kThreads / 32); ++w) {
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
    if constexpr (kCtas > 1) {
      at = count - taken;
      for (int c = 0; c < kCtas; ++c) at += sums[c].freed;
    }
    p.free_count_out[0] = static_cast<int>(min(at, static_cast<long long>(p.num_pages)));
  }

  // ------------------------------------------------------------------ slots
  if (near && kCtas > 1) {
    for (int i = tid; i <= p.batch; i += kThreads) {
      offsets[i] = p.cu_new[i];
      if (i < p.batch) lengths[i] = p.seqlens_out[i];
    }
  } else if (near && tid == 0) {
    offsets[0] = 0;
  }
  __syncthreads();
  auto offset = [&](int i) { return near ? offsets[i] : p.cu_new[i]; };
  auto length = [&](int r) { return near ? lengths[r] : p.seqlens_out[r]; };
  const int tokens = static_cast<int>(min(all_tokens, static_cast<uint32_t>(p.max_tokens)));
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 31) == 0;
  // A thread has runs of kRun slots: one every grid's width, or (kRun 8) as many as there
  // are for it one behind the other, so that it looks for a request once (256 prompts of
  // 1 .. 4096 tokens: 16.4 us a run every grid's width, 13.4 so).
  constexpr long long kWidth = static_cast<long long>(kRun) * kThreads * kCtas;
  const int runs = kRun > 1 ? static_cast<int>((p.max_tokens + kWidth - 1) / kWidth) : 1;
  const int first_run = kRun > 1 ? (warp * kCtas + rank) * 32 + lane : rank * kThreads + tid;
  for (long long c0 = static_cast<long long>(kRun) * runs * first_run; c0 < p.max_tokens; c0 += kWidth * runs) {
    int r = 0, end = 0, len = 0;
    if (c0 < tokens) {
      int hi = p.batch - 1;      // the first request that ends behind c0
      while (r < hi) {
        const int mid = (r + hi) >> 1;
        if (offset(mid + 1) > c0) hi = mid;
        else r = mid + 1;
      }
      end = offset(r + 1);
      len = length(r);
    }
    // Entry of the table for position `pos` of request r; the first row of its
    // page, or -1.
    auto entry = [&](int pos) { return p.page_table + static_cast<long long>(r) * p.max_pages + pos / kPage; };
    auto first_row = [&](int id) {
      if (id >= 0 && id < p.num_pages) return id * kPage;
      raise_error(kErrCheck);
      return -1;
    };
    auto to_request_of = [&](int t) {      // (requests without new tokens lie between)
      while (t >= end) {
        end = offset(++r + 1);
        len = length(r);
      }
    };
    for (int k = 0; k < runs; ++k) {
      const long long t0 = c0 + static_cast<long long>(kRun) * k;
      if (t0 >= p.max_tokens) break;
      int v[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[e] = -1;
      if (t0 < tokens) {
        to_request_of(static_cast<int>(t0));
        if (kRun > 1 && t0 + kRun <= end) {
          // One request's tokens, on one page or two.
          if (len >= 0) {
            const int pos = len - static_cast<int>(end - t0), row = pos % kPage;
            const int id_a = *entry(pos), id_b = *entry(pos + kRun - 1);
            const int a = first_row(id_a), b = first_row(id_b);
#pragma unroll
            for (int e = 0; e < kRun; ++e) v[e] = row + e < kPage ? a + row + e : b + row + e - kPage;
            if ((a | b) < 0) {
#pragma unroll
              for (int e = 0; e < kRun; ++e)
                if ((row + e < kPage ? a : b) < 0) v[e] = -1;
            }
          }
        } else {
          // Where each token's entry is (all of them first, so that the loads overlap).
          const int32_t* at[kRun];
          int row[kRun];
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            const int t = static_cast<int>(t0) + e;
            at[e] = nullptr;
            if (t >= tokens) continue;
            to_request_of(t);
            const int pos = len - (end - t);
            if (len >= 0) at[e] = entry(pos);
            row[e] = pos % kPage;
          }
#pragma unroll
          for (int e = 0; e < kRun; ++e) v[e] = at[e] ? *at[e] : -1;
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            if (!at[e]) continue;
            const int first = first_row(v[e]);
            v[e] = first < 0 ? -1 : first + row[e];
          }
        }
      }
      if (kRun == 8 && wide && t0 + kRun <= p.max_tokens) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = static_cast<uint32_t>(v[e % kRun]);
        st_global_32(p.slots + t0, w);
      } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
          if (t0 + e < p.max_tokens) p.slots[t0 + e] = v[e];
      }
    }
  }
  if (refused && kCtas > 1) cluster_sync();      // the others have read the lengths
  if (kCtas == 1) __syncthreads();
  if (refused)
    for (int r = r_lo + tid; r < r_hi; r += kThreads)
      if (p.seqlens_out[r] < 0) p.seqlens_out[r] = ~p.seqlens_out[r];
}

}  // namespace

// One CTA of 256 threads, or of 1024, where they have a request and a few slots each
// at most; else a cluster of 16, a thread eight slots in a row where there are many
// (a prompt's are on one page or two; a step's are on a page each, whose entries
// would be waited for one after another).  us on the device: 128 requests of a token
// 3.4 (in a cluster of 16: 10.9); 256 prompts of 1 .. 4096 tokens, half a million
// slots, 13.4 (with a slot at a time, for 4 / 8 / 16 CTAs, 42 / 30 / 21).
cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t s) {
  if (a.batch <= 256 && a.max_tokens <= 4 * 256)
    return launch_kernel(pages_kernel<256, 1, 1>, dim3(1), dim3(256), 0, s, false, 1, a);
  if (a.batch <= 1024 && a.max_tokens <= 4 * 1024)
    return launch_kernel(pages_kernel<1024, 1, 1>, dim3(1), dim3(1024), 0, s, false, 1, a);
  auto kern = a.max_tokens <= 4 * 1024 * kCluster ? pages_kernel<1024, kCluster, 1> : pages_kernel<1024, kCluster, 8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(kCluster), dim3(1024), 0, s, false, kCluster, a);
}

}  // namespace dsa
