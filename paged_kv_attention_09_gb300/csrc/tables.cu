// tables.cu — block tables, slot map, positions and query offsets of one serving step,
// built on the GPU from the requests' lengths and a ring of free pages.
//
// Request b holds c tokens in cache and brings n new ones (n < 0: it has ended).  It needs
// need = ceil((c + n) / 16) - ceil(c / 16) new pages; with cum the inclusive prefix sum of
// the needs in request order, it is served when need = 0 or cum <= the free pages, and its
// k-th new page is ring[(head + cum - need + k) mod N].  The new token at position p goes to
// slot page(p / 16) * 16 + p % 16.  Ended requests' pages are pushed behind the free ones.
//
// One launch.  Every block walks the requests in chunks of 1024 with a block-wide scan of
// (rows, pages) — lengths are 8 bytes a request and come from L2 after the first block — and
// keeps the chunk's offsets in shared memory; its own 1024 rows then find their request by
// binary search there.  So no block waits for another, whatever the batch, and a single
// long prompt spreads over as many blocks as a thousand short ones.  The first row of a new
// page writes the table entry.  The block that takes the last ticket (an atomic, no
// waiting: every block has read the ring by then) pushes the ended requests' pages and
// updates the pool, so that a step works on the pool in place and can be replayed from a
// CUDA graph.
//
// Bound by latency, not bytes: a 256-request decode step moves 9 KB.
#include <cuda_runtime.h>

#include <cstdint>

#include "abi.h"
#include "internal.h"
#include "nvtx.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                       // requests per thread of a chunk
constexpr int kChunk = kThreads * kPer;       // requests per chunk
constexpr int kRowsPerBlock = 1024;
constexpr int kMaxBlocks = 1024;  // more rows than 1024 per block are taken in strides

struct TablesArgs {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* bt;
  int32_t* context;
  int32_t* starts;     // may be null
  int32_t* positions;  // may be null
  int32_t* slots;
  int32_t* ring;
  int32_t* state;  // head, free pages, ticket
  int32_t* status;
  int B, MB, N, T;
};

struct Sums {
  long long rows, pages;
};

__device__ __forceinline__ Sums add(Sums a, Sums b) { return {a.rows + b.rows, a.pages + b.pages}; }

// Exclusive block-wide prefix sum; *total receives the block's sum.  The caller
// synchronises before `part` is used again.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Sums inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up{__shfl_up_sync(0xffffffffu, inc.rows, o), __shfl_up_sync(0xffffffffu, inc.pages, o)};
    if (lane >= o) inc = add(inc, up);
  }
  if (lane == 31) part[w] = inc;
  __syncthreads();
  Sums base{0, 0}, all{0, 0};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const Sums p = part[i];
    if (i < w) base = add(base, p);
    all = add(all, p);
  }
  *total = all;
  return {base.rows + inc.rows - v.rows, base.pages + inc.pages - v.pages};
}

__device__ __forceinline__ long long pages_of(long long tokens) { return (tokens + kPage - 1) / kPage; }

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a) {
  __shared__ int s_end[kChunk];     // end row of each request of the chunk (at most T)
  __shared__ int s_start[kChunk];   // its first row
  __shared__ int s_cached[kChunk];  // its cached tokens, -1 when its rows get no slot
  __shared__ int s_ring[kChunk];    // ring offset of its first new page from the head
  __shared__ Sums s_part[kWarps];
  __shared__ int s_last, s_any, s_alloc;
  __shared__ int s_cnt[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int head0 = a.state[0], free0 = a.state[1];
  const bool pool_ok = head0 >= 0 && head0 < a.N && free0 >= 0 && free0 <= a.N;
  const int head = pool_ok ? head0 : 0, count = pool_ok ? free0 : 0;
  if (tid == 0) {
    s_any = 0;
    s_alloc = 0;
  }
  int bits = pool_ok || blockIdx.x ? 0 : 0x1;  // PKV_DEV_BAD_PAGE
  __syncthreads();

  long long rows0 = 0, pages0 = 0;  // sums over the chunks before
  for (int c0 = 0; c0 < a.B; c0 += kChunk) {
    const bool mine = (c0 / kChunk) % gridDim.x == blockIdx.x;  // this block writes the chunk's outputs
    int c[kPer], n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c0 + tid * kPer + i;
      c[i] = b < a.B ? a.cached[b] : 0;
      n[i] = b < a.B ? a.fresh[b] : 0;
    }
    // rows first: a request whose rows pass the end of the row buffers gets no pages
    long long row_sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) row_sum += n[i] > 0 ? n[i] : 0;
    Sums total;
    // (pages depend on the rows' prefix only through that end check, so most launches
    // could scan both at once; the rows that do not fit are found with one extra scan)
    const Sums at = block_scan({row_sum, 0}, s_part, &total);
    __syncthreads();
    long long start = rows0 + at.rows;
    long long need[kPer], page_sum = 0;
    bool bad[kPer];
    int any = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c0 + tid * kPer + i;
      const long long rows = n[i] > 0 ? n[i] : 0, end = start + rows;
      bad[i] = c[i] < 0 || c[i] + rows > static_cast<long long>(a.MB) * kPage || (n[i] >= 0 && end > a.T);
      need[i] = bad[i] || n[i] < 0 ? 0 : pages_of(c[i] + rows) - pages_of(c[i]);
      page_sum += need[i];
      if (b < a.B && n[i] < 0 && !bad[i] && c[i] > 0) any = 1;
      if (mine && b < a.B && bad[i]) bits |= 0x2;  // PKV_DEV_BAD_LEN
      s_start[tid * kPer + i] = static_cast<int>(start < a.T ? start : a.T);
      s_end[tid * kPer + i] = static_cast<int>(end < a.T ? end : a.T);
      start = end;
    }
    if (any) s_any = 1;
    Sums page_total;
    const Sums pg = block_scan({0, page_sum}, s_part, &page_total);
    long long cum = pages0 + pg.pages;
    int alloc = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c0 + tid * kPer + i, k = tid * kPer + i;
      const long long before = cum;
      cum += need[i];
      const bool live = b < a.B && !bad[i] && n[i] >= 0;
      const bool served = live && (need[i] == 0 || cum <= count);
      if (served && need[i] > 0) alloc = static_cast<int>(cum);
      s_cached[k] = served ? c[i] : -1;
      s_ring[k] = served ? static_cast<int>(before < count ? before : count) : 0;
      if (mine && b < a.B) {
        a.context[b] = served ? c[i] + n[i] : 0;
        if (a.starts) a.starts[b + 1] = s_end[k];
        if (live && !served) bits |= 0x20;  // PKV_DEV_NO_PAGES
      }
    }
    if (alloc) atomicMax(&s_alloc, alloc);
    __syncthreads();
    // this block's rows of the chunk
    const int in_chunk = min(kChunk, a.B - c0);
    const int lo = s_start[0], hi = s_end[in_chunk - 1];
    for (long long t0 = static_cast<long long>(blockIdx.x) * kRowsPerBlock; t0 < hi;
         t0 += static_cast<long long>(gridDim.x) * kRowsPerBlock) {
      if (t0 + kRowsPerBlock <= lo) continue;
#pragma unroll
      for (int u = 0; u < kRowsPerBlock / kThreads; ++u) {
        const long long tl = t0 + u * kThreads + tid;
        if (tl < lo || tl >= hi) continue;
        const int t = static_cast<int>(tl);
        int l = 0, r = in_chunk - 1;  // the first request that ends behind row t
        while (l < r) {
          const int m = (l + r) >> 1;
          if (s_end[m] > t) r = m;
          else l = m + 1;
        }
        const int cached = s_cached[l];
        int slot = -1, pos = -1;
        if (cached >= 0) {
          const int p = cached + (t - s_start[l]);
          const int pn = p / kPage, have = (cached + kPage - 1) / kPage;
          int32_t* const entry = a.bt + static_cast<size_t>(c0 + l) * a.MB + pn;
          int page;
          if (pn >= have) {
            const long long q = static_cast<long long>(head) + s_ring[l] + (pn - have);
            page = a.ring[q >= a.N ? q - a.N : q];
            if (page < 0 || page >= a.N) page = -1;
            if (p % kPage == 0) *entry = page;
          } else {
            page = *entry;
          }
          if (page >= 0 && page < a.N) {
            slot = page * kPage + p % kPage;
            pos = p;
          } else {
            bits |= 0x1;  // PKV_DEV_BAD_PAGE
          }
        }
        a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
      }
    }
    rows0 += total.rows;
    pages0 += page_total.pages;
    __syncthreads();  // the chunk's arrays are free
  }
  // rows behind the last request: padding
  for (long long t = static_cast<long long>(blockIdx.x) * kThreads + tid; t < a.T;
       t += static_cast<long long>(gridDim.x) * kThreads) {
    if (t >= rows0) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
  }
  if (blockIdx.x == 0 && tid == 0 && a.starts) a.starts[0] = 0;

  // ---- the last block to finish returns pages and updates the pool
  if (gridDim.x > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(a.state + 2, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!s_last) {
      bits = __reduce_or_sync(0xffffffffu, bits);
      if (bits && lane == 0 && a.status) atomicOr(a.status, bits);
      return;
    }
    __threadfence();
  }
  const int alloc = s_alloc;
  const int room = a.N - (count - alloc);  // places for returned pages
  long long tail = static_cast<long long>(head) + count;
  int pushed = 0;
  if (s_any && pool_ok) {
    for (int c0 = 0; c0 < a.B; c0 += kChunk) {
      // page offsets of the chunk's ended requests, then all their table entries in order
      long long mine = 0;
      long long held[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = c0 + tid * kPer + i;
        const int c = b < a.B ? a.cached[b] : 0;
        const bool back = b < a.B && a.fresh[b] < 0 && c > 0 && c <= static_cast<long long>(a.MB) * kPage;
        held[i] = back ? pages_of(c) : 0;
        mine += held[i];
      }
      Sums total;
      long long at = block_scan({0, mine}, s_part, &total).pages;
      // (a pool holds at most 2^31 / 16 pages; more table entries than that are cut off)
      const int n = static_cast<int>(total.pages < 0x7fffffff ? total.pages : 0x7fffffff);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s_start[tid * kPer + i] = static_cast<int>(at < n ? at : n);
        at += held[i];
        s_end[tid * kPer + i] = static_cast<int>(at < n ? at : n);
      }
      __syncthreads();
      for (int j0 = 0; j0 < n; j0 += kThreads) {
        const int j = j0 + tid;
        int page = -1;
        if (j < n) {
          int l = 0, r = kChunk - 1;
          while (l < r) {
            const int m = (l + r) >> 1;
            if (s_end[m] > j) r = m;
            else l = m + 1;
          }
          page = a.bt[static_cast<size_t>(c0 + l) * a.MB + (j - s_start[l])];
          if (page >= a.N) bits |= 0x1;
        }
        const bool valid = page >= 0 && page < a.N;
        const unsigned votes = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) s_cnt[w] = __popc(votes);
        __syncthreads();
        int before = pushed + __popc(votes & ((1u << lane) - 1u)), all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          if (i < w) before += s_cnt[i];
          all += s_cnt[i];
        }
        if (valid) {
          if (before < room) a.ring[(tail + before) % a.N] = page;
          else bits |= 0x1;  // more pages than the pool has: returned twice
        }
        pushed += all;
        __syncthreads();
      }
      __syncthreads();
    }
    pushed = pushed < room ? pushed : room;
  }
  if (tid == 0) {
    if (pool_ok) {
      const long long h = static_cast<long long>(head) + alloc;
      a.state[0] = static_cast<int>(h >= a.N ? h - a.N : h);
      a.state[1] = count - alloc + pushed;
    }
    a.state[2] = 0;  // the ticket, ready for the next call
  }
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits && lane == 0 && a.status) atomicOr(a.status, bits);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_batch_tables(const pkv_page_pool* pool, const int32_t* cached_lens,
                                       const int32_t* new_lens, int32_t num_seqs,
                                       int32_t* block_tables, int32_t max_blocks_per_seq,
                                       int32_t* context_lens, int32_t* q_start_loc,
                                       int32_t* positions, int32_t* slot_mapping,
                                       int32_t max_tokens, int32_t* dev_status, void* stream) {
  PKV_RANGE("pkv_batch_tables");
  using pkv::aligned4;
  if (!pool || !pool->ring || !pool->state) return PKV_ERR_NULL;
  if (pool->page_size != pkv::kPage) return PKV_ERR_PAGE_SIZE;
  if (pool->num_pages < 1 || num_seqs < 0 || max_blocks_per_seq < 1 || max_tokens < 0)
    return PKV_ERR_SHAPE;
  if (static_cast<long long>(pool->num_pages) * pkv::kPage > 0x7fffffffLL ||
      static_cast<long long>(max_blocks_per_seq) * pkv::kPage > 0x7fffffffLL)
    return PKV_ERR_SHAPE;
  if (num_seqs > 0 && (!cached_lens || !new_lens || !block_tables || !context_lens))
    return PKV_ERR_NULL;
  if (max_tokens > 0 && !slot_mapping) return PKV_ERR_NULL;
  for (const void* p : {static_cast<const void*>(cached_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_tables), static_cast<const void*>(context_lens),
                        static_cast<const void*>(q_start_loc), static_cast<const void*>(positions),
                        static_cast<const void*>(slot_mapping), static_cast<const void*>(dev_status),
                        static_cast<const void*>(pool->ring), static_cast<const void*>(pool->state)})
    if (!aligned4(p)) return PKV_ERR_ALIGN;
  // blocks read every request's lengths while others write the outputs
  if (num_seqs > 0 && (context_lens == cached_lens || context_lens == new_lens))
    return PKV_ERR_UNSUPPORTED;
  pkv::TablesArgs a{cached_lens, new_lens,  block_tables, context_lens, q_start_loc,
                    positions,   slot_mapping, pool->ring, pool->state, dev_status,
                    num_seqs,    max_blocks_per_seq, pool->num_pages, max_tokens};
  long long blocks = (static_cast<long long>(max_tokens) + pkv::kRowsPerBlock - 1) / pkv::kRowsPerBlock;
  blocks = blocks < 1 ? 1 : blocks > pkv::kMaxBlocks ? pkv::kMaxBlocks : blocks;
  pkv::tables_kernel<<<static_cast<unsigned>(blocks), pkv::kThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
