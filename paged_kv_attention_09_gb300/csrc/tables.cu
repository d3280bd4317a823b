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
// page writes the table entry.  The last block also pushes the ended requests' pages: behind
// the free ones, so that the places written are never those that other blocks read new pages
// from.  The block that takes the last ticket (an atomic, no waiting: every block has read the
// pool's state by then) updates the state, so that a step works on the pool in place and can
// be replayed from a CUDA graph.
//
// Bound by latency, not bytes: a 256-request decode step moves 9 KB in 6.1 us (an empty launch
// takes about 2, the rest is four dependent round trips: lengths, pages or table entries, the
// ticket, the state).  A step of 511 requests with 32k prompt rows and ended requests takes
// 10.9 us, 14 with the ended requests' pages behind the other blocks' rows in one block.
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
// (A step of 32k rows: 11.5 us at 256, 10.9 at 1024, 12.9 at 2048.)
constexpr int kRowsPerBlock = 1024;
constexpr int kBackRounds = 8;  // returned pages per thread and round
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
  int32_t* state;  // head, free pages, ticket, pages returned
  int32_t* status;
  int B, MB, N, T;
};

// Prefix sums: new rows, new pages, and pages that ended requests return.
struct Sums {
  long long rows, need, back;
};

__device__ __forceinline__ Sums add(Sums a, Sums b) {
  return {a.rows + b.rows, a.need + b.need, a.back + b.back};
}

// Exclusive block-wide prefix sum; *total receives the block's sum.  The caller
// synchronises before `part` is used again.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Sums inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up{__shfl_up_sync(0xffffffffu, inc.rows, o), __shfl_up_sync(0xffffffffu, inc.need, o),
                  __shfl_up_sync(0xffffffffu, inc.back, o)};
    if (lane >= o) inc = add(inc, up);
  }
  if (lane == 31) part[w] = inc;
  __syncthreads();
  Sums base{0, 0, 0}, all{0, 0, 0};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const Sums p = part[i];
    if (i < w) base = add(base, p);
    all = add(all, p);
  }
  *total = all;
  return {base.rows + inc.rows - v.rows, base.need + inc.need - v.need, base.back + inc.back - v.back};
}

__device__ __forceinline__ long long pages_of(long long tokens) { return (tokens + kPage - 1) / kPage; }

// The first of n entries of ascending `end` that lies above x (there is one).
__device__ __forceinline__ int find_above(const int* end, int n, int x) {
  int l = 0, r = n - 1;
  while (l < r) {
    const int m = (l + r) >> 1;
    if (end[m] > x) r = m;
    else l = m + 1;
  }
  return l;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a) {
  __shared__ int s_end[kChunk];     // end row of each request of the chunk (at most T)
  __shared__ int s_start[kChunk];   // its first row
  __shared__ int s_cached[kChunk];  // its cached tokens, -1 when its rows get no slot
  __shared__ int s_ring[kChunk];    // ring offset of its first new page from the head
  __shared__ int s_back[kChunk];    // end of its returned pages among the chunk's
  __shared__ Sums s_part[kWarps];
  __shared__ int s_alloc;
  __shared__ int s_cnt[kBackRounds * kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int head0 = a.state[0], free0 = a.state[1];
  const bool pool_ok = head0 >= 0 && head0 < a.N && free0 >= 0 && free0 <= a.N;
  const int head = pool_ok ? head0 : 0, count = pool_ok ? free0 : 0;
  const long long cap = static_cast<long long>(a.MB) * kPage;
  if (tid == 0) s_alloc = 0;
  int bits = pool_ok || blockIdx.x ? 0 : 0x1;  // PKV_DEV_BAD_PAGE

  Sums before{0, 0, 0};  // sums over the chunks before
  for (int c0 = 0; c0 < a.B; c0 += kChunk) {
    const bool mine = (c0 / kChunk) % gridDim.x == blockIdx.x;  // this block writes the chunk's outputs
    int c[kPer], n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c0 + tid * kPer + i;
      c[i] = b < a.B ? a.cached[b] : 0;
      n[i] = b < a.B ? a.fresh[b] : 0;
    }
    Sums sum{0, 0, 0};
    long long need[kPer], back[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const long long rows = n[i] > 0 ? n[i] : 0;
      const bool bad = c[i] < 0 || c[i] + rows > cap;
      need[i] = bad || n[i] < 0 ? 0 : pages_of(c[i] + rows) - pages_of(c[i]);
      back[i] = bad || n[i] >= 0 ? 0 : pages_of(c[i]);
      sum = add(sum, {rows, need[i], back[i]});
    }
    Sums total;
    Sums at = block_scan(sum, s_part, &total);
    __syncthreads();
    if (before.rows + total.rows > a.T) {
      // some requests' rows pass the end of the row buffers: they get no pages
      long long end = before.rows + at.rows;
      sum = {0, 0, 0};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        end += n[i] > 0 ? n[i] : 0;
        if (end > a.T) need[i] = 0;
        sum.need += need[i];
      }
      Sums fitting;
      at.need = block_scan(sum, s_part, &fitting).need;
      total.need = fitting.need;
      __syncthreads();
    }
    long long start = before.rows + at.rows, cum = before.need + at.need, gone = at.back;
    int alloc = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c0 + tid * kPer + i, k = tid * kPer + i;
      const long long rows = n[i] > 0 ? n[i] : 0, end = start + rows, first = cum;
      const bool bad = c[i] < 0 || c[i] + rows > cap || (n[i] >= 0 && end > a.T);
      cum += need[i];
      gone += back[i];
      const bool live = b < a.B && !bad && n[i] >= 0;
      const bool served = live && (need[i] == 0 || cum <= count);
      if (served && need[i] > 0) alloc = static_cast<int>(cum);
      s_start[k] = static_cast<int>(start < a.T ? start : a.T);
      s_end[k] = static_cast<int>(end < a.T ? end : a.T);
      s_cached[k] = served ? c[i] : -1;
      s_ring[k] = served ? static_cast<int>(first < count ? first : count) : 0;
      s_back[k] = static_cast<int>(gone < 0x7fffffff ? gone : 0x7fffffff);
      if (mine && b < a.B) {
        a.context[b] = served ? c[i] + n[i] : 0;
        if (a.starts) a.starts[b + 1] = s_end[k];
        if (bad) bits |= 0x2;             // PKV_DEV_BAD_LEN
        if (live && !served) bits |= 0x20;  // PKV_DEV_NO_PAGES
      }
      start = end;
    }
    if (alloc) atomicMax(&s_alloc, alloc);
    before = add(before, total);
    __syncthreads();
    // this block's rows of the chunk
    const int in_chunk = min(kChunk, a.B - c0);
    const int lo = s_start[0], hi = s_end[in_chunk - 1];
    for (long long t0 = static_cast<long long>(blockIdx.x) * kRowsPerBlock; t0 < hi;
         t0 += static_cast<long long>(gridDim.x) * kRowsPerBlock) {
      if (t0 + kRowsPerBlock <= lo) continue;
      // the rows' pages are fetched together, before any table entry is written
      constexpr int R = kRowsPerBlock / kThreads;
      int page[R], p[R];
      int32_t* entry[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const long long t = t0 + u * kThreads + tid;
        page[u] = p[u] = -1;
        entry[u] = nullptr;
        if (t < lo || t >= hi) continue;
        const int l = find_above(s_end, in_chunk, static_cast<int>(t));
        const int cached = s_cached[l];
        if (cached < 0) continue;
        p[u] = cached + (static_cast<int>(t) - s_start[l]);
        const int pn = p[u] / kPage, have = (cached + kPage - 1) / kPage;
        int32_t* const e = a.bt + static_cast<size_t>(c0 + l) * a.MB + pn;
        if (pn >= have) {
          const long long q = static_cast<long long>(head) + s_ring[l] + (pn - have);
          page[u] = a.ring[q >= a.N ? q - a.N : q];
          if (p[u] % kPage == 0) entry[u] = e;
        } else {
          page[u] = *e;
        }
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const long long t = t0 + u * kThreads + tid;
        if (t < lo || t >= hi) continue;
        const bool good = page[u] >= 0 && page[u] < a.N;
        if (entry[u]) *entry[u] = good ? page[u] : -1;
        if (p[u] >= 0 && !good) bits |= 0x1;  // PKV_DEV_BAD_PAGE
        a.slots[t] = p[u] >= 0 && good ? page[u] * kPage + p[u] % kPage : -1;
        if (a.positions) a.positions[t] = good ? p[u] : -1;
      }
    }
    if (c0 + kChunk < a.B) __syncthreads();  // the chunk's arrays are free
  }
  // rows behind the last request: padding
  for (long long t = static_cast<long long>(blockIdx.x) * kThreads + tid; t < a.T;
       t += static_cast<long long>(gridDim.x) * kThreads) {
    if (t >= before.rows) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
  }
  if (blockIdx.x == 0 && tid == 0 && a.starts) a.starts[0] = 0;

  // ---- the last block's share: pages of ended requests go back
  const int room = a.N - count;  // places behind the free pages (more pages than that were
                                 // returned twice)
  const long long tail = static_cast<long long>(head) + count;
  int pushed = 0;
  if (blockIdx.x == gridDim.x - 1 && before.back > 0 && pool_ok) {
    for (int c0 = 0; c0 < a.B; c0 += kChunk) {
      if (a.B > kChunk) {  // (a single chunk's offsets are still in place)
        __syncthreads();
        long long back[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int b = c0 + tid * kPer + i;
          const int c = b < a.B ? a.cached[b] : 0;
          back[i] = b < a.B && a.fresh[b] < 0 && c > 0 && c <= cap ? pages_of(c) : 0;
          sum += back[i];
        }
        Sums total;
        long long gone = block_scan({0, 0, sum}, s_part, &total).back;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          gone += back[i];
          s_back[tid * kPer + i] = static_cast<int>(gone < 0x7fffffff ? gone : 0x7fffffff);
        }
        __syncthreads();
      }
      const int n = s_back[kChunk - 1];
      // table entries in request and page order, kBackRounds of them a thread at a time;
      // valid ones are numbered by counting them warp by warp
      for (long long j0 = 0; j0 < n; j0 += kBackRounds * kThreads) {
        int page[kBackRounds];
#pragma unroll
        for (int u = 0; u < kBackRounds; ++u) {
          const long long j = j0 + u * kThreads + tid;
          page[u] = -1;
          if (j < n) {
            const int l = find_above(s_back, kChunk, static_cast<int>(j));
            const int first = l ? s_back[l - 1] : 0;
            page[u] = a.bt[static_cast<size_t>(c0 + l) * a.MB + (j - first)];
          }
        }
        unsigned votes[kBackRounds];
#pragma unroll
        for (int u = 0; u < kBackRounds; ++u) {
          if (page[u] >= a.N) {
            bits |= 0x1;
            page[u] = -1;
          }
          votes[u] = __ballot_sync(0xffffffffu, page[u] >= 0);
          if (lane == 0) s_cnt[u * kWarps + w] = __popc(votes[u]);
        }
        __syncthreads();
        int all = pushed;
#pragma unroll
        for (int u = 0; u < kBackRounds; ++u) {
          int mine = 0;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            if (i == w) mine = all + __popc(votes[u] & ((1u << lane) - 1u));
            all += s_cnt[u * kWarps + i];
          }
          if (page[u] >= 0) {
            if (mine < room) a.ring[(tail + mine) % a.N] = page[u];
            else bits |= 0x1;  // more pages than the pool has: returned twice
          }
        }
        pushed = all;
        __syncthreads();
      }
    }
    pushed = pushed < room ? pushed : room;
  }
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits && lane == 0 && a.status) atomicOr(a.status, bits);

  // ---- the pool's state
  __syncthreads();
  if (tid != 0) return;
  if (gridDim.x > 1) {
    if (blockIdx.x == gridDim.x - 1) a.state[3] = pushed;
    __threadfence();
    if (atomicAdd(a.state + 2, 1) != static_cast<int>(gridDim.x) - 1) return;
    __threadfence();
    pushed = *static_cast<volatile int32_t*>(a.state + 3);
  }
  if (pool_ok) {
    const long long h = static_cast<long long>(head) + s_alloc;
    a.state[0] = static_cast<int>(h >= a.N ? h - a.N : h);
    a.state[1] = count - s_alloc + pushed;
  }
  a.state[2] = a.state[3] = 0;  // ready for the next call
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
  const long long bytes = 4ll * num_seqs;
  for (const int32_t* in : {cached_lens, new_lens}) {
    const long long apart = reinterpret_cast<const char*>(context_lens) - reinterpret_cast<const char*>(in);
    if (apart < bytes && -apart < bytes) return PKV_ERR_UNSUPPORTED;
  }
  pkv::TablesArgs a{cached_lens, new_lens,  block_tables, context_lens, q_start_loc,
                    positions,   slot_mapping, pool->ring, pool->state, dev_status,
                    num_seqs,    max_blocks_per_seq, pool->num_pages, max_tokens};
  long long blocks = (static_cast<long long>(max_tokens) + pkv::kRowsPerBlock - 1) / pkv::kRowsPerBlock;
  blocks = blocks < 1 ? 1 : blocks > pkv::kMaxBlocks ? pkv::kMaxBlocks : blocks;
  pkv::tables_kernel<<<static_cast<unsigned>(blocks), pkv::kThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
