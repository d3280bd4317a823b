// prefill_blk.cu — chunked-prefill attention over a block-scaled 8-bit cache on the
// 5th-generation tensor cores (tcgen05).
//
// out[row] = sum_t softmax_t(scale q[row] . (s_k code_k[t])) s_v code_v[t] over the keys t
// that the row sees (causal, and the last `window` of them), s_k and s_v the scales of the
// token's (page, kv head) block.  Codes (INT8, E4M3) are exact in FP16, so the products take
// the codes themselves and the scales stay outside, in FP32: s_k multiplies a page's 16
// scores, s_v its 16 probabilities.
//
// One block computes 128 query rows, (chunk token, query head) pairs of one GQA group,
// token-major, against the group's keys in tiles of 128 (8 pages):
//   warps 18-20  K: each takes every third run of 64 keys (4 pages).  Its codes come by bulk
//                copies into a slot of the warp's own, requested as soon as the slot is free
//                (a warp fetches for itself: no hand-over), and are written as FP16 operand
//                blocks (no-swizzle K-major core matrices); the pages' scales are copied into
//                a ring of eight tiles;
//   warps 21-23  V: the same; codes of keys that no row sees become zero (a stale E4M3 NaN
//                would survive a zero probability).  (Two warps for float queries, whose
//                second operand tile takes the room.)  A shared-memory round trip takes some
//                150 cycles in this kernel, so a page's loads are in flight together and every
//                wait, fence and arrival stands for 64 keys: one page a time and warp, each with
//                its own, took 2700 cycles a page;
//   warp 16      one thread issues S(i) = Q K^T (M = 128, N = 128) into one of two (head_dim 64:
//                three) score buffers of TMEM, warp 17 one thread O += P(i) V (M = 128, N = head_dim):
//                two issuers, since each barrier that one asks costs it as much as two MMAs;
//   warps 0-15   softmax, four threads per row, 32 keys each.  They share the row's running
//                maximum: it is raised only when a score passes it by 2^8, so nearly every
//                tile costs the four warps of 32 rows one barrier with a vote, not an exchange.  P overwrites
//                its own scores in TMEM, page by page (8 columns of FP16 high parts, 8 of
//                remainders: P keeps ~22 bits, two MMAs per page), so that the score buffers
//                fit beside O and the sum of its earlier segments (kSegment).
// What bounds it: a tile takes ~2500 cycles, of which the softmax's exponentials take 1024 on
// the special-function pipe; they do not overlap with the same warps' loads, votes and waits
// (~1300), since the four warps of a scheduler are the four parts of the same rows.  The MMAs
// take 1600 and the fills less.  Measured (cycles a tile; 4 x 512 tokens over 4096, 12 / 2 heads
// of 128, FP8B): 4400 with the codes through registers or asynchronous copies and one MMA
// issuer, 3300 with whole runs of 64 keys per warp and no bank conflicts, 2600 with two issuers.
// That workload: 54.3 us, 627 TFLOP/s; 2 chunks of 512 over 2048: 34.7 us; one chunk of 37: 8.7 us.
//
// Range of FP16: query rows are brought to [2^13, 2^14) by a power of two that goes into the
// score scale (float queries as high part + remainder); probabilities carry the V scale as
// 2^(log2 s_v + lg), lg raised or lowered when a page's scale leaves the range, so that
// P s_v stays below 2^15; the sum takes P s_v / 2^(log2 s_v + lg) back off.
// Every wait is bounded.
#include <cuda_fp16.h>
#include <math_constants.h>

#include <mutex>

#include "internal.h"
#include "prefill.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kParts = 4;                // softmax threads per query row
constexpr int kSoftWarps = 4 * kParts;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMmaWarp = kSoftWarps;
constexpr int kPvWarp = kMmaWarp + 1;
constexpr int kKWarp = kPvWarp + 1;
constexpr int kKWarps = 3;                // warps that fill the K ring
constexpr int kVWarp = kKWarp + kKWarps;
constexpr int kKeysB = 128;               // keys per tile
constexpr int kPagesB = kKeysB / kPage;
constexpr int kPartKeys = kKeysB / kParts, kPartPages = kPagesB / kParts;
// Key tiles whose products one accumulator takes.  The tensor core adds with truncation: over n
// additions a sum loses about n 2^-25 of itself, and a tile adds 16 times.  (Error of 512 rows over
// 2048 keys, relative, and time of 4 x 512 over 4096: segments of 2 tiles 0.4e-6, 57.0 us; 4 tiles
// 0.8e-6, 55.0; 8 tiles 1.7e-6, 54.1; one accumulator 4.3e-6, 52.9.  A sum in FP32 with rounding,
// key by key: 0.9e-6.)
constexpr int kSegment = 4;
constexpr int kScaleSlots = 8;
constexpr float kGainTop = 7.f;          // log2 of the largest scaled V scale

#ifdef PKV_TEST_HOOKS
// Test builds only: the softmax threads' first wait for scores gives up at once.
__device__ int g_test_prefill_blk_fail_first_wait = 0;
#endif

template <int D, bool QSPLIT>
struct BSmem {
  static constexpr int blk = kPage * D * 2;          // one FP16 page block (K or V)
  static constexpr int qTile = kRowsTC * D * 2;      // one FP16 query tile
  static constexpr int half = kPagesTC * blk;        // operand blocks of 64 keys
  static constexpr int SB = D == 128 ? 2 : 3;        // score buffers
  static constexpr int KST = 2;                      // K ring: tiles
  static constexpr int VST = QSPLIT ? 3 : 4;         // V ring: halves
  static constexpr int VW = QSPLIT ? 2 : 3;          // warps that fill the V ring
  static constexpr int threads = (kVWarp + VW) * 32;
  static constexpr int page = kPage * D;             // a page's codes
  static constexpr int raw = kPagesTC * page;        // a warp's slot: the codes of 64 keys
  static constexpr int q0 = 0;
  static constexpr int k0 = q0 + (QSPLIT ? 2 : 1) * qTile;
  static constexpr int v0 = k0 + KST * 2 * half;
  static constexpr int rk0 = v0 + VST * half;
  static constexpr int rv0 = rk0 + kKWarps * raw;
  // scales of a tile's pages: K [8], V [8]
  static constexpr int sc0 = rv0 + VW * raw;
  static constexpr int scSlot = 2 * kPagesB * 4;
  static constexpr int bar0 = sc0 + kScaleSlots * scSlot;
  // barriers by index
  static constexpr int kFull = 0, kEmpty = 2, vFull = 4, vEmpty = 8, sFull = 12, pFull = 15, oDone = 18,
                       fin = 21, qFull = 22, rawFull = 23, nbars = rawFull + kKWarps + VW;
  // (A wait by parity tells a phase only from the one before it.  sFull, pFull and oDone are one
  // barrier per score buffer: S(i + SB) waits for the products of tile i, so that on each of
  // them whoever waits for tile i does so after tile i - SB and before tile i + SB.)
  static constexpr int misc0 = bar0 + (nbars + nbars % 2) * 8;  // TMEM base address, abort flag; failed waits of the softmax quarters
  // row values exchanged by the softmax threads [part][row]; then the split merge's weights
  static constexpr int xch0 = misc0 + 32;
  static constexpr int total = xch0 + kParts * kRowsTC * 4;
  // TMEM columns: O [0, D), the earlier segments' sum [D, 2 D), then score buffers of 128
  // columns (part h's 32 keys at + 32 h)
  static constexpr int tCol = D, sCol = 2 * D;
  static constexpr int tmemCols = 512;
  static_assert(sCol + SB * kKeysB <= 512, "tensor memory");
  static_assert(total <= 227 * 1024, "shared memory");
};

// The four softmax warps of one TMEM lane quarter hold the four parts of the same 32 rows;
// quarters are independent of each other.  A vote of a quarter's threads (and their barrier),
// and their barrier alone.
__device__ __forceinline__ bool quarter_any(int quarter, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(1 + quarter), "n"(32 * kParts)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void quarter_sync(int quarter) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(5 + quarter), "n"(32 * kParts) : "memory");
}

// Four stored bytes -> their four code values in FP16, in order.
template <bool FP8>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FP8) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {  // byte b = code + 128 -> the f16 1024 + b, less 1152
    uint32_t a, b;
    asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(w), "r"(0x64646464u));
    asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(w), "r"(0x64646464u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}
// 4 bytes global -> shared asynchronously, and the groups they complete in.
__device__ __forceinline__ void fetch4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the N latest groups have landed
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16 stored bytes -> two 16-byte operand rows of 8 FP16 values, 128 bytes apart.
template <bool FP8>
__device__ __forceinline__ void store_codes16(uint8_t* dst, uint4 c) {
  uint4 a, b;
  codes4<FP8>(c.x, a.x, a.y);
  codes4<FP8>(c.y, a.z, a.w);
  codes4<FP8>(c.z, b.x, b.y);
  codes4<FP8>(c.w, b.z, b.w);
  *reinterpret_cast<uint4*>(dst) = a;
  *reinterpret_cast<uint4*>(dst + 128) = b;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (a, b) -> f16x2 high part and f16x2 remainder
__device__ __forceinline__ void split2(float2 a, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __float22half2_rn(a);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  float x, y;  // a - h, each one multiply-add of the FP16 part by -1
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.f16 %0, l, %5, %3;\n\tfma.rn.f32.f16 %1, h, %5, %4;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(hi), "f"(a.x), "f"(a.y), "h"(static_cast<unsigned short>(0xBC00)));
  const __half2 r = __floats2half2_rn(x, y);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

template <bool FP8, int D, bool QSPLIT>
__global__ void __launch_bounds__(BSmem<D, QSPLIT>::threads, 1)
    prefill_blk_kernel(const __grid_constant__ TParams p) {
  using Sm = BSmem<D, QSPLIT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::bar0);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sm::misc0);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Sm::misc0 + 4);
  volatile int* soft_fail = reinterpret_cast<volatile int*>(smem + Sm::misc0 + 16);
  __shared__ int s_err;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int tile = blockIdx.x / p.ksplit, ks = blockIdx.x % p.ksplit;
  const int row0 = tile * kRowsTC;
  // the warps that fetch codes: their place among K's or V's, and the first page ids, read
  // together with the lengths where the range's first page does not depend on those
  const bool fills = warp >= kKWarp, isK = warp < kVWarp;
  const int step = isK ? kKWarps : Sm::VW, w = warp - (isK ? kKWarp : kVWarp);
  const int q_first = kPagesTC * w + (lane & 3);
  const bool early = p.window == 0 && ks == 0;
  int ids = fills && early && q_first < p.MB ? p.bt[static_cast<size_t>(b) * p.MB + q_first] : -1;
  const int q0 = p.qsl[b];
  const int Lq = p.qsl[b + 1] - q0;
  const int L = p.lens[b];
  const int nrows = Lq > 0 ? Lq * p.G : 0;
  if (row0 >= nrows) return;

  int err = 0;
  if (L < 0 || L > p.MB * kPage) err |= 0x2;  // PKV_DEV_BAD_LEN
  if (Lq > L) err |= 0x8;                     // PKV_DEV_BAD_CHUNK
  const int last_row = min(row0 + kRowsTC, nrows) - 1;
  const int p_first = L - Lq + row0 / p.G;
  const int p_last = L - Lq + last_row / p.G;
  const int n_keys0 = err ? 0 : p_last + 1;
  // Sliding window of W tokens: row position pos sees keys pos - W + 1 .. pos; keys below
  // lo_blk are seen by no row of the block, keys below lo_max by some rows only.  Tiles are
  // counted from kb0, the first key of the page holding lo_blk.
  const int win = p.window;
  const int lo_blk = win > 0 ? max(0, p_first - win + 1) : 0;
  const int lo_max = win > 0 ? p_last - win + 1 : 0;
  const int kb0 = (lo_blk / kPage) * kPage;
  // this block's share of the key tiles: [t0, t1) of the row tile's range
  const int nt_all = err ? 0 : (n_keys0 - kb0 + kKeysB - 1) / kKeysB;
  const int t0 = ks * nt_all / p.ksplit, t1 = (ks + 1) * nt_all / p.ksplit;
  const int n_keys = err ? 0 : min(n_keys0, kb0 + t1 * kKeysB);
  const int kbase = err ? 0 : kb0 + t0 * kKeysB;
  const int n_pages = max(0, (n_keys - kbase + kPage - 1) / kPage);  // pages from kbase on
  const int n_tiles = t1 - t0;
  const int32_t* btw = p.bt + static_cast<size_t>(b) * p.MB + kbase / kPage;

  // ---- what a block's start waits for goes out before it is set up: the first codes and the
  // query rows.  A page id outside the pool is replaced by page 0 (every read stays inside the
  // cache) and flagged: the block's rows then become NaN.
  bool bad = false;
  auto checked = [&](int q, int id) -> int {  // -1: no such page
    if (q >= n_pages) return -1;
    if (id >= 0 && id < p.num_pages) return id;
    bad = true;
    return 0;
  };
  auto page_id = [&](int q) -> int { return checked(q, q < n_pages ? btw[q] : -1); };
  const int n_halves = 2 * n_tiles;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t slot = sbase + (isK ? Sm::rk0 : Sm::rv0) + w * Sm::raw;
  const uint32_t bar = smem_u32(&bars[Sm::rawFull + warp - kKWarp]);
  auto request = [&](int h) {  // the copies of run h, h = w, w + step, ...
    if (h < n_halves) {
      const int n = min(kPagesTC, max(0, n_pages - kPagesTC * h));  // its pages
      mbar_arrive_expect_tx_if(lane == 0, bar, n * Sm::page);
      const bool there = lane < n;
      const size_t blk = there ? static_cast<size_t>(ids) * p.Hkv + g : 0;
      __syncwarp();
      bulk_g2s_if(there, slot + lane * Sm::page, (isK ? p.k : p.v) + blk * Sm::page, Sm::page, bar,
                  l2_evict_last_policy());  // every row tile of the group rereads them
      if (isK && lane < kPagesTC) {
        const uint32_t at = sbase + Sm::sc0 + (h >> 1) % kScaleSlots * Sm::scSlot + ((h & 1) * kPagesTC + lane) * 4;
        if (there) {
          fetch4(at, p.ks + blk);
          fetch4(at + 4 * kPagesB, p.vs + blk);
        } else {  // no page: zeros (its keys are masked)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0) : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4 * kPagesB), "r"(0) : "memory");
        }
      }
      // the ids of the warp's next 64 keys (lanes 0 .. 3), loaded one run ahead: read when
      // needed they would cost a global round trip
      ids = page_id(kPagesTC * (h + step) + (lane & 3));
    }
    fetch_commit();
  };
  // softmax threads: row r (= TMEM lane 32 (warp % 4) + lane), part of the row
  const int r = tid & (kRowsTC - 1);
  const int part = tid / kRowsTC;
  const int rho = row0 + r;
  const bool valid_row = tid < kSoftThreads && rho < nrows;
  constexpr int N = D / kParts;                       // its columns of the query row
  constexpr int QN = QSPLIT ? N / 4 : N / 8;          // in 16-byte pieces
  uint4 qraw[QN];
#pragma unroll
  for (int i = 0; i < QN; ++i) qraw[i] = make_uint4(0u, 0u, 0u, 0u);
  if (n_tiles > 0) {
    if (fills) {
      if (lane == 0) {
        mbar_init(&bars[Sm::rawFull + warp - kKWarp], 1);
        fence_barrier_init();
      }
      __syncwarp();
      ids = checked(q_first, early || q_first >= n_pages ? ids : btw[q_first]);
      request(w);
    } else if (valid_row) {
      const size_t at = (static_cast<size_t>(q0 + rho / p.G) * p.Hq + g * p.G + rho % p.G) * D + N * part;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) + at * (QSPLIT ? 4 : 2));
#pragma unroll
      for (int i = 0; i < QN; ++i) qraw[i] = src[i];
    }
  }

  // ---- set-up: TMEM and barriers
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, Sm::tmemCols);
    tc::tmem_relinquish();
  }
  if (tid < Sm::rawFull) {
    const int i = tid;
    const int count = i >= Sm::kFull && i < Sm::kFull + Sm::KST     ? 2   // its halves
                      : (i >= Sm::pFull && i < Sm::pFull + Sm::SB) || i == Sm::qFull ? kSoftWarps
                      : i == Sm::fin                                ? 2  // one from each MMA issuer
                                                                    : 1;
    mbar_init(&bars[i], count);
    fence_barrier_init();
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) soft_fail[i] = 0;
    s_err = err;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  const int quarter = warp & 3;

  constexpr int UPP = D / 32;  // units of 32 pieces of 16 codes per page
  if (n_tiles > 0 && fills) {
    // ---------------------------------------------------------------- K and V codes
    bool ok = true;
    uint32_t phase = 0;
    int h = w;
    // K: thread -> 16 codes of one token, a piece of its D / 16.  The 8 lanes of a quarter warp
    // take 8 tokens along a diagonal, so that both their loads (rows of D bytes) and their
    // stores (16-byte rows of core matrices) fall into different banks.  V: the 16 tokens of
    // one head-dim row, unit u: rows 32 u .. + 31.
    uint32_t from[UPP], to[UPP];
#pragma unroll
    for (int u = 0; u < UPP; ++u) {
      const int l = lane & 7, k = lane >> 3;
      const int row = l + 8 * (D == 128 ? u >> 1 : u);
      const int piece = D == 128 ? (l + k + 4 * (u & 1)) & 7 : ((l >> 1) + k) & 3;
      from[u] = slot + (isK ? row * D + piece * 16 : lane * 16 + 512 * u);
      to[u] = isK ? tile_off(row, 16 * piece, D) : bf16_v_off(lane, 0) + 1024 * u;
    }
    for (; h < n_halves; h += step, phase ^= 1) {
      const int j = h >> 1, st = isK ? j % Sm::KST : h % Sm::VST, use = isK ? j / Sm::KST : h / Sm::VST;
      if (use > 0)
        ok = mbar_wait_warp(smem_u32(&bars[(isK ? Sm::kEmpty : Sm::vEmpty) + st]), (use - 1) & 1);
      ok = mbar_wait_warp(bar, phase) && ok;
      if (!ok) break;
      uint8_t* const dst = smem + (isK ? Sm::k0 + (2 * st + (h & 1)) * Sm::half : Sm::v0 + st * Sm::half);
      const int key0 = kbase + h * kKeysTC;
      const int n = min(kPagesTC, max(0, n_pages - kPagesTC * h));
      const bool edge = !isK && (key0 < lo_blk || key0 + kKeysTC > n_keys);
      auto load = [&](int q, uint4 (&c)[UPP]) {
#pragma unroll
        for (int u = 0; u < UPP; ++u) c[u] = lds_u4(from[u] + q * Sm::page);
      };
      uint4 cur[UPP], nxt[UPP];
      load(0, cur);
#pragma unroll
      for (int q = 0; q < kPagesTC; ++q) {
        if (q + 1 < kPagesTC) load(q + 1, nxt);
        if (q >= n) {
#pragma unroll
          for (int u = 0; u < UPP; ++u) cur[u] = make_uint4(0u, 0u, 0u, 0u);
        } else if (edge) {  // only tokens that some row sees
          const int key = key0 + q * kPage;
          uint32_t m[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            m[v] = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = key + 4 * v + e;
              if (t >= lo_blk && t < n_keys) m[v] |= 0xffu << (8 * e);
            }
          }
#pragma unroll
          for (int u = 0; u < UPP; ++u) {
            cur[u].x &= m[0]; cur[u].y &= m[1]; cur[u].z &= m[2]; cur[u].w &= m[3];
          }
        }
#pragma unroll
        for (int u = 0; u < UPP; ++u) {
          store_codes16<FP8>(dst + q * Sm::blk + to[u], cur[u]);
          cur[u] = nxt[u];
        }
      }
      fence_proxy_async_smem();
      fetch_wait<0>();  // this run's scales
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[(isK ? Sm::kFull : Sm::vFull) + st]);
      request(h + step);  // (every lane has read the slot)
    }
    if (!ok) *abort_flag = 1;
    // leave nothing in flight
    fetch_wait<0>();
    if (h < n_halves) (void)mbar_wait_warp(bar, phase);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&s_err, 0x1);  // PKV_DEV_BAD_PAGE
  } else if (n_tiles > 0 && (warp == kMmaWarp || warp == kPvWarp)) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_f16_f32(kRowsTC, kKeysB);
      constexpr uint32_t idO = tc::idesc_f16_f32(kRowsTC, D);
      constexpr uint32_t sboQK = (D / 8) * 128;  // 8-row groups of Q and of K
      const uint64_t dQhi = tc::smem_desc(sbase + Sm::q0, 128, sboQK);
      const uint64_t dQlo = tc::smem_desc(sbase + Sm::q0 + Sm::qTile, 128, sboQK);
      const uint64_t dK0 = tc::smem_desc(sbase + Sm::k0, 128, sboQK);
      const uint64_t dV0 = tc::smem_desc(sbase + Sm::v0, 128, 256);
      auto done_bar = [&](int i) { return &bars[Sm::oDone + i % Sm::SB]; };
      bool ok = true;
      if (warp == kMmaWarp) {
        // S of tile i, once its K is there and the last readers of its buffer, the P.V products
        // of tile i - SB, have completed
        ok = mbar_wait(&bars[Sm::qFull], 0);
        for (int i = 0; i < n_tiles && ok; ++i) {
          ok = (i < Sm::SB || mbar_wait(done_bar(i - Sm::SB), ((i - Sm::SB) / Sm::SB) & 1)) &&
               mbar_wait(&bars[Sm::kFull + i % Sm::KST], (i / Sm::KST) & 1) && !*abort_flag;
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t dK = tc::desc_add(dK0, (i % Sm::KST) * 2 * Sm::half);
          const uint32_t tS = tmem + Sm::sCol + kKeysB * (i % Sm::SB);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t bd = tc::desc_add(dK, k * 256);
            tc::mma_bf16(tS, tc::desc_add(dQhi, k * 256), bd, idS, k > 0);
            if constexpr (QSPLIT) tc::mma_bf16(tS, tc::desc_add(dQlo, k * 256), bd, idS, true);
          }
          tc::commit(&bars[Sm::sFull + i % Sm::SB]);
          tc::commit(&bars[Sm::kEmpty + i % Sm::KST]);
        }
      } else {
        // O += P V of tile i
        for (int i = 0; i < n_tiles && ok; ++i) {
          for (int h = 2 * i; h < 2 * i + 2 && ok; ++h)
            ok = mbar_wait(&bars[Sm::vFull + h % Sm::VST], (h / Sm::VST) & 1);
          ok = ok && mbar_wait(&bars[Sm::pFull + i % Sm::SB], (i / Sm::SB) & 1) && !*abort_flag;
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t tP = tmem + Sm::sCol + kKeysB * (i % Sm::SB);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int st = (2 * i + y) % Sm::VST;
            const uint64_t dV = tc::desc_add(dV0, st * Sm::half);
#pragma unroll
            for (int q = 0; q < kPagesTC; ++q) {
              const uint64_t bd = tc::desc_add(dV, q * Sm::blk);
#pragma unroll
              for (int half = 0; half < 2; ++half)
                tc::mma_bf16_ts(tmem, tP + 16 * (kPagesTC * y + q) + 8 * half, bd, idO,
                                !(i % kSegment == 0 && y == 0 && q == 0 && half == 0));
            }
            tc::commit(&bars[Sm::vEmpty + st]);
          }
          tc::commit(done_bar(i));
        }
      }
      if (!ok) *abort_flag = 1;
      // every MMA has completed before TMEM is released
      tc::commit(&bars[Sm::fin]);
      (void)mbar_wait(&bars[Sm::fin], 0);
    }
  } else if (n_tiles > 0 && warp < kSoftWarps) {
    // ---------------------------------------------------------------- the query rows
    // each thread brings its part of its row's columns; the parts exchange their largest
    // value, and the row becomes FP16 in [2^13, 2^14)
    float* xch = reinterpret_cast<float*>(smem + Sm::xch0);  // [part][row]
    float rs;
    {
      float x[N];
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        const uint32_t w4[4] = {qraw[i].x, qraw[i].y, qraw[i].z, qraw[i].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if constexpr (QSPLIT) {
            x[4 * i + u] = __uint_as_float(w4[u]);
          } else {
            x[8 * i + 2 * u] = __uint_as_float(w4[u] << 16);
            x[8 * i + 2 * u + 1] = __uint_as_float(w4[u] & 0xffff0000u);
          }
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
      xch[part * kRowsTC + r] = top;
      quarter_sync(quarter);
#pragma unroll
      for (int i = 0; i < kParts; ++i) top = fmaxf(top, xch[i * kRowsTC + r]);
      // top in [2^(e-1), 2^e): times 2^k, k = 14 - e
      const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xffu) - 126;
      const int k = min(14 - e, 126);
      // (a negative softmax scale turns the query round)
      const float f = copysignf(__uint_as_float(static_cast<uint32_t>(127 + k) << 23), p.scale_log2);
      rs = ldexpf(fabsf(p.scale_log2), -k);
      uint8_t* qhi = smem + Sm::q0;
#pragma unroll
      for (int c = 0; c < N / 8; ++c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          split2(make_float2(x[8 * c + 2 * u] * f, x[8 * c + 2 * u + 1] * f), h[u], l[u]);
        const uint32_t off = tile_off(r, N * part + 8 * c, D);
        *reinterpret_cast<uint4*>(qhi + off) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (QSPLIT) *reinterpret_cast<uint4*>(qhi + Sm::qTile + off) = make_uint4(l[0], l[1], l[2], l[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Sm::qFull]);
    }
    // ---------------------------------------------------------------- softmax rows
    const int pos = valid_row ? L - Lq + rho / p.G : p_first;
    const int lo_row = win > 0 ? pos - win + 1 : 0;  // first key of the row's window
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    constexpr int DP = D / kParts;  // columns of O that this thread rescales and writes
    const uint32_t tO = tmem + lane_base + DP * part, tT = tO + Sm::tCol;
    float m_used = -CUDART_INF_F, l = 0.f;
    float lg = 100.f;  // log2 of the gain on the V scales (the first tile brings it down)
    bool ok = true;
    // A quarter's threads pass the same barriers in every tile, whatever happens: a wait that
    // gave up only raises soft_fail, which all of them see in the same tile.
    int i = 0;
    for (; i < n_tiles; ++i) {
      ok = mbar_wait_warp(smem_u32(&bars[Sm::sFull + i % Sm::SB]), (i / Sm::SB) & 1) && ok;
#ifdef PKV_TEST_HOOKS
      if (i == 0 && g_test_prefill_blk_fail_first_wait) ok = false;  // a wait that gives up
#endif
      tc::fence_after_sync();
      const uint32_t tS = tmem + lane_base + Sm::sCol + kKeysB * (i % Sm::SB) + kPartKeys * part;
      const float* sc = reinterpret_cast<const float*>(smem + Sm::sc0 + (i % kScaleSlots) * Sm::scSlot);
      const float2 k2 = *reinterpret_cast<const float2*>(sc + kPartPages * part);
      const float2 v2 = *reinterpret_cast<const float2*>(sc + kPagesB + kPartPages * part);
      // (never 0: a masked score of -inf has to stay -inf; 1e-37 takes every score to 0)
      constexpr float kTiny = 1e-37f;
      const float kf[2] = {fmaxf(k2.x * rs, kTiny), fmaxf(k2.y * rs, kTiny)};
      const float lv[2] = {fast_log2(v2.x), fast_log2(v2.y)};  // (-inf: a page of zeros, or none)
      const float4 va = *reinterpret_cast<const float4*>(sc + kPagesB), vb = *reinterpret_cast<const float4*>(sc + kPagesB + 4);
      const float lv_top = fast_log2(fmaxf(fmax3(fmax3(va.x, va.y, va.z), fmax3(va.w, vb.x, vb.y), vb.z), vb.w));
      float s[kPartKeys];
      __syncwarp();
      tc::ld32(tS, s);
      const int key0 = kbase + i * kKeysB + kPartKeys * part;
      if (key0 + kPartKeys - 1 > p_first || key0 + kPartKeys > n_keys || key0 < lo_max) {
#pragma unroll
        for (int u = 0; u < kPartKeys; ++u)
          s[u] = (key0 + u <= pos && key0 + u >= lo_row) ? s[u] : -CUDART_INF_F;
      }
      // largest score: raw per page (the scales are positive), then scaled
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int q = 0; q < kPartPages; ++q) {
        const float* t = s + kPage * q;
        const float a = fmax3(t[0], t[1], t[2]), b = fmax3(t[3], t[4], t[5]), c = fmax3(t[6], t[7], t[8]),
                    d = fmax3(t[9], t[10], t[11]), e = fmax3(t[12], t[13], t[14]);
        mx = fmaxf(mx, kf[q] * fmaxf(fmax3(a, b, c), fmax3(d, e, t[15])));
      }
      const bool gain = lv_top + lg > kGainTop;  // (the same for every row)
      if (!ok) soft_fail[quarter] = 1;
      if (quarter_any(quarter, mx > m_used + kRescaleLog2 || gain || !ok)) {
        xch[part * kRowsTC + r] = mx;
        quarter_sync(quarter);
        float m_new = m_used;
#pragma unroll
        for (int q = 0; q < kParts; ++q) m_new = fmaxf(m_new, xch[q * kRowsTC + r]);
        const bool fail = soft_fail[quarter] != 0;
        quarter_sync(quarter);  // (xch and soft_fail are read)
        if (fail) {
          ok = false;
          break;
        }
        if (!(m_new > m_used + kRescaleLog2)) m_new = m_used;
        const float fl = m_new > m_used ? fast_exp2(m_used - m_new) : 1.f;
        const float lg_new = gain ? kGainTop - 4.f - ceilf(lv_top) : lg;
        const float f = fl * exp2f(lg_new - lg);
        if (i >= 1) {
          // O holds the earlier tiles: wait for their last P.V, then rescale
          ok = mbar_wait_warp(smem_u32(&bars[Sm::oDone + (i - 1) % Sm::SB]), ((i - 1) / Sm::SB) & 1);
          __syncwarp();
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < DP / 16; ++c) {
            float o[16];
            tc::ld16(tO + 16 * c, o);
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] *= f;
            tc::st16(tO + 16 * c, o);
            if (i > kSegment) {
              tc::ld16(tT + 16 * c, o);
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] *= f;
              tc::st16(tT + 16 * c, o);
            }
          }
        }
        l *= fl;
        m_used = m_new;
        lg = lg_new;
      }
      // (a part can meet a row's keys only in a later tile: while its max is still -inf,
      // every probability is 0, not exp2(-inf + inf))
      const float nm = m_used == -CUDART_INF_F ? 0.f : -m_used;
#pragma unroll
      for (int q = 0; q < kPartPages; ++q) {  // a page's 16 keys -> 8 columns of P, 8 of remainders
        uint32_t h[8], lo[8];
        // (a page of zeros has no say in the gain: its probabilities count with gain 1)
        const bool zero = lv[q] == -CUDART_INF_F;
        const float up = zero ? 0.f : lv[q] + lg;
        const float off = nm + up;
        const float2 kk = make_float2(kf[q], kf[q]), oo = make_float2(off, off);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 x = __ffma2_rn(make_float2(s[kPage * q + 2 * u], s[kPage * q + 2 * u + 1]), kk, oo);
          const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          sum = u == 0 ? pe : __fadd2_rn(sum, pe);
          split2(pe, h[u], lo[u]);
        }
        l = fmaf(sum.x + sum.y, fast_exp2(-up), l);
        tc::st8_nowait(tS + kPage * q, h);
        tc::st8_nowait(tS + kPage * q + 8, lo);
      }
      tc::st_wait();
      if (i > 0 && i % kSegment == 0) {
        // a segment ends: its accumulator joins the sum of the earlier ones
        ok = mbar_wait_warp(smem_u32(&bars[Sm::oDone + (i - 1) % Sm::SB]), ((i - 1) / Sm::SB) & 1) && ok;
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          float o[16];
          tc::ld16(tO + 16 * c, o);
          if (i > kSegment) {
            float t[16];
            tc::ld16(tT + 16 * c, t);
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] += t[u];
          }
          tc::st16(tT + 16 * c, o);
        }
      }
      tc::fence_before_sync();
      // (one arrival a warp: arrivals of 512 threads on one barrier are served one by one)
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Sm::pFull + i % Sm::SB]);
    }
    if (ok && i == n_tiles)  // the last P.V
      ok = mbar_wait_warp(smem_u32(&bars[Sm::oDone + (n_tiles - 1) % Sm::SB]), ((n_tiles - 1) / Sm::SB) & 1);
    __syncwarp();
    tc::fence_before_sync();
    // the row's sum over its parts (the maximum and the gain are common)
    xch[part * kRowsTC + r] = l;
    if (!ok) soft_fail[quarter] = 1;
    quarter_sync(quarter);
    if (soft_fail[quarter]) {
      *abort_flag = 1;
    } else {
      tc::fence_after_sync();
      float lsum = 0.f;
#pragma unroll
      for (int q = 0; q < kParts; ++q) lsum += xch[q * kRowsTC + r];
      // a split block leaves its unnormalised partial for the merge
      const bool partial = p.ksplit > 1;
      const float wt = (partial ? 1.f : 1.f / lsum) * exp2f(-lg);
      const size_t pidx = (static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r;
      if (partial && valid_row && part == 0) {
        p.ws_m[pidx] = m_used;
        p.ws_l[pidx] = lsum;
      }
      // The row is put together in shared memory (the K and V operands are done with) and
      // leaves as one bulk copy (the end of a block, last products included: 2.1 us; 3.7 us
      // with stores of single 16-byte pieces of 32 rows at a time).  Rows are padded by 16
      // bytes against bank conflicts.
      uint8_t* const orow = smem + Sm::k0 + r * (D * 4 + 16);
      __syncwarp();
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) {
        float o[16];
        tc::ld16(tO + 16 * c, o);
        if (n_tiles > kSegment) {
          float t[16];
          tc::ld16(tT + 16 * c, t);
#pragma unroll
          for (int u = 0; u < 16; ++u) o[u] += t[u];
        }
#pragma unroll
        for (int u = 0; u < 16; u += 4)
          *reinterpret_cast<float4*>(orow + (DP * part + 16 * c + u) * 4) =
              make_float4(o[u] * wt, o[u + 1] * wt, o[u + 2] * wt, o[u + 3] * wt);
      }
      fence_proxy_async_smem();
      quarter_sync(quarter);
      if (part == 0 && valid_row) {
        float* dst = partial ? p.ws_o + pidx * D
                             : p.out + (static_cast<size_t>(q0 + rho / p.G) * p.Hq + g * p.G + rho % p.G) * D;
        bulk_s2g(dst, orow, D * 4);
        bulk_store_wait();  // (arrived: a merge reads it, an error found late writes over it)
      }
    }
  }

  // ---- tear-down: errors become NaN rows; TMEM is released by the warp that took it
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (tid == 0 && *abort_flag) atomicOr(&s_err, 0x10);  // PKV_DEV_TIMEOUT
  __syncthreads();
  err = s_err;
  if (tid == 0 && err && p.dev_status) atomicOr(p.dev_status, err);
  if (err && valid_row) {
    float* dst = p.out + (static_cast<size_t>(q0 + rho / p.G) * p.Hq + g * p.G + rho % p.G) * D;
    for (int d = (D / kParts) * part; d < (D / kParts) * (part + 1); ++d) dst[d] = CUDART_NAN_F;
    if (p.ksplit > 1 && part == 0)  // a poisoned partial turns the merged row into NaN
      p.ws_m[(static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r] = CUDART_NAN_F;
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, Sm::tmemCols);
  if (p.ksplit > 1) {
    // a block with no key tiles (a short row range split more ways than it has tiles)
    // leaves an empty partial
    if (n_tiles == 0 && !err && valid_row && part == 0) {
      const size_t pidx = (static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r;
      p.ws_m[pidx] = -CUDART_INF_F;
      p.ws_l[pidx] = 0.f;
      for (int d = 0; d < D; d += 4)
        *reinterpret_cast<float4*>(p.ws_o + pidx * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    split_merge<D, Sm::threads>(p, tile, g, b, q0, nrows, err, tid, smem + Sm::xch0);
  }
}

template <bool FP8, int D, bool QSPLIT>
const void* blk_kernel() {
  return reinterpret_cast<const void*>(&prefill_blk_kernel<FP8, D, QSPLIT>);
}
struct BlkVariant {
  const void* fn;
  int smem, threads;
};
template <int D, bool QSPLIT>
BlkVariant variant_of(const void* fn) {
  return {fn, BSmem<D, QSPLIT>::total, BSmem<D, QSPLIT>::threads};
}
BlkVariant blk_variant(bool fp8, int D, bool qsplit) {
  if (D == 64) {
    if (qsplit) return variant_of<64, true>(fp8 ? blk_kernel<true, 64, true>() : blk_kernel<false, 64, true>());
    return variant_of<64, false>(fp8 ? blk_kernel<true, 64, false>() : blk_kernel<false, 64, false>());
  }
  if (qsplit) return variant_of<128, true>(fp8 ? blk_kernel<true, 128, true>() : blk_kernel<false, 128, true>());
  return variant_of<128, false>(fp8 ? blk_kernel<true, 128, false>() : blk_kernel<false, 128, false>());
}

constexpr int kMaxDevicesB = 64;
bool g_blk_attr[kMaxDevicesB][8];
std::mutex g_blk_mu;

}  // namespace

cudaError_t launch_prefill_blk(const PrefillArgs& a, int n_row_tiles, int ksplit, cudaStream_t st) {
  if (n_row_tiles == 0) return cudaSuccess;
  const TParams p = params_of(a, n_row_tiles, ksplit);
  const bool fp8 = a.c.dtype == kFP8B, qsplit = a.q_dtype == kF32;
  const BlkVariant v = blk_variant(fp8, a.c.D, qsplit);
  const int slot = (fp8 ? 4 : 0) + (a.c.D == 128 ? 2 : 0) + (qsplit ? 1 : 0);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevicesB) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(g_blk_mu);
    if (!g_blk_attr[dev][slot]) {
      e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
      if (e != cudaSuccess) return e;
      g_blk_attr[dev][slot] = true;
    }
  }
  const dim3 grid(n_row_tiles * ksplit, a.c.Hkv, a.B);
  void* args[] = {const_cast<TParams*>(&p)};
  return cudaLaunchKernel(v.fn, grid, dim3(v.threads), args, v.smem, st);
}

}  // namespace pkv

#ifdef PKV_TEST_HOOKS
// Test builds only: switches the give-up-at-once first score wait (see above) on or off.
extern "C" int pkv_test_prefill_blk_fail_first_wait(int on) {
  return cudaMemcpyToSymbol(pkv::g_test_prefill_blk_fail_first_wait, &on, sizeof(int)) == cudaSuccess ? 0 : 1;
}
#endif
