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
// token-major, against the group's keys in pairs of 64-key tiles (8 pages):
//   warps 9-12   K: fetch the pair's codes 16 bytes a thread, one pair ahead in registers,
//                and write them as FP16 operand tiles (no-swizzle K-major core matrices);
//                they also leave the pages' scales in a ring of four pairs;
//   warps 13-16  V: the same per 64-key tile; codes of keys that no row sees become zero
//                (a stale E4M3 NaN would survive a zero probability);
//   warp 8       one thread issues every MMA: S(p) = Q K^T (M = 128, N = 128) into one of
//                two score buffers of TMEM, O_g += P_g V (M = 128, N = head_dim) for the
//                two softmax groups g;
//   warps 0-7    softmax, two groups of four warps, one thread per row; group g takes the
//                pair's tile g with its own running max and sum and its own accumulator
//                O_g, merged once at the end.  P overwrites its own scores in TMEM, page by
//                page (8 columns of FP16 high parts, 8 of remainders: P keeps ~22 bits, two
//                MMAs per page), so that two score buffers fit beside the accumulators: the
//                scores of pair p + 1 are ready while the groups work on pair p.
//
// Range of FP16: query rows are brought to [2^13, 2^14) by a power of two that goes into the
// score scale (float queries as high part + remainder); probabilities carry the V scale as
// 2^(log2 s_v + lg), lg raised or lowered when a page's scale leaves the range, so that
// P s_v stays below 2^15.  The sum takes P s_v / s_v, so the rounding of the logarithm
// cancels.
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

constexpr int kSoftWarps = 8;  // two groups of 4 warps, one thread per query row
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMmaWarp = kSoftWarps;
constexpr int kKWarp = kMmaWarp + 1;
constexpr int kFillWarps = 4;  // warps that fill each of the K and V rings
constexpr int kVWarp = kKWarp + kFillWarps;
constexpr int kThreadsB = (kVWarp + kFillWarps) * 32;
constexpr int kPairPages = 2 * kPagesTC;
constexpr int kScaleSlots = 4;
constexpr float kGainTop = 7.f;  // log2 of the largest scaled V scale

#ifdef PKV_TEST_HOOKS
// Test builds only: each softmax group's first wait for scores gives up at once.
__device__ int g_test_prefill_blk_fail_first_wait = 0;
#endif

template <int D, bool QSPLIT>
struct BSmem {
  static constexpr int blk = kPage * D * 2;          // one FP16 page block (K or V)
  static constexpr int qTile = kRowsTC * D * 2;      // one FP16 query tile
  static constexpr int KSP = 2;                      // stages of the K ring (a tile pair each)
  static constexpr int KST = 4;                      // stages of the V ring (a tile each)
  static constexpr int kStage = kPairPages * blk, vStage = kPagesTC * blk;
  static constexpr int q0 = 0;
  static constexpr int k0 = q0 + (QSPLIT ? 2 : 1) * qTile;
  static constexpr int v0 = k0 + KSP * kStage;
  // scales of a pair's pages: K scale [8], log2 of the V scale [8], 1 / V scale [8]
  static constexpr int sc0 = v0 + KST * vStage;
  static constexpr int scSlot = 3 * kPairPages * 4;
  static constexpr int bar0 = sc0 + kScaleSlots * scSlot;
  // barriers by index
  static constexpr int kFull = 0, kEmpty = 2, vFull = 4, vEmpty = 8, sFull = 12, pFull = 14, oDone = 18,
                       fin = 20, xfin = 21, qFull = 22, nbars = 24;
  static constexpr int misc0 = bar0 + nbars * 8;  // TMEM base address, abort flag
  // row maxima of the queries, then the final exchange (max, sum, gain by group and row),
  // then the split merge's weights
  static constexpr int xch0 = misc0 + 16;
  static constexpr int total = xch0 + 4 * kRowsTC * 4 + 2 * kRowsTC * 4;
  // TMEM columns: O of group 0 [0, D), O of group 1 [D, 2D), score buffers at 2D + 128 b
  // (group g's 64 keys at + 64 g)
  static constexpr int sCol = 2 * D;
  static constexpr int tmemCols = 512;
  static_assert(2 * D + 4 * kKeysTC <= 512, "tensor memory");
};

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
// 16 stored bytes -> two 16-byte operand rows of 8 FP16 values, `step` bytes apart.
template <bool FP8>
__device__ __forceinline__ void store_codes16(uint8_t* dst, uint32_t step, uint4 c) {
  uint4 a, b;
  codes4<FP8>(c.x, a.x, a.y);
  codes4<FP8>(c.y, a.z, a.w);
  codes4<FP8>(c.z, b.x, b.y);
  codes4<FP8>(c.w, b.z, b.w);
  *reinterpret_cast<uint4*>(dst) = a;
  *reinterpret_cast<uint4*>(dst + step) = b;
}

// (a, b) -> f16x2 high part and f16x2 remainder
__device__ __forceinline__ void split2(float2 a, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __float22half2_rn(a);
  const float2 f = __half22float2(h);
  const __half2 r = __float22half2_rn(__fadd2_rn(a, make_float2(-f.x, -f.y)));
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

template <bool FP8, int D, bool QSPLIT>
__global__ void __launch_bounds__(kThreadsB, 1)
    prefill_blk_kernel(const __grid_constant__ TParams p) {
  using Sm = BSmem<D, QSPLIT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::bar0);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sm::misc0);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Sm::misc0 + 4);
  __shared__ int s_err;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int tile = blockIdx.x / p.ksplit, ks = blockIdx.x % p.ksplit;
  const int row0 = tile * kRowsTC;
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
  const int nt_all = err ? 0 : (n_keys0 - kb0 + kKeysTC - 1) / kKeysTC;
  const int t0 = ks * nt_all / p.ksplit, t1 = (ks + 1) * nt_all / p.ksplit;
  const int n_keys = err ? 0 : min(n_keys0, kb0 + t1 * kKeysTC);
  const int kbase = err ? 0 : kb0 + t0 * kKeysTC;
  const int n_pages = max(0, (n_keys - kbase + kPage - 1) / kPage);  // pages from kbase on
  const int n_tiles = t1 - t0, n_pairs = (n_tiles + 1) / 2;
  const int32_t* btw = p.bt + static_cast<size_t>(b) * p.MB + kbase / kPage;

  // ---- set-up: TMEM and barriers
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, Sm::tmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < Sm::nbars; ++i) {
      const bool filled = (i >= Sm::kFull && i < Sm::kFull + 2) || (i >= Sm::vFull && i < Sm::vFull + 4);
      const int count = filled                                       ? kFillWarps
                        : i >= Sm::pFull && i < Sm::pFull + 4        ? kSoftThreads / 2
                        : i == Sm::xfin || i == Sm::qFull            ? kSoftThreads
                                                                     : 1;
      mbar_init(&bars[i], count);
    }
    fence_barrier_init();
    *abort_flag = 0;
    s_err = err;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);

  // softmax threads: row r (= TMEM lane 32 (warp % 4) + lane) of group grp
  const int r = tid & (kRowsTC - 1);
  const int grp = tid / kRowsTC;
  const int rho = row0 + r;
  const bool valid_row = tid < kSoftThreads && rho < nrows;

  // A page id outside the pool is replaced by page 0 (every read stays inside the cache)
  // and flagged: the block's rows then become NaN.
  bool bad = false;
  auto page_id = [&](int q) -> int {  // -1: no such page
    if (q >= n_pages) return -1;
    const int id = btw[q];
    if (id >= 0 && id < p.num_pages) return id;
    bad = true;
    return 0;
  };

  if (n_tiles > 0 && warp >= kKWarp && warp < kVWarp) {
    // ---------------------------------------------------------------- K codes
    // thread -> 16 codes of one token; the 8 lanes of a quarter warp take 8 tokens, so that
    // their 16-byte operand rows are one core matrix (no bank conflicts)
    constexpr int PPS = D == 128 ? 1 : 2;             // pages per step of the four warps
    constexpr int STEPS = kPairPages / PPS;
    const int w = warp - kKWarp;
    const int sub = D == 128 ? 0 : w >> 1;
    const int row = 8 * (D == 128 ? w >> 1 : w & 1) + (lane & 7);
    const int piece = (D == 128 ? 4 * (w & 1) : 0) + (lane >> 3);
    const uint8_t* src = p.k + static_cast<size_t>(g) * kPage * D + row * D + piece * 16;
    const size_t stride = static_cast<size_t>(p.Hkv) * kPage * D;
    uint8_t* dst = smem + Sm::k0 + tile_off(sub * kPage + row, 16 * piece, D);
    uint4 raw[STEPS];
    float sk = 0.f, sv = 0.f;
    auto fetch1 = [&](int s, int ids) {
      const int id = __shfl_sync(0xffffffffu, ids, s * PPS + sub);
      raw[s] = id >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + id * stride)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto fetch_scales = [&](int ids) {
      sk = sv = 0.f;
      if (w == 0 && lane < kPairPages && ids >= 0) {
        sk = p.ks[static_cast<size_t>(ids) * p.Hkv + g];
        sv = p.vs[static_cast<size_t>(ids) * p.Hkv + g];
      }
    };
    int ids = page_id(lane & 7);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) fetch1(s, ids);
    fetch_scales(ids);
    ids = page_id(kPairPages + (lane & 7));
    bool ok = true;
    for (int j = 0; j < n_pairs; ++j) {
      const int st = j % Sm::KSP;
      if (j >= Sm::KSP) ok = mbar_wait_warp(smem_u32(&bars[Sm::kEmpty + st]), (j / Sm::KSP - 1) & 1);
      if (!ok || *abort_flag) break;
      const bool more = j + 1 < n_pairs;
      if (w == 0 && lane < kPairPages) {
        // (an all-zero block has scale 0 and zero codes: any K scale gives its zeros; a V
        // scale of 0, and pages past the end, are marked by a logarithm of -inf)
        float* sc = reinterpret_cast<float*>(smem + Sm::sc0 + (j % kScaleSlots) * Sm::scSlot);
        sc[lane] = sk == 0.f ? 1.f : sk;
        sc[kPairPages + lane] = sv == 0.f ? -CUDART_INF_F : log2f(sv);
        sc[2 * kPairPages + lane] = sv == 0.f ? 1.f : 1.f / sv;
      }
      if (more) fetch_scales(ids);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        store_codes16<FP8>(dst + st * Sm::kStage + s * PPS * Sm::blk, 128, raw[s]);
        if (more) fetch1(s, ids);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Sm::kFull + st]);
      ids = page_id((j + 2) * kPairPages + (lane & 7));
    }
    if (!ok) *abort_flag = 1;
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&s_err, 0x1);  // PKV_DEV_BAD_PAGE
  } else if (n_tiles > 0 && warp >= kVWarp) {
    // ---------------------------------------------------------------- V codes
    // thread -> the 16 tokens of one head-dim row of a page: two operand rows of 8 tokens
    constexpr int PPS = D == 128 ? 1 : 2;
    constexpr int STEPS = kPagesTC / PPS;  // per tile
    const int w = warp - kVWarp;
    const int sub = D == 128 ? 0 : w >> 1;
    const int d = (D == 128 ? 32 * w : 32 * (w & 1)) + lane;
    const uint8_t* src = p.v + static_cast<size_t>(g) * kPage * D + d * 16;
    const size_t stride = static_cast<size_t>(p.Hkv) * kPage * D;
    uint8_t* dst = smem + Sm::v0 + sub * Sm::blk + bf16_v_off(d, 0);
    uint4 raw[2][STEPS];  // the two tiles of a pair
    auto fetch1 = [&](int y, int s, int ids) {
      const int id = __shfl_sync(0xffffffffu, ids, y * kPagesTC + s * PPS + sub);
      raw[y][s] = id >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + id * stride)) : make_uint4(0u, 0u, 0u, 0u);
    };
    int ids = page_id(lane & 7);
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) fetch1(y, s, ids);
    ids = page_id(kPairPages + (lane & 7));
    bool ok = true;
    for (int j = 0; j < n_pairs && ok; ++j) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 2 * j + y, st = i % Sm::KST;
        if (i >= n_tiles) break;
        if (i >= Sm::KST) ok = mbar_wait_warp(smem_u32(&bars[Sm::vEmpty + st]), (i / Sm::KST - 1) & 1);
        if (*abort_flag) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          uint4 c = raw[y][s];
          const int key = kbase + i * kKeysTC + (s * PPS + sub) * kPage;  // of the page's token 0
          if (key < lo_blk || key + kPage > n_keys) {  // only tokens that some row sees
            uint32_t m[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              m[u] = 0u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = key + 4 * u + e;
                if (t >= lo_blk && t < n_keys) m[u] |= 0xffu << (8 * e);
              }
            }
            c.x &= m[0]; c.y &= m[1]; c.z &= m[2]; c.w &= m[3];
          }
          store_codes16<FP8>(dst + st * Sm::vStage + s * PPS * Sm::blk, 128, c);
          if (j + 1 < n_pairs) fetch1(y, s, ids);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Sm::vFull + st]);
      }
      ids = page_id((j + 2) * kPairPages + (lane & 7));
    }
    if (!ok) *abort_flag = 1;
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&s_err, 0x1);
  } else if (n_tiles > 0 && warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_f16_f32(kRowsTC, 2 * kKeysTC);
      constexpr uint32_t idO = tc::idesc_f16_f32(kRowsTC, D);
      constexpr uint32_t sboQK = (D / 8) * 128;  // 8-row groups of Q and of K
      const uint64_t dQhi = tc::smem_desc(sbase + Sm::q0, 128, sboQK);
      const uint64_t dQlo = tc::smem_desc(sbase + Sm::q0 + Sm::qTile, 128, sboQK);
      const uint64_t dK0 = tc::smem_desc(sbase + Sm::k0, 128, sboQK);
      const uint64_t dV0 = tc::smem_desc(sbase + Sm::v0, 128, 256);
      // S of pair pr, once the last readers of its buffer, the P.V products of pair pr - 2,
      // have completed (only MMAs into one accumulator are bound to run in order)
      auto issue_s = [&](int pr) -> bool {
        if (pr >= 2 && (!mbar_wait(&bars[Sm::oDone], pr & 1) || !mbar_wait(&bars[Sm::oDone + 1], pr & 1)))
          return false;
        if (!mbar_wait(&bars[Sm::kFull + pr % Sm::KSP], (pr / Sm::KSP) & 1) || *abort_flag) return false;
        tc::fence_after_sync();
        const uint64_t dK = tc::desc_add(dK0, (pr % Sm::KSP) * Sm::kStage);
        const uint32_t tS = tmem + Sm::sCol + 2 * kKeysTC * (pr & 1);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t bd = tc::desc_add(dK, k * 256);
          tc::mma_bf16(tS, tc::desc_add(dQhi, k * 256), bd, idS, k > 0);
          if constexpr (QSPLIT) tc::mma_bf16(tS, tc::desc_add(dQlo, k * 256), bd, idS, true);
        }
        tc::commit(&bars[Sm::sFull + (pr & 1)]);
        tc::commit(&bars[Sm::kEmpty + pr % Sm::KSP]);
        return true;
      };
      auto issue_pv = [&](int i) -> bool {
        const int y = i & 1, pr = i >> 1, st = i % Sm::KST;
        if (!mbar_wait(&bars[Sm::pFull + 2 * y + (pr & 1)], (pr >> 1) & 1)) return false;
        if (!mbar_wait(&bars[Sm::vFull + st], (i / Sm::KST) & 1) || *abort_flag) return false;
        tc::fence_after_sync();
        const uint64_t dV = tc::desc_add(dV0, st * Sm::vStage);
        const uint32_t tP = tmem + Sm::sCol + 2 * kKeysTC * (pr & 1) + kKeysTC * y;
#pragma unroll
        for (int q = 0; q < kPagesTC; ++q) {
          const uint64_t bd = tc::desc_add(dV, q * Sm::blk);
#pragma unroll
          for (int part = 0; part < 2; ++part)
            tc::mma_bf16_ts(tmem + D * y, tP + 16 * q + 8 * part, bd, idO, !(i < 2 && q == 0 && part == 0));
        }
        tc::commit(&bars[Sm::oDone + y]);
        tc::commit(&bars[Sm::vEmpty + st]);
        return true;
      };
      bool ok = mbar_wait(&bars[Sm::qFull], 0);
      for (int pr = 0; pr < min(2, n_pairs) && ok; ++pr) ok = issue_s(pr);
      for (int pr = 0; pr < n_pairs && ok; ++pr) {
        ok = issue_pv(2 * pr);
        if (ok && 2 * pr + 1 < n_tiles) ok = issue_pv(2 * pr + 1);
        if (ok && pr + 2 < n_pairs) ok = issue_s(pr + 2);
      }
      if (!ok) *abort_flag = 1;
      // every MMA has completed before TMEM is released
      tc::commit(&bars[Sm::fin]);
      (void)mbar_wait(&bars[Sm::fin], 0);
    }
  } else if (n_tiles > 0 && warp < kSoftWarps) {
    // ---------------------------------------------------------------- the query rows
    // each thread brings half of its row's columns; the two halves exchange their largest
    // value, and the row becomes FP16 in [2^13, 2^14)
    float* xch = reinterpret_cast<float*>(smem + Sm::xch0);
    float rs;
    {
      constexpr int N = D / 2;
      float x[N];
      if (valid_row) {
        const size_t at = (static_cast<size_t>(q0 + rho / p.G) * p.Hq + g * p.G + rho % p.G) * D + N * grp;
        if constexpr (!QSPLIT) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at);
#pragma unroll
          for (int i = 0; i < N / 8; ++i) {
            const uint4 v = src[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              x[8 * i + 2 * u] = __uint_as_float(w[u] << 16);
              x[8 * i + 2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
            }
          }
        } else {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            const float4 v = src[i];
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.f;
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
      xch[grp * kRowsTC + r] = top;
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
      top = fmaxf(top, xch[(grp ^ 1) * kRowsTC + r]);
      // top in [2^(e-1), 2^e): times 2^k, k = 14 - e
      const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xffu) - 126;
      const int k = min(14 - e, 126);
      const float f = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
      rs = ldexpf(p.scale_log2, -k);
      uint8_t* qhi = smem + Sm::q0;
#pragma unroll
      for (int c = 0; c < N / 8; ++c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          split2(make_float2(x[8 * c + 2 * u] * f, x[8 * c + 2 * u + 1] * f), h[u], l[u]);
        const uint32_t off = tile_off(r, N * grp + 8 * c, D);
        *reinterpret_cast<uint4*>(qhi + off) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (QSPLIT) *reinterpret_cast<uint4*>(qhi + Sm::qTile + off) = make_uint4(l[0], l[1], l[2], l[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[Sm::qFull]);
    }
    // ---------------------------------------------------------------- softmax rows
    const int pos = valid_row ? L - Lq + rho / p.G : p_first;
    const int lo_row = win > 0 ? pos - win + 1 : 0;  // first key of the row's window
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + lane_base + D * grp;
    float m_used = -CUDART_INF_F, l = 0.f;
    float lg = 100.f;  // log2 of the gain on the V scales (the first tile brings it down)
    bool ok = true;
    int n_mine = 0;  // tiles this group has finished
    for (int j = grp; j < n_tiles; j += 2, ++n_mine) {
      const int k = j >> 1;  // the pair
      ok = mbar_wait(&bars[Sm::sFull + (k & 1)], (k >> 1) & 1) && !*abort_flag;
#ifdef PKV_TEST_HOOKS
      if (k == 0 && g_test_prefill_blk_fail_first_wait) ok = false;  // a wait that gives up
#endif
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t tS = tmem + lane_base + Sm::sCol + 2 * kKeysTC * (k & 1) + kKeysTC * grp;
      float s[64];
      tc::ld64(tS, s);
      const float* sc = reinterpret_cast<const float*>(smem + Sm::sc0 + (k % kScaleSlots) * Sm::scSlot) +
                        kPagesTC * grp;
      const float4 k4 = *reinterpret_cast<const float4*>(sc);
      const float4 v4 = *reinterpret_cast<const float4*>(sc + kPairPages);
      const float4 i4 = *reinterpret_cast<const float4*>(sc + 2 * kPairPages);
      // (never 0: a masked score of -inf has to stay -inf; 1e-37 takes every score to 0)
      constexpr float kTiny = 1e-37f;
      const float kf[4] = {fmaxf(k4.x * rs, kTiny), fmaxf(k4.y * rs, kTiny), fmaxf(k4.z * rs, kTiny),
                           fmaxf(k4.w * rs, kTiny)};
      const float lv[4] = {v4.x, v4.y, v4.z, v4.w};
      const float iv[4] = {i4.x, i4.y, i4.z, i4.w};
      const int key0 = kbase + j * kKeysTC;
      if (key0 + kKeysTC - 1 > p_first || key0 + kKeysTC > n_keys || key0 < lo_max) {
#pragma unroll
        for (int u = 0; u < 64; ++u)
          s[u] = (key0 + u <= pos && key0 + u >= lo_row) ? s[u] : -CUDART_INF_F;
      }
      // largest score: raw per page (the scales are positive), then scaled
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = fmaxf(s[16 * q + u], s[16 * q + 8 + u]);
        mx = fmaxf(mx, kf[q] * fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmaxf(t[6], t[7])));
      }
      const float lv_top = fmaxf(fmaxf(lv[0], lv[1]), fmaxf(lv[2], lv[3]));
      const bool need = mx > m_used + kRescaleLog2;
      const bool gain = lv_top + lg > kGainTop;  // (the same for every row)
      if (__any_sync(0xffffffffu, need) || gain) {
        const float m_new = need ? mx : m_used;
        const float fl = need ? fast_exp2(m_used - m_new) : 1.f;
        const float lg_new = gain ? kGainTop - 2.f - ceilf(lv_top) : lg;
        const float f = fl * exp2f(lg_new - lg);
        if (k >= 1) {
          // O holds this group's earlier tiles: wait for their last P.V, then rescale
          ok = mbar_wait(&bars[Sm::oDone + grp], (k - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            tc::ld16(tO + 16 * c, o);
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] *= f;
            tc::st16(tO + 16 * c, o);
          }
        }
        l *= fl;
        m_used = m_new;
        lg = lg_new;
      }
      // (a group can meet a row's keys only in a later tile: while its max is still -inf,
      // every probability is 0, not exp2(-inf + inf))
      const float nm = m_used == -CUDART_INF_F ? 0.f : -m_used;
      const float ginv = exp2f(-lg);
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // a page's 16 keys -> 8 columns of P, 8 of remainders
        uint32_t h[8], lo[8];
        // (a page of zeros has no say in the gain: its probabilities count with gain 1)
        const bool zero = lv[q] == -CUDART_INF_F;
        const float off = nm + (zero ? 0.f : lv[q] + lg);
        const float2 k2 = make_float2(kf[q], kf[q]), o2 = make_float2(off, off);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 x = __ffma2_rn(make_float2(s[16 * q + 2 * u], s[16 * q + 2 * u + 1]), k2, o2);
          const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          sum = u == 0 ? pe : __fadd2_rn(sum, pe);
          split2(pe, h[u], lo[u]);
        }
        l = fmaf(sum.x + sum.y, zero ? 1.f : iv[q] * ginv, l);
        tc::st8_nowait(tS + 16 * q, h);
        tc::st8_nowait(tS + 16 * q + 8, lo);
      }
      tc::st_wait();
      tc::fence_before_sync();
      mbar_arrive(&bars[Sm::pFull + 2 * grp + (k & 1)]);
    }
    if (ok && n_mine > 0) {  // this group's last P.V
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[Sm::oDone + grp], (n_mine - 1) & 1));
    }
    tc::fence_before_sync();
    // the two groups' (max, sum, gain) of this row, exchanged once
    float* xm = xch;  // [group][row] (the queries' maxima are done with)
    float* xl = xm + 2 * kRowsTC;
    float* xg = xl + 2 * kRowsTC;  // one value per group and row, as the others
    xm[grp * kRowsTC + r] = m_used;
    xl[grp * kRowsTC + r] = l;
    if (r == 0) xg[grp] = lg;
    mbar_arrive(&bars[Sm::xfin]);
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[Sm::xfin], 0) && ok);
    if (!ok) *abort_flag = 1;
    if (ok) {
      tc::fence_after_sync();
      const float m_o = xm[(grp ^ 1) * kRowsTC + r], l_o = xl[(grp ^ 1) * kRowsTC + r];
      const float lg_o = xg[grp ^ 1];
      const float M = fmaxf(m_used, m_o);
      const float a_me = m_used == -CUDART_INF_F ? 0.f : fast_exp2(m_used - M);
      const float a_ot = m_o == -CUDART_INF_F ? 0.f : fast_exp2(m_o - M);
      const float lsum = l * a_me + l_o * a_ot;
      // a split block leaves its unnormalised partial for the merge
      const bool partial = p.ksplit > 1;
      const float inv = partial ? 1.f : 1.f / lsum;
      const float w_me = a_me * inv * exp2f(-lg), w_ot = a_ot * inv * exp2f(-lg_o);
      const float wA = grp == 0 ? w_me : w_ot, wB = grp == 0 ? w_ot : w_me;
      const bool hasB = n_tiles > 1;  // group 1's accumulator holds data
      const size_t pidx = (static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r;
      float* dst = !valid_row ? nullptr
                   : partial ? p.ws_o + pidx * D
                             : p.out + (static_cast<size_t>(q0 + rho / p.G) * p.Hq + g * p.G + rho % p.G) * D;
      if (partial && valid_row && grp == 0) {
        p.ws_m[pidx] = M;
        p.ws_l[pidx] = lsum;
      }
      // group grp writes head_dim columns [grp D/2, (grp + 1) D/2) of its row
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int col = (D / 2) * grp + 32 * c;
        float oa[32], ob[32];
        tc::ld32(tmem + lane_base + col, oa);
        if (hasB) {
          tc::ld32(tmem + lane_base + D + col, ob);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) ob[u] = 0.f;
        }
        if (dst) {
#pragma unroll
          for (int u = 0; u < 32; u += 4)
            *reinterpret_cast<float4*>(dst + col + u) =
                make_float4(oa[u] * wA + ob[u] * wB, oa[u + 1] * wA + ob[u + 1] * wB,
                            oa[u + 2] * wA + ob[u + 2] * wB, oa[u + 3] * wA + ob[u + 3] * wB);
        }
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
    for (int d = (D / 2) * grp; d < (D / 2) * (grp + 1); ++d) dst[d] = CUDART_NAN_F;
    if (p.ksplit > 1 && grp == 0)  // a poisoned partial turns the merged row into NaN
      p.ws_m[(static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r] = CUDART_NAN_F;
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, Sm::tmemCols);
  if (p.ksplit > 1) {
    // a block with no key tiles (a short row range split more ways than it has tiles)
    // leaves an empty partial
    if (n_tiles == 0 && !err && valid_row && grp == 0) {
      const size_t pidx = (static_cast<size_t>(tile_index(p, tile, g, b)) * p.ksplit + ks) * kRowsTC + r;
      p.ws_m[pidx] = -CUDART_INF_F;
      p.ws_l[pidx] = 0.f;
      for (int d = 0; d < D; d += 4)
        *reinterpret_cast<float4*>(p.ws_o + pidx * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    split_merge<D, kThreadsB>(p, tile, g, b, q0, nrows, err, tid, smem + Sm::xch0);
  }
}

template <bool FP8, int D, bool QSPLIT>
const void* blk_kernel() {
  return reinterpret_cast<const void*>(&prefill_blk_kernel<FP8, D, QSPLIT>);
}
struct BlkVariant {
  const void* fn;
  int smem;
};
BlkVariant blk_variant(bool fp8, int D, bool qsplit) {
  if (D == 64) {
    if (qsplit) return {fp8 ? blk_kernel<true, 64, true>() : blk_kernel<false, 64, true>(), BSmem<64, true>::total};
    return {fp8 ? blk_kernel<true, 64, false>() : blk_kernel<false, 64, false>(), BSmem<64, false>::total};
  }
  if (qsplit) return {fp8 ? blk_kernel<true, 128, true>() : blk_kernel<false, 128, true>(), BSmem<128, true>::total};
  return {fp8 ? blk_kernel<true, 128, false>() : blk_kernel<false, 128, false>(), BSmem<128, false>::total};
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
  return cudaLaunchKernel(v.fn, grid, dim3(kThreadsB), args, v.smem, st);
}

}  // namespace pkv

#ifdef PKV_TEST_HOOKS
// Test builds only: switches the give-up-at-once first score wait (see above) on or off.
extern "C" int pkv_test_prefill_blk_fail_first_wait(int on) {
  return cudaMemcpyToSymbol(pkv::g_test_prefill_blk_fail_first_wait, &on, sizeof(int)) == cudaSuccess ? 0 : 1;
}
#endif
