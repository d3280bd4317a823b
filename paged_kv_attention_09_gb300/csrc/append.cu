// append.cu — KV append: scatter new tokens' K/V rows into their cache slots.
//
// "Tiny-LLM-Inference Project_Status" (feature list: paged KV cache; dtype contract:
// FP32 or BF16 KV), "tinyloop Current Status" (KV cache modes table: INT8 and INT4 KV
// caches) and the TinyInfer review (item 2: INT8 or FP8 KV cache).  One warp per (token,
// kv head) writes both the K row and the V column of that slot; quantised rows go through
// the shared quantisers (kvrow.cuh).  INT4 K rows are written as whole 32-bit words and
// INT4 V bytes belong to one token each, so tokens of one call never share a byte.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"
#include "kvrow.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;

template <int NEW_DT>
__device__ __forceinline__ float load_src(const void* p, size_t i) {
  if constexpr (NEW_DT == kBF16) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  } else {
    return static_cast<const float*>(p)[i];
  }
}

template <int KV_DT, int NEW_DT, int D>
__global__ void __launch_bounds__(kWarps * 32)
    append_kernel(void* __restrict__ k_cache, void* __restrict__ v_cache,
                  float* __restrict__ k_scale, float* __restrict__ v_scale,
                  const void* __restrict__ k_new, const void* __restrict__ v_new,
                  const int32_t* __restrict__ slots, int T, int Hkv, int num_pages,
                  int32_t* dev_status) {
  constexpr int E = D / 32;  // elements per lane
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(T) * Hkv) return;
  const int tok = static_cast<int>(item / Hkv), h = static_cast<int>(item % Hkv);
  const int slot = slots[tok];
  if (slot < 0) return;
  if (slot >= num_pages * kPage) {
    if (lane == 0 && dev_status) atomicOr(dev_status, 0x4 /*PKV_DEV_BAD_SLOT*/);
    return;
  }
  const int page = slot / kPage, off = slot % kPage;
  const size_t src_row = (static_cast<size_t>(tok) * Hkv + h) * D;
  const size_t blk = static_cast<size_t>(page) * Hkv + h;  // (page, head) block index
  const size_t k_row = (blk * kPage + off) * D;            // K: [P][D] inside the block
  const size_t v_base = blk * D * kPage + off;             // V: [D][P] inside the block
  // (INT4: D/2 bytes per K row and D/2 row pairs of 16 bytes per V block)

#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const void* src = which ? v_new : k_new;
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = load_src<NEW_DT>(src, src_row + lane * E + e);

    if constexpr (KV_DT == kINT4) {
      int8_t code[E];
      const float s = quantize_row_int4<E>(x, code);
      uint8_t* dst = static_cast<uint8_t*>(which ? v_cache : k_cache) + blk * kPage * (D / 2);
      if (which == 0) {
        const uint32_t w = int4_k_word<E>(code, lane);
        if ((lane & (8 / E - 1)) == 0)
          reinterpret_cast<uint32_t*>(dst + off * (D / 2))[lane * E / 8] = w;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane * E + e;
          const uint8_t b = int4_v_byte<E>(code, e);
          if ((d & 15) < 8) dst[int4_v_pair(d) * kPage + int4_v_tpos(off)] = b;
        }
      }
      if (lane == 0) (which ? v_scale : k_scale)[blk * kPage + off] = s;
    } else if constexpr (KV_DT == kINT8 || KV_DT == kFP8) {
      uint8_t code[E];
      float s;
      if constexpr (KV_DT == kINT8) {
        int8_t c8[E];
        s = quantize_row_int8<E>(x, c8);
#pragma unroll
        for (int e = 0; e < E; ++e) code[e] = int8_stored(c8[e]);
      } else {
        s = quantize_row_fp8<E>(x, code);
      }
      uint8_t* dst = static_cast<uint8_t*>(which ? v_cache : k_cache);
      if (which == 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) dst[k_row + lane * E + e] = code[e];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) dst[v_base + static_cast<size_t>(lane * E + e) * kPage] = code[e];
      }
      if (lane == 0) (which ? v_scale : k_scale)[blk * kPage + off] = s;
    } else if constexpr (KV_DT == kBF16) {
      // tensor-core tile order inside the block (see bf16_k_off / bf16_v_off)
      uint8_t* blkp = static_cast<uint8_t*>(which ? v_cache : k_cache) + blk * kPage * D * 2;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 b = __float2bfloat16_rn(x[e]);
        const int d = lane * E + e;
        const int off_b = which == 0 ? bf16_k_off(off, d, D) : bf16_v_off(d, off);
        *reinterpret_cast<__nv_bfloat16*>(blkp + off_b) = b;
      }
    } else {
      float* dst = static_cast<float*>(which ? v_cache : k_cache);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (which == 0) dst[k_row + lane * E + e] = x[e];
        else dst[v_base + static_cast<size_t>(lane * E + e) * kPage] = x[e];
      }
    }
  }
}

// Block-scaled 8-bit formats: the scale belongs to the 16 tokens of a (page, kv head), so
// the new rows of one page are taken together.  They stand next to each other in the call in
// ascending order of their slots (a run).  One warp takes the runs that start within `group`
// consecutive tokens, for one kv head and one of K and V; for each run it finds the largest
// new value, grows the block's scale to hold it (rows before the run's first offset keep
// their place and are coded again when it grows; a run that starts the page starts its scale
// afresh), and stores the run.
//
// The old block is fetched whole, 16 bytes a lane, together with the new rows, before the
// scale is known: a decode step's append then waits for one round trip after the slots'.
// A V block has its tokens along the rows, so its bytes are merged in registers and stored
// as whole 16-byte rows; K rows are stored as they are, old rows only when coded again.
//
// Bound by latency: a decode step's tokens wait for their slot, then for one round of loads
// (256 tokens of 4 heads of 64, BF16: 4.0 us a launch, an empty one takes about 2); a prompt's
// are bound by the instructions that code and transpose (16k tokens of 2 heads of 128 BF16
// into INT8B: 18.0 us, 1.4 TB/s).
constexpr int kBlockWarps = 4;

// Four values -> the four stored bytes at scale s (inv = 1 / s: exact for FP8B, whose scales
// are powers of two; rounded for INT8B, NaN where 1 / s is not a normal number).
template <bool FP8>
__device__ __forceinline__ uint32_t block_codes4(float a, float b, float c, float d, float s, float inv) {
  if (s == 0.f) return FP8 ? 0u : 0x80808080u;
  if constexpr (FP8) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    // Adding 1.5 * 2^23 rounds to the nearest whole number, ties to even, and leaves
    // code + 128 in the low byte.  x * inv is within 2 units in the last place (2^-16 up to
    // 127) of the quotient, so it rounds to the same code unless it lies that near a half:
    // then, and for anything not finite, the division itself is taken.
    constexpr float kMagic = 12583040.f;
    const float y[4] = {a * inv, b * inv, c * inv, d * inv};
    float far = 0.f;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = y[i] + kMagic;
      u[i] = __float_as_uint(m);
      const float off = fabsf(y[i] - (m - kMagic));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(far) : "f"(off));
    }
    if (!(far < 0.4999f)) {
      const float x[4] = {a, b, c, d};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = __float_as_uint(fminf(fmaxf(__fdiv_rn(x[i], s), -127.f), 127.f) + kMagic);
    }
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  }
}
// Four stored bytes coded again (block_recode).
template <bool FP8>
__device__ __forceinline__ uint32_t block_recode4(uint32_t w, float by) {
  uint32_t m = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) m |= block_recode<FP8>((w >> (8 * b)) & 0xffu, by) << (8 * b);
  return m;
}

template <bool FP8, int NEW_DT, int D>
__global__ void __launch_bounds__(kBlockWarps * 32, NEW_DT == kBF16 ? 5 : 1)
    append_block_kernel(uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache,
                        float* __restrict__ k_scale, float* __restrict__ v_scale,
                        const void* __restrict__ k_new, const void* __restrict__ v_new,
                        const int32_t* __restrict__ slots, int T, int Hkv, int num_pages, int group,
                        int32_t* dev_status) {
  constexpr int E = D / 32;  // head-dim elements per lane; also 16-byte pieces of a block
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kBlockWarps + (threadIdx.x >> 5);
  const int which = static_cast<int>(item & 1);
  const int h = static_cast<int>((item >> 1) % Hkv);
  const long long base = (item >> 1) / Hkv * group;  // the first of the warp's tokens
  if (base >= T) return;
  // slots: lane 0 the token before the group, lanes 1 .. group its own, then those behind
  const long long at0 = base - 1 + lane;
  const int slot = at0 >= 0 && at0 < T ? slots[at0] : -1;
  const int prev = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool mine = lane >= 1 && lane <= group && slot >= 0;
  const bool inside = slot < num_pages * kPage;
  const bool joined = prev >= 0 && prev / kPage == slot / kPage;  // its page's run started before
  if (mine && (!inside || (joined && prev + 1 != slot)) && h == 0 && which == 0 && dev_status)
    atomicOr(dev_status, 0x4 /*PKV_DEV_BAD_SLOT*/);
  unsigned leaders = __ballot_sync(0xffffffffu, mine && inside && !joined);
  const void* const src = which ? v_new : k_new;

  while (leaders) {
    const int lead = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    // the run: tokens tok .. tok + n - 1 at offsets off .. off + n - 1 of the page
    const int first = __shfl_sync(0xffffffffu, slot, lead);
    const long long tok = base - 1 + lead;
    const int page = first / kPage, off = first % kPage;
    const unsigned follow = __ballot_sync(0xffffffffu, lane >= lead && off + (lane - lead) < kPage &&
                                                           slot == first + (lane - lead));
    const int n = __ffs(~(follow >> lead)) - 1;
    const size_t blk = static_cast<size_t>(page) * Hkv + h;
    uint8_t* const block = (which ? v_cache : k_cache) + blk * kPage * D;
    float* const scale = (which ? v_scale : k_scale) + blk;

    // old block (only where bytes of it may stay: rows before the run; V also rows behind
    // it): K 16-byte pieces lane + 32 i, V the 16 token bytes of head-dim rows lane * E + i
    const bool old_rows = off > 0, fetch = which ? n < kPage : old_rows;
    const float s_old = old_rows ? *scale : 0.f;
    uint4 was[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
      was[i] = fetch ? reinterpret_cast<const uint4*>(block)[which ? lane * E + i : lane + 32 * i]
                     : make_uint4(0u, 0u, 0u, 0u);
    // the token at page offset t, elements lane * E .. (BF16 pairs stay packed: 32 registers
    // fewer at head_dim 128, and 5 blocks fit an SM)
    constexpr int W = NEW_DT == kBF16 ? E / 2 : E;
    uint32_t raw[kPage][W];
#pragma unroll
    for (int t = 0; t < kPage; ++t) {
#pragma unroll
      for (int e = 0; e < W; ++e) raw[t][e] = 0u;
      if (t >= off && t < off + n) {
        const size_t at = (static_cast<size_t>(tok + t - off) * Hkv + h) * D + lane * E;
        const uint8_t* const p = static_cast<const uint8_t*>(src) + at * (NEW_DT == kBF16 ? 2 : 4);
        if constexpr (W == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          raw[t][0] = v.x; raw[t][1] = v.y; raw[t][2] = v.z; raw[t][3] = v.w;
        } else if constexpr (W == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          raw[t][0] = v.x; raw[t][1] = v.y;
        } else {
          raw[t][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    }
    auto value = [&](int t, int e) -> float {
      if constexpr (NEW_DT == kBF16) {
        const uint32_t v = raw[t][e / 2];
        return __uint_as_float(e & 1 ? v & 0xffff0000u : v << 16);
      } else {
        return __uint_as_float(raw[t][e]);
      }
    };
    float amax = 0.f;
    if constexpr (NEW_DT == kBF16) {
      __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int t = 0; t < kPage; ++t)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t v = raw[t][e] & 0x7fff7fffu;
          top = __hmax2(top, *reinterpret_cast<const __nv_bfloat162*>(&v));
        }
      const float2 f = __bfloat1622float2(top);
      amax = fmaxf(f.x, f.y);
    } else {
#pragma unroll
      for (int t = 0; t < kPage; ++t)
#pragma unroll
        for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(value(t, e)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float need = block_scale<FP8>(amax);
    const float s = old_rows ? fmaxf(s_old, need) : need;
    const bool again = old_rows && s > s_old;
    const float by = again ? __fdiv_rn(s_old, s) : 1.f;
    float inv = s != 0.f ? __fdiv_rn(1.f, s) : 0.f;
    if (!FP8 && !(s > 1e-37f && s < 1e37f)) inv = CUDART_NAN_F;  // (takes the division)
    if (lane == 0) *scale = s;

    if (which == 0) {  // K: a row of D bytes per token
      if (again) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if ((lane + 32 * i) * 16 / D >= off) continue;
          reinterpret_cast<uint4*>(block)[lane + 32 * i] =
              make_uint4(block_recode4<FP8>(was[i].x, by), block_recode4<FP8>(was[i].y, by),
                         block_recode4<FP8>(was[i].z, by), block_recode4<FP8>(was[i].w, by));
        }
      }
#pragma unroll
      for (int t = 0; t < kPage; ++t) {
        if (t < off || t >= off + n) continue;
        uint8_t* const row = block + t * D + lane * E;
        const uint32_t m = block_codes4<FP8>(value(t, 0), value(t, 1), value(t, E - 2), value(t, E - 1), s, inv);
        if constexpr (E == 4) *reinterpret_cast<uint32_t*>(row) = m;
        else *reinterpret_cast<uint16_t*>(row) = static_cast<uint16_t>(m);
      }
    } else {  // V: 16 token bytes per head-dim row; the lane's rows are lane * E ..
      // byte masks of the run's tokens and of the rows before it
      uint32_t m_new[4], m_old[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int lo = min(max(off - 4 * u, 0), 4), hi = min(max(off + n - 4 * u, 0), 4);
        const uint32_t below = lo == 4 ? ~0u : (1u << (8 * lo)) - 1u;
        m_old[u] = below;
        m_new[u] = (hi == 4 ? ~0u : (1u << (8 * hi)) - 1u) & ~below;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        uint32_t w[4] = {was[i].x, was[i].y, was[i].z, was[i].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (again && m_old[u]) w[u] = (w[u] & ~m_old[u]) | (block_recode4<FP8>(w[u], by) & m_old[u]);
          if (m_new[u])
            w[u] = (w[u] & ~m_new[u]) |
                   (block_codes4<FP8>(value(4 * u, i), value(4 * u + 1, i), value(4 * u + 2, i), value(4 * u + 3, i), s, inv) &
                    m_new[u]);
        }
        reinterpret_cast<uint4*>(block)[lane * E + i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <bool FP8>
cudaError_t launch_block(const CacheView& c, void* k, void* v, float* ks, float* vs, const void* kn,
                         const void* vn, int new_dtype, const int32_t* slots, int T,
                         int32_t* dev_status, cudaStream_t st) {
  // Tokens per warp: as few as keep the launch to about 32 warps an SM, all resident at once
  // (a decode step's tokens each lie in a page of their own and have their own warps; a
  // prompt's tokens share pages, and with one token per warp 15 of 16 only find that they do
  // not lead a run).  BF16 rows, 2 heads of 128, us at 1 / 4 / 8 / 16 tokens a warp: 4.6k tokens
  // 16.6 / 5.2 / 5.9 / 7.0, 16k tokens 54 / 23.2 / 20.1 / 17.9.
  int group = 1;
  while (group < 16 && 2ll * ((T + group - 1) / group) * c.Hkv > 152 * 32) group *= group == 1 ? 4 : 2;
  const long long items = 2ll * ((T + group - 1) / group) * c.Hkv;
  if (items / kBlockWarps >= 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((items + kBlockWarps - 1) / kBlockWarps));
  uint8_t* kb = static_cast<uint8_t*>(k);
  uint8_t* vb = static_cast<uint8_t*>(v);
  const bool nb = new_dtype == kBF16;
#define PKV_BLOCK(ND, DD)                                                                      \
  append_block_kernel<FP8, ND, DD><<<grid, kBlockWarps * 32, 0, st>>>(                         \
      kb, vb, ks, vs, kn, vn, slots, T, c.Hkv, c.num_pages, group, dev_status)
  if (c.D == 64) {
    if (nb) PKV_BLOCK(kBF16, 64);
    else PKV_BLOCK(kF32, 64);
  } else {
    if (nb) PKV_BLOCK(kBF16, 128);
    else PKV_BLOCK(kF32, 128);
  }
#undef PKV_BLOCK
  return cudaGetLastError();
}

template <int KV_DT, int NEW_DT>
cudaError_t launch_t(int D, dim3 grid, cudaStream_t st, void* k, void* v, float* ks,
                     float* vs, const void* kn, const void* vn, const int32_t* slots, int T,
                     int Hkv, int NP, int32_t* dev_status) {
  if (D == 64)
    append_kernel<KV_DT, NEW_DT, 64><<<grid, kWarps * 32, 0, st>>>(k, v, ks, vs, kn, vn, slots,
                                                                   T, Hkv, NP, dev_status);
  else
    append_kernel<KV_DT, NEW_DT, 128><<<grid, kWarps * 32, 0, st>>>(k, v, ks, vs, kn, vn, slots,
                                                                    T, Hkv, NP, dev_status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const CacheView& c, void* k_cache, void* v_cache, float* ks,
                          float* vs, const void* k_new, const void* v_new, int new_dtype,
                          const int32_t* slots, int T, int32_t* dev_status, cudaStream_t st) {
  const long long items = static_cast<long long>(T) * c.Hkv;
  const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps));
  const bool nb = new_dtype == kBF16;
  switch (c.dtype) {
    case kF32:
      return nb ? launch_t<kF32, kBF16>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                        slots, T, c.Hkv, c.num_pages, dev_status)
                : launch_t<kF32, kF32>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                       slots, T, c.Hkv, c.num_pages, dev_status);
    case kBF16:
      return nb ? launch_t<kBF16, kBF16>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                         slots, T, c.Hkv, c.num_pages, dev_status)
                : launch_t<kBF16, kF32>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                        slots, T, c.Hkv, c.num_pages, dev_status);
    case kINT8:
      return nb ? launch_t<kINT8, kBF16>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                         slots, T, c.Hkv, c.num_pages, dev_status)
                : launch_t<kINT8, kF32>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                        slots, T, c.Hkv, c.num_pages, dev_status);
    case kFP8:
      return nb ? launch_t<kFP8, kBF16>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                        slots, T, c.Hkv, c.num_pages, dev_status)
                : launch_t<kFP8, kF32>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                       slots, T, c.Hkv, c.num_pages, dev_status);
    case kINT4:
      return nb ? launch_t<kINT4, kBF16>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                         slots, T, c.Hkv, c.num_pages, dev_status)
                : launch_t<kINT4, kF32>(c.D, grid, st, k_cache, v_cache, ks, vs, k_new, v_new,
                                        slots, T, c.Hkv, c.num_pages, dev_status);
    case kINT8B:
      return launch_block<false>(c, k_cache, v_cache, ks, vs, k_new, v_new, new_dtype, slots, T,
                                 dev_status, st);
    case kFP8B:
      return launch_block<true>(c, k_cache, v_cache, ks, vs, k_new, v_new, new_dtype, slots, T,
                                dev_status, st);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
