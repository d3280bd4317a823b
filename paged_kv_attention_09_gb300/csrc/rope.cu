// rope.cu — rotary positions of query and key rows.
//
// Pair i of a head (elements i and i + rotary_dim/2, or 2i and 2i + 1) is turned by the angle
// pos * f_i, f_i = theta^(-2i/rotary_dim), optionally scaled for contexts longer than the
// trained one:
//   linear  f_i / factor
//   base    f_i of the base theta * factor^(rotary_dim / (rotary_dim - 2)): the fastest pair
//           keeps its frequency, the slowest is divided by factor
//   bands   g f_i + (1 - g) f_i / factor, g = clamp((r - low) / (high - low), 0, 1), r the
//           turns original_len * f_i / 2 pi that pair i makes over the trained length
// The transposed form turns by the opposite angle: it is the gradient of the forward one.
//
// Angles.  A float product pos * f_i is off by more than a radian at a few million
// positions, and double sincos is slow on this part.  The frequency is kept instead in turns
// as a 64-bit binary fraction, so that pos * f mod 2^64 is the exact fraction of a turn of
// that frequency (rounding f itself costs pos * 2^-54 turns); read as a signed number and
// converted to float it is the angle over pi in [-1, 1], which sincospif takes.
//
// A block takes a few consecutive tokens.  Their rows come into shared memory by bulk copies
// (one for a token's query heads, one for its key heads: contiguous kilobytes), while the
// threads work out each token's cosines and sines once; then every thread turns vector pairs
// in place (two 16-byte vectors; VE = 8 pairs for BF16, 4 for float) and the rows go out as
// they came.  So the launch's bytes in flight do not hang on registers or on how many heads a
// thread walks over, and partly turned heads cost nothing extra.  Rows, strides or sizes
// that are not multiples of 16 bytes take a plain element-by-element kernel.
// Bound by HBM: every element is read once and written once.  65536 tokens of 36 BF16 heads of
// 64: 91 us, 6.6 TB/s; 8192 tokens of 14 heads of 128 out of fused rows: 11.7 us, 5.0 TB/s (one
// wave of blocks: the launch's ramp and the last blocks' round trips are the rest); a decode
// step of 64 tokens is bound by latency, 2.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "abi.h"
#include "internal.h"
#include "nvtx.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
// Rows of a block, about.  (us at 8 / 12 / 16 / 24 KB: 8192 tokens of 14 BF16 heads of 128 out of
// fused rows 13.5 / 13.2 / 12.6 / 13.3, 65536 tokens of 36 heads of 64 126 / 97 / 93 / 96; with
// 256 threads and 16 KB 15.0 and 113.)
constexpr int kTileBytes = 16 * 1024;
constexpr int kMaxRowBytes = 96 * 1024;  // of one token, for the bulk-copy kernel
constexpr int kMaxTile = 32;

struct RopeArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int32_t* pos;
  int32_t* status;
  long long qs, ks, qos, kos;  // elements from one token to the next
  int Hq, Hk, T, D, rd;
  int tile;    // tokens per block
  float gain, sgn;
  uint64_t freq[PKV_ROPE_MAX_PAIRS];  // turns per position, as a fraction of 2^64
};

// Cosine and sine (with the gain) of pair i at a position >= 0.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int pos, int i) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * a.freq[i];
  // (scaled by 2^-63: the angle over pi, in [-1, 1])
  const float x = __ll2float_rn(static_cast<long long>(turns)) * 1.0842021724855044e-19f;
  float c, s;
  sincospif(x, &s, &c);
  return make_float2(c * a.gain, s * a.sgn);
}

// 16 bytes of elements as they are stored, and as floats.
template <typename T, int N>
__device__ __forceinline__ void widen(uint4 r, float (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  }
}
template <typename T, int N>
__device__ __forceinline__ uint4 narrow(const float (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
}

// Shared memory: the rows [tile][Hq + Hk][D], the angles [tile][VE / 2][units][2] (two pairs
// to 16 bytes, so that neighbouring units read neighbouring 16 bytes), the barrier.
template <typename T, int VE, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int t0 = blockIdx.x * a.tile, nt = min(a.tile, a.T - t0);
  const int H = a.Hq + a.Hk, D = a.D, half = a.rd / 2, units = half / VE;
  const uint32_t qb = a.Hq * D * sizeof(T), kb = a.Hk * D * sizeof(T), row = qb + kb;
  float* const angles = reinterpret_cast<float*>(smem + static_cast<size_t>(a.tile) * row);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(angles + 2 * a.tile * half);
  const int tid = threadIdx.x;

  // warp 0: one lane per token requests (and later returns) its rows; a token at a negative
  // position is padding and is left alone
  const bool live = tid < nt && a.pos[t0 + tid] >= 0;
  if (tid < 32) {
    const unsigned n = __popc(__ballot_sync(0xffffffffu, live));
    if (tid == 0) {
      mbar_init(bar, 1);
      fence_barrier_init();
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, n * row);
    }
    __syncwarp();
    if (live) {
      const uint64_t pol = l2_evict_first_policy();
      uint8_t* const dst = smem + tid * row;
      if (qb) bulk_g2s(dst, static_cast<const T*>(a.q) + (t0 + tid) * a.qs, qb, bar, pol);
      if (kb) bulk_g2s(dst + qb, static_cast<const T*>(a.k) + (t0 + tid) * a.ks, kb, bar, pol);
    }
  }
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, e = i - t * half;
    const int at = ((e % VE) / 2 * units + e / VE) * 2 + (e & 1);
    reinterpret_cast<float2*>(angles)[t * half + at] = turn_of(a, max(a.pos[t0 + t], 0), e);
  }
  __syncthreads();  // (the barrier is initialised, too)
  if (!mbar_wait(bar, 0)) {
    (void)mbar_wait(bar, 0);  // no copy may land in the memory of a block that has left
    if (a.status) atomicOr(a.status, 0x10);  // PKV_DEV_TIMEOUT
    return;
  }
  // A thread keeps the angles of VE pairs of a token and turns every `share`-th head by them (the
  // prefill above: 12.5 us with the angles read again for each head).
  const int share = max(1, min(H, kThreads / (nt * units))), per_token = share * units;
  for (int i = tid; i < nt * per_token; i += kThreads) {
    const int t = i / per_token, it = i - t * per_token, h0 = it / units, j = it - h0 * units;
    float c[VE], s[VE];
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      const float4 v = *reinterpret_cast<const float4*>(angles + 2 * (t * half + (e / 2 * units + j) * 2));
      c[e] = v.x; s[e] = v.y; c[e + 1] = v.z; s[e + 1] = v.w;
    }
    uint8_t* px = smem + t * row + (h0 * D + (HALF ? j * VE : 2 * j * VE)) * sizeof(T);
    for (int h = h0; h < H; h += share, px += share * D * sizeof(T)) {
      uint8_t* const py = px + (HALF ? half : VE) * sizeof(T);
      float x[VE], y[VE], u[VE], v[VE];
      widen<T, VE>(*reinterpret_cast<const uint4*>(px), x);
      widen<T, VE>(*reinterpret_cast<const uint4*>(py), y);
      if constexpr (HALF) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          u[e] = fmaf(x[e], c[e], -(y[e] * s[e]));
          v[e] = fmaf(y[e], c[e], x[e] * s[e]);
        }
      } else {  // pairs lie side by side: VE / 2 of them in each vector
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          u[2 * e] = fmaf(x[2 * e], c[e], -(x[2 * e + 1] * s[e]));
          u[2 * e + 1] = fmaf(x[2 * e + 1], c[e], x[2 * e] * s[e]);
          v[2 * e] = fmaf(y[2 * e], c[VE / 2 + e], -(y[2 * e + 1] * s[VE / 2 + e]));
          v[2 * e + 1] = fmaf(y[2 * e + 1], c[VE / 2 + e], y[2 * e] * s[VE / 2 + e]);
        }
      }
      *reinterpret_cast<uint4*>(px) = narrow<T, VE>(u);
      *reinterpret_cast<uint4*>(py) = narrow<T, VE>(v);
    }
  }
  fence_proxy_async_smem();  // the turned rows are visible to the copies
  __syncthreads();
  if (live) {
    const uint8_t* const src = smem + tid * row;
    if (qb) bulk_s2g(static_cast<T*>(a.q_out) + (t0 + tid) * a.qos, src, qb);
    if (kb) bulk_s2g(static_cast<T*>(a.k_out) + (t0 + tid) * a.kos, src + qb, kb);
    bulk_store_wait();
  }
}

// Element by element: one thread per (token, pair or copied column), over the heads.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_elements_kernel(const __grid_constant__ RopeArgs a) {
  const int half = a.rd / 2, units = half + a.D - a.rd;
  const long long idx = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long t = idx / units;
  const int j = static_cast<int>(idx - t * units);
  if (t >= a.T) return;
  const int pos = a.pos[t];
  if (pos < 0) return;
  const bool turned = j < half;
  const int ca = !turned ? a.rd + j - half : HALF ? j : 2 * j, cb = HALF ? ca + half : ca + 1;
  const float2 cs = turned ? turn_of(a, pos, j) : make_float2(0.f, 0.f);
  for (int h = 0; h < a.Hq + a.Hk; ++h) {
    const bool isq = h < a.Hq;
    const size_t at = static_cast<size_t>(isq ? h : h - a.Hq) * a.D;
    const T* p = isq ? static_cast<const T*>(a.q) + t * a.qs + at : static_cast<const T*>(a.k) + t * a.ks + at;
    T* o = isq ? static_cast<T*>(a.q_out) + t * a.qos + at : static_cast<T*>(a.k_out) + t * a.kos + at;
    if (!turned) {
      if (p != o) o[ca] = p[ca];
      continue;
    }
    const float x = static_cast<float>(p[ca]), y = static_cast<float>(p[cb]);
    o[ca] = static_cast<T>(fmaf(x, cs.x, -(y * cs.y)));
    o[cb] = static_cast<T>(fmaf(y, cs.x, x * cs.y));
  }
}

template <typename T>
const void* kernel_of(bool rows, bool half) {
  constexpr int VE = 16 / sizeof(T);
  if (rows)
    return half ? reinterpret_cast<const void*>(&rope_rows_kernel<T, VE, true>)
                : reinterpret_cast<const void*>(&rope_rows_kernel<T, VE, false>);
  return half ? reinterpret_cast<const void*>(&rope_elements_kernel<T, true>)
              : reinterpret_cast<const void*>(&rope_elements_kernel<T, false>);
}

// Turns per position of pair i as a fraction of 2^64 (frequencies are below one turn).
uint64_t turns_of(double f) {
  const double t = std::ldexp(f / 6.283185307179586476925, 64);
  return t >= 18446744073709549568.0 ? ~0ull : static_cast<uint64_t>(t);
}

// The frequencies of the description; false if it is out of range.
bool frequencies(const pkv_rope_params* r, uint64_t* freq) {
  const int rd = r->rotary_dim;
  if (!(r->theta > 1.0) || !std::isfinite(r->theta)) return false;
  if (r->scaling < PKV_ROPE_NONE || r->scaling > PKV_ROPE_BANDS) return false;
  const bool scaled = r->scaling != PKV_ROPE_NONE;
  if (scaled && (!(r->factor >= 1.0) || !std::isfinite(r->factor))) return false;
  if (r->scaling == PKV_ROPE_BANDS &&
      (!(r->low >= 0.0) || !(r->high > r->low) || !std::isfinite(r->high) || r->original_len < 1))
    return false;
  double theta = r->theta;
  if (r->scaling == PKV_ROPE_BASE && rd > 2)
    theta *= std::pow(r->factor, static_cast<double>(rd) / (rd - 2));
  for (int i = 0; i < rd / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rd);
    if (r->scaling == PKV_ROPE_LINEAR) {
      f /= r->factor;
    } else if (r->scaling == PKV_ROPE_BANDS) {
      const double turns = r->original_len * f / 6.283185307179586476925;
      double g = (turns - r->low) / (r->high - r->low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = g * f + (1.0 - g) * (f / r->factor);
    }
    freq[i] = turns_of(f);
  }
  return true;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_rope_plan_init(const pkv_rope_params* params, pkv_rope_plan* plan) {
  PKV_RANGE("pkv_rope_plan_init");
  if (!params || !plan) return PKV_ERR_NULL;
  const int rd = params->rotary_dim;
  if (rd < 2 || (rd & 1)) return PKV_ERR_SHAPE;
  if (rd > 2 * PKV_ROPE_MAX_PAIRS) return PKV_ERR_UNSUPPORTED;
  if (params->layout != PKV_ROPE_HALF && params->layout != PKV_ROPE_INTERLEAVED) return PKV_ERR_SHAPE;
  if (!std::isfinite(params->attention_factor) || params->attention_factor < 0.f) return PKV_ERR_SHAPE;
  pkv_rope_plan made{};
  if (!pkv::frequencies(params, made.freq)) return PKV_ERR_SHAPE;
  made.rotary_dim = rd;
  made.layout = params->layout;
  made.transposed = params->transposed != 0;
  made.attention_factor = params->attention_factor == 0.f ? 1.f : params->attention_factor;
  *plan = made;
  return PKV_OK;
}

extern "C" pkv_status pkv_rope(const pkv_rope_plan* plan, const void* q, void* q_out, int64_t q_stride,
                               int64_t q_out_stride, int32_t num_q_heads, const void* k, void* k_out,
                               int64_t k_stride, int64_t k_out_stride, int32_t num_kv_heads, int32_t dtype,
                               int32_t num_tokens, int32_t head_dim, const int32_t* positions,
                               int32_t* dev_status, void* stream) {
  PKV_RANGE("pkv_rope");
  if (!plan) return PKV_ERR_NULL;
  if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_DTYPE;
  const int rd = plan->rotary_dim;
  if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 ||
      num_q_heads + static_cast<long long>(num_kv_heads) > 65535 || rd < 2 || (rd & 1) || rd > head_dim)
    return PKV_ERR_SHAPE;
  if (head_dim > 2 * PKV_ROPE_MAX_PAIRS) return PKV_ERR_UNSUPPORTED;
  pkv::RopeArgs a{};
  const long long qrow = static_cast<long long>(num_q_heads) * head_dim;
  const long long krow = static_cast<long long>(num_kv_heads) * head_dim;
  a.qs = q_stride ? q_stride : qrow;
  a.qos = q_out_stride ? q_out_stride : qrow;
  a.ks = k_stride ? k_stride : krow;
  a.kos = k_out_stride ? k_out_stride : krow;
  if (a.qs < 0 || a.qos < 0 || a.ks < 0 || a.kos < 0) return PKV_ERR_SHAPE;
  if (num_tokens > 1 && (a.qs < qrow || a.qos < qrow || a.ks < krow || a.kos < krow)) return PKV_ERR_SHAPE;
  if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PKV_OK;
  if (!positions || (num_q_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || !k_out)))
    return PKV_ERR_NULL;
  // in place means row by row: the same rows at the same stride
  if ((num_q_heads > 0 && q == q_out && a.qs != a.qos) || (num_kv_heads > 0 && k == k_out && a.ks != a.kos))
    return PKV_ERR_SHAPE;
  const int elt = dtype == PKV_F32 ? 4 : 2, ve = 16 / elt;
  const uintptr_t bases = (num_q_heads ? reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) : 0) |
                          (num_kv_heads ? reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(k_out) : 0);
  if (bases % elt || !pkv::aligned4(positions) || !pkv::aligned4(dev_status)) return PKV_ERR_ALIGN;
  const long long strides = (num_q_heads ? a.qs | a.qos : 0) | (num_kv_heads ? a.ks | a.kos : 0);
  // bulk copies and 16-byte vectors when every row, every head and both halves of the turned
  // columns start on a 16-byte boundary; single elements otherwise
  const long long per_token = (qrow + krow) * elt;
  const bool rows = bases % 16 == 0 && strides % ve == 0 && head_dim % ve == 0 && (rd / 2) % ve == 0 &&
                    per_token <= pkv::kMaxRowBytes;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.pos = positions;
  a.status = dev_status;
  a.Hq = num_q_heads;
  a.Hk = num_kv_heads;
  a.T = num_tokens;
  a.D = head_dim;
  a.rd = rd;
  a.gain = plan->attention_factor;
  a.sgn = plan->transposed ? -a.gain : a.gain;
  for (int i = 0; i < rd / 2; ++i) a.freq[i] = plan->freq[i];
  long long blocks;
  size_t smem = 0;
  if (rows) {
    // Tokens per block: about kTileBytes of rows, fewer while that would leave SMs without a
    // block (a decode step's tokens get a block each).
    long long tile = pkv::kTileBytes / per_token;
    const long long spread = (num_tokens + 152 * 4 - 1) / (152 * 4);
    if (tile > spread) tile = spread;
    if (tile > pkv::kMaxTile) tile = pkv::kMaxTile;
    if (tile < 1) tile = 1;
    a.tile = static_cast<int>(tile);
    blocks = (num_tokens + tile - 1) / tile;
    smem = static_cast<size_t>(tile) * (per_token + (rd / 2) * sizeof(float2)) + 16;
  } else {
    blocks = (static_cast<long long>(num_tokens) * (rd / 2 + head_dim - rd) + pkv::kThreads - 1) / pkv::kThreads;
  }
  if (blocks > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  const bool half = plan->layout == PKV_ROPE_HALF;
  const void* fn = dtype == PKV_F32 ? pkv::kernel_of<float>(rows, half) : pkv::kernel_of<__nv_bfloat16>(rows, half);
  if (smem > 48 * 1024 &&  // (rows of very many heads)
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) != cudaSuccess)
    return PKV_ERR_LAUNCH;
  void* args[] = {&a};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(pkv::kThreads), args, smem,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
