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
// One thread owns one token's VE pairs (two 16-byte vectors of every head; VE = 8 for
// BF16, 4 for float) and walks over the heads: its VE cosines and sines stay in registers,
// no shared memory, no barrier, and the loads of several heads are in flight at once.  Heads
// are divided among several threads only while the launch would otherwise not fill the GPU.
// Bound by HBM: every element is read once and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "abi.h"
#include "internal.h"
#include "nvtx.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;

struct RopeArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int32_t* pos;
  long long qs, ks, qos, kos;  // elements from one token to the next
  int Hq, Hk, T, D, rd;
  int units;  // threads per token and head group: turned pair vectors, then copied ones
  int turned;
  int groups;
  float gain, sgn;
  uint64_t freq[PKV_ROPE_MAX_PAIRS];  // turns per position, as a fraction of 2^64
};

// N consecutive elements as floats
template <typename T, int N>
__device__ __forceinline__ void load(const T* p, float (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (N == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      x[0] = __bfloat162float(*p);
    }
  } else {
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      x[0] = *p;
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (N == 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *p = __float2bfloat16_rn(x[0]);
    }
  } else {
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *p = x[0];
  }
}

// T: element type; VE: pairs per thread (16-byte vectors, or 1 for sizes and strides that
// are not multiples of them); HALF: half layout, else interleaved.
template <typename T, int VE, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  const long long idx = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long t = idx / a.units;
  const int j = static_cast<int>(idx - t * a.units);
  if (t >= a.T) return;
  const int pos = a.pos[t];
  if (pos < 0) return;  // padding: the row is left alone
  const T* q = static_cast<const T*>(a.q) + t * a.qs;
  const T* k = static_cast<const T*>(a.k) + t * a.ks;
  T* qo = static_cast<T*>(a.q_out) + t * a.qos;
  T* ko = static_cast<T*>(a.k_out) + t * a.kos;
  const int H = a.Hq + a.Hk, D = a.D;
  auto from = [&](int h) { return h < a.Hq ? q + static_cast<size_t>(h) * D : k + static_cast<size_t>(h - a.Hq) * D; };
  auto to = [&](int h) { return h < a.Hq ? qo + static_cast<size_t>(h) * D : ko + static_cast<size_t>(h - a.Hq) * D; };
  if (j >= a.turned) {  // columns that are not turned, copied when the output is elsewhere
    const int col = a.rd + (j - a.turned) * VE;
    for (int h = blockIdx.y; h < H; h += a.groups) {
      if (from(h) == to(h)) continue;
      float x[VE];
      load<T, VE>(from(h) + col, x);
      store<T, VE>(to(h) + col, x);
    }
    return;
  }
  const int ca = HALF ? j * VE : 2 * j * VE;         // first vector's column
  const int cb = HALF ? ca + a.rd / 2 : ca + VE;     // second vector's
  float c[VE], s[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * a.freq[j * VE + e];
    // (scaled by 2^-63: the angle over pi, in [-1, 1])
    const float x = __ll2float_rn(static_cast<long long>(turns)) * 1.0842021724855044e-19f;
    sincospif(x, &s[e], &c[e]);
    c[e] *= a.gain;
    s[e] *= a.sgn;
  }
#pragma unroll 4
  for (int h = blockIdx.y; h < H; h += a.groups) {
    const T* p = from(h);
    T* o = to(h);
    float x[VE], y[VE], u[VE], v[VE];
    load<T, VE>(p + ca, x);
    load<T, VE>(p + cb, y);
    if constexpr (HALF || VE == 1) {
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
    store<T, VE>(o + ca, u);
    store<T, VE>(o + cb, v);
  }
}

template <typename T, int VE>
const void* kernel_of(bool half) {
  return half ? reinterpret_cast<const void*>(&rope_kernel<T, VE, true>)
              : reinterpret_cast<const void*>(&rope_kernel<T, VE, false>);
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
                               void* stream) {
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
  if (bases % elt || !pkv::aligned4(positions)) return PKV_ERR_ALIGN;
  const long long strides = (num_q_heads ? a.qs | a.qos : 0) | (num_kv_heads ? a.ks | a.kos : 0);
  // 16-byte vectors when every row, every head and both halves of the turned columns start
  // on a 16-byte boundary; single elements otherwise
  const bool vec = bases % 16 == 0 && strides % ve == 0 && head_dim % ve == 0 && (rd / 2) % ve == 0;
  const int per = vec ? ve : 1;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.pos = positions;
  a.Hq = num_q_heads;
  a.Hk = num_kv_heads;
  a.T = num_tokens;
  a.D = head_dim;
  a.rd = rd;
  a.turned = rd / 2 / per;
  const bool elsewhere = (num_q_heads && q != q_out) || (num_kv_heads && k != k_out);
  a.units = a.turned + (elsewhere ? (head_dim - rd) / per : 0);
  a.gain = plan->attention_factor;
  a.sgn = plan->transposed ? -a.gain : a.gain;
  for (int i = 0; i < rd / 2; ++i) a.freq[i] = plan->freq[i];
  // Heads per thread: all of them once the tokens alone give every SM a few hundred threads.
  const long long threads = static_cast<long long>(num_tokens) * a.units;
  const int H = num_q_heads + num_kv_heads;
  const long long want = 152 * 512;
  long long groups = threads >= want ? 1 : (want + threads - 1) / threads;
  a.groups = static_cast<int>(groups > H ? H : groups);
  const long long blocks = (threads + pkv::kThreads - 1) / pkv::kThreads;
  if (blocks > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  const void* fn;
  const bool half = plan->layout == PKV_ROPE_HALF;
  if (dtype == PKV_F32) fn = vec ? pkv::kernel_of<float, 4>(half) : pkv::kernel_of<float, 1>(half);
  else fn = vec ? pkv::kernel_of<__nv_bfloat16, 8>(half) : pkv::kernel_of<__nv_bfloat16, 1>(half);
  void* args[] = {&a};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(blocks), a.groups), dim3(pkv::kThreads), args,
                                         0, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
