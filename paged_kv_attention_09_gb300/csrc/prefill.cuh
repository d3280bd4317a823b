// prefill.cuh — what the chunked-prefill kernels share: the launch parameters, the operand
// tile layout, and the merge of row tiles whose key range several blocks shared.
#pragma once
#include <math_constants.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kRowsTC = 128;      // query rows per block (MMA M)
constexpr int kKeysTC = 64;       // keys per tile (MMA N of S)
constexpr int kPagesTC = kKeysTC / kPage;
constexpr float kRescaleLog2 = 8.f;  // raise the running max only beyond this margin

struct TParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;  // block scales (block-scaled formats)
  const float* vs;
  const void* q;
  const int32_t* qsl;
  const int32_t* bt;
  const int32_t* lens;
  float* out;
  int32_t* dev_status;
  // key-range split: each row tile's key tiles are divided among ksplit blocks, which
  // leave partial (max, sum, O) states in the workspace for the last of them to merge
  int ksplit;
  float* ws_o;      // [tile][split][row][D]
  float* ws_m;      // [tile][split][row]
  float* ws_l;      // [tile][split][row]
  int* ws_ticket;   // [tile]
  int q_dtype, Hkv, Hq, G, MB, num_pages;
  int window;  // sliding window in tokens (0: none)
  float scale_log2;
};

// Byte offset of element (row, col) in a no-swizzle K-major tile whose K extent is
// kext elements: core matrix (row / 8, col / 8), row % 8, element col % 8.
__device__ __forceinline__ uint32_t tile_off(int row, int col, int kext) {
  return ((((row >> 3) * (kext >> 3)) + (col >> 3)) << 7) + ((row & 7) << 4) + ((col & 7) << 1);
}

// Index of a row tile of the launch: [sequence][kv head][row tile].
__device__ __forceinline__ int tile_index(const TParams& p, int tile, int g, int b) {
  return (b * p.Hkv + g) * (gridDim.x / p.ksplit) + tile;
}

// Key-range split: the block that takes a row tile's last ticket (an atomic, no waiting)
// merges the ksplit partial states of its 128 rows, in split order, into the output,
// and resets the ticket.  `scratch`: ((ksplit + 1) x 128) floats of shared memory.
template <int D, int kThreads>
__device__ __noinline__ void split_merge(const TParams& p, int tile, int g, int b, int q0, int nrows,
                                         int err, int tid, uint8_t* scratch) {
  __shared__ int s_last;
  // The parameters are read once into registers: this function is not inlined, so each
  // use of p would be a load through a generic pointer, repeated after every store.
  const int KS = p.ksplit, G = p.G, Hq = p.Hq;
  float* const out = p.out;
  const float* const ws_o = p.ws_o;
  const float* const ws_m = p.ws_m;
  const float* const ws_l = p.ws_l;
  const int tix = tile_index(p, tile, g, b);
  __threadfence();
  __syncthreads();
  int* ticket = p.ws_ticket + tix;
  if (tid == 0) s_last = atomicAdd(ticket, 1) == KS - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const size_t base = static_cast<size_t>(tix) * KS * kRowsTC;
  const int row0 = tile * kRowsTC;
  float* wts = reinterpret_cast<float*>(scratch);  // [split][row], then [row] 1 / sum
  if (tid < kRowsTC) {
    const int r = tid;
    float m[3], l[3];
#pragma unroll
    for (int s = 0; s < 3; ++s) {  // every load in flight at once
      m[s] = s < KS ? __ldcg(ws_m + base + s * kRowsTC + r) : -CUDART_INF_F;
      l[s] = s < KS ? __ldcg(ws_l + base + s * kRowsTC + r) : 0.f;
    }
    const bool poisoned = isnan(m[0]) || isnan(m[1]) || isnan(m[2]);
    const float M = fmaxf(fmaxf(m[0], m[1]), m[2]);
    float L = 0.f;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const float f = m[s] == -CUDART_INF_F ? 0.f : fast_exp2(m[s] - M);
      if (s < KS) wts[s * kRowsTC + r] = f;
      L += l[s] * f;
    }
    wts[KS * kRowsTC + r] = poisoned ? CUDART_NAN_F : 1.f / L;
  }
  __syncthreads();
  if (!err) {
    constexpr int D4 = D / 4;
    constexpr int CH = 4;  // output chunks per thread and round: their loads go out together
    for (int c0 = tid; c0 < kRowsTC * D4; c0 += CH * kThreads) {
      float4 v[CH][3];
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int c = c0 + u * kThreads;
        const int r = c / D4, d4 = c % D4;
#pragma unroll
        for (int s = 0; s < 3; ++s)
          v[u][s] = c < kRowsTC * D4 && s < KS
                        ? __ldcg(reinterpret_cast<const float4*>(ws_o + (base + s * kRowsTC + r) * D) + d4)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int c = c0 + u * kThreads;
        const int r = c / D4, d4 = c % D4;
        const int rho = row0 + r;
        if (c >= kRowsTC * D4 || rho >= nrows) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          if (s < KS) {
            const float f = wts[s * kRowsTC + r];
            acc.x += v[u][s].x * f; acc.y += v[u][s].y * f; acc.z += v[u][s].z * f; acc.w += v[u][s].w * f;
          }
        }
        const float inv = wts[KS * kRowsTC + r];
        float* dst = out + (static_cast<size_t>(q0 + rho / G) * Hq + g * G + rho % G) * D;
        reinterpret_cast<float4*>(dst)[d4] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      }
    }
  }
  if (tid == 0) *ticket = 0;  // leave the counter ready for the next call
}

// The parameters of a launch over n_row_tiles x ksplit blocks per (sequence, kv head).
TParams params_of(const PrefillArgs& a, int n_row_tiles, int ksplit) {
  TParams p{};
  p.k = static_cast<const uint8_t*>(a.c.k);
  p.v = static_cast<const uint8_t*>(a.c.v);
  p.ks = a.c.ks;
  p.vs = a.c.vs;
  p.q = a.q;
  p.qsl = a.q_start_loc;
  p.bt = a.block_tables;
  p.lens = a.context_lens;
  p.out = a.out;
  p.dev_status = a.dev_status;
  p.q_dtype = a.q_dtype;
  p.Hkv = a.c.Hkv;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.MB = a.MB;
  p.num_pages = a.c.num_pages;
  p.window = a.c.window;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.ksplit = ksplit;
  if (ksplit > 1) {
    const size_t tiles = static_cast<size_t>(n_row_tiles) * a.c.Hkv * a.B;
    uint8_t* base = static_cast<uint8_t*>(a.ws);
    p.ws_ticket = reinterpret_cast<int*>(base);
    float* f = reinterpret_cast<float*>(base + ((tiles * 4 + 255) / 256) * 256);
    const size_t rows = tiles * ksplit * kRowsTC;
    p.ws_o = f;
    p.ws_m = f + rows * a.c.D;
    p.ws_l = p.ws_m + rows;
  }
  return p;
}

}  // namespace
}  // namespace pkv
