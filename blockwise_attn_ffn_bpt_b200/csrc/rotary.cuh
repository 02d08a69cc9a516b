// Rotary positions of the queries and keys, forward and backward.
//
// For a pair of dimensions (x0, x1) of a head at position pos, with f the
// pair's radians per position, a = pos f and magnitude m:
//     y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a).
// The map is linear and its transpose turns by -a: the gradient is the same
// kernel with the sign of the sine flipped.
//
// Bound by HBM: every element is read once and written once. The angles cost
// little because a token's rot / 2 angles serve all of its heads, queries and
// keys: a block computes them once per token into shared memory. An angle is
// taken in turns in fp64 (pos * f / 2 pi, less its nearest whole number), so
// that positions in the millions keep fp32 accuracy in what is left; the sine
// and cosine of the remainder are then fp32.
#pragma once

#include "ptx.cuh"

namespace bpt {

constexpr int ROT_THREADS = 256;
constexpr int ROT_MAX_PAIRS = 64;           // rot <= 128
constexpr int ROT_TABLE = 8 * ROT_MAX_PAIRS;  // angles of a block's tokens
constexpr int ROT_UNROLL = 4;

struct RotaryTensor {
  const void* x;
  void* y;
  long long bs_x, ld_x, bs_y, ld_y;  // elements between sequences and between tokens
};

struct RotaryArgs {
  RotaryTensor t[2];      // queries, keys
  int heads0, heads1;
  int in_place0, in_place1;
  int tokens, s;          // b * s, and the tokens of a sequence
  int dh, rot;
  int tile, units, chunk; // tokens of a block; vector pairs of a token, and of a block's part of it
  const void* positions;  // int32 or int64 [b, s] (pos_stride between sequences), or null: offset + t
  int pos64;
  long long pos_stride, offset;
  float magnitude, sine;  // sine: +magnitude, or -magnitude for the transpose
  double turns[ROT_MAX_PAIRS];
};

template <typename T, int W>
struct alignas(sizeof(T) * W) Vec {
  T v[W];
};

__device__ __forceinline__ float rot_to_float(float x) { return x; }
__device__ __forceinline__ float rot_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void rot_from_float(float x, float& y) { y = x; }
__device__ __forceinline__ void rot_from_float(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// One unit is W pairs: two vectors of W elements, which are the pairs' first
// and second halves (the half layout: j and j + rot / 2) or W interleaved
// pairs. W fills 16 bytes where rot / 2 is a multiple of it and every row is
// aligned, and is 1 otherwise.
template <typename T, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ float2 table[ROT_TABLE];
  const int tok0 = blockIdx.x * a.tile;
  const int ntok = min(a.tile, a.tokens - tok0);
  const int pairs = a.rot >> 1;
  for (int i = threadIdx.x; i < ntok * pairs; i += ROT_THREADS) {
    const int tt = i / pairs, j = i - tt * pairs;
    const int tok = tok0 + tt, beta = tok / a.s, t = tok - beta * a.s;
    long long pos = a.offset + t;
    if (a.positions != nullptr) {
      const long long at = beta * a.pos_stride + t;
      pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
    }
    const double turn = (double)pos * a.turns[j];
    float sn, cs;
    sincospif(2.0f * (float)(turn - rint(turn)), &sn, &cs);
    table[i] = make_float2(cs * a.magnitude, sn * a.sine);
  }
  __syncthreads();

  const int per_head = a.dh / (2 * W), rotated = a.rot / (2 * W);
  const int u0 = blockIdx.y * a.chunk, nu = min(a.chunk, a.units - u0);
  const int total = ntok * nu;
  for (int i0 = threadIdx.x; i0 < total; i0 += ROT_THREADS * ROT_UNROLL) {
    Vec<T, W> p[ROT_UNROLL], q[ROT_UNROLL];
    T* out[ROT_UNROLL];
    const float2* ang[ROT_UNROLL];
    int gap[ROT_UNROLL];
#pragma unroll
    for (int k = 0; k < ROT_UNROLL; ++k) {
      const int i = i0 + k * ROT_THREADS;
      out[k] = nullptr;
      if (i >= total) continue;
      const int tt = i / nu, u = u0 + i - tt * nu;
      int head = u / per_head;
      const int v = u - head * per_head;
      const bool keys = head >= a.heads0;
      if (keys) head -= a.heads0;
      const bool turned = v < rotated;
      if (!turned && (keys ? a.in_place1 : a.in_place0)) continue;
      const RotaryTensor& x = a.t[keys ? 1 : 0];
      const int tok = tok0 + tt, beta = tok / a.s, t = tok - beta * a.s;
      // dimensions of the two vectors
      const int d0 = (INTERLEAVED || !turned) ? 2 * W * v : W * v;
      gap[k] = (INTERLEAVED || !turned) ? W : a.rot >> 1;
      const long long col = (long long)head * a.dh + d0;
      const T* src = static_cast<const T*>(x.x) + beta * x.bs_x + t * x.ld_x + col;
      out[k] = static_cast<T*>(x.y) + beta * x.bs_y + t * x.ld_y + col;
      ang[k] = turned ? table + tt * pairs + W * v : nullptr;
      p[k] = *reinterpret_cast<const Vec<T, W>*>(src);
      q[k] = *reinterpret_cast<const Vec<T, W>*>(src + gap[k]);
    }
#pragma unroll
    for (int k = 0; k < ROT_UNROLL; ++k) {
      if (out[k] == nullptr) continue;
      if (ang[k] != nullptr) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 cs = ang[k][e];
          if (INTERLEAVED) {  // pair e of the unit: elements 2e, 2e + 1 of the two vectors together
            T& lo = 2 * e < W ? p[k].v[2 * e % W] : q[k].v[2 * e % W];
            T& hi = 2 * e + 1 < W ? p[k].v[(2 * e + 1) % W] : q[k].v[(2 * e + 1) % W];
            const float x0 = rot_to_float(lo), x1 = rot_to_float(hi);
            rot_from_float(x0 * cs.x - x1 * cs.y, lo);
            rot_from_float(x1 * cs.x + x0 * cs.y, hi);
          } else {
            const float x0 = rot_to_float(p[k].v[e]), x1 = rot_to_float(q[k].v[e]);
            rot_from_float(x0 * cs.x - x1 * cs.y, p[k].v[e]);
            rot_from_float(x1 * cs.x + x0 * cs.y, q[k].v[e]);
          }
        }
      }
      *reinterpret_cast<Vec<T, W>*>(out[k]) = p[k];
      *reinterpret_cast<Vec<T, W>*>(out[k] + gap[k]) = q[k];
    }
  }
}

}  // namespace bpt
