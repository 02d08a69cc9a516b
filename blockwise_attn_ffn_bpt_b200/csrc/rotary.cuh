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
  int tile, units, chunk; // tokens of a block; units of a token, and of a block's part of it
  int head_shift;         // log2 of the units of a head
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

// Place in the table of angle j of a token: the W angles of a unit are read as
// W / 2 vectors of two angles, and the same vector of neighbouring units lies
// side by side, so that the reads of a warp meet no bank twice.
template <int W>
__device__ __forceinline__ int rot_place(int j, int pairs) {
  if (W == 1) return j;
  const int v = j / W, e = j % W;
  return ((e >> 1) * (pairs / W) + v) * 2 + (e & 1);
}

// One unit is W pairs: two vectors of W elements, which are the pairs' first
// and second halves (the half layout: j and j + rot / 2) or W interleaved
// pairs. W fills 16 bytes where rot / 2 is a multiple of it and every row is
// aligned, and is 1 otherwise. A block has at most ROT_UNROLL units a thread:
// their loads are issued first and fly while the angles are computed.
template <typename T, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ alignas(16) float2 table[ROT_TABLE];
  const int tok0 = blockIdx.x * a.tile;
  const int ntok = min(a.tile, a.tokens - tok0);
  const int beta0 = tok0 / a.s, first = tok0 - beta0 * a.s;
  const int pairs = a.rot >> 1;
  const int rotated = a.rot / (2 * W);
  const int u0 = blockIdx.y * a.chunk, nu = min(a.chunk, a.units - u0);
  const int total = ntok * nu;

  Vec<T, W> p[ROT_UNROLL], q[ROT_UNROLL];
  T* out[ROT_UNROLL];
  int ang[ROT_UNROLL];  // first angle of the unit, or -1 where nothing turns
#pragma unroll
  for (int k = 0; k < ROT_UNROLL; ++k) {
    const int i = threadIdx.x + k * ROT_THREADS;
    out[k] = nullptr;
    if (i >= total) continue;
    const int tt = ntok == 1 ? 0 : i / nu, u = u0 + i - tt * nu;
    int head = u >> a.head_shift;
    const int v = u & ((1 << a.head_shift) - 1);
    const bool keys = head >= a.heads0;
    if (keys) head -= a.heads0;
    const bool turned = v < rotated;
    if (!turned && (keys ? a.in_place1 : a.in_place0)) continue;
    const RotaryTensor& x = a.t[keys ? 1 : 0];
    int beta = beta0, t = first + tt;
    if (t >= a.s) {
      beta += t / a.s;
      t %= a.s;
    }
    // dimensions of the two vectors
    const int d0 = (INTERLEAVED || !turned) ? 2 * W * v : W * v;
    const int gap = (INTERLEAVED || !turned) ? W : a.rot >> 1;
    const long long col = (long long)head * a.dh + d0;
    const T* src = static_cast<const T*>(x.x) + beta * x.bs_x + t * x.ld_x + col;
    out[k] = static_cast<T*>(x.y) + beta * x.bs_y + t * x.ld_y + col;
    ang[k] = turned ? tt * pairs + (W == 1 ? v : 2 * v) : -1;
    p[k] = *reinterpret_cast<const Vec<T, W>*>(src);
    q[k] = *reinterpret_cast<const Vec<T, W>*>(src + gap);
  }

  for (int i = threadIdx.x; i < ntok * pairs; i += ROT_THREADS) {
    const int tt = i / pairs, j = i - tt * pairs;
    int beta = beta0, t = first + tt;
    if (t >= a.s) {
      beta += t / a.s;
      t %= a.s;
    }
    long long pos = a.offset + t;
    if (a.positions != nullptr) {
      const long long at = beta * a.pos_stride + t;
      pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
    }
    const double turn = (double)pos * a.turns[j];
    float sn, cs;
    sincospif(2.0f * (float)(turn - rint(turn)), &sn, &cs);
    table[tt * pairs + rot_place<W>(j, pairs)] = make_float2(cs * a.magnitude, sn * a.sine);
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < ROT_UNROLL; ++k) {
    if (out[k] == nullptr) continue;
    const bool turned = ang[k] >= 0;
    if (turned) {
      float2 cs[W];
      if (W == 1) {
        cs[0] = table[ang[k]];
      } else {
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const float4 two = *reinterpret_cast<const float4*>(&table[ang[k] + e * (pairs / W)]);
          cs[e] = make_float2(two.x, two.y);
          cs[(e + 1) % W] = make_float2(two.z, two.w);
        }
      }
#pragma unroll
      for (int e = 0; e < W; ++e) {
        // pair e: of the two vectors, or of both as one run of interleaved pairs
        T& lo = !INTERLEAVED ? p[k].v[e] : 2 * e < W ? p[k].v[2 * e % W] : q[k].v[2 * e % W];
        T& hi = !INTERLEAVED ? q[k].v[e] : 2 * e + 1 < W ? p[k].v[(2 * e + 1) % W] : q[k].v[(2 * e + 1) % W];
        const float x0 = rot_to_float(lo), x1 = rot_to_float(hi);
        rot_from_float(x0 * cs[e].x - x1 * cs[e].y, lo);
        rot_from_float(x1 * cs[e].x + x0 * cs[e].y, hi);
      }
    }
    *reinterpret_cast<Vec<T, W>*>(out[k]) = p[k];
    *reinterpret_cast<Vec<T, W>*>(out[k] + ((INTERLEAVED || !turned) ? W : a.rot >> 1)) = q[k];
  }
}

}  // namespace bpt
