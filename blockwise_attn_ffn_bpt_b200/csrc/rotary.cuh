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
// that positions in the millions keep fp32 accuracy in what is left. Sine and
// cosine are fp32's of the remainder in fp32, plus the first order of what that
// rounding leaves (up to 9e-8 rad), rounded once with the magnitude.
#pragma once

#include "ptx.cuh"

namespace bpt {

// Measured at 8192 tokens of 64 heads of 128 in bf16 (268 MB in all, 41 us at
// the copy's rate), device time: 4 units a thread loaded at once and 2 tokens a
// block, 75 us (2 blocks fit an SM); one unit ahead and 8 tokens a block, 50.6
// us with 5 blocks an SM, 52.8 with 4, 50.6 with 6; grids of 2, 4 and 8 rounds
// of blocks 55.7, 52.8 and 58.8 us.
constexpr int ROT_THREADS = 256;
constexpr int ROT_BLOCKS = 5;                 // of an SM
constexpr int ROT_ROUNDS = 4;                 // of the grid, at least, before a block takes more tokens
constexpr int ROT_MAX_PAIRS = 64;             // rot <= 128
constexpr int ROT_TABLE = 8 * ROT_MAX_PAIRS;  // angles of a block's tokens
constexpr int ROT_CHUNK = 1024;               // units of one token that a block takes at most

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
// aligned, and otherwise the largest part of that for which both hold: the 8192
// tokens above take 47 us with 16 bytes, 62 with 8 (rot = 24), 99 with 4 (rot = 20)
// and 178 with 2. A thread takes every ROT_THREADS-th unit of the
// block's tokens, with the next one's loads in flight (the first one's while the
// block computes its angles).
template <typename T, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(ROT_THREADS, ROT_BLOCKS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ alignas(16) float2 table[ROT_TABLE];
  grid_dependency_wait();
  grid_dependents_start();
  const int tok0 = blockIdx.x * a.tile;
  const int ntok = min(a.tile, a.tokens - tok0);
  const int beta0 = tok0 / a.s, first = tok0 - beta0 * a.s;
  const int pairs = a.rot >> 1;
  const int rotated = a.rot / (2 * W);
  const int u0 = blockIdx.y * a.chunk, nu = min(a.chunk, a.units - u0);

  // the thread's next unit: unit u of the block's part of token tt
  int tt = threadIdx.x / nu, u = threadIdx.x - tt * nu;
  const int step_tt = ROT_THREADS / nu, step_u = ROT_THREADS - step_tt * nu;

  struct Unit {
    Vec<T, W> p, q;
    T* out;
    int angle;  // its first angle, or -1 where nothing turns
  };
  auto load = [&](Unit& x) {
    x.out = nullptr;
    if (tt >= ntok) return;
    int head = (u0 + u) >> a.head_shift;
    const int v = (u0 + u) & ((1 << a.head_shift) - 1);
    const bool keys = head >= a.heads0;
    if (keys) head -= a.heads0;
    const bool turned = v < rotated;
    int beta = beta0, t = first + tt;
    if (t >= a.s) {
      beta += t / a.s;
      t %= a.s;
    }
    if (turned || !(keys ? a.in_place1 : a.in_place0)) {
      const RotaryTensor& y = a.t[keys ? 1 : 0];
      // dimensions of the two vectors
      const int d0 = (INTERLEAVED || !turned) ? 2 * W * v : W * v;
      const long long col = (long long)head * a.dh + d0;
      const T* src = static_cast<const T*>(y.x) + beta * y.bs_x + t * y.ld_x + col;
      x.out = static_cast<T*>(y.y) + beta * y.bs_y + t * y.ld_y + col;
      x.angle = turned ? tt * pairs + (W == 1 ? v : 2 * v) : -1;
      x.p = *reinterpret_cast<const Vec<T, W>*>(src);
      x.q = *reinterpret_cast<const Vec<T, W>*>(src + ((INTERLEAVED || !turned) ? W : a.rot >> 1));
    }
    tt += step_tt;
    u += step_u;
    if (u >= nu) {
      u -= nu;
      ++tt;
    }
  };
  auto turn = [&](Unit& x) {
    if (x.out == nullptr) return;
    const bool turned = x.angle >= 0;
    if (turned) {
      float2 cs[W];
      if (W == 1) {
        cs[0] = table[x.angle];
      } else {
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const float4 two = *reinterpret_cast<const float4*>(&table[x.angle + e * (pairs / W)]);
          cs[e] = make_float2(two.x, two.y);
          cs[(e + 1) % W] = make_float2(two.z, two.w);
        }
      }
#pragma unroll
      for (int e = 0; e < W; ++e) {
        // pair e: of the two vectors, or of both as one run of interleaved pairs
        T& lo = !INTERLEAVED ? x.p.v[e] : 2 * e < W ? x.p.v[2 * e % W] : x.q.v[2 * e % W];
        T& hi = !INTERLEAVED ? x.q.v[e] : 2 * e + 1 < W ? x.p.v[(2 * e + 1) % W] : x.q.v[(2 * e + 1) % W];
        const float x0 = rot_to_float(lo), x1 = rot_to_float(hi);
        rot_from_float(x0 * cs[e].x - x1 * cs[e].y, lo);
        rot_from_float(x1 * cs[e].x + x0 * cs[e].y, hi);
      }
    }
    *reinterpret_cast<Vec<T, W>*>(x.out) = x.p;
    *reinterpret_cast<Vec<T, W>*>(x.out + ((INTERLEAVED || !turned) ? W : a.rot >> 1)) = x.q;
  };

  Unit now, next;
  load(now);

  for (int i = threadIdx.x; i < ntok * pairs; i += ROT_THREADS) {
    const int ti = i / pairs, j = i - ti * pairs;
    int beta = beta0, t = first + ti;
    if (t >= a.s) {
      beta += t / a.s;
      t %= a.s;
    }
    long long pos = a.offset + t;
    if (a.positions != nullptr) {
      const long long at = beta * a.pos_stride + t;
      pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
    }
    const double turns = (double)pos * a.turns[j];
    const double part = turns - rint(turns);
    const float turn = (float)part, rest = 6.2831853f * (float)(part - (double)turn);
    float sn, cs;
    sincospif(2.0f * turn, &sn, &cs);
    table[ti * pairs + rot_place<W>(j, pairs)] =
        make_float2(fmaf(cs, a.magnitude, -sn * rest * a.magnitude), fmaf(sn, a.sine, cs * rest * a.sine));
  }
  __syncthreads();

  while (true) {
    const bool more = tt < ntok;
    if (more) load(next);
    turn(now);
    if (!more) break;
    now = next;
  }
}

}  // namespace bpt
