// The key/value cache held in 4 bits: layout, and the kernels that store
// tokens into it and load them back.
//
// Per token, head and group of 64 dimensions, with x the 64 bf16 values:
//     min = min x,  scale = bf16((max x - min) / 15),  r = 1 / scale (fp32)
//     code = rint((x - min) r) in 0 .. 15,   value = min + scale code.
// A scale below the smallest normal number counts as 0 (every code 0); a group
// that holds an infinity or a NaN, or whose range overflows, reads back as NaN.
//
// Layout: [b][kv_heads][capacity / 64] blocks, a block being 64 tokens of one
// head: [K codes 64 x dh/2 bytes][K parameters 64 x dh/64 x 4 bytes][V codes]
// [V parameters], 9216 bytes for dh = 128. A block is what one bulk copy of the
// attention fetches and what one of its warps works on. A row of codes is dh/8
// words of 32 bits; word u holds dimensions 8u .. 8u + 7, dimension 8u + i in
// bits 4i .. 4i + 3, and its place in the row is chosen so that the attention's
// shared-memory reads are wide and free of bank conflicts (kv4_k_place,
// kv4_v_place). K words are rotated left by 3 bits: a nibble then lands in bits
// 3 .. 6 of a 16-bit half, where it completes a bf16 of value 16 + code.
// Parameters are two bf16: scale in the lower half of 32 bits, min in the upper.
#pragma once

#include "ptx.cuh"

namespace bpt {

constexpr int KV4_BLOCK = 64;  // tokens of a block
constexpr int KV4_GROUP = 64;  // dimensions that share a scale and a minimum

template <int DH>
struct Kv4 {
  static constexpr int GROUPS = DH / KV4_GROUP;
  static constexpr int ROW = DH / 2;         // bytes of a row of codes
  static constexpr int PROW = GROUPS * 4;    // bytes of a row of parameters
  static constexpr int K_PARAMS = KV4_BLOCK * ROW;
  static constexpr int V_CODES = K_PARAMS + KV4_BLOCK * PROW;
  static constexpr int V_PARAMS = V_CODES + KV4_BLOCK * ROW;
  static constexpr int BYTES = 2 * V_CODES;
};

// Place in its row of K's word u: the four lanes that share a row in the
// attention's matrix instructions take one contiguous quarter of it each.
template <int DH>
__host__ __device__ constexpr int kv4_k_place(int u) {
  return (u & 3) * (DH / 32) + (u >> 2);
}

// Place in row r of V's word u: a lane takes the words of its 8 dimensions of
// every group next to each other, and the halves of the row are swapped in two
// rows of four, so that the lanes of four rows meet no bank twice.
template <int DH>
__host__ __device__ constexpr int kv4_v_place(int u, int r) {
  return DH == 64 ? u : ((((u & 7) ^ (((r >> 1) & 1) << 2)) << 1) | (u >> 3));
}

struct Kv4Dims {
  int b, kv_heads, capacity;
  __host__ __device__ long long blocks() const { return capacity / KV4_BLOCK; }
};

// Records a length, start or count that points outside the cache, unless the
// stream's status word already holds an error.
__device__ __forceinline__ void record_range(int* status) { atomicCAS(status, (int)BPT_OK, (int)BPT_ERR_RANGE); }

// A token count read from device memory, cut to [0, most].
__device__ __forceinline__ int clamp_count(int n, int most, int* status) {
  if (n >= 0 && n <= most) return n;
  record_range(status);
  return n < 0 ? 0 : most;
}

constexpr int KV4_THREADS = 256;

struct Kv4StoreArgs {
  uint8_t* cache;
  Kv4Dims d;
  const __nv_bfloat16* x[2];      // k, v: token (beta, t) at beta * bs + t * ld, head after head
  long long bs[2], ld[2];
  int n;
  const int* start;   // [b]: place of the sequence's first new token
  const int* counts;  // [b], or null: n for every sequence
  int* status;
};

// 16 bytes of x to the word of 8 codes, with the group's parameters.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& raw, uint32_t& params) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&raw);
  // NaN-propagating extremes, over the 8 lanes that hold the group
  __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(x[0], x[1]), __hmin2_nan(x[2], x[3]));
  __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
  }
  const __nv_bfloat16 lo16 = __hmin_nan(__low2bfloat16(lo2), __high2bfloat16(lo2));
  const float lo = __bfloat162float(lo16);
  const float range = __bfloat162float(__hmax_nan(__low2bfloat16(hi2), __high2bfloat16(hi2))) - lo;
  if (!(range < __int_as_float(0x7f800000))) {  // not finite: the group reads back as NaN
    params = 0x7fc00000u;
    return 0;
  }
  const __nv_bfloat16 scale16 = __float2bfloat16_rn(__fdiv_rn(range, 15.0f));
  const float scale = __bfloat162float(scale16);
  const bool live = scale >= 1.17549435e-38f;
  const float r = live ? __fdiv_rn(1.0f, scale) : 0.0f;
  params = (live ? (uint32_t)__bfloat16_as_ushort(scale16) : 0u) | ((uint32_t)__bfloat16_as_ushort(lo16) << 16);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(x[i]);
    // adding 1.5 * 2^23 rounds the exact product to a whole number, ties to
    // even, and leaves it in the low bits; at most 15 (1 + 2^-8) before that
    const float c0 = fmaf(f.x - lo, r, 12582912.0f), c1 = fmaf(f.y - lo, r, 12582912.0f);
    word |= (__float_as_uint(c0) & 15u) << (8 * i);
    word |= (__float_as_uint(c1) & 15u) << (8 * i + 4);
  }
  return word;
}

// A thread takes 8 dimensions of K and of V of one token and head: 16 bytes
// in, one word out each. Bound by HBM.
template <int DH>
__global__ void __launch_bounds__(KV4_THREADS) kv4_store_kernel(const Kv4StoreArgs a) {
  constexpr int U = DH / 8;
  using L = Kv4<DH>;
  const unsigned i = blockIdx.x * (unsigned)KV4_THREADS + threadIdx.x;
  const int u = i % U;
  const unsigned rest = i / U;
  const int t = rest / a.d.kv_heads, head = rest - (unsigned)t * a.d.kv_heads;
  for (int beta = blockIdx.y; beta < a.d.b; beta += gridDim.y) {
    const int count = a.counts == nullptr ? a.n : clamp_count(a.counts[beta], a.n, a.status);
    const long long at = (long long)a.start[beta] + t;
    bool live = t < count;
    if (live && (at < 0 || at >= a.d.capacity)) {
      record_range(a.status);
      live = false;
    }
    uint4 raw[2] = {};
    if (live) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        raw[w] = __ldcs(reinterpret_cast<const uint4*>(a.x[w] + beta * a.bs[w] + t * a.ld[w] + head * DH + u * 8));
    }
    uint32_t pk, pv;  // whole warps quantise: the extremes are shuffled between 8 lanes
    const uint32_t wk = kv4_quantise(raw[0], pk), wv = kv4_quantise(raw[1], pv);
    if (!live) continue;
    const int r = at % KV4_BLOCK;
    uint8_t* block = a.cache + (((long long)beta * a.d.kv_heads + head) * a.d.blocks() + at / KV4_BLOCK) * L::BYTES;
    *reinterpret_cast<uint32_t*>(block + r * L::ROW + kv4_k_place<DH>(u) * 4) = __funnelshift_l(wk, wk, 3);
    *reinterpret_cast<uint32_t*>(block + L::V_CODES + r * L::ROW + kv4_v_place<DH>(u, r) * 4) = wv;
    if (u % 8 == 0) {
      *reinterpret_cast<uint32_t*>(block + L::K_PARAMS + r * L::PROW + u / 8 * 4) = pk;
      *reinterpret_cast<uint32_t*>(block + L::V_PARAMS + r * L::PROW + u / 8 * 4) = pv;
    }
  }
}

struct Kv4LoadArgs {
  const uint8_t* cache;
  Kv4Dims d;
  __nv_bfloat16* x[2];  // k, v [b, n, kv_heads * dh]
  int n;
  const int* start;     // [b], or null: 0
  const int* lens;      // [b]: tokens at or past it read as zero
  int* status;
};

// min + scale c of the 8 codes of a word, as bf16.
__device__ __forceinline__ uint4 kv4_values(uint32_t word, uint32_t params) {
  const float scale = __uint_as_float(params << 16), lo = __uint_as_float(params & 0xffff0000u);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c0 = (float)((word >> (8 * i)) & 15u), c1 = (float)((word >> (8 * i + 4)) & 15u);
    out[i] = pack_bf16x2(fmaf(c0, scale, lo), fmaf(c1, scale, lo));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The store's mapping the other way round. Bound by HBM (its writes).
template <int DH>
__global__ void __launch_bounds__(KV4_THREADS) kv4_load_kernel(const Kv4LoadArgs a) {
  constexpr int U = DH / 8;
  using L = Kv4<DH>;
  const unsigned i = blockIdx.x * (unsigned)KV4_THREADS + threadIdx.x;
  const int u = i % U;
  const unsigned rest = i / U;
  const int t = rest / a.d.kv_heads, head = rest - (unsigned)t * a.d.kv_heads;
  if (t >= a.n) return;
  for (int beta = blockIdx.y; beta < a.d.b; beta += gridDim.y) {
    const int len = clamp_count(a.lens[beta], a.d.capacity, a.status);
    const long long at = (a.start == nullptr ? 0LL : (long long)a.start[beta]) + t;
    if (at < 0) record_range(a.status);
    uint4 k = {}, v = {};
    if (at >= 0 && at < len) {
      const int r = at % KV4_BLOCK;
      const uint8_t* block =
          a.cache + (((long long)beta * a.d.kv_heads + head) * a.d.blocks() + at / KV4_BLOCK) * L::BYTES;
      const uint32_t wk = *reinterpret_cast<const uint32_t*>(block + r * L::ROW + kv4_k_place<DH>(u) * 4);
      const uint32_t wv = *reinterpret_cast<const uint32_t*>(block + L::V_CODES + r * L::ROW + kv4_v_place<DH>(u, r) * 4);
      const uint32_t pk = *reinterpret_cast<const uint32_t*>(block + L::K_PARAMS + r * L::PROW + u / 8 * 4);
      const uint32_t pv = *reinterpret_cast<const uint32_t*>(block + L::V_PARAMS + r * L::PROW + u / 8 * 4);
      k = kv4_values(__funnelshift_r(wk, wk, 3), pk);
      v = kv4_values(wv, pv);
    }
    const long long to = ((beta * (long long)a.n + t) * a.d.kv_heads + head) * DH + u * 8;
    *reinterpret_cast<uint4*>(a.x[0] + to) = k;
    *reinterpret_cast<uint4*>(a.x[1] + to) = v;
  }
}

}  // namespace bpt
