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
// kv4_v_place). K words are rotated left by 3 bits: three shifts (0, 5 and 12 bits
// to the right) then take the four nibbles of every 16-bit half to bits 3 .. 6,
// 2 .. 5, 6 .. 9 and 3 .. 6, within its 10 lowest bits, where one mask more leaves
// a subnormal fp16 number (kv4_attention.cuh). Parameters are two bf16: scale in
// the lower half of 32 bits, min in the upper.
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

// rint((x - lo) r) of the exact difference, where that has more bits than fp32.
__device__ __forceinline__ uint32_t kv4_code_wide(float x, float lo, float r) {
  // the difference as a sum of two (Knuth's two-sum), each times r exact in fp64
  const float d = __fsub_rn(x, lo), b = __fsub_rn(d, x);
  const float rest = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(lo, b));
  const double p = (double)d * (double)r, more = (double)rest * (double)r;
  double c = rint(p);
  const double f = p - c;  // exact; within half of c, and `more` may lead out of that
  const bool odd = (int)c & 1;
  if (more > 0.5 - f || (odd && more == 0.5 - f && more != 0.0)) c += 1.0;
  else if (more < -0.5 - f || (odd && more == -0.5 - f && more != 0.0)) c -= 1.0;
  return (uint32_t)c;
}

// Whether a code of 16 values may depend on what their fp32 difference from lo
// leaves out: that is not zero, and the product without it next to a tie. (Calls,
// not inline: 16 values' codes in fp64 take the store from 40 registers to 69 and
// the example below from 64 to 84 us, were they in its line.)
__device__ __noinline__ bool kv4_near_tie(uint4 xs, uint4 ys, float lo, float r) {
  const uint32_t raw[8] = {xs.x, xs.y, xs.z, xs.w, ys.x, ys.y, ys.z, ys.w};
  const uint64_t minus = f2_pack(-lo, -lo), times = f2_pack(r, r), neg = f2_pack(-1.0f, -1.0f);
  const uint64_t magic = f2_pack(12582912.0f, 12582912.0f);
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t x = f2_pack(__uint_as_float(raw[i] << 16), __uint_as_float(raw[i] & 0xffff0000u));
    const uint64_t d = f2_add(x, minus), b = f2_fma(x, neg, d);
    const uint64_t rest = f2_add(f2_fma(f2_fma(b, neg, d), neg, x), f2_fma(b, neg, minus));
    const uint64_t away = f2_fma(d, times, f2_fma(f2_fma(d, times, magic), neg, magic));  // from the code
    float r0, r1, a0, a1;
    f2_unpack(rest, r0, r1);
    f2_unpack(away, a0, a1);
    // what is left out moves the product by 16 times 2^-24 at most
    near |= (r0 != 0.f && fabsf(a0) > 0.49999f) || (r1 != 0.f && fabsf(a1) > 0.49999f);
  }
  return near;
}

// The codes of 16 values, as two words, where kv4_near_tie.
__device__ __noinline__ uint2 kv4_words_wide(uint4 x, uint4 y, float lo, float r) {
  uint32_t word[2] = {};
  const uint32_t raw[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    word[i / 4] = word[i / 4] * 16u + kv4_code_wide(__uint_as_float(raw[i] & 0xffff0000u), lo, r);
    word[i / 4] = word[i / 4] * 16u + kv4_code_wide(__uint_as_float(raw[i] << 16), lo, r);
  }
  return make_uint2(word[0], word[1]);
}

// 16 values of x (bf16, packed) to two words of codes, with the group's
// parameters; 4 neighbouring lanes hold the 64 values of a group.
__device__ __forceinline__ void kv4_quantise(const uint32_t (&raw)[8], uint32_t (&word)[2], uint32_t& params) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(raw);
  // NaN-propagating extremes, both as minimums: (min x, min -x)
  __nv_bfloat162 lo2 = x[0], hi2 = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = __hmin2_nan(lo2, x[i]);
    hi2 = __hmax2_nan(hi2, x[i]);
  }
  __nv_bfloat162 ends = __halves2bfloat162(__hmin_nan(__low2bfloat16(lo2), __high2bfloat16(lo2)),
                                           __hneg(__hmax_nan(__low2bfloat16(hi2), __high2bfloat16(hi2))));
  ends = __hmin2_nan(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
  ends = __hmin2_nan(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
  const __nv_bfloat16 lo16 = __low2bfloat16(ends);
  const float lo = __bfloat162float(lo16);
  const float range = -__high2float(ends) - lo;
  const bool finite = range < __int_as_float(0x7f800000);  // else the group reads back as NaN
  // range / 15: a product with the rounded reciprocal, corrected by its exact
  // residual (Markstein 1990), which leaves the correctly rounded quotient
  constexpr float fifteenth = 1.0f / 15.0f;
  const float q = range * fifteenth;
  const __nv_bfloat16 scale16 = __float2bfloat16_rn(fmaf(fmaf(-15.0f, q, range), fifteenth, q));
  const float scale = __bfloat162float(scale16);
  const bool live = finite && scale >= 1.17549435e-38f;
  const float r = live ? __frcp_rn(scale) : 0.0f;
  params = !finite ? 0x7fc00000u
                   : (live ? (uint32_t)__bfloat16_as_ushort(scale16) : 0u) | ((uint32_t)__bfloat16_as_ushort(lo16) << 16);
  const uint64_t minus = f2_pack(-lo, -lo), times = f2_pack(r, r), magic = f2_pack(12582912.0f, 12582912.0f);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    // Adding 1.5 * 2^23 rounds the exact product of the difference to a whole
    // number, ties to even, and leaves it (at most 15 (1 + 2^-8) before that) in
    // the low bits of 0x4b400000; those constants add up to 0x4b400000 (16^8 - 1)
    // / 15.
    uint32_t sum = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint32_t two = raw[4 * w + i];
      float lo_code, hi_code;
      f2_unpack(f2_fma(f2_add(f2_pack(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u)), minus), times, magic),
                lo_code, hi_code);
      sum = sum * 16u + __float_as_uint(hi_code);
      sum = sum * 16u + __float_as_uint(lo_code);
    }
    word[w] = live ? sum - 0x4b400000u * 0x11111111u : 0u;
  }
  // The difference of two bf16 is exact in fp32 unless one is below 2^-14 of the
  // other. Where that is the minimum, or where so small an x could lie next to a tie
  // (it is within 2^-10 steps of 0), the codes are looked at again.
  const float zero = -lo * r;  // 0's code before it is rounded
  const bool small = lo != 0.f && fabsf(lo) < 0x1p-14f * range;
  if (live && (small || fabsf(zero - rintf(zero)) > 0.5f - 0x1p-10f)) {
    const uint4 x = make_uint4(raw[0], raw[1], raw[2], raw[3]), y = make_uint4(raw[4], raw[5], raw[6], raw[7]);
    if (kv4_near_tie(x, y, lo, r)) {
      const uint2 exact = kv4_words_wide(x, y, lo, r);
      word[0] = exact.x;
      word[1] = exact.y;
    }
  }
}

// 32 bytes that are read once.
__device__ __forceinline__ void load_stream32(const void* p, uint32_t (&x)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
               : "l"(p));
}

// A thread takes 16 dimensions of K and of V of one token and head: 32 bytes
// in, two words out of each. 4 x 8192 tokens of 16 heads of 128 (343 MB in and
// out, 52 us at the copy's rate): 63 us, 5.4 TB/s. Bound by the issue of its
// instructions (80% of the slots) close behind the memory: the look at what fp32 differences leave
// out costs 4 us of it; 8 dimensions a thread took 105 us, unpacked arithmetic and
// two divisions a group 69.
template <int DH, bool WIDE>
__global__ void __launch_bounds__(KV4_THREADS, 6) kv4_store_kernel(const __grid_constant__ Kv4StoreArgs a) {
  constexpr int U = DH / 16;
  using L = Kv4<DH>;
  grid_dependency_wait();
  grid_dependents_start();
  const unsigned i = blockIdx.x * (unsigned)KV4_THREADS + threadIdx.x;
  const int u = i % U;
  const unsigned rest = i / U;
  const int t = rest / (unsigned)a.d.kv_heads, head = rest - (unsigned)t * a.d.kv_heads;
  for (int beta = blockIdx.y; beta < a.d.b; beta += gridDim.y) {
    const int count = a.counts == nullptr ? a.n : clamp_count(a.counts[beta], a.n, a.status);
    const long long at = (long long)a.start[beta] + t;
    bool live = t < count;
    if (live && (at < 0 || at >= a.d.capacity)) {
      record_range(a.status);
      live = false;
    }
    uint32_t raw[2][8] = {};
    if (live) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const __nv_bfloat16* src = a.x[w] + beta * a.bs[w] + t * a.ld[w] + (head * DH + u * 16);
        if (WIDE) {
          load_stream32(src, raw[w]);
        } else {
          const uint4 x = reinterpret_cast<const uint4*>(src)[0], y = reinterpret_cast<const uint4*>(src)[1];
          raw[w][0] = x.x, raw[w][1] = x.y, raw[w][2] = x.z, raw[w][3] = x.w;
          raw[w][4] = y.x, raw[w][5] = y.y, raw[w][6] = y.z, raw[w][7] = y.w;
        }
      }
    }
    uint32_t pk, pv, wk[2], wv[2];  // whole warps quantise: the extremes are shuffled between 4 lanes
    kv4_quantise(raw[0], wk, pk);
    kv4_quantise(raw[1], wv, pv);
    if (!live) continue;
    const int r = at % KV4_BLOCK;
    uint8_t* block = a.cache + (((long long)beta * a.d.kv_heads + head) * a.d.blocks() + at / KV4_BLOCK) * L::BYTES;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      *reinterpret_cast<uint32_t*>(block + r * L::ROW + kv4_k_place<DH>(2 * u + w) * 4) = __funnelshift_l(wk[w], wk[w], 3);
      *reinterpret_cast<uint32_t*>(block + L::V_CODES + r * L::ROW + kv4_v_place<DH>(2 * u + w, r) * 4) = wv[w];
    }
    if (u % 4 == 0) {
      *reinterpret_cast<uint32_t*>(block + L::K_PARAMS + r * L::PROW + u / 4 * 4) = pk;
      *reinterpret_cast<uint32_t*>(block + L::V_PARAMS + r * L::PROW + u / 4 * 4) = pv;
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
  uint32_t zero;        // 0
};

// (x & mask) | MAGIC in one operation. The mask comes in a register that the
// compiler does not know (a kernel argument is part of it): with two constants
// it makes two operations.
template <uint32_t MAGIC>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "n"(MAGIC));
  return y;
}

// min + scale c of the 8 codes of a word, as bf16. mask: 15.
__device__ __forceinline__ void kv4_values(uint32_t word, uint32_t params, uint32_t mask, uint32_t* out) {
  const float scale = __uint_as_float(params << 16), lo = __uint_as_float(params & 0xffff0000u);
  const uint64_t minus = f2_pack(-8388608.0f, -8388608.0f), times = f2_pack(scale, scale), plus = f2_pack(lo, lo);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 2^23 + c is exact in fp32, and so is c again
    const uint64_t c = f2_add(f2_pack(__uint_as_float(and_or<0x4b000000u>(word >> (8 * i), mask)),
                                      __uint_as_float(and_or<0x4b000000u>(word >> (8 * i + 4), mask))), minus);
    float x0, x1;
    f2_unpack(f2_fma(c, times, plus), x0, x1);
    out[i] = pack_bf16x2(x0, x1);
  }
}

// 32 bytes that this kernel does not read again.
__device__ __forceinline__ void store_stream32(void* p, const uint32_t (&x)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// The store's mapping the other way round: 16 dimensions of K and V a thread.
// Bound by HBM (its writes): 60 us, 5.7 TB/s, at the store's example. The outputs'
// rows are 128 bytes or more, so every 32 bytes are aligned where their start is
// (WIDE).
template <int DH, bool WIDE>
__global__ void __launch_bounds__(KV4_THREADS) kv4_load_kernel(const __grid_constant__ Kv4LoadArgs a) {
  constexpr int U = DH / 16;
  using L = Kv4<DH>;
  grid_dependency_wait();
  grid_dependents_start();
  const unsigned i = blockIdx.x * (unsigned)KV4_THREADS + threadIdx.x;
  const int u = i % U;
  const unsigned rest = i / U;
  const int t = rest / (unsigned)a.d.kv_heads, head = rest - (unsigned)t * a.d.kv_heads;
  if (t >= a.n) return;
  for (int beta = blockIdx.y; beta < a.d.b; beta += gridDim.y) {
    const int len = clamp_count(a.lens[beta], a.d.capacity, a.status);
    const int first = a.start == nullptr ? 0 : a.start[beta];
    if (first < 0 || first > a.d.capacity) record_range(a.status);
    const long long at = (long long)first + t;
    uint32_t x[2][8] = {};
    if (at >= 0 && at < len) {
      const int r = at % KV4_BLOCK;
      const uint8_t* block =
          a.cache + (((long long)beta * a.d.kv_heads + head) * a.d.blocks() + at / KV4_BLOCK) * L::BYTES;
      uint32_t word[2][2], params[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        word[0][w] = reinterpret_cast<const uint32_t*>(block + r * L::ROW)[kv4_k_place<DH>(2 * u + w)];
        word[1][w] = reinterpret_cast<const uint32_t*>(block + L::V_CODES + r * L::ROW)[kv4_v_place<DH>(2 * u + w, r)];
        params[w] = reinterpret_cast<const uint32_t*>(block + (w ? L::V_PARAMS : L::K_PARAMS) + r * L::PROW)[u / 4];
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        kv4_values(__funnelshift_r(word[0][w], word[0][w], 3), params[0], 15u + a.zero, x[0] + 4 * w);
        kv4_values(word[1][w], params[1], 15u + a.zero, x[1] + 4 * w);
      }
    }
    const long long to = ((beta * (long long)a.n + t) * a.d.kv_heads + head) * DH + u * 16;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (WIDE) {
        store_stream32(a.x[w] + to, x[w]);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(a.x[w] + to);
        dst[0] = make_uint4(x[w][0], x[w][1], x[w][2], x[w][3]);
        dst[1] = make_uint4(x[w][4], x[w][5], x[w][6], x[w][7]);
      }
    }
  }
}

}  // namespace bpt
