// Eviction from the 4-bit cache by accumulated attention weight: of a
// sequence's len tokens, each key/value head keeps the `recent` newest and the
// heaviest of the others, `keep` in all (ties: the lowest place), in their
// order, and their rows move to another cache.
//
// Selection is a radix select of the need-th largest weight: its bits, made
// monotone as a whole number, are fixed 11, 11 and 10 at a time from histograms
// of the candidates that agree so far. Which tied tokens stay then follows from
// their order alone, so the result does not depend on any order of the atomics.
#pragma once

#include "kv4_cache.cuh"

namespace bpt {

constexpr int EVICT_THREADS = 1024;
constexpr int EVICT_BINS = 2048;

struct Kv4SelectArgs {
  const float* weights;  // [b, kv_heads, capacity]
  Kv4Dims d;
  const int* lens;
  int keep, recent;
  int* kept;             // [b, kv_heads, keep], -1 past the kept ones
  int* lens_out;         // [b]
  int* status;
};

// A weight as a whole number of the same order; both zeros are equal, and NaN
// is the heaviest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t x = __float_as_uint(w + 0.0f);
  return x ^ ((x >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(EVICT_THREADS) kv4_select_kernel(const Kv4SelectArgs a) {
  __shared__ int hist[EVICT_BINS];
  __shared__ int warp_sum[32], warp_tie[32];
  __shared__ int s_bin, s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = a.d.b * a.d.kv_heads;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const int beta = row / a.d.kv_heads;
    const int len = clamp_count(a.lens[beta], a.d.capacity, a.status);
    const int left = min(len, a.keep), recent = min(a.recent, left);
    const int old = len - recent, need = left - recent;  // choose `need` of the `old` first tokens
    const float* w = a.weights + (long long)row * a.d.capacity;
    int* kept = a.kept + (long long)row * a.keep;
    if (tid == 0 && row == beta * a.d.kv_heads) a.lens_out[beta] = left;
    for (int i = tid; i < a.keep; i += EVICT_THREADS)
      if (i >= need) kept[i] = i < left ? old + i - need : -1;
    if (need == old) {
      for (int i = tid; i < need; i += EVICT_THREADS) kept[i] = i;
      continue;
    }
    if (need == 0) continue;
    // the need-th largest key, digit by digit
    uint32_t prefix = 0, mask = 0;
    int want = need;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      __syncthreads();
      for (int i = tid; i < EVICT_BINS; i += EVICT_THREADS) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < old; i += EVICT_THREADS) {
        const uint32_t key = weight_key(w[i]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // from the top: thread i holds bins BINS - 1 - 2i and BINS - 2 - 2i
      const int hi = hist[EVICT_BINS - 1 - 2 * tid], lo = hist[EVICT_BINS - 2 - 2 * tid];
      int sum = hi + lo;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      int before = sum - hi - lo;
      for (int i = 0; i < warp; ++i) before += warp_sum[i];
      if (before < want && want <= before + hi + lo) {  // exactly one thread
        const bool in_hi = want <= before + hi;
        s_bin = EVICT_BINS - (in_hi ? 1 : 2) - 2 * tid;
        s_need = want - before - (in_hi ? 0 : hi);
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << shift;
      mask |= (uint32_t)((1 << bits) - 1) << shift;
      want = s_need;
    }
    // keys above `prefix` stay, and the first `want` of those equal to it;
    // each warp takes a run of whole 32s and first counts what stays before it
    const int run = ((old + 1023) / 1024) * 32;
    const int lo = min(warp * run, old), hi = min(lo + run, old);
    int more = 0, tie = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      const uint32_t key = weight_key(w[i]);
      more += key > prefix;
      tie += key == prefix;
    }
    more = __reduce_add_sync(0xffffffffu, more);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
      warp_sum[warp] = more;
      warp_tie[warp] = tie;
    }
    __syncthreads();
    int above = 0, ties = 0;
    for (int i = 0; i < warp; ++i) {
      above += warp_sum[i];
      ties += warp_tie[i];
    }
    const uint32_t below = (1u << lane) - 1;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < hi ? weight_key(w[i]) : 0u;
      const uint32_t m_above = __ballot_sync(0xffffffffu, i < hi && key > prefix);
      const uint32_t m_tie = __ballot_sync(0xffffffffu, i < hi && key == prefix);
      const int tie_at = ties + __popc(m_tie & below);
      const bool stays = (m_above >> lane & 1) || ((m_tie >> lane & 1) && tie_at < want);
      if (stays) kept[above + __popc(m_above & below) + min(tie_at, want)] = i;
      above += __popc(m_above);
      ties += __popc(m_tie);
    }
    __syncthreads();
  }
}

struct Kv4MoveArgs {
  const uint8_t* src;
  uint8_t* dst;
  Kv4Dims d, d_out;
  const float* weights;
  float* weights_out;  // [b, kv_heads, capacity_out], zero past the kept tokens
  const int* kept;
  const int* lens_out;
  int keep;
};

// A team of lanes moves one row, 16 bytes of codes a lane, then its parameters
// and weight. The halves of V's row change places where the two rows' places
// differ in that bit (kv4_v_place). Bound by HBM.
template <int DH>
__global__ void __launch_bounds__(KV4_THREADS) kv4_move_kernel(const Kv4MoveArgs a) {
  using L = Kv4<DH>;
  constexpr int C = L::ROW / 16, TEAM = 2 * C;  // 16-byte pieces of a row of codes; lanes: K's, then V's
  const int piece = threadIdx.x % TEAM;
  const int j = blockIdx.x * (KV4_THREADS / TEAM) + threadIdx.x / TEAM;
  const int rows = a.d.b * a.d.kv_heads;
  if (j >= a.d_out.capacity) return;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int left = a.lens_out[row / a.d.kv_heads];
    if (j >= left) {
      if (piece == 0) a.weights_out[(long long)row * a.d_out.capacity + j] = 0.f;
      continue;
    }
    const int i = a.kept[(long long)row * a.keep + j];
    const int ri = i % KV4_BLOCK, rj = j % KV4_BLOCK;
    const uint8_t* from = a.src + ((long long)row * a.d.blocks() + i / KV4_BLOCK) * L::BYTES;
    uint8_t* to = a.dst + ((long long)row * a.d_out.blocks() + j / KV4_BLOCK) * L::BYTES;
    if (piece < C) {
      *reinterpret_cast<uint4*>(to + rj * L::ROW + piece * 16) =
          *reinterpret_cast<const uint4*>(from + ri * L::ROW + piece * 16);
    } else {
      const int c = piece - C;
      const int swap = DH == 64 ? 0 : ((ri ^ rj) & 2);  // places differ by 4 pairs of words = 2 pieces
      *reinterpret_cast<uint4*>(to + L::V_CODES + rj * L::ROW + (c ^ swap) * 16) =
          *reinterpret_cast<const uint4*>(from + L::V_CODES + ri * L::ROW + c * 16);
    }
    if (piece < 2) {
      const int at = piece == 0 ? L::K_PARAMS : L::V_PARAMS;
#pragma unroll
      for (int g = 0; g < L::GROUPS; ++g)
        *reinterpret_cast<uint32_t*>(to + at + rj * L::PROW + g * 4) =
            *reinterpret_cast<const uint32_t*>(from + at + ri * L::PROW + g * 4);
      if (piece == 0)
        a.weights_out[(long long)row * a.d_out.capacity + j] = a.weights[(long long)row * a.d.capacity + i];
    }
  }
}

}  // namespace bpt
