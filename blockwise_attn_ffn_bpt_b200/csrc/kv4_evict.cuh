// Eviction from the 4-bit cache by accumulated attention weight: of a
// sequence's len tokens, each key/value head keeps the `recent` newest and the
// heaviest of the others, `keep` in all (ties: the lowest place), in their
// order, and their rows move to another cache.
//
// Selection is a radix select of the need-th largest weight: its bits, made
// monotone as a whole number, are fixed 11, 11 and 10 at a time from histograms
// of the candidates that agree so far; it ends early where all that agree stay.
// Which tied tokens stay then follows from their order alone, so the result does
// not depend on any order of the atomics. Bound by latencies: 7 us for a few
// hundred tokens (two or three passes of five barriers each), 17 us for 64 rows
// of 32768.
#pragma once

#include "gemm_pair.cuh"  // cluster rank, barrier and addresses
#include "kv4_cache.cuh"

namespace bpt {

constexpr int EVICT_THREADS = 1024;
constexpr int EVICT_SHORT = 256;  // threads for many short rows (evict_threads)
constexpr int EVICT_BINS = 2048;
// Copies of the histogram, one to every second or fourth lane: weights of a few
// octaves share few bins of the first digit, and lanes that add to one bin take
// turns. (48 KB of it and of the cluster's totals are there without asking.)
constexpr int evict_copies(int cl, int threads) { return cl > 1 || threads == EVICT_SHORT ? 2 : 4; }
constexpr int EVICT_CACHED = 40960;  // tokens of a block whose keys stay in shared memory (160 KB)

struct Kv4SelectArgs {
  const float* weights;  // [b, kv_heads, capacity]
  Kv4Dims d;
  const int* lens;
  int keep, recent;
  int* kept;             // [b, kv_heads, keep], -1 past the kept ones
  int* lens_out;         // [b]
  int* status;
};

// Shared memory of the cluster's block r.
__device__ __forceinline__ int cluster_load(uint32_t addr, int r) {
  int x;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(addr, (uint32_t)r)) : "memory");
  return x;
}
__device__ __forceinline__ int2 cluster_load2(uint32_t addr, int r) {
  int2 x;
  asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(mapa_shared(addr, (uint32_t)r)) : "memory");
  return x;
}

// A weight as a whole number of the same order; both zeros are equal, and NaN
// is the heaviest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t x = __float_as_uint(w + 0.0f);
  return x ^ ((x >> 31) ? 0xffffffffu : 0x80000000u);
}

// The keys of 4 weights. Past `old` they are 0, below every weight's.
__device__ __forceinline__ uint4 weight_keys(const float4& w, int i, int old) {
  return make_uint4(i < old ? weight_key(w.x) : 0u, i + 1 < old ? weight_key(w.y) : 0u,
                    i + 2 < old ? weight_key(w.z) : 0u, i + 3 < old ? weight_key(w.w) : 0u);
}

// A cluster of CL blocks a (sequence, head), each with an equal part of its
// tokens. The keys of up to EVICT_CACHED tokens a block stay in shared memory
// after the first pass; longer rows are read again, from L2.
template <int CL, bool CACHED, int THREADS>
__global__ void __launch_bounds__(THREADS) kv4_select_kernel(const __grid_constant__ Kv4SelectArgs a) {
  extern __shared__ uint4 cached[];
  constexpr int COPIES = evict_copies(CL, THREADS), PER = EVICT_BINS / THREADS;  // bins of a thread
  static_assert(CL == 1 || PER == 2, "clusters read two bins a thread");
  __shared__ int hist[COPIES][EVICT_BINS];
  __shared__ int warp_sum[32], warp_tie[32];
  __shared__ int s_bin, s_need, s_count;
  // what the other blocks of the cluster read: the histogram (by turns, so that
  // one barrier a pass will do) and the block's counts of the last step
  __shared__ alignas(8) int s_total[CL > 1 ? 2 : 1][CL > 1 ? EVICT_BINS : 1];
  __shared__ int s_above, s_ties;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL > 1 ? (int)cluster_ctarank() : 0;
  const int rows = a.d.b * a.d.kv_heads;
  grid_dependency_wait();
  grid_dependents_start();
  for (int row = blockIdx.x / CL; row < rows; row += gridDim.x / CL) {
    const int beta = row / a.d.kv_heads;
    const int len = clamp_count(a.lens[beta], a.d.capacity, a.status);
    const int left = min(len, a.keep), recent = min(a.recent, left);
    const int old = len - recent, need = left - recent;  // choose `need` of the `old` first tokens
    const float* w = a.weights + (long long)row * a.d.capacity;
    int* kept = a.kept + (long long)row * a.keep;
    if (rank == 0 && tid == 0 && row == beta * a.d.kv_heads) a.lens_out[beta] = left;
    const int first = rank * THREADS + tid;
    for (int i = need + first; i < a.keep; i += CL * THREADS) kept[i] = i < left ? old + i - need : -1;
    if (need == old) {
      for (int i = first; i < need; i += CL * THREADS) kept[i] = i;
      continue;
    }
    if (need == 0) continue;
    // this block's part, in groups of 4 tokens
    const int every = (old + 3) / 4, share = (every + CL - 1) / CL, quad0 = min(rank * share, every);
    const int quads = min(share, every - quad0);
    auto keys_of = [&](int i, bool read) -> uint4 {
      if (CACHED && !read) return cached[i];
      const uint4 k = weight_keys(reinterpret_cast<const float4*>(w)[quad0 + i], 4 * (quad0 + i), old);
      if (CACHED) cached[i] = k;
      return k;
    };
    // the need-th largest key, digit by digit
    uint32_t prefix = 0, mask = 0;
    int want = need;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t digit = (1u << bits) - 1;
      __syncthreads();
      for (int i = tid; i < COPIES * EVICT_BINS; i += THREADS) (&hist[0][0])[i] = 0;
      __syncthreads();
      auto count = [&](uint32_t key) {
        if ((key & mask) == prefix) atomicAdd(&hist[lane % COPIES][(key >> shift) & digit], 1);
      };
#pragma unroll 4
      for (int i = tid; i < quads; i += THREADS) {
        const uint4 k = keys_of(i, pass == 0);
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      }
      __syncthreads();
      // from the top: thread i holds the PER bins from BINS - 1 - PER i down
      const int top = EVICT_BINS - 1 - PER * tid;
      int bin[PER] = {};
#pragma unroll
      for (int p = 0; p < PER; ++p)
#pragma unroll
        for (int x = 0; x < COPIES; ++x) bin[p] += hist[x][top - p];
      if constexpr (CL > 1) {
        int* mine = s_total[pass & 1];
        mine[top] = bin[0];
        mine[top - 1] = bin[1];
        cluster_sync_all();
        bin[0] = bin[1] = 0;
#pragma unroll
        for (int r = 0; r < CL; ++r) {
          const int2 x = cluster_load2(smem_addr(mine + top - 1), r);
          bin[1] += x.x;
          bin[0] += x.y;
        }
      }
      int all = 0;
#pragma unroll
      for (int p = 0; p < PER; ++p) all += bin[p];
      int sum = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      int before = sum - all + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
      if (before < want && want <= before + all) {  // exactly one thread
#pragma unroll
        for (int p = 0; p < PER; ++p) {
          if (before < want && want <= before + bin[p]) {
            s_bin = top - p;
            s_need = want - before;
            s_count = bin[p];
          }
          before += bin[p];
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << shift;
      mask |= digit << shift;
      want = s_need;
      if (want == s_count && prefix != 0) {  // all that agree so far stay: they count as above
        --prefix;
        want = 0;
        break;
      }
    }
    // keys above `prefix` stay, and the first `want` of those equal to it;
    // each warp takes a run of whole 128s and first counts what stays before it
    const int run = (quads + THREADS - 1) / THREADS * 32;
    const int lo = min(warp * run, quads), hi = min(lo + run, quads);
    int more = 0, tie = 0;
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) {
      const uint4 k = keys_of(i, false);
      more += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
      tie += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    more = __reduce_add_sync(0xffffffffu, more);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
      warp_sum[warp] = more;
      warp_tie[warp] = tie;
    }
    __syncthreads();
    int above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
    int ties = __reduce_add_sync(0xffffffffu, lane < warp ? warp_tie[lane] : 0);
    if constexpr (CL > 1) {
      if (tid == THREADS - 1) {
        s_above = above + more;
        s_ties = ties + tie;
      }
      cluster_sync_all();
      for (int r = 0; r < rank; ++r) {
        above += cluster_load(smem_addr(&s_above), r);
        ties += cluster_load(smem_addr(&s_ties), r);
      }
    }
    const uint32_t below = (1u << lane) - 1;
    if (want == 0) {  // no ties to choose from
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const uint4 k = i < hi ? keys_of(i, false) : make_uint4(0, 0, 0, 0);
        const bool s0 = k.x > prefix, s1 = k.y > prefix, s2 = k.z > prefix, s3 = k.w > prefix;
        const uint32_t b0 = __ballot_sync(0xffffffffu, s0), b1 = __ballot_sync(0xffffffffu, s1);
        const uint32_t b2 = __ballot_sync(0xffffffffu, s2), b3 = __ballot_sync(0xffffffffu, s3);
        int at = above + __popc(b0 & below) + __popc(b1 & below) + __popc(b2 & below) + __popc(b3 & below);
        if (s0) kept[at++] = 4 * (quad0 + i);
        if (s1) kept[at++] = 4 * (quad0 + i) + 1;
        if (s2) kept[at++] = 4 * (quad0 + i) + 2;
        if (s3) kept[at] = 4 * (quad0 + i) + 3;
        above += __popc(b0) + __popc(b1) + __popc(b2) + __popc(b3);
      }
    } else {
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const uint4 k4 = i < hi ? keys_of(i, false) : make_uint4(0, 0, 0, 0);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        int at = above, tied = ties;
        bool is_above[4], is_tie[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          is_above[e] = k[e] > prefix;
          is_tie[e] = i < hi && k[e] == prefix;
          const uint32_t b_above = __ballot_sync(0xffffffffu, is_above[e]), b_tie = __ballot_sync(0xffffffffu, is_tie[e]);
          at += __popc(b_above & below);
          tied += __popc(b_tie & below);
          above += __popc(b_above);
          ties += __popc(b_tie);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (is_above[e] || (is_tie[e] && tied < want)) kept[at + min(tied, want)] = 4 * (quad0 + i) + e;
          at += is_above[e];
          tied += is_tie[e];
        }
      }
    }
    if constexpr (CL > 1)
      cluster_sync_all();  // no block ends, or starts on its next row, before the others have read its counts
    else
      __syncthreads();
  }
}

// Blocks of a cluster: more where a row is long and the rows alone leave SMs
// idle (two blocks on an SM gain nothing). Device time, 1 against 2 and 4 blocks:
// 4 rows of 8192 tokens 11.3, 12.4, 12.3 us, of 32768 tokens 18.8, 15.8, 14.8, 2
// rows of 131072 tokens 69, 42, 22; 64 rows of 32768 tokens 23.9, 20.0, 30.7. That
// is with full rows; the host knows the capacity alone, and the rows may be short:
// an eviction from 64 rows of 4096 tokens takes 9.0 us with that capacity (one
// block), 12.4 with 32768 (two).
inline int evict_cluster(long long rows, int capacity) {
  if (capacity < 16384) return 1;
  return rows * 4 <= KVA_MAX_SMS ? 4 : rows * 2 <= KVA_MAX_SMS ? 2 : 1;
}

// Threads of a block: few where the rows, two blocks of 1024 an SM, would take a
// second round, and are short. Device time of the selection, 1024 against 256: 1440
// rows of 512 tokens 42.6, 20.4 us; 1024 of 2048 34.4, 22.2, of 4096 38.6, 28.8; 296
// of 4096 12.3, 13.2; 64 of 2048 5.3, 6.7. As above with full rows: an eviction
// from 1440 rows of 512 takes 29 us with a capacity of 512 or 4096 (256 threads),
// 50 with 32768 (1024).
inline int evict_threads(int cl, long long rows, int capacity) {
  return cl == 1 && rows > KVA_MAX_SMS * 2 && capacity <= 4096 ? EVICT_SHORT : EVICT_THREADS;
}

typedef void (*EvictKernel)(const Kv4SelectArgs);
inline EvictKernel evict_kernel(int cl, bool cached, int threads) {
  if (threads == EVICT_SHORT) return kv4_select_kernel<1, true, EVICT_SHORT>;  // such rows are always cached
  if (cl == 4) return cached ? kv4_select_kernel<4, true, EVICT_THREADS> : kv4_select_kernel<4, false, EVICT_THREADS>;
  if (cl == 2) return cached ? kv4_select_kernel<2, true, EVICT_THREADS> : kv4_select_kernel<2, false, EVICT_THREADS>;
  return cached ? kv4_select_kernel<1, true, EVICT_THREADS> : kv4_select_kernel<1, false, EVICT_THREADS>;
}

inline bool evict_set_attributes() {
  bool ok = true;
  for (int cl : {1, 2, 4})
    ok = ok && cudaFuncSetAttribute(evict_kernel(cl, true, EVICT_THREADS), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    EVICT_CACHED * 4) == cudaSuccess;
  return ok;
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

constexpr int MOVE_ROWS = 4;

// A team of lanes moves MOVE_ROWS rows at a time, 16 bytes of codes of each a
// lane, then their parameters and weights. The halves of V's row change places
// where the two rows' places differ in that bit (kv4_v_place). Bound by HBM: 64
// rows of 32768 tokens, 4096 kept, 24 us, where the kept rows (every eighth) cost
// the 64-byte sectors around their parameters too, 122 MB in all; and by the
// latency of two reads in a row (a place, then its row), hence several rows at
// once (one at a time: 39 us).
template <int DH>
__global__ void __launch_bounds__(KV4_THREADS) kv4_move_kernel(const __grid_constant__ Kv4MoveArgs a) {
  using L = Kv4<DH>;
  constexpr int C = L::ROW / 16, TEAM = 2 * C, TEAMS = KV4_THREADS / TEAM;  // lanes: K's 16-byte pieces, then V's
  const int piece = threadIdx.x % TEAM;
  const int j0 = blockIdx.x * (TEAMS * MOVE_ROWS) + threadIdx.x / TEAM;
  const int rows = a.d.b * a.d.kv_heads;
  grid_dependency_wait();
  grid_dependents_start();
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int left = a.lens_out[row / a.d.kv_heads];
    const uint8_t* src = a.src + (long long)row * a.d.blocks() * L::BYTES;
    uint8_t* dst = a.dst + (long long)row * a.d_out.blocks() * L::BYTES;
    int from[MOVE_ROWS];
#pragma unroll
    for (int k = 0; k < MOVE_ROWS; ++k) {
      const int j = j0 + k * TEAMS;
      from[k] = j < left ? a.kept[(long long)row * a.keep + j] : -1;
    }
    uint4 codes[MOVE_ROWS];
    uint32_t params[MOVE_ROWS][L::GROUPS];
    float weight[MOVE_ROWS];
#pragma unroll
    for (int k = 0; k < MOVE_ROWS; ++k) {
      weight[k] = 0.f;
      if (from[k] < 0) continue;
      const int r = from[k] % KV4_BLOCK;
      const uint8_t* block = src + (long long)(from[k] / KV4_BLOCK) * L::BYTES;
      const int at = (piece < C ? 0 : L::V_CODES) + r * L::ROW + (piece < C ? piece : piece - C) * 16;
      codes[k] = *reinterpret_cast<const uint4*>(block + at);
      if (piece < 2) {
#pragma unroll
        for (int g = 0; g < L::GROUPS; ++g)
          params[k][g] = reinterpret_cast<const uint32_t*>(block + (piece == 0 ? L::K_PARAMS : L::V_PARAMS) + r * L::PROW)[g];
      }
      if (piece == 2) weight[k] = a.weights[(long long)row * a.d.capacity + from[k]];
    }
#pragma unroll
    for (int k = 0; k < MOVE_ROWS; ++k) {
      const int j = j0 + k * TEAMS;
      if (piece == 2 && j < a.d_out.capacity) a.weights_out[(long long)row * a.d_out.capacity + j] = weight[k];
      if (from[k] < 0) continue;
      const int r = j % KV4_BLOCK;
      // V's words of a place differ by 4 pairs of words, which is 2 pieces
      const int swap = DH == 64 || piece < C ? 0 : ((from[k] ^ j) & 2);
      uint8_t* block = dst + (long long)(j / KV4_BLOCK) * L::BYTES;
      const int at = (piece < C ? 0 : L::V_CODES) + r * L::ROW + ((piece < C ? piece : piece - C) ^ swap) * 16;
      *reinterpret_cast<uint4*>(block + at) = codes[k];
      if (piece < 2) {
#pragma unroll
        for (int g = 0; g < L::GROUPS; ++g)
          reinterpret_cast<uint32_t*>(block + (piece == 0 ? L::K_PARAMS : L::V_PARAMS) + r * L::PROW)[g] = params[k][g];
      }
    }
  }
}

}  // namespace bpt
