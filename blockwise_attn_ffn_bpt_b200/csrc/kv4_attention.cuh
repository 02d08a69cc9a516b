// Attention of new tokens over the 4-bit cache (kv4_cache.cuh).
//
// For a token's query q (one head) and the cached tokens u that it sees:
//     s_u = q . K_u / sqrt(dh),  o = sum_u 2^(c s_u - lse2) V_u,
//     lse2 = log2 sum_u 2^(c s_u),  c = log2 e,
// with a running maximum and sum over one pass of the cache; the weights of a
// cached token, summed over the queries that share its head, are added to
// weights[u] by a further kernel from the scores that the first one leaves.
//
// Bound by HBM: 144 bytes a cached token and head (dh = 128) for 4 dh flops a
// query, so the codes have to become matrix operands in as few instructions as
// possible. The queries that share a head (heads / kv_heads times the new
// tokens) are the 8 columns of m16n8k16 products, 16 cached tokens (K) or 16
// dimensions (V) their rows:
//     S^T[16 tokens, 8] = K[16, dh] Q^T,   O^T[dh, 8] += V^T[dh, 16] P^T.
// A nibble that lies within the 10 lowest bits of a 16-bit half is, masked, a
// subnormal fp16 number: code 2^e, exactly, with e from its place. So one
// operation (and a shift for some) makes an operand of two codes, and nothing
// has to be taken off the products; powers of two that differ by the place are
// in the other operand (K) or taken out at the end (V). Scale and minimum enter
// after the product with K and before the one with V, for groups of 64 dims:
//     s = sum over groups of scale (q . code) + min (sum q),
//     o = sum_u P' code + sum_u p min,   P' = p scale.
// q enters as fp16 times a power of two that takes its largest element to 2^14
// (exact but for elements 2^-25 below that). P' enters as fp16 times a factor w
// of its column and group, w P' being at most 2^14 and 2^7 where w is set: what
// lies 2^-31 below the largest P' so far is lost, everything above 2^-21 of it
// keeps fp16's 11 bits. w falls when a P' would pass 2^14, and rises with the
// softmax's maximum, which takes the P' of the tokens before with it; it is at
// most 2^125, so that of the smallest scales 2^-150 is lost, as fp32 does itself.
//
// The sum of P' code, 7.5 times that of P' and more, would lose the values' small
// mean over many tokens in its roundings. So every KVA_CENTRE blocks 7.5 sum P'
// is taken off it, and the second sum is of p mid, mid = min + 7.5 scale. (At
// 32768 tokens of equal weight o was 1.6e-2 off in the norm with an offset of
// 135 P' a token in that sum until its end; the rounding of o to bf16 alone is
// 1.7e-3.) The sum taken off is that of the fp16 numbers that met the codes, so
// that a rounding error meets code - 7.5, which is of either sign: P' of nearly
// equal weights all round the same way. (With scores within 1e-4 at 20000 tokens
// o was 5.5e-2 off in the norm with the sum of the P' before their rounding.)
//
// The cached blocks of all sequences and heads, one after the other, are split
// evenly over the warps of the device, whatever the lengths. A warp works on
// its run alone: bulk copies into its own ring of stages, its own maximum, sum
// and O^T; it leaves a partial result for each (sequence, head) that its run
// touches, and kv4_join_kernel joins those.
//
// The products are mma.sync's: its operands are made in registers, where the
// codes are unpacked, while tcgen05 would take them from shared or tensor memory,
// a write and a read of four times the cache's bytes more. They fill a quarter of
// the tensor pipe's cycles (28% with one query a head, 24% with 8, over 8 x 8191
// tokens of 32 heads of 128).
//
// Measured: 8 contexts of 32768 tokens, 32 heads of 128 (1.2 GB) 183 us, 6.6 TB/s;
// 16 of 4096 tokens (302 MB) 55 us, 46 us of it at the memory's rate, the others
// being the start (3 us until the first blocks arrive) and the end (warps that
// finish one after another). What bounds it then is the memory; in calls without
// pause also the 1 kW power cap.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "kv4_cache.cuh"
#include "kv4_split.h"

namespace bpt {

constexpr int KVA_MAX_SMS = 148;      // the split does not grow past it (workspaces are sized without a device)
// Blocks between two takings off of the codes' mean. 256 heads over 32 of 128, 16 x
// 32768 tokens: with 16, o was 3.5e-4 off beside its rounding and the call took
// 417.6 us, with 8 2.4e-4 and 418.2, with 4 2.2e-4 (2e-4 of it the weights' fp16)
// and 419.7; with 512 heads 757, 759 and 764 us.
constexpr int KVA_CENTRE = 8;
constexpr float KVA_HIGH = 16384.0f, KVA_WIDEST = 0x1p125f;  // of w P' and of w (whose reciprocal is a normal number)
constexpr float KVA_LAZY = 8.0f;      // the maximum is raised when a score passes it by this (log2)

// Warps of an SM and stages of a warp: the rings take 216 KB in every case, and
// the registers of that many warps hold what NT blocks of 8 columns need.
template <int DH, int NT>
struct KvaCfg {
  static constexpr int WARPS = DH == 128 ? (NT == 1 ? 12 : 8) : (NT == 1 ? 16 : 12);
  static constexpr int STAGES = DH == 128 ? (NT == 1 ? 2 : 3) : (NT == 1 ? 3 : 4);
  static constexpr int RING = WARPS * STAGES * Kv4<DH>::BYTES;
  static constexpr int SMEM = RING + WARPS * STAGES * 8 + 16 + 128;
};

inline int kva_warps(int dh, int nt) {
  if (dh == 128) return nt == 1 ? KvaCfg<128, 1>::WARPS : KvaCfg<128, 2>::WARPS;
  return nt == 1 ? KvaCfg<64, 1>::WARPS : KvaCfg<64, 2>::WARPS;
}

struct Kv4AttnArgs {
  const __nv_bfloat16* q;  // token (beta, t) at beta * bs + t * ld
  long long bs_q, ld_q;
  const uint8_t* cache;
  Kv4Dims d;
  const int* lens;         // [b], the new tokens among them
  int n, heads, causal;
  int cols, cols_block, blocks_of_cols;  // queries that share a head; those of one pass over it; passes
  int max_warps;
  float score_scale;       // log2(e) / sqrt(dh)
  __nv_bfloat16* o;        // [b, n, heads * dh]
  float* lse2;             // [b, heads, n], or null
  float* scores;           // [b, kv_heads, cols, capacity] in log2 units, or null
  float* part_o;           // [slots][cols_block][dh]: sums of a run, not divided
  float2* part_ml;         // [slots][cols_block]: maximum and sum
  int* status;
};

// Cached tokens that new token t of a sequence of `len` tokens sees.
__device__ __forceinline__ int kv4_seen(int len, int n, int t, int causal) {
  return causal ? max(len - n + 1 + t, 0) : len;
}

__device__ __forceinline__ int kva_blocks(const Kv4AttnArgs& a, int beta) {
  return (min(max(a.lens[beta], 0), a.d.capacity) + KV4_BLOCK - 1) / KV4_BLOCK;
}

// Called by a whole warp: the split, and the units before sequence `beta`.
__device__ __forceinline__ KvaSplit kva_split(const Kv4AttnArgs& a, int beta, uint32_t& before) {
  const uint32_t per = (uint32_t)a.d.kv_heads * a.blocks_of_cols;
  uint32_t total = 0, prior = 0;
  for (int i = lane_id(); i < a.d.b; i += 32) {
    const uint32_t nb = kva_blocks(a, i);
    const uint32_t units = kva_units(nb);
    total += units;
    if (i < beta) prior += units;
  }
  before = __reduce_add_sync(0xffffffffu, prior) * per;
  return KvaSplit(__reduce_add_sync(0xffffffffu, total) * per, (uint32_t)a.max_warps);
}

// The place of unit t, and the run of n units from there (whole warp).
__device__ __forceinline__ KvaPlace kva_find(const Kv4AttnArgs& a, uint32_t t, int n, int rows) {
  uint32_t base = 0;
  const int lane = lane_id();
  for (int b0 = 0; b0 < a.d.b; b0 += 32) {
    const uint32_t nb = b0 + lane < a.d.b ? kva_blocks(a, b0 + lane) : 0;
    const uint32_t units = kva_units(nb) * rows;
    uint32_t sum = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + sum > t);
    if (past) {
      const int src = __ffs(past) - 1;
      const uint32_t blocks = __shfl_sync(0xffffffffu, nb, src);
      return KvaPlace::in_sequence(b0 + src, blocks, t - (base + __shfl_sync(0xffffffffu, sum - units, src)), n);
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return KvaPlace{a.d.b, 0, 0, 0, 0};
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// d = A B + c, fp16 operands
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

__device__ __forceinline__ float scale_of(uint32_t params) { return __uint_as_float(params << 16); }
__device__ __forceinline__ float min_of(uint32_t params) { return __uint_as_float(params & 0xffff0000u); }

// Lane (g, t) = (lane / 4, lane % 4). Row k of a 16-row product is the cached
// token kva_token(k) of the 16: lane t of V's operand then reads rows t, 7 - t,
// 8 + t and 15 - t, four neighbouring rows in every read of the warp, and the
// two rows of K that 8 lanes read together lie in different halves of the banks.
__device__ __forceinline__ int kva_token(int k) { return (k & 1) ? 7 - (k >> 1) : k >> 1; }

// NT blocks of 8 columns. With fewer queries than columns (NT = 1, F > 1) the 8
// columns hold F copies of 8 / F queries, and copy f meets only the f-th of F
// groups of 16 tokens (its queries are zero in the products of the others), so
// that one accumulator ends up with the scores of 16 F tokens and the softmax
// costs a lane F times less; the copies' sums are added at the end of the run.
//
// DIRECT: instead of the even split over the device, a block takes one segment,
// splits it over its warps and joins their sums itself, which saves the second
// kernel (kva_direct).
template <int DH, int NT, int F, bool DIRECT>
__global__ void __launch_bounds__(KvaCfg<DH, NT>::WARPS * 32, 1) kv4_attention_kernel(const __grid_constant__ Kv4AttnArgs a) {
  static_assert(NT == 1 || F == 1, "copies of the queries fill one block of columns");
  using L = Kv4<DH>;
  using C = KvaCfg<DH, NT>;
  constexpr int G = L::GROUPS, KW = DH / 32;  // groups; words of a K row that a lane takes
  constexpr int CW = 8 / F, J = 4 / F;        // columns of a copy; accumulators that 64 tokens need
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_addr(smem_raw) + 127u) & ~127u;
  volatile int* flag = reinterpret_cast<volatile int*>(smem_raw + (smem - smem_addr(smem_raw)) + C::RING + C::WARPS * C::STAGES * 8);
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem + warp * C::STAGES * L::BYTES;
  const uint32_t bars = smem + C::RING + warp * C::STAGES * 8;
  if (threadIdx.x == 0) *flag = 0;
  if (lane == 0)
    for (int i = 0; i < C::STAGES; ++i) mbar_init(bars + i * 8, 1);
  fence_mbar_init();
  __syncthreads();
  const Abort ab{flag, a.status};
  grid_dependency_wait();
  grid_dependents_start();  // not earlier: the kernels behind read lens and the weights before they wait

  const int rows = a.d.kv_heads * a.blocks_of_cols, group = a.heads / a.d.kv_heads;
  if (blockIdx.x == 0 && warp == 0)
    for (int i = lane; i < a.d.b; i += 32) clamp_count(a.lens[i], a.d.capacity, a.status);
  int w = 0;
  KvaPlace at;
  if constexpr (DIRECT) {
    const int beta = blockIdx.x / rows, nb = kva_blocks(a, beta), each = nb / C::WARPS, rest = nb - each * C::WARPS;
    at = KvaPlace{beta, (int)blockIdx.x - beta * rows, each * warp + min(warp, rest), nb, each + (warp < rest)};
  } else {
    uint32_t unused;
    const KvaSplit split = kva_split(a, 0, unused);
    w = warp * gridDim.x + blockIdx.x;  // neighbours of a run on different SMs
    if (w >= (int)split.warps || split.total == 0) return;
    const uint32_t t0 = split.first(w);
    at = kva_find(a, t0, (int)(split.first(w + 1) - t0), rows);
  }
  KvaPlace next = at;

  auto blocks_of = [&](int beta) { return kva_blocks(a, beta); };
  int issued = 0;
  auto issue = [&]() {  // the next block of the run into its stage
    if (next.left <= 0) return;
    if (lane == 0) {
      const uint32_t bar = bars + issued % C::STAGES * 8;
      const uint8_t* src =
          a.cache + (((long long)next.beta * a.d.kv_heads + next.row / a.blocks_of_cols) * a.d.blocks() + next.blk) * L::BYTES;
      mbar_arrive_expect_tx(bar, L::BYTES);
      bulk_load(ring + issued % C::STAGES * L::BYTES, src, L::BYTES, bar);
    }
    ++issued;
    next.advance(blocks_of, a.d.b, rows, 1);
  };
  const int fold = 2 * t / CW;           // the copy that this lane's two columns of a result belong to
  const int row_fold = F == 1 ? 0 : g / CW;  // the copy that this lane's column of an operand belongs to
  const float lazy = KVA_LAZY / a.score_scale;
  // where this lane's words and parameters lie in a block, the compile-time
  // parts left out (8 rows on, V's words lie in the same order)
  const uint32_t k_at = kva_token(g) * L::ROW + t * (L::ROW / 4);
  const uint32_t v_at[2] = {L::V_CODES + t * L::ROW + kv4_v_place<DH>(g, t) * 4u,
                            L::V_CODES + (7 - t) * L::ROW + kv4_v_place<DH>(g, 7 - t) * 4u};
  const int token = fold * 16 + kva_token(g);  // of this lane's results: 16 F j + token, and 8 on
  // DIRECT: the warp's sums, in its ring once its blocks are done with
  float* own_o = reinterpret_cast<float*>(smem_raw + (ring - smem_addr(smem_raw)));
  float2* own_ml = reinterpret_cast<float2*>(own_o + 8 * NT * DH);
  int done = 0;
  bool lost = false, summed = false;
  while (at.left > 0) {
    // one segment's part of the run
    const int len = min(max(a.lens[at.beta], 0), a.d.capacity);
    const int kvh = at.row / a.blocks_of_cols, cb = at.row - kvh * a.blocks_of_cols;
    const int col0 = cb * 8 * NT;
    uint32_t qf[NT][F][KW][4];
    float qs[NT][G][2], unit[NT][2];  // sums of q; what a product of q with codes is times q and codes
    int lim[NT][2];
    uint4 raw[NT][KW];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = col0 + nt * 8 + g % CW;
      const bool real = col < a.cols;
      const int tok = real ? col / group : 0, head = kvh * group + (real ? col - tok * group : 0);
      const __nv_bfloat16* q = a.q + at.beta * a.bs_q + tok * a.ld_q + (long long)head * DH;
#pragma unroll
      for (int i = 0; i < KW; ++i)
        raw[nt][i] = real ? *reinterpret_cast<const uint4*>(q + (i * 4 + t) * 8) : make_uint4(0, 0, 0, 0);
    }
    if (issued == 0)  // the first blocks, behind the queries: those would wait for all of them
      for (int i = 0; i < C::STAGES; ++i) issue();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t top = 0;  // largest |q|, as bits
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t y[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(y[e] & 0x7fffu, y[e] >> 16 & 0x7fffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^14 over the power of two in it, as the bits of an exponent
      const int up = min(268 - (int)(top >> 7), 250);  // times 2 is finite still
      const float times = __int_as_float(up << 23);
      float sum[G] = {};
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t y[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = scale_of(y[e]);
          x[2 * e + 1] = min_of(y[e]);
          sum[i / 2] += x[2 * e] + x[2 * e + 1];
        }
        // dimensions e and e + 4 meet codes times 8, 4, 64 and 8 (2^-24)
        constexpr float place[4] = {1.0f, 2.0f, 0.125f, 1.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t two = pack_half2(x[e] * (times * place[e]), x[e + 4] * (times * place[e]));
#pragma unroll
          for (int f = 0; f < F; ++f) qf[nt][f][i][e] = row_fold == f ? two : 0u;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        unit[nt][e] = __int_as_float(min(275 - __shfl_sync(0xffffffffu, up, (2 * t + e) * 4), 255) << 23);
#pragma unroll
      for (int gi = 0; gi < G; ++gi) {
        sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 1);
        sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) qs[nt][gi][e] = __shfl_sync(0xffffffffu, sum[gi], (2 * t + e) * 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[nt][e] = kv4_seen(len, a.n, (col0 + nt * 8 + (2 * t + e) % CW) / group, a.causal);
    }
    const int lim_all = kv4_seen(len, a.n, col0 / group, a.causal);  // seen by every column

    // m: the maximum's reference, in units of a score before score_scale; the
    // sums of a lane are of its own tokens until the end of the run
    float o[NT][G][4][4] = {};
    float m[NT][2], ref[NT][2] = {}, l[NT][2] = {}, off[NT][G][2] = {};  // ref: m score_scale, or 0 for none
    float part[NT][G][2] = {};  // sums of w P', as rounded, not yet taken off o
    float wide[NT][G][2];  // w of the comment above
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) wide[nt][gi][e] = KVA_WIDEST;
      }

    // One block of 64 tokens. WHOLE: every column sees all of them.
    auto block = [&](auto whole_tag, uint32_t blk, int key0) {
      constexpr bool WHOLE = decltype(whole_tag)::value;
      float s[J][NT][4];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float acc[NT][G][4];
#pragma unroll
        for (int f = 0; f < F; ++f) {
          uint32_t ka[KW], kb[KW];
          lds(blk + k_at + (j * F + f) * 16 * L::ROW, ka);
          lds(blk + k_at + ((j * F + f) * 16 + 8) * L::ROW, kb);
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            uint32_t xa[4], xb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // the words are rotated left by 3: nibbles 0 (and 4) in bits 3 .. 6, and 5 bits
              // on nibbles 1 in bits 2 .. 5 and 2 in bits 6 .. 9, and 12 bits on 3 in 3 .. 6
              constexpr int shift[4] = {0, 5, 5, 12};
              constexpr uint32_t mask[4] = {0x00780078u, 0x003c003cu, 0x03c003c0u, 0x00780078u};
              xa[e] = __funnelshift_r(ka[i], ka[i], shift[e]) & mask[e];
              xb[e] = __funnelshift_r(kb[i], kb[i], shift[e]) & mask[e];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t(&b)[4] = qf[nt][f][i];
              float(&d)[4] = acc[nt][i / 2];
              float none[4] = {};
              mma16816(d, xa[0], xb[0], xa[1], xb[1], b[0], b[1], f == 0 && i % 2 == 0 ? none : d);
              mma16816(d, xa[2], xb[2], xa[3], xb[3], b[2], b[3], d);
            }
          }
        }
        const int ra = j * F * 16 + token;
        uint32_t pa[G], pb[G];
        lds(blk + L::K_PARAMS + ra * L::PROW, pa);
        lds(blk + L::K_PARAMS + (ra + 8) * L::PROW, pb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t(&p)[G] = e < 2 ? pa : pb;
            float x = scale_of(p[0]) * acc[nt][0][e], y = min_of(p[0]) * qs[nt][0][e & 1];
#pragma unroll
            for (int gi = 1; gi < G; ++gi) {
              x = fmaf(scale_of(p[gi]), acc[nt][gi][e], x);
              y = fmaf(min_of(p[gi]), qs[nt][gi][e & 1], y);
            }
            x = fmaf(x, unit[nt][e & 1], y);
            if (!WHOLE && key0 + ra + (e >> 1) * 8 >= lim[nt][e & 1]) x = -INFINITY;
            s[j][nt][e] = x;
          }
      }
      if (a.scores != nullptr) {
        float* to = a.scores + ((long long)at.beta * a.d.kv_heads + kvh) * a.cols * a.d.capacity + key0 + token;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = col0 + nt * 8 + (2 * t + (e & 1)) % CW;
            if (col < a.cols)
#pragma unroll
              for (int j = 0; j < J; ++j)
                to[(long long)col * a.d.capacity + j * F * 16 + (e >> 1) * 8] = s[j][nt][e] * a.score_scale;
          }
      }

      // the maximum: raised only where a score passes it by more than KVA_LAZY
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
          for (int j = 1; j < J; ++j) x = max3f(x, s[j][nt][e], s[j][nt][e + 2]);
          top[nt][e] = x;
          grow |= x > m[nt][e] + lazy;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float now = fmaxf(m[nt][e], top[nt][e]);
#pragma unroll
            for (int x = CW / 2; x < 32; x <<= 1)  // all lanes that hold this column or a copy of it
              now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, x));
            const float f = m[nt][e] == -INFINITY ? 0.f : ex2_approx((m[nt][e] - now) * a.score_scale);
            const float back = m[nt][e] == -INFINITY ? INFINITY : ex2_approx((now - m[nt][e]) * a.score_scale);
            m[nt][e] = now;
            ref[nt][e] = now == -INFINITY ? 0.f : now * a.score_scale;
            l[nt][e] *= f;
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
              off[nt][gi][e] *= f;
              // the P' so far fall by f: w rises by as much and their sum stays, as long as w can
              float& w = wide[nt][gi][e];
              const float more = w * back, now_o = more <= KVA_WIDEST ? 1.0f : __fdividef(KVA_WIDEST * f, w);
              w = fminf(more, KVA_WIDEST);
              part[nt][gi][e] *= now_o;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][gi][i][e] *= now_o;
                o[nt][gi][i][e + 2] *= now_o;
              }
            }
          }
      }

#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int ra = j * F * 16 + token;
        uint32_t va[G], vb[G];
        lds(blk + L::V_PARAMS + ra * L::PROW, va);
        lds(blk + L::V_PARAMS + (ra + 8) * L::PROW, vb);
        uint32_t bf[NT][G][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4], y[G][4], high = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2_approx(fmaf(s[j][nt][e], a.score_scale, -ref[nt][e & 1]));
            l[nt][e & 1] += p[e];
          }
#pragma unroll
          for (int gi = 0; gi < G; ++gi) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t pr = e < 2 ? va[gi] : vb[gi];
              y[gi][e] = p[e] * scale_of(pr);
              // a token that is not seen may have any parameters, NaN among them
              const bool live = WHOLE || key0 + ra + (e >> 1) * 8 < lim[nt][e & 1];
              if (!live) y[gi][e] = 0.f;
              if (live) off[nt][gi][e & 1] = fmaf(p[e], fmaf(7.5f, scale_of(pr), min_of(pr)), off[nt][gi][e & 1]);
            }
            high = max3f(high, y[gi][0] * wide[nt][gi][0], y[gi][1] * wide[nt][gi][1]);
            high = max3f(high, y[gi][2] * wide[nt][gi][0], y[gi][3] * wide[nt][gi][1]);
          }
          if (__any_sync(0xffffffffu, high > KVA_HIGH)) {
#pragma unroll
            for (int gi = 0; gi < G; ++gi)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(y[gi][e], y[gi][e + 2]);
#pragma unroll
                for (int x = CW / 2; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                float& w = wide[nt][gi][e];
                if (top * w > KVA_HIGH) {  // the power of two that takes it to 2^7
                  const float less = __int_as_float((261 - (__float_as_int(top) >> 23)) << 23), now_o = __fdividef(less, w);
                  w = less;
                  part[nt][gi][e] *= now_o;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    o[nt][gi][i][e] *= now_o;
                    o[nt][gi][i][e + 2] *= now_o;
                  }
                }
              }
          }
#pragma unroll
          for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const __half2 two = __floats2half2_rn(y[gi][2 * x] * wide[nt][gi][0], y[gi][2 * x + 1] * wide[nt][gi][1]);
              const float2 rounded = __half22float2(two);
              part[nt][gi][0] += rounded.x;
              part[nt][gi][1] += rounded.y;
              bf[nt][gi][x] = transpose8(*reinterpret_cast<const uint32_t*>(&two));
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
          uint32_t v[4][G];  // this lane's words of four tokens
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            lds(blk + v_at[x & 1] + ((j * F + f) * 16 + (x >> 1) * 8) * L::ROW, v[x]);
          }
#pragma unroll
          for (int gi = 0; gi < G; ++gi) {
            const uint32_t lo0 = __byte_perm(v[0][gi], v[1][gi], 0x5410), hi0 = __byte_perm(v[0][gi], v[1][gi], 0x7632);
            const uint32_t lo1 = __byte_perm(v[2][gi], v[3][gi], 0x5410), hi1 = __byte_perm(v[2][gi], v[3][gi], 0x7632);
            uint32_t b[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) b[nt][x] = F == 1 || row_fold == f ? bf[nt][gi][x] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // nibbles 0 and 2 in bits 0 .. 3, 1 and 3 (times 16) in bits 4 .. 7
              auto code = [&](uint32_t x) { return x >> (i / 2 * 8) & (i % 2 ? 0x00f000f0u : 0x000f000fu); };
              const uint32_t a0 = code(lo0), a1 = code(hi0), a2 = code(lo1), a3 = code(hi1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][gi][i], a0, a1, a2, a3, b[nt][0], b[nt][1], o[nt][gi][i]);
            }
          }
        }
      }
    };

    auto over_lanes = [](float x) {  // of a column and its copies
#pragma unroll
      for (int y = CW / 2; y < 32; y <<= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
      return x;
    };
    auto over_copies = [](float x) {
#pragma unroll
      for (int y = CW / 2; y < 4; y <<= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
      return x;
    };
    auto centre = [&]() {  // takes 7.5 times the sum of the rounded P' off o, off each copy its own
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float all = part[nt][gi][e];
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) all += __shfl_xor_sync(0xffffffffu, all, y);
            part[nt][gi][e] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = all * (i % 2 ? -7.5f * 0x1p-20f : -7.5f * 0x1p-24f);
              o[nt][gi][i][e] += x;
              o[nt][gi][i][e + 2] += x;
            }
          }
    };

    const int piece = min(at.nb - at.blk, at.left);
    for (int k = 0; k < piece; ++k) {
      const int stage = done % C::STAGES;
      if (!warp_wait(bars + stage * 8, (done / C::STAGES) & 1, ab)) {
        // the copies still in flight land before the warp leaves its ring
        for (int i = done + 1; i < issued; ++i) {
          const unsigned long long since = global_timer_ns();
          while (!mbar_try_wait(bars + i % C::STAGES * 8, (i / C::STAGES) & 1) &&
                 global_timer_ns() - since < kWaitTimeoutNs) {}
        }
        lost = true;
        break;
      }
      const int key0 = (at.blk + k) * KV4_BLOCK;
      if (key0 + KV4_BLOCK <= lim_all)
        block(std::true_type{}, ring + stage * L::BYTES, key0);
      else
        block(std::false_type{}, ring + stage * L::BYTES, key0);
      __syncwarp();  // every lane has read the stage
      ++done;
      issue();
      if (k % KVA_CENTRE == KVA_CENTRE - 1) centre();
    }

    if (lost) break;

    // the run's sums for this segment
    const long long slot = (long long)at.beta * rows + at.row + w;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum = over_lanes(l[nt][e]);
        const int c = nt * 8 + 2 * t + e;
        const bool real = 2 * t < CW && col0 + c < a.cols;
        const long long to = slot * a.cols_block + c;
        if (real && g == 0) (DIRECT ? own_ml + c : a.part_ml + to)[0] = make_float2(m[nt][e] * a.score_scale, sum);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
          const float per = 1.0f / wide[nt][gi][e], add = over_lanes(fmaf(-7.5f * per, part[nt][gi][e], off[nt][gi][e]));
          float x[8];  // dimensions 8u .. 8u + 7 of word u = 8 gi + g
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float unit = i % 2 ? 0x1p20f : 0x1p24f;
            x[i] = fmaf(over_copies(o[nt][gi][i][e]) * unit, per, add);
            x[i + 4] = fmaf(over_copies(o[nt][gi][i][e + 2]) * unit, per, add);
          }
          if (real) {
            float4* dst = reinterpret_cast<float4*>((DIRECT ? own_o + c * DH : a.part_o + to * DH) + (gi * 8 + g) * 8);
            dst[0] = make_float4(x[0], x[1], x[2], x[3]);
            dst[1] = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      }
    summed = true;
    at.advance(blocks_of, a.d.b, rows, piece);
  }

  if constexpr (DIRECT) {
    if (!summed && lane < 8 * NT) own_ml[lane] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    const int beta = blockIdx.x / rows, row = blockIdx.x - beta * rows;
    const int kvh = row / a.blocks_of_cols, col0 = (row - kvh * a.blocks_of_cols) * 8 * NT;
    const int cols = min(a.cols - col0, 8 * NT);
    const float* o0 = reinterpret_cast<const float*>(smem_raw + (smem - smem_addr(smem_raw)));
    constexpr int STRIDE = C::STAGES * L::BYTES / 4;  // from warp to warp
    for (int i = threadIdx.x; i < cols * DH; i += C::WARPS * 32) {
      const int c = i / DH;
      float m = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
      for (int v = 0; v < C::WARPS; ++v) m = fmaxf(m, reinterpret_cast<const float2*>(o0 + v * STRIDE + 8 * NT * DH)[c].x);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int v = 0; v < C::WARPS; ++v) {
        const float2 ml = reinterpret_cast<const float2*>(o0 + v * STRIDE + 8 * NT * DH)[c];
        const float k = ex2_approx(ml.x - ref);
        sum = fmaf(ml.y, k, sum);
        // a warp without blocks has left nothing here (one whose blocks are all
        // masked has left zeros)
        if (ml.x != -INFINITY || ml.y != 0.f) x = fmaf(o0[v * STRIDE + i], k, x);
      }
      const bool none = sum == 0.f;  // a row that sees no token is zero
      const int tok = (col0 + c) / group, head = kvh * group + col0 + c - tok * group;
      a.o[(((long long)beta * a.n + tok) * a.heads + head) * DH + i - c * DH] = __float2bfloat16_rn(none ? 0.f : x / sum);
      if (i == c * DH && a.lse2 != nullptr) a.lse2[((long long)beta * a.heads + head) * a.n + tok] = none ? -INFINITY : ref + log2f(sum);
    }
  }
}

// The kernel for `cols` queries that share a head: one block of columns up to 8
// of them, with as many copies as fit; two blocks (16 a pass) above that.
inline int kva_col_blocks(int cols) { return cols <= 8 ? 1 : 2; }

typedef void (*KvaKernel)(const Kv4AttnArgs);
template <int DH, bool DIRECT>
KvaKernel kva_kernel(int cols) {
  if (cols <= 2) return kv4_attention_kernel<DH, 1, 4, DIRECT>;
  if (cols <= 4) return kv4_attention_kernel<DH, 1, 2, DIRECT>;
  return cols <= 8 ? kv4_attention_kernel<DH, 1, 1, DIRECT> : kv4_attention_kernel<DH, 2, 1, DIRECT>;
}

inline KvaKernel kva_kernel(int dh, int cols, bool direct) {
  if (dh == 128) return direct ? kva_kernel<128, true>(cols) : kva_kernel<128, false>(cols);
  return direct ? kva_kernel<64, true>(cols) : kva_kernel<64, false>(cols);
}

inline int kva_smem(int dh, int cols) {
  if (dh == 128) return cols <= 8 ? KvaCfg<128, 1>::SMEM : KvaCfg<128, 2>::SMEM;
  return cols <= 8 ? KvaCfg<64, 1>::SMEM : KvaCfg<64, 2>::SMEM;
}

// Whether every segment gets a thread block of its own (DIRECT). It saves the
// join, about 3.5 us, and costs the SMs that have no segment: a warp then has
// `blocks` / `warps` blocks of tokens instead of that times segments / SMs, at
// about 2 us a block. Device time of one call, direct against split: 4 segments
// of 200 tokens (dh = 64) 4.6 against 8.2 us; 32 segments (dh = 128) of 1000
// tokens 8.8 against 10.0, of 2000 tokens 12.1 against 10.1; 128 segments of 3000
// tokens 15.4 against 18.1. These are for caches that are full: the host knows the
// capacity alone, and a block with a long sequence among short ones keeps the
// others waiting. So a warp takes 4 blocks at most: 148 segments (dh = 128) of just
// those 48 15.3 against 19.5 us, with lengths spread evenly 15.0 against 15.1,
// with one full sequence of 37 14.6 against 10.5; of 8192 tokens, which would be 11
// blocks, 33.8 against 36.1, 31.6 against 22.8 and 30.9 against 12.2.
constexpr int KVA_DIRECT = 4;
inline bool kva_direct(long long segments, int blocks, int warps) {
  return segments <= KVA_MAX_SMS && blocks <= KVA_DIRECT * warps &&
         (long long)blocks * (KVA_MAX_SMS - segments) * 10 <= 16LL * warps * KVA_MAX_SMS;
}

inline bool kva_set_attributes() {
  bool ok = true;
  for (int dh : {64, 128})
    for (int cols : {2, 4, 8, 16})
      for (bool direct : {false, true})
        ok = ok && cudaFuncSetAttribute(kva_kernel(dh, cols, direct), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kva_smem(dh, cols)) == cudaSuccess;
  return ok;
}

constexpr int KVJ_UNROLL = 4;
constexpr int kvj_threads(int warps) { return (warps < 8 ? 8 : warps) * 32; }

// Joins the partial results of the columns of all (sequence, head)s: WARPS warps
// a column (8 columns a block with one), each taking every WARPS-th of its
// partial results, KVJ_UNROLL in flight, a lane DH / 32 dimensions. It is
// launched while the attention still runs and waits for it here, so that its
// start costs nothing. Bound by the latency of its reads (kvj_warps).
template <int DH, int WARPS>
__global__ void __launch_bounds__(kvj_threads(WARPS)) kv4_join_kernel(const __grid_constant__ Kv4AttnArgs a) {
  constexpr int E = DH / 32, COLS = kvj_threads(WARPS) / 32 / WARPS;
  static_assert(WARPS == 1 || COLS == 1, "a block joins one column, or a warp does");
  __shared__ float s_m[WARPS], s_l[WARPS], s_o[WARPS > 1 ? WARPS : 1][WARPS > 1 ? DH : 1];
  const int warp = warp_id() % WARPS, lane = lane_id();
  const int rows = a.d.kv_heads * a.blocks_of_cols, group = a.heads / a.d.kv_heads;
  const int all = a.d.kv_heads * a.cols, chunks = (all + COLS - 1) / COLS;
  grid_dependents_start();
  bool waited = false;
  int last = -1, nb = 0;
  uint32_t before = 0;
  KvaSplit split(0, 1);
  auto column = [&](int beta, int x0) {
    if (beta != last) {
      split = kva_split(a, beta, before);
      nb = kva_blocks(a, beta);
      last = beta;
    }
    const bool real = x0 < all;
    const int kvh = x0 / a.cols, col = x0 - kvh * a.cols;
    const int per = a.cols_block, cb = col / per, c = col - cb * per;
    const int tok = col / group, head = kvh * group + col - tok * group;
    const int row = kvh * a.blocks_of_cols + cb;
    int w0 = 0, w1 = -1;
    if (nb > 0 && real) {
      const uint32_t first = before + kva_first_block(row, nb);
      w0 = split.warp_of(first);
      w1 = split.warp_of(first + nb - 1);
    }
    if (!waited) {
      grid_dependency_wait();
      waited = true;
    }
    const long long at0 = ((long long)beta * rows + row) * a.cols_block + c;
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int w = w0 + warp; w <= w1; w += WARPS * KVJ_UNROLL) {
      float2 ml[KVJ_UNROLL];
      float x[KVJ_UNROLL][E];
#pragma unroll
      for (int u = 0; u < KVJ_UNROLL; ++u) {
        const int v = w + u * WARPS;
        const long long at = at0 + (long long)v * a.cols_block;
        ml[u] = v <= w1 ? __ldcg(&a.part_ml[at]) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = v <= w1 ? __ldcg(&a.part_o[at * DH + e * 32 + lane]) : 0.f;
      }
      float now = m;
#pragma unroll
      for (int u = 0; u < KVJ_UNROLL; ++u) now = fmaxf(now, ml[u].x);
      const float ref = now == -INFINITY ? 0.f : now, f = ex2_approx(m - ref);
      m = now;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int u = 0; u < KVJ_UNROLL; ++u) {
        const float k = ex2_approx(ml[u].x - ref);
        l = fmaf(ml[u].y, k, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(x[u][e], k, o[e]);
      }
    }
    // a row that sees no token is zero
    __nv_bfloat16* to = a.o + (((long long)beta * a.n + tok) * a.heads + head) * DH;
    float* lse2 = a.lse2 == nullptr ? nullptr : a.lse2 + ((long long)beta * a.heads + head) * a.n + tok;
    if constexpr (WARPS == 1) {
      if (!real) return;
#pragma unroll
      for (int e = 0; e < E; ++e) to[e * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
      if (lane == 0 && lse2 != nullptr) *lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    } else {
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
      __syncthreads();
      float top = s_m[0];
#pragma unroll
      for (int i = 1; i < WARPS; ++i) top = fmaxf(top, s_m[i]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) sum = fmaf(s_l[i], ex2_approx(s_m[i] - ref), sum);
      const bool none = sum == 0.f;
      if (threadIdx.x < DH) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) x = fmaf(s_o[i][threadIdx.x], ex2_approx(s_m[i] - ref), x);
        to[threadIdx.x] = __float2bfloat16_rn(none ? 0.f : x / sum);
      }
      if (threadIdx.x == 0 && lse2 != nullptr) *lse2 = none ? -INFINITY : ref + log2f(sum);
      __syncthreads();
    }
  };
  if constexpr (WARPS == 1) {
    // a run of columns a block, 8 at a time: they mostly share a sequence. (Their number is below 2^31: b n heads is.)
    const unsigned items = (unsigned)a.d.b * (unsigned)chunks, each = items / gridDim.x, rest = items - each * gridDim.x;
    const unsigned from = each * blockIdx.x + min(blockIdx.x, rest), until = from + each + (blockIdx.x < rest ? 1u : 0u);
    for (unsigned item = from; item < until; ++item) {
      const unsigned beta = item / (unsigned)chunks;
      column((int)beta, (int)(item - beta * (unsigned)chunks) * COLS + warp_id());
    }
  } else {
    for (int beta = blockIdx.y; beta < a.d.b; beta += gridDim.y) column(beta, blockIdx.x);
  }
}

// Warps a column: one where blocks of 8 (4 of them fit an SM) would take a second
// round, 32 where few columns have many partial results each. Device time of one
// call, with 1, 8 and 32: 27520 columns 63, 174, 761 us; 1024 39.1, 44.6, 68; 768
// 27.4, 28.1, 48; 512 37.3, 36.3, 51; 128 of 55 partial results 74, 65, 67; 64 of
// 111 67, 47, 46; 32 of 222 64, 34, 30; 32 of 592 109, 31, 17.
inline int kvj_warps(long long columns, long long segments, int max_warps) {
  if (columns > KVA_MAX_SMS * 4) return 1;
  return columns <= KVA_MAX_SMS * 2 && max_warps / segments > 64 ? 32 : 8;
}

inline KvaKernel kvj_kernel(int dh, int warps) {
  if (dh == 128) return warps == 1 ? kv4_join_kernel<128, 1> : warps == 8 ? kv4_join_kernel<128, 8> : kv4_join_kernel<128, 32>;
  return warps == 1 ? kv4_join_kernel<64, 1> : warps == 8 ? kv4_join_kernel<64, 8> : kv4_join_kernel<64, 32>;
}

struct Kv4WeightsArgs {
  const float* scores;  // as in Kv4AttnArgs
  const float* lse2;    // [b, heads, n]
  float* weights;       // [b, kv_heads, capacity]
  Kv4Dims d;
  const int* lens;
  int n, heads, causal;
};

// weights[u] += sum over the queries that share u's head of 2^(score - lse2):
// V times 4 cached tokens a thread. Bound by the latency of its reads (the scores
// come from L2 where they fit): what does not wait for the kernels ahead is read
// before they end, the scores of Q queries at a time after. 64 rows of about 27000
// tokens, 4 queries each: 10 us with V = Q = 2, 16 with one vector a thread and
// every read after the wait.
constexpr int KVW_THREADS = 128;

template <int V, int Q>
__global__ void __launch_bounds__(KVW_THREADS, Q > 2 ? 4 : 8) kv4_weights_kernel(const __grid_constant__ Kv4WeightsArgs a) {
  constexpr int STEP = KVW_THREADS * 4;
  const int group = a.heads / a.d.kv_heads, cols = group * a.n;
  const int key = blockIdx.x * STEP * V + threadIdx.x * 4;
  const int rows = a.d.b * a.d.kv_heads;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int beta = row / a.d.kv_heads, kvh = row - beta * a.d.kv_heads;
    float* to = a.weights + (long long)row * a.d.capacity;
    float4 old[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key + v * STEP < a.d.capacity) old[v] = *reinterpret_cast<const float4*>(to + key + v * STEP);
    const int len = min(max(a.lens[beta], 0), a.d.capacity);
    grid_dependency_wait();
    grid_dependents_start();
    if (key >= len) continue;
    const float* s = a.scores + (long long)row * cols * a.d.capacity + key;
    const float* lse2 = a.lse2 + ((long long)beta * a.heads + kvh * group) * a.n;
    float sum[V][4] = {};
    int t = 0, h = 0;  // token and head of the next query
    for (int c = 0; c < cols; c += Q) {
      float4 x[Q][V];
      float l[Q];
      int seen[Q];
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        seen[k] = 0;
        if (c + k < cols) {
          seen[k] = kv4_seen(len, a.n, t, a.causal);
          l[k] = __ldcg(lse2 + h * a.n + t);
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (key + v * STEP < len) x[k][v] = __ldcs(reinterpret_cast<const float4*>(s + (long long)(c + k) * a.d.capacity + v * STEP));
          if (++h == group) {
            h = 0;
            ++t;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < Q; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int at = key + v * STEP;
          if (at < seen[k]) sum[v][0] += ex2_approx(x[k][v].x - l[k]);
          if (at + 1 < seen[k]) sum[v][1] += ex2_approx(x[k][v].y - l[k]);
          if (at + 2 < seen[k]) sum[v][2] += ex2_approx(x[k][v].z - l[k]);
          if (at + 3 < seen[k]) sum[v][3] += ex2_approx(x[k][v].w - l[k]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = key + v * STEP;
      if (at < len)  // past the length nothing changes
        *reinterpret_cast<float4*>(to + at) = make_float4(old[v].x + sum[v][0], at + 1 < len ? old[v].y + sum[v][1] : old[v].y,
                                                          at + 2 < len ? old[v].z + sum[v][2] : old[v].z,
                                                          at + 3 < len ? old[v].w + sum[v][3] : old[v].w);
    }
  }
}

// Whether the blocks of <2, 2> are too few to hide the latency of a read, and the
// queries many: <1, 8> then. Device time of the kernel with <2, 2> and <1, 8>: 18
// blocks, 88 queries 24.1 and 9.8 us; 256 blocks, 8 queries 3.8 and 2.5; 864 blocks,
// 22 queries 10.7 and 13.0; 472 blocks, 4 queries 4.4 and 5.6. The blocks are
// counted by the capacity; those past a sequence's length end at once.
inline bool kvw_few(long long rows, int capacity, int cols) {
  return cols >= 8 && rows * ((capacity + KVW_THREADS * 8 - 1) / (KVW_THREADS * 8)) <= KVA_MAX_SMS * 4;
}

}  // namespace bpt
