// Attention of new tokens over the 4-bit cache (kv4_cache.cuh).
//
// For a token's query q (one head) and the cached tokens u that it sees:
//     s_u = q . K_u / sqrt(dh),  o = sum_u 2^(c s_u - lse2) V_u,
//     lse2 = log2 sum_u 2^(c s_u),  c = log2 e,
// with a running maximum and sum over one pass of the cache; the weights of a
// cached token, summed over the queries that share its head, are added to
// weights[u] by a second kernel from the scores that the first one leaves.
#pragma once

#include "kv4_cache.cuh"

namespace bpt {

constexpr int KVA_THREADS = 256;

struct Kv4AttnArgs {
  const __nv_bfloat16* q;  // token (beta, t) at beta * bs + t * ld
  long long bs_q, ld_q;
  const uint8_t* cache;
  Kv4Dims d;
  const int* lens;         // [b], the new tokens among them
  int n, heads, causal;
  float score_scale;       // log2(e) / sqrt(dh)
  __nv_bfloat16* o;        // [b, n, heads * dh]
  float* lse2;             // [b, heads, n]
  float* scores;           // [b, kv_heads, group * n, capacity] in log2 units, or null
  int* status;
};

// Cached tokens that new token t of a sequence of `len` tokens sees.
__device__ __forceinline__ int kv4_seen(int len, int n, int t, int causal) {
  return causal ? max(len - n + 1 + t, 0) : len;
}

// One block a query: teams of dh/8 lanes take the cached tokens in turn, a lane
// 8 dimensions of each, and the teams' sums are joined at the end.
template <int DH>
__global__ void __launch_bounds__(KVA_THREADS) kv4_attention_kernel(const Kv4AttnArgs a) {
  constexpr int U = DH / 8, TEAMS = KVA_THREADS / U;
  using L = Kv4<DH>;
  __shared__ float s_o[TEAMS][DH], s_m[TEAMS], s_l[TEAMS];
  const int group = a.heads / a.d.kv_heads;
  const int u = threadIdx.x % U, team = threadIdx.x / U;
  const long long queries = (long long)a.d.b * a.n * a.heads;
  for (long long query = blockIdx.x; query < queries; query += gridDim.x) {
    const int head = query % a.heads;
    const long long tok = query / a.heads;
    const int beta = tok / a.n, t = tok - (long long)beta * a.n;
    const int kvh = head / group;
    const int len = clamp_count(a.lens[beta], a.d.capacity, a.status);
    const int seen = kv4_seen(len, a.n, t, a.causal);
    const uint4 raw = *reinterpret_cast<const uint4*>(a.q + beta * a.bs_q + t * a.ld_q + head * DH + u * 8);
    float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&raw)[i]);
      q[2 * i] = f.x;
      q[2 * i + 1] = f.y;
    }
    const uint8_t* base = a.cache + ((long long)beta * a.d.kv_heads + kvh) * a.d.blocks() * L::BYTES;
    float* scores = a.scores == nullptr
                        ? nullptr
                        : a.scores + (((long long)beta * a.d.kv_heads + kvh) * group * a.n +
                                      (t * group + head - kvh * group)) * a.d.capacity;
    const int rounds = (seen + TEAMS - 1) / TEAMS;
    for (int k = 0; k < rounds; ++k) {
      const int at = k * TEAMS + team;
      const bool live = at < seen;
      const int key = live ? at : 0, r = key % KV4_BLOCK;
      const uint8_t* block = base + (long long)(key / KV4_BLOCK) * L::BYTES;
      uint32_t wk = *reinterpret_cast<const uint32_t*>(block + r * L::ROW + kv4_k_place<DH>(u) * 4);
      const uint32_t wv = *reinterpret_cast<const uint32_t*>(block + L::V_CODES + r * L::ROW + kv4_v_place<DH>(u, r) * 4);
      const uint32_t pk = *reinterpret_cast<const uint32_t*>(block + L::K_PARAMS + r * L::PROW + u / 8 * 4);
      const uint32_t pv = *reinterpret_cast<const uint32_t*>(block + L::V_PARAMS + r * L::PROW + u / 8 * 4);
      wk = __funnelshift_r(wk, wk, 3);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dot = fmaf(q[i], fmaf((float)((wk >> (4 * i)) & 15u), __uint_as_float(pk << 16), __uint_as_float(pk & 0xffff0000u)), dot);
#pragma unroll
      for (int x = 1; x < U; x <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      const float s = dot * a.score_scale;
      if (!live) continue;
      if (scores != nullptr && u == 0) scores[key] = s;
      const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
      const float keep = ex2_approx(m - ref), p = ex2_approx(s - ref);
      m = top;
      l = fmaf(l, keep, p);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = fmaf(o[i], keep, p * fmaf((float)((wv >> (4 * i)) & 15u), __uint_as_float(pv << 16), __uint_as_float(pv & 0xffff0000u)));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) s_o[team][u * 8 + i] = o[i];
    if (u == 0) {
      s_m[team] = m;
      s_l[team] = l;
    }
    __syncthreads();
    if (threadIdx.x < DH) {
      float top = -INFINITY;
      for (int x = 0; x < TEAMS; ++x) top = fmaxf(top, s_m[x]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, out = 0.f;
      for (int x = 0; x < TEAMS; ++x) {
        const float w = ex2_approx(s_m[x] - ref);
        sum = fmaf(s_l[x], w, sum);
        out = fmaf(s_o[x][threadIdx.x], w, out);
      }
      const bool none = sum == 0.f;  // a row that sees no token is zero
      a.o[query * DH + threadIdx.x] = __float2bfloat16_rn(none ? 0.f : out / sum);
      if (threadIdx.x == 0) a.lse2[((long long)beta * a.heads + head) * a.n + t] = none ? -INFINITY : ref + log2f(sum);
    }
    __syncthreads();
  }
}

struct Kv4WeightsArgs {
  const float* scores;  // as Kv4AttnArgs
  const float* lse2;    // [b, heads, n]
  float* weights;       // [b, kv_heads, capacity]
  Kv4Dims d;
  const int* lens;
  int n, heads, causal;
};

// weights[u] += sum over the queries that share u's head of 2^(score - lse2).
__global__ void __launch_bounds__(KVA_THREADS) kv4_weights_kernel(const Kv4WeightsArgs a) {
  const int group = a.heads / a.d.kv_heads, cols = group * a.n;
  const int key = blockIdx.x * KVA_THREADS + threadIdx.x;
  const int rows = a.d.b * a.d.kv_heads;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int beta = row / a.d.kv_heads, kvh = row - beta * a.d.kv_heads;
    const int len = min(max(a.lens[beta], 0), a.d.capacity);
    if (key >= len) continue;
    const float* s = a.scores + (long long)row * cols * a.d.capacity + key;
    float sum = 0.f;
    for (int c = 0; c < cols; ++c) {
      const int t = c / group, head = kvh * group + c - t * group;
      if (key < kv4_seen(len, a.n, t, a.causal))
        sum += ex2_approx(s[(long long)c * a.d.capacity] - a.lse2[((long long)beta * a.heads + head) * a.n + t]);
    }
    a.weights[(long long)row * a.d.capacity + key] += sum;
  }
}

}  // namespace bpt
