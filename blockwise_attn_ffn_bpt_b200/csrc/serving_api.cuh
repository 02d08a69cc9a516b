// Entry points of rotary positions and of the 4-bit key/value cache: argument
// checks and launches. Included by bpt_api.cu, whose checks, status words and
// launch log they share.
#pragma once

#include "kv4_attention.cuh"
#include "kv4_cache.cuh"
#include "kv4_evict.cuh"
#include "rotary.cuh"

namespace bpt {
namespace {

// Token rows of one tensor: row (beta, t) at p + beta * bs + t * ld bytes,
// `width` bytes long.
struct TokenRows {
  const void* p;
  int b, s;
  long long bs, ld;
  size_t width;
  size_t extent() const { return (size_t)((b - 1) * bs + (s - 1) * ld) + width; }
  Range range() const { return rng(p, extent()); }
};

// Strides that keep every byte of the tensor within 2^62 of its start.
bool strides_ok(const TokenRows& r) {
  const long long most = 1LL << 62;
  if (r.bs < 0 || r.ld < 0) return false;
  if (r.b > 1 && r.bs > most / r.b) return false;
  if (r.s > 1 && r.ld > most / r.s) return false;
  return r.b * r.bs + r.s * r.ld <= most;
}

// Whether no two rows of one tensor share a byte (required of outputs).
bool rows_distinct(const TokenRows& r) {
  const long long w = (long long)r.width;
  if (r.s > 1 && r.ld < w) return false;
  if (r.b > 1 && r.bs < w) return false;
  if (r.s == 1 || r.b == 1) return true;
  return r.bs >= (r.s - 1) * r.ld + w || r.ld >= (r.b - 1) * r.bs + w;
}

// Whether two tensors may share a byte. Rows of one buffer side by side (q, k
// and v of a fused projection) have the same strides and do not.
bool rows_overlap(const TokenRows& x, const TokenRows& y) {
  if (!overlap(x.range(), y.range())) return false;
  if (x.b != y.b || x.s != y.s || (x.b > 1 && x.bs != y.bs) || (x.s > 1 && x.ld != y.ld)) return true;
  long long period = 0;  // every row of both starts at a multiple of it from the first one
  if (x.b == 1)
    period = x.s == 1 ? 0 : x.ld;
  else if (x.s == 1)
    period = x.bs;
  else if (x.ld > 0 && x.bs % x.ld == 0)
    period = x.ld;
  else if (x.bs > 0 && x.ld % x.bs == 0)
    period = x.bs;
  if (period <= 0) return true;
  const long long d = (long long)((reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p)));
  const long long at = ((d % period) + period) % period;
  return !(at >= (long long)x.width && at + (long long)y.width <= period);
}

bool same_rows(const TokenRows& x, const TokenRows& y) {
  return x.p == y.p && (x.b == 1 || x.bs == y.bs) && (x.s == 1 || x.ld == y.ld);
}

bool aligned(const TokenRows& r, long long a) {
  return reinterpret_cast<uintptr_t>(r.p) % a == 0 && (r.b == 1 || r.bs % a == 0) && (r.s == 1 || r.ld % a == 0);
}

int check_dh(int dh) { return dh == 64 || dh == 128 ? BPT_OK : BPT_ERR_SHAPE; }

size_t kv4_bytes(int b, int kv_heads, int capacity, int dh) {
  return (size_t)b * kv_heads * (capacity / KV4_BLOCK) * (dh == 128 ? Kv4<128>::BYTES : Kv4<64>::BYTES);
}

// b sequences of n new tokens (n = 0 where there are none) on a cache
int check_kv4(int b, int n, int kv_heads, int capacity, int dh) {
  const long long most = 0x7fffffffLL;
  if (b < 0 || n < 0 || kv_heads <= 0 || capacity <= 0 || capacity % KV4_BLOCK) return BPT_ERR_SHAPE;
  BPT_TRY(check_dh(dh));
  if ((long long)b * kv_heads > most || (long long)b * n > most) return BPT_ERR_SHAPE;
  if ((long long)n * kv_heads > most / (dh / 8)) return BPT_ERR_SHAPE;
  if ((double)b * kv_heads * capacity * dh > 4e18) return BPT_ERR_SHAPE;
  return BPT_OK;
}

// Launches a kernel, in clusters of `cl` blocks where cl > 1, that may start
// before the one ahead of it on the stream has ended: it waits for that itself
// (grid_dependency_wait), with its launch behind it. What follows it may start
// so too, whatever it is, because every kernel launched here waits in all its
// blocks: its end is also the end of all before it.
template <typename Args>
int launch_kernel(void (*kernel)(const Args), const Args& args, dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                  int cl = 1) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess) return BPT_OK;
  cudaGetLastError();
  return BPT_ERR_CUDA;
}

unsigned grid_y(long long rows) { return (unsigned)std::min<long long>(rows, 65535); }

template <typename T, int W>
int launch_rotary(const RotaryArgs& a, bool interleaved, dim3 grid, cudaStream_t st) {
  return launch_kernel(interleaved ? rotary_kernel<T, W, true> : rotary_kernel<T, W, false>, a, grid, ROT_THREADS, 0, st);
}

struct Kv4AttnLayout {
  size_t lse = 0, ml = 0, o = 0, scores = 0, total = 0;
  int cols = 0, cols_block = 0, passes = 0, warps = 0, max_warps = 0;
  long long segments = 0;
  bool direct = false;
};

Kv4AttnLayout kv4_attn_layout(int b, int n, int heads, int kv_heads, int capacity, int dh, bool weights) {
  Kv4AttnLayout l;
  l.cols = heads / kv_heads * n;
  const int pass = 8 * kva_col_blocks(l.cols);  // more queries take further passes over the head's tokens
  l.cols_block = std::min(l.cols, pass);
  l.passes = (l.cols + pass - 1) / pass;
  l.segments = (long long)b * kv_heads * l.passes;
  l.warps = kva_warps(dh, pass / 8);
  l.direct = kva_direct(l.segments, capacity / KV4_BLOCK, l.warps);
  l.max_warps = (int)std::min<long long>(l.segments * (capacity / KV4_BLOCK), (long long)KVA_MAX_SMS * l.warps);
  size_t at = 0;
  auto take = [&](size_t& to, size_t bytes) {
    to = at;
    at += align_up(bytes, 256);
  };
  if (!l.direct) {
    const size_t slots = (size_t)l.segments + l.max_warps;
    take(l.ml, slots * l.cols_block * 8);
    take(l.o, slots * l.cols_block * dh * 4);
  }
  if (weights) {
    take(l.lse, (size_t)b * heads * n * 4);
    take(l.scores, (size_t)b * heads * n * capacity * 4);
  }
  l.total = at;
  return l;
}

int check_kv4_attention(int b, int n, int heads, int kv_heads, int capacity, int dh) {
  BPT_TRY(check_kv4(b, n, kv_heads, capacity, dh));
  if (heads <= 0 || heads % kv_heads) return BPT_ERR_SHAPE;
  if ((long long)b * n * heads > 0x7fffffffLL) return BPT_ERR_SHAPE;
  if ((double)b * n * heads * capacity > 1e18) return BPT_ERR_SHAPE;
  const int cols = heads / kv_heads * n, pass = 8 * kva_col_blocks(cols);
  if ((double)b * kv_heads * ((cols + pass - 1) / pass) * (capacity / KV4_BLOCK + KVA_SWITCH) > 2147483647.0)
    return BPT_ERR_SHAPE;
  return BPT_OK;
}

}  // namespace
}  // namespace bpt

extern "C" {

int bpt_rotary_frequencies(int rot, double base, int scaling, double factor, int original, double low_turns,
                           double high_turns, double* inv_freq, float* magnitude) {
  if (rot < 2 || rot > 2 * ROT_MAX_PAIRS || rot % 2) return BPT_ERR_SHAPE;
  if (!(base > 0.0) || !std::isfinite(base)) return BPT_ERR_SHAPE;
  if (scaling < BPT_ROTARY_PLAIN || scaling > BPT_ROTARY_RAMP) return BPT_ERR_SHAPE;
  if (!(factor >= 1.0) || !std::isfinite(factor)) return BPT_ERR_SHAPE;
  if (scaling == BPT_ROTARY_BASE && rot == 2) return BPT_ERR_SHAPE;
  if (scaling == BPT_ROTARY_RAMP && (original <= 0 || !(low_turns < high_turns))) return BPT_ERR_SHAPE;
  if (!inv_freq || !magnitude) return BPT_ERR_NULL;
  constexpr double two_pi = 6.283185307179586476925286766559;
  if (scaling == BPT_ROTARY_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
  *magnitude = 1.0f;
  if (scaling == BPT_ROTARY_RAMP) *magnitude = (float)(0.1 * std::log(factor) + 1.0);
  for (int j = 0; j < rot / 2; ++j) {
    const double f = std::pow(base, -2.0 * j / rot);
    double keep = 1.0;  // the share of f that is not divided by the factor
    if (scaling == BPT_ROTARY_LINEAR) keep = 0.0;
    if (scaling == BPT_ROTARY_RAMP)
      keep = std::min(1.0, std::max(0.0, (original * f / two_pi - low_turns) / (high_turns - low_turns)));
    inv_freq[j] = f * (keep + (1.0 - keep) / factor);
  }
  return BPT_OK;
}

int bpt_rotary(int dtype, const void* q, long long bs_q, long long ld_q, const void* k, long long bs_k,
               long long ld_k, int b, int s, int heads, int kv_heads, int dh, int rot, int interleaved,
               const double* inv_freq, float magnitude, const void* positions, int position_bytes,
               long long position_stride, long long offset, int inverse, void* q_out, long long bs_qo,
               long long ld_qo, void* k_out, long long bs_ko, long long ld_ko, void* stream) {
  if (dtype != BPT_DTYPE_BF16 && dtype != BPT_DTYPE_F32) return BPT_ERR_DTYPE;
  if (positions && position_bytes != 4 && position_bytes != 8) return BPT_ERR_DTYPE;
  if (b < 0 || s < 0 || heads <= 0 || kv_heads < 0) return BPT_ERR_SHAPE;
  BPT_TRY(check_dh(dh));
  if (rot < 2 || rot > dh || rot % 2) return BPT_ERR_SHAPE;
  if ((long long)b * s > 0x7fffffffLL || ((long long)heads + kv_heads) * dh > 0x7fffffffLL / 64) return BPT_ERR_SHAPE;
  if (position_stride < 0) return BPT_ERR_SHAPE;
  if ((long long)b * s == 0) return BPT_OK;
  const bool keys = kv_heads > 0;
  if (!q || !q_out || !inv_freq || (keys && (!k || !k_out))) return BPT_ERR_NULL;
  const int es = dtype == BPT_DTYPE_F32 ? 4 : 2;
  TokenRows in[2] = {{q, b, s, bs_q * es, ld_q * es, (size_t)heads * dh * es},
                     {k, b, s, bs_k * es, ld_k * es, (size_t)kv_heads * dh * es}};
  TokenRows out[2] = {{q_out, b, s, bs_qo * es, ld_qo * es, (size_t)heads * dh * es},
                      {k_out, b, s, bs_ko * es, ld_ko * es, (size_t)kv_heads * dh * es}};
  const int nt = keys ? 2 : 1;
  const TokenRows pos{positions, b, s, position_stride * position_bytes, position_bytes, (size_t)position_bytes};
  if (positions && (!strides_ok(pos) || reinterpret_cast<uintptr_t>(positions) % position_bytes))
    return strides_ok(pos) ? BPT_ERR_ALIGN : BPT_ERR_SHAPE;
  int w = 16 / es;  // elements of a vector: 16 bytes, or fewer as the rows are aligned
  bool in_place[2] = {false, false};
  for (int i = 0; i < nt; ++i) {
    if (!strides_ok(in[i]) || !strides_ok(out[i]) || !rows_distinct(out[i])) return BPT_ERR_SHAPE;
    if (!aligned(in[i], es) || !aligned(out[i], es)) return BPT_ERR_ALIGN;
    while (w > 1 && !(aligned(in[i], w * es) && aligned(out[i], w * es))) w /= 2;
    in_place[i] = same_rows(in[i], out[i]);
  }
  for (int i = 0; i < nt; ++i) {
    for (int j = 0; j < nt; ++j)
      if (!(i == j && in_place[i]) && rows_overlap(out[i], in[j])) return BPT_ERR_ALIAS;
    if (positions && overlap(out[i].range(), pos.range())) return BPT_ERR_ALIAS;
  }
  if (keys && rows_overlap(out[0], out[1])) return BPT_ERR_ALIAS;

  // the turned part of a head is whole vectors of its pairs' halves
  while ((rot / 2) % w) w /= 2;
  RotaryArgs a{};
  for (int i = 0; i < nt; ++i)
    a.t[i] = {in[i].p, const_cast<void*>(out[i].p), in[i].bs / es, in[i].ld / es, out[i].bs / es, out[i].ld / es};
  a.heads0 = heads;
  a.heads1 = kv_heads;
  a.in_place0 = in_place[0];
  a.in_place1 = in_place[1];
  a.tokens = b * s;
  a.s = s;
  a.dh = dh;
  a.rot = rot;
  a.units = (heads + kv_heads) * (dh / (2 * w));
  while ((1 << a.head_shift) < dh / (2 * w)) ++a.head_shift;
  // tokens of a block: up to what its table of angles holds, as many as give every
  // thread a unit, and more as long as that leaves a few rounds of blocks for every
  // SM (5490 tokens of 4 heads of 64 in fp32, 32 units each, took 13.4 us with a
  // token a block, 5.8 with 8); a token of very many heads is shared by several blocks
  a.chunk = std::min(a.units, ROT_CHUNK);
  const long long blocks = (long long)KVA_MAX_SMS * ROT_BLOCKS * ROT_ROUNDS;
  a.tile = (int)std::max<long long>(1, std::min<long long>(ROT_TABLE / (rot / 2), std::max<long long>(ROT_THREADS / a.units, a.tokens / blocks)));
  a.positions = positions;
  a.pos64 = position_bytes == 8;
  a.pos_stride = position_stride;
  a.offset = offset;
  a.magnitude = magnitude;
  a.sine = inverse ? -magnitude : magnitude;
  for (int j = 0; j < rot / 2; ++j) a.turns[j] = inv_freq[j] / 6.283185307179586476925286766559;
  int sms = 0;
  BPT_TRY(check_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(((long long)a.tokens + a.tile - 1) / a.tile), (a.units + a.chunk - 1) / a.chunk);
  LaunchScope ls("rotary", st);
  if (es == 4)
    return w == 4   ? launch_rotary<float, 4>(a, interleaved, grid, st)
           : w == 2 ? launch_rotary<float, 2>(a, interleaved, grid, st)
                    : launch_rotary<float, 1>(a, interleaved, grid, st);
  return w == 8   ? launch_rotary<__nv_bfloat16, 8>(a, interleaved, grid, st)
         : w == 4 ? launch_rotary<__nv_bfloat16, 4>(a, interleaved, grid, st)
         : w == 2 ? launch_rotary<__nv_bfloat16, 2>(a, interleaved, grid, st)
                  : launch_rotary<__nv_bfloat16, 1>(a, interleaved, grid, st);
}

size_t bpt_kv4_cache_bytes(int b, int kv_heads, int capacity, int dh) {
  if (check_kv4(b, 0, kv_heads, capacity, dh) != BPT_OK) return 0;
  return kv4_bytes(b, kv_heads, capacity, dh);
}

int bpt_kv4_store(void* cache, int b, int kv_heads, int capacity, int dh, const void* k, long long bs_k,
                  long long ld_k, const void* v, long long bs_v, long long ld_v, int n, const int* start,
                  const int* counts, void* stream) {
  BPT_TRY(check_kv4(b, n, kv_heads, capacity, dh));
  if (b == 0 || n == 0) return BPT_OK;
  if (!cache || !k || !v || !start) return BPT_ERR_NULL;
  const size_t width = (size_t)kv_heads * dh * 2;
  const TokenRows rk{k, b, n, bs_k * 2, ld_k * 2, width}, rv{v, b, n, bs_v * 2, ld_v * 2, width};
  if (!strides_ok(rk) || !strides_ok(rv)) return BPT_ERR_SHAPE;
  if (!aligned16(cache) || !aligned(rk, 16) || !aligned(rv, 16)) return BPT_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(counts)) & 3u) return BPT_ERR_ALIGN;
  const Range rc = rng(cache, kv4_bytes(b, kv_heads, capacity, dh));
  if (overlap(rc, rk.range()) || overlap(rc, rv.range()) || overlap(rc, rng(start, (size_t)b * 4)) ||
      (counts && overlap(rc, rng(counts, (size_t)b * 4))))
    return BPT_ERR_ALIAS;
  int sms = 0;
  BPT_TRY(check_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Kv4StoreArgs a{reinterpret_cast<uint8_t*>(cache), {b, kv_heads, capacity}};
  a.x[0] = reinterpret_cast<const __nv_bfloat16*>(k);
  a.x[1] = reinterpret_cast<const __nv_bfloat16*>(v);
  a.bs[0] = bs_k;
  a.bs[1] = bs_v;
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  a.n = n;
  a.start = start;
  a.counts = counts;
  BPT_TRY(stream_status_word(st, &a.status));
  const long long units = (long long)n * kv_heads * (dh / 16);
  const dim3 grid((unsigned)((units + KV4_THREADS - 1) / KV4_THREADS), grid_y(b));
  const bool wide = aligned(rk, 32) && aligned(rv, 32);  // 32-byte loads
  {
    LaunchScope ls("kv4_store", st);
    auto kernel = dh == 128 ? (wide ? kv4_store_kernel<128, true> : kv4_store_kernel<128, false>)
                            : (wide ? kv4_store_kernel<64, true> : kv4_store_kernel<64, false>);
    BPT_TRY(launch_kernel(kernel, a, grid, KV4_THREADS, 0, st));
  }
  return BPT_OK;
}

int bpt_kv4_load(const void* cache, int b, int kv_heads, int capacity, int dh, const int* start, const int* lens,
                 int n, void* k, void* v, void* stream) {
  BPT_TRY(check_kv4(b, n, kv_heads, capacity, dh));
  if (b == 0 || n == 0) return BPT_OK;
  if (!cache || !k || !v || !lens) return BPT_ERR_NULL;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v)) return BPT_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(lens)) & 3u) return BPT_ERR_ALIGN;
  const size_t act = (size_t)b * n * kv_heads * dh * 2;
  const Range outs[2] = {rng(k, act), rng(v, act)};
  const Range in[3] = {rng(cache, kv4_bytes(b, kv_heads, capacity, dh)), rng(lens, (size_t)b * 4),
                       rng(start, start ? (size_t)b * 4 : 0)};
  if (overlap(outs[0], outs[1])) return BPT_ERR_ALIAS;
  for (const Range& o : outs)
    for (const Range& r : in)
      if (overlap(o, r)) return BPT_ERR_ALIAS;
  int sms = 0;
  BPT_TRY(check_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Kv4LoadArgs a{reinterpret_cast<const uint8_t*>(cache), {b, kv_heads, capacity}};
  a.x[0] = reinterpret_cast<__nv_bfloat16*>(k);
  a.x[1] = reinterpret_cast<__nv_bfloat16*>(v);
  a.n = n;
  a.start = start;
  a.lens = lens;
  BPT_TRY(stream_status_word(st, &a.status));
  const long long units = (long long)n * kv_heads * (dh / 16);
  const dim3 grid((unsigned)((units + KV4_THREADS - 1) / KV4_THREADS), grid_y(b));
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;  // 32-byte stores
  {
    LaunchScope ls("kv4_load", st);
    auto kernel = dh == 128 ? (wide ? kv4_load_kernel<128, true> : kv4_load_kernel<128, false>)
                            : (wide ? kv4_load_kernel<64, true> : kv4_load_kernel<64, false>);
    BPT_TRY(launch_kernel(kernel, a, grid, KV4_THREADS, 0, st));
  }
  return BPT_OK;
}

size_t bpt_kv4_attention_workspace_bytes(int b, int n, int heads, int kv_heads, int capacity, int dh,
                                         int with_weights) {
  if (check_kv4_attention(b, n, heads, kv_heads, capacity, dh) != BPT_OK || b == 0 || n == 0) return 0;
  return kv4_attn_layout(b, n, heads, kv_heads, capacity, dh, with_weights != 0).total;
}

int bpt_kv4_attention(const void* q, long long bs_q, long long ld_q, const void* cache, const int* lens, int b,
                      int n, int heads, int kv_heads, int capacity, int dh, int causal, void* o, float* lse2,
                      float* weights, void* workspace, size_t ws_bytes, void* stream) {
  BPT_TRY(check_kv4_attention(b, n, heads, kv_heads, capacity, dh));
  if (b == 0 || n == 0) return BPT_OK;
  const Kv4AttnLayout L = kv4_attn_layout(b, n, heads, kv_heads, capacity, dh, weights != nullptr);
  if (!q || !cache || !lens || !o || (!workspace && L.total)) return BPT_ERR_NULL;
  const TokenRows rq{q, b, n, bs_q * 2, ld_q * 2, (size_t)heads * dh * 2};
  if (!strides_ok(rq)) return BPT_ERR_SHAPE;
  if (!aligned16(cache) || !aligned(rq, 16) || !aligned16(o) || !aligned16(lse2) || !aligned16(weights))
    return BPT_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return BPT_ERR_ALIGN;
  if (ws_bytes < L.total) return BPT_ERR_NOMEM;
  const size_t rows = (size_t)b * n * heads;
  const Range in[3] = {rq.range(), rng(cache, kv4_bytes(b, kv_heads, capacity, dh)), rng(lens, (size_t)b * 4)};
  const Range outs[4] = {rng(o, rows * dh * 2), rng(lse2, lse2 ? rows * 4 : 0),
                         rng(weights, weights ? (size_t)b * kv_heads * capacity * 4 : 0), rng(workspace, L.total)};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : in)
      if (overlap(outs[i], r)) return BPT_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return BPT_ERR_ALIAS;
  }
  int sms = 0;
  BPT_TRY(check_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  Kv4AttnArgs a{};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.bs_q = bs_q;
  a.ld_q = ld_q;
  a.cache = reinterpret_cast<const uint8_t*>(cache);
  a.d = {b, kv_heads, capacity};
  a.lens = lens;
  a.n = n;
  a.heads = heads;
  a.causal = causal != 0;
  a.score_scale = (float)(1.4426950408889634 / std::sqrt((double)dh));
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.lse2 = lse2 || !weights ? lse2 : reinterpret_cast<float*>(ws + L.lse);
  a.scores = weights ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  a.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  a.part_o = reinterpret_cast<float*>(ws + L.o);
  a.cols = L.cols;
  a.cols_block = L.cols_block;
  a.blocks_of_cols = L.passes;
  const int most = std::min(sms, KVA_MAX_SMS);
  a.max_warps = std::min(L.max_warps, most * L.warps);
  BPT_TRY(stream_status_word(st, &a.status));
  {
    LaunchScope ls("kv4_attention", st);
    const unsigned grid = L.direct ? (unsigned)L.segments : (unsigned)std::min(most, (a.max_warps + L.warps - 1) / L.warps);
    BPT_TRY(launch_kernel(kva_kernel(dh, L.cols, L.direct), a, grid, L.warps * 32, kva_smem(dh, L.cols), st));
  }
  if (!L.direct) {
    LaunchScope ls("kv4_join", st);
    const long long columns = (long long)b * kv_heads * L.cols;
    const int warps = kvj_warps(columns, L.segments, L.max_warps), threads = kvj_threads(warps);
    const long long runs = std::min<long long>((long long)b * ((kv_heads * L.cols + 7) / 8), KVA_MAX_SMS * 8);
    const dim3 grid = warps == 1 ? dim3((unsigned)runs) : dim3((unsigned)(kv_heads * L.cols), grid_y(b));
    BPT_TRY(launch_kernel(kvj_kernel(dh, warps), a, grid, threads, 0, st));
  }
  if (weights) {
    LaunchScope ls("kv4_weights", st);
    const Kv4WeightsArgs w{a.scores, a.lse2, weights, a.d, lens, n, heads, a.causal};
    const bool few = kvw_few((long long)b * kv_heads, capacity, L.cols);
    const int per = KVW_THREADS * 4 * (few ? 1 : 2);
    const dim3 grid((unsigned)((capacity + per - 1) / per), grid_y((long long)b * kv_heads));
    BPT_TRY(launch_kernel(few ? kv4_weights_kernel<1, 8> : kv4_weights_kernel<2, 2>, w, grid, KVW_THREADS, 0, st));
  }
  return BPT_OK;
}

int bpt_kv4_evict(const void* cache, const float* weights, const int* lens, int b, int kv_heads, int capacity,
                  int dh, int keep, int recent, void* cache_out, int capacity_out, float* weights_out, int* lens_out,
                  int* kept, void* stream) {
  BPT_TRY(check_kv4(b, 0, kv_heads, capacity, dh));
  BPT_TRY(check_kv4(b, 0, kv_heads, capacity_out, dh));
  if (keep <= 0 || keep > capacity_out || recent < 0 || recent > keep) return BPT_ERR_SHAPE;
  if (b == 0) return BPT_OK;
  if (!cache || !weights || !lens || !cache_out || !weights_out || !lens_out || !kept) return BPT_ERR_NULL;
  const void* wide[4] = {cache, cache_out, weights, weights_out};
  for (const void* p : wide)
    if (!aligned16(p)) return BPT_ERR_ALIGN;
  const void* ints[3] = {lens, lens_out, kept};
  for (const void* p : ints)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return BPT_ERR_ALIGN;
  const size_t rows = (size_t)b * kv_heads;
  const Range in[3] = {rng(cache, kv4_bytes(b, kv_heads, capacity, dh)), rng(weights, rows * capacity * 4),
                       rng(lens, (size_t)b * 4)};
  const Range outs[4] = {rng(cache_out, kv4_bytes(b, kv_heads, capacity_out, dh)),
                         rng(weights_out, rows * capacity_out * 4), rng(lens_out, (size_t)b * 4),
                         rng(kept, rows * keep * 4)};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : in)
      if (overlap(outs[i], r)) return BPT_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return BPT_ERR_ALIAS;
  }
  int sms = 0;
  BPT_TRY(check_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* status = nullptr;
  BPT_TRY(stream_status_word(st, &status));
  const Kv4Dims d{b, kv_heads, capacity}, d_out{b, kv_heads, capacity_out};
  {
    LaunchScope ls("kv4_select", st);
    const Kv4SelectArgs a{weights, d, lens, keep, recent, kept, lens_out, status};
    const int cl = evict_cluster((long long)rows, capacity);
    const size_t share = (size_t)(capacity / 4 + cl - 1) / cl * 4;  // tokens of a block
    const bool cached = share <= EVICT_CACHED;
    const int threads = evict_threads(cl, (long long)rows, capacity);
    BPT_TRY(launch_kernel(evict_kernel(cl, cached, threads), a, dim3((unsigned)rows * cl), threads, cached ? share * 4 : 0,
                          st, cl));
  }
  {
    LaunchScope ls("kv4_move", st);
    const Kv4MoveArgs a{reinterpret_cast<const uint8_t*>(cache), reinterpret_cast<uint8_t*>(cache_out), d, d_out,
                        weights, weights_out, kept, lens_out, keep};
    const int per = KV4_THREADS / (dh == 128 ? 8 : 4) * MOVE_ROWS;
    const dim3 grid((unsigned)((capacity_out + per - 1) / per), grid_y((long long)rows));
    BPT_TRY(launch_kernel(dh == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, a, grid, KV4_THREADS, 0, st));
  }
  return BPT_OK;
}

}  // extern "C"
