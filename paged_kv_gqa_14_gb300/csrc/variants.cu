// Paged attention with a bucketed position bias, and differential attention: one kernel that is right for every
// call, a CTA to a (sequence, output head), its warps over the keys in turn, fp32 throughout.
#include "common.cuh"
#include "internal.h"
#include "variants.cuh"

namespace pkv {
namespace {

struct RowsParams {
  const bf16* q;
  int64_t q_st, q_sh;
  const bf16* k_cache;
  const bf16* v_cache;
  int64_t num_blocks;
  int bs_log2;
  const int32_t* block_tables;
  int64_t bt_stride, max_ctx;
  const int32_t* context_lens;
  const int32_t* qsl;
  bf16* out;
  int64_t o_st, o_sh, num_tokens;
  int hkv, group, num_seqs;
  float qscale;
  unsigned int* err;
  BiasArgs bias;
  DiffArgs diff;
};

constexpr int kRowWarps = 8;

template <int D, int V>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int PER = D / 32;            // dims of a head to a lane
  constexpr int MAPS = V == kDiff ? 2 : 1;
  constexpr int W = MAPS * PER;          // output numbers of a lane
  __shared__ float s_m[kRowWarps][MAPS], s_l[kRowWarps][MAPS], s_o[kRowWarps][MAPS][32 * W];
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x, head = blockIdx.y;
  for (int x = 0; x < b; ++x)
    if (p.qsl[x + 1] < p.qsl[x]) return;  // (flagged by that sequence's CTAs)
  const int s0 = p.qsl[b], s1 = p.qsl[b + 1], n = s1 - s0, ctx = p.context_lens[b];
  if (n <= 0 || s0 < 0 || s1 > p.num_tokens || ctx < n || ctx > p.max_ctx) {
    if (threadIdx.x == 0 && (n < 0 || s0 < 0 || s1 > p.num_tokens || (n > 0 && ctx < n))) raise_error(p.err, PKV_DEVERR_SPAN);
    else if (threadIdx.x == 0 && n > 0) raise_error(p.err, PKV_DEVERR_CONTEXT);
    return;
  }
  const int g = head / p.group;
  for (int row = 0; row < n; ++row) {
    const int pos = ctx - n + row;
    float q[MAPS][PER], acc[MAPS][W], m[MAPS], l[MAPS];
    for (int c = 0; c < MAPS; ++c) {
      const bf16* src = p.q + static_cast<int64_t>(s0 + row) * p.q_st + static_cast<int64_t>(MAPS * head + c) * p.q_sh;
      for (int x = 0; x < PER; ++x) q[c][x] = __bfloat162float(src[lane * PER + x]);
      for (int x = 0; x < W; ++x) acc[c][x] = 0.f;
      m[c] = NEG_INF;
      l[c] = 0.f;
    }
    for (int j = warp; j <= pos; j += kRowWarps) {
      int blk = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + (j >> p.bs_log2)];
      if (blk < 0 || blk >= p.num_blocks) {
        raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
        blk = 0;
      }
      const int64_t at = (((static_cast<int64_t>(blk) << p.bs_log2) + (j & ((1 << p.bs_log2) - 1))) * p.hkv + MAPS * g) * D;
      float v[W];
      for (int c = 0; c < MAPS; ++c)
        for (int x = 0; x < PER; ++x) v[c * PER + x] = __bfloat162float(p.v_cache[at + c * D + lane * PER + x]);
      for (int c = 0; c < MAPS; ++c) {
        float s = 0.f;
        for (int x = 0; x < PER; ++x) s = fmaf(q[c][x], __bfloat162float(p.k_cache[at + c * D + lane * PER + x]), s);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.qscale;
        if (V == kBias) {
          int i = 0;
          while (i + 1 < p.bias.num_buckets && p.bias.starts[i + 1] <= pos - j) ++i;
          s += bias_at(p.bias, i, head);
        }
        const float mn = fmaxf(m[c], s);
        if (mn == NEG_INF && s == NEG_INF) continue;
        const float f = exp2f(m[c] - mn), w = exp2f(s - mn);
        m[c] = mn;
        l[c] = l[c] * f + w;
        for (int x = 0; x < W; ++x) acc[c][x] = acc[c][x] * f + w * v[x];
      }
    }
    for (int c = 0; c < MAPS; ++c) {
      if (lane == 0) s_m[warp][c] = m[c], s_l[warp][c] = l[c];
      for (int x = 0; x < W; ++x) s_o[warp][c][lane * W + x] = acc[c][x];
    }
    __syncthreads();
    if (warp == 0) {
      float x[W];
      for (int c = 0; c < MAPS; ++c) {
        float M = NEG_INF, den = 0.f, num[W] = {};
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, s_m[w][c]);
        for (int w = 0; w < kRowWarps && M != NEG_INF; ++w) {
          const float f = exp2f(s_m[w][c] - M);
          den += f * s_l[w][c];
          for (int y = 0; y < W; ++y) num[y] += f * s_o[w][c][lane * W + y];
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        float f = inv;
        if (c == 1) f *= p.diff.lambda[static_cast<int64_t>(s0 + row) * p.diff.lambda_st + head];
        for (int y = 0; y < W; ++y) x[y] = c == 0 ? num[y] * f : x[y] - num[y] * f;
      }
      bf16* dst = p.out + static_cast<int64_t>(s0 + row) * p.o_st + static_cast<int64_t>(head) * p.o_sh;
      if (V == kDiff) {
        float f = p.diff.out_scale;
        if (p.diff.norm_weight) {
          float ss = 0.f;
          for (int y = 0; y < W; ++y) ss = fmaf(x[y], x[y], ss);
          for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          f *= 1.f / sqrtf(ss / (2 * D) + p.diff.norm_eps);
        }
        for (int y = 0; y < W; ++y) {
          const int d = (y / PER) * D + lane * PER + y % PER;
          dst[d] = __float2bfloat16(x[y] * f * (p.diff.norm_weight ? p.diff.norm_weight[d] : 1.f));
        }
      } else {
        for (int y = 0; y < W; ++y) dst[lane * PER + y] = __float2bfloat16(x[y]);
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_variant_rows(const AttnArgs& a, cudaStream_t stream) {
  RowsParams p{};
  p.q = static_cast<const bf16*>(a.q);
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.k_cache = static_cast<const bf16*>(a.k_cache);
  p.v_cache = static_cast<const bf16*>(a.v_cache);
  p.num_blocks = a.num_blocks;
  p.bs_log2 = a.bs_log2;
  p.block_tables = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.max_ctx = max_context(a.max_blocks, a.bs_log2);
  p.context_lens = a.context_lens;
  p.qsl = a.qsl;
  p.out = static_cast<bf16*>(a.out);
  p.o_st = a.o_st;
  p.o_sh = a.o_sh;
  p.num_tokens = a.num_tokens;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.num_seqs = static_cast<int>(a.num_seqs);
  p.qscale = a.scale * 1.4426950408889634f;
  p.err = a.err;
  if (a.bias) p.bias = *a.bias;
  if (a.diff) p.diff = *a.diff;
  const dim3 grid(static_cast<unsigned>(a.num_seqs), static_cast<unsigned>(a.variant == kDiff ? a.hq / 2 : a.hq));
  const auto kernel = a.variant == kDiff ? (a.head_dim == 128 ? rows_kernel<128, kDiff> : rows_kernel<64, kDiff>)
                                         : (a.head_dim == 128 ? rows_kernel<128, kBias> : rows_kernel<64, kBias>);
  return launch_kernel(false, kernel, grid, dim3(kRowWarps * 32), 0, stream, p);
}

}  // namespace pkv
