// Decode split-K with a position bias, and of differential attention, over the bf16 cache.
//
// The work decomposition is the 8-bit decode's (decode_q8.cu): a unit is 8 page-heads of 16 tokens (16 at d 64), 32 KB
// of K and as much of V; every CTA finds its own units, each an equal share of all entries' units; an entry cut by
// CTA boundaries leaves one state (m, l, acc) for each piece, joined by a kernel after this one or, for the smallest
// batches, by the CTA that writes the last piece.  For a page and a kv head, a consumer warp computes
//   S^T [16 x 8] = K [16 x d] . Q^T [d x 8]          mma.sync m16n8k16, bf16 -> fp32
//   s = S scale log2(e) (+ bias),  p = 2^(s - m), m raised only when a score exceeds it, to 20 above (kVarSlack)
//   O^T [W x 8] += V^T [W x 16] . P^T [16 x 8]       p rounded to bf16, l the sum of what is multiplied
// kBias: W = d.  A page all of whose keys lie in the last bucket adds one number; in other pages each lane looks up the
// bucket of one key (while the page's copies are on their way).
// kDiff: the heads 2g and 2g + 1 of a pair are the k heads of its two maps, and both maps weigh both v heads: W = 2 d.
// A page is still read once: the pair's two warps read the same V from shared memory, which has the room.  What the rounding
// leaves of a weight is a second bf16, multiplied too: the difference takes out what the maps share and leaves their roundings (a
// warp's products are 2.5 times the plain decode's.  2000 keys, maps of correlation 0.99, lambda 1, with the norm: 0.0017 off in
// relative norm, which is the output's rounding, with one part 0.0105; 256 entries 180.6 us, with one part 177.7).  The
// states of both maps meet when a segment ends: x = o_0 - lambda o_1, the norm and the output are a warp's to a head, in fp32.
//
// Bound: DRAM.  GB300, of a copy's 6787 GB/s: kDiff 256 entries of up to 2048 keys, 16/8 heads d 128, 181 us (0.93), one of
// 131,053 keys, 32/8, 91 us (0.87, of which 10 us start, flush and merge); kBias 256 entries 168 us (0.97), 50 of 8192 keys,
// 28/4, 129 us (0.95).  Short batches are the launch, the plan and the joining of pieces: 4 entries of up to 100 keys 7.4 us
// a call, 32 of up to 1152 15.3.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "decode.cuh"
#include "decode_tc.cuh"
#include "variants.cuh"

namespace pkv {

bool make_pool_map_pages(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D, int pages);

namespace {

constexpr int kConsumers = kDecodeWarps * 32;
constexpr int kProducers = 4;  // warps
constexpr int kThreads = kConsumers + kProducers * 32;
constexpr int kWarpsAll = kThreads / 32;
// (kDiff has half as many output heads to share among the CTAs, each of twice the width and two maps)
template <int V>
constexpr int kMergeThreads = V == kDiff ? 1024 : 512;  // (131,053 keys, 32/8 heads: 512 threads 94 us, 1024 90.5)

// What the last steps of a row need.
struct RowEnd {
  bf16* out;
  int64_t o_st, o_sh;
  DiffArgs diff;
};

struct DecodeVarParams {
  CUtensorMap tmap_k;  // 5-D {64, 16 (8) rows, Hkv d / 64, pages of a block, num_blocks}, box {64, 16 (8), all, box_pages, 1}
  CUtensorMap tmap_v;
  DecodeParams p;
  int group;
  int self_plan, plan_early, num_seqs;
  int64_t num_tokens, max_ctx;
  int box_pages;  // pages of a block that one copy brings
  unsigned long long tag;  // this call's own, below 2^48, when the pieces are joined here; 0: by the merge kernel
  RowEnd end;
  BiasArgs bias;
};

template <int D>
struct DecodeVarCfg {
  static constexpr int PPW = 128 / D;                              // pages of a warp in a unit
  static constexpr int kPartBytes = kDecodeWarps * PPW * 16 * D * 2;  // K (or V) of a stage: 32 KB
  static constexpr int kStageBytes = 2 * kPartBytes;
  static constexpr int STAGES = 3;
  static constexpr int kBarBytes = 256 + 512;                      // barriers and flags, each warp's meta words
  static constexpr int kStartBytes = kMaxBuckets * 4;
  static constexpr int kMlBytes = kDecodeWarps * 8 * 8;
  static constexpr int xbuf_bytes(int g) {
    const int states = kDecodeWarps * g * D * 4, merge = kConsumers * 24 + 64;
    return states > merge ? states : merge;
  }
  static constexpr int smem_bytes(int g) {
    return 1024 + STAGES * kStageBytes + kBarBytes + kStartBytes + kMlBytes + xbuf_bytes(g);
  }
  static_assert(smem_bytes(8) <= 227 * 1024, "shared memory budget");
};

// Pages of block `blk` from its page `page` on, all heads: {dim, token, head and 64-dim half, page, block}.
__device__ __forceinline__ void tma_load_pages_bf16(void* dst_smem, const CUtensorMap* map, int page, int blk,
                                                    uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(page), "r"(blk), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Columns `q4` (four numbers of the 2 D or D of a row) of an output head, x their values before the norm; kDiff: f the
// factor of the norm and of out_scale.
template <int V>
__device__ __forceinline__ void write_cols4(const RowEnd& e, int64_t tq, int head, int d0, float4 x, float f) {
  if (V == kDiff) {
    if (e.diff.norm_weight) {
      const float4 w = *reinterpret_cast<const float4*>(e.diff.norm_weight + d0);
      x.x *= w.x, x.y *= w.y, x.z *= w.z, x.w *= w.w;
    }
    x.x *= f, x.y *= f, x.z *= f, x.w *= f;
  }
  uint2 o;
  o.x = pack_bf16x2(x.x, x.y);
  o.y = pack_bf16x2(x.z, x.w);
  *reinterpret_cast<uint2*>(e.out + tq * e.o_st + static_cast<int64_t>(head) * e.o_sh + d0) = o;
}
// The factor of a row of 2 D numbers whose squares sum to ss.
template <int D>
__device__ __forceinline__ float row_factor(const DiffArgs& d, float ss) {
  return d.norm_weight ? d.out_scale * (1.f / sqrtf(ss * (1.f / (2 * D)) + d.norm_eps)) : d.out_scale;
}

// The output heads [j0, j1) of an entry whose `n` pieces are in slots slot0 on: out = sum 2^(m - M) acc / sum 2^(m - M) l
// of each map, then the row's last steps.  Called by all NT threads; a column is four numbers of one map, its pieces
// shared by `lanes` threads where there are many.
template <int D, int V, int NT>
__device__ void merge_heads(const Plan& plan, const RowEnd& end, int hq, int group, int64_t slot0, int n, int64_t tq,
                            int j0, int j1, unsigned char* sm) {
  constexpr int MAPS = V == kDiff ? 2 : 1;
  constexpr int W4 = MAPS * D / 4;  // columns of a map
  constexpr int CQ = MAPS * W4;     // columns of an output head
  constexpr int kBatch = 4;
  const float NEG_INF = -__int_as_float(0x7f800000);
  float4* s_num = reinterpret_cast<float4*>(sm);             // [NT]
  float2* s_ml = reinterpret_cast<float2*>(sm + NT * 16);    // [NT]
  float* s_ss = reinterpret_cast<float*>(sm + NT * 24);      // [NT / 32]
  int lanes = 1;
  while (lanes * kBatch < n && lanes < NT / CQ) lanes <<= 1;
  const int heads = NT / (CQ * lanes);
  const int tid = threadIdx.x;
  const int col = tid % CQ, hp = tid / CQ % heads, pl = tid / (CQ * heads);
  const int c = col / W4, q = col % W4;
  for (int base = j0; base < j1; base += heads) {
    const int j = base + hp;
    const bool have = j < j1;
    const int e = V == kDiff ? (2 * (j / group) + c) * group + j % group : j;
    float M = NEG_INF, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = pl; have && k0 < n; k0 += kBatch * lanes) {
      float2 ml[kBatch];
      float4 a[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = make_float2(NEG_INF, 0.f);
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k * lanes < n) {
          const int64_t sh = (slot0 + k0 + k * lanes) * hq + e;
          ml[k] = __ldcg(reinterpret_cast<const float2*>(plan.part_ml + sh * 2));
          a[k] = __ldcg(reinterpret_cast<const float4*>(plan.part_acc + sh * (MAPS * D)) + q);
        }
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, ml[k].x);
      const float b = Mn == NEG_INF ? 0.f : Mn;
      const float f = fast_exp2(M - b);
      den *= f;
      num.x *= f, num.y *= f, num.z *= f, num.w *= f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = fast_exp2(ml[k].x - b);
        den = fmaf(w, ml[k].y, den);
        num.x = fmaf(w, a[k].x, num.x);
        num.y = fmaf(w, a[k].y, num.y);
        num.z = fmaf(w, a[k].z, num.z);
        num.w = fmaf(w, a[k].w, num.w);
      }
      M = Mn;
    }
    if (lanes > 1) {  // (heads * CQ threads to a set of columns, the sets behind one another)
      s_num[tid] = num;
      s_ml[tid] = make_float2(M, den);
      named_bar_sync(1, NT);
      if (pl == 0) {
        for (int k = 1; k < lanes; ++k) {
          const float2 ml = s_ml[tid + k * CQ * heads];
          const float4 o = s_num[tid + k * CQ * heads];
          const float Mn = fmaxf(M, ml.x), b = Mn == NEG_INF ? 0.f : Mn;
          const float w1 = fast_exp2(M - b), w2 = fast_exp2(ml.x - b);
          den = den * w1 + ml.y * w2;
          num.x = num.x * w1 + o.x * w2;
          num.y = num.y * w1 + o.y * w2;
          num.z = num.z * w1 + o.z * w2;
          num.w = num.w * w1 + o.w * w2;
          M = Mn;
        }
      }
    }
    const float inv = inverse_or_0(den);
    num.x *= inv, num.y *= inv, num.z *= inv, num.w *= inv;
    const bool mine = have && pl == 0 && c == 0;
    if (V == kDiff) {
      named_bar_sync(1, NT);  // (the sums above are read)
      if (pl == 0 && c == 1) s_num[tid] = num;
      named_bar_sync(1, NT);
      float4 x = num;
      if (mine) {
        const float la = end.diff.lambda[tq * end.diff.lambda_st + j];
        const float4 o = s_num[tid + W4];
        x.x -= la * o.x, x.y -= la * o.y, x.z -= la * o.z, x.w -= la * o.w;
      }
      float ss = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;  // (of c = 0: whole warps)
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if constexpr (W4 > 32) {
        if ((tid & 31) == 0) s_ss[tid >> 5] = ss;
        named_bar_sync(1, NT);
        ss = s_ss[(tid >> 5) & ~1] + s_ss[(tid >> 5) | 1];
      }
      if (mine) write_cols4<V>(end, tq, j, 4 * q, x, row_factor<D>(end.diff, ss));
    } else if (mine) {
      write_cols4<V>(end, tq, j, 4 * q, num, 1.f);
    }
    named_bar_sync(1, NT);  // shared memory is used again
  }
}

struct MergeParams {
  Plan plan;
  RowEnd end;
  int hq, group;
};

// The pieces of entries cut by CTA boundaries: CTA c - 1 looks at the boundary between decode CTAs c - 1 and c, and the
// n - 1 boundaries inside an entry of n pieces share its output heads.  The decode leaves for each of its CTAs
// {entry, its first unit, end unit, query row}, {W, 0, 0, 0}; entry -1 for a CTA without units.
template <int D, int V>
__global__ void __launch_bounds__(kMergeThreads<V>) merge_variant_kernel(const __grid_constant__ MergeParams p) {
  __shared__ __align__(16) unsigned char sm[kMergeThreads<V> * 24 + 128];
  pdl_wait();
  pdl_trigger();
  const int c = static_cast<int>(blockIdx.x) + 1;
  const int4 rec = p.plan.cta_rec[2 * c];
  const int W = p.plan.cta_rec[2 * c + 1].x;
  if (rec.x < 0 || rec.y >= c * W) return;  // (an entry starts at the boundary, or the units end before it)
  const int c0 = rec.y / W;                 // the entry's first CTA
  const int n = (rec.z - 1) / W - c0 + 1;
  const int heads = V == kDiff ? p.hq / 2 : p.hq;
  const int per = ceil_div(heads, n - 1);
  const int j0 = (c - 1 - c0) * per;
  if (j0 < heads)
    merge_heads<D, V, kMergeThreads<V>>(p.plan, p.end, p.hq, p.group, c0 + rec.x, n, rec.w, j0, min(heads, j0 + per), sm);
}

// A small batch's pieces are joined in the decode kernel itself: the CTA that writes the last of an entry's pieces
// joins them all; no thread waits for another CTA.  Nothing zeroes the workspace before, so a counter carries the call's
// tag: a word with another tag counts as none, and the last arrival leaves a word that no call's tag matches (a
// captured call keeps its tag in every replay).
__device__ __forceinline__ bool last_piece(unsigned long long* counter, unsigned long long tag, int of) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(counter);
  while (true) {
    const unsigned long long seen = (old >> 16) == tag ? old & 0xffffull : 0ull;
    const bool last = seen == static_cast<unsigned long long>(of - 1);
    const unsigned long long was = atomicCAS(counter, old, last ? 0ull : (tag << 16 | (seen + 1)));
    if (was == old) return last;
    old = was;
  }
}

// Sums of two counters over the block's threads before this one, and over all of them.
__device__ __forceinline__ int2 scan_pairs(int2 v, int2& total, int2* sm /* [kWarpsAll] */) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, off), b = __shfl_up_sync(0xffffffffu, x.y, off);
    if (lane >= off) {
      x.x += a;
      x.y += b;
    }
  }
  __syncthreads();  // (sm may still be read from before)
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  int2 before = make_int2(0, 0);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarpsAll; ++w) {
    const int2 t = sm[w];
    if (w < warp) before.x += t.x, before.y += t.y;
    total.x += t.x;
    total.y += t.y;
  }
  return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// TWO: 8-token blocks, a page of 16 tokens is two of them; else a page lies in one block.
template <int D, int V, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    decode_variant_kernel(const __grid_constant__ DecodeVarParams P) {
  using C = DecodeVarCfg<D>;
  constexpr int PPW = C::PPW;
  constexpr int STAGES = C::STAGES;
  constexpr int KS = D / 16;                   // k-steps of QK^T, m-tiles of P.V for one v head
  constexpr int HALVES = D / 64;               // 64-dim chunks of a head's row
  constexpr int NV = V == kDiff ? 2 : 1;       // v heads that a map weighs
  constexpr int PER = D / 32;                  // numbers of a lane where a warp holds a head's row
  const DecodeParams& p = P.p;
  const int G = P.group;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* stages = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes);
  uint64_t* empty = full + STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + STAGES);
  volatile int* last_flag = abort_flag + 2;
  int* warp_meta = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(full) + 256);
  int* starts = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(full) + C::kBarBytes);
  float2* xml = reinterpret_cast<float2*>(reinterpret_cast<unsigned char*>(starts) + C::kStartBytes);  // [warp][head]
  float* xbuf = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(xml) + C::kMlBytes);         // [warp][head][D]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kDecodeWarps);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kDecodeWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_v)) : "memory");
  }
  if (V == kBias)
    for (int i = threadIdx.x; i < P.bias.num_buckets; i += kThreads) starts[i] = P.bias.starts[i];
  const int hkv = p.hkv;
  const int wpp = kDecodeWarps / hkv;  // warps (pages at a time) to a kv head
  const int ppu = wpp * PPW;           // pages of a unit
  int4* first_rec = reinterpret_cast<int4*>(warp_meta + 64);  // [2]
  int mode = 0;  // 0: everything before this kernel has finished; 1, 2: streaming early, as in the plain decode
  int U, W, ubeg, uend;
  if (P.self_plan) {
    // Every CTA scans the batch and writes the entries that its own units touch.  An entry is a row: a sequence's one
    // new token, or each row of a longer span.
    if (!P.plan_early && !p.stream_early) pdl_wait();
    if (p.stream_early) pdl_trigger();
    int2* scan = reinterpret_cast<int2*>(warp_meta + 72);
    int s0 = 0, span = 0, ctx = 0, end_b = P.num_seqs;  // sequences from end_b on are skipped
    auto look = [&](int b) -> int2 {  // (entries, units) of sequence b
      int2 v = make_int2(0, 0);
      span = 0;
      int s1 = 0;
      s0 = 0;
      if (b < P.num_seqs) {
        s0 = p.qsl[b];
        s1 = p.qsl[b + 1];
        ctx = p.context_lens[b];
      }
      end_b = before_first_back(b, s0, s1, end_b, warp_meta + 120);
      if (b < end_b) {
        const int n = s1 - s0;
        if (s0 < 0 || s1 > P.num_tokens || (n > 0 && ctx < n)) {
          if (blockIdx.x == 0) raise_error(p.err, PKV_DEVERR_SPAN);
        } else if (n > 0 && ctx > P.max_ctx) {
          if (blockIdx.x == 0) raise_error(p.err, PKV_DEVERR_CONTEXT);
        } else {
          span = n;
          v.x = n;
          for (int r = 0; r < n; ++r) v.y += ceil_div(ceil_div(ctx - n + r + 1, kPageTokens), ppu);
        }
      } else if (b == end_b && b < P.num_seqs && blockIdx.x == 0) {
        raise_error(p.err, PKV_DEVERR_SPAN);
      }
      return v;
    };
    const int tid = static_cast<int>(threadIdx.x);
    int2 v = make_int2(0, 0), tot, ex = make_int2(0, 0);
    U = 0;
    for (int base = 0; base < P.num_seqs; base += kThreads) {
      v = look(base + tid);
      ex = scan_pairs(v, tot, scan);
      U += tot.y;
    }
    W = max(1, ceil_div(U, static_cast<int>(gridDim.x)));
    ubeg = static_cast<int>(blockIdx.x) * W;
    uend = min(U, ubeg + W);
    if (P.plan_early && !p.stream_early) pdl_wait();  // from here on the workspace is written
    if (!p.stream_early) pdl_trigger();
    if (ubeg < uend) {
      int2 carry = make_int2(0, 0);
      for (int base = 0; base < P.num_seqs; base += kThreads) {
        if (P.num_seqs > kThreads) {
          v = look(base + tid);
          ex = scan_pairs(v, tot, scan);
        }
        int unit = carry.y + ex.y;
        if (span > 0 && unit < uend && unit + v.y > ubeg) {
          for (int r = 0; r < span; ++r) {
            const int ctx_r = ctx - span + r + 1;
            const int end = unit + ceil_div(ceil_div(ctx_r, kPageTokens), ppu);
            if (unit < uend && end > ubeg) {
              const int i = carry.x + ex.x + r;
              p.plan.dec_seq[i] = base + tid;
              p.plan.dec_unit[i] = unit;
              p.plan.dec_unit[i + 1] = end;  // (the next entry's start: the same value from both)
              p.plan.dec_ctx[i] = ctx_r;
              p.plan.dec_tq[i] = s0 + r;
              if (unit <= ubeg) {
                first_rec[0] = make_int4(i, unit, end, base + tid);
                first_rec[1] = make_int4(ctx_r, s0 + r, 0, 0);
              }
            }
            unit = end;
          }
        }
        carry.x += tot.x;
        carry.y += tot.y;
      }
    }
    // (streaming early: an entry that is a row of a longer span has new keys before its last page)
    if (p.stream_early) mode = __syncthreads_or(span > 1 || P.num_seqs > kThreads) ? 2 : 1;
    __syncthreads();  // the records, and barrier initialisation
  } else {
    pdl_wait();
    pdl_trigger();
    U = p.plan.header[1];
    W = p.plan.header[2];
    ubeg = static_cast<int>(blockIdx.x) * W;
    uend = min(U, ubeg + W);
    if (threadIdx.x < 2) first_rec[threadIdx.x] = p.plan.cta_rec[2 * blockIdx.x + threadIdx.x];
    __syncthreads();  // the records, and barrier initialisation
  }
  // (meaningless, and unused, for a CTA without units)
  const int4 rec0 = first_rec[0], rec1 = first_rec[1];
  // (without the tag: for the merge kernel, over the start record)
  if (P.tag == 0 && threadIdx.x == 0) {
    p.plan.cta_rec[2 * blockIdx.x] = ubeg < uend ? make_int4(rec0.x, rec0.y, rec0.z, rec1.y) : make_int4(-1, 0, 0, 0);
    p.plan.cta_rec[2 * blockIdx.x + 1] = make_int4(W, 0, 0, 0);
  }
  if (ubeg >= uend) {  // CTA-uniform
    if (mode != 0) pdl_wait();  // (the grid ends after the work before it even if no CTA has units)
    return;
  }
  const int i_first = rec0.x;
  const int* dec_unit = p.plan.dec_unit;
  const uint32_t page_bytes = static_cast<uint32_t>(hkv * 16 * D * 2);
  // a stage: [K|V][page][8-row half (TWO)][kv head][64-dim half][16 (TWO: 8) rows][128 B]
  constexpr uint32_t kChunk = TWO ? 1024 : 2048;                    // a 64-dim half of a head
  constexpr uint32_t kHead = HALVES * kChunk;
  const uint32_t row8_off = TWO ? page_bytes / 2 : 1024u;           // rows 8..15

  if (warp >= kDecodeWarps) {
    // ------------------------------------------------------------------ producer warps
    if (p.fault_no_copies) return;
    const uint64_t pol = l2_policy_evict_first();
    // Each takes K or V of one half of a unit's pages, a lane to a page.
    const int kv = warp & 1, part = (warp - kDecodeWarps) >> 1;
    const int bp = (ppu * part >> 1) + lane;
    const bool lane_has_page = bp < ppu * (part + 1) >> 1;
    const bool lane_copies = (bp & (P.box_pages - 1)) == 0;
    const int blk_shift = TWO ? 0 : p.bs_log2 - 4;  // page gp lies in block gp >> blk_shift
    // A unit as this lane copies it, read one unit ahead, so that the latency of the block table is never between a
    // free stage and its copies.
    struct Unit {
      int blk, blk2, page0, bytes;
      bool page, half2, late;  // this lane copies blk, and blk2; the unit may hold what the kernel before writes
    };
    int i = i_first;
    int ustart = rec0.y, unext = rec0.z, ctx = rec1.x;
    const int32_t* table = p.block_tables + static_cast<int64_t>(rec0.w) * p.bt_stride;
    auto fetch = [&](int u) -> Unit {
      while (u >= unext) {
        ++i;
        ustart = unext;
        unext = dec_unit[i + 1];
        ctx = p.plan.dec_ctx[i];
        table = p.block_tables + static_cast<int64_t>(p.plan.dec_seq[i]) * p.bt_stride;
      }
      const int pg0 = (u - ustart) * ppu;
      const int npg = min(ppu, ceil_div(ctx, 16) - pg0);
      const int gp = pg0 + bp;
      Unit n;
      n.page = lane_has_page && bp < npg;
      n.half2 = TWO && n.page && gp * 16 + 8 < ctx;
      n.blk = n.blk2 = 0;
      if (n.page) n.blk = table[TWO ? 2 * gp : gp >> blk_shift];
      if (n.half2) n.blk2 = table[2 * gp + 1];
      n.page0 = TWO ? 0 : gp & ((1 << blk_shift) - 1);
      // (a last half page past the context is not loaded)
      const bool tail_half = TWO && (pg0 + npg - 1) * 16 + 8 >= ctx;
      // (a copy brings pages of its block past the context as well, which nobody reads)
      const int brought = (npg + P.box_pages - 1) & -P.box_pages;
      n.bytes = 2 * (brought * static_cast<int>(page_bytes) - (tail_half ? static_cast<int>(page_bytes) / 2 : 0));
      n.late = mode == 2 || pg0 + npg - 1 >= (ctx - 1) >> 4;
      return n;
    };
    int s = 0;
    uint32_t phase = 1;  // of empty[s]: a fresh barrier passes a wait for phase 1
    int u = ubeg;
    bool waited = mode == 0;
    Unit next = fetch(ubeg);
    for (; u < uend; ++u) {
      Unit cur = next;
      if (u + 1 < uend) next = fetch(u + 1);
      if (u - ubeg >= STAGES && !wait_or_abort(&empty[s], phase, p.err, abort_flag)) break;
      if (!waited && cur.late) {
        pdl_wait();
        waited = true;
      }
      if (warp == kDecodeWarps && lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(cur.bytes));
      __syncwarp();
      if (cur.page) {
        if (cur.blk < 0 || cur.blk >= p.num_blocks || cur.blk2 < 0 || cur.blk2 >= p.num_blocks) {
          raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);  // a bad id is read as block 0
          if (cur.blk < 0 || cur.blk >= p.num_blocks) cur.blk = 0;
          if (cur.blk2 < 0 || cur.blk2 >= p.num_blocks) cur.blk2 = 0;
        }
        unsigned char* dst = stages + s * C::kStageBytes + kv * C::kPartBytes + bp * page_bytes;
        const CUtensorMap* map = kv ? &P.tmap_v : &P.tmap_k;
        if (lane_copies) tma_load_pages_bf16(dst, map, cur.page0, cur.blk, &full[s], pol);
        if (TWO && cur.half2) tma_load_pages_bf16(dst + page_bytes / 2, map, 0, cur.blk2, &full[s], pol);
      }
      if (++s == STAGES) {
        s = 0;
        phase ^= 1;
      }
    }
    // every copy issued has landed before the CTA may leave (also after another warp has given up)
    const int issued = u - ubeg;
    for (int k = max(0, issued - STAGES); k < issued; ++k)
      mbar_wait(&full[k % STAGES], (k / STAGES) & 1, p.err);
    return;
  }

  // -------------------------------------------------------------------- consumer warps
  if (mode != 0) pdl_wait();  // q is written by the kernel before
  const int pw = warp / hkv;
  const int h = warp - pw * hkv;  // kv head
  const int gr = lane >> 2, tig = lane & 3;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const uint32_t stage_base = smem_u32(stages);
  const bool hv = gr < G;
  // q head of group member g of this warp's kv head
  auto q_head = [&](int g) { return V == kDiff ? 2 * ((h >> 1) * G + g) + (h & 1) : h * G + g; };
  uint32_t qb[KS][2];     // Q^T B fragments: head gr (zero past G), dims of k-step kk
  float acc[NV][KS][4];   // O^T: dims 16 mt + gr (+8) of v head, heads 2 tig (+1)
  float mref[2], lsum[2];
  float cfar[2] = {0.f, 0.f};  // (kBias) the last bucket's bias of heads 2 tig, 2 tig + 1
  int far = 0;                 // and its first distance
  if (V == kBias) {
    far = P.bias.starts[P.bias.num_buckets - 1];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * tig + j < G) cfar[j] = bias_at(P.bias, P.bias.num_buckets - 1, h * G + 2 * tig + j);
  }
  bool ok = true;
  int* meta = warp_meta + 4 * warp;  // the next entry, read from the plan while the segment runs
  auto load_q = [&](int64_t row_tq) {
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
        p.q + row_tq * p.q_st + static_cast<int64_t>(q_head(hv ? gr : 0)) * p.q_sh);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      qb[kk][0] = hv ? qrow[kk * 8 + tig] : 0u;
      qb[kk][1] = hv ? qrow[kk * 8 + 4 + tig] : 0u;
    }
  };
  // segments: the parts of consecutive entries that lie in this CTA's units [ubeg, uend)
  int s = 0;
  uint32_t phase = 0;
  int u = ubeg;
  int i = i_first, ustart = rec0.y, unext = rec0.z, ctx = rec1.x, tq = rec1.y;
  load_q(tq);
  while (true) {
    const int npages = ceil_div(ctx, 16);
    const int u1 = min(unext, uend);
    if (unext < uend && lane < 3) {  // the next entry
      const int* src = lane == 0 ? dec_unit + i + 2 : lane == 1 ? p.plan.dec_ctx + i + 1 : p.plan.dec_tq + i + 1;
      cp_async_word(smem_u32(meta + lane), src);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) acc[v][mt][0] = acc[v][mt][1] = acc[v][mt][2] = acc[v][mt][3] = 0.f;
    mref[0] = mref[1] = NEG_INF;
    lsum[0] = lsum[1] = 0.f;
    for (; u < u1; ++u) {
      // the biases of keys gr and gr + 8 of this warp's first page of the unit, for heads 2 tig and 2 tig + 1
      float bb[4];
      auto look_up = [&](int pg) {
        bb[0] = bb[2] = cfar[0];
        bb[1] = bb[3] = cfar[1];
        if (ctx - 1 - (pg * 16 + 15) < far) {  // (warp-uniform) some key is nearer than the last bucket
          const int at = bucket_of(starts, P.bias.num_buckets, max(ctx - 1 - (pg * 16 + (lane & 15)), 0));
          const int b0 = __shfl_sync(0xffffffffu, at, gr), b1 = __shfl_sync(0xffffffffu, at, gr + 8);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (2 * tig + j < G) {
              bb[j] = bias_at(P.bias, b0, h * G + 2 * tig + j);
              bb[2 + j] = bias_at(P.bias, b1, h * G + 2 * tig + j);
            }
        }
      };
      if (V == kBias) look_up((u - ustart) * ppu + pw);
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(&full[s], phase, p.err, abort_flag));
#pragma unroll
      for (int w = 0; w < PPW; ++w) {
        const int up = pw + w * wpp;  // page of the unit
        const int pg = (u - ustart) * ppu + up;
        if (V == kBias && w > 0) look_up(pg);
        if (!ok || pg >= npages) continue;
        const int rows = min(16, ctx - pg * 16);
        const uint32_t kbase = stage_base + s * C::kStageBytes + up * page_bytes + h * kHead;
        const uint32_t vbase = stage_base + s * C::kStageBytes + C::kPartBytes + up * page_bytes +
                               (V == kDiff ? h & ~1 : h) * kHead;
        if (rows < 16) {
          // keys past the context: zero their V rows so 0 * (unused slot) cannot poison P.V (of a pair's heads by both
          // of its warps, each before it reads them)
          unsigned char* vgen = stages + (vbase - stage_base);
          for (int idx = lane; idx < (16 - rows) * 8 * HALVES * NV; idx += 32) {
            const int ch = idx / ((16 - rows) * 8);
            const int r2 = idx - ch * (16 - rows) * 8;
            const int t = rows + (r2 >> 3);
            *reinterpret_cast<uint4*>(vgen + ch * kChunk + (t >> 3) * row8_off + (t & 7) * 128 + ((r2 & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        // S^T = K . Q^T, two chains
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        {
          const int r = (lane & 7) + 8 * ((lane >> 3) & 1);
          const uint32_t rsel = (r >> 3) * row8_off;
          const int csel = lane >> 4;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            uint32_t a[4];
            ldsm_x4_tc(a, kbase + (kk >> 2) * kChunk + rsel + chunk_off(r, 2 * (kk & 3) + csel));
            mma_16816(kk & 1 ? sb : sa, a, qb[kk][0], qb[kk][1]);
          }
        }
        // scores in the log2 domain, keys past the context masked by select
        const bool v0 = gr < rows, v1 = gr + 8 < rows;
        float sc[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float t = V == kBias ? fmaf(sa[x] + sb[x], p.qscale, bb[x]) : (sa[x] + sb[x]) * p.qscale;
          sc[x] = (x < 2 ? v0 : v1) ? t : NEG_INF;
        }
        float pm0 = fmaxf(sc[0], sc[2]), pm1 = fmaxf(sc[1], sc[3]);
        if (__any_sync(0xffffffffu, pm0 > mref[0] || pm1 > mref[1])) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            pm0 = fmaxf(pm0, __shfl_xor_sync(0xffffffffu, pm0, off));
            pm1 = fmaxf(pm1, __shfl_xor_sync(0xffffffffu, pm1, off));
          }
          const float mn0 = pm0 > mref[0] ? pm0 + kVarSlack : mref[0], mn1 = pm1 > mref[1] ? pm1 + kVarSlack : mref[1];
          const float c0 = mref[0] == mn0 ? 1.f : fast_exp2(mref[0] - mn0);
          const float c1 = mref[1] == mn1 ? 1.f : fast_exp2(mref[1] - mn1);
          mref[0] = mn0;
          mref[1] = mn1;
          lsum[0] *= c0;
          lsum[1] *= c1;
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              acc[v][mt][0] *= c0;
              acc[v][mt][1] *= c1;
              acc[v][mt][2] *= c0;
              acc[v][mt][3] *= c1;
            }
        }
        const float b0 = mref[0] == NEG_INF ? 0.f : mref[0], b1 = mref[1] == NEG_INF ? 0.f : mref[1];
        const float wt[4] = {fast_exp2(sc[0] - b0), fast_exp2(sc[1] - b1), fast_exp2(sc[2] - b0), fast_exp2(sc[3] - b1)};
        const uint32_t p0 = pack_bf16x2(wt[0], wt[1]), p1 = pack_bf16x2(wt[2], wt[3]);
        // (kDiff: what the rounding leaves of a weight is multiplied too)
        uint32_t r0 = 0, r1 = 0;
        if (V == kDiff) {
          r0 = pack_bf16x2(wt[0] - bf16lo(p0), wt[1] - bf16hi(p0));
          r1 = pack_bf16x2(wt[2] - bf16lo(p1), wt[3] - bf16hi(p1));
        }
        // (l sums what P.V weighs with, so that a row's weights add up to 1 whatever their rounding)
        lsum[0] += bf16lo(p0) + bf16lo(p1);
        lsum[1] += bf16hi(p0) + bf16hi(p1);
        if (V == kDiff) {
          lsum[0] += bf16lo(r0) + bf16lo(r1);
          lsum[1] += bf16hi(r0) + bf16hi(r1);
        }
        // P^T (tokens x heads) -> B fragments (k = token, n = head) by an 8x8 transpose
        const uint32_t pb0 = movmatrix_t(p0), pb1 = movmatrix_t(p1);
        const uint32_t rb0 = V == kDiff ? movmatrix_t(r0) : 0u, rb1 = V == kDiff ? movmatrix_t(r1) : 0u;
        // O^T += V^T . P^T
        {
          const int r = (lane & 7) + 8 * (lane >> 4);
          const uint32_t rsel = (r >> 3) * row8_off;
          const int csel = (lane >> 3) & 1;
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              uint32_t a[4];
              ldsm_x4_t_tc(a, vbase + v * kHead + (mt >> 2) * kChunk + rsel + chunk_off(r, 2 * (mt & 3) + csel));
              mma_16816(acc[v][mt], a, pb0, pb1);
              if (V == kDiff) mma_16816(acc[v][mt], a, rb0, rb1);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == STAGES) {
        s = 0;
        phase ^= 1;
      }
    }

    // ---------------------------------------------------------------- segment flush
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const bool more = unext < uend;
    const int nx_unext = meta[0], nx_ctx = meta[1], nx_tq = meta[2];  // (unused unless more)
    if (more) load_q(nx_tq);  // (arrives while the states are joined)
    float L0 = lsum[0], L1 = lsum[1];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      L0 += __shfl_xor_sync(0xffffffffu, L0, off);
      L1 += __shfl_xor_sync(0xffffffffu, L1, off);
    }
    // (a row of xbuf is xored with its head, so that the eight gr and four tig of a store use different banks)
    auto xsw = [](int g) { return ((g >> 1) & 3) << 3; };
    auto put = [&](int v) {
      float* xb = xbuf + warp * G * D;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int g = 2 * tig + j;
        if (g < G) {
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            xb[g * D + ((16 * mt + gr) ^ xsw(g))] = acc[v][mt][j];
            xb[g * D + ((16 * mt + gr + 8) ^ xsw(g))] = acc[v][mt][2 + j];
          }
          if (gr == 0 && v == 0) xml[warp * 8 + g] = make_float2(mref[j], j ? L1 : L0);
        }
      }
    };
    // this lane's PER numbers of kv head hh, member g, from the warps that hold its pages
    auto gather = [&](int hh, int g, float (&num)[PER], float& M, float& den) {
      M = NEG_INF;
      for (int k = 0; k < wpp; ++k) M = fmaxf(M, xml[(hh + k * hkv) * 8 + g].x);
      const float b = M == NEG_INF ? 0.f : M;
      den = 0.f;
#pragma unroll
      for (int x = 0; x < PER; ++x) num[x] = 0.f;
      for (int k = 0; k < wpp; ++k) {
        const float2 ml = xml[(hh + k * hkv) * 8 + g];
        const float w = fast_exp2(ml.x - b);  // a warp with no pages: m = -inf -> w = 0
        den = fmaf(w, ml.y, den);
        const float* row = xbuf + ((hh + k * hkv) * G + g) * D + ((PER * lane) ^ xsw(g));
#pragma unroll
        for (int x = 0; x < PER; x += 2) {
          const float2 o = *reinterpret_cast<const float2*>(row + x);
          num[x] = fmaf(w, o.x, num[x]);
          num[x + 1] = fmaf(w, o.y, num[x + 1]);
        }
      }
    };
    auto store_bf16 = [&](int64_t at, const float (&x)[PER]) {
      if constexpr (PER == 4) {
        uint2 o;
        o.x = pack_bf16x2(x[0], x[1]);
        o.y = pack_bf16x2(x[2], x[3]);
        *reinterpret_cast<uint2*>(P.end.out + at) = o;
      } else {
        *reinterpret_cast<uint32_t*>(P.end.out + at) = pack_bf16x2(x[0], x[1]);
      }
    };
    const bool whole = ustart >= ubeg && unext <= uend;  // the entry's every unit is this CTA's
    if (!whole) {
      // a piece's slot: CTA and entry grow together along the pieces, so their sum names each once
      const int64_t slot_h = static_cast<int64_t>(static_cast<int>(blockIdx.x) + i) * p.hq;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        put(v);
        named_bar_sync(1, kConsumers);
        for (int e = warp; e < p.hq; e += kDecodeWarps) {
          float num[PER], M, den;
          gather(e / G, e % G, num, M, den);
          float* dst = p.plan.part_acc + (slot_h + e) * (NV * D) + v * D + PER * lane;
#pragma unroll
          for (int x = 0; x < PER; x += 2) *reinterpret_cast<float2*>(dst + x) = make_float2(num[x], num[x + 1]);
          if (lane == 0 && v == 0) *reinterpret_cast<float2*>(p.plan.part_ml + (slot_h + e) * 2) = make_float2(M, den);
        }
        named_bar_sync(1, kConsumers);
      }
      if (P.tag) {
        const int c0 = ustart / W, chunks = (unext - 1) / W - c0 + 1;
        __threadfence();
        named_bar_sync(1, kConsumers);
        // (the counter is in the start record of CTA c0, which starts at most one entry of several pieces)
        if (threadIdx.x == 0)
          *last_flag = last_piece(reinterpret_cast<unsigned long long*>(p.plan.cta_rec + 2 * c0), P.tag, chunks);
        named_bar_sync(1, kConsumers);
        if (*last_flag) {
          __threadfence();
          merge_heads<D, V, kConsumers>(p.plan, P.end, p.hq, G, c0 + i, chunks, tq, 0, V == kDiff ? p.hq / 2 : p.hq,
                                        reinterpret_cast<unsigned char*>(xbuf));
        }
        named_bar_sync(1, kConsumers);
      }
    } else if (V == kBias) {
      put(0);
      named_bar_sync(1, kConsumers);
      for (int e = warp; e < p.hq; e += kDecodeWarps) {
        float num[PER], M, den;
        gather(e / G, e % G, num, M, den);
        const float inv = inverse_or_0(den);
#pragma unroll
        for (int x = 0; x < PER; ++x) num[x] *= inv;
        store_bf16(static_cast<int64_t>(tq) * P.end.o_st + static_cast<int64_t>(e) * P.end.o_sh + PER * lane, num);
      }
      named_bar_sync(1, kConsumers);
    } else {
      // a warp to an output head, which waits in registers for its second half of the columns
      constexpr int kRounds = 4;  // up to 32 output heads
      const int heads = p.hq / 2;
      float x[kRounds][NV][PER];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        put(v);
        named_bar_sync(1, kConsumers);
#pragma unroll
        for (int rd = 0; rd < kRounds; ++rd) {
          const int j = warp + rd * kDecodeWarps;
          if (j < heads) {
            float o[PER], M, den;
            gather(2 * (j / G), j % G, x[rd][v], M, den);
            const float inv0 = inverse_or_0(den);
            gather(2 * (j / G) + 1, j % G, o, M, den);
            const float f1 = inverse_or_0(den) * P.end.diff.lambda[static_cast<int64_t>(tq) * P.end.diff.lambda_st + j];
#pragma unroll
            for (int y = 0; y < PER; ++y) x[rd][v][y] = x[rd][v][y] * inv0 - o[y] * f1;
          }
        }
        named_bar_sync(1, kConsumers);
      }
#pragma unroll
      for (int rd = 0; rd < kRounds; ++rd) {
        const int j = warp + rd * kDecodeWarps;
        if (j < heads) {
          float ss = 0.f;
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int y = 0; y < PER; ++y) ss = fmaf(x[rd][v][y], x[rd][v][y], ss);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float f = row_factor<D>(P.end.diff, ss);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int d0 = v * D + PER * lane;
#pragma unroll
            for (int y = 0; y < PER; ++y)
              x[rd][v][y] *= P.end.diff.norm_weight ? f * P.end.diff.norm_weight[d0 + y] : f;
            store_bf16(static_cast<int64_t>(tq) * P.end.o_st + static_cast<int64_t>(j) * P.end.o_sh + d0, x[rd][v]);
          }
        }
      }
    }
    if (!more) break;
    ++i;
    ustart = unext;  // entries are consecutive: the next one starts where this one ends
    unext = nx_unext;
    ctx = nx_ctx;
    tq = nx_tq;
    __syncwarp();  // every lane has read meta
  }
}

// Tags of this process's calls: 48 bits, never 0, from a start that two runs seldom share (the words they
// are compared with are whatever the workspace held before).
unsigned long long new_tag() {
  static std::atomic<unsigned long long> count{
      static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0xD1B54A32D192ED03ull};
  unsigned long long t;
  do t = count.fetch_add(1) & 0xffffffffffffull;
  while (t == 0);
  return t;
}

template <int D, int V, bool TWO>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  using C = DecodeVarCfg<D>;
  // (the largest any group needs, so the limit is raised once)
  if (const cudaError_t e = set_smem_once<decode_variant_kernel<D, V, TWO>>(C::smem_bytes(8)); e != cudaSuccess) return e;
  DecodeVarParams P{};
  P.box_pages = TWO ? 1 : std::min(kDecodeWarps / a.hkv * C::PPW, 1 << (a.bs_log2 - 4));
  if (!make_pool_map_pages(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D, P.box_pages) ||
      !make_pool_map_pages(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D, P.box_pages))
    return cudaErrorInvalidValue;
  DecodeParams& p = P.p;
  p.q = static_cast<const bf16*>(a.q);
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.num_blocks = a.num_blocks;
  p.bs_log2 = a.bs_log2;
  p.block_tables = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.context_lens = a.context_lens;
  p.qsl = a.qsl;
  p.hkv = a.hkv;
  p.hq = a.hq;
  p.qscale = a.scale * kLog2e;
  p.plan = a.plan;
  p.err = a.err;
  p.fault_no_copies = a.fault == PKV_FAULT_DECODE_NO_COPIES;
  p.stream_early = a.stream_early && self_plan;
  P.group = a.hq / a.hkv;
  P.self_plan = self_plan ? 1 : 0;
  P.plan_early = a.plan_early;
  P.num_seqs = static_cast<int>(a.num_seqs);
  P.num_tokens = a.num_tokens;
  P.max_ctx = max_context(a.max_blocks, a.bs_log2);
  P.end.out = static_cast<bf16*>(a.out);
  P.end.o_st = a.o_st;
  P.end.o_sh = a.o_sh;
  if (a.diff) P.end.diff = *a.diff;
  if (a.bias) P.bias = *a.bias;
  // Pieces are joined by the kernel after this one or, where there is little to join, by the CTA that writes the last, which
  // saves a launch but has one CTA read it all.  GB300, replayed graph, in the kernel / after it: 4 sequences of up to 100
  // keys, 14/2 heads d 64, kDiff 12.8 / 16.9 us, kBias 12.8 / 14.8, 8/2 d 128 17.1 / 21.0 and 14.8 / 14.8, but 16/8 d 128
  // 25.2 / 17.1 and 18.9 / 14.8, 32/8 d 128 35.6 / 18.9 and 23.0 / 15.2; 64 of 64, 8/2 d 128, 14.8 / 17.5 and 12.8 / 13.7, 16/8
  // d 128 31.2 / 29.2 and 22.4 / 21.0; one of 4096, 14/2 d 64, 33.2 / 16.9 and 27.1 / 16.9.
  const int64_t units = ceil_div64(ceil_div64(P.max_ctx, kPageTokens), kDecodeWarps / a.hkv * C::PPW);
  const bool merge_here = self_plan && a.num_seqs * P.max_ctx <= (1 << 13) && units <= 8 && a.hq * D <= 1024;
  P.tag = merge_here ? new_tag() : 0;
  record_kernel_event(PKV_KERNEL_DECODE, false, stream);
  cudaError_t e = launch_pdl(decode_variant_kernel<D, V, TWO>, dim3(a.decode_ctas), dim3(kThreads), C::smem_bytes(P.group),
                             stream, P);
  if (e == cudaSuccess && !merge_here && a.decode_ctas > 1) {
    MergeParams M;
    M.plan = a.plan;
    M.end = P.end;
    M.hq = a.hq;
    M.group = P.group;
    // (beside prefill tiles not launched early: its CTAs, waiting for the decode, would take the SMs that
    // the prefill's are to run on)
    e = launch_kernel(self_plan, merge_variant_kernel<D, V>, dim3(a.decode_ctas - 1), dim3(kMergeThreads<V>), 0, stream, M);
  }
  record_kernel_event(PKV_KERNEL_DECODE, true, stream);
  return e;
}

template <int D, int V>
cudaError_t launch_bs(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  return a.bs_log2 == 3 ? launch<D, V, true>(a, stream, self_plan) : launch<D, V, false>(a, stream, self_plan);
}

}  // namespace

cudaError_t launch_decode_variant(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  if (a.variant == kBias)
    return a.head_dim == 128 ? launch_bs<128, kBias>(a, stream, self_plan) : launch_bs<64, kBias>(a, stream, self_plan);
  return a.head_dim == 128 ? launch_bs<128, kDiff>(a, stream, self_plan) : launch_bs<64, kDiff>(a, stream, self_plan);
}

}  // namespace pkv
