// Decode split-K over an 8-bit cache: the work decomposition, split states and merge of the bf16
// decode (decode_tc.cuh), over pages of half the bytes.
//
// For one page (16 tokens) of one kv head and its G query heads:
//   S^T [16 x 8] = K8 [16 x d] . Q^T [d x 8]     mma.sync m16n8k16, f16 -> fp32
//   s = S 2^ek 2^eq scale log2(e),  p = 2^(s - m)
//   O^T [d x 8] += (V8 2^(ev - r))^T [d x 16] . P^T [16 x 8]
// The held values become f16 exactly (int8: seven bits, e4m3: four), the page's K scale 2^ek is a
// factor of its scores in fp32, and each q row enters as q 2^-eq with its largest magnitude in
// [2^14, 2^15), so that what a bf16 q loses in f16 is below 2^-39 of its largest component.  V is taken
// relative to a reference exponent r of the warp: V 2^(ev - r) is exact in f16 for ev - r in
// [kQ8RefLow, kQ8RefHigh], and when a page's scale leaves that window r moves to it and the fp32 sums
// are multiplied by 2^(old r - new r).  p is rounded to f16 (11 bits) with m chosen so that the
// largest is near 2^kQ8Lift: what is flushed is below 2^-32 of the row's largest weight.
//
// m is not the running maximum: it is raised only when a score exceeds it by more than 8 (one vote
// per page in place of two shuffle reductions and a rescale of the sums).  The sums of a row refer
// to the same m, so the result is the same.
//
// Fragments come straight from the 8-bit rows with 16-byte reads: the order of the contraction's
// index is free, so lane (g, t) reads d/4 consecutive bytes of rows g and g + 8 of K (four bytes
// to a k-step; q is loaded in the same order), and d/8 consecutive bytes of rows 2t, 2t+1,
// 2t+8, 2t+9 of V, whose bytes of two tokens are interleaved before they become f16 pairs.  With
// the TMA's swizzle these reads have no bank conflicts at d = 128.
//
// A unit is 8 page-heads (16 at d 64): 16 KB of K and 16 KB of V.  Sixteen consumer warps in two
// groups take the units in turn, so that four warps to a scheduler hide the latency of one page's chain
// (wait, K, scores, weights, V).  Four producing warps copy pages by TMA and their scales by cp.async; both
// complete the same mbarrier.
//
// Bound: memory, between a start and an end of about 15 us.  Measured on GB300: one sequence of 131,072 keys
// (32/8 heads, d 128) 52 us, of which the keys' bytes take 38 (7.2 TB/s, some of them from L2); every CTA's plan 2.0,
// its first page 2.3 after that, the flush 2 and the merge 3.  256 sequences of up to 2048 keys (16/8) 104 us (5.3 TB/s
// over all of it), 50 of 8192 (28/4) 77.  An entry costs a CTA 4.2 us besides its keys (one unit's chain, the flush and the
// next entry's q, with the instructions of a path that is run once), which short contexts pay and long ones hide.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "decode.cuh"
#include "decode_tc.cuh"
#include "q8.cuh"

namespace pkv {

bool make_pool_map_heads_q8(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D,
                            int pages);

namespace {

constexpr int kGroups = 2;                        // consumer warps in groups of kDecodeWarps
constexpr int kWarps = kGroups * kDecodeWarps;
constexpr int kConsumers = kWarps * 32;
constexpr int kProducers = 4;  // warps
static_assert(kGroups == 2, "the flush folds two groups' states");
constexpr int kThreads = kConsumers + 128;  // + the producer's warpgroup

struct DecodeQ8Params {
  CUtensorMap tmap_k;  // 5-D: {d, 16 (8), Hkv, pages of a block, num_blocks} of bytes, box {d, 16 (8), Hkv, box_pages, 1}
  CUtensorMap tmap_v;
  DecodeParams p;
  const float* k_scale;
  const float* v_scale;
  int group;
  // without the planner kernel (a step without prefill tiles): the batch, from which every CTA finds
  // its own units
  int self_plan, plan_early, num_seqs;
  int64_t num_tokens, max_ctx;
  int box_pages;  // pages of a block that one copy brings
  unsigned long long tag;  // this call's own, below 2^48, when the pieces are merged here; 0: by the merge kernel
};

template <int D>
struct DecodeQ8Cfg {
  static constexpr int PPW = q8_pages_per_warp(D);
  static constexpr int kPartBytes = kDecodeWarps * PPW * 16 * D;  // K (or V) of a stage: 16 KB
  static constexpr int kScaleBytes = 2 * kDecodeWarps * PPW * 2 * 4;  // [K|V][page][half][head]
  static constexpr int kStageBytes = 2 * kPartBytes;
  // A multiple of the groups: a stage is then always the same group's, whose waits follow its phases in
  // order.  (Shared between groups, one could wait for a stage's next phase before its present one
  // has completed, and a parity wait would let it pass.)
  static constexpr int STAGES = 6;
  static constexpr int kBarBytes = 256 + 512;  // barriers and flags, each warp's meta words
  static constexpr int smem_bytes(int g) {
    return 1024 + kBarBytes + kDecodeWarps * g * (D + 2) * 4 + STAGES * (kStageBytes + kScaleBytes);
  }
  static_assert(STAGES % kGroups == 0 && smem_bytes(8) <= 227 * 1024, "ring");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pages of block `blk` from its page `page` on, all heads: {d, token, head, page, block}.
__device__ __forceinline__ void tma_load_pages(void* dst_smem, const CUtensorMap* map, int page, int blk, uint64_t* bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(page), "r"(blk), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// A decode CTA's record for the merge, written over its start record: the entry that holds its first
// unit, {entry, first unit, end unit, query row}, {W, 0, 0, 0}; entry -1 for a CTA without units.
struct MergeParams {
  Plan plan;
  bf16* out;
  int64_t o_st, o_sh;
  int hq;
};

constexpr int kMergeThreads = 512;

// The states of an entry cut by CTA boundaries, joined: out = sum 2^(m - M) acc / sum 2^(m - M) l.
// CTA c - 1 looks at boundary c between decode CTAs c - 1 and c.  The n - 1 boundaries inside an entry of n
// pieces share its columns (a column: four dims of a q head) in groups of eight, 128 bytes of a piece;
// where a CTA has fewer columns than threads its threads share the pieces as well and join their sums.  So two
// pieces take one CTA, and those of a context that is on every SM take every SM.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_q8_kernel(const __grid_constant__ MergeParams p) {
  constexpr int kQ = D / 4;
  constexpr int kBatch = 4;
  constexpr int kWarpsM = kMergeThreads / 32;
  __shared__ float4 s_num[kWarpsM][32];
  __shared__ float2 s_ml[kWarpsM][32];
  const float NEG_INF = -__int_as_float(0x7f800000);
  pdl_wait();
  pdl_trigger();
  const int c = static_cast<int>(blockIdx.x) + 1;
  const int4 rec = p.plan.cta_rec[2 * c];
  const int W = p.plan.cta_rec[2 * c + 1].x;
  if (rec.x < 0 || rec.y >= c * W) return;  // (an entry starts at the boundary, or the units end before it)
  const int c0 = rec.y / W;                 // the entry's first CTA
  const int n = (rec.z - 1) / W - c0 + 1;
  const int64_t slot0 = c0 + rec.x;
  const int ncol = p.hq * kQ;
  const int per = ceil_div(ceil_div(ncol, n - 1), 8) * 8;
  const int col0 = (c - 1 - c0) * per, col1 = min(ncol, col0 + per);
  int width = 8;  // columns at a time
  while (width < per && width < kMergeThreads) width <<= 1;
  const int lanes = kMergeThreads / width;  // threads to a column
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int base = col0; base < col1; base += width) {  // (more than once only with a thread to a column)
    const int col = base + (threadIdx.x & (width - 1));
    const int h = col / kQ, q = col & (kQ - 1);
    float M = NEG_INF, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    const int end = col < col1 ? n : 0;
    for (int k0 = threadIdx.x / width; k0 < end; k0 += kBatch * lanes) {
      float2 ml[kBatch];
      float4 a[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = make_float2(NEG_INF, 0.f);
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k * lanes < end) {
          const int64_t sh = (slot0 + k0 + k * lanes) * p.hq + h;
          ml[k] = *reinterpret_cast<const float2*>(p.plan.part_ml + sh * 2);
          a[k] = *(reinterpret_cast<const float4*>(p.plan.part_acc + sh * D) + q);
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
    if (lanes > 1) {
      auto join = [&](float m2, float d2, float4 n2) {
        const float Mn = fmaxf(M, m2);
        const float b = Mn == NEG_INF ? 0.f : Mn;
        const float w1 = fast_exp2(M - b), w2 = fast_exp2(m2 - b);
        den = den * w1 + d2 * w2;
        num.x = num.x * w1 + n2.x * w2;
        num.y = num.y * w1 + n2.y * w2;
        num.z = num.z * w1 + n2.z * w2;
        num.w = num.w * w1 + n2.w * w2;
        M = Mn;
      };
      __syncwarp();
      for (int off = width; off < 32; off <<= 1) {
        float4 n2;
        n2.x = __shfl_xor_sync(0xffffffffu, num.x, off);
        n2.y = __shfl_xor_sync(0xffffffffu, num.y, off);
        n2.z = __shfl_xor_sync(0xffffffffu, num.z, off);
        n2.w = __shfl_xor_sync(0xffffffffu, num.w, off);
        const float m2 = __shfl_xor_sync(0xffffffffu, M, off), d2 = __shfl_xor_sync(0xffffffffu, den, off);
        join(m2, d2, n2);
      }
      s_num[warp][lane] = num;
      s_ml[warp][lane] = make_float2(M, den);
      __syncthreads();
      const int step = max(width >> 5, 1);  // warps to a set of columns
      if (warp >= step || lane >= width) return;
      for (int w = warp + step; w < kWarpsM; w += step) join(s_ml[w][lane].x, s_ml[w][lane].y, s_num[w][lane]);
    }
    if (col < col1) {
      const float inv = 1.f / den;
      uint2 o;
      o.x = pack_bf16x2(num.x * inv, num.y * inv);
      o.y = pack_bf16x2(num.z * inv, num.w * inv);
      *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(rec.w) * p.o_st + static_cast<int64_t>(h) * p.o_sh + 4 * q) = o;
    }
  }
}

// A small batch's pieces are merged in the decode kernel itself: the CTA that writes the last of an
// entry's pieces merges them all (finish_pieces); no thread waits for another CTA.  Nothing zeroes the
// workspace before, so a counter carries the call's tag: a word with another tag counts as none, and the
// last arrival leaves a word that no call's tag matches (a captured call keeps its tag in every replay).
__device__ __forceinline__ bool last_arrival(unsigned long long* counter, unsigned long long tag, int of) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(counter);
  while (true) {
    const unsigned long long seen = (old >> 16) == tag ? old & 0xffffull : 0ull;
    const bool last = seen == static_cast<unsigned long long>(of - 1);
    const unsigned long long was = atomicCAS(counter, old, last ? 0ull : (tag << 16 | (seen + 1)));
    if (was == old) return last;
    old = was;
  }
}

// Entry i's `chunks` pieces, CTAs c0 on, this CTA's among them just written.  (The counter is in the start
// record of CTA c0, which starts at most one entry of several pieces.)
template <int D>
__device__ void finish_pieces(const DecodeParams& p, unsigned long long tag, int i, int64_t tq, int c0, int chunks,
                              volatile int* last_flag) {
  constexpr int kQ = D / 4;
  constexpr int kBatch = 4;
  const float NEG_INF = -__int_as_float(0x7f800000);
  __threadfence();
  named_bar_sync(1, kConsumers);
  if (threadIdx.x == 0)
    *last_flag = last_arrival(reinterpret_cast<unsigned long long*>(p.plan.cta_rec + 2 * c0), tag, chunks);
  named_bar_sync(1, kConsumers);
  if (!*last_flag) return;
  __threadfence();
  for (int item = threadIdx.x; item < p.hq * kQ; item += kConsumers) {
    const int h = item / kQ, q = item - h * kQ;
    float M = NEG_INF, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < chunks; k0 += kBatch) {
      float2 ml[kBatch];
      float4 a[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = make_float2(NEG_INF, 0.f);
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < chunks) {
          const int64_t sh = static_cast<int64_t>(c0 + i + k0 + k) * p.hq + h;
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p.plan.part_ml + sh * 2));
          a[k] = __ldcg(reinterpret_cast<const float4*>(p.plan.part_acc + sh * D) + q);
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
    const float inv = 1.f / den;
    uint2 o;
    o.x = pack_bf16x2(num.x * inv, num.y * inv);
    o.y = pack_bf16x2(num.z * inv, num.w * inv);
    *reinterpret_cast<uint2*>(p.out + tq * p.o_st + static_cast<int64_t>(h) * p.o_sh + 4 * q) = o;
  }
}

// Sums of two counters over the block's threads before this one, and over all of them.
__device__ __forceinline__ int2 block_scan2(int2 v, int2& total, int2* sm /* [kThreads / 32] */) {
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
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 t = sm[w];
    if (w < warp) before.x += t.x, before.y += t.y;
    total.x += t.x;
    total.y += t.y;
  }
  return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// TWO: 8-token blocks, a page of 16 tokens is two of them; else a page lies in one block.
template <int D, int FMT, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q8_kernel(const __grid_constant__ DecodeQ8Params P) {
  using C = DecodeQ8Cfg<D>;
  constexpr int PPW = C::PPW;
  constexpr int KS = D / 16;       // k-steps of QK^T, m-tiles of P.V
  constexpr int HALVES = TWO ? 2 : 1;
  const DecodeParams& p = P.p;
  const int G = P.group;
  constexpr int STAGES = C::STAGES;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* stages = smem;
  float* scales = reinterpret_cast<float*>(smem + STAGES * C::kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * (C::kStageBytes + C::kScaleBytes));
  uint64_t* empty = full + STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + STAGES);
  volatile int* last_flag = abort_flag + 2;
  int* warp_meta = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(full) + 256);
  float* xbuf = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(full) + C::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1 + 32 * kProducers);  // the TMA bytes' arrival and every producer lane's cp.async
      mbar_init(&empty[s], kDecodeWarps);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_v)) : "memory");
  }
  const int hkv = p.hkv;
  const int wpp = kDecodeWarps / hkv;  // warps (pages at a time) to a kv head
  const int ppu = wpp * PPW;           // pages of a unit
  int4* first_rec = reinterpret_cast<int4*>(warp_meta + 64);  // [2]
  int mode = 0;  // 0: everything before this kernel has finished; 1, 2: streaming early, as in the bf16 decode
  int U, W, ubeg, uend;
  if (P.self_plan) {
    // Every CTA scans the batch (two passes over context_lens and query_start_loc, one block scan each,
    // about a microsecond) and writes the entries that its own units touch: no planner kernel before
    // this one.  An entry is a row: a sequence's one new token, or each row of a longer span.
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
    int2 v = make_int2(0, 0), tot, ex;
    U = 0;
    for (int base = 0; base < P.num_seqs; base += kThreads) {
      v = look(base + tid);
      ex = block_scan2(v, tot, scan);
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
          ex = block_scan2(v, tot, scan);
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
    // Streaming early: an entry that is a row of a longer span has new keys before its last page.  With fewer than
    // four kv heads nothing is copied early either: copies of 4 or 8 bytes go through L1, whose sector holds the
    // scales of other blocks too, newest ones among them, as they were before the append changed them.
    if (p.stream_early) mode = __syncthreads_or(span > 1 || P.num_seqs > kThreads || hkv < 4) ? 2 : 1;
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
  const uint32_t page_bytes = static_cast<uint32_t>(hkv * 16 * D);
  // a stage: [K|V][page][half][kv head][16 / HALVES rows][D bytes]
  const uint32_t half_off = static_cast<uint32_t>(hkv * 8 * D);  // (TWO) rows 8..15
  const uint32_t head_off = 16 * D / HALVES;
  const uint32_t row8_off = TWO ? half_off : 8 * D;

  // Registers: 64 a thread for the producer's warpgroup and 104 for the consumers', within the 96 of the
  // launch (640 threads).
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------------ producer warps
    if (p.fault_no_copies) return;
    const uint64_t pol = l2_policy_evict_first();
    // Each takes K or V of one half of a unit's pages, a lane to a page: a warp's lanes issue their copies one
    // after the other, about 60 ns each.  Measured on GB300, 268 MB of keys of 1 kv head, d 128, blocks of 8 (1 KB a
    // copy) and of 16: one warp 116 and 77 us, two 90 and 66, four 75 and 60.
    const int kv = warp & 1, part = (warp - kWarps) >> 1;
    const int bp = (ppu * part >> 1) + lane;
    const bool lane_has_page = bp < ppu * (part + 1) >> 1;
    const bool lane_copies = (bp & (P.box_pages - 1)) == 0;
    const float* scale_src = kv ? P.v_scale : P.k_scale;
    const uint32_t scale_dst0 = smem_u32(scales) + static_cast<uint32_t>((kv * ppu + bp) * HALVES * hkv * 4);
    const int blk_shift = TWO ? 0 : p.bs_log2 - 4;  // page gp lies in block gp >> blk_shift
    // A unit as this lane copies it: its page's block (and second block), the page in it, the bytes of the whole
    // unit, and whether it may hold what the kernel before the planner writes.  Read one unit ahead, so
    // that the latency of the block table is never between a free stage and its copies.
    struct Unit {
      int blk, blk2, page0, bytes;
      bool page, half2, late;  // this lane copies blk, and blk2
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
      // streaming early: any row (and the scale) of the block that holds the newest key may still change
      n.late = mode == 2 || pg0 + npg - 1 >= (((ctx - 1) >> p.bs_log2) << p.bs_log2) >> 4;
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
      if (warp == kWarps && lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(cur.bytes));
      __syncwarp();
      if (cur.page) {
        if (cur.blk < 0 || cur.blk >= p.num_blocks || cur.blk2 < 0 || cur.blk2 >= p.num_blocks) {
          raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);  // a bad id is read as block 0
          if (cur.blk < 0 || cur.blk >= p.num_blocks) cur.blk = 0;
          if (cur.blk2 < 0 || cur.blk2 >= p.num_blocks) cur.blk2 = 0;
        }
        unsigned char* dst = stages + s * C::kStageBytes + kv * C::kPartBytes + bp * page_bytes;
        const CUtensorMap* map = kv ? &P.tmap_v : &P.tmap_k;
        if (lane_copies) tma_load_pages(dst, map, cur.page0, cur.blk, &full[s], pol);
        if (TWO && cur.half2) tma_load_pages(dst + half_off, map, 0, cur.blk2, &full[s], pol);
        // the blocks' scales, hkv floats each (a power of two of them, so aligned to the copy's size)
        uint32_t sd = scale_dst0 + static_cast<uint32_t>(s * C::kScaleBytes);
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
          if (half == 0 || cur.half2) {
            const float* src = scale_src + static_cast<int64_t>(half ? cur.blk2 : cur.blk) * hkv;
            if (hkv == 8) {
              cp_async_l2(sd, src);
              cp_async_l2(sd + 16, src + 4);
            } else if (hkv == 4) {
              cp_async_l2(sd, src);
            } else if (hkv == 2) {
              cp_async<8>(sd, src);
            } else {
              cp_async<4>(sd, src);
            }
          }
          sd += hkv * 4;
        }
      }
      cp_async_arrive(&full[s]);
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
  asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
  if (mode != 0) pdl_wait();  // q is written by the kernel before the planner
  const int wg = warp / kDecodeWarps;  // this warp's group: units ubeg + wg, ubeg + wg + kGroups, ..
  const int pw = (warp % kDecodeWarps) / hkv;
  const int h = warp % kDecodeWarps - pw * hkv;
  const int gr = lane >> 2, tig = lane & 3;
  const float NEG_INF = -__int_as_float(0x7f800000);

  uint32_t qb[KS][2];  // Q^T B fragments (f16): head gr, dims tig d/4 + 4 kk + 0..1 and + 2..3
  float fq[2];         // scale log2(e) 2^eq of heads 2tig, 2tig + 1
  float acc[KS][4];    // O^T: dims gr d/8 + 2mt (+1), heads 2tig (+1), in units of 2^(ref - 127)
  float mref[2], lsum[2];
  const uint32_t stage_base = smem_u32(stages);
  const bool hv = gr < G;
  bool ok = true;
  int* meta = warp_meta + 4 * warp;  // what the flush needs, read from the plan while the segment runs
  uint4 raw_q[KS / 2];
  auto read_q = [&](int64_t row_tq) {
    const uint4* qrow = reinterpret_cast<const uint4*>(
        p.q + row_tq * p.q_st + static_cast<int64_t>(h * G + (hv ? gr : 0)) * p.q_sh + tig * (D / 4));
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) raw_q[x] = hv ? qrow[x] : make_uint4(0u, 0u, 0u, 0u);
  };
  // q 2^-eq in f16, eq putting the head's largest magnitude in [2^14, 2^15)
  auto take_q = [&]() {
    unsigned mx = 0;
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) {
      const uint32_t w[4] = {raw_q[x].x, raw_q[x].y, raw_q[x].z, raw_q[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) mx = max(mx, max(w[y] & 0x7fffu, (w[y] >> 16) & 0x7fffu));
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = min(max(static_cast<int>(mx >> 7), 30), 254);  // biased exponent of the largest
    const float up = q8_exp2(127 + 14 + 127 - e);              // 2^(14 - (e - 127))
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) {
      const uint32_t w[4] = {raw_q[x].x, raw_q[x].y, raw_q[x].z, raw_q[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) qb[2 * x + (y >> 1)][y & 1] = pack_f16x2(bf16lo(w[y]) * up, bf16hi(w[y]) * up);
    }
    const float f = p.qscale * q8_exp2(e - 14);
    fq[0] = __shfl_sync(0xffffffffu, f, (2 * tig) << 2);  // head 2 tig is lane group gr = 2 tig's
    fq[1] = __shfl_sync(0xffffffffu, f, (2 * tig + 1) << 2);
  };
  // segments: the parts of consecutive entries that lie in this CTA's units [ubeg, uend)
  int s = wg;  // stage and phase of this group's next unit
  uint32_t phase = 0;
  int u = ubeg + wg;  // this group's next unit
  int i = i_first, ustart = rec0.y, unext = rec0.z, ctx = rec1.x, tq = rec1.y;
  read_q(tq);
  while (true) {
    take_q();
    const int npages = ceil_div(ctx, 16);
    const int u1 = min(unext, uend);
    if (unext < uend && lane < 3) {  // the next entry
      const int* src = lane == 0 ? dec_unit + i + 2 : lane == 1 ? p.plan.dec_ctx + i + 1 : p.plan.dec_tq + i + 1;
      cp_async<4>(smem_u32(meta + lane), src);
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    mref[0] = mref[1] = NEG_INF;
    lsum[0] = lsum[1] = 0.f;
    int ref = 0;  // biased exponent of the V reference; 0: none yet
    int peak = 0;  // the highest it has been: how far down it may come (kQ8MaxDown)
    for (; u < u1; u += kGroups) {
      if (ok) ok = wait_or_abort(&full[s], phase, p.err, abort_flag);
#pragma unroll
      for (int w = 0; w < PPW; ++w) {
        const int up = pw + w * wpp;  // page of the unit
        const int pg = (u - ustart) * ppu + up;
        if (!ok || pg >= npages) continue;
        const int rows = min(16, ctx - pg * 16);
        const uint32_t kbase = stage_base + s * C::kStageBytes + up * page_bytes + h * head_off;
        const uint32_t vbase = kbase + C::kPartBytes;
        const float* sc_k = scales + s * (C::kScaleBytes / 4) + up * HALVES * hkv + h;
        const float* sc_v = sc_k + ppu * HALVES * hkv;
        const float ks0 = sc_k[0], ks1 = TWO ? sc_k[hkv] : ks0;  // (a half past the context: unused)
        int ev0 = __float_as_int(sc_v[0]) >> 23;
        int ev1 = TWO && rows > 8 ? __float_as_int(sc_v[hkv]) >> 23 : ev0;

        // S^T = K . Q^T, two chains
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < KS / 4; ++x) {  // 16 bytes of rows gr and gr + 8: four k-steps
          const uint32_t off = chunk8_off<D>(gr, KS / 4 * tig + x);
          const uint4 r0 = lds128(kbase + off), r1 = lds128(kbase + row8_off + off);
          const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t a0, a1, a2, a3;
            q8_to_f16<FMT>(w0[y], a0, a2);
            q8_to_f16<FMT>(w1[y], a1, a3);
            mma_f16(y & 1 ? sb : sa, a0, a1, a2, a3, qb[4 * x + y][0], qb[4 * x + y][1]);
          }
        }
        // scores in the log2 domain, keys past the context masked by select
        const bool v0 = gr < rows, v1 = gr + 8 < rows;
        float sc[4];
        sc[0] = v0 ? (sa[0] + sb[0]) * (fq[0] * ks0) : NEG_INF;
        sc[1] = v0 ? (sa[1] + sb[1]) * (fq[1] * ks0) : NEG_INF;
        sc[2] = v1 ? (sa[2] + sb[2]) * (fq[0] * ks1) : NEG_INF;
        sc[3] = v1 ? (sa[3] + sb[3]) * (fq[1] * ks1) : NEG_INF;
        float pm0 = fmaxf(sc[0], sc[2]), pm1 = fmaxf(sc[1], sc[3]);
        if (__any_sync(0xffffffffu, pm0 - mref[0] > kQ8Slack || pm1 - mref[1] > kQ8Slack)) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            pm0 = fmaxf(pm0, __shfl_xor_sync(0xffffffffu, pm0, off));
            pm1 = fmaxf(pm1, __shfl_xor_sync(0xffffffffu, pm1, off));
          }
          const float mn0 = fmaxf(mref[0], pm0), mn1 = fmaxf(mref[1], pm1);
          const float c0 = mref[0] == mn0 ? 1.f : fast_exp2(mref[0] - mn0);
          const float c1 = mref[1] == mn1 ? 1.f : fast_exp2(mref[1] - mn1);
          mref[0] = mn0;
          mref[1] = mn1;
          lsum[0] *= c0;
          lsum[1] *= c1;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            acc[mt][0] *= c0;
            acc[mt][1] *= c1;
            acc[mt][2] *= c0;
            acc[mt][3] *= c1;
          }
        }
        // (the difference before the lift: m - 7 is rounded where m is large, and a weight could pass f16's range)
        const float b0 = mref[0] == NEG_INF ? 0.f : mref[0], b1 = mref[1] == NEG_INF ? 0.f : mref[1];
        sc[0] = fast_exp2((sc[0] - b0) + kQ8Lift);
        sc[1] = fast_exp2((sc[1] - b1) + kQ8Lift);
        sc[2] = fast_exp2((sc[2] - b0) + kQ8Lift);
        sc[3] = fast_exp2((sc[3] - b1) + kQ8Lift);
        lsum[0] += sc[0] + sc[2];
        lsum[1] += sc[1] + sc[3];
        // P^T (tokens x heads) -> B fragments (k = token, n = head) by an 8x8 transpose
        const uint32_t pb0 = movmatrix_t(pack_f16x2(sc[0], sc[1]));
        const uint32_t pb1 = movmatrix_t(pack_f16x2(sc[2], sc[3]));

        // O^T += V^T . P^T; the two halves of a page one after the other when their scales are too
        // far apart for one reference (8-token blocks only)
        const int passes = TWO && (ev0 - ev1 > -kQ8RefLow || ev1 - ev0 > -kQ8RefLow) ? 2 : 1;
        for (int pass = 0; pass < passes; ++pass) {
          const int ea = passes == 2 ? (pass ? ev1 : ev0) : ev0, eb = passes == 2 ? ea : ev1;
          const int top = max(ea, eb);
          if (ref == 0) {
            ref = peak = top;
          } else if (top - ref > kQ8RefHigh || min(ea, eb) - ref < kQ8RefLow) {  // (warp-uniform)
            // the reference moves to this page's scale, unless that is too far below the highest so far
            const int sh = ref - top;
            peak = max(peak, top);
            if (peak - top <= kQ8MaxDown) {
              const float f = sh >= -126 ? q8_exp2(127 + sh) : 0.f;
#pragma unroll
              for (int mt = 0; mt < KS; ++mt) {
                acc[mt][0] *= f;
                acc[mt][1] *= f;
                acc[mt][2] *= f;
                acc[mt][3] *= f;
              }
              ref = top;
            }
          }
          uint32_t sA, oA, sB, oB;
          q8_f16_pow2(ea - ref, sA, oA);
          if constexpr (TWO) {
            q8_f16_pow2(eb - ref, sB, oB);
          } else {
            sB = sA;
            oB = oA;
          }
          const uint32_t b0p = passes == 2 && pass == 1 ? 0u : pb0, b1p = passes == 2 && pass == 0 ? 0u : pb1;
          const uint32_t z0 = 2 * tig, z1 = 2 * tig + 1;  // this lane's rows (and + 8)
          constexpr int NW = D / 32;  // 4-byte words of a row to a lane
          uint32_t r0[NW], r1[NW], r2[NW], r3[NW];
          if constexpr (D == 128) {
            const uint4 a = lds128(vbase + chunk8_off<D>(z0, gr)), b = lds128(vbase + chunk8_off<D>(z1, gr));
            const uint4 c = lds128(vbase + row8_off + chunk8_off<D>(z0, gr)),
                        d = lds128(vbase + row8_off + chunk8_off<D>(z1, gr));
            r0[0] = a.x, r0[1] = a.y, r0[2] = a.z, r0[3] = a.w;
            r1[0] = b.x, r1[1] = b.y, r1[2] = b.z, r1[3] = b.w;
            r2[0] = c.x, r2[1] = c.y, r2[2] = c.z, r2[3] = c.w;
            r3[0] = d.x, r3[1] = d.y, r3[2] = d.z, r3[3] = d.w;
          } else {
            const uint32_t in = (gr & 1) * 8;
            const uint2 a = lds64(vbase + chunk8_off<D>(z0, gr >> 1) + in), b = lds64(vbase + chunk8_off<D>(z1, gr >> 1) + in);
            const uint2 c = lds64(vbase + row8_off + chunk8_off<D>(z0, gr >> 1) + in),
                        d = lds64(vbase + row8_off + chunk8_off<D>(z1, gr >> 1) + in);
            r0[0] = a.x, r0[1] = a.y;
            r1[0] = b.x, r1[1] = b.y;
            r2[0] = c.x, r2[1] = c.y;
            r3[0] = d.x, r3[1] = d.y;
          }
          if (FMT == PKV_Q8_E4M3 && rows < 16) {
            // keys past the context: e4m3 bytes there may be NaN, and 0 NaN would poison P.V
#pragma unroll
            for (int x = 0; x < NW; ++x) {
              if (z0 >= rows) r0[x] = 0u;
              if (z1 >= rows) r1[x] = 0u;
              if (z0 + 8 >= rows) r2[x] = 0u;
              if (z1 + 8 >= rows) r3[x] = 0u;
            }
          }
#pragma unroll
          for (int x = 0; x < NW; ++x) {
            // bytes of tokens z0, z1 (and z0 + 8, z1 + 8) interleaved: [z0 d0, z1 d0, z0 d1, z1 d1], then d2, d3
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a0, a1, a2, a3;
              q8_to_f16_scaled<FMT>(__byte_perm(r0[x], r1[x], y ? 0x7362 : 0x5140), sA, oA, a0, a1);
              q8_to_f16_scaled<FMT>(__byte_perm(r2[x], r3[x], y ? 0x7362 : 0x5140), sB, oB, a2, a3);
              mma_f16(acc[2 * x + y], a0, a1, a2, a3, b0p, b1p);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      s += kGroups;
      if (s >= STAGES) {
        s -= STAGES;
        phase ^= 1;
      }
    }

    // ---------------------------------------------------------------- segment flush
    // The state (m + 8, l 2^-15, acc 2^(ref - 127 - 15)): weights relative to 2^(m + 8), at most 1.
    float L0 = lsum[0], L1 = lsum[1];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      L0 += __shfl_xor_sync(0xffffffffu, L0, off);
      L1 += __shfl_xor_sync(0xffffffffu, L1, off);
    }
    constexpr float kDown = 1.f / 32768.f;
    const float unit = q8_exp2(ref > 0 ? ref : 1);
    // the second group's warps leave their states for the first group's, which fold them into their own
    // (xbuf: [warp][head] rows of D floats, then their (m, l).  A row's 16-byte chunks are xored with tig, spread so
    // that eight lanes' accesses, two gr by four tig, use different banks)
    auto xsw = [](int g) { return D == 128 ? (g >> 1 & 3) << 2 : ((g >> 1 & 1) | (g & 4)) << 2; };
    float* xb = xbuf + (warp % kDecodeWarps) * G * D;
    float2* xml = reinterpret_cast<float2*>(xbuf + kDecodeWarps * G * D);
    float2* xm = xml + (warp % kDecodeWarps) * G;
    auto put = [&](float m0, float m1, float l0, float l1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int hh = 2 * tig + j;
        if (hh < G) {
#pragma unroll
          for (int mt = 0; mt < KS; mt += 2)
            *reinterpret_cast<float4*>(xb + hh * D + (gr * (D / 8) + 2 * mt ^ xsw(hh))) =
                make_float4(acc[mt][j], acc[mt][2 + j], acc[mt + 1][j], acc[mt + 1][2 + j]);
          if (gr == 0) xm[hh] = make_float2(j ? m1 : m0, j ? l1 : l0);
        }
      }
    };
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[mt][j] *= kDown * unit;
    mref[0] += 15.f - kQ8Lift;
    mref[1] += 15.f - kQ8Lift;
    L0 *= kDown;
    L1 *= kDown;
    if (wg == 1) put(mref[0], mref[1], L0, L1);
    named_bar_sync(1, kConsumers);
    if (wg == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int hh = 2 * tig + j;
        if (hh < G) {
          const float2 ml = xm[hh];
          const float M = fmaxf(mref[j], ml.x);
          const float b = M == NEG_INF ? 0.f : M;
          const float w0 = fast_exp2(mref[j] - b), w1 = fast_exp2(ml.x - b);
          float& L = j ? L1 : L0;
          L = L * w0 + ml.y * w1;
          mref[j] = M;
#pragma unroll
          for (int mt = 0; mt < KS; mt += 2) {
            const float4 o = *reinterpret_cast<const float4*>(xb + hh * D + (gr * (D / 8) + 2 * mt ^ xsw(hh)));
            acc[mt][j] = acc[mt][j] * w0 + o.x * w1;
            acc[mt][2 + j] = acc[mt][2 + j] * w0 + o.y * w1;
            acc[mt + 1][j] = acc[mt + 1][j] * w0 + o.z * w1;
            acc[mt + 1][2 + j] = acc[mt + 1][2 + j] * w0 + o.w * w1;
          }
        }
      }
      if (wpp > 1) {
        __syncwarp();  // (m, l) read by every lane
        put(mref[0], mref[1], L0, L1);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const bool more = unext < uend;
    const int nx_unext = meta[0], nx_ctx = meta[1], nx_tq = meta[2];  // (unused unless more)
    const bool whole = ustart >= ubeg && unext <= uend;  // the entry's every unit is this CTA's
    if (more) read_q(nx_tq);  // (arrives while the states are merged)
    // a piece's slot: CTA and entry grow together along the pieces, so their sum names each once
    const int64_t slot_h = static_cast<int64_t>(static_cast<int>(blockIdx.x) + i) * p.hq;
    auto write4 = [&](int hq, int d0, float4 num, float M, float den, float inv) {
      if (whole) {
        uint2 o;
        o.x = pack_bf16x2(num.x * inv, num.y * inv);
        o.y = pack_bf16x2(num.z * inv, num.w * inv);
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(tq) * p.o_st + static_cast<int64_t>(hq) * p.o_sh + d0) = o;
      } else {
        *reinterpret_cast<float4*>(p.plan.part_acc + (slot_h + hq) * D + d0) = num;
        if (d0 == 0) *reinterpret_cast<float2*>(p.plan.part_ml + (slot_h + hq) * 2) = make_float2(M, den);
      }
    };
    if (wpp == 1) {  // a warp of the first group holds its head's state
      if (wg == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (2 * tig + j < G) {
            const float den = j ? L1 : L0, inv = 1.f / den;
#pragma unroll
            for (int mt = 0; mt < KS; mt += 2)
              write4(h * G + 2 * tig + j, gr * (D / 8) + 2 * mt,
                     make_float4(acc[mt][j], acc[mt][2 + j], acc[mt + 1][j], acc[mt + 1][2 + j]), mref[j], den, inv);
          }
        }
      }
    } else {
      named_bar_sync(1, kConsumers);
      for (int item = threadIdx.x; item < hkv * G * (D / 4); item += kConsumers) {
        const int hh = item / (G * (D / 4));
        const int rem3 = item - hh * G * (D / 4);
        const int g = rem3 / (D / 4);
        const int d0 = (rem3 - g * (D / 4)) * 4;
        float M = NEG_INF;
        for (int k = 0; k < wpp; ++k) M = fmaxf(M, xml[(hh + k * hkv) * G + g].x);
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
        for (int k = 0; k < wpp; ++k) {
          const int row = (hh + k * hkv) * G + g;
          const float w = fast_exp2(xml[row].x - M);  // a warp with no pages: m = -inf -> w = 0
          den = fmaf(w, xml[row].y, den);
          const float4 x = *reinterpret_cast<const float4*>(xbuf + row * D + (d0 ^ xsw(g)));
          num.x = fmaf(w, x.x, num.x);
          num.y = fmaf(w, x.y, num.y);
          num.z = fmaf(w, x.z, num.z);
          num.w = fmaf(w, x.w, num.w);
        }
        write4(hh * G + g, d0, num, M, den, 1.f / den);
      }
    }
    named_bar_sync(1, kConsumers);
    if (!whole && P.tag) {
      const int c0 = ustart / W;
      finish_pieces<D>(p, P.tag, i, tq, c0, (unext - 1) / W - c0 + 1, last_flag);
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
unsigned long long next_tag() {
  static std::atomic<unsigned long long> count{
      static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ull};
  unsigned long long t;
  do t = count.fetch_add(1) & 0xffffffffffffull;
  while (t == 0);
  return t;
}

template <int D, int FMT, bool TWO>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  using C = DecodeQ8Cfg<D>;
  // (the largest any group needs, so the limit is raised once)
  if (const cudaError_t e = set_smem_once<decode_q8_kernel<D, FMT, TWO>>(C::smem_bytes(8)); e != cudaSuccess) return e;
  DecodeQ8Params P;
  // Pages of a block are copied together where a unit holds several (few kv heads): a copy costs about 60 ns of the
  // SM's copy engine besides its bytes.  Measured on GB300, 268 MB of keys of 1 kv head, d 128, blocks of 128: page
  // by page 75.6 us, eight pages at a time 58.0 (d 64: 103.8, 64.2).
  P.box_pages = TWO ? 1 : std::min(kDecodeWarps / a.hkv * C::PPW, 1 << (a.bs_log2 - 4));
  if (!make_pool_map_heads_q8(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D, P.box_pages) ||
      !make_pool_map_heads_q8(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D, P.box_pages))
    return cudaErrorInvalidValue;
  DecodeParams& p = P.p;
  p.q = static_cast<const bf16*>(a.q);
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.k_cache = nullptr;
  p.v_cache = nullptr;
  p.num_blocks = a.num_blocks;
  p.bs_log2 = a.bs_log2;
  p.block_tables = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.context_lens = a.context_lens;
  p.qsl = a.qsl;
  p.out = static_cast<bf16*>(a.out);
  p.o_st = a.o_st;
  p.o_sh = a.o_sh;
  p.hkv = a.hkv;
  p.hq = a.hq;
  p.qscale = a.scale * 1.4426950408889634f;
  p.plan = a.plan;
  p.err = a.err;
  p.fault_no_copies = a.fault == PKV_FAULT_DECODE_NO_COPIES;
  p.stream_early = a.stream_early;
  P.k_scale = a.k_scale;
  P.v_scale = a.v_scale;
  P.group = a.hq / a.hkv;
  P.self_plan = self_plan ? 1 : 0;
  P.plan_early = a.plan_early;
  P.num_seqs = static_cast<int>(a.num_seqs);
  P.num_tokens = a.num_tokens;
  P.max_ctx = max_context(a.max_blocks, a.bs_log2);
  // Pieces merged in the kernel or by one after it.  In it: one launch less, but the merge of an entry is one
  // CTA's.  Measured on GB300 (32/8 heads, d 128), in the kernel / after it: 4 sequences of up to 100 keys 8.7 / 10.7
  // us, 64 of 64 16.3 / 19.2, 64 of 128 16.7 / 19.2; 64 of 256 21.8 / 19.9, 256 of 64 25.1 / 24.4, one of 4096 21.4 /
  // 18.7, 32 of up to 1152 16.2 / 14.8.
  const int64_t units = ceil_div64(ceil_div64(P.max_ctx, kPageTokens), kDecodeWarps / a.hkv * C::PPW);
  const bool merge_here = self_plan && a.num_seqs * P.max_ctx <= (1 << 13) && units <= 8;
  P.tag = merge_here ? next_tag() : 0;
  record_kernel_event(PKV_KERNEL_DECODE, false, stream);
  cudaError_t e = launch_pdl(decode_q8_kernel<D, FMT, TWO>, dim3(a.decode_ctas), dim3(kThreads),
                             C::smem_bytes(P.group), stream, P);
  if (e == cudaSuccess && !merge_here && a.decode_ctas > 1) {
    MergeParams M;
    M.plan = a.plan;
    M.out = p.out;
    M.o_st = a.o_st;
    M.o_sh = a.o_sh;
    M.hq = a.hq;
    // (beside prefill tiles not launched early: its CTAs, waiting for the decode, would take the SMs that
    // the prefill's are to run on)
    e = launch_kernel(self_plan, merge_q8_kernel<D>, dim3(a.decode_ctas - 1), dim3(kMergeThreads), 0,
                      stream, M);
  }
  record_kernel_event(PKV_KERNEL_DECODE, true, stream);
  return e;
}

template <int D, int FMT>
cudaError_t launch_bs(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  return a.bs_log2 == 3 ? launch<D, FMT, true>(a, stream, self_plan) : launch<D, FMT, false>(a, stream, self_plan);
}

}  // namespace

cudaError_t launch_decode_q8(const AttnArgs& a, cudaStream_t stream, bool self_plan) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch_bs<128, PKV_Q8_INT8>(a, stream, self_plan)
                             : launch_bs<64, PKV_Q8_INT8>(a, stream, self_plan);
  return a.head_dim == 128 ? launch_bs<128, PKV_Q8_E4M3>(a, stream, self_plan)
                           : launch_bs<64, PKV_Q8_E4M3>(a, stream, self_plan);
}

}  // namespace pkv
