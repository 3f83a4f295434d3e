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
// A unit is 8 page-heads a warp (two at d 64): 16 KB of K and 16 KB of V.  The producer warp copies
// pages by TMA and their scales by cp.async; both complete the same mbarrier.
#include <cuda.h>

#include "decode.cuh"
#include "decode_tc.cuh"
#include "q8.cuh"

namespace pkv {

bool make_pool_map_heads_q8(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D);

namespace {

struct DecodeQ8Params {
  CUtensorMap tmap_k;  // 4-D: {d, block_size, Hkv, num_blocks} of bytes, box {d, min(block_size, 16), Hkv, 1}
  CUtensorMap tmap_v;
  DecodeParams p;
  const float* k_scale;
  const float* v_scale;
  int group;
  int stages;
};

template <int D>
struct DecodeQ8Cfg {
  static constexpr int PPW = q8_pages_per_warp(D);
  static constexpr int kPartBytes = kDecodeWarps * PPW * 16 * D;  // K (or V) of a stage: 16 KB
  static constexpr int kScaleBytes = 2 * kDecodeWarps * PPW * 2 * 4;  // [K|V][page][half][head]
  static constexpr int kStageBytes = 2 * kPartBytes;
  static constexpr int kMaxStages = 8;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemLimit = 227 * 1024;
  static constexpr int xbuf_bytes(int g) { return kDecodeWarps * g * (D + 2) * 4; }
  static constexpr int stages(int g) {
    const int fit = (kSmemLimit - 1024 - kBarBytes - xbuf_bytes(g)) / (kStageBytes + kScaleBytes);
    return fit < kMaxStages ? fit : kMaxStages;
  }
  static constexpr int smem_bytes(int g) {
    return 1024 + kBarBytes + xbuf_bytes(g) + stages(g) * (kStageBytes + kScaleBytes);
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// TWO: 8-token blocks, a page of 16 tokens is two of them; else a page lies in one block.
template <int D, int FMT, bool TWO>
__global__ void __launch_bounds__((kDecodeWarps + 1) * 32, 1)
    decode_q8_kernel(const __grid_constant__ DecodeQ8Params P) {
  using C = DecodeQ8Cfg<D>;
  constexpr int PPW = C::PPW;
  constexpr int KS = D / 16;       // k-steps of QK^T, m-tiles of P.V
  constexpr int HALVES = TWO ? 2 : 1;
  const DecodeParams& p = P.p;
  const int G = P.group;
  const int STAGES = P.stages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* stages = smem;
  float* scales = reinterpret_cast<float*>(smem + STAGES * C::kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * (C::kStageBytes + C::kScaleBytes));
  uint64_t* empty = full + C::kMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kMaxStages);
  volatile int* last_flag = abort_flag + 2;
  volatile int* stream_mode = abort_flag + 4;
  float* xbuf = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(full) + C::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 33);  // the TMA bytes' arrival and every producer lane's cp.async
      mbar_init(&empty[s], kDecodeWarps);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kDecodeWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_v)) : "memory");
  }
  // the plan: as in the bf16 decode (mode 0: all earlier work has finished; 1, 2: streaming early)
  int mode = 0;
  if (p.stream_early) {
    if (threadIdx.x == 0) {
      int v;
      const long long t0 = clock64();
      while ((v = ld_acquire_gpu(p.plan.header + kPlanReadyWord)) == 0 && clock64() - t0 < kPlanReadySpinClocks)
        __nanosleep(64);
      *stream_mode = v;
    }
    __syncthreads();
    mode = *stream_mode;
    if (mode == 0) pdl_wait();
  } else {
    pdl_wait();
  }
  pdl_trigger();
  const int* hdr = p.plan.header;
  const int U = hdr[1];
  const int W = hdr[2];
  const int4 rec0 = p.plan.cta_rec[2 * blockIdx.x];
  const int4 rec1 = p.plan.cta_rec[2 * blockIdx.x + 1];
  const int i_first = rec0.x;
  const int ubeg = blockIdx.x * W;
  const int uend = min(U, ubeg + W);
  if (ubeg >= uend) return;  // CTA-uniform
  const int* dec_unit = p.plan.dec_unit;
  __syncthreads();  // barrier initialisation visible to every warp
  const int hkv = p.hkv;
  const int wpp = kDecodeWarps / hkv;  // warps (pages at a time) to a kv head
  const int ppu = wpp * PPW;           // pages of a unit
  const uint32_t page_bytes = static_cast<uint32_t>(hkv * 16 * D);
  // a stage: [K|V][page][half][kv head][16 / HALVES rows][D bytes]
  const uint32_t half_off = static_cast<uint32_t>(hkv * 8 * D);  // (TWO) rows 8..15
  const uint32_t head_off = 16 * D / HALVES;
  const uint32_t row8_off = TWO ? half_off : 8 * D;

  if (warp == kDecodeWarps) {
    // ------------------------------------------------------------------ producer warp
    if (p.fault_no_copies) return;
    const uint64_t pol = l2_policy_evict_first();
    const int kv = lane / ppu;  // lane -> (K or V, page) of the unit; 2 ppu <= 32
    const int bp = lane - kv * ppu;
    const bool lane_has_page = lane < 2 * ppu;
    const float* scale_src = kv ? P.v_scale : P.k_scale;
    const uint32_t scale_dst0 = smem_u32(scales) + static_cast<uint32_t>((kv * ppu + bp) * HALVES * hkv * 4);
    int i = i_first;
    int ustart = rec0.y, unext = rec0.z;
    int b = rec0.w;
    int ctx = rec1.x;
    int npages = ceil_div(ctx, 16);
    const int blk_shift = TWO ? 0 : p.bs_log2 - 4;  // page gp lies in block gp >> blk_shift
    const int row_mask = (1 << p.bs_log2) - 1;
    int s = 0;
    uint32_t phase = 1;  // of empty[s]: a fresh barrier passes a wait for phase 1
    int u = ubeg;
    bool waited = mode == 0;
    for (; u < uend; ++u) {
      while (u >= unext) {
        ++i;
        ustart = unext;
        unext = dec_unit[i + 1];
        b = p.plan.dec_seq[i];
        ctx = p.plan.dec_ctx[i];
        npages = ceil_div(ctx, 16);
      }
      const int pg0 = (u - ustart) * ppu;
      const int npg = min(ppu, npages - pg0);
      const bool issue = lane_has_page && bp < npg;
      const int gp = pg0 + bp;
      int blk = 0, blk2 = -1;
      if (issue) {  // requested before the wait for the stage
        const int32_t* row = p.block_tables + static_cast<int64_t>(b) * p.bt_stride;
        blk = row[TWO ? 2 * gp : gp >> blk_shift];
        if (TWO && gp * 16 + 8 < ctx) blk2 = row[2 * gp + 1];
      }
      if (u - ubeg >= STAGES && !wait_or_abort(&empty[s], phase, p.err, abort_flag)) break;
      if (issue) {
        if (blk < 0 || blk >= p.num_blocks) {
          raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
          blk = 0;
        }
        if (TWO && gp * 16 + 8 < ctx && (blk2 < 0 || blk2 >= p.num_blocks)) {
          raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
          blk2 = 0;
        }
      }
      // streaming early: the kernel before the planner may write any row (and the scale) of the block
      // that holds the newest key, so pages from that block's first on wait for it
      if (!waited && (mode == 2 || pg0 + npg - 1 >= (((ctx - 1) >> p.bs_log2) << p.bs_log2) >> 4)) {
        pdl_wait();
        waited = true;
      }
      const bool tail_half = TWO && (pg0 + npg - 1) * 16 + 8 >= ctx;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], 2u * (npg * page_bytes - (tail_half ? page_bytes / 2 : 0u)));
      __syncwarp();
      if (issue) {
        unsigned char* dst = stages + s * C::kStageBytes + kv * C::kPartBytes + bp * page_bytes;
        const CUtensorMap* map = kv ? &P.tmap_v : &P.tmap_k;
        tma_load_4d(dst, map, 0, TWO ? 0 : (gp * 16) & row_mask, 0, blk, &full[s], pol);
        if (TWO && blk2 >= 0) tma_load_4d(dst + half_off, map, 0, 0, 0, blk2, &full[s], pol);
        // the blocks' scales, hkv floats each (a power of two of them, so aligned to the copy's size)
        uint32_t sd = scale_dst0 + static_cast<uint32_t>(s * C::kScaleBytes);
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
          const int bk = half ? blk2 : blk;
          if (bk >= 0) {
            const float* src = scale_src + static_cast<int64_t>(bk) * hkv;
            if (hkv == 8) {
              cp_async<16>(sd, src);
              cp_async<16>(sd + 16, src + 4);
            } else if (hkv == 4) {
              cp_async<16>(sd, src);
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
    // every copy issued has landed before the CTA may leave
    const int issued = u - ubeg;
    for (int k = max(0, issued - STAGES); k < issued; ++k)
      wait_or_abort(&full[k % STAGES], (k / STAGES) & 1, p.err, abort_flag);
    return;
  }

  // -------------------------------------------------------------------- consumer warps
  if (mode != 0) pdl_wait();  // q is written by the kernel before the planner
  const int pw = warp / hkv;
  const int h = warp - pw * hkv;
  const int gr = lane >> 2, tig = lane & 3;
  const float NEG_INF = -__int_as_float(0x7f800000);

  uint32_t qb[KS][2];  // Q^T B fragments (f16): head gr, dims tig d/4 + 4 kk + 0..1 and + 2..3
  float fq[2];         // scale log2(e) 2^eq of heads 2tig, 2tig + 1
  float acc[KS][4];    // O^T: dims gr d/8 + 2mt (+1), heads 2tig (+1), in units of 2^(ref - 127)
  float mref[2], lsum[2];
  int ref = 0;         // biased exponent of the V reference; 0: none yet
  int i = i_first;
  int ustart = 0, unext = 0, ctx = 0, npages = 0;
  int64_t tq = 0;
  bool seg_start = true;
  bool ok = true;
  const uint32_t stage_base = smem_u32(stages);
  const bool hv = gr < G;
  // the next segment's entry and its raw q row are read while this segment runs
  int nx_unext = 0, nx_ctx = 0;
  int64_t nx_tq = 0;
  uint4 nx_q[KS / 2];
  bool nx_pending = false, nx_have_q = false;
  int chunks = 1, slot0 = 0;
  auto read_q = [&](int64_t row_tq, uint4 (&dst)[KS / 2]) {
    const uint4* qrow = reinterpret_cast<const uint4*>(
        p.q + row_tq * p.q_st + static_cast<int64_t>(h * G + (hv ? gr : 0)) * p.q_sh + tig * (D / 4));
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) dst[x] = hv ? qrow[x] : make_uint4(0u, 0u, 0u, 0u);
  };
  // q 2^-eq in f16, eq putting the head's largest magnitude in [2^14, 2^15)
  auto take_q = [&](const uint4 (&raw)[KS / 2]) {
    unsigned mx = 0;
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) {
      const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) mx = max(mx, max(w[y] & 0x7fffu, (w[y] >> 16) & 0x7fffu));
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = min(max(static_cast<int>(mx >> 7), 30), 254);  // biased exponent of the largest
    const float up = q8_exp2(127 + 14 + 127 - e);              // 2^(14 - (e - 127))
#pragma unroll
    for (int x = 0; x < KS / 2; ++x) {
      const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) qb[2 * x + (y >> 1)][y & 1] = pack_f16x2(bf16lo(w[y]) * up, bf16hi(w[y]) * up);
    }
    const float f = p.qscale * q8_exp2(e - 14);
    fq[0] = __shfl_sync(0xffffffffu, f, (2 * tig) << 2);  // head 2 tig is lane group gr = 2 tig's
    fq[1] = __shfl_sync(0xffffffffu, f, (2 * tig + 1) << 2);
  };
  int s = 0;
  uint32_t phase = 0;
  for (int u = ubeg; u < uend; ++u) {
    if (seg_start) {
      if (i == i_first) {
        ustart = rec0.y;
        unext = rec0.z;
        ctx = rec1.x;
        tq = rec1.y;
      } else {
        ustart = unext;
        unext = nx_unext;
        ctx = nx_ctx;
        tq = nx_tq;
      }
      if (!nx_have_q) read_q(tq, nx_q);
      take_q(nx_q);
      npages = ceil_div(ctx, 16);
      chunks = p.plan.dec_chunks[i];
      slot0 = p.plan.dec_slot[i];
      nx_pending = unext < uend;
      nx_have_q = false;
      if (nx_pending) {
        nx_unext = dec_unit[i + 2];
        nx_ctx = p.plan.dec_ctx[i + 1];
        nx_tq = p.plan.dec_tq[i + 1];
      }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
      mref[0] = mref[1] = NEG_INF;
      lsum[0] = lsum[1] = 0.f;
      ref = 0;
      seg_start = false;
    }
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
      if (__any_sync(0xffffffffu, pm0 > mref[0] + kQ8Slack || pm1 > mref[1] + kQ8Slack)) {
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
      const float b0 = (mref[0] == NEG_INF ? 0.f : mref[0]) - kQ8Lift, b1 = (mref[1] == NEG_INF ? 0.f : mref[1]) - kQ8Lift;
      sc[0] = fast_exp2(sc[0] - b0);
      sc[1] = fast_exp2(sc[1] - b1);
      sc[2] = fast_exp2(sc[2] - b0);
      sc[3] = fast_exp2(sc[3] - b1);
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
          ref = top;
        } else if (top - ref > kQ8RefHigh || min(ea, eb) - ref < kQ8RefLow) {  // (warp-uniform)
          // the reference moves to this page's scale, unless that is too far down to count
          const int sh = ref - top;
          if (sh <= kQ8MaxDown) {
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
    if (++s == STAGES) {
      s = 0;
      phase ^= 1;
    }
    if (nx_pending && !nx_have_q) {
      read_q(nx_tq, nx_q);
      nx_have_q = true;
    }
    const bool seg_end = (u + 1 == unext) || (u + 1 == uend);
    if (!seg_end) continue;

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
    float* xb = xbuf + warp * G * (D + 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int hh = 2 * tig + j;
      if (hh < G) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
          *reinterpret_cast<float2*>(xb + hh * (D + 2) + gr * (D / 8) + 2 * mt) =
              make_float2(acc[mt][j] * kDown * unit, acc[mt][2 + j] * kDown * unit);
        if (gr == 0) {
          xb[hh * (D + 2) + D] = mref[j] + (15.f - kQ8Lift);
          xb[hh * (D + 2) + D + 1] = (j ? L1 : L0) * kDown;
        }
      }
    }
    named_bar_sync(1, kDecodeWarps * 32);
    {
      const int slot = slot0 + (static_cast<int>(blockIdx.x) - ustart / W);
      for (int item = threadIdx.x; item < hkv * G * (D / 4); item += kDecodeWarps * 32) {
        const int hh = item / (G * (D / 4));
        const int rem3 = item - hh * G * (D / 4);
        const int g = rem3 / (D / 4);
        const int d0 = (rem3 - g * (D / 4)) * 4;
        float M = NEG_INF;
        for (int k = 0; k < wpp; ++k) M = fmaxf(M, xbuf[((hh + k * hkv) * G + g) * (D + 2) + D]);
        float num[4] = {0.f, 0.f, 0.f, 0.f};
        float den = 0.f;
        for (int k = 0; k < wpp; ++k) {
          const float* e = xbuf + ((hh + k * hkv) * G + g) * (D + 2);
          const float w = fast_exp2(e[D] - M);  // a warp with no pages: m = -inf -> w = 0
          den = fmaf(w, e[D + 1], den);
#pragma unroll
          for (int x = 0; x < 4; ++x) num[x] = fmaf(w, e[d0 + x], num[x]);
        }
        const int hq = hh * G + g;
        if (chunks == 1) {
          const float inv = 1.f / den;
          uint2 o;
          o.x = pack_bf16x2(num[0] * inv, num[1] * inv);
          o.y = pack_bf16x2(num[2] * inv, num[3] * inv);
          *reinterpret_cast<uint2*>(p.out + tq * p.o_st + static_cast<int64_t>(hq) * p.o_sh + d0) = o;
        } else {
          const int64_t sh = static_cast<int64_t>(slot) * p.hq + hq;
          *reinterpret_cast<float4*>(p.plan.part_acc + sh * D + d0) = make_float4(num[0], num[1], num[2], num[3]);
          if (d0 == 0) *reinterpret_cast<float2*>(p.plan.part_ml + sh * 2) = make_float2(M, den);
        }
      }
    }
    named_bar_sync(1, kDecodeWarps * 32);
    if (chunks > 1) finish_split<D>(p, i, tq, chunks, slot0, last_flag);
    seg_start = true;
    ++i;
  }
}

template <int D, int FMT, bool TWO>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  using C = DecodeQ8Cfg<D>;
  // (the largest any group needs, so the limit is raised once)
  if (const cudaError_t e = set_smem_once<decode_q8_kernel<D, FMT, TWO>>(C::kSmemLimit); e != cudaSuccess) return e;
  DecodeQ8Params P;
  if (!make_pool_map_heads_q8(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D) ||
      !make_pool_map_heads_q8(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D))
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
  P.stages = C::stages(P.group);
  record_kernel_event(PKV_KERNEL_DECODE, false, stream);
  const cudaError_t e = launch_pdl(decode_q8_kernel<D, FMT, TWO>, dim3(a.decode_ctas), dim3((kDecodeWarps + 1) * 32),
                                   C::smem_bytes(P.group), stream, P);
  record_kernel_event(PKV_KERNEL_DECODE, true, stream);
  return e;
}

template <int D, int FMT>
cudaError_t launch_bs(const AttnArgs& a, cudaStream_t stream) {
  return a.bs_log2 == 3 ? launch<D, FMT, true>(a, stream) : launch<D, FMT, false>(a, stream);
}

}  // namespace

cudaError_t launch_decode_q8(const AttnArgs& a, cudaStream_t stream) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch_bs<128, PKV_Q8_INT8>(a, stream) : launch_bs<64, PKV_Q8_INT8>(a, stream);
  return a.head_dim == 128 ? launch_bs<128, PKV_Q8_E4M3>(a, stream) : launch_bs<64, PKV_Q8_E4M3>(a, stream);
}

}  // namespace pkv
