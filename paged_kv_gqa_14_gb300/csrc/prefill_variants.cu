// Prefill-chunk attention with a position bias, and of differential attention, on the 5th-generation tensor cores.
//
// The causal rule and the stacking of heads are the plain prefill's (prefill_tc.cuh): a Q tile's 128 rows are
// P = floor(128 / G) positions of a span times the G output heads of one kv head (kBias) or pair of them (kDiff).
// A pass is one Q tile against one k head:
//   S = Q K^T  (M 128, N 128, K d),  O += P V  (M 128, N W, K 128)      tcgen05.mma kind::f16, accumulators in TMEM
// with W = d, or for kDiff W = 2 d, the pair's two v heads side by side.  A kDiff item is two passes, one for each
// map; the first leaves its normalised rows in the workspace (fp32, 128 x 2 d, written and read again by the same
// threads, so nothing has to be waited for), the second subtracts, normalises and writes the output.
//
// One CTA of twelve warps, one Q tile at a time:
//   warp 0      Q tile and K tiles of 128 keys (TMA)
//   warp 1      V, in stages of 16 KB (TMA)
//   warp 2, 3   issue of QK^T; of P V (a warp each: what a warp does around its products costs as much as they)
//   warps 4-7   softmax of the even tiles, thread = row; warps 8-11 that of the odd ones
// S has two buffers (three where TMEM has room), each half of the softmax works on its own, and P overlays the S that it
// came from.  Both halves weigh with one reference m of a row, so that one O takes all: m goes from tile to tile
// through shared memory (a half reads the tile before's as soon as that is known, long before its weights are), it is
// raised only when a row's maximum exceeds it by more than 8, and the half that raises it rescales O, once the P V
// of every tile before has landed.  Each half sums its own weights; the sums meet when the pass ends.
//
// TMA boxes are whole blocks of a head, both 64-dim halves and for V both heads of a pair at once: the pool as {64 dims,
// 8 rows, half, head, group of 8 rows} lands as [group][head][half][8 rows][128 bytes], which a shared-memory
// descriptor takes with its own strides.
//
// Every wait is bounded; a CTA that times out sets PKV_DEVERR_TIMEOUT and finishes without further work.
#include <cuda.h>

#include "decode_tc.cuh"
#include "prefill.cuh"
#include "prefill_tc.cuh"
#include "tcgen05.cuh"
#include "variants.cuh"

namespace pkv {

bool make_pool_map_rows8(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D, int heads,
                         int groups);
bool make_q_map_parts(CUtensorMap* m, const AttnArgs& a, int parts);

namespace {

constexpr int kPvThreads = 384;

struct PrefillVarParams {
  CUtensorMap tmap_q;  // 4-D {d, parts (1; kDiff 2), output heads, tokens}, box {64, 1, G, P}
  CUtensorMap tmap_k;  // 5-D {64, 8 rows, d / 64, Hkv, groups of 8 rows}, box {64, 8, all, 1, a block's, 16 at most}
  CUtensorMap tmap_v;  // the same, box {64, 8, all, W / d, a block's, a stage's at most}
  PrefillParams p;
  int group;  // G
  int prows;  // P
  BiasArgs bias;
  DiffArgs diff;
};

template <int D, int V>
struct PrefillVarCfg {
  static constexpr int BK = 128;
  static constexpr int W = V == kDiff ? 2 * D : D;
  static constexpr int HALVES = D / 64;
  static constexpr int CB = W / 64;                // 64-column blocks of O
  static constexpr int kQHalf = 128 * 128;         // [128 rows][64 dims]
  static constexpr int kQBytes = HALVES * kQHalf;
  static constexpr int kKTile = BK * D * 2;
  static constexpr int KST = D == 128 ? 2 : 4;     // K stages
  static constexpr int kVStage = 16384;
  static constexpr int VG = kVStage / (2 * W);     // keys of a V stage: 32, 64 or 128
  static constexpr int GPT = BK / VG;              // V stages of a tile
  static constexpr int VST = V == kDiff ? (D == 128 ? 7 : 6) : (D == 128 ? 5 : 4);
  static constexpr int NS = W == 256 ? 2 : 3;      // S buffers of 128 columns
  static constexpr uint32_t COL_O = 128 * NS;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + kQBytes;
  static constexpr int OFF_V = OFF_K + KST * kKTile;
  static constexpr int OFF_M = OFF_V + VST * kVStage;  // [2][128] m of the last tile of either half
  static constexpr int OFF_EX = OFF_M + 1024;          // [2][2][128] exchanges at the end of a pass
  static constexpr int OFF_IDX = OFF_EX + 2048;        // (kBias) bucket of each distance, bytes
  static constexpr int OFF_TAB = OFF_IDX + (V == kBias ? kMaxBucketStart + 16 : 0);  // (kBias) [bucket][head] log2 domain
  static constexpr int OFF_BAR = OFF_TAB + (V == kBias ? kMaxBuckets * 64 * 4 : 0);
  static constexpr int kSmemBytes = OFF_BAR + 512 + 1024;  // + barriers + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(COL_O + W <= 512, "TMEM columns");
};

__device__ __forceinline__ void tma_load_rows8(void* dst_smem, const CUtensorMap* map, int head, int rowgroup,
                                               uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(rowgroup), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_q(void* dst_smem, const CUtensorMap* map, int c0, int part, int head, int token,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(part), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}

template <int D, int V>
__global__ void __launch_bounds__(kPvThreads, 1) prefill_variant_kernel(const __grid_constant__ PrefillVarParams P) {
  using C = PrefillVarCfg<D, V>;
  constexpr int W = C::W, NS = C::NS, KST = C::KST, VST = C::VST, HALVES = C::HALVES;
  const PrefillParams& p = P.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  float* mref = reinterpret_cast<float*>(smem + C::OFF_M);
  float* exch = reinterpret_cast<float*>(smem + C::OFF_EX);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;       // a pass's every QK completed
  uint64_t* k_full = bars + 2;        // [4]
  uint64_t* k_empty = bars + 6;       // [4]
  uint64_t* v_full = bars + 10;       // [8]
  uint64_t* v_empty = bars + 18;      // [8]
  uint64_t* s_full = bars + 26;       // [3] S buffer written
  uint64_t* p_full = bars + 29;       // [3] P written over it
  uint64_t* pv_done = bars + 32;      // [3] the P V that reads it completed
  uint64_t* o_free = bars + 35;       // O of a pass is read
  uint64_t* m_known = bars + 36;      // [2][4] a half's warp has written the tile's m
  uint64_t* pair = bars + 44;         // [4] the two warps of the same rows at the end of a pass
  uint64_t* fin = bars + 48;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 49);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 50);
  static_assert(KST <= 4 && VST <= 8 && NS <= 3, "barrier layout");
  const float NEG_INF = -__int_as_float(0x7f800000);

  // (a shuffle's result is uniform to the compiler, and so is what follows from it)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < KST; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
    for (int i = 0; i < VST; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1);
    for (int i = 0; i < NS; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4), mbar_init(&pv_done[i], 1);
    mbar_init(o_free, 8);
    for (int i = 0; i < 8; ++i) mbar_init(&m_known[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 2);
    mbar_init(fin, 2);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_v)) : "memory");
  }
  if (warp == 2) {  // while the planner still runs
    tc5::alloc(tmem_slot, 512);
    tc5::relinquish();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  pdl_wait();
  pdl_trigger();
  const int hp = V == kDiff ? p.hkv / 2 : p.hkv;  // items of a Q tile's positions
  const int total = uniform(p.plan.header[3]) * hp;
  const int nact = min(max(uniform(p.plan.header[5]), 0), static_cast<int>(gridDim.x));
  if (static_cast<int>(blockIdx.x) >= total || static_cast<int>(blockIdx.x) >= nact) {  // no item in any wave
    if (warp == 2) tc5::dealloc(tmem, 512);
    return;
  }
  const int far = V == kBias ? P.bias.starts[P.bias.num_buckets - 1] : 0;  // the last bucket's first distance
  if (V == kBias) {
    // the bucket of each distance up to `far`, and the biases in the log2 domain
    for (int i = warp; i < P.bias.num_buckets; i += kPvThreads / 32) {
      const int end = i + 1 < P.bias.num_buckets ? P.bias.starts[i + 1] : far + 1;
      for (int n = P.bias.starts[i] + lane; n < end; n += 32) smem[C::OFF_IDX + n] = static_cast<unsigned char>(i);
    }
    float* tab = reinterpret_cast<float*>(smem + C::OFF_TAB);
    for (int i = threadIdx.x; i < P.bias.num_buckets * p.hq; i += kPvThreads)
      tab[i] = bias_at(P.bias, i / p.hq, i % p.hq);
    __syncthreads();
  }
  const int G = P.group;
  const int PR = P.prows;
  const uint64_t pol = l2_policy_evict_last();  // K/V tiles are read again by the other items

  // every role walks the CTA's passes by itself: body(pass)
  struct Pass {
    int no, item_no;  // passes and tiles of this CTA before this one
    int t0, g0;       // tiles, V stages before it
    int h, part;      // kv head or pair; map
    int b, s0, q0, pos0, rows, kv_end, nkt;
  };
  constexpr int kParts = V == kDiff ? 2 : 1;
  auto for_passes = [&](auto&& body) {
    Pass it;
    it.no = it.t0 = it.g0 = 0;
    for (int wave = 0; wave * nact < total; ++wave) {
      const int ord = snake_order(wave, blockIdx.x, nact);
      if (ord >= total) continue;
      const int item = total - 1 - ord;  // later (longer) tiles of each span first
      const int ti = item / hp;
      it.h = item - ti * hp;
      it.b = uniform(p.plan.pf_seq[ti]);
      it.s0 = uniform(p.qsl[it.b]);
      const int n = uniform(p.qsl[it.b + 1]) - it.s0;
      it.q0 = uniform(p.plan.pf_tile[ti]) * PR;
      it.pos0 = uniform(p.context_lens[it.b]) - n + it.q0;
      it.rows = min(PR, n - it.q0);
      it.kv_end = it.pos0 + it.rows;  // keys [0, kv_end) are visible to some row
      it.nkt = ceil_div(it.kv_end, C::BK);
      for (it.part = 0; it.part < kParts; ++it.part) {
        body(it);
        it.t0 += it.nkt;
        it.g0 += ceil_div(it.kv_end, C::VG);
        ++it.no;
      }
    }
  };
  const int bs = 1 << p.bs_log2;

  // Registers: 72 + 216 + 216 a thread of the three warpgroups, the 3 x 168 of the launch.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const uint32_t one = lane == 0;
    if (warp == 0) {
      // ------------------------------------------------------------- Q and K by TMA
      int q_issued = 0, k_issued = 0;
      for_passes([&](const Pass& it) {
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        auto fetch = [&](int jt) -> int {  // the block of this lane's box of tile jt
          const int key0 = jt * C::BK + lane * bs;
          return (jt < it.nkt && lane * bs < C::BK && key0 < it.kv_end) ? btrow[key0 >> p.bs_log2] : 0;
        };
        bool ok = !*abort_flag;
        int nb0 = fetch(0), nb1 = fetch(1);
        if (ok && it.no > 0) ok = warp_wait(q_empty, (it.no - 1) & 1, p.err, abort_flag);
        if (ok) {
          if (lane == 0) mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(HALVES * G * PR * 128));
          __syncwarp();
          if (lane < HALVES)
            tma_load_q(smem + C::OFF_Q + lane * C::kQHalf, &P.tmap_q, lane * 64, it.part, it.h * G, it.s0 + it.q0, q_full);
          ++q_issued;
        }
        const int head = V == kDiff ? 2 * it.h + it.part : it.h;
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          int blk = nb0;
          nb0 = nb1;
          nb1 = fetch(jt + 2);
          const int f = it.t0 + jt, ks = f % KST;
          if (f >= KST) ok = warp_wait(&k_empty[ks], (f / KST - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          const int nbox = ceil_div(min(C::BK, it.kv_end - jt * C::BK), bs);
          if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], static_cast<uint32_t>(nbox * bs * D * 2));
          __syncwarp();
          if (lane < nbox) {
            if (blk < 0 || blk >= p.num_blocks) {
              raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
              blk = 0;
            }
            tma_load_rows8(smem + C::OFF_K + ks * C::kKTile + lane * bs * D * 2, &P.tmap_k, head, blk << (p.bs_log2 - 3),
                           &k_full[ks], pol);
          }
          k_issued = f + 1;
        }
      });
      // every copy issued has landed before the CTA may leave, also after another role has given up
      if (q_issued > 0) mbar_wait(q_full, (q_issued - 1) & 1, p.err);
      for (int f = max(0, k_issued - KST); f < k_issued; ++f) mbar_wait(&k_full[f % KST], (f / KST) & 1, p.err);
    } else if (warp == 1) {
      // -------------------------------------------------------------------- V by TMA
      int issued = 0;
      const int box = min(bs, C::VG);  // rows of a box
      const int nbox_all = C::VG / box;
      for_passes([&](const Pass& it) {
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        const int ng = ceil_div(it.kv_end, C::VG);
        auto fetch = [&](int g) -> int {
          const int key0 = g * C::VG + lane * box;
          return (g < ng && lane < nbox_all && key0 < it.kv_end) ? btrow[key0 >> p.bs_log2] : 0;
        };
        bool ok = !*abort_flag;
        int nb0 = fetch(0), nb1 = fetch(1), nb2 = fetch(2);
        const int head = V == kDiff ? 2 * it.h : it.h;
        for (int g = 0; g < ng && ok; ++g) {
          int blk = nb0;
          nb0 = nb1;
          nb1 = nb2;
          nb2 = fetch(g + 3);
          const int f = it.g0 + g, vs = f % VST;
          if (f >= VST) ok = warp_wait(&v_empty[vs], (f / VST - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          const int nbox = ceil_div(min(C::VG, it.kv_end - g * C::VG), box);
          if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], static_cast<uint32_t>(nbox * box * W * 2));
          __syncwarp();
          if (lane < nbox) {
            if (blk < 0 || blk >= p.num_blocks) {
              raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
              blk = 0;
            }
            const int in_block = (g * C::VG + lane * box) & (bs - 1);
            tma_load_rows8(smem + C::OFF_V + vs * C::kVStage + lane * box * W * 2, &P.tmap_v, head,
                           (blk << (p.bs_log2 - 3)) + (in_block >> 3), &v_full[vs], pol);
          }
          issued = f + 1;
        }
      });
      for (int f = max(0, issued - VST); f < issued; ++f) mbar_wait(&v_full[f % VST], (f / VST) & 1, p.err);
    } else if (warp == 2) {
      // ------------------------------------------------------------------- S = Q K^T
      constexpr uint32_t kIdesc = tc5::idesc_bf16_f32(128, 128);
      const uint64_t qd = tc5::smem_desc_sw128(sb + C::OFF_Q, 16, 1024);
      const uint64_t kd0 = tc5::smem_desc_sw128(sb + C::OFF_K, 16, HALVES * 1024);
      for_passes([&](const Pass& it) {
        bool ok = warp_wait(q_full, it.no & 1, p.err, abort_flag);
#pragma unroll 1
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          const int f = it.t0 + jt, ks = f % KST, sbuf = f % NS;
          ok = warp_wait(&k_full[ks], (f / KST) & 1, p.err, abort_flag);
          // (the P V that reads the P that this S overwrites)
          if (ok && f >= NS) ok = warp_wait(&pv_done[sbuf], (f / NS - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          tc5::fence_after();
          const uint64_t kd = kd0 + static_cast<uint32_t>(ks * (C::kKTile >> 4));
          const uint32_t sd = tmem + 128u * sbuf;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t qo = (kk >> 2) * static_cast<uint64_t>(C::kQHalf >> 4) + (kk & 3) * static_cast<uint64_t>(32 >> 4);
            const uint64_t ko = (kk >> 2) * static_cast<uint64_t>(1024 >> 4) + (kk & 3) * static_cast<uint64_t>(32 >> 4);
            if (kk == 0)
              tc5::mma_ss_warp<false>(one, sd, qd, kd, kIdesc);
            else
              tc5::mma_ss_warp<true>(one, sd, qd + qo, kd + ko, kIdesc);
          }
          tc5::commit_warp(one, &s_full[sbuf]);
          tc5::commit_warp(one, &k_empty[ks]);
          if (jt == it.nkt - 1) tc5::commit_warp(one, q_empty);
        }
      });
      tc5::commit_warp(one, fin);
      __syncwarp();
    } else {
      // --------------------------------------------------------------------- O += P V
      constexpr uint32_t kIdesc = tc5::idesc_bf16_f32(128, W, true);
      constexpr uint32_t kRows8 = C::CB * 1024;  // 8 keys of all W columns
      const uint64_t vd0 = tc5::smem_desc_sw128(sb + C::OFF_V, 1024, kRows8);
      const uint32_t od = tmem + C::COL_O;
      for_passes([&](const Pass& it) {
        bool ok = !*abort_flag;
#pragma unroll 1
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          const int f = it.t0 + jt, sbuf = f % NS;
          ok = warp_wait(&p_full[sbuf], (f / NS) & 1, p.err, abort_flag);
          // (a pass's first P V overwrites O)
          if (ok && jt == 0 && it.no > 0) ok = warp_wait(o_free, (it.no - 1) & 1, p.err, abort_flag);
          const uint32_t pt = tmem + 128u * sbuf;
#pragma unroll 1
          for (int g = 0; g < C::GPT && ok; ++g) {
            const int vis = it.kv_end - jt * C::BK - g * C::VG;  // keys of the stage that some row sees
            if (vis <= 0) break;
            const int gi = it.g0 + jt * C::GPT + g, vs = gi % VST;
            ok = warp_wait(&v_full[vs], (gi / VST) & 1, p.err, abort_flag);
            if (!ok) break;
            if (vis < C::VG) {
              // keys that no row sees: zero, so that 0 * (unused slot) cannot poison O
              unsigned char* vb = smem + C::OFF_V + vs * C::kVStage;
              for (int idx = lane; idx < (C::VG - vis) * C::CB * 8; idx += 32) {
                const int t = vis + idx / (C::CB * 8), c = idx % (C::CB * 8);
                *reinterpret_cast<uint4*>(vb + (t >> 3) * kRows8 + (c >> 3) * 1024 + (t & 7) * 128 + ((c & 7) << 4)) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc5::fence_after();
            const uint64_t vd = vd0 + static_cast<uint32_t>(vs * (C::kVStage >> 4));
            const uint32_t pg = pt + static_cast<uint32_t>(g * (C::VG / 2));  // two keys to a column
            if (jt == 0 && g == 0)
              tc5::mma_ts_warp<false>(one, od, pg, vd, kIdesc);
            else
              tc5::mma_ts_warp<true>(one, od, pg, vd, kIdesc);
#pragma unroll
            for (int kk = 1; kk < C::VG / 16; ++kk)
              tc5::mma_ts_warp<true>(one, od, pg + 8u * kk, vd + kk * static_cast<uint64_t>(2 * kRows8 >> 4), kIdesc);
            tc5::commit_warp(one, &v_empty[vs]);
          }
          if (ok) tc5::commit_warp(one, &pv_done[sbuf]);
        }
      });
      tc5::commit_warp(one, fin);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ------------------------------------------------------------------------ softmax
    const int wg = (warp - 4) >> 2;  // the half: tiles of this parity
    const int sw = warp & 3;         // TMEM lanes 32 sw .. 32 sw + 31
    const int r = 32 * sw + lane;
    const int rt = r / G;       // position within the Q tile
    const int rg = r - rt * G;  // member of the group
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * sw) << 16);
    const uint32_t to = tlane + C::COL_O;
    const float* tab = reinterpret_cast<const float*>(smem + C::OFF_TAB);
    const unsigned char* idx = smem + C::OFF_IDX;
    int ex_no = 0;  // exchanges with the other half's warp so far
    // x of this warp's rows against the other half's, through shared memory; false: a wait gave up
    auto exchange = [&](float x, float& other) -> bool {
      float* slot = exch + (ex_no & 1) * 256;
      slot[wg * 128 + r] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pair[sw]);
      const bool ok = warp_wait(&pair[sw], ex_no & 1, p.err, abort_flag);
      other = slot[(1 - wg) * 128 + r];
      ++ex_no;
      return ok;
    };
    for_passes([&](const Pass& it) {
      const bool live = rt < it.rows;
      // (a row past the span's sees everything: its scores need no mask and go nowhere)
      const int pos = live ? it.pos0 + rt : INT32_MAX;
      const int posb = live ? it.pos0 + rt : it.kv_end - 1;
      const int bh = V == kBias ? it.h * G + (live ? rg : 0) : 0;  // the bias's head
      const float cfar = V == kBias ? tab[(P.bias.num_buckets - 1) * p.hq + bh] : 0.f;
      // (a bias that would swallow scores is added to each, so that it does)
      const bool cfar_large = V == kBias && fabsf(cfar) > 1048576.f && cfar != NEG_INF;
      float m_own = NEG_INF, l_run = 0.f;
      bool ok = !*abort_flag;
      const int first = (it.t0 + wg) & 1;  // this half's first tile of the pass
#pragma unroll 1
      for (int jt = first; jt < it.nkt && ok; jt += 2) {
        const int f = it.t0 + jt, sbuf = f % NS;
        const uint32_t ts = tlane + 128u * sbuf;
        ok = warp_wait(&s_full[sbuf], (f / NS) & 1, p.err, abort_flag);
        if (!ok) break;
        tc5::fence_after();
        float sc[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tc5::ld32(ts + 32u * c, v);
#pragma unroll
          for (int x = 0; x < 32; ++x) sc[32 * c + x] = v[x];
        }
        tc5::wait_ld();
        const int key0 = jt * C::BK;
        float mul = p.qscale, add = cfar;
        if (V == kBias && __any_sync(0xffffffffu, posb - (key0 + C::BK - 1) < far || cfar_large)) {
          // some key is nearer than the last bucket
          const float* tb = tab + bh;
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const int n = min(max(posb - key0 - c, 0), far);
            sc[c] = fmaf(sc[c], p.qscale, tb[idx[n] * p.hq]);
          }
          mul = 1.f;
          add = 0.f;
        }
        if (__any_sync(0xffffffffu, key0 + C::BK - 1 > pos)) {
          const int last = pos - key0;  // (may be negative: none)
#pragma unroll
          for (int c = 0; c < 128; ++c) sc[c] = c <= last ? sc[c] : NEG_INF;
        }
        float mx8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(sc[x], sc[8 + x]);
#pragma unroll
        for (int c = 16; c < 128; c += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(fmaxf(mx8[x], sc[c + x]), sc[c + 8 + x]);
        const float mraw = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const float mx = V == kBias ? fmaf(mraw, mul, add) : mraw * mul;  // (-inf stays -inf)
        // the row's m after the tile before, which the other half has
        float m_prev = NEG_INF;
        if (jt > 0) {
          ok = warp_wait(&m_known[(1 - wg) * 4 + sw], ((f - 1) >> 1) & 1, p.err, abort_flag);
          if (!ok) break;
          m_prev = mref[(1 - wg) * 128 + r];
        }
        const bool up = mx - m_prev > kVarSlack;
        const float m_new = up ? mx : m_prev;
        mref[wg * 128 + r] = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m_known[wg * 4 + sw]);
        const bool any_up = __any_sync(0xffffffffu, up);
        const float corr = up ? fast_exp2(m_prev - m_new) : 1.f;
        l_run *= m_own == m_new ? 1.f : fast_exp2(m_own - m_new);
        m_own = m_new;
        const float base = m_new == NEG_INF ? 0.f : m_new;
        // weights 2^(s - m), rounded to bf16 for P V; l sums the rounded ones, so that they add up to 1
        const float2 mul2 = make_float2(mul, mul);
        const float2 add2 = make_float2(add - base, add - base);
        float2 ls4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ls4[x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float pk[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float2 t = ffma2(make_float2(sc[64 * c + 2 * x], sc[64 * c + 2 * x + 1]), mul2, add2);
            const uint32_t w = pack_bf16x2(fast_exp2(t.x), fast_exp2(t.y));
            ls4[x & 3] = fadd2(ls4[x & 3], make_float2(bf16lo(w), bf16hi(w)));
            pk[x] = __uint_as_float(w);
          }
          tc5::st32(ts + 32u * c, pk);  // P over S: column c holds keys 2c, 2c + 1
        }
        const float2 ls2 = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
        l_run += ls2.x + ls2.y;
        if (jt > 0 && any_up) {
          // O is rescaled once the P V of every tile before has landed in it
          ok = warp_wait(&pv_done[(f - 1) % NS], ((f - 1) / NS) & 1, p.err, abort_flag);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll 1
          for (int c = 0; c < W / 32; ++c) {
            float o[32];
            tc5::ld32(to + 32u * c, o);
            tc5::wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= corr;
            tc5::st32(to + 32u * c, o);
          }
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sbuf]);
      }
      // ------------------------------------------------------------- the pass's rows
      const int last = it.t0 + it.nkt - 1;  // its last tile, and the half that had it
      float M = m_own;
      if (ok && (last & 1) != wg) {
        ok = warp_wait(&m_known[(1 - wg) * 4 + sw], (last >> 1) & 1, p.err, abort_flag);
        M = mref[(1 - wg) * 128 + r];
      }
      l_run *= m_own == M ? 1.f : fast_exp2(m_own - M);
      float l_other = 0.f;
      if (ok) ok = exchange(l_run, l_other);
      if (ok) ok = warp_wait(&pv_done[last % NS], (last / NS) & 1, p.err, abort_flag);
      if (!ok) return;
      tc5::fence_after();
      const float inv = inverse_or_0(l_run + l_other);
      constexpr int HW = W / 2;  // columns of either half
      const uint32_t tc = to + static_cast<uint32_t>(wg * HW);
      const int row = it.s0 + it.q0 + rt;
      const int head = it.h * G + rg;
      bf16* orow = p.out + static_cast<int64_t>(row) * p.o_st + static_cast<int64_t>(head) * p.o_sh + wg * HW;
      float o[HW];
#pragma unroll
      for (int c = 0; c < HW / 32; ++c) {
        float v[32];
        tc5::ld32(tc + 32u * c, v);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[32 * c + x] = v[x];
      }
      tc5::wait_ld();
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);  // O is read: the next pass's P V may overwrite it
      if (V == kDiff) {
        float4* own = reinterpret_cast<float4*>(p.plan.scratch) +
                      (static_cast<int64_t>(blockIdx.x) * (W / 4) + wg * (HW / 4)) * 128 + r;
        if (it.part == 0) {
#pragma unroll
          for (int c = 0; c < HW / 4; ++c)
            own[c * 128] = make_float4(o[4 * c] * inv, o[4 * c + 1] * inv, o[4 * c + 2] * inv, o[4 * c + 3] * inv);
          return;
        }
        const float la = live ? P.diff.lambda[static_cast<int64_t>(row) * P.diff.lambda_st + head] * inv : 0.f;
#pragma unroll
        for (int c = 0; c < HW / 4; ++c) {
          const float4 a = own[c * 128];
          o[4 * c] = a.x - la * o[4 * c];
          o[4 * c + 1] = a.y - la * o[4 * c + 1];
          o[4 * c + 2] = a.z - la * o[4 * c + 2];
          o[4 * c + 3] = a.w - la * o[4 * c + 3];
        }
        float scale = P.diff.out_scale;
        if (P.diff.norm_weight) {
          float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < HW; ++c) ss[c & 3] = fmaf(o[c], o[c], ss[c & 3]);
          const float mine = (ss[0] + ss[1]) + (ss[2] + ss[3]);
          float theirs = 0.f;
          if (!exchange(mine, theirs)) return;
          // (the same sum in both halves)
          scale *= 1.f / sqrtf((wg == 0 ? mine + theirs : theirs + mine) * (1.f / W) + P.diff.norm_eps);
          const float4* nw = reinterpret_cast<const float4*>(P.diff.norm_weight + wg * HW);
#pragma unroll
          for (int c = 0; c < HW / 4; ++c) {
            const float4 w = __ldg(nw + c);
            o[4 * c] *= w.x, o[4 * c + 1] *= w.y, o[4 * c + 2] *= w.z, o[4 * c + 3] *= w.w;
          }
        }
#pragma unroll
        for (int c = 0; c < HW; ++c) o[c] *= scale;
      } else {
#pragma unroll
        for (int c = 0; c < HW; ++c) o[c] *= inv;
      }
      if (live) {
#pragma unroll
        for (int x = 0; x < HW / 8; ++x) {
          uint4 u;
          u.x = pack_bf16x2(o[8 * x + 0], o[8 * x + 1]);
          u.y = pack_bf16x2(o[8 * x + 2], o[8 * x + 3]);
          u.z = pack_bf16x2(o[8 * x + 4], o[8 * x + 5]);
          u.w = pack_bf16x2(o[8 * x + 6], o[8 * x + 7]);
          *reinterpret_cast<uint4*>(orow + 8 * x) = u;
        }
      }
    });
  }
  __syncthreads();  // every role has finished its last pass
  if (warp == 2) {  // no MMA may be in flight when TMEM is released
    mbar_wait(fin, 0, p.err);
    __syncwarp();
    tc5::fence_after();
    tc5::dealloc(tmem, 512);
  }
}

template <int D, int V>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  using C = PrefillVarCfg<D, V>;
  if (const cudaError_t e = set_smem_once<prefill_variant_kernel<D, V>>(C::kSmemBytes); e != cudaSuccess) return e;
  PrefillVarParams P{};
  const int bs8 = 1 << (a.bs_log2 - 3);  // groups of 8 rows of a block
  const int heads = V == kDiff ? 2 : 1;
  if (!make_q_map_parts(&P.tmap_q, a, heads) ||
      !make_pool_map_rows8(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D, 1, bs8) ||
      !make_pool_map_rows8(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D, heads,
                           bs8 < C::VG / 8 ? bs8 : C::VG / 8))
    return cudaErrorInvalidValue;
  P.p = make_prefill_params(a);
  P.group = a.hq / a.hkv;
  P.prows = kTcPrefillRows / P.group;
  if (a.bias) P.bias = *a.bias;
  if (a.diff) P.diff = *a.diff;
  record_kernel_event(PKV_KERNEL_PREFILL, false, stream);
  const cudaError_t e = launch_kernel(pdl, prefill_variant_kernel<D, V>, dim3(static_cast<unsigned>(prefill_variant_grid(a))),
                                      dim3(kPvThreads), C::kSmemBytes, stream, P);
  record_kernel_event(PKV_KERNEL_PREFILL, true, stream);
  return e;
}

}  // namespace

// One CTA per SM, at most one per item.
int64_t prefill_variant_grid(const AttnArgs& a) {
  const int prows = kTcPrefillRows / (a.hq / a.hkv);
  const int64_t max_items = (a.num_tokens / prows + a.num_seqs + 1) * (a.variant == kDiff ? a.hkv / 2 : a.hkv);
  const int64_t cap = device_sm_count();
  return max_items < cap ? max_items : cap;
}

cudaError_t launch_prefill_variant(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  if (a.variant == kBias)
    return a.head_dim == 128 ? launch<128, kBias>(a, stream, pdl) : launch<64, kBias>(a, stream, pdl);
  return a.head_dim == 128 ? launch<128, kDiff>(a, stream, pdl) : launch<64, kDiff>(a, stream, pdl);
}

}  // namespace pkv
