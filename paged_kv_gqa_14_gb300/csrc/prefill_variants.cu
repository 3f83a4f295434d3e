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
// One CTA of sixteen warps, one Q tile at a time:
//   warp 0      Q tile and K tiles of 128 keys (TMA)
//   warp 1      V, in stages of 16 KB (TMA)
//   warps 2, 3  issue of S = Q K^T, of the even and of the odd tiles
//   warp 4 (5)  issue of O += P V (at W 256 a warp for either half of the columns)
//   warps 8-15  softmax, two threads to a row: warps 8-11 the first 64 keys of a tile, warps 12-15 the others
// (A product is issued at the pace at which the tensor cores take it, and a wait costs a warp 60 to 100 clocks even where
// there is nothing to wait for: one warp for all products took 3800 clocks a tile, two 2350, of which the products are 1536.)
// S is free again once the softmax has read it into registers, and P has two buffers of its own, so the tensor cores run
// ahead of the softmax by a tile or two (one S buffer at W 256, two where TMEM has room).  A row's two threads exchange their
// maxima through shared memory, so that both weigh with one reference m and one O takes all; m is raised only when a
// score exceeds it, to 20 above (kVarSlack), and O is rescaled then, once the P V of every tile before has landed (either half
// of the columns by one of the two warps).  Each thread sums its own weights; the sums meet when the pass ends.
// (Whole rows to a thread, the tiles to the two halves in turn: with one S buffer the next S then waits until a half is free to
// read this one, 1109 us for a differential chunk of 3528 tokens behind 12,288 keys, 28/4 heads d 128.)
//
// Few items behind long contexts: up to four pairs of CTAs, a cluster, take an item together, a range of its key tiles each,
// and join through distributed shared memory (the difference's first map through its workspace).  GB300, four spans of 12
// behind 7000 keys as a difference, 24/4 heads d 64: 45 us, by one pair each 113; pieces of fewer than 8 / share tiles are not
// made, since the joining takes 2 to 3 us.
//
// Two CTAs of a cluster take an item together, two Q tiles of the same span and heads, each with copies of K and V of its
// own.  (They share nothing, but run beside each other at the same keys: as CTAs without clusters the prompts below took 128
// us for 119, a late chunk with the bias 696 for 675 and the differential one 861 for 840.)
//
// TMA boxes are whole blocks of a head, both 64-dim halves and for V both heads of a pair at once: the pool as {64 dims,
// 8 rows, half, head, group of 8 rows} lands as [group][head][half][8 rows][128 bytes], which a shared-memory
// descriptor takes with its own strides.
//
// Bound: kDiff the tensor cores (at d 128 1536 clocks of products to a tile that takes about 2000) and what the last round of
// items leaves idle; kBias the softmax (about 2000 clocks a tile; of 1900, before scores were rounded in a step of their own,
// powers were 900, maxima 365, the exchange 230, hand-over and fetch the rest).  GB300, that chunk 852 us (0.66 of the library's bf16 rate); with a bias 3700 tokens 695 us (0.57); five
// prompts of up to 2048 tokens, 14/2 heads d 64, 123 us, where each item's diagonal, first scores and last rows weigh most.
//
// Every wait is bounded; a CTA that times out sets PKV_DEVERR_TIMEOUT and finishes without further work.
#include <cuda.h>

#include <atomic>
#include <type_traits>

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

constexpr int kPvThreads = 512;

struct PrefillVarParams {
  CUtensorMap tmap_q;  // 4-D {d, parts (1; kDiff 2), output heads, tokens}, box {64, 1, G, P}
  CUtensorMap tmap_k;  // 5-D {64, 8 rows, d / 64, Hkv, groups of 8 rows}, box {64, 8, all, 1, a block's}
  CUtensorMap tmap_v;  // the same, box {64, 8, all, W / d, a block's, a stage's at most}
  PrefillParams p;
  int group;  // G
  int prows;  // P
  BiasArgs bias;
  DiffArgs diff;
  int pieces;           // pairs of CTAs in a cluster, which may share an item
  int fault_no_copies;  // test-only: the loaders issue nothing
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
  // Two tiles' worth of stages of either, so that a tile's place in the ring and its phase follow from its number alone:
  // K stage f & 1, V stages from GPT (f & 1) on, all in phase (f >> 1) & 1.
  static constexpr int KST = 2;
  static constexpr int VG = W == 256 ? 32 : 64;    // keys of a V stage
  static constexpr int GPT = BK / VG;              // V stages of a tile
  static constexpr int VST = 2 * GPT;
  static constexpr int kVStage = VG * W * 2;
  static constexpr int PVW = W == 256 ? 2 : 1;     // warps that issue P V, W / PVW columns each
  static constexpr int NS = W == 256 ? 1 : 2;      // S buffers of 128 columns
  static constexpr uint32_t COL_P = 128 * NS;      // P: two buffers of 64 columns
  static constexpr uint32_t COL_O = COL_P + 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + kQBytes;
  static constexpr int OFF_V = OFF_K + KST * kKTile;
  static constexpr int OFF_EX = OFF_V + VST * kVStage;  // [2][2][128] exchanges between the threads of a row
  static constexpr int OFF_IDX = OFF_EX + 2048;         // (kBias) bucket of each distance, bytes
  // (kBias) in the log2 domain, [head][distance], a head's row `tab_row` apart; or where that is too long [bucket][head]
  static constexpr int kTabFloats = kMaxBuckets * 64;
  static constexpr int OFF_TAB = OFF_IDX + (V == kBias ? kMaxBucketStart + 16 : 0);
  static constexpr int OFF_BAR = OFF_TAB + (V == kBias ? kTabFloats * 4 : 0);
  static constexpr int kSmemBytes = OFF_BAR + 512;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(COL_O + W <= 512, "TMEM columns");
};

__device__ __forceinline__ void tma_load_rows8(void* dst_smem, const CUtensorMap* map, int head, int rowgroup, uint64_t* bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(rowgroup), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Shared memory of the cluster's CTA `rank` at this CTA's shared address `a`.
__device__ __forceinline__ uint32_t peer_smem(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 ld_peer_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void tma_load_q(void* dst_smem, const CUtensorMap* map, int c0, int part, int head, int token,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(part), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}

// Every weight is 2^kCutShift larger, which the division by l takes out again: a row's largest, 2^-20, is held exactly and would
// lose nothing in the cut, where the others lose 0.0028 on average (half of 2^-7 / mantissa); a row of few keys would feel that
// (rows of 12 to 14 keys: 0.0025 off the 64-bit result in relative norm, of which the output's rounding is 0.0016).
constexpr float kCutShift = 0.004f;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// SHARE: pairs of a cluster may share an item.  (An instance of its own, since what it adds to every role costs the others'
// long chunks 3 %: 847 us of the differential chunk became 873.)
template <int D, int V, bool SHARE>
__global__ void __launch_bounds__(kPvThreads, 1) prefill_variant_kernel(const __grid_constant__ PrefillVarParams P) {
  using C = PrefillVarCfg<D, V>;
  constexpr int W = C::W, NS = C::NS, KST = C::KST, VST = C::VST, HALVES = C::HALVES;
  const PrefillParams& p = P.p;
  extern __shared__ __align__(1024) unsigned char smem[];  // (swizzle atoms are 1024 bytes; no room for slack at W 256)
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {  // (CTA-uniform; never so far)
    if (threadIdx.x == 0) raise_error(P.p.err, PKV_DEVERR_TIMEOUT);
    return;
  }
  float* exch = reinterpret_cast<float*>(smem + C::OFF_EX);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;       // a pass's every QK completed
  uint64_t* k_full = bars + 2;        // [2]
  uint64_t* k_empty = bars + 4;       // [2]
  uint64_t* v_full = bars + 10;       // [8]
  uint64_t* v_empty = bars + 18;      // [8]
  // of the even and the odd tiles
  uint64_t* s_full = bars + 26;       // [2] S written
  uint64_t* s_free = bars + 28;       // [2] S read into registers
  uint64_t* p_full = bars + 30;       // [2] P written
  uint64_t* pv_done = bars + 32;      // [2] P V completed
  uint64_t* o_free = bars + 34;       // O of a pass is read
  uint64_t* pair = bars + 43;         // [4] the two warps of the same rows have written what they exchange
  uint64_t* fin = bars + 51;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 52);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 53);
  static_assert(KST == 2 && VST <= 8 && NS <= 2, "barrier layout");
  const float NEG_INF = -__int_as_float(0x7f800000);

  // (a shuffle's result is uniform to the compiler, and so is what follows from it)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < KST; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
    for (int i = 0; i < VST; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], C::PVW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], C::PVW);
    }
    mbar_init(o_free, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 2);
    mbar_init(fin, 2 + C::PVW);
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
  // An item is a pair's, the first Q tile the even CTA's and the second the odd one's.  Few items: `share` pairs of a cluster
  // take one, a range of its key tiles each, and join their states in the end.
  const int nact = min(max(uniform(p.plan.header[5]), 0), static_cast<int>(gridDim.x)) >> 1;
  int share = SHARE ? P.pieces : 1;
  while (SHARE && share > 1 && total * share > nact) share >>= 1;
  const int rank = static_cast<int>(blockIdx.x) & 1, at = static_cast<int>(blockIdx.x) >> 1;
  const int taker = SHARE ? at / share : at, piece = SHARE ? at - taker * share : 0;
  const int in_cluster = SHARE ? static_cast<int>(blockIdx.x) & (2 * P.pieces - 1) : 0;
  if (taker >= total || at >= nact) {  // no item in any wave
    if (SHARE) {  // (others of the cluster may have one)
      cluster_barrier();
      cluster_barrier();
    }
    if (warp == 2) tc5::dealloc(tmem, 512);
    return;
  }
  const int far = V == kBias ? P.bias.starts[P.bias.num_buckets - 1] : 0;  // the last bucket's first distance
  // Distances up to far + 63, all that a group of 64 keys with one nearer than `far` can hold; rows apart by about 32 / G
  // banks, so that a warp's 32 / G positions of G heads read different ones.
  const int tab_row = far + 64 + ((32 / P.group - (far + 64)) & 31);
  const bool by_distance = V == kBias && p.hq * tab_row <= C::kTabFloats;
  if (V == kBias) {
    // the bucket of each distance up to `far`, and the biases in the log2 domain
    for (int i = warp; i < P.bias.num_buckets; i += kPvThreads / 32) {
      const int end = i + 1 < P.bias.num_buckets ? P.bias.starts[i + 1] : far + 1;
      for (int n = P.bias.starts[i] + lane; n < end; n += 32) smem[C::OFF_IDX + n] = static_cast<unsigned char>(i);
    }
    __syncthreads();
    float* tab = reinterpret_cast<float*>(smem + C::OFF_TAB);
    if (by_distance) {
      for (int i = threadIdx.x; i < p.hq * tab_row; i += kPvThreads)
        tab[i] = bias_at(P.bias, smem[C::OFF_IDX + min(i % tab_row, far)], i / tab_row);
    } else {
      for (int i = threadIdx.x; i < P.bias.num_buckets * p.hq; i += kPvThreads)
        tab[i] = bias_at(P.bias, i / p.hq, i % p.hq);
    }
    __syncthreads();
  }
  const int G = P.group;
  const int PR = P.prows;
  const uint64_t pol = l2_policy_evict_last();  // K/V tiles are read again by the other items

  // Every role walks the CTA's passes by itself: body(pass).  What an item's pass needs comes by two reads, one depending
  // on the other: they are made two and one items ahead, so that no pass starts with waiting for them.
  struct Pass {
    int no;        // passes of this CTA before this one
    int t0;        // tiles before it
    int h, part;   // kv head or pair; map
    int b, s0, q0, pos0, rows;
    int key0, keys, nkt;  // the keys [key0, key0 + keys), visible to some row of the pair (key0 0 but for a shared item)
    bool shared;          // the cluster's `share` pairs have a range of the keys each
  };
  constexpr int kParts = V == kDiff ? 2 : 1;
  auto item_of = [&](int wave) -> int {  // later (longer) tiles of each span first; -1: none in this or a later wave
    const int ord = snake_order(wave, taker, nact);
    return wave * nact < total && ord < total ? total - 1 - ord : -1;
  };
  auto for_passes = [&](auto&& body) -> Pass {
    Pass it{};
    int item = item_of(0), next = item_of(1);
    int tile = 0, s0 = 0, s1 = 0, ctx = 0, b = 0, next_b = 0, next_tile = 0;
    if (item >= 0) {
      b = p.plan.pf_seq[item / hp];
      tile = p.plan.pf_tile[item / hp];
      s0 = p.qsl[b];
      s1 = p.qsl[b + 1];
      ctx = p.context_lens[b];
    }
    if (next >= 0) {
      next_b = p.plan.pf_seq[next / hp];
      next_tile = p.plan.pf_tile[next / hp];
    }
    for (int wave = 0; item >= 0; ++wave) {
      it.h = item - item / hp * hp;
      it.b = uniform(b);
      it.s0 = uniform(s0);
      const int n = uniform(s1) - it.s0;
      const int first = uniform(tile) * 2 * PR;  // the item's first position
      it.q0 = first + rank * PR;
      it.pos0 = uniform(ctx) - n + it.q0;
      it.rows = min(PR, n - it.q0);  // (of the second tile none or fewer, where the span ends before it)
      it.keys = it.pos0 - rank * PR + min(2 * PR, n - first);
      it.nkt = ceil_div(it.keys, C::BK);
      it.shared = SHARE && share > 1 && it.nkt >= kPrefillShareTiles;
      if (SHARE && share > 1) {  // (of an item that is not shared the first pair has every key)
        const int per = it.shared ? ceil_div(it.nkt, share) : it.nkt;
        it.key0 = min(piece * per, it.nkt) * C::BK;
        it.keys = min(it.keys - it.key0, per * C::BK);
        it.nkt = ceil_div(max(it.keys, 0), C::BK);
      }
      item = next;
      b = next_b;
      tile = next_tile;
      if (item >= 0) {
        s0 = p.qsl[b];
        s1 = p.qsl[b + 1];
        ctx = p.context_lens[b];
      }
      next = item >= 0 ? item_of(wave + 2) : -1;
      if (next >= 0) {
        next_b = p.plan.pf_seq[next / hp];
        next_tile = p.plan.pf_tile[next / hp];
      }
      if (SHARE && it.nkt == 0) break;  // a piece without keys
      for (it.part = 0; it.part < kParts; ++it.part) {
        body(it);
        it.t0 += it.nkt;
        ++it.no;
      }
    }
    return it;
  };
  const int bs = 1 << p.bs_log2;
  // (the same as warp_wait, a few clocks less where the phase has completed already)
  auto ready_or_wait = [&](uint64_t* bar, int phase) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, static_cast<uint32_t>(phase) & 1u))) return true;
    return warp_wait(bar, static_cast<uint32_t>(phase) & 1u, p.err, abort_flag);
  };

  // Registers: 88 + 88 + 168 + 168 a thread of the four warpgroups, the 4 x 128 of the launch.
  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const uint32_t one = lane == 0;
    if (warp == 0) {
      // ------------------------------------------------------------- Q and K by TMA
      int q_issued = 0, k_issued = 0;
      const int box = min(bs, C::BK);  // rows of a box
      const int per = C::BK / box;     // boxes of a tile
      const int my_key = lane * box;   // this lane's box of a tile
      for_passes([&](const Pass& it) {
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        auto fetch = [&](int jt) -> int {  // the block of this lane's box of tile jt
          const int key = jt * C::BK + my_key;
          return (jt < it.nkt && lane < per && key < it.keys) ? btrow[((SHARE ? it.key0 : 0) + key) >> p.bs_log2] : -1;
        };
        bool ok = __all_sync(0xffffffffu, !*abort_flag) && !P.fault_no_copies;
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
          const int f = it.t0 + jt, ks = f & 1;
          if (f >= KST) ok = ready_or_wait(&k_empty[ks], (f >> 1) - 1);
          if (!ok) break;
          const int key = jt * C::BK + my_key;
          const int nbox = ceil_div(min(C::BK, it.keys - jt * C::BK), box);
          if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], static_cast<uint32_t>(nbox * box * D * 2));
          __syncwarp();
          if (lane < per && key < it.keys) {
            if (blk < 0 || blk >= p.num_blocks) {
              raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
              blk = 0;
            }
            tma_load_rows8(smem + C::OFF_K + ks * C::kKTile + my_key * D * 2, &P.tmap_k, head,
                           (blk << (p.bs_log2 - 3)) + ((((SHARE ? it.key0 : 0) + key) & (bs - 1)) >> 3), &k_full[ks], pol);
          }
          k_issued = f + 1;
        }
      });
      // every copy issued has landed before the CTA may leave, also after another role has given up
      if (q_issued > 0) mbar_wait(q_full, (q_issued - 1) & 1, p.err);
      for (int f = max(0, k_issued - KST); f < k_issued; ++f) mbar_wait(&k_full[f % KST], (f / KST) & 1, p.err);
    } else if (warp == 1) {
      // -------------------------------------------------------------------- V by TMA
      int issued = 0;                  // stages
      const int box = min(bs, C::VG);  // rows of a box
      const int per = C::VG / box;     // boxes of a stage
      const int my_stage = lane / per, my_key = lane * box;  // this lane's box of a tile
      for_passes([&](const Pass& it) {
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        auto fetch = [&](int jt) -> int {
          const int key = jt * C::BK + my_key;
          return (jt < it.nkt && my_stage < C::GPT && key < it.keys) ? btrow[((SHARE ? it.key0 : 0) + key) >> p.bs_log2] : -1;
        };
        bool ok = __all_sync(0xffffffffu, !*abort_flag) && !P.fault_no_copies;
        int nb0 = fetch(0), nb1 = fetch(1);
        const int head = V == kDiff ? 2 * it.h : it.h;
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          int blk = nb0;
          nb0 = nb1;
          nb1 = fetch(jt + 2);
          const int f = it.t0 + jt;
          const int key = jt * C::BK + my_key;
          const bool mine = my_stage < C::GPT && key < it.keys;
          if (mine && (blk < 0 || blk >= p.num_blocks)) {
            raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
            blk = 0;
          }
          const int group = (blk << (p.bs_log2 - 3)) + ((((SHARE ? it.key0 : 0) + key) & (bs - 1)) >> 3);
#pragma unroll
          for (int g = 0; g < C::GPT; ++g) {
            const int vs = C::GPT * (f & 1) + g;
            if (f >= 2) ok = ready_or_wait(&v_empty[vs], (f >> 1) - 1);
            if (!ok) break;
            // (a stage whose keys no row sees is handed on empty)
            const int nbox = min(max(ceil_div(it.keys - jt * C::BK - g * C::VG, box), 0), per);
            if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], static_cast<uint32_t>(nbox * box * W * 2));
            __syncwarp();
            if (mine && my_stage == g)
              tma_load_rows8(smem + C::OFF_V + vs * C::kVStage + (lane - g * per) * box * W * 2, &P.tmap_v, head, group,
                             &v_full[vs], pol);
            ++issued;
          }
        }
      });
      for (int i = max(0, issued - VST); i < issued; ++i) mbar_wait(&v_full[i % VST], (i / VST) & 1, p.err);
    } else if (warp < 4) {
      // ------------------------------------------------------- S = Q K^T of the tiles of one parity
      constexpr uint32_t kIdesc = tc5::idesc_bf16_f32(128, 128);
      const int par = warp & 1;
      const uint64_t qd = tc5::smem_desc_sw128(sb + C::OFF_Q, 16, 1024);
      const uint64_t kd = tc5::smem_desc_sw128(sb + C::OFF_K + par * C::kKTile, 16, HALVES * 1024);
      const uint32_t q_lo = static_cast<uint32_t>(qd), q_hi = static_cast<uint32_t>(qd >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(kd), k_hi = static_cast<uint32_t>(kd >> 32);
      const uint32_t sd = tmem + (NS == 2 ? 128u * par : 0u);
      uint64_t* kf = k_full + par;
      uint64_t* ke = k_empty + par;
      uint64_t* sf = s_full + par;
      uint64_t* before = s_free + (NS == 2 ? par : 1 - par);  // of the tile that had the S buffer before
      for_passes([&](const Pass& it) {
        bool ok = warp_wait(q_full, it.no & 1, p.err, abort_flag);
        const int first = (it.t0 + par) & 1;
        if (ok && first >= it.nkt && lane == 0) mbar_arrive(q_empty);  // none of the pass's tiles
#pragma unroll 1
        for (int jt = first; jt < it.nkt && ok; jt += 2) {
          const int f = it.t0 + jt;
          ok = ready_or_wait(kf, f >> 1);
          if (ok && f >= NS) ok = ready_or_wait(before, (f - NS) >> 1);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qo = (kk >> 2) * (C::kQHalf >> 4) + (kk & 3) * (32 >> 4);
            const uint32_t ko = (kk >> 2) * (1024 >> 4) + (kk & 3) * (32 >> 4);
            if (kk == 0)
              tc5::mma_ss_warp<false>(one, sd, q_lo, q_hi, k_lo, k_hi, kIdesc);
            else
              tc5::mma_ss_warp<true>(one, sd, q_lo + qo, q_hi, k_lo + ko, k_hi, kIdesc);
          }
          tc5::commit_warp(one, sf);
          tc5::commit_warp(one, ke);
          if (jt + 2 >= it.nkt) tc5::commit_warp(one, q_empty);
        }
      });
      tc5::commit_warp(one, fin);
      __syncwarp();
    } else if (warp < 4 + C::PVW) {
      // ------------------------------------------------- O += P V, all columns or a half of them
      constexpr int NW = W / C::PVW;
      constexpr uint32_t kIdesc = tc5::idesc_bf16_f32(128, NW, true);
      constexpr uint32_t kRows8 = C::CB * 1024;  // 8 keys of all W columns
      constexpr int kCols = NW / 64;             // this warp's 64-column blocks
      const uint32_t c0 = static_cast<uint32_t>((warp - 4) * kCols);
      const uint64_t vd = tc5::smem_desc_sw128(sb + C::OFF_V + c0 * 1024, 1024, kRows8);
      const uint32_t v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
      const uint32_t od = tmem + C::COL_O + c0 * 64;
      const uint32_t pt = tmem + C::COL_P;
      for_passes([&](const Pass& it) {
        bool ok = __all_sync(0xffffffffu, !*abort_flag);
        // tile jt of parity PAR, FIRST of the pass (overwrites O), LAST (with keys that no row sees)
        auto tile = [&](auto par_, auto first_, auto last_, int jt) {
          constexpr int PAR = decltype(par_)::value;
          constexpr bool FIRST = decltype(first_)::value, LAST = decltype(last_)::value;
          const int f = it.t0 + jt;
          ok = ready_or_wait(&p_full[PAR], f >> 1);
          if (FIRST && ok && it.no > 0) ok = ready_or_wait(o_free, it.no - 1);
#pragma unroll
          for (int g = 0; g < C::GPT; ++g) {
            constexpr int VG = C::VG;
            const int vs = C::GPT * PAR + g;
            if (ok) ok = ready_or_wait(&v_full[vs], f >> 1);
            if (!ok) return;
            if (LAST) {
              const int vis = it.keys - jt * C::BK - g * VG;  // keys of the stage that some row sees
              if (vis < VG) {
                // keys that no row sees: zero, so that 0 * (unused slot) cannot poison O
                unsigned char* vb = smem + C::OFF_V + vs * C::kVStage + c0 * 1024;
                constexpr int kLanes = kCols * 8;  // 16-byte chunks of a row
                unsigned char* mine = vb + (lane % kLanes >> 3) * 1024 + ((lane & 7) << 4);
#pragma unroll 4
                for (int t = max(vis, 0) + lane / kLanes; t < VG; t += 32 / kLanes)
                  *reinterpret_cast<uint4*>(mine + (t >> 3) * kRows8 + (t & 7) * 128) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
            tc5::fence_after();
#pragma unroll
            for (int kk = 0; kk < VG / 16; ++kk) {
              const uint32_t a = pt + 64u * PAR + g * (VG / 2) + 8u * kk;  // two keys to a column
              const uint32_t b = v_lo + vs * (C::kVStage >> 4) + kk * (2 * kRows8 >> 4);
              if (FIRST && g == 0 && kk == 0)
                tc5::mma_ts_warp<false>(one, od, a, b, v_hi, kIdesc);
              else
                tc5::mma_ts_warp<true>(one, od, a, b, v_hi, kIdesc);
            }
            tc5::commit_warp(one, &v_empty[vs]);
          }
          tc5::commit_warp(one, &pv_done[PAR]);
        };
        using T = std::true_type;
        using F = std::false_type;
        using P0 = std::integral_constant<int, 0>;
        using P1 = std::integral_constant<int, 1>;
        auto either = [&](auto first_, auto last_, int jt) {
          if ((it.t0 + jt) & 1)
            tile(P1{}, first_, last_, jt);
          else
            tile(P0{}, first_, last_, jt);
        };
        if (!ok) return;
        if (it.nkt == 1) {
          either(T{}, T{}, 0);
          return;
        }
        either(T{}, F{}, 0);
#pragma unroll 1
        for (int jt = 1; jt < it.nkt - 1 && ok; ++jt) either(F{}, F{}, jt);
        if (ok) either(F{}, T{}, it.nkt - 1);
      });
      tc5::commit_warp(one, fin);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // ------------------------------------------------------------------------ softmax
    const int wg = (warp - 8) >> 2;  // keys 64 wg .. 64 wg + 63 of a tile
    const int sw = warp & 3;         // TMEM lanes 32 sw .. 32 sw + 31
    const int r = 32 * sw + lane;
    const int rt = r / G;       // position within the Q tile
    const int rg = r - rt * G;  // member of the group
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * sw) << 16);
    const uint32_t to = tlane + C::COL_O;
    const float* tab = reinterpret_cast<const float*>(smem + C::OFF_TAB);
    const unsigned char* idx = smem + C::OFF_IDX;
    int ex_no = 0;  // exchanges so far
    // of a shared item: the state of this thread's row in each map, and where its sums are left (row by row)
    float m_of[2] = {NEG_INF, NEG_INF}, l_of[2] = {0.f, 0.f};
    float* const left0 = V == kDiff ? p.plan.scratch + static_cast<int64_t>(blockIdx.x) * 128 * W : nullptr;
    const uint32_t left1 = sb + C::OFF_V;  // 16-byte pieces of a row xored with the row, so that rows use different banks
    const uint32_t left_ml = sb + C::OFF_K;
    // x of this thread against the other's of its row; false: a wait gave up.  (Two slots in turn: a warp writes one again only
    // after the exchange between, to which the other came after it had read it.)
    auto exchange = [&](float x, float& other) -> bool {
      float* slot = exch + (ex_no & 1) * 256;
      slot[wg * 128 + r] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pair[sw]);
      const bool ok = ready_or_wait(&pair[sw], ex_no);
      other = slot[(1 - wg) * 128 + r];
      ++ex_no;
      return ok;
    };
    const Pass end = for_passes([&](const Pass& it) {
      const bool live = rt < it.rows;
      // (a row past the span's sees everything: its scores need no mask and go nowhere)
      const int pos = live ? it.pos0 + rt : INT32_MAX;
      const int posb = live ? it.pos0 + rt : (SHARE ? it.key0 : 0) + it.keys - 1;
      const int bh = V == kBias ? it.h * G + (live ? rg : 0) : 0;  // the bias's head
      const float cfar = V == kBias ? tab[by_distance ? bh * tab_row + far : (P.bias.num_buckets - 1) * p.hq + bh] : 0.f;
      // (a bias that would swallow scores is added to each, so that it does)
      const bool cfar_large = V == kBias && fabsf(cfar) > 1048576.f && cfar != NEG_INF;
      float m_run = NEG_INF, l_run = 0.f;
      bool ok = __all_sync(0xffffffffu, !*abort_flag);
      float sc[64];
      auto fetch = [&](int f) -> bool {  // S of tile f on its way into registers
        if (!ready_or_wait(&s_full[f & 1], f >> 1)) return false;
        tc5::fence_after();
        const uint32_t ts = tlane + 128u * (f % NS) + 64u * wg;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v[32];
          tc5::ld32(ts + 32u * c, v);
#pragma unroll
          for (int x = 0; x < 32; ++x) sc[32 * c + x] = v[x];
        }
        return true;
      };
      if (ok) ok = fetch(it.t0);
#pragma unroll 1
      for (int jt = 0; jt < it.nkt && ok; ++jt) {
        const int f = it.t0 + jt, par = f & 1;
        tc5::wait_ld();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[par]);
        const int key0 = (SHARE ? it.key0 : 0) + jt * C::BK + 64 * wg;
        float mul = p.qscale, add = cfar;
        if (V == kBias && __any_sync(0xffffffffu, posb - (key0 + 63) < far || cfar_large)) {
          // some key is nearer than the last bucket
          const int n0 = posb - key0;
          if (by_distance) {
            // (a warp's rows may lie a few positions past what a row of the table holds, all of them in the last bucket; and
            // keys after the row, masked below, read what lies before the table)
            const float* tb = tab + bh * tab_row + min(n0, far + 63);
#pragma unroll
            for (int c = 0; c < 64; ++c) sc[c] = fmaf(sc[c], p.qscale, tb[-c]);
          } else {
            const float* tb = tab + bh;
#pragma unroll
            for (int c = 0; c < 64; ++c) sc[c] = fmaf(sc[c], p.qscale, tb[idx[min(max(n0 - c, 0), far)] * p.hq]);
          }
          mul = 1.f;
          add = 0.f;
        }
        if (__any_sync(0xffffffffu, key0 + 63 > pos)) {
          const int last = pos - key0;  // (may be negative: none)
#pragma unroll
          for (int c = 0; c < 64; ++c) sc[c] = c <= last ? sc[c] : NEG_INF;
        }
        float mx8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) mx8[x] = max3(sc[x], sc[8 + x], sc[16 + x]);
#pragma unroll
        for (int c = 24; c < 56; c += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x) mx8[x] = max3(mx8[x], sc[c + x], sc[c + 8 + x]);
#pragma unroll
        for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(mx8[x], sc[56 + x]);
        const float mraw = max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        const float mine = V == kBias ? fmaf(mraw, mul, add) : mraw * mul;  // (-inf stays -inf)
        float theirs = NEG_INF;
        ok = exchange(mine, theirs);
        if (!ok) break;
        const float mx = fmaxf(mine, theirs);
        const bool up = mx > m_run;
        const bool any_up = __any_sync(0xffffffffu, up);
        const float raised = mx + (kVarSlack - kCutShift);
        const float corr = up ? fast_exp2(m_run - raised) : 1.f;
        m_run = up ? raised : m_run;
        l_run *= corr;
        const float base = m_run == NEG_INF ? 0.f : m_run;
        // (looked at here and used below: what it takes passes with the weights)
        const bool p_free = f < 2 || mbar_test_wait(&pv_done[par], static_cast<uint32_t>((f >> 1) - 1) & 1u);
        // weights 2^(s - m), cut to bf16 for P V (a byte permutation where a conversion would go to the unit of the powers
        // of two).  l sums the cut ones: what all weights lose alike drops out, and what is left of the cut, at most 2^-8 of a
        // weight either way, is what rounding to the nearest would leave; kCutShift has the largest weight lose as much as the
        // others on average.
        // (A score is rounded as the row's maximum was, before the difference: fused into one step a row whose scores pass 2^30
        // had weights as far above 1, or below, as fp32 rounds its maximum.  Two steps cost 853 us for 840 of the differential
        // chunk, 691 for 674 of that with the bias; a look whether a row needs them 845 and 707.)
        const float2 mul2 = make_float2(mul, mul), add2 = make_float2(add, add), base2 = make_float2(-base, -base);
        float2 ls4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ls4[x] = make_float2(0.f, 0.f);
        float pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float2 t = fadd2(ffma2(make_float2(sc[2 * x], sc[2 * x + 1]), mul2, add2), base2);
          const uint32_t w = __byte_perm(__float_as_uint(fast_exp2(t.x)), __float_as_uint(fast_exp2(t.y)), 0x7632);
          ls4[x & 3] = fadd2(ls4[x & 3], make_float2(bf16lo(w), bf16hi(w)));
          pk[x] = __uint_as_float(w);
        }
        if (!__all_sync(0xffffffffu, p_free)) {  // this P buffer is read by the P V of tile f - 2
          ok = warp_wait(&pv_done[par], static_cast<uint32_t>((f >> 1) - 1) & 1u, p.err, abort_flag);
          if (!ok) break;
        }
        tc5::fence_after();
        tc5::st32(tlane + C::COL_P + 64u * par + 32u * wg, pk);  // a column holds two keys
        if (jt + 1 < it.nkt) {
          ok = fetch(f + 1);  // (its S needs nothing of this tile's but that its own is read)
          if (!ok) break;
        }
        const float2 ls2 = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
        l_run += ls2.x + ls2.y;
        if (jt > 0 && any_up) {
          // O is rescaled once the P V of every tile before has landed in it, this warp's half of the columns here
          // (that of tile f - 2 has: p_free)
          ok = warp_wait(&pv_done[1 - par], ((f - 1) >> 1) & 1, p.err, abort_flag);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll 1
          for (int c = 0; c < W / 64; ++c) {
            const uint32_t at = to + static_cast<uint32_t>(wg * (W / 2) + 32 * c);
            float o[32];
            tc5::ld32(at, o);
            tc5::wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= corr;
            tc5::st32(at, o);
          }
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[par]);
      }
      // ------------------------------------------------------------- the pass's rows
      const int last = it.t0 + it.nkt - 1;
      float l_other = 0.f;
      if (ok) ok = exchange(l_run, l_other);
      if (ok) ok = warp_wait(&pv_done[last & 1], (last >> 1) & 1, p.err, abort_flag);
      if (!ok) return;
      tc5::fence_after();
      const float l_all = l_run + l_other;
      const float inv = inverse_or_0(l_all);
      constexpr int HW = W / 2;  // columns of either half, 32 at a time
      constexpr int NC = HW / 32;
      const uint32_t tc = to + static_cast<uint32_t>(wg * HW);
      const int row = it.s0 + it.q0 + rt;
      const int head = it.h * G + rg;
      bf16* orow = p.out + static_cast<int64_t>(row) * p.o_st + static_cast<int64_t>(head) * p.o_sh + wg * HW;
      auto o_is_read = [&]() {  // the next pass's P V may overwrite it
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      };
      auto write32 = [&](int c, const float (&o)[32]) {
        if (live) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint4 u;
            u.x = pack_bf16x2(o[8 * x + 0], o[8 * x + 1]);
            u.y = pack_bf16x2(o[8 * x + 2], o[8 * x + 3]);
            u.z = pack_bf16x2(o[8 * x + 4], o[8 * x + 5]);
            u.w = pack_bf16x2(o[8 * x + 6], o[8 * x + 7]);
            *reinterpret_cast<uint4*>(orow + 32 * c + 8 * x) = u;
          }
        }
      };
      if (SHARE && it.shared) {
        // (every product of this CTA that reads V has completed when the last pass's have, and no copy is to come)
        if (it.part == 0)
          m_of[0] = m_run, l_of[0] = l_all;
        else
          m_of[1] = m_run, l_of[1] = l_all;
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          float o[32];
          tc5::ld32(tc + 32u * c, o);
          tc5::wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int at4 = wg * (HW / 4) + 8 * c + x;
            float4* dst = V == kDiff && it.part == 0
                              ? reinterpret_cast<float4*>(left0) + r * (W / 4) + at4
                              : reinterpret_cast<float4*>(smem + C::OFF_V + r * (W * 4) + ((at4 ^ (r & 7)) << 4));
            *dst = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
        o_is_read();
        return;
      }
      if constexpr (V == kDiff) {
        float4* own = reinterpret_cast<float4*>(p.plan.scratch) +
                      (static_cast<int64_t>(blockIdx.x) * (W / 4) + wg * (HW / 4)) * 128 + r;
        if (it.part == 0) {
#pragma unroll 1
          for (int c = 0; c < NC; ++c) {
            float o[32];
            tc5::ld32(tc + 32u * c, o);
            tc5::wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x)
              own[(8 * c + x) * 128] = make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
          }
          o_is_read();
          return;
        }
        const float la = live ? P.diff.lambda[static_cast<int64_t>(row) * P.diff.lambda_st + head] * inv : 0.f;
        const float4* nw = reinterpret_cast<const float4*>(P.diff.norm_weight + wg * HW);
        float scale = P.diff.out_scale, ss = 0.f;
        // x = a_0 V - lambda a_1 V; with the norm back into O's columns until the row's squares are summed
        float4 a[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) a[x] = own[x * 128];
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          float o[32];
          tc5::ld32(tc + 32u * c, o);
          float4 next[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) next[x] = c + 1 < NC ? own[(8 * c + 8 + x) * 128] : a[x];
          tc5::wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            o[4 * x] = a[x].x - la * o[4 * x];
            o[4 * x + 1] = a[x].y - la * o[4 * x + 1];
            o[4 * x + 2] = a[x].z - la * o[4 * x + 2];
            o[4 * x + 3] = a[x].w - la * o[4 * x + 3];
            a[x] = next[x];
          }
          if (P.diff.norm_weight) {
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 32; ++x) s4[x & 3] = fmaf(o[x], o[x], s4[x & 3]);
            ss += (s4[0] + s4[1]) + (s4[2] + s4[3]);
            tc5::st32(tc + 32u * c, o);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= scale;
            write32(c, o);
          }
        }
        if (P.diff.norm_weight) {
          tc5::wait_st();
          float theirs = 0.f;
          if (!exchange(ss, theirs)) return;
          // (the same sum in both threads)
          scale *= 1.f / sqrtf((wg == 0 ? ss + theirs : theirs + ss) * (1.f / W) + P.diff.norm_eps);
#pragma unroll 1
          for (int c = 0; c < NC; ++c) {
            float o[32];
            tc5::ld32(tc + 32u * c, o);
            tc5::wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float4 w = __ldg(nw + 8 * c + x);
              o[4 * x] *= w.x * scale;
              o[4 * x + 1] *= w.y * scale;
              o[4 * x + 2] *= w.z * scale;
              o[4 * x + 3] *= w.w * scale;
            }
            write32(c, o);
          }
        }
        o_is_read();
      } else {
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          float o[32];
          tc5::ld32(tc + 32u * c, o);
          tc5::wait_ld();
          if (c == NC - 1) o_is_read();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] *= inv;
          write32(c, o);
        }
      }
    });
    if (SHARE && end.shared) {
      if (wg == 0) {
#pragma unroll
        for (int c = 0; c < kParts; ++c)
          *reinterpret_cast<float2*>(smem + C::OFF_K + (c * 128 + r) * 8) = make_float2(m_of[c], l_of[c]);
      }
      cluster_barrier();
      // Every share-th row is this piece's, a warp to a row and 16 / share of them to a warp: with f = 2^(m - M) over the pieces'
      // sum of 2^(m - M) l (kDiff: the second map's times -lambda) the row is the sum of f o over pieces and maps.
      const uint32_t first = static_cast<uint32_t>(in_cluster - 2 * piece);  // the same tile's CTA of piece 0
      constexpr int CH = (W / 4 + 31) / 32;                                   // 16-byte pieces of a row to a lane
      const int log_share = share == 4 ? 2 : 1, rows = 16 >> log_share;
      auto row_of = [&](int i) { return ((warp - 8 + 8 * i) << log_share) + piece; };
      float f = 0.f;
      {  // a lane to a row, a map and a piece
        const int k = lane & (share - 1), c = V == kDiff ? lane >> log_share & 1 : 0;
        const int row = row_of((V == kDiff ? lane >> (log_share + 1) : lane >> log_share) & (rows - 1)), jt = row / G;
        const float2 ml = ld_peer_f2(peer_smem(left_ml + (c * 128 + row) * 8, first + 2 * k));
        float M = ml.x;
        for (int off = 1; off < share; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float w = ml.y == 0.f ? 0.f : fast_exp2(ml.x - (M == NEG_INF ? 0.f : M));
        float den = w * ml.y;
        for (int off = 1; off < share; off <<= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
        f = w * inverse_or_0(den);
        if (V == kDiff && c == 1 && jt < end.rows)
          f *= -P.diff.lambda[static_cast<int64_t>(end.s0 + end.q0 + jt) * P.diff.lambda_st + end.h * G + row - jt * G];
      }
      const bool ok = __all_sync(0xffffffffu, !*abort_flag);
#pragma unroll 2
      for (int i = 0; i < rows; ++i) {
        const int row = row_of(i), jt = row / G, jg = row - jt * G;
        const bool mine = ok && jt < end.rows;  // (warp-uniform)
        float4 x[CH];
#pragma unroll
        for (int y = 0; y < CH; ++y) x[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
#pragma unroll
          for (int k = 0; k < kPrefillSharePairs; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, (((i * kParts) + c) << log_share) + (k & (share - 1)));
            if (!mine || k >= share || fk == 0.f) continue;  // (this piece holds no key of the row)
#pragma unroll
            for (int y = 0; y < CH; ++y) {
              const int at4 = W / 4 < 32 ? lane & (W / 4 - 1) : lane + 32 * y;
              const float4 o = V == kDiff && c == 0
                                   ? __ldcg(reinterpret_cast<const float4*>(left0 + 2 * (k - piece) * (128 * W) + row * W) + at4)
                                   : ld_peer_f4(peer_smem(left1 + row * (W * 4) + ((at4 ^ (row & 7)) << 4), first + 2 * k));
              x[y] = make_float4(fmaf(fk, o.x, x[y].x), fmaf(fk, o.y, x[y].y), fmaf(fk, o.z, x[y].z), fmaf(fk, o.w, x[y].w));
            }
          }
        }
        float scale = 1.f;
        if (V == kDiff) {
          scale = P.diff.out_scale;
          if (P.diff.norm_weight) {
            float ss = 0.f;
#pragma unroll
            for (int y = 0; y < CH; ++y) ss += x[y].x * x[y].x + x[y].y * x[y].y + x[y].z * x[y].z + x[y].w * x[y].w;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            scale *= 1.f / sqrtf(ss * (1.f / W) + P.diff.norm_eps);
          }
        }
        if (!mine || (W / 4 < 32 && lane >= W / 4)) continue;
        bf16* orow = p.out + static_cast<int64_t>(end.s0 + end.q0 + jt) * p.o_st + static_cast<int64_t>(end.h * G + jg) * p.o_sh;
#pragma unroll
        for (int y = 0; y < CH; ++y) {
          const int at4 = lane + 32 * y;
          float4 w = make_float4(scale, scale, scale, scale);
          if (V == kDiff && P.diff.norm_weight) {
            const float4 nw = __ldg(reinterpret_cast<const float4*>(P.diff.norm_weight) + at4);
            w = make_float4(nw.x * scale, nw.y * scale, nw.z * scale, nw.w * scale);
          }
          uint2 u;
          u.x = pack_bf16x2(x[y].x * w.x, x[y].y * w.y);
          u.y = pack_bf16x2(x[y].z * w.z, x[y].w * w.w);
          *reinterpret_cast<uint2*>(orow + 4 * at4) = u;
        }
      }
    } else if (SHARE) {
      cluster_barrier();
    }
  }
  if (SHARE && warp < 8) cluster_barrier();  // (the softmax's joins shared items behind it)
  __syncthreads();  // every role has finished its last pass
  if (warp == 2) {  // no product may be in flight when TMEM is released
    mbar_wait(fin, 0, p.err);
    __syncwarp();
    tc5::fence_after();
    tc5::dealloc(tmem, 512);
  }
  if (SHARE) cluster_barrier();  // no CTA leaves while another may still read its rows
}

// Clusters of `pieces` pairs of CTAs that the device holds at a time (asked once for each device and size).
template <int D, int V, bool SHARE>
int max_clusters(int pieces) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  std::atomic<int>& slot = known[dev][pieces >> 1];
  int n = slot.load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pieces));
    cfg.blockDim = dim3(kPvThreads);
    cfg.dynamicSmemBytes = PrefillVarCfg<D, V>::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(2 * pieces), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, prefill_variant_kernel<D, V, SHARE>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = -1;
    }
    slot.store(n);
  }
  return n > 0 ? n : 0;
}

template <int D, int V, bool SHARE>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  using C = PrefillVarCfg<D, V>;
  if (const cudaError_t e = set_smem_once<prefill_variant_kernel<D, V, SHARE>>(C::kSmemBytes); e != cudaSuccess) return e;
  PrefillVarParams P{};
  const int bs8 = 1 << (a.bs_log2 - 3);  // groups of 8 rows of a block
  const int heads = V == kDiff ? 2 : 1;
  if (!make_q_map_parts(&P.tmap_q, a, heads) ||
      !make_pool_map_rows8(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D, 1, bs8 < C::BK / 8 ? bs8 : C::BK / 8) ||
      !make_pool_map_rows8(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D, heads,
                           bs8 < C::VG / 8 ? bs8 : C::VG / 8))
    return cudaErrorInvalidValue;
  P.p = make_prefill_params(a);
  P.group = a.hq / a.hkv;
  P.prows = kTcPrefillRows / P.group;
  if (a.bias) P.bias = *a.bias;
  if (a.diff) P.diff = *a.diff;
  P.fault_no_copies = a.fault == PKV_FAULT_PREFILL_NO_COPIES;
  cudaLaunchConfig_t cfg = {};
  P.pieces = prefill_variant_pieces(a);
  const int64_t grid = prefill_variant_grid(a), fit = 2ll * P.pieces * max_clusters<D, V, SHARE>(P.pieces);
  cfg.gridDim = dim3(static_cast<unsigned>(fit > 0 && fit < grid ? fit : grid));
  cfg.blockDim = dim3(kPvThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(2 * P.pieces), 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  record_kernel_event(PKV_KERNEL_PREFILL, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_variant_kernel<D, V, SHARE>, P);
  record_kernel_event(PKV_KERNEL_PREFILL, true, stream);
  return e;
}

}  // namespace

// Pairs of CTAs in a cluster, which may share an item: more than one where the tokens beyond one a sequence, were they all in
// one span, would not give half the pairs an item (the kernel then decides by the items there are), and a context may be long
// enough.  (GB300, spans of 223 and 249 behind 1969 keys, 16/2 heads d 64: 33 us shared by four pairs, 42 by two, 50 by one
// each; four prompts of 238, which nobody shares: 20.5 us in pairs, 22 in clusters of eight.)
int prefill_variant_pieces(const AttnArgs& a) {
  const int prows = 2 * (kTcPrefillRows / (a.hq / a.hkv));
  const int64_t extra = a.num_tokens - a.num_seqs + 1;
  const int64_t items = ceil_div64(extra > 0 ? extra : 1, prows) * (a.variant == kDiff ? a.hkv / 2 : a.hkv);
  const int64_t pairs = device_sm_count() / 2;
  if (max_context(a.max_blocks, a.bs_log2) < kPrefillShareTiles * 128) return 1;
  return items * 4 <= pairs ? kPrefillSharePairs : items * 2 <= pairs ? 2 : 1;
}

// One CTA per SM, at most a pair per item or, where pairs may share items, a cluster.
int64_t prefill_variant_grid(const AttnArgs& a) {
  const int prows = 2 * (kTcPrefillRows / (a.hq / a.hkv));
  const int64_t pieces = prefill_variant_pieces(a);
  const int64_t max_items = (a.num_tokens / prows + a.num_seqs + 1) * (a.variant == kDiff ? a.hkv / 2 : a.hkv);
  const int64_t clusters = device_sm_count() / (2 * pieces);
  return 2 * pieces * (max_items < clusters ? max_items : clusters);
}

template <bool SHARE>
static cudaError_t launch_variant(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  if (a.variant == kBias)
    return a.head_dim == 128 ? launch<128, kBias, SHARE>(a, stream, pdl) : launch<64, kBias, SHARE>(a, stream, pdl);
  return a.head_dim == 128 ? launch<128, kDiff, SHARE>(a, stream, pdl) : launch<64, kDiff, SHARE>(a, stream, pdl);
}
cudaError_t launch_prefill_variant(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  return prefill_variant_pieces(a) > 1 ? launch_variant<true>(a, stream, pdl) : launch_variant<false>(a, stream, pdl);
}

}  // namespace pkv
