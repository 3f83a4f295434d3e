// Prefill-chunk attention over an 8-bit cache on the 5th-generation tensor cores.
//
// The causal rule and the stacking of heads are the bf16 prefill's (prefill_tc.cuh): a Q tile's 128 rows are
// P = floor(128 / G) positions of a span times the G query heads of one kv head.  The tensor cores read
// neither int8 nor a scale per block, so every K/V tile of 128 keys is turned into f16 in shared memory
// first, and an item is two Q tiles, A and B (2 P positions), so that each converted tile feeds four
// products, S = Q K^T and O += P V of either (tcgen05.mma kind::f16, accumulators in TMEM):
//
//   held 2^(e - ref)  with ref one exponent per tile for K and one per item for V
//
// which is exact in f16 while e is not far below ref (the products are then those of the
// dequantised cache); S is multiplied by 2^ref 2^eq in the softmax, where q entered as q 2^-eq
// with its largest magnitude in [2^14, 2^15), and O is in units of 2^ref.  The V reference moves to
// a tile whose scales leave the window around it; the softmax warps then rescale O as they do when
// a row's maximum grows.
//
// One CTA of twenty warps:
//   warps 0-3    the MMA issue, in steps of 64 keys: QK of A and of B, PV of A and of B (a warp to each scheduler)
//   warp 4       TMA producer: raw K and V tiles in turn (one box per block), scales by cp.async, four stages
//   warps 5-7    Q tiles: plain loads (any strides), row maximum, f16, swizzled store
//   warps 8-11   softmax of A, thread = row: S from TMEM, P (f16) back over it, O rescale, output
//   warps 12-15  softmax of B
//   warps 16-19  conversion of the raw tiles into three f16 stages (K0 V0 K1 V1 ..)
// TMEM holds two S buffers of 64 columns and O for either Q tile, all of it at d 128, so P overlays the S
// it came from; a Q tile's QK of step s + 1 waits for its PV of step s - 1.  A step's products take the tensor cores
// 1,264 clocks (two Q tiles, measured alone); what an issuing warp does around them costs as much again (its waits
// about 130 clocks each even when nothing is to be waited for), so each of the four has a warp: one warp for
// all took 4,400 clocks a step, one for a Q tile 2,900.  Items follow one another without a CTA barrier, and
// every wait is bounded.
//
// Few items (short spans, few heads) would leave most SMs idle while each walks a long context alone: then two,
// four or eight CTAs of a cluster share an item, each a range of its key tiles, and join their rows through
// distributed shared memory, out = sum 2^(m - M) l o / sum 2^(m - M) l.  Two spans of up to 14 tokens after 3,273, 2
// heads, d 64: 75 us alone, 25 shared.
//
// Bound: the softmax warps, and their wait for S.  3700 tokens after 12,288 (28/4 heads, d 128) take 765 us, 0.52 of
// the bf16 library rate; the tensor pipe is busy 41 % of it, and a scheduler issues in 55 % of its cycles.  A step of
// 64 keys takes a softmax warp 2,200 clocks: 550 of waiting for S, 260 for its TMEM read, 340 for the maximum, 740 for
// the weights, 270 for sums and checks.  Tried and slower: S in one buffer with P in columns of its own, so that
// the next QK does not wait for P V (830 us; at d 64 two buffers of each, 802 against 697); part of the powers of two
// on the FMA pipe by a polynomial (a quarter of them 969 us, an eighth 838).
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "decode_tc.cuh"
#include "prefill.cuh"
#include "prefill_tc.cuh"
#include "q8.cuh"
#include "tcgen05.cuh"

namespace pkv {

bool make_pool_map_q8(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D);

namespace {

constexpr int kPqThreads = 640;
constexpr float kExactScore = 2097152.f;  // scores (log2 domain) up to which m's rounding is at most 2^-3
constexpr int kConvWarps = 4;

struct PrefillQ8Params {
  CUtensorMap tmap_k;  // 4-D {d, Hkv, block_size, num_blocks} of bytes, box {d, 1, block_size, 1}
  CUtensorMap tmap_v;
  PrefillParams p;
  const float* k_scale;
  const float* v_scale;
  const uint8_t* v_cache;
  int group;  // G
  int prows;  // floor(128 / G): positions of a Q tile
  int pieces;  // CTAs of a cluster, 1: launched without clusters
  int fault_no_copies;  // test-only: the producer issues nothing
};

template <int D>
struct PrefillQ8Cfg {
  static constexpr int BK = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int kBlk = 128 * 128;       // [128 rows][64 f16], 128-byte swizzled
  static constexpr int kTile = HALVES * kBlk;  // a Q, K or V tile in f16
  static constexpr int kRaw = BK * D;          // a K or V tile as held
  static constexpr int RST = 4;                // raw stages (K and V tiles in turn)
  static constexpr int TST = 3;                // f16 stages (K and V tiles in turn)
  static constexpr int OFF_Q = 0;              // A, B
  static constexpr int OFF_T = 2 * kTile;
  static constexpr int OFF_RAW = OFF_T + TST * kTile;
  static constexpr int OFF_QE = OFF_RAW + RST * kRaw;  // [3][A|B][128] biased exponents of the rows' largest, bytes
  static constexpr int OFF_SC = OFF_QE + 3 * 256;      // [RST][K|V][16] scales
  static constexpr int OFF_REF = OFF_SC + RST * 32 * 4;  // [4] {K reference, V reference}
  static constexpr int OFF_BAR = OFF_REF + 4 * 8;
  static constexpr int kSmemBytes = OFF_BAR + 32 * 8 + 1024;  // + barriers + alignment slack
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int SK = 64;           // keys of a step
  static constexpr uint32_t COL_S = 0;    // [A|B][2 buffers] of 64 columns
  static constexpr uint32_t COL_O = 256;  // A; B D further
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// Instruction descriptor of a kind::f16 MMA with f16 operands (as tc5::idesc_bf16_f32, whose
// operand format fields are 0 for f16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major = false) {
  return tc5::idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// The products as issued by a whole converged warp, of which one lane (`one` != 0) executes them: with every
// operand uniform in the warp's control flow the instructions follow one another; issued from a branch that
// only one lane takes they were 165 (both operands in shared memory) and 115 clocks apart, whatever N, and bound
// the kernel.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACC ? 1 : 0), "r"(one)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "n"(ACC ? 1 : 0), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(one)
      : "memory");
}

// All threads of the cluster's CTAs, each from its own role's code.
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

template <int D, int FMT>
__global__ void __launch_bounds__(kPqThreads, 1) prefill_q8_kernel(const __grid_constant__ PrefillQ8Params P) {
  using C = PrefillQ8Cfg<D>;
  const PrefillParams& p = P.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  unsigned char* qexp = smem + C::OFF_QE;
  volatile int* refs = reinterpret_cast<volatile int*>(smem + C::OFF_REF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_full = bars + 0;   // [4] TMA bytes and the producer lanes' cp.async
  uint64_t* raw_empty = bars + 4;  // [4] converted
  uint64_t* t_full = bars + 8;     // [3] f16 tile written
  uint64_t* t_empty = bars + 11;   // [3] each Q tile's products with it completed
  uint64_t* q_full = bars + 14;
  uint64_t* q_empty = bars + 15;   // each Q tile's QKs of an item completed
  uint64_t* s_full = bars + 16;    // [A|B][2] S buffer written
  uint64_t* p_full = bars + 20;    // [A|B][2] P written over it
  uint64_t* pv_done = bars + 24;   // [A|B][2] the P.V that reads it completed
  uint64_t* fin = bars + 28;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 29);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* nan_seen = reinterpret_cast<volatile int*>(bars + 31);  // a NaN of V was taken out of a tile
  const float NEG_INF = -__int_as_float(0x7f800000);

  // (a shuffle's result is uniform to the compiler, and so is what follows from it: the MMA descriptors are then
  // made in uniform registers, where the instruction takes them)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::RST; ++s) {
      mbar_init(&raw_full[s], 33);
      mbar_init(&raw_empty[s], kConvWarps);
    }
    for (int s = 0; s < C::TST; ++s) {
      mbar_init(&t_full[s], kConvWarps);
      mbar_init(&t_empty[s], 2);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&pv_done[x], 1);
    }
    mbar_init(q_full, 3);
    mbar_init(q_empty, 2);
    mbar_init(fin, 4);
    fence_mbar_init();
    *abort_flag = 0;
    *nan_seen = 0;
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_v)) : "memory");
  }
  if (warp == 1) {  // while the planner still runs
    tc5::alloc(tmem_slot, C::TMEM_COLS);
    tc5::relinquish();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  pdl_wait();
  pdl_trigger();
  const int total = uniform(p.plan.header[3]) * p.hkv;
  const int nact = min(max(uniform(p.plan.header[5]), 0), static_cast<int>(gridDim.x));
  // Few items: `share` CTAs of a cluster take one, a range of its key tiles each, and join their states in the end.
  int share = P.pieces;
  while (share > 1 && total * share > nact) share >>= 1;
  const int taker = static_cast<int>(blockIdx.x) / share, piece = static_cast<int>(blockIdx.x) - taker * share;
  if (taker >= total || static_cast<int>(blockIdx.x) >= nact) {  // no item in any wave
    if (share > 1) {  // (others of the cluster may have one)
      cluster_barrier();
      cluster_barrier();
    }
    if (warp == 1) tc5::dealloc(tmem, C::TMEM_COLS);
    return;
  }
  const int G = P.group;
  const int PR = P.prows;
  const uint64_t pol = l2_policy_evict_last();  // K/V tiles are read again by the other items

  // every role walks the CTA's items by itself: body(item)
  struct Item {
    int no;                // items of this CTA before this one
    int t_glob, t_of[2];   // before it: key tiles, and steps of Q tile A and of B
    int h, b, s0, q0, pos0;
    int rows[2], nst_of[2];  // positions and steps of A and B
    int key0, kv_end;        // the keys [key0, kv_end), visible to some row (key0 0 but for a shared item)
    int nkt, nst;            // key tiles, steps
  };
  auto for_items = [&](auto&& body) {
    Item it;
    it.no = it.t_glob = it.t_of[0] = it.t_of[1] = 0;
    for (int wave = 0; wave * nact < total; ++wave) {
      const int ord = share > 1 ? taker : snake_order(wave, blockIdx.x, nact);
      if (ord >= total) continue;
      const int item = total - 1 - ord;  // later (longer) tiles of each span first
      const int ti = item / p.hkv;
      it.h = item - ti * p.hkv;
      it.b = uniform(p.plan.pf_seq[ti]);
      it.s0 = uniform(p.qsl[it.b]);
      const int n = uniform(p.qsl[it.b + 1]) - it.s0;
      it.q0 = uniform(p.plan.pf_tile[ti]) * 2 * PR;
      it.pos0 = uniform(p.context_lens[it.b]) - n + it.q0;
      it.rows[0] = min(PR, n - it.q0);
      it.rows[1] = min(PR, n - it.q0 - it.rows[0]);
      it.kv_end = it.pos0 + it.rows[0] + it.rows[1];
      it.nkt = ceil_div(it.kv_end, C::BK);
      it.key0 = 0;
      if (share > 1) {
        const int per = ceil_div(it.nkt, share), first = min(piece * per, it.nkt);
        it.nkt = min(per, it.nkt - first);
        it.key0 = first * C::BK;
        it.kv_end = min(it.kv_end, it.key0 + it.nkt * C::BK);
      }
      it.nst = max(ceil_div(it.kv_end - it.key0, C::SK), 0);
      it.nst_of[0] = max(ceil_div(min(it.pos0 + it.rows[0], it.kv_end) - it.key0, C::SK), 0);
      it.nst_of[1] = it.rows[1] > 0 ? it.nst : 0;
      body(it);
      it.t_glob += it.nkt;
      it.t_of[0] += it.nst_of[0];
      it.t_of[1] += it.nst_of[1];
      ++it.no;
    }
  };
  const int bs = 1 << p.bs_log2;

  // Registers: 56 + 56 + 136 + 136 + 96 a thread of the five warpgroups, the 5 x 96 of the launch.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // --------------------------------------------------------- MMA issue of one kind, of one Q tile
    const uint32_t one = lane == 0;
    const int x = warp & 1;
    const uint32_t sd0 = tmem + C::COL_S + 128u * x;
    uint64_t* pd = pv_done + 2 * x;
    if (warp < 2) {
      // S[f % 2] = Q K^T, once the P.V that reads the P it overwrites (two steps before) is done.  A tile is
      // given back when this Q tile's products with it have completed (at once if it sees none of it).
      constexpr uint32_t kIdesc = idesc_f16_f32(128, C::SK);
      // (a descriptor's low bits are the address in units of 16 bytes)
      const uint64_t qd = tc5::smem_desc_k128(sb + C::OFF_Q + x * C::kTile), kd0 = tc5::smem_desc_k128(sb + C::OFF_T);
      uint64_t* sf = s_full + 2 * x;
      for_items([&](const Item& it) {
        const int nst_x = x ? it.nst_of[1] : it.nst_of[0], t_x = x ? it.t_of[1] : it.t_of[0];
        bool ok = warp_wait(q_full, it.no & 1, p.err, abort_flag);
        if (ok && nst_x == 0 && one) mbar_arrive(q_empty);
#pragma unroll 1
        for (int st = 0; st < it.nst && ok; ++st) {
          const int u = 2 * (it.t_glob + (st >> 1)), ts = u % C::TST;
          if (!(st & 1)) ok = warp_wait(&t_full[ts], (u / C::TST) & 1, p.err, abort_flag);
          if (st < nst_x) {
            const int f = t_x + st;
            if (ok && f >= 2) ok = warp_wait(&pd[f & 1], ((f >> 1) - 1) & 1, p.err, abort_flag);
            if (!ok) break;
            tc5::fence_after();
            const uint64_t kd = kd0 + static_cast<uint32_t>(ts * (C::kTile >> 4) + (st & 1) * (C::SK * 128 >> 4));
            const uint32_t sd = sd0 + 64u * (f & 1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (kk >> 2) * static_cast<uint64_t>(C::kBlk >> 4) + (kk & 3) * static_cast<uint64_t>(32 >> 4);
              if (kk == 0)
                mma_ss<false>(one, sd, qd, kd, kIdesc);
              else
                mma_ss<true>(one, sd, qd + off, kd + off, kIdesc);
            }
            commit_one(one, &sf[f & 1]);
            if (st == nst_x - 1) commit_one(one, q_empty);
          }
          if (ok && ((st & 1) || st == it.nst - 1)) commit_one(one, &t_empty[ts]);
        }
      });
    } else {
      // O += P V
      constexpr uint32_t kIdesc = idesc_f16_f32(128, D, true);
      const uint64_t vd0 = tc5::smem_desc_mn128(sb + C::OFF_T, C::kBlk);
      const uint32_t od = tmem + C::COL_O + static_cast<uint32_t>(D) * x;
      uint64_t* pf = p_full + 2 * x;
      for_items([&](const Item& it) {
        const int nst_x = x ? it.nst_of[1] : it.nst_of[0], t_x = x ? it.t_of[1] : it.t_of[0];
        bool ok = !*abort_flag;
#pragma unroll 1
        for (int st = 0; st < it.nst && ok; ++st) {
          const int u = 2 * (it.t_glob + (st >> 1)) + 1, ts = u % C::TST;
          if (!(st & 1)) ok = warp_wait(&t_full[ts], (u / C::TST) & 1, p.err, abort_flag);
          if (st < nst_x) {
            const int f = t_x + st;
            if (ok) ok = warp_wait(&pf[f & 1], (f >> 1) & 1, p.err, abort_flag);
            if (!ok) break;
            tc5::fence_after();
            // (an item's first P.V overwrites O: its P comes from warps that have read the last item's)
            const uint64_t vd = vd0 + static_cast<uint32_t>(ts * (C::kTile >> 4) + (st & 1) * (C::SK * 128 >> 4));
            const uint32_t pt = sd0 + 64u * (f & 1);
            if (st == 0)
              mma_ts<false>(one, od, pt, vd, kIdesc);
            else
              mma_ts<true>(one, od, pt, vd, kIdesc);
#pragma unroll
            for (int kk = 1; kk < C::SK / 16; ++kk) mma_ts<true>(one, od, pt + 8u * kk, vd + kk * (2048 >> 4), kIdesc);
            commit_one(one, &pd[f & 1]);
          }
          if (ok && ((st & 1) || st == it.nst - 1)) commit_one(one, &t_empty[ts]);
        }
      });
    }
    commit_one(one, fin);  // every product this warp issued
    __syncwarp();
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 4) {
      // ----------------------------------------------------------------- TMA producer
      int issued = 0;  // tiles
      for_items([&](const Item& it) {
        const int lb = lane & 15;  // this lane's block of the tile
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        auto fetch_block = [&](int jt) -> int {
          const int key0 = it.key0 + jt * C::BK + lb * bs;
          return (jt < it.nkt && lb * bs < C::BK && key0 < it.kv_end) ? btrow[key0 >> p.bs_log2] : 0;
        };
        bool ok = !*abort_flag && !P.fault_no_copies;
        int nb0 = fetch_block(0), nb1 = fetch_block(1);
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          int blk = nb0;
          nb0 = nb1;
          nb1 = fetch_block(jt + 2);
          const int nbox = ceil_div(min(C::BK, it.kv_end - it.key0 - jt * C::BK), bs);
          if (lb < nbox && (blk < 0 || blk >= p.num_blocks)) {
            raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
            blk = 0;
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int u = 2 * (it.t_glob + jt) + kv;  // K and V tiles in turn
            const int rs = u % C::RST;
            if (u >= C::RST) {
              ok = warp_wait(&raw_empty[rs], (u / C::RST - 1) & 1, p.err, abort_flag);
              if (!ok) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[rs], static_cast<uint32_t>(nbox * bs * D));
            __syncwarp();
            if (lane < nbox)
              tma_load_4d(smem + C::OFF_RAW + rs * C::kRaw + lane * bs * D, kv ? &P.tmap_v : &P.tmap_k, 0, it.h, 0,
                          blk, &raw_full[rs], pol);
            // the scales of both come with K's tile (K: lanes 0-15, V: 16-31)
            if (kv == 0 && lb < nbox)
              cp_async<4>(sb + C::OFF_SC + (rs * 32 + lane) * 4,
                          (lane >= 16 ? P.v_scale : P.k_scale) + static_cast<int64_t>(blk) * p.hkv + it.h);
            cp_async_arrive(&raw_full[rs]);
            issued = u + 1;
          }
        }
      });
      // every copy issued has landed before the CTA may leave, also after another role has given up
      for (int u = max(0, issued - C::RST); u < issued; ++u) mbar_wait(&raw_full[u % C::RST], (u / C::RST) & 1, p.err);
    } else {
      // ---------------------------------------------------------------------- Q tiles
      // D / 8 lanes to a row, one 16-byte chunk each; row groups in turn among the three warps
      constexpr int LR = D / 8;       // lanes to a row
      constexpr int RI = 32 / LR;     // rows of a group
      constexpr int NG = 256 / RI;    // groups: A's rows, then B's
      constexpr int NB = 4;           // groups loaded at a time
      const int c = lane % LR, sub = lane / LR;
      for_items([&](const Item& it) {
        bool ok = !*abort_flag;
        unsigned char* qe = qexp + (it.no % 3) * 256;
        const bf16* base = p.q + static_cast<int64_t>(it.s0 + it.q0) * p.q_st + static_cast<int64_t>(it.h * G) * p.q_sh + c * 8;
        uint4 w[NB];
        auto load = [&](int g0) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int r = (g0 + 3 * i) * RI + sub, x = r >> 7;
            const int rt = (r & 127) / G, rg = (r & 127) - rt * G;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < 256 && rt < (x ? it.rows[1] : it.rows[0]))
              w[i] = *reinterpret_cast<const uint4*>(base + static_cast<int64_t>(x * PR + rt) * p.q_st + rg * p.q_sh);
          }
        };
        if (ok) load(warp - 5);  // requested before the wait for the tiles' space
        if (ok && it.no > 0) ok = warp_wait(q_empty, (it.no - 1) & 1, p.err, abort_flag);
        if (ok) {
#pragma unroll 1
          for (int g0 = warp - 5; g0 < NG; g0 += 3 * NB) {
            if (g0 != warp - 5) load(g0);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              if (g0 + 3 * i >= NG) break;
              const int r = (g0 + 3 * i) * RI + sub;
              const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
              unsigned mx = 0;
#pragma unroll
              for (int y = 0; y < 4; ++y) mx = max(mx, max(v[y] & 0x7fffu, (v[y] >> 16) & 0x7fffu));
#pragma unroll
              for (int off = 1; off < LR; off <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
              const int e = min(max(static_cast<int>(mx >> 7), 30), 254);  // biased exponent of the row's largest
              const float up = q8_exp2(127 + 14 + 127 - e);
              uint32_t o[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) o[y] = pack_f16x2(bf16lo(v[y]) * up, bf16hi(v[y]) * up);
              sts128(sb + C::OFF_Q + (r >> 7) * C::kTile + (c >> 3) * C::kBlk + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
                     o[0], o[1], o[2], o[3]);
              if (c == 0) qe[r] = static_cast<unsigned char>(e);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
      });
    }
  } else if (warp >= 16) {
    // ------------------------------------------------------------------- conversion
    const int cw = warp - 16;  // rows 32 cw .. 32 cw + 31 of each tile
    // an 8-lane phase takes 64 bytes of two rows whose swizzles differ, so that neither the
    // 16-byte reads nor the 16-byte writes conflict: rows x and x ^ 5 (128-byte rows), x and x ^ 1 (64)
    const int ph = lane >> 3, sel = (lane >> 2) & 1, cq = lane & 3;
    const int r8 = D == 128 ? (sel ? ph ^ 5 : ph) : 2 * ph + sel;
    for_items([&](const Item& it) {
      bool ok = !*abort_flag;
      int vref = 0;  // biased exponent of O's unit; 0: no tile of this item yet
      int vpeak = 0;  // the highest it has been: how far down it may come (kQ8MaxDown)
      for (int jt = 0; jt < it.nkt && ok; ++jt) {
        const int g = it.t_glob + jt;
        const int vis = it.kv_end - it.key0 - jt * C::BK;  // keys of this tile that some row sees
        const int nbox = ceil_div(min(C::BK, vis), bs);
        int ee = 0, kref = 0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int u = 2 * g + kv;
          const int rs = u % C::RST, ts = u % C::TST;
          ok = warp_wait(&raw_full[rs], (u / C::RST) & 1, p.err, abort_flag);
          if (!ok) break;
          if (kv == 0) {
            // lane: the scale exponent of one block of the tile (K: lanes 0-15, V: 16-31)
            ee = (__float_as_int(*reinterpret_cast<const float*>(smem + C::OFF_SC + (rs * 32 + lane) * 4)) >> 23) & 0xff;
            const bool have = (lane & 15) < nbox;
            const int ktop = __reduce_max_sync(0xffffffffu, have && lane < 16 ? ee : 0);
            const int kmin = __reduce_min_sync(0xffffffffu, have && lane < 16 ? ee : 255);
            const int vtop = __reduce_max_sync(0xffffffffu, have && lane >= 16 ? ee : 0);
            const int vmin = __reduce_min_sync(0xffffffffu, have && lane >= 16 ? ee : 255);
            // scales far apart within a tile: the reference below the largest leaves more room beneath
            kref = ktop - kmin > -kQ8RefLow ? ktop - kQ8RefHigh : ktop;
            const int vnew = vtop - vmin > -kQ8RefLow ? vtop - kQ8RefHigh : vtop;
            if (vref == 0 || ((vtop - vref > kQ8RefHigh || vmin - vref < kQ8RefLow) && vpeak - vnew <= kQ8MaxDown))
              vref = vnew;
            vpeak = max(vpeak, vref);
          }
          if (u >= C::TST) {
            ok = warp_wait(&t_empty[ts], (u / C::TST - 1) & 1, p.err, abort_flag);
            if (!ok) break;
          }
          // (read by both softmaxes before they write P of this tile; the slot's next use waits for a later P.V)
          if (kv == 0 && cw == 0 && lane == 0) {
            refs[2 * (g & 3)] = kref;
            refs[2 * (g & 3) + 1] = vref;
          }
          const uint32_t src = sb + C::OFF_RAW + rs * C::kRaw + 32 * cw * D;
          const uint32_t dst = sb + C::OFF_T + ts * C::kTile + 32 * cw * 128;
          const int ref = kv ? vref : kref;
          if (FMT == PKV_Q8_E4M3 && kv == 1 && it.key0 + jt * C::BK + C::BK - 1 > it.pos0) {
            // keys that some rows of the item do not see: their NaN is taken out of the raw tile (0 times NaN would
            // poison those rows), and the rows that do see it get it back in the end.  (In a loop of its own over the
            // bytes that this lane converts next: done on the registers below, the conversion of every tile was slower
            // and a chunk took 905 us for 765.)
#pragma unroll 1
            for (int x = 0; x < 4 * (D / 64); ++x) {
              const int row = 32 * cw + 8 * (x & 3) + r8;
              if (row >= vis || it.key0 + jt * C::BK + row <= it.pos0) continue;
              const uint32_t at = src + chunk8_off<D>(8 * (x & 3) + r8, 4 * (x >> 2) + cq);
              const uint4 v = lds128(at);
              const uint32_t n[4] = {e4m3_nan_bits(v.x) >> 7, e4m3_nan_bits(v.y) >> 7, e4m3_nan_bits(v.z) >> 7,
                                     e4m3_nan_bits(v.w) >> 7};
              if ((n[0] | n[1] | n[2] | n[3]) != 0u) {
                *nan_seen = 1;
                sts128(at, v.x & ~(n[0] * 0xffu), v.y & ~(n[1] * 0xffu), v.z & ~(n[2] * 0xffu), v.w & ~(n[3] * 0xffu));
              }
            }
          }
          // (an offset of whole 8-row atoms leaves the swizzle as it is)
          uint4 w[4][D / 64];
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int c4 = 0; c4 < D / 64; ++c4) w[a][c4] = lds128(src + chunk8_off<D>(8 * a + r8, 4 * c4 + cq));
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int e = __shfl_sync(0xffffffffu, ee, 16 * kv + ((32 * cw + 8 * a) >> p.bs_log2));
            uint32_t s2, off2;
            q8_f16_pow2(e - ref, s2, off2);
            const bool zero = kv == 1 && 32 * cw + 8 * a + r8 >= vis;  // keys no row sees: 0 * NaN would poison P.V
#pragma unroll
            for (int c4 = 0; c4 < D / 64; ++c4) {
              uint32_t o[8];
              q8_to_f16_scaled<FMT>(w[a][c4].x, s2, off2, o[0], o[1]);
              q8_to_f16_scaled<FMT>(w[a][c4].y, s2, off2, o[2], o[3]);
              q8_to_f16_scaled<FMT>(w[a][c4].z, s2, off2, o[4], o[5]);
              q8_to_f16_scaled<FMT>(w[a][c4].w, s2, off2, o[6], o[7]);
              if (zero) {
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = 0u;
              }
              const int c = 4 * c4 + cq;
              const uint32_t row = dst + (c >> 2) * C::kBlk + (8 * a + r8) * 128;
              const int q = 2 * (c & 3);
              sts128(row + ((q ^ r8) << 4), o[0], o[1], o[2], o[3]);
              sts128(row + (((q + 1) ^ r8) << 4), o[4], o[5], o[6], o[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&t_full[ts]);
            mbar_arrive(&raw_empty[rs]);
          }
        }
      }
    });
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    // -------------------------------------------------------------------- softmax
    const int x = (warp - 8) >> 2;  // Q tile
    const int sw = warp & 3;        // TMEM lanes 32 sw .. 32 sw + 31
    const int r = 32 * sw + lane;
    const int rt = r / G;       // position within the Q tile
    const int rg = r - rt * G;  // q head within the group
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * sw) << 16);
    const uint32_t to = tlane + C::COL_O + static_cast<uint32_t>(D) * x;
    for_items([&](const Item& it) {
      const bool live = rt < (x ? it.rows[1] : it.rows[0]);
      const int nst_x = x ? it.nst_of[1] : it.nst_of[0], t_x = x ? it.t_of[1] : it.t_of[0];
      // (a row past the span's, its q zero, sees everything: its scores need no mask and go nowhere)
      const int pos = live ? it.pos0 + x * PR + rt : INT32_MAX;
      float m_run = NEG_INF, l_run = 0.f;
      float qf = 0.f;
      int vref = 0;
      bool ok = !*abort_flag;
      // One step; 0: a wait gave up, 1: done, 2: left as it was, because a row's maximum became one whose rounding
      // counts.  S fac - m in one rounding has the rounding of m in every exponent: a factor that all weights of a row
      // share, and that would overflow f16 (or take them all to 0) where m is large.  `large` steps, a loop of their
      // own for the rest of the item, round a score as m was.  (In the same loop: 805 to 880 us for a chunk's 765.)
      auto step = [&](auto large, int st) -> int {
        const int f = t_x + st;
        const int g = it.t_glob + (st >> 1);
        const uint32_t ts = tlane + C::COL_S + 128u * x + 64u * (f & 1);
        ok = warp_wait(&s_full[2 * x + (f & 1)], (f >> 1) & 1, p.err, abort_flag);
        if (!ok) return 0;
        tc5::fence_after();
        if (st == 0) qf = p.qscale * q8_exp2(static_cast<int>(qexp[(it.no % 3) * 256 + 128 * x + r]) - 14);
        float sc[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v[32];
          tc5::ld32(ts + 32u * c, v);
#pragma unroll
          for (int y = 0; y < 32; ++y) sc[32 * c + y] = v[y];
        }
        // scores are S fac in the log2 domain (kept from underflowing to 0, which would turn a masked
        // -inf into NaN)
        const float fac = fmaxf(qf * q8_exp2(refs[2 * (g & 3)]), 1.17549435e-38f);
        const int vnew = refs[2 * (g & 3) + 1];
        tc5::wait_ld();
        const int key0 = it.key0 + st * C::SK;
        if (key0 + C::SK - 1 > pos) {
          const int last = pos - key0;  // (may be negative: none)
#pragma unroll
          for (int c = 0; c < 64; ++c) sc[c] = c <= last ? sc[c] : NEG_INF;
        }
        float mx4[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) mx4[y] = fmaxf(sc[y], sc[4 + y]);
#pragma unroll
        for (int c = 8; c < 64; c += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) mx4[y] = fmaxf(fmaxf(mx4[y], sc[c + y]), sc[c + 4 + y]);
        const float mx = fac * fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const bool up = mx - m_run > kQ8Slack;  // (m_run + 8 may be rounded up)
        const bool any_up = __any_sync(0xffffffffu, up);
        if (!decltype(large)::value && any_up && __any_sync(0xffffffffu, up && fabsf(mx) > kExactScore)) return 2;
        float corr = up ? fast_exp2(m_run - mx) : 1.f;  // (0 from the first key that a row sees on)
        m_run = up ? mx : m_run;
        const float m_fin = m_run == NEG_INF ? 0.f : m_run, base = m_fin - kQ8Lift;
        l_run *= corr;
        // O to the new unit (the item's first P.V overwrites it)
        if (vnew != vref && st > 0) {
          const int sh = vref - vnew;
          corr *= sh >= -126 ? q8_exp2(127 + sh) : 0.f;
        }
        const bool resc = any_up || vnew != vref;  // (of some row of the warp)
        vref = vnew;
        const float2 f2 = make_float2(fac, fac);
        const float2 nb2 = make_float2(-base, -base);
        float2 ls4[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) ls4[y] = make_float2(0.f, 0.f);
        float pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float2 t;
          if constexpr (decltype(large)::value)  // (the difference is exact, the lift apart from it)
            t = make_float2(__fadd_rn(__fadd_rn(__fmul_rn(sc[c], fac), -m_fin), kQ8Lift),
                            __fadd_rn(__fadd_rn(__fmul_rn(sc[c + 1], fac), -m_fin), kQ8Lift));
          else
            t = ffma2(make_float2(sc[c], sc[c + 1]), f2, nb2);
          const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
          ls4[(c >> 1) & 3] = fadd2(ls4[(c >> 1) & 3], e);
          pk[c >> 1] = __uint_as_float(pack_f16x2(e.x, e.y));
        }
        tc5::st32(ts, pk);  // P over S
        const float2 ls2 = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
        l_run += ls2.x + ls2.y;
        if (st > 0 && resc) {
          // O is rescaled once the P.V of every step before has landed in it
          ok = warp_wait(&pv_done[2 * x + ((f - 1) & 1)], ((f - 1) >> 1) & 1, p.err, abort_flag);
          if (!ok) return 0;
          tc5::fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc5::ld32(to + 32u * c, o);
            tc5::wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] *= corr;
            tc5::st32(to + 32u * c, o);
          }
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + (f & 1)]);
        return 1;
      };
      int st = 0, how = 1;
      for (; st < nst_x && ok; ++st)
        if ((how = step(std::false_type{}, st)) != 1) break;
      if (how == 2)
#pragma unroll 1
        for (; st < nst_x && ok; ++st)
          if (step(std::true_type{}, st) != 1) break;
      if (nst_x > 0) {
        const int f = t_x + nst_x - 1;
        if (ok) ok = warp_wait(&pv_done[2 * x + (f & 1)], (f >> 1) & 1, p.err, abort_flag);
        tc5::fence_after();
      }
      const float inv = live && nst_x > 0 ? q8_exp2(vref) / l_run : 0.f;
      // columns of this row in which a key that it sees, but not every row of the item, holds a NaN: looked for in the
      // pool itself, once the conversion has met one (so seldom that its time does not count)
      uint32_t nan_at[D / 32] = {};
      if constexpr (FMT == PKV_Q8_E4M3) {
        if (*nan_seen && live) {
          const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
          for (int key = max(it.pos0 + 1, it.key0); key <= min(pos, it.kv_end - 1); ++key) {
            int blk = btrow[key >> p.bs_log2];
            if (blk < 0 || blk >= p.num_blocks) blk = 0;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(P.v_cache +
                (((static_cast<int64_t>(blk) << p.bs_log2) + (key & (bs - 1))) * p.hkv + it.h) * D);
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              for (int y = 0; y < 8; ++y) {
                const uint32_t n = e4m3_nan_bits(v[8 * c + y]) >> 7;  // bits 0, 8, 16, 24
                nan_at[c] |= ((n | n >> 7 | n >> 14 | n >> 21) & 15u) << (4 * y);
              }
          }
        }
        __syncwarp();  // (lanes looked through different numbers of keys)
      }
      auto put_nan = [&](int c, float (&o)[32]) {
        if constexpr (FMT == PKV_Q8_E4M3) {
          if (nan_at[c] == 0u) return;
#pragma unroll
          for (int y = 0; y < 32; ++y)
            if (nan_at[c] >> y & 1u) o[y] = __int_as_float(0x7fffffff);
        }
      };
      if (share > 1) {
        // Every product of both Q tiles has completed once all eight warps are here: the tiles' space takes the
        // rows (each normalised by its own sum) and their (m, l).  16-byte pieces of a row are xored with the row
        // number, so that eight rows' lanes use different banks.
        named_bar_sync(2, 256);
        const int row = 128 * x + r;
        const uint32_t orow = sb + row * (D * 4);
        if (nst_x > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc5::ld32(to + 32u * c, o);
            tc5::wait_ld();
            put_nan(c, o);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              sts128(orow + (((8 * c + y) ^ (row & 7)) << 4), __float_as_uint(o[4 * y] * inv), __float_as_uint(o[4 * y + 1] * inv),
                     __float_as_uint(o[4 * y + 2] * inv), __float_as_uint(o[4 * y + 3] * inv));
          }
        }
        *reinterpret_cast<float2*>(smem + 256 * D * 4 + row * 8) = make_float2(m_run, ok ? l_run : __int_as_float(0x7fffffff));
        cluster_barrier();
        // this CTA's share of the rows: out = sum 2^(m - M) l o / sum 2^(m - M) l over the pieces
        const int first_peer = static_cast<int>(blockIdx.x) % P.pieces - piece;
        const int own = 256 / share;
        const int who = (warp - 8) * 32 + lane;
        for (int i = who; i < own * (D / 4); i += 256) {
          const int jrow = piece * own + i / (D / 4), c = i % (D / 4);
          const int jx = jrow >> 7, jt = (jrow & 127) / G, jg = (jrow & 127) - jt * G;
          if (jt >= (jx ? it.rows[1] : it.rows[0])) continue;
          float M = NEG_INF;
          for (int k = 0; k < share; ++k) M = fmaxf(M, ld_peer_f2(peer_smem(sb + 256 * D * 4 + jrow * 8, first_peer + k)).x);
          const float base = M == NEG_INF ? 0.f : M;
          float den = 0.f;
          float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < share; ++k) {
            const float2 ml = ld_peer_f2(peer_smem(sb + 256 * D * 4 + jrow * 8, first_peer + k));
            if (ml.y == 0.f) continue;  // this piece holds no key of the row, and no row
            const float w = fast_exp2(ml.x - base) * ml.y;
            const float4 o = ld_peer_f4(peer_smem(sb + jrow * (D * 4) + ((c ^ (jrow & 7)) << 4), first_peer + k));
            den += w;
            num.x = fmaf(w, o.x, num.x);
            num.y = fmaf(w, o.y, num.y);
            num.z = fmaf(w, o.z, num.z);
            num.w = fmaf(w, o.w, num.w);
          }
          const float id = 1.f / den;
          uint2 u;
          u.x = pack_bf16x2(num.x * id, num.y * id);
          u.y = pack_bf16x2(num.z * id, num.w * id);
          *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(it.s0 + it.q0 + jx * PR + jt) * p.o_st +
                                    static_cast<int64_t>(it.h * G + jg) * p.o_sh + 4 * c) = u;
        }
      } else if (nst_x > 0 && ok) {
        bf16* orow = p.out + static_cast<int64_t>(it.s0 + it.q0 + x * PR + rt) * p.o_st +
                     static_cast<int64_t>(it.h * G + rg) * p.o_sh;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc5::ld32(to + 32u * c, o);
          tc5::wait_ld();
          put_nan(c, o);
          if (live) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint4 u;
              u.x = pack_bf16x2(o[8 * y + 0] * inv, o[8 * y + 1] * inv);
              u.y = pack_bf16x2(o[8 * y + 2] * inv, o[8 * y + 3] * inv);
              u.z = pack_bf16x2(o[8 * y + 4] * inv, o[8 * y + 5] * inv);
              u.w = pack_bf16x2(o[8 * y + 6] * inv, o[8 * y + 7] * inv);
              *reinterpret_cast<uint4*>(orow + 32 * c + 8 * y) = u;
            }
          }
        }
      }
      tc5::fence_before();
    });
  }
  if (share > 1) {
    if (warp < 8 || warp >= 16) cluster_barrier();  // (the softmax warps' is above)
    cluster_barrier();                              // no CTA leaves while another reads its rows
  }
  __syncthreads();  // every role has finished its last item

  if (warp == 1) {  // no MMA may be in flight when TMEM is released
    mbar_wait(fin, 0, p.err);
    __syncwarp();
    tc5::fence_after();
    tc5::dealloc(tmem, C::TMEM_COLS);
  }
}

// Clusters of `pieces` CTAs that fit the device at a time (asked once for each device and size).
template <int D, int FMT>
int max_clusters(int pieces) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  std::atomic<int>& slot = known[dev][pieces == 8 ? 3 : pieces == 4 ? 2 : 1];
  int n = slot.load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pieces));
    cfg.blockDim = dim3(kPqThreads);
    cfg.dynamicSmemBytes = PrefillQ8Cfg<D>::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(pieces), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, prefill_q8_kernel<D, FMT>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = -1;
    }
    slot.store(n);
  }
  return n > 0 ? n : 0;
}

template <int D, int FMT>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  using C = PrefillQ8Cfg<D>;
  if (const cudaError_t e = set_smem_once<prefill_q8_kernel<D, FMT>>(C::kSmemBytes); e != cudaSuccess) return e;
  PrefillQ8Params P;
  if (!make_pool_map_q8(&P.tmap_k, a.k_cache, a.num_blocks, a.bs_log2, a.hkv, D) ||
      !make_pool_map_q8(&P.tmap_v, a.v_cache, a.num_blocks, a.bs_log2, a.hkv, D))
    return cudaErrorInvalidValue;
  P.p = make_prefill_params(a);
  P.k_scale = a.k_scale;
  P.v_scale = a.v_scale;
  P.v_cache = static_cast<const uint8_t*>(a.v_cache);
  P.group = a.hq / a.hkv;
  P.prows = kTcPrefillRows / P.group;
  P.fault_no_copies = a.fault == PKV_FAULT_PREFILL_NO_COPIES;
  int64_t grid = prefill_q8_grid(a);
  P.pieces = prefill_q8_pieces(a);
  if (P.pieces > 1) {
    const int64_t fit = static_cast<int64_t>(max_clusters<D, FMT>(P.pieces)) * P.pieces;
    if (fit > 0)
      grid = grid < fit ? grid : fit;
    else
      P.pieces = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPqThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (P.pieces > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n++].val.clusterDim = {static_cast<unsigned>(P.pieces), 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  record_kernel_event(PKV_KERNEL_PREFILL, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_q8_kernel<D, FMT>, P);
  record_kernel_event(PKV_KERNEL_PREFILL, true, stream);
  return e;
}

}  // namespace

// CTAs of a cluster that may share an item: more than one where the tokens beyond one a sequence, were they
// all in one span, would not give half the SMs an item (the kernel then decides by the items there are).
int prefill_q8_pieces(const AttnArgs& a) {
  const int64_t prows = 2 * (kTcPrefillRows / (a.hq / a.hkv));
  const int64_t extra = a.num_tokens - a.num_seqs + 1;  // tokens of the longest span there can be, at least
  const int64_t items = ceil_div64(extra > 0 ? extra : 1, prows) * a.hkv;
  return items * 8 <= device_sm_count() ? 8 : items * 2 <= device_sm_count() ? 4 : 1;
}

// One CTA per SM, at most one per item or, where CTAs may share items, a cluster.
int64_t prefill_q8_grid(const AttnArgs& a) {
  const int prows = 2 * (kTcPrefillRows / (a.hq / a.hkv));
  const int64_t pieces = prefill_q8_pieces(a);
  const int64_t max_items = (a.num_tokens / prows + a.num_seqs + 1) * a.hkv * pieces;
  const int64_t cap = device_sm_count() / pieces * pieces;
  return max_items < cap ? max_items : cap;
}

cudaError_t launch_prefill_q8(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch<128, PKV_Q8_INT8>(a, stream, pdl) : launch<64, PKV_Q8_INT8>(a, stream, pdl);
  return a.head_dim == 128 ? launch<128, PKV_Q8_E4M3>(a, stream, pdl) : launch<64, PKV_Q8_E4M3>(a, stream, pdl);
}

}  // namespace pkv
