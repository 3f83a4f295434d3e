// Prefill-chunk attention over an 8-bit cache on the 5th-generation tensor cores.
//
// Items, causal rule and the tcgen05 products are the bf16 prefill's (prefill_tc.cuh): an item is
// (sequence, floor(128 / G) positions of its span, kv head), its 128-row Q tile stacks the G query
// heads of the kv head, and S = Q K^T and O += P V run as kind::f16 with accumulators in TMEM.
// The tensor cores read neither int8 nor a scale per block, so every K/V tile of 128 keys is
// turned into f16 in shared memory first:
//
//   held 2^(e - ref)  with ref one exponent per tile for K and one per item for V
//
// which is exact in f16 while e is not far below ref (the products are then those of the
// dequantised cache); S is multiplied by 2^ref 2^eq in the softmax, where q entered as q 2^-eq
// with its largest magnitude in [2^14, 2^15), and O is in units of 2^ref.  The V reference moves to
// a tile whose scales leave the window around it; the softmax warps then rescale O as they do when
// a row's maximum grows.
//
// One CTA of twelve warps:
//   warp 0      TMA producer: raw K and V tiles (one box per block), scales by cp.async, two stages
//   warp 1      TMEM, and the MMA issue from one thread
//   warps 2, 3  Q tiles: plain loads (any strides), row maximum, f16, swizzled store
//   warps 4-7   softmax, thread = row: S from TMEM, P (f16) back to TMEM, O rescale, output
//   warps 8-11  conversion of the raw tiles to f16
// Items follow one another without a CTA barrier, and every wait is bounded.
#include <cuda.h>

#include "decode_tc.cuh"
#include "prefill.cuh"
#include "prefill_tc.cuh"
#include "q8.cuh"
#include "tcgen05.cuh"

namespace pkv {

bool make_pool_map_q8(CUtensorMap* m, const void* base, int64_t num_blocks, int bs_log2, int hkv, int D);

namespace {

constexpr int kPqThreads = 384;
constexpr int kConvWarps = 4;

struct PrefillQ8Params {
  CUtensorMap tmap_k;  // 4-D {d, Hkv, block_size, num_blocks} of bytes, box {d, 1, block_size, 1}
  CUtensorMap tmap_v;
  PrefillParams p;
  const float* k_scale;
  const float* v_scale;
  int group;  // G
  int prows;  // floor(128 / G): positions per item
};

template <int D>
struct PrefillQ8Cfg {
  static constexpr int BK = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int kBlk = 128 * 128;          // [128 rows][64 f16], 128-byte swizzled
  static constexpr int kTile = HALVES * kBlk;     // a Q, K or V tile in f16
  static constexpr int kRaw = BK * D;             // a K or V tile as held
  static constexpr int RST = 2;                   // raw stages (K and V)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = kTile;             // two stages
  static constexpr int OFF_V = OFF_K + 2 * kTile; // two stages
  static constexpr int OFF_RAW = OFF_V + 2 * kTile;
  static constexpr int OFF_QF = OFF_RAW + RST * 2 * kRaw;  // [3][128] row factors
  static constexpr int OFF_SC = OFF_QF + 3 * 128 * 4;      // [RST][K|V][16] scales
  static constexpr int OFF_REF = OFF_SC + RST * 32 * 4;    // [4] {K reference, V reference}
  static constexpr int OFF_BAR = OFF_REF + 4 * 8;
  static constexpr int kSmemBytes = OFF_BAR + 26 * 8 + 16 + 1024;  // + barriers + alignment slack
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 256;
  static constexpr uint32_t COL_P = 384;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// Instruction descriptor of a kind::f16 MMA with f16 operands (as tc5::idesc_bf16_f32, whose
// operand format fields are 0 for f16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major = false) {
  return tc5::idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}

template <int D, int FMT>
__global__ void __launch_bounds__(kPqThreads, 1) prefill_q8_kernel(const __grid_constant__ PrefillQ8Params P) {
  using C = PrefillQ8Cfg<D>;
  const PrefillParams& p = P.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  float* qfac = reinterpret_cast<float*>(smem + C::OFF_QF);
  volatile int* refs = reinterpret_cast<volatile int*>(smem + C::OFF_REF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_full = bars + 0;   // [2] TMA bytes and the producer lanes' cp.async
  uint64_t* raw_empty = bars + 2;  // [2] converted
  uint64_t* q_full = bars + 4;
  uint64_t* q_empty = bars + 5;    // every QK of an item completed
  uint64_t* k_full = bars + 6;     // [2]
  uint64_t* k_empty = bars + 8;    // [2]
  uint64_t* v_full = bars + 10;    // [2]
  uint64_t* v_empty = bars + 12;   // [2]
  uint64_t* s_full = bars + 14;    // [2]
  uint64_t* s_free = bars + 16;    // [2]
  uint64_t* p_full = bars + 18;    // [2]
  uint64_t* pv_done = bars + 20;   // [2]
  uint64_t* o_free = bars + 22;
  uint64_t* fin = bars + 23;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 24);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 25);
  const float NEG_INF = -__int_as_float(0x7f800000);
  // P.V of tile t completes pv_done[t % 2] for the (t / 2)-th time
  auto pv_wait = [&](int t) { return warp_wait(&pv_done[t & 1], (t >> 1) & 1, p.err, abort_flag); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&raw_full[s], 33);
      mbar_init(&raw_empty[s], kConvWarps);
      mbar_init(&k_full[s], kConvWarps);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], kConvWarps);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 2);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 4);
    mbar_init(fin, 1);
    fence_mbar_init();
    *abort_flag = 0;
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
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int total = p.plan.header[3] * p.hkv;
  const int nact = min(max(p.plan.header[5], 0), static_cast<int>(gridDim.x));
  if (static_cast<int>(blockIdx.x) >= total || static_cast<int>(blockIdx.x) >= nact) {  // no item in any wave
    if (warp == 1) tc5::dealloc(tmem, C::TMEM_COLS);
    return;
  }
  const int G = P.group;
  const int PR = P.prows;
  const uint64_t pol = l2_policy_evict_last();  // K/V tiles are read again by the other items

  // every role walks the CTA's items by itself: body(item)
  struct Item {
    int no, t_glob;  // items and tiles of this CTA before this one
    int h, b, s0, q0, qrows, pos0, kv_end, nkt;
  };
  auto for_items = [&](auto&& body) {
    Item it;
    it.no = it.t_glob = 0;
    for (int wave = 0; wave * nact < total; ++wave) {
      const int ord = snake_order(wave, blockIdx.x, nact);
      if (ord >= total) continue;
      const int item = total - 1 - ord;  // later (longer) tiles of each span first
      const int ti = item / p.hkv;
      it.h = item - ti * p.hkv;
      it.b = p.plan.pf_seq[ti];
      it.s0 = p.qsl[it.b];
      const int n = p.qsl[it.b + 1] - it.s0;
      it.q0 = p.plan.pf_tile[ti] * PR;
      it.qrows = min(PR, n - it.q0);
      it.pos0 = p.context_lens[it.b] - n + it.q0;
      it.kv_end = it.pos0 + it.qrows;  // keys [0, kv_end) are visible to some row
      it.nkt = ceil_div(it.kv_end, C::BK);
      body(it);
      it.t_glob += it.nkt;
      ++it.no;
    }
  };
  const int bs = 1 << p.bs_log2;

  // Registers go to the softmax warps (a row of 128 scores each): 120 + 240 + 144 a thread of the
  // three warpgroups, the 3 x 168 of the launch.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 0) {
      // ----------------------------------------------------------------- TMA producer
      for_items([&](const Item& it) {
        const bool is_v = lane >= 16;
        const int lb = lane & 15;  // this lane's block of the tile (K: lanes 0-15, V: 16-31)
        const int32_t* btrow = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        auto fetch_block = [&](int jt) -> int {
          const int key0 = jt * C::BK + lb * bs;
          return (jt < it.nkt && lb * bs < C::BK && key0 < it.kv_end) ? btrow[key0 >> p.bs_log2] : 0;
        };
        bool ok = !*abort_flag;
        int nb0 = fetch_block(0), nb1 = fetch_block(1);
        for (int jt = 0; jt < it.nkt && ok; ++jt) {
          const int f = it.t_glob + jt;
          const int rs = f % C::RST;
          int blk = nb0;
          nb0 = nb1;
          nb1 = fetch_block(jt + 2);
          if (f >= C::RST) {
            ok = warp_wait(&raw_empty[rs], (f / C::RST - 1) & 1, p.err, abort_flag);
            if (!ok) break;
          }
          const int nbox = ceil_div(min(C::BK, it.kv_end - jt * C::BK), bs);
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[rs], static_cast<uint32_t>(2 * nbox * bs * D));
          __syncwarp();
          if (lb < nbox) {
            if (blk < 0 || blk >= p.num_blocks) {
              raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
              blk = 0;
            }
            tma_load_4d(smem + C::OFF_RAW + (2 * rs + (is_v ? 1 : 0)) * C::kRaw + lb * bs * D,
                is_v ? &P.tmap_v : &P.tmap_k, 0, it.h, 0, blk, &raw_full[rs], pol);
            cp_async<4>(sb + C::OFF_SC + (rs * 32 + lane) * 4,
                (is_v ? P.v_scale : P.k_scale) + static_cast<int64_t>(blk) * p.hkv + it.h);
          }
          cp_async_arrive(&raw_full[rs]);
        }
      });
    } else if (warp == 1) {
      // ------------------------------------------------------------------- MMA issuer
      if (lane == 0) {
        for_items([&](const Item& it) {
          constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128);
          constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, true);
          bool ok = wait_or_abort(q_full, it.no & 1, p.err, abort_flag);
          auto issue_pv = [&](int fp, bool first) -> bool {
            const int s = fp & 1;
            if (!wait_or_abort(&v_full[s], (fp >> 1) & 1, p.err, abort_flag)) return false;
            if (!wait_or_abort(&p_full[s], (fp >> 1) & 1, p.err, abort_flag)) return false;
            // the item's first P.V overwrites O: the previous item's epilogue must have read it
            if (first && it.no > 0 && !wait_or_abort(o_free, (it.no - 1) & 1, p.err, abort_flag)) return false;
            tc5::fence_after();
            const uint32_t vst = sb + C::OFF_V + s * C::kTile;
#pragma unroll
            for (int kk = 0; kk < C::BK / 16; ++kk)
              tc5::mma_ts(tmem + C::COL_O, tmem + C::COL_P + 64u * s + 8u * kk,
                  tc5::smem_desc_mn128(vst + kk * 2048, C::kBlk), kIdescPV, (first && kk == 0) ? 0u : 1u);
            tc5::commit(&pv_done[s]);
            tc5::commit(&v_empty[s]);
            return true;
          };
          for (int jt = 0; jt < it.nkt && ok; ++jt) {
            const int f = it.t_glob + jt;
            const int s = f & 1;
            ok = wait_or_abort(&k_full[s], (f >> 1) & 1, p.err, abort_flag);
            if (ok && f >= 2) ok = wait_or_abort(&s_free[s], ((f >> 1) - 1) & 1, p.err, abort_flag);
            if (!ok) break;
            tc5::fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::kBlk + (kk & 3) * 32;
              tc5::mma_ss(tmem + 128u * s, tc5::smem_desc_k128(sb + C::OFF_Q + off),
                  tc5::smem_desc_k128(sb + C::OFF_K + s * C::kTile + off), kIdescQK, kk > 0 ? 1u : 0u);
            }
            tc5::commit(&s_full[s]);
            tc5::commit(&k_empty[s]);
            if (jt == it.nkt - 1) tc5::commit(q_empty);
            if (jt > 0) ok = issue_pv(f - 1, jt == 1);
          }
          if (ok) issue_pv(it.t_glob + it.nkt - 1, it.nkt == 1);
        });
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------------- Q tiles
      // warp 2: rows 0-63, warp 3: rows 64-127; D / 8 lanes to a row, one 16-byte chunk each
      for_items([&](const Item& it) {
        bool ok = !*abort_flag;
        constexpr int LR = D / 8;         // lanes to a row
        constexpr int RI = 32 / LR;       // rows an instruction
        constexpr int NI = 64 / RI;       // row groups of this warp
        const int c = lane % LR, sub = lane / LR;
        float* qf = qfac + (it.no % 3) * 128;
        uint4 w[16];
        auto load = [&](int base) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = 64 * (warp - 2) + (base + x) * RI + sub;
            const int rt = r / G, rg = r - rt * G;
            w[x] = make_uint4(0u, 0u, 0u, 0u);
            if (rt < it.qrows)
              w[x] = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(it.s0 + it.q0 + rt) * p.q_st +
                  static_cast<int64_t>(it.h * G + rg) * p.q_sh + c * 8);
          }
        };
        if (ok) load(0);  // requested before the wait for the tile's space
        if (ok && it.no > 0) ok = warp_wait(q_empty, (it.no - 1) & 1, p.err, abort_flag);
        if (ok) {
#pragma unroll
          for (int base = 0; base < NI; base += 16) {
            if (base > 0) load(base);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const int r = 64 * (warp - 2) + (base + x) * RI + sub;
              const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
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
              sts128(sb + C::OFF_Q + (c >> 3) * C::kBlk + r * 128 + (((c & 7) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              if (c == 0) qf[r] = p.qscale * q8_exp2(e - 14);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
      });
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 144;");
    // ------------------------------------------------------------------- conversion
    const int cw = warp - 8;  // rows 32 cw .. 32 cw + 31 of each tile
    for_items([&](const Item& it) {
      bool ok = !*abort_flag;
      int vref = 0;  // biased exponent of O's unit; 0: no tile of this item yet
      for (int jt = 0; jt < it.nkt && ok; ++jt) {
        const int f = it.t_glob + jt;
        const int rs = f % C::RST;
        const int s = f & 1;
        ok = warp_wait(&raw_full[rs], (f / C::RST) & 1, p.err, abort_flag);
        if (!ok) break;
        const int vis = it.kv_end - jt * C::BK;  // keys of this tile that some row sees
        const int nbox = ceil_div(min(C::BK, vis), bs);
        // lane: the scale exponent of one block of the tile (K: lanes 0-15, V: 16-31)
        const int ee = (__float_as_int(*reinterpret_cast<const float*>(smem + C::OFF_SC + (rs * 32 + lane) * 4)) >> 23) & 0xff;
        const bool have = (lane & 15) < nbox;
        const int ktop = __reduce_max_sync(0xffffffffu, have && lane < 16 ? ee : 0);
        const int kmin = __reduce_min_sync(0xffffffffu, have && lane < 16 ? ee : 255);
        const int vtop = __reduce_max_sync(0xffffffffu, have && lane >= 16 ? ee : 0);
        const int vmin = __reduce_min_sync(0xffffffffu, have && lane >= 16 ? ee : 255);
        // scales far apart within a tile: the reference below the largest leaves more room beneath
        const int kref = ktop - kmin > -kQ8RefLow ? ktop - kQ8RefHigh : ktop;
        const int vnew = vtop - vmin > -kQ8RefLow ? vtop - kQ8RefHigh : vtop;
        if (vref == 0)
          vref = vnew;
        else if ((vtop - vref > kQ8RefHigh || vmin - vref < kQ8RefLow) && vref - vnew <= kQ8MaxDown)
          vref = vnew;
        if (f >= 2) ok = warp_wait(&k_empty[s], ((f >> 1) - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        if (cw == 0 && lane == 0) {  // (read by the softmax warps before they free S of this tile)
          refs[2 * (f & 3)] = kref;
          refs[2 * (f & 3) + 1] = vref;
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (kv == 1) {
            if (f >= 2) ok = warp_wait(&v_empty[s], ((f >> 1) - 1) & 1, p.err, abort_flag);
            if (!ok) break;
          }
          const uint32_t src = sb + C::OFF_RAW + (2 * rs + kv) * C::kRaw;
          const uint32_t dst = sb + (kv ? C::OFF_V : C::OFF_K) + s * C::kTile;
          const int ref = kv ? vref : kref;
          // an 8-lane phase takes 64 bytes of two rows whose swizzles differ, so that neither the
          // 16-byte reads nor the 16-byte writes conflict: rows x and x ^ 5 (128-byte rows), x and x ^ 1 (64)
          const int ph = lane >> 3, sel = (lane >> 2) & 1, cq = lane & 3;
          const int r8 = D == 128 ? (sel ? ph ^ 5 : ph) : 2 * ph + sel;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int r = 32 * cw + 8 * a + r8;
            const int e = __shfl_sync(0xffffffffu, ee, 16 * kv + ((32 * cw + 8 * a) >> p.bs_log2));
            uint32_t s2, off2;
            q8_f16_pow2(e - ref, s2, off2);
            const bool zero = kv == 1 && r >= vis;  // keys no row sees: 0 * NaN would poison P.V
#pragma unroll
            for (int c4 = 0; c4 < D / 64; ++c4) {
              const int c = 4 * c4 + cq;
              const uint4 w = lds128(src + chunk8_off<D>(r, c));
              uint32_t o[8];
              q8_to_f16_scaled<FMT>(w.x, s2, off2, o[0], o[1]);
              q8_to_f16_scaled<FMT>(w.y, s2, off2, o[2], o[3]);
              q8_to_f16_scaled<FMT>(w.z, s2, off2, o[4], o[5]);
              q8_to_f16_scaled<FMT>(w.w, s2, off2, o[6], o[7]);
              if (zero) {
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = 0u;
              }
              const uint32_t row = dst + (c >> 2) * C::kBlk + r * 128;
              const int q = 2 * (c & 3);
              sts128(row + ((q ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              sts128(row + (((q + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv ? &v_full[s] : &k_full[s]);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
      }
    });
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    // -------------------------------------------------------------------- softmax
    const int sw = warp - 4;  // TMEM lanes 32 sw .. 32 sw + 31
    const int r = 32 * sw + lane;
    const int rt = r / G;          // position within the item
    const int rg = r - rt * G;     // q head within the group
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * sw) << 16);
    for_items([&](const Item& it) {
      const bool live = rt < it.qrows;
      const int pos = it.pos0 + rt;
      float m_run = NEG_INF, l_run = 0.f;
      float qf = 0.f;
      int vref = 0;
      bool ok = !*abort_flag;
      for (int jt = 0; jt < it.nkt && ok; ++jt) {
        const int f = it.t_glob + jt;
        const int s = f & 1;
        ok = warp_wait(&s_full[s], (f >> 1) & 1, p.err, abort_flag);
        if (!ok) break;
        tc5::fence_after();
        if (jt == 0) qf = qfac[(it.no % 3) * 128 + r];
        // scores are S fac in the log2 domain (kept from underflowing to 0, which would turn a masked
        // -inf into NaN)
        const float fac = fmaxf(qf * q8_exp2(refs[2 * (f & 3)]), 1.17549435e-38f);
        const int vnew = refs[2 * (f & 3) + 1];
        float sc[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tc5::ld32(trow + 128u * s + 32u * c, v);
#pragma unroll
          for (int x = 0; x < 32; ++x) sc[32 * c + x] = v[x];
        }
        tc5::wait_ld();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[s]);
        const int key0 = jt * C::BK;
        float mx8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) mx8[x] = NEG_INF;
        if (live && key0 + C::BK - 1 <= pos) {
#pragma unroll
          for (int c = 0; c < 128; ++c) mx8[c & 7] = fmaxf(mx8[c & 7], sc[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            sc[c] = (live && key0 + c <= pos) ? sc[c] : NEG_INF;
            mx8[c & 7] = fmaxf(mx8[c & 7], sc[c]);
          }
        }
        const float mx = fac * fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
            fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        float corr = 1.f;
        bool resc = false;
        if (m_run == NEG_INF) {
          m_run = mx;
        } else if (mx > m_run + kQ8Slack) {
          corr = fast_exp2(m_run - mx);
          m_run = mx;
          resc = true;
        }
        const float base = (m_run == NEG_INF ? 0.f : m_run) - kQ8Lift;
        const float2 f2 = make_float2(fac, fac);
        const float2 nb2 = make_float2(-base, -base);
        float2 ls4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ls4[x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float2 t = ffma2(make_float2(sc[c], sc[c + 1]), f2, nb2);
          sc[c] = fast_exp2(t.x);
          sc[c + 1] = fast_exp2(t.y);
          ls4[(c >> 1) & 3] = fadd2(ls4[(c >> 1) & 3], make_float2(sc[c], sc[c + 1]));
        }
        const float2 ls2 = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
        l_run = l_run * corr + (ls2.x + ls2.y);
        // O to the new unit (the item's first P.V overwrites it)
        if (vnew != vref && jt > 0) {
          const int sh = vref - vnew;
          corr *= sh >= -126 ? q8_exp2(127 + sh) : 0.f;
          resc = true;
        }
        vref = vnew;
        if (jt > 0 && __any_sync(0xffffffffu, resc)) {
          // O is rescaled only once every P.V issued so far has landed in it
          ok = pv_wait(f - 1);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc5::ld32(trow + C::COL_O + 32u * c, o);
            tc5::wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= corr;
            tc5::st32(trow + C::COL_O + 32u * c, o);
          }
          tc5::wait_st();
        }
        if (f >= 2) {  // this P buffer was read by the P.V of tile f - 2
          ok = pv_wait(f - 2);
          if (!ok) break;
          tc5::fence_after();
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float pk[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) pk[x] = __uint_as_float(pack_f16x2(sc[64 * c + 2 * x], sc[64 * c + 2 * x + 1]));
          tc5::st32(trow + C::COL_P + 64u * s + 32u * c, pk);
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
      }
      if (ok) ok = pv_wait(it.t_glob + it.nkt - 1);
      if (ok) {
        tc5::fence_after();
        const float inv = live ? q8_exp2(vref) / l_run : 0.f;
        bf16* orow = p.out + static_cast<int64_t>(it.s0 + it.q0 + rt) * p.o_st + static_cast<int64_t>(it.h * G + rg) * p.o_sh;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc5::ld32(trow + C::COL_O + 32u * c, o);
          tc5::wait_ld();
          if (live) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint4 u;
              u.x = pack_bf16x2(o[8 * x + 0] * inv, o[8 * x + 1] * inv);
              u.y = pack_bf16x2(o[8 * x + 2] * inv, o[8 * x + 3] * inv);
              u.z = pack_bf16x2(o[8 * x + 4] * inv, o[8 * x + 5] * inv);
              u.w = pack_bf16x2(o[8 * x + 6] * inv, o[8 * x + 7] * inv);
              *reinterpret_cast<uint4*>(orow + 32 * c + 8 * x) = u;
            }
          }
        }
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
    });
  }
  __syncthreads();  // every role has finished its last item

  if (warp == 1) {  // no MMA may be in flight when TMEM is released
    if (lane == 0) {
      tc5::commit(fin);
      mbar_wait(fin, 0, p.err);
    }
    __syncwarp();
    tc5::fence_after();
    tc5::dealloc(tmem, C::TMEM_COLS);
  }
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
  P.group = a.hq / a.hkv;
  P.prows = kTcPrefillRows / P.group;
  record_kernel_event(PKV_KERNEL_PREFILL, false, stream);
  const cudaError_t e = launch_kernel(pdl, prefill_q8_kernel<D, FMT>, dim3(static_cast<unsigned>(prefill_q8_grid(a))),
                                      dim3(kPqThreads), C::kSmemBytes, stream, P);
  record_kernel_event(PKV_KERNEL_PREFILL, true, stream);
  return e;
}

}  // namespace

// One CTA per SM, at most one per item.
int64_t prefill_q8_grid(const AttnArgs& a) {
  const int prows = kTcPrefillRows / (a.hq / a.hkv);
  const int64_t max_items = (a.num_tokens / prows + a.num_seqs + 1) * a.hkv;
  const int64_t cap = device_sm_count();
  return max_items < cap ? max_items : cap;
}

cudaError_t launch_prefill_q8(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch<128, PKV_Q8_INT8>(a, stream, pdl) : launch<64, PKV_Q8_INT8>(a, stream, pdl);
  return a.head_dim == 128 ? launch<128, PKV_Q8_E4M3>(a, stream, pdl) : launch<64, PKV_Q8_E4M3>(a, stream, pdl);
}

}  // namespace pkv
