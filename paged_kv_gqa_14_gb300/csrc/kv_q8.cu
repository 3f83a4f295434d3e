// The 8-bit cache written and read back: fused RoPE + quantisation + append, and the way back to
// bf16.
//
// Append.  The unit is one block of one sequence, because the block's new tokens share a scale: for
// every (K or V, head), a task, four warps (one, where there are four new rows or fewer) read its new rows once,
// find their largest magnitude, take the smallest power of two that holds it (and the block's present scale, if
// rows are there already), round those rows to a scale that grew, and write the new rows.  So a scale is decided
// in one place, and the result does not depend on the order of tokens or CTAs.  Other CTAs of the block
// rotate its tokens' q rows.
//
// The number of blocks a step touches is known on the device only.  A span of n tokens touches at
// most n / bs + 2 blocks, so blocks are numbered from start_b = qsl[b] / bs + 2 b, a non-decreasing
// function of b that leaves room for them all, and a CTA finds its sequence by a warp-wide
// search; with few tokens to a sequence (a decode step) the CTAs are numbered by token instead, and
// those of a block's first new token work.
//
// RoPE for a value that is rounded to eight bits: near a rounding border the fp32 error of sincosf
// decides which way a key goes, so the rotation is carried to 2^-27 of |x| + |y| (the bound; the most of
// four million was 2^-28.3) before it is rounded to fp32.  The angle modulo a turn is exact (RopeFreqs);
// with k the nearest quarter turn and j the nearest 1/64 of one, sin and cos of j pi/128 come from a
// table in two floats, the first of 16 bits, and the rest, |d| <= pi/256, enters through
// sin d = d - d^3/6 and cos d - 1 = -d^2/2 + d^4/24.  A bf16 value times a 16-bit float is exact in
// fp32, and the two exact products are added with their rounding error kept (TwoSum), so one rounding
// to fp32 remains (to odd, see rot).
//
// Bound: for prompts the instructions (2 B in and out per q value, 2 B in and 1 B out per k and v value would be
// 18 us where it takes 40: 8,445 tokens, 16/8 heads, d 128), for a decode step the chain of reads that find a
// token's block (7 us for 8 to 256 tokens).  A task by one warp, sixteen rows in its registers, is less work to
// order, but all its code runs once and waits for instructions a quarter of the time: 46 us; rows shared by four
// warps and tasks in a loop 38 (the rotation rounded to odd another 2).
#include <math.h>

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "q8.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 16;  // rows whose (cos, sin) table and raw values are held at a time
constexpr int kTaskWarps = 4;  // warps that share a task, kChunk / kTaskWarps rows each (one if that is all its rows)

// sin and cos of j pi / 128, j = 0 .. 32: hi has 16 significant bits, hi + lo is good to 2^-41.
struct RopeTrig {
  float s_hi[33], s_lo[33], c_hi[33], c_lo[33];
};

// The last b in [0, n) with start(b) <= x (start non-decreasing), or -1; every lane gets it.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int64_t x, int lane, F start) {
  int lo = 0, hi = n - 1;
  for (int round = 0; round < 8 && lo <= hi; ++round) {  // 32 samples a round: 32^7 covers any int
    const int len = hi - lo + 1;
    const int stride = len <= 32 ? 1 : (len + 31) / 32;
    const int idx = lo + lane * stride;
    const int k = __popc(__ballot_sync(0xffffffffu, idx <= hi && start(idx) <= x)) - 1;
    if (k < 0) return -1;  // (only in the first round)
    if (stride == 1) return lo + k;
    lo += k * stride;
    hi = min(hi, lo + stride - 1);
  }
  return lo;
}

// (cos, sin) of 2 pi turn / 2^64 as {cos hi, cos lo, sin hi, sin lo}, hi of 16 bits.
__device__ __forceinline__ float4 trig_of_turn(unsigned long long turn, const float4* tab) {
  const unsigned k = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
  const long long rem = static_cast<long long>(turn - (static_cast<unsigned long long>(k) << 62));
  const int j = static_cast<int>((rem + (1ll << 55)) >> 56);  // -32 .. 32
  const int d_int = static_cast<int>((rem - (static_cast<long long>(j) << 56)) >> 24);  // |.| <= 2^31
  constexpr float kTwoPiOver2p40 = static_cast<float>(6.283185307179586 / 1099511627776.0);
  const float d = static_cast<float>(d_int) * kTwoPiOver2p40;
  const float d2 = d * d;
  const float sd = fmaf(d * d2, -1.f / 6.f, d);
  const float cd = d2 * fmaf(d2, 1.f / 24.f, -0.5f);  // cos d - 1
  const float4 t = tab[j < 0 ? -j : j];  // {s_hi, s_lo, c_hi, c_lo}
  const float sh = j < 0 ? -t.x : t.x, sl = j < 0 ? -t.y : t.y;
  const float sf = sh + sl, cf = t.z + t.w;
  const float s_lo = sl + fmaf(sf, cd, cf * sd);
  const float c_lo = t.w + fmaf(cf, cd, -(sf * sd));
  switch (k & 3u) {
    case 0: return make_float4(t.z, c_lo, sh, s_lo);
    case 1: return make_float4(-sh, -s_lo, t.z, c_lo);
    case 2: return make_float4(-t.z, -c_lo, -sh, -s_lo);
    default: return make_float4(sh, s_lo, -t.z, -c_lo);
  }
}

// x ch + y sh + (x cl + y sl) with one rounding at the end: x, y have 8 bits and ch, sh 16, so the
// two products are exact.  That rounding is to odd (a sum that is not exact takes the neighbour whose last bit is
// set), so that the rounding to eight bits after it goes as it would from the sum itself: never to a tie that
// the sum is not.
__device__ __forceinline__ float rot(float x, float ch, float cl, float y, float sh, float sl) {
  const float p = x * ch, q = y * sh;
  const float s = p + q;
  const float t = s - p;
  const float e = (p - (s - t)) + (q - t);
  const float c = e + fmaf(x, cl, y * sl);
  const float r = s + c;
  const float b = r - s;
  const float rest = (s - (r - b)) + (c - b);
  int u = __float_as_int(r);
  if (rest != 0.f && (u & 1) == 0) u += (rest < 0.f) == (r < 0.f) ? 1 : -1;  // (r = 0 is exact; a NaN stays one)
  return __int_as_float(u);
}

struct AppendParams {
  bf16* q;
  int64_t q_st, q_sh;
  const bf16* k;
  int64_t k_st, k_sh;
  const bf16* v;
  int64_t v_st, v_sh;
  const int32_t* bt;
  int64_t bt_stride, max_blocks;
  const int32_t* ctxl;
  const int32_t* qsl;
  int num_seqs;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  int64_t num_tokens, num_blocks;
  int bs_log2, hq, hkv;
  int by_token;
  int ny;  // CTAs (blockIdx.y) that share a block's k and v; the rest take its q
  unsigned int* err;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 3)
    kv_append_q8_kernel(const __grid_constant__ AppendParams p, const __grid_constant__ RopeFreqs fr,
                        const __grid_constant__ RopeTrig tg) {
  constexpr int HALF = D / 2;
  constexpr int LPR = D / 4;         // lanes to a row: four values each, (2 l', 2 l' + 1) of either half
  constexpr int RPS = 32 / LPR;      // rows a warp takes in a step
  constexpr int STEPS = kChunk / kTaskWarps / RPS;
  constexpr int QC = HALF / 8;       // 16-byte chunk pairs of a q head row
  // a k CTA's {cos hi, cos lo, sin hi, sin lo}, even pairs before odd ones (a lane takes a pair of each), or a
  // q CTA's {cos, sin}, a gap after every eight (a lane takes eight in a row): no bank conflicts either way
  __shared__ float4 cs[kChunk][HALF];
  static_assert((HALF + HALF / 8) * sizeof(float2) <= HALF * sizeof(float4), "the q table fits");
  __shared__ unsigned long long freq[HALF];
  __shared__ float4 tab[33];
  __shared__ float part_amax[kWarps / kTaskWarps][2][kTaskWarps];
  extern __shared__ unsigned task_amax[];  // [2 hkv], blocks of more than kChunk rows: the bits, then the exponent

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < HALF) freq[tid] = fr.F[tid];
  if (tid >= kThreads - 33) {
    const int j = tid - (kThreads - 33);
    tab[j] = make_float4(tg.s_hi[j], tg.s_lo[j], tg.c_hi[j], tg.c_lo[j]);
  }
  pdl_wait();  // q, k, v and the tables may come from the previous kernel
  pdl_trigger();

  // the sequence b and logical block jb of this CTA
  const int bs_log2 = p.bs_log2;
  const int64_t c = blockIdx.x;
  const int32_t* qsl = p.qsl;
  int b;
  if (p.by_token)
    b = warp_search(p.num_seqs, c, lane, [&](int i) -> int64_t { return qsl[i]; });
  else
    b = warp_search(p.num_seqs, c, lane, [&](int i) -> int64_t { return (qsl[i] >> bs_log2) + 2ll * i; });
  if (b < 0) return;
  const int64_t s0 = qsl[b], n = static_cast<int64_t>(qsl[b + 1]) - s0, ctx = p.ctxl[b];
  if (n <= 0) {
    if (n < 0 && tid == 0 && blockIdx.y == 0) raise_error(p.err, PKV_DEVERR_SPAN);
    return;
  }
  if (s0 < 0 || s0 + n > p.num_tokens || ctx < n) {
    if (tid == 0 && blockIdx.y == 0) raise_error(p.err, PKV_DEVERR_SPAN);
    return;
  }
  const int64_t first = ctx - n;  // position of the span's first token
  const int64_t c_first = p.by_token ? s0 : (s0 >> bs_log2) + 2ll * b;
  if (c < c_first) {  // (the search may end behind c where starts go back)
    if (tid == 0 && blockIdx.y == 0) raise_error(p.err, PKV_DEVERR_SPAN);
    return;
  }
  int64_t jb;
  if (p.by_token) {
    if (c - s0 >= n) return;  // a row outside every span
    const int64_t pos = first + (c - s0);
    if (c != s0 && (pos & ((1 << bs_log2) - 1)) != 0) return;  // not its block's first new token
    jb = pos >> bs_log2;
  } else {
    jb = (first >> bs_log2) + (c - c_first);
    if (jb > ((ctx - 1) >> bs_log2)) return;
  }
  const int64_t p_lo = max(first, jb << bs_log2), p_hi = min(ctx, (jb + 1) << bs_log2);
  const int r0 = static_cast<int>(p_lo - (jb << bs_log2));  // rows there already
  const int m = static_cast<int>(p_hi - p_lo);              // new rows
  const int64_t t0 = s0 + (p_lo - first);                   // their first token
  int blk = -1;
  if (jb >= p.max_blocks) {
    if (tid == 0 && blockIdx.y == 0) raise_error(p.err, PKV_DEVERR_CONTEXT);
  } else {
    blk = p.bt[b * p.bt_stride + jb];
    if (blk < 0 || blk >= p.num_blocks) {
      if (tid == 0 && blockIdx.y == 0) raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
      blk = -1;
    }
  }
  const int hkv = p.hkv;
  const int ntasks = 2 * hkv;  // task < hkv: K of that head, else V
  const int lr = lane % LPR, lrow = lane / LPR;
  const int64_t block_row = static_cast<int64_t>(blk) << bs_log2;  // (unused when blk < 0)
  __syncthreads();  // freq and tab

  auto each_angle = [&](int c0, auto&& put) {
    const int rows = min(kChunk, m - c0);
    for (int idx = tid; idx < rows * HALF; idx += kThreads) {
      const int r = idx / HALF, i = idx - r * HALF;
      put(r, i, trig_of_turn(static_cast<unsigned long long>(p_lo + c0 + r) * freq[i], tab));
    }
  };

  if (static_cast<int>(blockIdx.y) >= p.ny) {
    // ------------------------------------------------------------------ q rows, every head, in place
    // (fp32, rounded to bf16; eight pairs a thread at a time, kBatch of them requested before the angles)
    constexpr int kBatch = 4;
    const int nq = gridDim.y - p.ny;
    const int per_row = p.hq * QC;
    for (int c0 = (blockIdx.y - p.ny) * kChunk; c0 < m; c0 += nq * kChunk) {
      const int items = min(kChunk, m - c0) * per_row;
      uint4 lo[kBatch], hi[kBatch];
      auto place = [&](int idx, int& r, int& ch) -> bf16* {
        r = idx / per_row;
        const int rest = idx - r * per_row, h = rest / QC;
        ch = rest - h * QC;
        return p.q + (t0 + c0 + r) * p.q_st + h * p.q_sh + ch * 8;
      };
      auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int idx = base + j * kThreads;
          if (idx < items) {
            int r, ch;
            const bf16* at = place(idx, r, ch);
            lo[j] = *reinterpret_cast<const uint4*>(at);
            hi[j] = *reinterpret_cast<const uint4*>(at + HALF);
          }
        }
      };
      load(tid);
      __syncthreads();  // (the last chunk's table has been read)
      each_angle(c0, [&](int r, int i, float4 t) {
        reinterpret_cast<float2*>(cs[r])[i + (i >> 3)] = make_float2(t.x + t.y, t.z + t.w);
      });
      __syncthreads();
      for (int base = tid; base < items; base += kBatch * kThreads) {
        if (base != tid) load(base);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int idx = base + j * kThreads;
          if (idx >= items) break;
          int r, ch;
          bf16* at = place(idx, r, ch);
          uint32_t* aw = reinterpret_cast<uint32_t*>(&lo[j]);
          uint32_t* ew = reinterpret_cast<uint32_t*>(&hi[j]);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 f0 = reinterpret_cast<const float2*>(cs[r])[ch * 9 + 2 * w];
            const float2 f1 = reinterpret_cast<const float2*>(cs[r])[ch * 9 + 2 * w + 1];
            const float c0f = f0.x, s0f = f0.y, c1f = f1.x, s1f = f1.y;
            const float x0 = bf16lo(aw[w]), x1 = bf16hi(aw[w]), y0 = bf16lo(ew[w]), y1 = bf16hi(ew[w]);
            aw[w] = pack_bf16x2(x0 * c0f - y0 * s0f, x1 * c1f - y1 * s1f);
            ew[w] = pack_bf16x2(y0 * c0f + x0 * s0f, y1 * c1f + x1 * s1f);
          }
          *reinterpret_cast<uint4*>(at) = lo[j];
          *reinterpret_cast<uint4*>(at + HALF) = hi[j];
        }
      }
    }
    return;
  }

  // ---------------------------------------------------------------------------- k and v tasks
  if (blk < 0) return;  // (CTA-uniform) the block has no place: nothing is written
  auto build_table = [&](int c0) {
    each_angle(c0, [&](int r, int i, float4 t) { cs[r][(i & 1) * (HALF / 2) + (i >> 1)] = t; });
  };
  const int tw = m <= kChunk / kTaskWarps ? 1 : kTaskWarps;
  const int groups = kWarps / tw, group = warp / tw, wi = warp % tw;
  const int wrow = wi * (kChunk / kTaskWarps);  // this warp's first row of a chunk
  static_assert(kWarps / kTaskWarps == 2, "a barrier each");
  auto task_sync = [&] {  // the task's warps (with tw > 1)
    if (group == 0)
      named_bar_sync(1, kTaskWarps * 32);
    else
      named_bar_sync(2, kTaskWarps * 32);
  };
  // four values of each of this lane's rows, rows c0 + wrow + i RPS + lrow: as read, then as fp32 (k rotated)
  struct Rows {
    uint32_t lo[STEPS], hi[STEPS];
  };
  float4 x[STEPS];
  auto load_rows = [&](int task, int c0, Rows& raw) {
    const bool is_v = task >= hkv;
    const int h = is_v ? task - hkv : task;
    const bf16* src = is_v ? p.v + t0 * p.v_st + h * p.v_sh : p.k + t0 * p.k_st + h * p.k_sh;
    const int64_t st = is_v ? p.v_st : p.k_st;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = c0 + wrow + i * RPS + lrow;
      raw.lo[i] = raw.hi[i] = 0u;
      if (r < m) {
        const bf16* row = src + r * st + 2 * lr;
        raw.lo[i] = *reinterpret_cast<const uint32_t*>(row);
        raw.hi[i] = *reinterpret_cast<const uint32_t*>(row + HALF);
      }
    }
  };
  auto to_values = [&](int task, const Rows& raw) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const float x0 = bf16lo(raw.lo[i]), x1 = bf16hi(raw.lo[i]), y0 = bf16lo(raw.hi[i]), y1 = bf16hi(raw.hi[i]);
      if (task >= hkv) {
        x[i] = make_float4(x0, x1, y0, y1);
      } else {
        const float4* row = cs[wrow + i * RPS + lrow];
        const float4 a = row[lr], e = row[HALF / 2 + lr];  // pairs 2 lr and 2 lr + 1
        x[i] = make_float4(rot(x0, a.x, a.y, y0, -a.z, -a.w), rot(x1, e.x, e.y, y1, -e.z, -e.w),
                           rot(y0, a.x, a.y, x0, a.z, a.w), rot(y1, e.x, e.y, x1, e.z, e.w));
      }
    }
  };
  // the largest finite magnitude of this warp's rows, as its bits (magnitudes order like their bits, infinities
  // and NaN last); its sign set: there are values that are not finite
  auto rows_amax = [&](int c0) -> float {
    constexpr unsigned kInf = 0x7f800000u;
    unsigned a = 0u;
    auto take = [&](bool finite_only) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        if (c0 + wrow + i * RPS + lrow >= m) continue;
        const float y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const unsigned b = __float_as_uint(y[j]) & 0x7fffffffu;
          a = max(a, finite_only && b >= kInf ? 0u : b);
        }
      }
      a = __reduce_max_sync(0xffffffffu, a);
    };
    take(false);
    if (a >= kInf) {  // (warp-uniform)
      if (lane == 0) raise_error(p.err, PKV_DEVERR_NONFINITE);
      a = 0u;
      take(true);
      return -__uint_as_float(a);
    }
    return __uint_as_float(a);
  };
  auto old_exp = [&](int task) -> int {
    if (r0 == 0) return 0;
    const bool is_v = task >= hkv;
    const int h = is_v ? task - hkv : task;
    const unsigned bits = __float_as_uint((is_v ? p.v_scale : p.k_scale)[static_cast<int64_t>(blk) * hkv + h]);
    return min(max(static_cast<int>((bits >> 23) & 0xffu), kQ8MinScaleExp), 253);
  };
  // The block's scale from the new rows' amax and, with rows there already, its present one (which every warp of
  // the task has read); rows there already are rounded to a scale that grew, by the task's warps in turn.
  // Returns the biased exponent.
  auto settle_scale = [&](int task, float amax, int e_old) -> int {
    const bool is_v = task >= hkv;
    const int h = is_v ? task - hkv : task;
    int e = q8_scale_exp<FMT>(amax);
    if (r0 > 0) {
      if (e > e_old) {
        uint8_t* base = (is_v ? p.v_cache : p.k_cache) + (block_row * hkv + h) * D + 4 * lr;
        const float f = q8_exp2(max(127 + e_old - e, 1));  // (below 2^-126 every value rounds to 0 anyway)
        for (int r = wi * RPS + lrow; r < r0; r += tw * RPS) {
          uint32_t* at = reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(r) * hkv * D);
          float y[4];
          q8_to_f32<FMT>(*at, y);
          *at = q8_pack2<FMT>(y[0] * f, y[1] * f) | (q8_pack2<FMT>(y[2] * f, y[3] * f) << 16);
        }
      } else {
        e = e_old;
      }
    }
    if (wi == 0 && lane == 0) (is_v ? p.v_scale : p.k_scale)[static_cast<int64_t>(blk) * hkv + h] = q8_exp2(e);
    return e;
  };
  // (plain: every value is finite and fits the scale, and int8 needs no clamps)
  auto write_rows = [&](int task, int c0, int e, bool plain) {
    const bool is_v = task >= hkv;
    const int h = is_v ? task - hkv : task;
    uint8_t* base = (is_v ? p.v_cache : p.k_cache) + ((block_row + r0) * hkv + h) * D + 2 * lr;
    const float inv = q8_inv_exp2(e);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = c0 + wrow + i * RPS + lrow;
      if (r < m) {
        uint8_t* at = base + static_cast<int64_t>(r) * hkv * D;
        uint32_t a, b;
        if (plain) {
          a = q8_pack2_plain<FMT>(x[i].x, x[i].y, inv);
          b = q8_pack2_plain<FMT>(x[i].z, x[i].w, inv);
        } else {
          a = q8_pack2<FMT>(x[i].x * inv, x[i].y * inv);
          b = q8_pack2<FMT>(x[i].z * inv, x[i].w * inv);
        }
        *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(a);
        *reinterpret_cast<uint16_t*>(at + HALF) = static_cast<uint16_t>(b);
      }
    }
  };

  // this CTA's share of the tasks, in a row (so that with CTAs enough only half of them need the angles), its
  // groups in turn
  const int per = (ntasks + p.ny - 1) / p.ny;
  const int task0 = static_cast<int>(blockIdx.y) * per + group, end = min(ntasks, task0 - group + per);
  const bool any_k = task0 - group < hkv;
  Rows raw;
  if (m <= kChunk) {
    // a task's rows are requested before the angles are computed, and the next one's before this one's amax
    int task = task0;
    int e_old = 0;
    if (task < end) {
      load_rows(task, 0, raw);
      e_old = old_exp(task);
    }
    if (any_k) build_table(0);
    __syncthreads();
#pragma unroll 1
    for (int turn = 0; task < end; turn ^= 1) {
      to_values(task, raw);
      const int next = task + groups, e_task = e_old;
      if (next < end) {
        load_rows(next, 0, raw);
        e_old = old_exp(next);
      }
      float amax = rows_amax(0);
      bool finite = !signbit(amax);
      amax = fabsf(amax);
      if (tw > 1) {
        float* part = part_amax[group][turn];  // (its last readers have passed the barrier of the turn between)
        if (lane == 0) part[wi] = finite ? amax : -amax;
        task_sync();
#pragma unroll
        for (int w = 0; w < kTaskWarps; ++w) {
          amax = fmaxf(amax, fabsf(part[w]));
          finite = finite && !signbit(part[w]);
        }
      }
      const int e = settle_scale(task, amax, e_task);
      write_rows(task, 0, e, finite && e < q8_max_exp<FMT>());
      task = next;
    }
    return;
  }
  // a block of more rows: the amax over all chunks first, then every chunk again
  for (int task = tid; task < ntasks; task += kThreads) task_amax[task] = 0u;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int c0 = 0; c0 < m; c0 += kChunk) {
      int task = task0;
      if (task < end) load_rows(task, c0, raw);
      __syncthreads();
      if (any_k) build_table(c0);
      __syncthreads();
#pragma unroll 1
      while (task < end) {
        to_values(task, raw);
        const int next = task + groups;
        if (next < end) load_rows(next, c0, raw);
        if (pass == 0) {
          const float a = fabsf(rows_amax(c0));
          if (lane == 0) atomicMax(task_amax + task, __float_as_uint(a));
        } else {
          write_rows(task, c0, static_cast<int>(task_amax[task]), false);
        }
        task = next;
      }
    }
    if (pass == 1) break;
    __syncthreads();
#pragma unroll 1
    for (int task = task0; task < end; task += groups) {
      const int e_old = old_exp(task);
      const float amax = __uint_as_float(task_amax[task]);
      task_sync();  // the present scale and the amax have been read by every warp
      const int e = settle_scale(task, amax, e_old);
      if (wi == 0 && lane == 0) task_amax[task] = static_cast<unsigned>(e);
    }
  }
}

// ------------------------------------------------------------------------------ reading back
struct ReadParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* bt;
  int64_t bt_stride, max_blocks;
  const int32_t* ctxl;
  const int32_t* rsl;
  int num_seqs;
  bf16* k_out;
  int64_t ko_st, ko_sh;
  bf16* v_out;
  int64_t vo_st, vo_sh;
  int64_t num_rows, num_blocks;
  int bs_log2, hkv;
  int rows;  // of a warp, at most 32
  unsigned int* err;
};

// bf16(held * scale), a warp to p.rows consecutive output rows (one search for them), whose 16-value pieces its
// lanes take in turn, kReadBatch of them requested together: at 1 kv head a row is eight or sixteen pieces, and
// a row to a step left lanes idle (524,288 rows of d 64 160 us, now 41).  Bound: memory; 50 sequences of up to 8192
// keys, 4 heads d 128, 191 us, 0.96 of a copy's rate.
constexpr int kReadBatch = 4;
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_q8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int CH = D / 16;  // 16-value pieces of a head row
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * p.rows;
  if (row0 >= p.num_rows) return;
  const int b0 = warp_search(p.num_seqs, row0, lane, [&](int i) -> int64_t { return p.rsl[i]; });
  // lane r < rows: the pool row of output row row0 + r (-1: none) and its block
  int64_t slot = -1;
  if (b0 >= 0 && lane < p.rows && row0 + lane < p.num_rows) {
    const int64_t row = row0 + lane;
    // the last sequence that starts at or before the row: in strides that double, then between the last two (a lane's
    // sequence is mostly b0 or the next, but a batch may have any number without rows between them)
    int b = b0;
    for (int step = 1; step > 0;) {
      if (step < p.num_seqs - b && p.rsl[b + step] <= row) {
        b += step;
        step <<= 1;
      } else {
        while ((step >>= 1) > 0)
          if (step < p.num_seqs - b && p.rsl[b + step] <= row) b += step;
      }
    }
    const int64_t s0 = p.rsl[b], n = static_cast<int64_t>(p.rsl[b + 1]) - s0, ctx = p.ctxl[b];
    if (row - s0 < n) {
      const int64_t pos = ctx - n + (row - s0);
      // (row < s0: the search may end behind the row where starts go back)
      if (s0 < 0 || row < s0 || s0 + n > p.num_rows || ctx < n) {
        raise_error(p.err, PKV_DEVERR_SPAN);
      } else if ((pos >> p.bs_log2) >= p.max_blocks) {
        raise_error(p.err, PKV_DEVERR_CONTEXT);
      } else {
        const int blk = p.bt[b * p.bt_stride + (pos >> p.bs_log2)];
        if (blk < 0 || blk >= p.num_blocks)
          raise_error(p.err, PKV_DEVERR_BLOCK_RANGE);
        else
          slot = (static_cast<int64_t>(blk) << p.bs_log2) + (pos & ((1 << p.bs_log2) - 1));
      }
    } else if (n < 0) {
      raise_error(p.err, PKV_DEVERR_SPAN);
    }
  }
  const int per_row = p.hkv * CH;  // pieces of a row of K, and of V
  const int items = p.rows * 2 * per_row;
  for (int base = lane; base - lane < items; base += 32 * kReadBatch) {
    uint4 w[kReadBatch];
    float f[kReadBatch];
    bf16* dst[kReadBatch];
#pragma unroll
    for (int j = 0; j < kReadBatch; ++j) {
      const int idx = base + 32 * j;
      const int r = idx / (2 * per_row);
      const int64_t s = __shfl_sync(0xffffffffu, slot, r & 31);
      dst[j] = nullptr;
      if (idx < items && s >= 0) {
        const int in_row = idx - r * 2 * per_row;
        const bool is_v = in_row >= per_row;
        const int rest = is_v ? in_row - per_row : in_row;
        const int h = rest / CH, ch = rest - h * CH;
        w[j] = *reinterpret_cast<const uint4*>((is_v ? p.v_cache : p.k_cache) + s * p.hkv * D + rest * 16);
        f[j] = (is_v ? p.v_scale : p.k_scale)[(s >> p.bs_log2) * p.hkv + h];
        dst[j] = (is_v ? p.v_out + (row0 + r) * p.vo_st + h * p.vo_sh : p.k_out + (row0 + r) * p.ko_st + h * p.ko_sh) +
                 ch * 16;
      }
    }
#pragma unroll
    for (int j = 0; j < kReadBatch; ++j) {
      if (dst[j] == nullptr) continue;
      const uint32_t in[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        q8_to_f32<FMT>(in[i], x);
        o[2 * i] = pack_bf16x2(x[0] * f[j], x[1] * f[j]);
        o[2 * i + 1] = pack_bf16x2(x[2] * f[j], x[3] * f[j]);
      }
      uint4* out = reinterpret_cast<uint4*>(dst[j]);
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

const RopeTrig& rope_trig() {
  static const RopeTrig t = [] {
    RopeTrig r;
    for (int j = 0; j <= 32; ++j) {
      const double a = j * (M_PI / 128.0);
      auto split = [](double x, float* hi, float* lo) {
        int e = 0;
        const double m = frexp(x, &e);  // x = m 2^e, m in [0.5, 1) or 0
        *hi = static_cast<float>(ldexp(nearbyint(ldexp(m, 16)), e - 16));
        *lo = static_cast<float>(x - static_cast<double>(*hi));
      };
      split(sin(a), &r.s_hi[j], &r.s_lo[j]);
      split(cos(a), &r.c_hi[j], &r.c_lo[j]);
    }
    return r;
  }();
  return t;
}

template <int D, int FMT>
cudaError_t launch_append(const Q8AppendArgs& a, cudaStream_t stream) {
  AppendParams p;
  p.q = static_cast<bf16*>(a.q);
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.k = static_cast<const bf16*>(a.k);
  p.k_st = a.k_st;
  p.k_sh = a.k_sh;
  p.v = static_cast<const bf16*>(a.v);
  p.v_st = a.v_st;
  p.v_sh = a.v_sh;
  p.bt = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctxl = a.context_lens;
  p.qsl = a.qsl;
  p.num_seqs = static_cast<int>(a.num_seqs);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.num_blocks;
  p.bs_log2 = a.bs_log2;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.err = a.err;
  // numbered by token, or by block with two spare numbers to a sequence: whichever is fewer CTAs
  const int64_t by_block = (a.num_tokens >> a.bs_log2) + 2 * a.num_seqs;
  p.by_token = a.num_tokens <= by_block;
  // A block's k and v tasks sixteen to a CTA, or fewer, down to two, where there are few blocks: a CTA's start (four
  // reads that depend on one another) is long beside its work, so no more of them than run at once, or half as
  // many more where a block has several chunks.  Its q by CTAs of their own, a chunk each.  Measured on GB300 (16/8
  // heads, d 128), 1 / 2 / 3 / 6 CTAs an SM: 256 decodes 6.9 / 7.9 / 9.8 / - us; 8192 tokens in blocks of 16 30.6 /
  // 30.6 / 32.1 / 36.5, of 64 75 / 41.7 / 47.8 / 48.4, of 128 139 / 58.3 / 48.0 / 47.9.
  const int chunks = p.by_token || (1 << a.bs_log2) <= kChunk ? 1 : (1 << a.bs_log2) / kChunk;
  const int64_t blocks = p.by_token ? a.num_tokens : by_block;
  const int64_t sms = device_sm_count();
  const int64_t target = p.by_token ? sms : chunks == 1 ? 2 * sms : 3 * sms;
  const int64_t least = (2 * a.hkv + 15) / 16, wanted = (target + blocks - 1) / blocks;
  p.ny = static_cast<int>(wanted <= least ? least : wanted < a.hkv ? wanted : a.hkv);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.ny + chunks));
  record_kernel_event(PKV_KERNEL_APPEND, false, stream);
  const cudaError_t e =
      launch_pdl(kv_append_q8_kernel<D, FMT>, grid, dim3(kThreads), sizeof(unsigned) * 2 * a.hkv, stream, p,
                 rope_freqs(a.theta, a.head_dim), rope_trig());
  record_kernel_event(PKV_KERNEL_APPEND, true, stream);
  return e;
}

template <int D, int FMT>
cudaError_t launch_read(const Q8ReadArgs& a, cudaStream_t stream) {
  ReadParams p;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.bt = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctxl = a.context_lens;
  p.rsl = a.rsl;
  p.num_seqs = static_cast<int>(a.num_seqs);
  p.k_out = static_cast<bf16*>(a.k_out);
  p.ko_st = a.ko_st;
  p.ko_sh = a.ko_sh;
  p.v_out = static_cast<bf16*>(a.v_out);
  p.vo_st = a.vo_st;
  p.vo_sh = a.vo_sh;
  p.num_rows = a.num_rows;
  p.num_blocks = a.num_blocks;
  p.bs_log2 = a.bs_log2;
  p.hkv = a.hkv;
  p.err = a.err;
  // Rows of a warp: two, four or eight pieces to a lane.  Few, and a small call fills the GPU; many, and the
  // search and the block table's entry serve more bytes.  Measured on GB300, two / four / eight: a quarter of a
  // million pieces 7.5 / 9.4 / 10.6 us, half a million 8.8 / 9.9 / 10.8, one million 13.4 / 12.7 / 15.1, two
  // 23.3 / 20.7 / 21.5, four 47.2 / 41.4 / 41.3, 33 million 331 / 279 / 269.
  const int per_row = 2 * a.hkv * (D / 16);
  const int64_t pieces = a.num_rows * per_row;
  const int lane_pieces = pieces < (1 << 20) ? 2 : pieces < (1 << 22) ? 4 : 8;
  p.rows = 32 * lane_pieces / per_row;
  if (p.rows < 1) p.rows = 1;
  const int64_t per_cta = static_cast<int64_t>(kWarps) * p.rows;
  return launch_pdl(kv_read_q8_kernel<D, FMT>, dim3(static_cast<unsigned>((a.num_rows + per_cta - 1) / per_cta)),
                    dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_append_q8(const Q8AppendArgs& a, cudaStream_t stream) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch_append<128, PKV_Q8_INT8>(a, stream) : launch_append<64, PKV_Q8_INT8>(a, stream);
  return a.head_dim == 128 ? launch_append<128, PKV_Q8_E4M3>(a, stream) : launch_append<64, PKV_Q8_E4M3>(a, stream);
}

cudaError_t launch_kv_read_q8(const Q8ReadArgs& a, cudaStream_t stream) {
  if (a.format == PKV_Q8_INT8)
    return a.head_dim == 128 ? launch_read<128, PKV_Q8_INT8>(a, stream) : launch_read<64, PKV_Q8_INT8>(a, stream);
  return a.head_dim == 128 ? launch_read<128, PKV_Q8_E4M3>(a, stream) : launch_read<64, PKV_Q8_E4M3>(a, stream);
}

}  // namespace pkv
