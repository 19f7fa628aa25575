// Attention of the video tokens to an encoder's states of another length, forward (sm_100a:
// tcgen05 + TMEM + TMA), persistent.
//
//   s_ij = scale q_i . k_j over the valid keys j of the batch item
//   lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
//
// One pass over the keys with a running reference maximum and sum in fp32. A row without a valid
// key gives 0 and lse = -inf.
//
// Work unit: 256 query rows (two blocks A and B of one 128-row tensor tile) of one item and key
// head, over all its key tiles or, where the units alone would leave SMs idle, over one of
// several parts of them; a second kernel then joins the parts. One CTA per SM takes every
// gridDim-th unit: units of one key head are neighbours, so its keys and values stay in L2.
// Each key tile is 128 keys wide: at N = 64 the tensor pipe would wait for shared memory (the
// two operands of a 128 x 64 x 16 step are read in 48 cycles and multiplied in 32; of a
// 128 x 128 x 16 step, 64 and 64).
//
// CTA roles (512 threads): warps 0-3 and 4-7 are the softmax of blocks A and B, a row (TMEM lane)
// a thread; warps 8-11 write the finished blocks out (normalise, stage in shared memory, one
// copy of the whole block); lane 0 of warp 12 loads Q and the K ring; warp 13 loads the V ring
// and zeroes rows of masked keys; warp 14 issues all products. A block's scores are 128
// TMEM columns, P overwrites them as bf16 pairs, and the block's next scores follow its P V in the
// pipe's issue order. One thread issues for A and B in turn: that keeps the blocks half a period
// apart, so that one multiplies while the other exponentiates (with an issuer for each, their
// products interleaved in the pipe, both softmaxes waited and then shared the exponential unit:
// 4200 cycles for a key tile of both blocks, the sum of the two parts).
//
// Roundings to fewer bits: P to bf16 for the P V product, the output once. The sum of a row is
// that of the unrounded probabilities.
//
// Measured, one B200, 12 heads of 128: 32760 queries over 512 keys 110 us (0.93 PFLOP/s; profiled by
// itself, with cold caches, 123 us, the tensor pipe 47 % busy, DRAM 16 %), over 4096 keys 706 and 788 us in two passes (1.17 and 1.05 PFLOP/s),
// over 128 keys 52 us (0.5 PFLOP/s, 3.9 TB/s). What bounds it is the chain of a block, scores to
// maximum to exponentials to P V to the next scores, some 2000 cycles of softmax and 1100 to 1400
// of products for a key tile, of which two blocks hide half; with few key tiles, the change of units.
#include "cross.cuh"
#include "once.cuh"

#include <math.h>

namespace bsa {
namespace {

using namespace cross;

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128;
constexpr int kRegsSoftmax = 176;
constexpr int kRegsOut = 64;
constexpr int kRegsControl = 96;
static_assert(128 * (2 * kRegsSoftmax + kRegsOut + kRegsControl) <= kThreads * kRegsLaunch,
              "register split above the launch's pool");
constexpr float kRescaleLog2 = 8.0f;     // O is rescaled only past 2^8 of growth

template <int D>
struct Cfg {
  static constexpr int kTile = kCrossTile * D * 2;        // bytes of a 128-row tile
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kOut = kV + kStages * kTile;       // staging of one finished block
  static constexpr int kInv = kOut + kTile;               // [2][128] 1 / row sum
  static constexpr int kBar = kInv + 2 * kCrossTile * 4;
  // kfull, kempty, vfull, vempty, vland [kStages each]; qfull, qempty, sfull, pfull (by half), odone, lfull,
  // oempty [2 each]; drain
  static constexpr int kBars = 5 * kStages + 17;
  static constexpr int kMisc = kBar + 8 * kBars;          // TMEM base, abort
  static constexpr int kSmem = 1024 + kMisc + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

template <int D>
struct Bars {
  static constexpr int S = Cfg<D>::kStages;
  uint32_t b0;
  __device__ uint32_t kfull(int s) const { return b0 + 8 * s; }
  __device__ uint32_t kempty(int s) const { return b0 + 8 * (S + s); }
  __device__ uint32_t vfull(int s) const { return b0 + 8 * (2 * S + s); }
  __device__ uint32_t vempty(int s) const { return b0 + 8 * (3 * S + s); }
  __device__ uint32_t vland(int s) const { return b0 + 8 * (4 * S + s); }
  __device__ uint32_t qfull(int x) const { return b0 + 8 * (5 * S + x); }
  __device__ uint32_t qempty(int x) const { return b0 + 8 * (5 * S + 2 + x); }
  __device__ uint32_t sfull(int x) const { return b0 + 8 * (5 * S + 4 + x); }
  __device__ uint32_t pfull(int x, int half) const { return b0 + 8 * (5 * S + 6 + 2 * x + half); }
  __device__ uint32_t odone(int x) const { return b0 + 8 * (5 * S + 10 + x); }
  __device__ uint32_t lfull(int x) const { return b0 + 8 * (5 * S + 12 + x); }
  __device__ uint32_t oempty(int x) const { return b0 + 8 * (5 * S + 14 + x); }
  __device__ uint32_t drain() const { return b0 + 8 * (5 * S + 16); }
};

struct FwdArgs {
  CrossGeom g;
  KeySet keys;
  int units, splits, nqb;            // nqb: pairs of query tiles of a key head
  FastDiv by_nqb, by_splits;
  int qb_mul, kb_mul, vb_mul;        // 0 where one item's tensor serves every item
  __nv_bfloat16* out;
  float* lse;
  float* part_o;                     // splits > 1: [splits, B, N, H, D], each part's own output
  float* part_lse;                   // [splits, B, H, N], in units of log 2
  uint32_t* err;
  float scale_log2;
};

// One unit: its item, key head, first token, and its range of key tiles. Units follow one another
// in the same object, so that an item's length is read once.
struct Unit {
  int b = -1, hkv, n0, part, t0, t1, len;
  __device__ __forceinline__ void open(const FwdArgs& a, int u) {
    const int before = b;
    const int rest = (int)a.by_nqb.q((uint32_t)u), bh = (int)a.by_splits.q((uint32_t)rest);
    part = rest - bh * a.splits;
    b = (int)a.g.by_hkv.q((uint32_t)bh);
    hkv = bh - b * a.g.Hkv;
    n0 = (u - rest * a.nqb) * 2 * a.g.tpt;
    if (b != before) len = item_keys(a.keys, b, a.g.M).x;
    const int nt = (len + kCrossTile - 1) / kCrossTile;
    t0 = 0;
    t1 = nt;
    if (a.splits > 1) {
      t0 = (int)((long long)nt * part / a.splits);
      t1 = (int)((long long)nt * (part + 1) / a.splits);
    }
  }
};

// Scores of masked keys (clear bits of `w`) become -inf, whatever they were: the maximum and the
// exponentials then need no mask.
__device__ __forceinline__ void mask32(uint32_t* r, uint32_t w) {
#pragma unroll
  for (int c = 0; c < 32; ++c) r[c] = ((w >> c) & 1u) ? r[c] : 0xff800000u;
}

// Row maximum over 32 columns, in four chains.
__device__ __forceinline__ void max32(const uint32_t* r, float (&m)[4]) {
#pragma unroll
  for (int c = 0; c < 32; c += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max3(m[j], __uint_as_float(r[c + 2 * j]), __uint_as_float(r[c + 2 * j + 1]));
}

// p = 2^(c s - m) of 32 columns, stored as 16 columns of bf16 pairs; their fp32 sum joins `sum`.
__device__ __forceinline__ void exp32(const uint32_t* r, float c, float m, uint64_t (&sum)[2], uint32_t taddr) {
  const uint64_t cc = f2(c, c), mm = f2(-m, -m);
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    uf2(ffma2(f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), cc, mm), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    pk[i] = pack_bf16x2(p0, p1);
    sum[i & 1] = fadd2(sum[i & 1], f2(p0, p1));
  }
  tmem_st_x16(taddr, pk);
}

// A key tile in the order in which the issuer meets them: the tiles of a unit, then the next unit
// with any. `rows[x]` counts the units of block x so far, empty ones included.
struct TileCursor {
  Unit t;
  int u, kt, t0, t1;
  bool valid, has_b;
  uint32_t rows[2];
  __device__ __forceinline__ void open(const FwdArgs& a, int from) {
    for (u = from; u < a.units; u += gridDim.x) {
      t.open(a, u);
      has_b = t.n0 + a.g.tpt < a.g.N;
      ++rows[0];
      rows[1] += has_b;
      t0 = kt = t.t0;
      t1 = t.t1;
      if (t0 < t1) {
        valid = true;
        return;
      }
    }
    valid = false;
  }
  __device__ __forceinline__ void next(const FwdArgs& a) {
    if (++kt == t1) open(a, u + (int)gridDim.x);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const FwdArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = ptx::smem_u32(smem);
  const CrossGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars<D> bar{sbase + C::kBar};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  float* s_inv = reinterpret_cast<float*>(smem + C::kInv);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(bar.kfull(s), 1);
      ptx::mbar_init(bar.kempty(s), 1);
      ptx::mbar_init(bar.vfull(s), 1);
      ptx::mbar_init(bar.vempty(s), 1);
      ptx::mbar_init(bar.vland(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(bar.qfull(x), 1);
      ptx::mbar_init(bar.qempty(x), 1);
      ptx::mbar_init(bar.sfull(x), 1);
      for (int h = 0; h < 2; ++h) ptx::mbar_init(bar.pfull(x, h), 4);     // one arrival per softmax warp
      ptx::mbar_init(bar.odone(x), 1);
      ptx::mbar_init(bar.lfull(x), 4);
      ptx::mbar_init(bar.oempty(x), 4);       // one per output warp
    }
    ptx::mbar_init(bar.drain(), 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 14) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;           // S_A at 0, S_B at 128, O_A at 256, O_B at 256 + D

  if (warp >= 12) {
    ptx::setmaxnreg_dec<kRegsControl>();
    if (warp == 12) {
      // ------------------------------------------------------------- Q and the K ring
      if (lane == 0) {
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        uint32_t nk = 0, nq[2] = {0, 0};
        bool ok = true;
        const uint32_t qbytes = (uint32_t)(g.G * g.tpt * D * 2);
        Unit t, f;
        for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
          t.open(a, u);
          auto load_q = [&](int x) {
            const int n = t.n0 + x * g.tpt;
            if (n >= g.N) return true;
            if (nq[x] > 0 && !wait_phase(bar.qempty(x), (nq[x] - 1) & 1, abort, a.err)) return false;
            ptx::mbar_arrive_expect_tx(bar.qfull(x), qbytes);
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb)
              tma_load_4d(sbase + C::kQ + x * C::kTile + cb * (kCrossTile * 128), &tmQ, bar.qfull(x), cb * 64,
                          t.hkv * g.G, n, t.b * a.qb_mul);
            ++nq[x];
            return true;
          };
          for (int kt = t.t0; kt < t.t1 && ok; ++kt) {
            // Q_A, first key tile, Q_B, the other key tiles: what the first products need first
            if (kt == t.t0 && !load_q(0)) { ok = false; break; }
            const int s = (int)(nk % S);
            if (!wait_phase(bar.kempty(s), ((nk / S) & 1) ^ 1, abort, a.err)) { ok = false; break; }
            ptx::mbar_arrive_expect_tx(bar.kfull(s), C::kTile);
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb)
              tma_load_4d(sbase + C::kK + s * C::kTile + cb * (kCrossTile * 128), &tmK, bar.kfull(s), cb * 64, t.hkv,
                          kt * kCrossTile, t.b * a.kb_mul);
            ++nk;
            if (kt == t.t0 && !load_q(1)) { ok = false; break; }
              // The next unit's queries come from HBM meanwhile: their buffers are free only when
              // this unit's last scores are done.
              if (kt == t.t0 && u + (int)gridDim.x < a.units) {
                f.open(a, u + (int)gridDim.x);
                for (int x = 0; x < 2; ++x)
                  if (f.t0 < f.t1 && f.n0 + x * g.tpt < g.N)
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                      tma_prefetch_4d(&tmQ, cb * 64, f.hkv * g.G, f.n0 + x * g.tpt, f.b * a.qb_mul);
              }
          }
        }
        // Never leave with copies in flight.
        int zero = 0;
        for (uint32_t s = 0; s < S; ++s)
          if (nk > s) wait_phase(bar.kfull((int)s), ((nk - 1 - s) / S) & 1, &zero, a.err);
        for (int x = 0; x < 2; ++x)
          if (nq[x] > 0) wait_phase(bar.qfull(x), (nq[x] - 1) & 1, &zero, a.err);
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------- the V ring
      // A tile with masked keys lands on a barrier of its own; its masked rows are zeroed before
      // the issuer sees it (zero probability times an infinity would be a NaN).
      uint32_t nv = 0, land[S];
#pragma unroll
      for (int s = 0; s < S; ++s) land[s] = 0;
      bool ok = true;
      Unit t;
      for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
        t.open(a, u);
        for (int kt = t.t0; kt < t.t1; ++kt) {
          const int s = (int)(nv % S);
          if (!warp_wait(bar.vempty(s), ((nv / S) & 1) ^ 1, abort, a.err)) { ok = false; break; }
          // keys past M are filled with zeros by the copy itself
          const uint4 w = tile_bits(a.keys, t.b, kt, g.nkt, t.len);
          const bool scrub = (a.keys.bits || a.keys.kv_len) && !all_set(w);
          const uint32_t full = scrub ? bar.vland(s) : bar.vfull(s);
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(full, C::kTile);
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb)
              tma_load_4d(sbase + C::kV + s * C::kTile + cb * (kCrossTile * 128), &tmV, full, cb * 64, t.hkv,
                          kt * kCrossTile, t.b * a.vb_mul);
          }
          __syncwarp();
          if (scrub) {
            uint32_t ph = 0;
#pragma unroll
            for (int i = 0; i < S; ++i)
              if (i == s) ph = land[i]++ & 1;
            // the copy is in flight: its landing is waited for even when the launch is given up
            int zero = 0;
            const bool in = __all_sync(0xffffffffu, wait_phase(bar.vland(s), ph, &zero, a.err));
            if (!in) { *abort = 1; ok = false; break; }
            zero_masked_rows<D>(smem + C::kV + s * C::kTile, w, lane);
            if (lane == 0) ptx::mbar_arrive(bar.vfull(s));
          }
          ++nv;
        }
      }
      int zero = 0;
      for (uint32_t s = 0; s < S; ++s)
        if (nv > s) wait_phase(bar.vfull((int)s), ((nv - 1 - s) / S) & 1, &zero, a.err);
    } else if (warp == 14) {
      // ------------------------------------------------------------- MMA issuer
      // For each key tile, A and then B: P V of this tile, then the scores of the next (which
      // may be the next unit's first). The warp runs whole; one lane issues.
      uint32_t nk = 0, nv = 0, np[2] = {0, 0}, nq[2] = {0, 0};
      auto wait = [&](uint32_t b, uint32_t ph) { return warp_wait(b, ph, abort, a.err); };
      TileCursor nxt;
      nxt.rows[0] = nxt.rows[1] = 0;
      nxt.open(a, blockIdx.x);
      auto scores = [&](int x) {
        const int s = (int)(nk % S);
        if (nxt.kt == nxt.t0 && !wait(bar.qfull(x), nq[x]++ & 1)) return false;
        if (x == 0 && !wait(bar.kfull(s), (nk / S) & 1)) return false;
        ptx::tc_fence_after();
        const bool last = nxt.kt == nxt.t1 - 1, release = x == 1 || !nxt.has_b;
        if (elect_one()) {
          product_nt<D>(tmem + 128u * (uint32_t)x, sbase + C::kQ + x * C::kTile, sbase + C::kK + s * C::kTile);
          ptx::mma_commit(bar.sfull(x));
          if (last) ptx::mma_commit(bar.qempty(x));
          if (release) ptx::mma_commit(bar.kempty(s));
        }
        __syncwarp();
        nk += release;
        return true;
      };
      bool ok = !nxt.valid || (scores(0) && (!nxt.has_b || scores(1)));
      while (ok && nxt.valid) {
        const bool first = nxt.kt == nxt.t0, last = nxt.kt == nxt.t1 - 1, has_b = nxt.has_b;
        const uint32_t rows[2] = {nxt.rows[0], nxt.rows[1]};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x == 0 || has_b) {
            const int s = (int)(nv % S);
            if (x == 0 && !wait(bar.vfull(s), (nv / S) & 1)) { ok = false; break; }
            if (!wait(bar.pfull(x, 0), np[x] & 1)) { ok = false; break; }
            // The unit before must have been read out of O. Behind the probabilities, not ahead of
            // them: this warp passes over units without keys, whose phases of oempty it does not see,
            // and the probabilities say that the softmax has seen all but the last (a wait that is
            // two phases behind looks complete).
            if (first && rows[x] > 1 && !wait(bar.oempty(x), rows[x] & 1)) { ok = false; break; }
            ptx::tc_fence_after();
            const uint32_t o_tmem = tmem + 256u + (uint32_t)(x * D), p_tmem = tmem + 128u * (uint32_t)x;
            const uint32_t v_smem = sbase + C::kV + s * C::kTile;
            if (elect_one()) product_nn_half<D, 0>(o_tmem, p_tmem, 32, v_smem, !first);
            __syncwarp();
            if (!wait(bar.pfull(x, 1), np[x]++ & 1)) { ok = false; break; }
            ptx::tc_fence_after();
            const bool release = x == 1 || !has_b;
            if (elect_one()) {
              product_nn_half<D, 1>(o_tmem, p_tmem, 32, v_smem, true);
              if (last) ptx::mma_commit(bar.odone(x));
              if (release) ptx::mma_commit(bar.vempty(s));
            }
            __syncwarp();
            nv += release;
          }
          if (x == 0) nxt.next(a);            // behind a P V, which the pipe is still busy with
          if (nxt.valid && (x == 0 || nxt.has_b) && !scores(x)) { ok = false; break; }
        }
      }
      // Never free TMEM under a running product.
      int zero = 0;
      if (elect_one()) ptx::mma_commit(bar.drain());
      wait_phase(bar.drain(), 0, &zero, a.err);
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- output
    ptx::setmaxnreg_dec<kRegsOut>();
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int row_tok = (int)g.by_G.q((uint32_t)row), row_head = row - row_tok * g.G;
    uint8_t* stage = smem + C::kOut;
    uint32_t nl[2] = {0, 0}, no[2] = {0, 0};
    bool ok = true;
    Unit t;
    for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
      t.open(a, u);
      const bool any = t.t1 > t.t0;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int first = t.n0 + x * g.tpt;
        if (first >= g.N) continue;
        ok = warp_wait(bar.lfull(x), nl[x]++ & 1, abort, a.err) &&
             (!any || warp_wait(bar.odone(x), no[x]++ & 1, abort, a.err));
        if (threadIdx.x == 256) store_read();                 // the staging is free again
        __syncwarp();
        ok = bar_all(1, 128, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const float inv = s_inv[x * kCrossTile + row];
        const uint32_t o_tmem = tmem + 256u + (uint32_t)(x * D) + lane_base;
        const int tok = first + row_tok, head = t.hkv * g.G + row_head;
        const bool mine = row < g.G * g.tpt && tok < g.N;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          __syncwarp();                           // lanes without a row of their own stored nothing
          uint32_t o[32];
          if (any) {
            tmem_ld_x32(o_tmem + 32 * ch, o);
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (a.splits == 1) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              pk[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
            put_row32(stage, row, ch, pk);
          } else if (mine) {
            float4* dst = reinterpret_cast<float4*>(
                a.part_o + ((((long long)t.part * g.B + t.b) * g.N + tok) * g.H + head) * D + 32 * ch);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                                   __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar.oempty(x));
        __syncwarp();
        if (a.splits == 1) {
          fence_proxy_async();
          bar_sync(1, 128);
          if (threadIdx.x == 256) {
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb)
              tma_store_4d(&tmO, sbase + C::kOut + cb * (kCrossTile * 128), cb * 64, t.hkv * g.G, first, t.b);
            store_commit();
          }
        }
      }
    }
    if (threadIdx.x == 256) store_done();
  } else {
    // --------------------------------------------------------------- softmax
    ptx::setmaxnreg_inc<kRegsSoftmax>();
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + 128u * (uint32_t)x + lane_base;
    const uint32_t o_tmem = tmem + 256u + (uint32_t)(x * D) + lane_base;
    const int row_tok = (int)g.by_G.q((uint32_t)row), row_head = row - row_tok * g.G;
    const float c = a.scale_log2;
    uint32_t ns = 0, nu = 0;
    bool ok = true;
    Unit t;
    for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
      t.open(a, u);
      const int first = t.n0 + x * g.tpt;
      if (first >= g.N) continue;
      float m_run = -INFINITY, l = 0.f;
      for (int kt = t.t0; kt < t.t1; ++kt) {
        const uint4 w = tile_bits(a.keys, t.b, kt, g.nkt, t.len);
        if (!warp_wait(bar.sfull(x), ns++ & 1, abort, a.err)) { ok = false; break; }
        ptx::tc_fence_after();
        uint32_t r[128];
#pragma unroll
        for (int h = 0; h < 4; ++h) tmem_ld_x32(s_tmem + 32 * h, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * h]));
        ptx::tmem_wait_ld();
        if (!all_set(w)) {
          mask32(&r[0], w.x);
          mask32(&r[32], w.y);
          mask32(&r[64], w.z);
          mask32(&r[96], w.w);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 4; ++h) max32(&r[32 * h], mx);
        const float mb = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
        bool resc = false;
        if (m_run == -INFINITY) m_run = mb;            // nothing of this row is in O yet but zeros
        else resc = mb > m_run + kRescaleLog2;
        if (__any_sync(0xffffffffu, resc)) {
          // These scores follow the previous tile's P V in the pipe, so O holds exactly the
          // tiles before this one.
          const float alpha = resc ? ex2(m_run - mb) : 1.0f;
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            __syncwarp();
            uint32_t o[16];
            tmem_ld_x16(o_tmem + 16 * h, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st_x16(o_tmem + 16 * h, o);
          }
          l *= alpha;
          if (resc) m_run = mb;
        }
        const float m = m_run == -INFINITY ? 0.0f : m_run;
        uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        // P goes to the issuer in two halves: the first 64 keys multiply V while the others are
        // exponentiated
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          exp32(&r[64 * h], c, m, sum, s_tmem + 32 * h);
          exp32(&r[64 * h + 32], c, m, sum, s_tmem + 32 * h + 16);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar.pfull(x, h));
        }
        float s0, s1;
        uf2(fadd2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      // 1 / l for the output warps, once they have read the unit before; the lse from here
      if (nu > 0 && !warp_wait(bar.oempty(x), (nu - 1) & 1, abort, a.err)) break;
      ++nu;
      s_inv[x * kCrossTile + row] = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : NAN);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar.lfull(x));
      const int tok = first + row_tok, head = t.hkv * g.G + row_head;
      if (row < g.G * g.tpt && tok < g.N) {
        const float lse2 = l > 0.f ? (m_run == -INFINITY ? 0.0f : m_run) + __log2f(l) : (l == 0.f ? -INFINITY : NAN);
        const long long at = ((long long)t.b * g.H + head) * g.N + tok;
        if (a.splits > 1) a.part_lse[(long long)t.part * g.B * g.H * g.N + at] = lse2;
        else if (a.lse) a.lse[at] = lse2 * 0.69314718055994531f;
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 14) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of split keys: weights 2^(lse_p - lse) in fp32, in the order of the parts.
// One warp per (item, token, head).
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(CrossGeom g, int splits, const float* __restrict__ part_o,
                                                         const float* __restrict__ part_lse,
                                                         __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  const long long rows = (long long)g.B * g.N * g.H;
  const long long at = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= rows) return;
  const int head = (int)(at % g.H);
  const long long bn = at / g.H;
  const int tok = (int)(bn % g.N), b = (int)(bn / g.N);
  const long long at_lse = ((long long)b * g.H + head) * g.N + tok;
  float top = -INFINITY;
  bool nan = false;
  for (int p = 0; p < splits; ++p) {
    const float z = part_lse[p * rows + at_lse];
    nan |= isnan(z);
    top = fmaxf(top, z);
  }
  constexpr int V = D / 32;
  float o[V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  if (top > -INFINITY || nan)
    for (int p = 0; p < splits; ++p) {
      const float z = part_lse[p * rows + at_lse];
      if (z == -INFINITY) continue;                    // a part without a valid key holds zeros
      const float w = ex2(z - top);
      sum += w;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] += w * part_o[(p * rows + at) * D + lane * V + i];
    }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : NAN);
#pragma unroll
  for (int i = 0; i < V; ++i) out[at * D + lane * V + i] = __float2bfloat16_rn(o[i] * inv);
  if (lse && lane == 0)
    lse[at_lse] = sum > 0.f ? (top + __log2f(sum)) * 0.69314718055994531f : (sum == 0.f ? -INFINITY : NAN);
}

// Key mask (and kv_len) of one item per block: packed bits, last valid key + 1, valid keys.
__global__ void __launch_bounds__(256) pack_keys_kernel(int M, int nkt, const int* __restrict__ kv_len,
                                                        const uint8_t* __restrict__ key_mask, int2* __restrict__ plan,
                                                        uint32_t* __restrict__ bits) {
  __shared__ int s_last, s_count;
  if (threadIdx.x == 0) s_last = s_count = 0;
  __syncthreads();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int len = kv_len ? min(max(kv_len[b], 0), M) : M;
  const uint8_t* m = key_mask + (long long)b * M;
  int last = 0, count = 0;
  for (int w = threadIdx.x >> 5; w < 4 * nkt; w += blockDim.x >> 5) {
    const int j = 32 * w + lane;
    const uint32_t word = __ballot_sync(0xffffffffu, j < len && m[j] != 0);
    if (lane == 0) bits[(long long)b * 4 * nkt + w] = word;
    if (word) last = 32 * w + 32 - __clz(word);
    count += __popc(word);
  }
  if (lane == 0) {
    atomicMax(&s_last, last);
    atomicAdd(&s_count, count);
  }
  __syncthreads();
  if (threadIdx.x == 0) plan[b] = make_int2(s_last, s_count);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

template <int D>
cudaError_t run_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                    const FwdArgs& a, cudaStream_t s) {
  // set anew for every call: a device reset forgets it
  cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  static OncePerDevice once;
  e = once([] {
    // A register split above what the launch provides would wait forever in setmaxnreg.
    cudaFuncAttributes fa;
    const cudaError_t r = cudaFuncGetAttributes(&fa, cross_fwd_kernel<D>);
    if (r != cudaSuccess) return r;
    return fa.numRegs * kThreads < 128 * (2 * kRegsSoftmax + kRegsOut + kRegsControl) ? cudaErrorInvalidConfiguration
                                                                                    : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  cross_fwd_kernel<D><<<a.units < kCrossSms ? a.units : kCrossSms, kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, mo, a);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  const long long rows = (long long)a.g.B * a.g.N * a.g.H;
  cross_join_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a.g, a.splits, a.part_o, a.part_lse, a.out, a.lse);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

bool make_map_4d(CUtensorMap* m, const void* base, int d, int heads, int tokens, int items, const CrossStride& s,
                 int box_heads, int box_tokens) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  // The stride of an axis of one index is never used; any valid value serves. Items at stride 0
  // share one copy, which the kernels address as item 0.
  const cuuint64_t one = (cuuint64_t)d * 2;
  const bool shared = s.b == 0 && items > 1;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens, shared ? 1u : (cuuint64_t)items};
  cuuint64_t strides[3] = {heads > 1 ? (cuuint64_t)s.h * 2 : one, tokens > 1 ? (cuuint64_t)s.n * 2 : one,
                           dims[3] > 1 ? (cuuint64_t)s.b * 2 : one};
  cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_pack_keys(const CrossGeom& g, const int* kv_len, const uint8_t* key_mask, int2* plan,
                             uint32_t* bits, cudaStream_t s) {
  pack_keys_kernel<<<g.B, 256, 0, s>>>(g.M, g.nkt, kv_len, key_mask, plan, bits);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_cross_fwd(const CrossCall& c, void* out, float* lse, cudaStream_t s) {
  const CrossGeom& g = c.g;
  const CrossWs w = cross_ws(g);
  FwdArgs a;
  a.g = g;
  a.keys = {c.kv_len, nullptr, nullptr};
  if (c.key_mask) {
    int2* plan = reinterpret_cast<int2*>(c.ws + w.plan);
    uint32_t* bits = reinterpret_cast<uint32_t*>(c.ws + w.bits);
    const cudaError_t e = launch_pack_keys(g, c.kv_len, c.key_mask, plan, bits, s);
    if (e != cudaSuccess) return e;
    a.keys = {nullptr, plan, bits};
  }
  a.splits = cross_splits(g);
  a.nqb = ceil_div(g.nqt, 2);
  a.by_nqb = FastDiv((uint32_t)a.nqb);
  a.by_splits = FastDiv((uint32_t)a.splits);
  a.units = g.B * g.Hkv * a.splits * a.nqb;
  a.qb_mul = c.sq.b == 0 && g.B > 1 ? 0 : 1;
  a.kb_mul = c.sk.b == 0 && g.B > 1 ? 0 : 1;
  a.vb_mul = c.sv.b == 0 && g.B > 1 ? 0 : 1;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(c.ws + w.part);
  a.part_lse = a.part_o + (size_t)a.splits * g.B * g.N * g.H * g.d;
  a.err = reinterpret_cast<uint32_t*>(c.ws);
  a.scale_log2 = c.scale * 1.4426950408889634f;
  const CrossStride dense = {(long long)g.N * g.H * g.d, (long long)g.H * g.d, g.d};
  CUtensorMap mq, mk, mv, mo;
  if (!make_map_4d(&mq, c.q, g.d, g.H, g.N, g.B, c.sq, g.G, g.tpt) ||
      !make_map_4d(&mk, c.k, g.d, g.Hkv, g.M, g.B, c.sk, 1, kCrossTile) ||
      !make_map_4d(&mv, c.v, g.d, g.Hkv, g.M, g.B, c.sv, 1, kCrossTile) ||
      !make_map_4d(&mo, out, g.d, g.H, g.N, g.B, dense, g.G, g.tpt))
    return cudaErrorInvalidValue;
  return g.d == 128 ? run_fwd<128>(mq, mk, mv, mo, a, s) : run_fwd<64>(mq, mk, mv, mo, a, s);
}

}  // namespace bsa
