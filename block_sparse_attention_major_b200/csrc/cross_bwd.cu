// Gradients of the attention of the video tokens to an encoder's states (sm_100a: tcgen05 + TMEM
// + TMA), persistent.
//
//   p_ij = exp(scale q_i . k_j - lse_i),  t_ij = do_i . v_j,  D_i = sum_c do_ic out_ic
//   ds_ij = p_ij (t_ij - D_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// Three kernels. The row statistics (lse in units of log 2, D) are computed once (D again where one
// key tile holds a row). Then one kernel keeps 128 query rows and walks the keys (dq; in parts of
// them where the rows are few), and one keeps 128 keys and walks the query rows (dk, dv), each
// computing the scores and t again: seven products where one kernel would need
// five, but no sum crosses a CTA on the way, so there are no atomics, and repeated calls give
// identical bits. The rows of all query heads of a key head are one walk, so their sum is taken
// in the accumulators.
//
// The dk, dv kernel works on transposed tiles: S^T = K Q^T and T^T = V dO^T have a key a row, and
// P^T and dS^T, written back as bf16 pairs, are the left operands of dv += P^T dO, dk += dS^T Q.
// Its (item, key head, key tile) units, of one step a query tile, are cut into one equal range
// of steps a CTA; a CTA that holds a whole unit writes dk and dv, the parts of a cut unit go to
// the workspace in fp32 and a last kernel adds them in the order of the CTAs.
//
// In both kernels 8 warps do the elementwise part (a thread has half a row: 64 columns), one
// thread issues all products in the order in which their operands get ready, and the products of
// the next tile's scores and of the previous one's gradient run under the exponentials.
//
// Roundings to fewer bits: P and dS to bf16 ahead of their products, the gradients once.
//
// Measured, one B200, 32760 queries, 512 keys, 12 heads of 128: statistics 42 us (4.8 TB/s), dq 155 us
// (1.0 PFLOP/s of the 6 N M H d that it runs; profiled by itself 171 us, the tensor pipe 48 % busy, the
// rest is the chain from T through dS to the next T and the change of units), dk and dv 165 us (1.25
// PFLOP/s of 8 N M H d; by itself 176 us, 66 % busy; its products read 128 bytes a cycle from shared memory, all there is, and every copy of Q
// and dO takes some of it), the join 8 us. Over 4096 keys 1.13 to 1.25 and 1.3 PFLOP/s (two passes).
#include "cross.cuh"

#include <math.h>

namespace bsa {
namespace {

using namespace cross;

constexpr int kThreads = 384;

struct BwdArgs {
  CrossGeom g;
  KeySet keys;
  float2* stats;                    // [B, H, N]: (lse / log 2, D); +inf for a row without a key
  const int* prefix;                // key tiles of the items before b; null: every item has nkt
  int kb_mul, vb_mul, qb_mul;
  __nv_bfloat16 *dk, *dv;
  float* part;                      // cut units: [CTA][first / last][dk, dv][128][D]; before that, with split
                                    // keys, dq unscaled: [splits, B, H, N, D]
  int splits;                       // parts of the keys of a dq unit
  uint32_t* err;
  float scale, scale_log2;
  FastDiv by_nqt, by_splits;
};

__device__ __forceinline__ int key_tiles(const BwdArgs& a, int b) {
  return (item_keys(a.keys, b, a.g.M).x + kCrossTile - 1) / kCrossTile;
}

// Place of (lse, D) of row r of query tile qt of (b, hkv), or -1 for rows past the tokens or the tile's
// heads, which take lse = +inf: their probabilities are zero.
__device__ __forceinline__ long long stats_at(const BwdArgs& a, int b, int hkv, int qt, int r) {
  const CrossGeom& g = a.g;
  const int rt = (int)g.by_G.q((uint32_t)r), tok = qt * g.tpt + rt, head = hkv * g.G + r - rt * g.G;
  if (r >= g.G * g.tpt || tok >= g.N) return -1;
  return ((long long)b * g.H + head) * g.N + tok;
}
__device__ __forceinline__ float2 row_stats(const BwdArgs& a, int b, int hkv, int qt, int r) {
  const long long i = stats_at(a, b, hkv, qt, r);
  return i < 0 ? make_float2(INFINITY, 0.f) : a.stats[i];
}

// -------------------------------------------------------------------------------- dq
template <int D>
struct CfgQ {
  static constexpr int kTile = kCrossTile * D * 2;
  // a key tile is held from its scores to its dq product, a value tile for one product only
  static constexpr int kKS = 3, kVS = D == 128 ? 1 : 2;
  static constexpr int kQ = 0, kDo = kTile, kK = 2 * kTile, kV = kK + kKS * kTile;
  static constexpr int kOut = kV + kVS * kTile;             // staging of a finished block
  static constexpr int kSum = kOut + kTile;                 // [2][128] sums of half rows
  static constexpr int kBar = kSum + 2 * kCrossTile * 4;
  // kfull, kempty, kland [kKS]; vfull, vempty [kVS]; sfull [2]; qfull, qempty, dofull, doempty, tfull, dsfull,
  // done, drain
  static constexpr int kBars = 3 * kKS + 2 * kVS + 2 + 8;
  static constexpr int kMisc = kBar + 8 * kBars;
  static constexpr int kSmem = 1024 + kMisc + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

// kSplit: the keys of a unit in parts (few query rows); kept out of the other form, which it slowed
// by 5 %.
template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmDq, const BwdArgs a, int units) {
  using C = CfgQ<D>;
  constexpr int KS = C::kKS, VS = C::kVS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = ptx::smem_u32(smem);
  const CrossGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b0 = sbase + C::kBar;
  auto kfull = [&](int s) { return b0 + 8 * s; };
  auto kempty = [&](int s) { return b0 + 8 * (KS + s); };
  auto kland = [&](int s) { return b0 + 8 * (2 * KS + s); };
  auto vfull = [&](int s) { return b0 + 8 * (3 * KS + s); };
  auto vempty = [&](int s) { return b0 + 8 * (3 * KS + VS + s); };
  auto sfull = [&](int s) { return b0 + 8 * (3 * KS + 2 * VS + s); };
  const uint32_t b1 = b0 + 8 * (3 * KS + 2 * VS + 2);
  const uint32_t qfull = b1, qempty = b1 + 8, dofull = b1 + 16, doempty = b1 + 24, tfull = b1 + 32, dsfull = b1 + 40,
                 done = b1 + 48, drain = b1 + 56;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) ptx::mbar_init(b0 + 8 * i, b0 + 8 * i == dsfull ? 8 : 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;                 // S buffers at 0 and 128, T at 256, dq at 384

  auto wait = [&](uint32_t b, uint32_t ph) { return wait_phase(b, ph, abort, a.err); };
  // unit -> (query tile, part of the keys, key head, item); query tiles fastest, so that neighbours
  // share keys
  auto decode = [&](int u, int& qt, int& hkv, int& b, int& part) {
    const int rest = (int)a.by_nqt.q((uint32_t)u);
    qt = u - rest * g.nqt;
    const int bh = kSplit ? (int)a.by_splits.q((uint32_t)rest) : rest;
    part = kSplit ? rest - bh * a.splits : 0;
    b = (int)g.by_hkv.q((uint32_t)bh);
    hkv = bh - b * g.Hkv;
  };
  // key tiles of a part: [t0, t1)
  auto tiles_of = [&](int nt, int part, int& t0, int& t1) {
    t0 = 0;
    t1 = nt;
    if (kSplit) {
      t0 = (int)((long long)nt * part / a.splits);
      t1 = (int)((long long)nt * (part + 1) / a.splits);
    }
  };

  if (warp == 8) {
    // ------------------------------------------------------------- Q, dO and the V ring
    if (lane == 0) {
      uint32_t nq = 0, nv = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)(g.G * g.tpt * D * 2);
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        int qt, hkv, b, part, t0, t1;
        decode(u, qt, hkv, b, part);
        tiles_of(key_tiles(a, b), part, t0, t1);
        if (u + (int)gridDim.x < units) {           // the next unit's rows come from HBM meanwhile
          int qf, hf, bf, pf;
          decode(u + (int)gridDim.x, qf, hf, bf, pf);
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb) {
            tma_prefetch_4d(&tmQ, cb * 64, hf * g.G, qf * g.tpt, bf * a.qb_mul);
            tma_prefetch_4d(&tmDo, cb * 64, hf * g.G, qf * g.tpt, bf);
          }
        }
        if (t0 == t1) continue;
        if (nq > 0 && !wait(qempty, (nq - 1) & 1)) break;
        ptx::mbar_arrive_expect_tx(qfull, bytes);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
          tma_load_4d(sbase + C::kQ + cb * 16384, &tmQ, qfull, cb * 64, hkv * g.G, qt * g.tpt, b * a.qb_mul);
        if (nq > 0 && !wait(doempty, (nq - 1) & 1)) {
          ++nq;
          ptx::mbar_arrive_expect_tx(dofull, 0);   // keeps the drain below in step
          break;
        }
        ptx::mbar_arrive_expect_tx(dofull, bytes);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
          tma_load_4d(sbase + C::kDo + cb * 16384, &tmDo, dofull, cb * 64, hkv * g.G, qt * g.tpt, b);
        ++nq;
        for (int i = t0; i < t1; ++i) {
          const int s = (int)(nv % VS);
          if (!wait(vempty(s), ((nv / VS) & 1) ^ 1)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(vfull(s), C::kTile);
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(sbase + C::kV + s * C::kTile + cb * 16384, &tmV, vfull(s), cb * 64, hkv, i * kCrossTile,
                        b * a.vb_mul);
          ++nv;
        }
      }
      int zero = 0;                                 // never leave with copies in flight
      for (uint32_t s = 0; s < VS; ++s)
        if (nv > s) wait_phase(vfull((int)s), ((nv - 1 - s) / VS) & 1, &zero, a.err);
      if (nq > 0) {
        wait_phase(qfull, (nq - 1) & 1, &zero, a.err);
        wait_phase(dofull, (nq - 1) & 1, &zero, a.err);
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------- the K ring
    // K is the right operand of dq += dS K, a sum over the keys: rows of masked keys, whose dS
    // is zero, are zeroed, so that what they hold does not matter.
    uint32_t nk = 0, land[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) land[s] = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      int qt, hkv, b, part, t0, t1;
      decode(u, qt, hkv, b, part);
      const int len = item_keys(a.keys, b, g.M).x;
      tiles_of((len + kCrossTile - 1) / kCrossTile, part, t0, t1);
      for (int i = t0; i < t1; ++i) {
        const int s = (int)(nk % KS);
        if (!warp_wait(kempty(s), ((nk / KS) & 1) ^ 1, abort, a.err)) { ok = false; break; }
        const uint4 w = tile_bits(a.keys, b, i, g.nkt, len);
        const bool scrub = (a.keys.bits || a.keys.kv_len) && !all_set(w);
        const uint32_t full = scrub ? kland(s) : kfull(s);
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(full, C::kTile);
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(sbase + C::kK + s * C::kTile + cb * 16384, &tmK, full, cb * 64, hkv, i * kCrossTile, b * a.kb_mul);
        }
        __syncwarp();
        if (scrub) {
          uint32_t ph = 0;
#pragma unroll
          for (int j = 0; j < KS; ++j)
            if (j == s) ph = land[j]++ & 1;
          int zero = 0;
          const bool in = __all_sync(0xffffffffu, wait_phase(kland(s), ph, &zero, a.err));
          if (!in) { *abort = 1; ok = false; break; }
          zero_masked_rows<D>(smem + C::kK + s * C::kTile, w, lane);
          if (lane == 0) ptx::mbar_arrive(kfull(s));
        }
        ++nk;
      }
    }
    int zero = 0;
    for (uint32_t s = 0; s < KS; ++s)
      if (nk > s) wait_phase(kfull((int)s), ((nk - 1 - s) / KS) & 1, &zero, a.err);
  } else if (warp == 9) {
    // ------------------------------------------------------------- MMA issuer
    // S(0), T(0), S(1); then, once a tile's dS is written: T of the next tile (this tile's was read
    // for dS), dq += dS K, and S of the tile after (over this tile's dS). The next dS needs the
    // first of the three only, so the others run under it. The warp runs whole; one lane issues.
    uint32_t ns = 0, nk = 0, nv = 0, nds = 0, nq = 0;
    bool ok = true;
    auto all_wait = [&](uint32_t b, uint32_t ph) { return warp_wait(b, ph, abort, a.err); };
    auto scores = [&](bool last) {
      const int s = (int)(ns % KS);
      if (!all_wait(kfull(s), (ns / KS) & 1)) return false;
      ptx::tc_fence_after();
      if (elect_one()) {
        product_nt<D>(tmem + 128u * (ns & 1), sbase + C::kQ, sbase + C::kK + s * C::kTile);
        ptx::mma_commit(sfull((int)(ns & 1)));
        if (last) ptx::mma_commit(qempty);
      }
      __syncwarp();
      ++ns;
      return true;
    };
    auto tee = [&](bool last) {
      const int s = (int)(nv % VS);
      if (!all_wait(vfull(s), (nv / VS) & 1)) return false;
      ptx::tc_fence_after();
      if (elect_one()) {
        product_nt<D>(tmem + 256u, sbase + C::kDo, sbase + C::kV + s * C::kTile);
        ptx::mma_commit(tfull);
        ptx::mma_commit(vempty(s));
        if (last) ptx::mma_commit(doempty);
      }
      __syncwarp();
      ++nv;
      return true;
    };
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      int qt, hkv, b, part, t0, t1;
      decode(u, qt, hkv, b, part);
      tiles_of(key_tiles(a, b), part, t0, t1);
      const int nt = t1 - t0;
      if (nt == 0) continue;
      if (!all_wait(qfull, nq & 1) || !scores(nt == 1)) break;
      if (!all_wait(dofull, nq & 1) || !tee(nt == 1)) break;
      if (nt > 1 && !scores(nt == 2)) break;
      ++nq;
      for (int i = 0; i < nt; ++i) {
        if (!all_wait(dsfull, nds++ & 1)) { ok = false; break; }
        ptx::tc_fence_after();
        if (i + 1 < nt && !tee(i + 2 == nt)) { ok = false; break; }
        const int s = (int)(nk % KS);
        if (elect_one()) {
          product_nn<D>(tmem + 384u, tmem + 128u * (nk & 1), 64, sbase + C::kK + s * C::kTile, i > 0);
          ptx::mma_commit(kempty(s));
          if (i == nt - 1) ptx::mma_commit(done);
        }
        __syncwarp();
        ++nk;
        if (i + 2 < nt && !scores(i + 3 == nt)) { ok = false; break; }
      }
    }
    int zero = 0;                                   // never free TMEM under a running product
    if (elect_one()) ptx::mma_commit(drain);
    wait_phase(drain, 0, &zero, a.err);
  } else if (warp < 8) {
    // ------------------------------------------------------------- dS and the epilogue
    // A finished unit is written out between the probabilities and the dS of the next unit's
    // first tile: its last product and the store run under them, and the accumulator is read
    // before the dS that lets the next unit overwrite it.
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c = a.scale_log2;
    uint32_t n = 0, nd = 0;
    bool ok = true;
    int held = -1;                                  // the unit whose gradient is still in the accumulator
    // A warp whose wait ran out says so at the next barrier of the eight warps before it leaves: others
    // may have seen the same phase complete, and they would wait there for good. There always is
    // one (a unit whose tiles are worked on is finished later), and no wait stands between the two
    // barriers of finish().
    auto give_up = [&] {
      bar_all(1, 256, false);
      return false;
    };
    // Waits for the last product of unit `from` (none if it has no key) and stores its block.
    auto finish = [&](int from, bool any) {
      bool in = !any || warp_wait(done, nd & 1, abort, a.err);
      nd += any;
      if (threadIdx.x == 0) store_read();           // the staging is free again
      __syncwarp();
      in = bar_all(1, 256, in);
      if (!in) return false;
      ptx::tc_fence_after();
      int qt = 0, hkv = 0, b = 0, part = 0;
      if (kSplit || threadIdx.x == 0) decode(from, qt, hkv, b, part);
      const long long at = kSplit ? stats_at(a, b, hkv, qt, row) : 0;          // (b, head, token)
      const uint32_t o_tmem = tmem + 384u + (uint32_t)(half * (D / 2)) + lane_base;
#pragma unroll 1
      for (int ch = 0; ch < D / 64; ++ch) {
        __syncwarp();                               // lanes without a row of their own stored nothing
        uint32_t o[32], pk[16];
        if (any) {
          tmem_ld_x32(o_tmem + 32 * ch, o);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (kSplit) {
          // [part][B, H, N][D]: the join turns them into rows of tokens
          if (at >= 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.part + (((long long)part * g.B * g.H * g.N + at) * D +
                                                            half * (D / 2) + 32 * ch));
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          continue;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          pk[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * a.scale, __uint_as_float(o[2 * k + 1]) * a.scale);
        put_row32(smem + C::kOut, row, half * (D / 64) + ch, pk);
      }
      if (kSplit) return true;
      fence_proxy_async();
      bar_sync(1, 256);
      if (threadIdx.x == 0) {
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
          tma_store_4d(&tmDq, sbase + C::kOut + cb * 16384, cb * 64, hkv * g.G, qt * g.tpt, b);
        store_commit();
      }
      return true;
    };
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      int qt, hkv, b, part, t0, t1;
      decode(u, qt, hkv, b, part);
      const int2 ik = item_keys(a.keys, b, g.M);
      const int nt = (ik.x + kCrossTile - 1) / kCrossTile;
      tiles_of(nt, part, t0, t1);
      if (t0 == t1) {
        if (held >= 0 && !finish(held, true)) break;
        held = -1;
        if (!finish(u, false)) break;
        continue;
      }
      const float2 st = row_stats(a, b, hkv, qt, row);
      const uint64_t cc = f2(c, c), mm = f2(-st.x, -st.x);
      uint64_t dd = f2(-st.y, -st.y);
      for (int i = t0; i < t1; ++i, ++n) {
        const uint4 w4 = tile_bits(a.keys, b, i, g.nkt, ik.x);
        const bool full = all_set(w4);
        const uint32_t w[2] = {half ? w4.z : w4.x, half ? w4.w : w4.y};
        const uint32_t s_tmem = tmem + 128u * (n & 1) + 64u * (uint32_t)half + lane_base;
        const uint32_t t_tmem = tmem + 256u + 64u * (uint32_t)half + lane_base;
        if (!warp_wait(sfull((int)(n & 1)), (n >> 1) & 1, abort, a.err)) { ok = give_up(); break; }
        ptx::tc_fence_after();
        uint32_t p[64];
        tmem_ld_x32(s_tmem, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
        tmem_ld_x32(s_tmem + 32, *reinterpret_cast<uint32_t(*)[32]>(&p[32]));
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x0, x1;
          uf2(ffma2(f2(__uint_as_float(p[2 * k]), __uint_as_float(p[2 * k + 1])), cc, mm), x0, x1);
          p[2 * k] = __float_as_uint(ex2(x0));
          p[2 * k + 1] = __float_as_uint(ex2(x1));
        }
        if (held >= 0) {
          ok = finish(held, true);
          held = -1;
          if (!ok) break;
        }
        ok = warp_wait(tfull, n & 1, abort, a.err);
        if (nt == 1) {
          // The whole row is here: D = sum_j p t, instead of the sum over the rounded output, whose
          // error is the larger against dS the fewer keys share a row. The two halves of a row
          // meet in shared memory; the dk, dv kernel reads the same D.
          float* s_sum = reinterpret_cast<float*>(smem + C::kSum);
          if (ok) {
            ptx::tc_fence_after();
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t t[32];
              tmem_ld_x32(t_tmem + 32 * h, t);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k)
                sum += ((w[h] >> k) & 1u) ? __uint_as_float(t[k]) * __uint_as_float(p[32 * h + k]) : 0.f;
            }
            s_sum[half * kCrossTile + row] = sum;
          }
          ok = bar_all(1, 256, ok);
          if (ok) {
            const float sum = s_sum[row] + s_sum[kCrossTile + row];
            dd = f2(-sum, -sum);
            const long long at = stats_at(a, b, hkv, qt, row);
            if (half == 0 && at >= 0) a.stats[at].y = sum;
            __syncwarp();
          }
        } else if (!ok) {
          give_up();
        }
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t t[32], pk[16];
          tmem_ld_x32(t_tmem + 32 * h, t);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float d0, d1;
            uf2(fmul2(fadd2(f2(__uint_as_float(t[2 * k]), __uint_as_float(t[2 * k + 1])), dd),
                      f2(__uint_as_float(p[32 * h + 2 * k]), __uint_as_float(p[32 * h + 2 * k + 1]))),
                d0, d1);
            if (!full) {
              d0 = ((w[h] >> (2 * k)) & 1u) ? d0 : 0.f;
              d1 = ((w[h] >> (2 * k + 1)) & 1u) ? d1 : 0.f;
            }
            pk[k] = pack_bf16x2(d0, d1);
          }
          // one valid key: its weight is 1 whatever the scores, and nothing has a gradient
          if (ik.y == 1)
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[k] = 0u;
          tmem_st_x16(s_tmem + 16 * h, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(dsfull);
      }
      if (!ok) break;
      held = u;
    }
    if (ok && held >= 0) finish(held, true);
    if (threadIdx.x == 0) store_done();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ dk, dv
template <int D>
struct CfgK {
  static constexpr int kTile = kCrossTile * D * 2;
  static constexpr int kS = 2;                              // stages of Q and of dO
  static constexpr int kK = 0, kV = kTile, kQ = 2 * kTile, kDo = kQ + kS * kTile;
  static constexpr int kStats = kDo + kS * kTile;           // [stage][128] lse, then [stage][128] D
  static constexpr int kBar = kStats + 2 * kS * kCrossTile * 4;
  // qfull, qempty, dofull, doempty, stfull, stempty [kS]; kvfull, kvempty, sfull, tfull, pfull, dsfull, done, drain
  static constexpr int kBars = 6 * kS + 8;
  static constexpr int kMisc = kBar + 8 * kBars;
  static constexpr int kSmem = 1024 + kMisc + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

// Steps of the dk, dv kernel: unit u = (item, key head, key tile) has nqt of them, unit after
// unit; CTA c does [total c / grid, total (c + 1) / grid).
struct Steps {
  long long total, lo, hi;
  __device__ __forceinline__ Steps(const BwdArgs& a, int cta, int grid) {
    const long long tiles = a.prefix ? a.prefix[a.g.B] : (long long)a.g.B * a.g.nkt;
    total = tiles * a.g.Hkv * a.g.nqt;
    lo = total * cta / grid;
    hi = total * (cta + 1) / grid;
  }
};
__device__ __forceinline__ void unit_of(const BwdArgs& a, long long u, int& b, int& hkv, int& kt) {
  const CrossGeom& g = a.g;
  if (!a.prefix) {
    kt = (int)(u % g.nkt);
    const long long bh = u / g.nkt;
    hkv = (int)(bh % g.Hkv);
    b = (int)(bh / g.Hkv);
    return;
  }
  int lo = 0, hi = g.B - 1;                         // the last item that starts at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)a.prefix[mid] * g.Hkv <= u) lo = mid;
    else hi = mid - 1;
  }
  b = lo;
  const int nt = a.prefix[b + 1] - a.prefix[b];
  const long long rest = u - (long long)a.prefix[b] * g.Hkv;
  hkv = (int)(rest / nt);
  kt = (int)(rest % nt);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const BwdArgs a) {
  using C = CfgK<D>;
  constexpr int S = C::kS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = ptx::smem_u32(smem);
  const CrossGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b0 = sbase + C::kBar;
  auto qfull = [&](int s) { return b0 + 8 * s; };
  auto qempty = [&](int s) { return b0 + 8 * (S + s); };
  auto dofull = [&](int s) { return b0 + 8 * (2 * S + s); };
  auto doempty = [&](int s) { return b0 + 8 * (3 * S + s); };
  auto stfull = [&](int s) { return b0 + 8 * (4 * S + s); };
  auto stempty = [&](int s) { return b0 + 8 * (5 * S + s); };
  const uint32_t b1 = b0 + 8 * (6 * S);
  const uint32_t kvfull = b1, kvempty = b1 + 8, sfull = b1 + 16, tfull = b1 + 24, pfull = b1 + 32, dsfull = b1 + 40,
                 done = b1 + 48, drain = b1 + 56;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  float* s_lse = reinterpret_cast<float*>(smem + C::kStats);
  float* s_del = s_lse + S * kCrossTile;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      const uint32_t b = b0 + 8 * i;
      const bool eight = b == pfull || b == dsfull || (i >= 5 * S && i < 6 * S);
      ptx::mbar_init(b, eight ? 8 : (i >= 4 * S && i < 5 * S) ? 32 : 1);
    }
    *abort = 0;
    ptx::fence_mbar_init();
  }
  // Rows that no copy fills (128 is not a multiple of the heads) enter sums over the rows: zero.
  if (g.G * g.tpt < kCrossTile) {
    for (int i = threadIdx.x; i < 2 * S * C::kTile / 16; i += kThreads)
      *reinterpret_cast<uint4*>(smem + C::kQ + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;                 // S^T at 0, T^T at 128, dv at 256, dk at 256 + D

  const Steps st(a, blockIdx.x, gridDim.x);
  auto wait = [&](uint32_t b, uint32_t ph) { return wait_phase(b, ph, abort, a.err); };
  // Segments of this CTA's range: unit u, query tiles [t0, t1).
  auto segment = [&](long long at, long long& u, int& t0, int& t1) {
    u = at / g.nqt;
    t0 = (int)(at - u * g.nqt);
    const long long left = st.hi - at;
    t1 = (int)(left < g.nqt - t0 ? t0 + left : g.nqt);
  };

  if (warp == 8) {
    // ------------------------------------------------------------- K, V, and the Q and dO rings
    if (lane == 0) {
      uint32_t nseg = 0, nq = 0, nd = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)(g.G * g.tpt * D * 2);
      for (long long at = st.lo; at < st.hi && ok;) {
        long long u;
        int t0, t1, b, hkv, kt;
        segment(at, u, t0, t1);
        unit_of(a, u, b, hkv, kt);
        if (nseg > 0 && !wait(kvempty, (nseg - 1) & 1)) break;
        ptx::mbar_arrive_expect_tx(kvfull, 2 * C::kTile);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb) {
          tma_load_4d(sbase + C::kK + cb * 16384, &tmK, kvfull, cb * 64, hkv, kt * kCrossTile, b * a.kb_mul);
          tma_load_4d(sbase + C::kV + cb * 16384, &tmV, kvfull, cb * 64, hkv, kt * kCrossTile, b * a.vb_mul);
        }
        ++nseg;
        for (int t = t0; t < t1; ++t) {
          const int s = (int)(nq % S);
          if (!wait(qempty(s), ((nq / S) & 1) ^ 1)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(qfull(s), bytes);
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(sbase + C::kQ + s * C::kTile + cb * 16384, &tmQ, qfull(s), cb * 64, hkv * g.G, t * g.tpt,
                        b * a.qb_mul);
          ++nq;
          if (!wait(doempty(s), ((nd / S) & 1) ^ 1)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(dofull(s), bytes);
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(sbase + C::kDo + s * C::kTile + cb * 16384, &tmDo, dofull(s), cb * 64, hkv * g.G, t * g.tpt, b);
          ++nd;
        }
        at += t1 - t0;
      }
      int zero = 0;                                 // never leave with copies in flight
      for (uint32_t s = 0; s < S; ++s) {
        if (nq > s) wait_phase(qfull((int)s), ((nq - 1 - s) / S) & 1, &zero, a.err);
        if (nd > s) wait_phase(dofull((int)s), ((nd - 1 - s) / S) & 1, &zero, a.err);
      }
      if (nseg > 0) wait_phase(kvfull, (nseg - 1) & 1, &zero, a.err);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------- row statistics
    uint32_t n = 0;
    bool ok = true;
    for (long long at = st.lo; at < st.hi && ok;) {
      long long u;
      int t0, t1, b, hkv, kt;
      segment(at, u, t0, t1);
      unit_of(a, u, b, hkv, kt);
      for (int t = t0; t < t1; ++t, ++n) {
        const int s = (int)(n % S);
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = row_stats(a, b, hkv, t, 32 * i + lane);
        if (!warp_wait(stempty(s), ((n / S) & 1) ^ 1, abort, a.err)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s_lse[s * kCrossTile + 32 * i + lane] = -v[i].x;
          s_del[s * kCrossTile + 32 * i + lane] = -v[i].y;
        }
        ptx::mbar_arrive(stfull(s));
      }
      at += t1 - t0;
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------- MMA issuer
    // S(0), T(0); then for each query tile: dv += P dO, S of the next tile (over P, which that
    // product has read), dk += dS Q, T of the next tile (over dS). The warp runs whole; one lane
    // issues.
    uint32_t nseg = 0, ns = 0, nt = 0, n = 0;
    bool ok = true;
    auto all_wait = [&](uint32_t b, uint32_t ph) { return warp_wait(b, ph, abort, a.err); };
    auto scores = [&]() {
      const int s = (int)(ns % S);
      if (!all_wait(qfull(s), (ns / S) & 1)) return false;
      ptx::tc_fence_after();
      if (elect_one()) {
        product_nt<D>(tmem, sbase + C::kK, sbase + C::kQ + s * C::kTile);
        ptx::mma_commit(sfull);
      }
      __syncwarp();
      ++ns;
      return true;
    };
    auto tee = [&]() {
      const int s = (int)(nt % S);
      if (!all_wait(dofull(s), (nt / S) & 1)) return false;
      ptx::tc_fence_after();
      if (elect_one()) {
        product_nt<D>(tmem + 128u, sbase + C::kV, sbase + C::kDo + s * C::kTile);
        ptx::mma_commit(tfull);
      }
      __syncwarp();
      ++nt;
      return true;
    };
    for (long long at = st.lo; at < st.hi && ok;) {
      long long u;
      int t0, t1;
      segment(at, u, t0, t1);
      if (!all_wait(kvfull, nseg++ & 1) || !scores() || !tee()) break;
      for (int t = t0; t < t1; ++t, ++n) {
        const int s = (int)(n % S);
        const bool more = t + 1 < t1;
        if (!all_wait(pfull, n & 1)) { ok = false; break; }
        ptx::tc_fence_after();
        if (elect_one()) {
          product_nn<D>(tmem + 256u, tmem, 64, sbase + C::kDo + s * C::kTile, t > t0);
          ptx::mma_commit(doempty(s));
        }
        __syncwarp();
        if (more && !scores()) { ok = false; break; }
        if (!all_wait(dsfull, n & 1)) { ok = false; break; }
        ptx::tc_fence_after();
        if (elect_one()) {
          product_nn<D>(tmem + 256u + (uint32_t)D, tmem + 128u, 64, sbase + C::kQ + s * C::kTile, t > t0);
          ptx::mma_commit(qempty(s));
          if (!more) {
            ptx::mma_commit(kvempty);
            ptx::mma_commit(done);
          }
        }
        __syncwarp();
        if (more && !tee()) { ok = false; break; }
      }
      at += t1 - t0;
    }
    int zero = 0;                                   // never free TMEM under a running product
    if (elect_one()) ptx::mma_commit(drain);
    wait_phase(drain, 0, &zero, a.err);
  } else if (warp < 8) {
    // ------------------------------------------------------------- P, dS and the epilogue
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + 64u * (uint32_t)half + lane_base, t_tmem = s_tmem + 128u;
    const uint64_t cc = f2(a.scale_log2, a.scale_log2);
    uint32_t n = 0, nseg = 0;
    bool ok = true;
    for (long long at = st.lo; at < st.hi && ok;) {
      long long u;
      int t0, t1, b, hkv, kt;
      segment(at, u, t0, t1);
      unit_of(a, u, b, hkv, kt);
      const int2 ik = item_keys(a.keys, b, g.M);
      for (int t = t0; t < t1; ++t, ++n) {
        const int s = (int)(n % S);
        const float* lse = s_lse + s * kCrossTile + 64 * half;
        const float* del = s_del + s * kCrossTile + 64 * half;
        if (!warp_wait(stfull(s), (n / S) & 1, abort, a.err)) { ok = false; break; }
        if (!warp_wait(sfull, n & 1, abort, a.err)) { ok = false; break; }
        ptx::tc_fence_after();
        uint32_t p[64];
        tmem_ld_x32(s_tmem, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
        tmem_ld_x32(s_tmem + 32, *reinterpret_cast<uint32_t(*)[32]>(&p[32]));
        ptx::tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 l = *reinterpret_cast<const float4*>(lse + 32 * h + 4 * k);
            uint32_t* q = &p[32 * h + 4 * k];
            float x0, x1, x2, x3;
            uf2(ffma2(f2(__uint_as_float(q[0]), __uint_as_float(q[1])), cc, f2(l.x, l.y)), x0, x1);
            uf2(ffma2(f2(__uint_as_float(q[2]), __uint_as_float(q[3])), cc, f2(l.z, l.w)), x2, x3);
            x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
            pk[2 * k] = pack_bf16x2(x0, x1);
            pk[2 * k + 1] = pack_bf16x2(x2, x3);
            q[0] = __float_as_uint(x0), q[1] = __float_as_uint(x1);
            q[2] = __float_as_uint(x2), q[3] = __float_as_uint(x3);
          }
          tmem_st_x16(s_tmem + 16 * h, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(pfull);
        if (!warp_wait(tfull, n & 1, abort, a.err)) { ok = false; break; }
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t tt[32], pk[16];
          tmem_ld_x32(t_tmem + 32 * h, tt);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 d = *reinterpret_cast<const float4*>(del + 32 * h + 4 * k);
            const uint32_t* q = &p[32 * h + 4 * k];
            float d0, d1, d2, d3;
            uf2(fmul2(fadd2(f2(__uint_as_float(tt[4 * k]), __uint_as_float(tt[4 * k + 1])), f2(d.x, d.y)),
                      f2(__uint_as_float(q[0]), __uint_as_float(q[1]))), d0, d1);
            uf2(fmul2(fadd2(f2(__uint_as_float(tt[4 * k + 2]), __uint_as_float(tt[4 * k + 3])), f2(d.z, d.w)),
                      f2(__uint_as_float(q[2]), __uint_as_float(q[3]))), d2, d3);
            pk[2 * k] = pack_bf16x2(d0, d1);
            pk[2 * k + 1] = pack_bf16x2(d2, d3);
          }
          // one valid key: its weight is 1 whatever the scores, and nothing has a gradient
          if (ik.y == 1)
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[k] = 0u;
          tmem_st_x16(t_tmem + 16 * h, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(dsfull);
          ptx::mbar_arrive(stempty(s));
        }
      }
      if (!ok) break;
      if (!warp_wait(done, nseg++ & 1, abort, a.err)) break;
      ptx::tc_fence_after();
      // dv of this key by the lower four warps, dk by the upper four
      const uint4 w4 = tile_bits(a.keys, b, kt, g.nkt, ik.x);
      const int wi = row >> 5;
      const uint32_t word = wi == 0 ? w4.x : wi == 1 ? w4.y : wi == 2 ? w4.z : w4.w;
      const bool valid = (word >> (row & 31)) & 1u;
      const int key = kt * kCrossTile + row;
      const bool whole = t0 == 0 && t1 == g.nqt;
      const float sc = half ? a.scale : 1.0f;
      const uint32_t o_tmem = tmem + 256u + (uint32_t)(half * D) + lane_base;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        __syncwarp();                               // keys past M were not stored
        uint32_t o[32];
        tmem_ld_x32(o_tmem + 32 * ch, o);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = valid ? __float_as_uint(__uint_as_float(o[k]) * sc) : 0u;
        if (whole) {
          if (key < g.M) {
            uint4* dst = reinterpret_cast<uint4*>((half ? a.dk : a.dv) + (((long long)b * g.M + key) * g.Hkv + hkv) * D + 32 * ch);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 v;
              v.x = pack_bf16x2(__uint_as_float(o[8 * k + 0]), __uint_as_float(o[8 * k + 1]));
              v.y = pack_bf16x2(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3]));
              v.z = pack_bf16x2(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5]));
              v.w = pack_bf16x2(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7]));
              dst[k] = v;
            }
          }
        } else {
          // a cut unit is the first or the last of this CTA's range
          const int slot = 2 * blockIdx.x + (at == st.lo ? 0 : 1);
          float4* dst = reinterpret_cast<float4*>(a.part + (((long long)slot * 2 + half) * kCrossTile + row) * D + 32 * ch);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]), __uint_as_float(o[4 * k + 2]),
                                 __uint_as_float(o[4 * k + 3]));
        }
      }
      at += t1 - t0;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The rest of dk and dv: sums of the parts of cut units, zeros for key tiles past an item's
// last valid key. Grid: eighths of a key tile (16 keys), key tile, key head and item; a thread
// has four neighbouring elements of dk and of dv.
template <int D>
__global__ void __launch_bounds__(16 * D / 4) cross_dkv_join_kernel(BwdArgs a, int grid) {
  const CrossGeom& g = a.g;
  const int kt = blockIdx.y, hkv = blockIdx.z % g.Hkv, b = blockIdx.z / g.Hkv;
  const int nt = key_tiles(a, b);
  const int r = blockIdx.x * 16 + threadIdx.x / (D / 4), c4 = threadIdx.x % (D / 4), key = kt * kCrossTile + r;
  int c0 = 0, c1 = -1;
  long long first = 0, total = 0;
  if (kt < nt) {
    const long long tiles = a.prefix ? a.prefix[g.B] : (long long)g.B * g.nkt;
    total = tiles * g.Hkv * g.nqt;
    const long long u = (a.prefix ? (long long)a.prefix[b] : (long long)b * g.nkt) * g.Hkv + (long long)hkv * nt + kt;
    first = u * g.nqt;
    const long long last = first + g.nqt - 1;
    c0 = (int)(first * grid / total);
    c1 = (int)(last * grid / total);
    while (c0 > 0 && total * c0 / grid > first) --c0;
    while (total * (c0 + 1) / grid <= first) ++c0;
    while (c1 > 0 && total * c1 / grid > last) --c1;
    while (total * (c1 + 1) / grid <= last) ++c1;
    if (c0 == c1) return;                           // written by its CTA
  }
  if (key >= g.M) return;
  float4 sv = make_float4(0.f, 0.f, 0.f, 0.f), sk = sv;
  for (int c = c0; c <= c1; ++c) {
    const long long lo = total * c / grid;
    if (lo == total * (c + 1) / grid) continue;     // fewer steps than CTAs: this one had none
    // the unit is the CTA's first if the CTA starts inside it or at its start
    const int slot = 2 * c + (lo >= first ? 0 : 1);
    const float4* p = reinterpret_cast<const float4*>(a.part) + ((long long)slot * 2 * kCrossTile + r) * (D / 4) + c4;
    const float4 pv = p[0], pk = p[kCrossTile * (D / 4)];
    sv.x += pv.x, sv.y += pv.y, sv.z += pv.z, sv.w += pv.w;
    sk.x += pk.x, sk.y += pk.y, sk.z += pk.z, sk.w += pk.w;
  }
  const long long at = (((long long)b * g.M + key) * g.Hkv + hkv) * D + 4 * c4;
  *reinterpret_cast<uint2*>(a.dv + at) = make_uint2(pack_bf16x2(sv.x, sv.y), pack_bf16x2(sv.z, sv.w));
  *reinterpret_cast<uint2*>(a.dk + at) = make_uint2(pack_bf16x2(sk.x, sk.y), pack_bf16x2(sk.z, sk.w));
}

// dq from the parts of split keys, added in their order: four neighbouring elements a thread.
template <int D>
__global__ void __launch_bounds__(256) cross_dq_join_kernel(CrossGeom g, int splits, float scale,
                                                            const float* __restrict__ part,
                                                            __nv_bfloat16* __restrict__ dq) {
  const long long rows = (long long)g.B * g.N * g.H;
  const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) / (D / 4);
  const int c4 = threadIdx.x % (D / 4);
  if (at >= rows) return;
  const int head = (int)(at % g.H);
  const long long bn = at / g.H, b = bn / g.N, tok = bn % g.N;
  const float4* p = reinterpret_cast<const float4*>(part) + ((b * g.H + head) * g.N + tok) * (D / 4) + c4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < splits; ++i) {
    const float4 v = p[(long long)i * rows * (D / 4)];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  *reinterpret_cast<uint2*>(dq + at * D + 4 * c4) =
      make_uint2(pack_bf16x2(s.x * scale, s.y * scale), pack_bf16x2(s.z * scale, s.w * scale));
}

// Row statistics: (lse / log 2, sum over the row of do out), one row of D elements by D/8 lanes,
// four rows a thread so that enough loads are in flight. A row without a key gets lse = +inf,
// which makes its probabilities zero. Grid: rows of an item, item. One block also writes the
// prefix sums of the items' key tiles.
template <int D>
__global__ void __launch_bounds__(256) cross_stats_kernel(CrossGeom g, KeySet keys, const __nv_bfloat16* __restrict__ out,
                                                          const __nv_bfloat16* __restrict__ dout,
                                                          const float* __restrict__ lse, float2* __restrict__ stats,
                                                          int* __restrict__ prefix) {
  constexpr int L = D / 8, kRows = 256 / L;         // lanes of a row; rows of a pass
  if (blockIdx.x == 0 && blockIdx.y == 0 && prefix && threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0;
    for (int i0 = 0; i0 < g.B; i0 += 32) {
      const int b = i0 + lane;
      const int nt = b < g.B ? (item_keys(keys, b, g.M).x + kCrossTile - 1) / kCrossTile : 0;
      int incl = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (b < g.B) prefix[b] = run + incl - nt;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[g.B] = run;
  }
  const uint32_t rows = (uint32_t)g.N * (uint32_t)g.H;      // of an item, below 2^31
  const uint32_t r0 = blockIdx.x * (4u * kRows) + threadIdx.x / L;
  const int part = threadIdx.x % L;
  const long long item = (long long)blockIdx.y * rows;
  uint4 o[4], d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = r0 + (uint32_t)(i * kRows);
    o[i] = d[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      o[i] = *reinterpret_cast<const uint4*>(out + (item + r) * D + part * 8);
      d[i] = *reinterpret_cast<const uint4*>(dout + (item + r) * D + part * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = r0 + (uint32_t)(i * kRows);
    const uint32_t ov[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, dv[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s += __uint_as_float(ov[k] << 16) * __uint_as_float(dv[k] << 16);
      s += __uint_as_float(ov[k] & 0xffff0000u) * __uint_as_float(dv[k] & 0xffff0000u);
    }
#pragma unroll
    for (int k = L / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (part == 0 && r < rows) {
      const uint32_t tok = r / (uint32_t)g.H, head = r - tok * (uint32_t)g.H;
      const long long at = ((long long)blockIdx.y * g.H + head) * g.N + tok;
      const float z = lse[at];
      stats[at] = z == -INFINITY ? make_float2(INFINITY, 0.f) : make_float2(z * 1.4426950408889634f, s);
    }
  }
}

template <int D>
cudaError_t run_bwd(const CUtensorMap& mq, const CUtensorMap& mdo, const CUtensorMap& mk, const CUtensorMap& mv,
                    const CUtensorMap& mdq, const BwdArgs& a, const __nv_bfloat16* out, const __nv_bfloat16* dout, const float* lse,
                    float2* stats, int* prefix, __nv_bfloat16* dq, cudaStream_t s) {
  const CrossGeom& g = a.g;
  const auto dq_kernel = a.splits > 1 ? cross_dq_kernel<D, true> : cross_dq_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CfgQ<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(cross_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CfgK<D>::kSmem);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)g.N * g.H, per = 4 * 256 / (D / 8);
  cross_stats_kernel<D><<<dim3((unsigned)((rows + per - 1) / per), g.B), 256, 0, s>>>(g, a.keys, out, dout, lse, stats, prefix);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int units = g.B * g.Hkv * a.splits * g.nqt;
  dq_kernel<<<units < kCrossSms ? units : kCrossSms, kThreads, CfgQ<D>::kSmem, s>>>(mq, mdo, mk, mv, mdq, a, units);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.splits > 1) {
    const long long quads = (long long)g.B * g.N * g.H * (D / 4);
    cross_dq_join_kernel<D><<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(g, a.splits, a.scale, a.part, dq);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const long long steps = (long long)g.B * g.Hkv * g.nkt * g.nqt;
  const int grid = (int)(steps < kCrossSms ? steps : kCrossSms);
  cross_dkv_kernel<D><<<grid, kThreads, CfgK<D>::kSmem, s>>>(mq, mdo, mk, mv, a);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cross_dkv_join_kernel<D><<<dim3(8, g.nkt, g.B * g.Hkv), 16 * D / 4, 0, s>>>(a, grid);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_bwd(const CrossCall& c, const void* out, const float* lse, const void* dout, void* dq,
                             void* dk, void* dv, cudaStream_t s) {
  const CrossGeom& g = c.g;
  const CrossWs w = cross_ws(g);
  BwdArgs a;
  a.g = g;
  a.keys = {c.kv_len, nullptr, nullptr};
  if (c.key_mask) {
    int2* plan = reinterpret_cast<int2*>(c.ws + w.plan);
    uint32_t* bits = reinterpret_cast<uint32_t*>(c.ws + w.bits);
    const cudaError_t e = launch_pack_keys(g, c.kv_len, c.key_mask, plan, bits, s);
    if (e != cudaSuccess) return e;
    a.keys = {nullptr, plan, bits};
  }
  float2* stats = reinterpret_cast<float2*>(c.ws + w.stats);
  int* prefix = c.key_mask || c.kv_len ? reinterpret_cast<int*>(c.ws + w.prefix) : nullptr;
  a.stats = stats;
  a.prefix = prefix;
  a.kb_mul = c.sk.b == 0 && g.B > 1 ? 0 : 1;
  a.vb_mul = c.sv.b == 0 && g.B > 1 ? 0 : 1;
  a.qb_mul = c.sq.b == 0 && g.B > 1 ? 0 : 1;
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.part = reinterpret_cast<float*>(c.ws + w.part);
  a.err = reinterpret_cast<uint32_t*>(c.ws);
  a.scale = c.scale;
  a.by_nqt = FastDiv((uint32_t)g.nqt);
  a.splits = cross_dq_splits(g);
  a.by_splits = FastDiv((uint32_t)a.splits);
  a.scale_log2 = c.scale * 1.4426950408889634f;
  const CrossStride dense = {(long long)g.N * g.H * g.d, (long long)g.H * g.d, g.d};
  CUtensorMap mq, mdo, mk, mv, mdq;
  if (!make_map_4d(&mq, c.q, g.d, g.H, g.N, g.B, c.sq, g.G, g.tpt) ||
      !make_map_4d(&mdo, dout, g.d, g.H, g.N, g.B, dense, g.G, g.tpt) ||
      !make_map_4d(&mdq, dq, g.d, g.H, g.N, g.B, dense, g.G, g.tpt) ||
      !make_map_4d(&mk, c.k, g.d, g.Hkv, g.M, g.B, c.sk, 1, kCrossTile) ||
      !make_map_4d(&mv, c.v, g.d, g.Hkv, g.M, g.B, c.sv, 1, kCrossTile))
    return cudaErrorInvalidValue;
  const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(out);
  const __nv_bfloat16* d = static_cast<const __nv_bfloat16*>(dout);
  __nv_bfloat16* q = static_cast<__nv_bfloat16*>(dq);
  return g.d == 128 ? run_bwd<128>(mq, mdo, mk, mv, mdq, a, o, d, lse, stats, prefix, q, s)
                    : run_bwd<64>(mq, mdo, mk, mv, mdq, a, o, d, lse, stats, prefix, q, s);
}

}  // namespace bsa
