// Shared parts of the attention of the video tokens to an encoder's states: what a call is,
// its workspace, and the device helpers of its forward and backward kernels.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"
#include "tmem_ops.cuh"

namespace bsa {

constexpr int kCrossTile = 128;      // query rows and keys of a tile
constexpr int kCrossSms = 148;       // SMs of the part: bounds persistent grids and their workspace

// One call. The H / Hkv = G query heads of a key head are handled together: a query tile holds
// tpt = floor(128 / G) tokens, row r = (token r / G, head r % G), so that a key tile is read
// once for all of them and dk, dv sum over them where they are computed.
struct CrossGeom {
  int B, H, Hkv, d, N, M;
  int G, tpt;                        // query heads of a key head; tokens of a query tile
  int nqt, nkt;                      // query tiles (of one key head), key tiles
  FastDiv by_hkv, by_G;
};

inline CrossGeom make_cross(const bsa_cross_geom& g) {
  CrossGeom c;
  c.B = g.B; c.H = g.H; c.Hkv = g.Hkv; c.d = g.d; c.N = g.N; c.M = g.M;
  c.G = g.H / g.Hkv;
  c.tpt = kCrossTile / c.G;
  c.nqt = ceil_div(g.N, c.tpt);
  c.nkt = ceil_div(g.M, kCrossTile);
  c.by_hkv = FastDiv((uint32_t)g.Hkv);
  c.by_G = FastDiv((uint32_t)c.G);
  return c;
}

// Which keys a batch item attends to: all (both null), the first kv_len[b] (clamped to [0, M]),
// or, with a mask, the set bits of its packed words; `plan` then holds (last valid key + 1,
// number of valid keys).
struct KeySet {
  const int* kv_len;
  const int2* plan;
  const uint32_t* bits;              // [B, 4 nkt]
};

// Keys that an item reaches (0: none) and the number of valid ones.
__device__ __forceinline__ int2 item_keys(const KeySet& ks, int b, int M) {
  if (ks.plan) return ks.plan[b];
  if (!ks.kv_len) return make_int2(M, M);
  const int n = min(max(ks.kv_len[b], 0), M);
  return make_int2(n, n);
}

// Valid keys of key tile kt as 4 words of 32.
__device__ __forceinline__ uint4 tile_bits(const KeySet& ks, int b, int kt, int nkt, int len) {
  if (ks.bits) return reinterpret_cast<const uint4*>(ks.bits)[(long long)b * nkt + kt];
  const int n = len - kt * kCrossTile;
  auto word = [&](int i) -> uint32_t {
    const int m = n - 32 * i;
    return m >= 32 ? 0xffffffffu : m <= 0 ? 0u : ((1u << m) - 1u);
  };
  return make_uint4(word(0), word(1), word(2), word(3));
}
__device__ __forceinline__ bool all_set(uint4 w) { return (w.x & w.y & w.z & w.w) == 0xffffffffu; }

// -------------------------------------------------------------------- workspace layout
// [0, 256)  error word; then, 256-aligned: plan int2 [B], packed key bits u32 [B, 4 nkt], prefix of
// the items' key tiles int [B + 1], row statistics float2 [B, H, N] (backward), and one region
// that the forward pass uses for the partial results of split keys, the backward pass for those of
// dq and then for the partial dk, dv of its blocks.
struct CrossWs {
  size_t plan, bits, prefix, stats, part, total;
};

// Parts that the keys are split into when the query tiles alone do not fill the device. Joining
// takes a launch and some 3 us, so short walks stay whole (one query and 12 heads over 512 keys:
// 11.0 us, in 4 parts 6.3 + 3.0 us and the launch), and a part has at least two tiles (1024 keys:
// 11.1 us in parts of 4 tiles, 7.1 us in parts of 1, the join 2.9 and 4.1 us).
inline int cross_parts(const CrossGeom& g, int row_units) {
  const long long units = (long long)g.B * g.Hkv * row_units;
  if (units * 2 > kCrossSms || g.nkt < 8) return 1;
  const long long s = kCrossSms / units, most = g.nkt / 2;
  return (int)(s < most ? s : most);
}

inline int cross_splits(const CrossGeom& g) { return cross_parts(g, ceil_div(g.nqt, 2)); }   // forward
inline int cross_dq_splits(const CrossGeom& g) { return cross_parts(g, g.nqt); }

inline CrossWs cross_ws(const CrossGeom& g) {
  CrossWs w;
  size_t off = 256;
  w.plan = off; off = align256(off + (size_t)g.B * sizeof(int2));
  w.bits = off; off = align256(off + (size_t)g.B * g.nkt * 16);
  w.prefix = off; off = align256(off + ((size_t)g.B + 1) * sizeof(int));
  w.stats = off; off = align256(off + (size_t)g.B * g.H * g.N * sizeof(float2));
  w.part = off;
  const int s = cross_splits(g);
  const size_t fwd = s > 1 ? (size_t)s * g.B * g.N * g.H * (g.d + 1) * sizeof(float) : 0;
  const int sq = cross_dq_splits(g);
  const size_t dq = sq > 1 ? (size_t)sq * g.B * g.N * g.H * g.d * sizeof(float) : 0;
  const size_t dkv = (size_t)kCrossSms * 2 * 2 * kCrossTile * g.d * sizeof(float);
  const size_t bwd = dq > dkv ? dq : dkv;             // dq is joined before dk, dv begin
  w.total = align256(off + (fwd > bwd ? fwd : bwd));
  return w;
}

// ------------------------------------------------------------------------ device helpers
namespace cross {

// Bounded wait for the phase of parity `parity`: each try suspends the thread for at most 200 ns, so
// giving up takes between a third of a second and seven seconds. Gives up at once when another
// thread has set *abort; on time-out it sets *abort and the error bit. Kept short because it
// stands at every hand-over of warps that run little else: with a clock in it, the code of the
// waits alone displaced the others' from the instruction cache.
constexpr int kWaitTries = 1 << 25;
template <int kTries = kWaitTries>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kTries; ++i) {
    if (ptx::mbar_try_wait_ns(bar, parity, 200)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  atomicOr(err, BSA_KERR_WAIT_TIMEOUT);
  return false;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// All lanes take the same decision after a per-thread bounded wait.
template <int kTries = kWaitTries>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  return __all_sync(0xffffffffu, wait_phase<kTries>(bar, parity, abort, err));
}

// Box of a 4-D map (columns, heads, tokens, items) into shared memory.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int h, int n,
                                            int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c), "r"(h), "r"(n), "r"(b)
      : "memory");
}
// The same box into L2 only.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c, int h, int n, int b) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c), "r"(h), "r"(n), "r"(b)
               : "memory");
}
// The reverse copy; the part of the box outside the tensor is not written. Completion goes by
// this thread's bulk groups: `store_read` waits until the shared memory may be written again.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c, int h, int n, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c), "r"(h), "r"(n), "r"(b)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whole warps only, and converged ones (as with the tcgen05 reads and writes of TMEM): a __syncwarp
// stands between them and a branch that only some lanes take.
// A barrier of `threads` threads that also tells all of them whether all said yes: after a bounded
// wait, so that threads whose wait ran out and threads whose did not leave together.
__device__ __forceinline__ bool bar_all(int id, int threads, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)yes)
      : "memory");
  return r != 0;
}

// 32 columns of a row (16 bf16 pairs) into columns 32 ch .. of a [D/64][128 rows][128 B] tile with
// the 128-byte swizzle (16-byte piece i of row r at i xor (r mod 8)).
__device__ __forceinline__ void put_row32(uint8_t* tile, int row, int ch, const uint32_t (&pk)[16]) {
  uint8_t* p = tile + (ch >> 1) * (kCrossTile * 128) + row * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(p + ((((ch & 1) * 4 + i) ^ (row & 7)) << 4)) =
        make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
}

// Orders this thread's shared-memory writes before later reads by the tensor pipe and the copies.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Zeroes the rows of masked keys in a [D/64][128 rows][128 B] tile (the whole warp): a row whose
// probability is zero must not bring an infinity or a NaN into a product over the keys.
template <int D>
__device__ __forceinline__ void zero_masked_rows(uint8_t* tile, uint4 w, int lane) {
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (uint32_t miss = ~word[i]; miss; miss &= miss - 1) {
      const int row = 32 * i + __ffs(miss) - 1;
      if (lane < 8 * (D / 64))
        *reinterpret_cast<uint4*>(tile + (lane >> 3) * (kCrossTile * 128) + row * 128 + (lane & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    }
  fence_proxy_async();
  __syncwarp();
}

// One lane of a converged warp, always the same one. The issuing warps run whole, and only the
// products and commits themselves are left to this lane: their descriptors are then values of the
// warp, which the tensor instructions take as they are. (Issued from a loop of one lane, each
// product's operands were moved over one by one, between the softmax warps' instructions: 120
// cycles a step of 64.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// D[128 x 128] = A B^T of two K-major tiles, D/16 steps of 16 columns.
template <int D>
__device__ __forceinline__ void product_nt(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(128, 128, 0, 0);
  const uint64_t ad = ptx::smem_desc_sw128(a_smem, 16, 1024), bd = ptx::smem_desc_sw128(b_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t o = (uint64_t)(((kk >> 2) * (kCrossTile * 128) + (kk & 3) * 32) >> 4);
    ptx::mma_ss(d_tmem, ad + o, bd + o, id, kk > 0 ? 1u : 0u);
  }
}

// D[128 x D] (+)= A B of a bf16 A in TMEM (128 contraction columns: 64 32-bit columns, the second
// half `gap` columns after the first) and a tile B whose rows are the contraction.
template <int D, int kHalf>
__device__ __forceinline__ void product_nn_half(uint32_t d_tmem, uint32_t a_tmem, int gap, uint32_t b_smem, bool accumulate) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(128, D, 0, 1);
  const uint64_t bd = ptx::smem_desc_sw128(b_smem, kCrossTile * 128, 1024);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    ptx::mma_ts(d_tmem, a_tmem + (uint32_t)(k * 8 + kHalf * gap), bd + (uint64_t)((4 * kHalf + k) * (2048 >> 4)), id,
                (k > 0 || kHalf || accumulate) ? 1u : 0u);
}
template <int D>
__device__ __forceinline__ void product_nn(uint32_t d_tmem, uint32_t a_tmem, int gap, uint32_t b_smem, bool accumulate) {
  product_nn_half<D, 0>(d_tmem, a_tmem, gap, b_smem, accumulate);
  product_nn_half<D, 1>(d_tmem, a_tmem, gap, b_smem, true);
}

}  // namespace cross

// Tensor maps of one call: q-like tensors (boxes of one query tile's tokens and heads) and
// k-like ones (boxes of 128 keys of one head), 64 columns wide with the 128-byte swizzle.
struct CrossStride {
  long long b, n, h;                 // elements
};
bool make_map_4d(CUtensorMap* m, const void* base, int d, int heads, int tokens, int items, const CrossStride& s,
                 int box_heads, int box_tokens);

// Packs a key mask (and kv_len) into `bits` and `plan`.
cudaError_t launch_pack_keys(const CrossGeom& g, const int* kv_len, const uint8_t* key_mask, int2* plan,
                             uint32_t* bits, cudaStream_t s);

struct CrossCall {
  CrossGeom g;
  CrossStride sq, sk, sv;
  const void *q, *k, *v;
  const int* kv_len;
  const uint8_t* key_mask;
  float scale;
  uint8_t* ws;
};
cudaError_t launch_cross_fwd(const CrossCall& c, void* out, float* lse, cudaStream_t s);
cudaError_t launch_cross_bwd(const CrossCall& c, const void* out, const float* lse, const void* dout, void* dq,
                             void* dk, void* dv, cudaStream_t s);

}  // namespace bsa
