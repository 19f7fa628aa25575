// Layer norm over the last axis, forward and backward, with the reduction of the weight's and
// bias's gradients.
//
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd (offset + w) + b
//   g  = dy (offset + w),  h = (x - mean) rstd
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// Rows are grouped into items of `per` consecutive rows; w and b are absent, shared by every
// row (one item of all rows) or one row per item (the modulation of a diffusion transformer).
// Everything is computed in fp32 from one read of each row, held in registers: the variance
// is the sum of squared distances from the mean (no cancellation on rows far from zero). The
// one rounding to fewer bits is that of the stored y and dx.
//
// Both passes are bound by HBM (2 C reads and writes a row forward, 3 C backward). Layout:
// a thread holds slots of 8 elements (one 16-byte load of bf16, two of fp32), so a row of up
// to 256 elements takes 8, 16 or 32 lanes and a block several rows, and a longer row takes a
// block of its own, with 2 or 4 slots a thread. Each thread copies its own slots of
// the next three groups of rows to shared memory while one group is at work: the bytes in
// flight cost no registers and no barrier. Rows of another even width go in pairs of elements, and odd widths (or
// addresses that allow no more) in single coalesced loads without copies ahead.
// The grid is persistent: each block takes one contiguous range of rows and in the backward pass
// keeps the column sums of the rows it has seen. It writes them as one partial row for each item that its range meets; a second kernel adds
// the partials of an item in the order of the blocks. No atomics: repeated calls give
// identical bits.
//
// Measured, one B200, two passes alike: 75600 x 5120 bf16 forward 285 us (5.4 TB/s of the 6.6 that a
// copy reaches), backward with the weight's gradient 463 us (5.0 TB/s); 65520 x 1536, fp32 to bf16,
// 108 and 198 us (5.6 and 5.1 TB/s); 393120 rows of 128 bf16 46 and 81 us (4.3 and 3.7 TB/s; fewer
// bytes a reduction: the forward pass has 72 % of its issue slots busy, the backward pass 45 %); the
// even width 5450 2.4 and 2.8 TB/s; odd widths 0.9 to 1.2 TB/s forward (1001, 1537, 2049 to 2559, 4097)
// and 0.9 to 1.6 backward, single elements without copies ahead; 8200 to 10240 bf16 3.3 to 4.0 and
// 1.8 to 1.9 TB/s.
#include "f32x2.cuh"
#include "norm.cuh"

namespace bsa {
namespace {

struct NormArgs {
  const void* x;
  const void* dy;          // backward
  const void* w;           // nullable; [C] or [items, C]
  const void* b;           // nullable (forward)
  void* y;                 // y, or dx
  float* mean;             // nullable in the forward pass
  float* rstd;
  float* part;             // backward: partial dw, then partial db, [blocks + items, C] each
  long long rows, per;     // per: rows of an item
  long long slots;         // blocks + items
  int C;
  int tpr;                 // threads of a row
  bool w_bf16, w_items;
  float eps, offset;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Column of element j of slot k of thread t: runs of E neighbouring elements a thread, neighbouring
// threads on neighbouring runs. E = 8 (16 bytes of bf16) or, where one side is fp32, 4 (16 bytes
// of that); 2 for rows of an even width that is not a multiple of 8; 1 for odd widths and
// addresses that allow no more.
template <int E>
__device__ __forceinline__ int column(int t, int k, int j, int tpr) {
  return ((k * (8 / E) + j / E) * tpr + t) * E + j % E;
}
// Eight elements of a row in registers: from global memory one by one, or (E > 1) from the runs
// that the thread has copied to shared memory.
template <typename T, int E>
struct Slot {
  static constexpr int kWords = 2 * sizeof(T);      // 32-bit words
  uint32_t v[kWords];
  __device__ __forceinline__ void load(const T* row, int t, int k, int tpr, int C, bool ok) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<E>(t, k, j, tpr);
      const float f = (ok && c < C) ? to_f(row[c]) : 0.f;
      if (sizeof(T) == 4) v[j] = __float_as_uint(f);
      else if (j & 1) v[j >> 1] |= __float_as_uint(f);
      else v[j >> 1] = __float_as_uint(f) >> 16;
    }
  }
  __device__ __forceinline__ void take(const uint4* p, int plane) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = p[i * plane];
      v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
    }
  }
  // Elements 2 i and 2 i + 1.
  __device__ __forceinline__ uint64_t pair(int i) const { return f2(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ float get(int j) const {
    if (sizeof(T) == 4) return __uint_as_float(v[j & (kWords - 1)]);
    return __uint_as_float((j & 1) ? (v[j >> 1] & 0xffff0000u) : (v[j >> 1] << 16));
  }
};

// 16-byte places of a slot, and the copy of one slot to the thread's own places in shared memory
// (`plane` apart; zeros past the row's end or for a row that is not there). Nobody else reads
// them, so waiting for one's own copies is all the ordering there is.
template <typename T>
constexpr int kPieces = sizeof(T) / 2;
template <int E, typename T>
__device__ __forceinline__ void copy_slot(uint4* dst, int plane, const T* row, int t, int k, int tpr, int C, bool ok) {
  constexpr int kBytes = E * sizeof(T);
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
  for (int i = 0; i < 8 / E; ++i) {
    const int c = column<E>(t, k, i * E, tpr), off = i * kBytes;
    const bool in = ok && c < C;
    const T* src = in ? row + c : row;
    const uint32_t at = to + (uint32_t)((off >> 4) * 16 * plane + (off & 15));
    if (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src), "r"(in ? 16 : 0) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(src), "n"(kBytes), "r"(in ? kBytes : 0)
                   : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Copies of one thread land in any order: a place must not be the target of a second one before
// the first has been waited for. Zero fills past an item's rows are still under way when its last
// row is done.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int E, typename T>
__device__ __forceinline__ void store_slot(T* row, int t, int k, int tpr, int C, const float (&o)[8]) {
  if (E == 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<E>(t, k, j, tpr);
      if (c < C) put(row + c, o[j]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8 / E; ++i) {
    const int c = column<E>(t, k, i * E, tpr);
    if (c >= C) continue;
    if (sizeof(T) == 4) {
      if (E == 2) *reinterpret_cast<float2*>(row + c) = make_float2(o[2 * i], o[2 * i + 1]);
      else *reinterpret_cast<float4*>(row + c) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(o[E * i + 2 * h], o[E * i + 2 * h + 1]);
        u[h] = *reinterpret_cast<const uint32_t*>(&p);
      }
      if (E == 8) *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
      else if (E == 4) *reinterpret_cast<uint2*>(row + c) = make_uint2(u[0], u[1]);
      else *reinterpret_cast<uint32_t*>(row + c) = u[0];
    }
  }
}

// (offset +) w or b of the columns of one slot, or `absent`; zero past C. Held in registers for an
// item: read again for every group of rows they cost as much L2 traffic as the rows.
template <int E>
__device__ __forceinline__ void load_affine(const void* p, bool bf16, long long at, float add, float absent, int t,
                                            int k, int tpr, int C, uint64_t (&o)[4]) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = column<E>(t, k, j, tpr);
    v[j] = c < C ? absent : 0.f;
    if (p && c < C)
      v[j] = add + (bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at + c])
                         : static_cast<const float*>(p)[at + c]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f2(v[2 * i], v[2 * i + 1]);
}

// Sums of S values over the threads of a row, left in every one of them. tpr <= 32: lanes of
// one warp. Else the block is one row: warp sums meet in `red` [S][32]; the caller alternates
// two such arrays, so that one barrier a call is enough.
template <int S>
__device__ __forceinline__ void row_sum(float (&s)[S], int tpr, float* red) {
  const int w = tpr < 32 ? tpr : 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < w)
#pragma unroll
      for (int i = 0; i < S; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < S; ++i) red[i * 32 + warp] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < S; ++i) {
    s[i] = lane < nw ? red[i * 32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  }
}

// Rows are taken in groups of U a lane group; all but one of a ring of groups are on their way to
// shared memory while one is at work (E > 1). Four groups, fewer where the pieces of an SM's
// threads are over 200 KB.
template <typename XT, int VPT, int U>
constexpr int kFwdPieces = U* VPT* kPieces<XT>;
template <typename XT, typename YT, int VPT, int U>
constexpr int kBwdPieces = U* VPT*(kPieces<XT> + kPieces<YT>);
constexpr int ring_depth(int pieces, int threads_sm) {
  const int d = 204800 / (16 * pieces * threads_sm);
  return d < 1 ? 1 : d > 4 ? 4 : d;
}

template <typename XT, typename YT, int E, int VPT, int U, int T, int kPerSm>
__global__ void __launch_bounds__(T, kPerSm) norm_fwd_kernel(NormArgs a) {
  __shared__ float red[2][U * 32];
  extern __shared__ uint4 ring[];         // [kDepth][piece][thread]
  constexpr bool kAhead = E > 1;
  constexpr int P = kPieces<XT>, kDepth = ring_depth(kFwdPieces<XT, VPT, U>, T * kPerSm);
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const int plane = blockDim.x;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  YT* y = static_cast<YT*>(a.y);
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  const long long step = (long long)rpb * U;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per), wat = a.w_items ? item * C : 0;
    uint64_t w[VPT][4], b[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      load_affine<E>(a.w, a.w_bf16, wat, a.offset, 1.f, t, k, tpr, C, w[k]);
      load_affine<E>(a.b, a.w_bf16, wat, 0.f, 0.f, t, k, tpr, C, b[k]);
    }
    int put = 0, got = 0;                 // ring stages
    auto request = [&](long long base) {
      if (kAhead) {
        uint4* dst = ring + put * (kFwdPieces<XT, VPT, U> * plane) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub;
#pragma unroll
          for (int k = 0; k < VPT; ++k)
            copy_slot<E>(dst + (u * VPT + k) * P * plane, plane, x + (r < end ? r : r0) * C, t, k, tpr, C, r < end);
        }
        copies_commit();
        put = put + 1 == kDepth ? 0 : put + 1;
      }
    };
    for (int i = 0; i < kDepth - 1; ++i) request(r0 + i * step);
    for (long long base = r0; base < end; base += step) {
      Slot<XT, E> xs[U][VPT];
      request(base + (kDepth - 1) * step);
      if constexpr (kAhead) {
        copies_wait<kDepth - 1>();
        const uint4* src = ring + got * (kFwdPieces<XT, VPT, U> * plane) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < VPT; ++k) xs[u][k].take(src + (u * VPT + k) * P * plane, plane);
        got = got + 1 == kDepth ? 0 : got + 1;
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub;
#pragma unroll
          for (int k = 0; k < VPT; ++k) xs[u][k].load(x + (r < end ? r : base) * C, t, k, tpr, C, r < end);
        }
      }
      float m[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i & 1] = fadd2(sum[i & 1], xs[u][k].pair(i));
        float s0, s1;
        uf2(fadd2(sum[0], sum[1]), s0, s1);
        m[u] = s0 + s1;
      }
      row_sum<U>(m, tpr, red[0]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        m[u] *= inv_c;
        const uint64_t nm = f2(-m[u], -m[u]);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint64_t d = fadd2(xs[u][k].pair(i), nm);
            if (E > 1) {
              if (column<E>(t, k, 2 * i, tpr) >= C) d = 0ull;
            } else {
              float d0, d1;
              uf2(d, d0, d1);
              d = f2(column<E>(t, k, 2 * i, tpr) < C ? d0 : 0.f, column<E>(t, k, 2 * i + 1, tpr) < C ? d1 : 0.f);
            }
            sum[i & 1] = ffma2(d, d, sum[i & 1]);
          }
        float s0, s1;
        uf2(fadd2(sum[0], sum[1]), s0, s1);
        v[u] = s0 + s1;
      }
      row_sum<U>(v, tpr, red[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub;
        v[u] = 1.0f / sqrtf(v[u] * inv_c + a.eps);
        if (t == 0 && r < end) {
          if (a.mean) a.mean[r] = m[u];
          if (a.rstd) a.rstd[r] = v[u];
        }
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub;
          const uint64_t nm = f2(-m[u], -m[u]), rs = f2(v[u], v[u]);
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            uf2(ffma2(fmul2(fadd2(xs[u][k].pair(i), nm), rs), w[k][i], b[k][i]), o[2 * i], o[2 * i + 1]);
          if (r < end) store_slot<E>(y + r * C, t, k, tpr, C, o);
        }
      }
    }
    if (kAhead) copies_wait<0>();         // see copies_wait: the next item starts at the first stage again
    r0 = end;
  }
}

template <typename XT, typename YT, int E, int VPT, int U, int T, int kPerSm>
__global__ void __launch_bounds__(T, kPerSm) norm_bwd_kernel(NormArgs a) {
  __shared__ float red[2][2 * U * 32];
  extern __shared__ uint4 ring[];         // [kDepth][piece][thread]
  constexpr bool kAhead = E > 1;
  constexpr int PX = kPieces<XT>, PY = kPieces<YT>, kDepth = ring_depth(kBwdPieces<XT, YT, VPT, U>, T * kPerSm);
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const int plane = blockDim.x;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  const YT* dy = static_cast<const YT*>(a.dy);
  XT* dx = static_cast<XT*>(a.y);
  // several rows a block: their column sums [2][C] meet here, behind the ring
  float* acc = reinterpret_cast<float*>(ring + (kAhead ? kDepth * kBwdPieces<XT, YT, VPT, U> * plane : 0));
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  const long long step = (long long)rpb * U;
  int flip = 0;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per), wat = a.w_items ? item * C : 0;
    uint64_t w[VPT][4], dw[VPT][4], db[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_affine<E>(a.w, a.w_bf16, wat, a.offset, 1.f, t, k, tpr, C, w[k]);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) dw[k][i] = db[k][i] = 0ull;
    int put = 0, got = 0;                 // ring stages
    auto request = [&](long long base) {
      if (kAhead) {
        uint4* dst = ring + put * (kBwdPieces<XT, YT, VPT, U> * plane) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub, q = r < end ? r : r0;
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            copy_slot<E>(dst + (u * VPT + k) * (PX + PY) * plane, plane, x + q * C, t, k, tpr, C, r < end);
            copy_slot<E>(dst + ((u * VPT + k) * (PX + PY) + PX) * plane, plane, dy + q * C, t, k, tpr, C, r < end);
          }
        }
        copies_commit();
        put = put + 1 == kDepth ? 0 : put + 1;
      }
    };
    for (int i = 0; i < kDepth - 1; ++i) request(r0 + i * step);
    for (long long base = r0; base < end; base += step) {
      Slot<XT, E> xs[U][VPT];
      Slot<YT, E> gs[U][VPT];
      float m[U], rs[U], s[2 * U];
      request(base + (kDepth - 1) * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub, q = r < end ? r : base;
        // a row that is not there: dy is zero, and so is h, whatever another row's statistics are
        m[u] = r < end ? a.mean[q] : 0.f;
        rs[u] = r < end ? a.rstd[q] : 0.f;
      }
      if constexpr (kAhead) {
        copies_wait<kDepth - 1>();
        const uint4* src = ring + got * (kBwdPieces<XT, YT, VPT, U> * plane) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            xs[u][k].take(src + (u * VPT + k) * (PX + PY) * plane, plane);
            gs[u][k].take(src + ((u * VPT + k) * (PX + PY) + PX) * plane, plane);
          }
        got = got + 1 == kDepth ? 0 : got + 1;
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub, q = r < end ? r : base;
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            xs[u][k].load(x + q * C, t, k, tpr, C, r < end);
            gs[u][k].load(dy + q * C, t, k, tpr, C, r < end);
          }
        }
      }
      uint64_t s1[U], s2[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s1[u] = s2[u] = 0ull;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint64_t nm = f2(-m[u], -m[u]), r2 = f2(rs[u], rs[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // Past the row's end dy is zero, so neither sum sees the element: sum g h is taken as
            // rstd sum g (x - mean), since h = (0 - mean) rstd may be infinite there where the row's
            // own are not.
            const uint64_t d = gs[u][k].pair(i), e = fadd2(xs[u][k].pair(i), nm), h = fmul2(e, r2), g = fmul2(d, w[k][i]);
            s1[u] = fadd2(s1[u], g);
            s2[u] = ffma2(g, e, s2[u]);
            dw[k][i] = ffma2(d, h, dw[k][i]);
            db[k][i] = fadd2(db[k][i], d);
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float p0, p1;
        uf2(s1[u], p0, p1);
        s[2 * u] = p0 + p1;
        uf2(s2[u], p0, p1);
        s[2 * u + 1] = p0 + p1;
      }
      row_sum<2 * U>(s, tpr, red[flip]);
      flip ^= 1;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub;
          const float c1 = s[2 * u] * inv_c, c2 = s[2 * u + 1] * rs[u] * inv_c;
          const uint64_t nm = f2(-m[u], -m[u]), r2 = f2(rs[u], rs[u]), n1 = f2(-c1, -c1), n2 = f2(-c2, -c2);
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t h = fmul2(fadd2(xs[u][k].pair(i), nm), r2);
            uf2(fmul2(ffma2(h, n2, ffma2(gs[u][k].pair(i), w[k][i], n1)), r2), o[2 * i], o[2 * i + 1]);
          }
          if (r < end) store_slot<E>(dx + r * C, t, k, tpr, C, o);
        }
      }
    }
    if (kAhead) copies_wait<0>();
    if (a.part) {
      // this block's partial row of the item: block + item counts up along the blocks' ranges,
      // so no two (block, item) pairs share it
      float* pw = a.part + (blockIdx.x + (a.w_items ? item : 0)) * C;
      float* pb = pw + a.slots * C;
      float vw[VPT][8], vb[VPT][8];
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uf2(dw[k][i], vw[k][2 * i], vw[k][2 * i + 1]);
          uf2(db[k][i], vb[k][2 * i], vb[k][2 * i + 1]);
        }
      if (rpb == 1) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = column<E>(t, k, j, tpr);
            if (c < C) pw[c] = vw[k][j], pb[c] = vb[k][j];
          }
      } else {
        for (int g = 0; g < rpb; ++g) {     // the rows' sums one after the other, in a fixed order
          if (sub == g)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int c = column<E>(t, k, j, tpr);
                if (c < C) {
                  acc[c] = g == 0 ? vw[k][j] : acc[c] + vw[k][j];
                  acc[C + c] = g == 0 ? vb[k][j] : acc[C + c] + vb[k][j];
                }
              }
          __syncthreads();
        }
        for (int c = threadIdx.x; c < C; c += blockDim.x) pw[c] = acc[c], pb[c] = acc[C + c];
        __syncthreads();
      }
    }
    r0 = end;
  }
}

// dw (blockIdx.z = 0) or db (1) of item blockIdx.y: the partial rows of the blocks whose range
// meets the item's rows, summed in the order of the blocks. 32 columns a block, 32 partial
// rows at a time.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ part, long long slots,
                                                           long long rows, long long per, int blocks, int C,
                                                           float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[32][33];
  float* out = blockIdx.z ? db : dw;
  if (!out) return;
  const long long item = blockIdx.y, first = item * per, last = min(rows, first + per) - 1;
  // block k covers rows [rows k / blocks, rows (k + 1) / blocks)
  long long b0 = first * blocks / rows, b1 = last * blocks / rows;
  while (b0 > 0 && rows * b0 / blocks > first) --b0;
  while (rows * (b0 + 1) / blocks <= first) ++b0;
  while (b1 > 0 && rows * b1 / blocks > last) --b1;
  while (rows * (b1 + 1) / blocks <= last) ++b1;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < C) {
    const float* p = part + (blockIdx.z ? slots * C : 0) + item * C + c;
    for (long long k = b0 + threadIdx.y; k <= b1; k += 32) v += p[k * C];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < C) out[item * C + cc] = v;
}

// Threads of a row, slots a thread and threads of a block for a row of C elements. More slots a
// thread mean fewer warps a row, and the reductions, whose cost goes by the warp, are what a
// block waits for (75600 rows of 5120 with 1 slot and 20 warps: 389 us); registers set the limit:
// a slot takes 4 (bf16) or 8 of the row and 16 of w and b, or 24 of w, dw and db.
// `built` is the thread count that the kernel of the launch is compiled for: norm_blocks reckons what
// is resident on an SM by it, and run_norm takes the kernel by it.
struct NormShape {
  int tpr, vpt, threads, built;
};
NormShape norm_shape(int C, bool bwd, bool fp32, int run) {
  const int slots = ceil_div(C, 8), most = run == 1 ? 1 : bwd || fp32 || run == 2 ? 2 : 4;
  NormShape n;
  if (slots <= 32 * most) {                         // a warp or less
    n.vpt = slots <= 32 ? 1 : slots <= 64 ? 2 : 4;
    n.tpr = slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
    n.threads = n.built = 256;
    return n;
  }
  if (run == 1) {                                    // no copies ahead: as many threads as go
    n.vpt = slots <= 640 ? 1 : slots <= 1024 ? 2 : 4;
  } else {                                          // the fewest lanes without work, then the fewest threads
    n.vpt = most == 4 && 128 * ceil_div(slots, 128) <= 64 * ceil_div(slots, 64) ? 4 : 2;
    if (slots > 1024) n.vpt = 4;
  }
  n.threads = n.tpr = 32 * ceil_div(slots, 32 * n.vpt);
  if (run == 1) n.built = n.vpt > 1 ? 512 : n.threads > 256 ? 640 : 256;
  else n.built = n.threads <= 256 ? 256 : n.vpt == 2 && n.threads <= 320 ? 320 : 512;
  return n;
}

constexpr int kNormSms = 148;     // SMs of the part; the workspace is sized without asking the device

// Rows that a lane group takes together: more make fewer reductions, fewer leave registers.
template <typename XT, int E, int VPT>
constexpr int kFwdU = E == 1 ? 1 : VPT == 1 ? 8 / sizeof(XT) : VPT == 2 ? 4 / sizeof(XT) : 1;
template <int E, int VPT>
constexpr int kBwdU = E > 1 && VPT == 1 ? 2 : 1;

// Blocks an SM that a kernel is built for: registers to hold nearly everything (what does not fit goes
// through L2, since the copies ahead leave L1 little: a backward pass with 216 bytes of it a
// thread took twice as long). What is left of it: some 60 to 120 bytes a thread in the backward
// form of 320 threads, up to 30 forward, 460 to 1120 in the backward forms of four slots (widths
// above 8192) and 660 forward where such a width is odd. Two blocks an SM end at 320 threads, 5120
// elements at two slots a thread: wider rows have 9 to 16 warps an SM, and no second form was
// measured for them.
constexpr int per_sm(int vpt, int T, bool bwd, int E) {
  return T > 320 ? 1 : vpt > 1 ? 2 : (bwd ? 2 : 3) + (E == 1 ? 1 : 0);
}

// Blocks of a launch: enough to fill the device, never more than there are rows for one each of a
// block's lane groups.
int norm_blocks(const NormShape& n, long long rows, bool bwd, int run) {
  const long long step = n.threads / n.tpr, need = (rows + step - 1) / step;
  const long long full = (long long)kNormSms * (per_sm(n.vpt, n.built, bwd, run) * n.built / n.threads);
  return (int)(need < full ? need : full);
}

// `most`: the largest shared memory that a launch of this kernel takes. Above 48 KB, static arrays
// included, it needs leave, asked for at every launch (a device reset forgets it) and for the most,
// so that launches of other sizes on other threads do not take it away.
template <auto kKernel>
cudaError_t start(const NormArgs& a, int blocks, int threads, size_t smem, size_t most, cudaStream_t s) {
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
  }
  kKernel<<<blocks, threads, smem, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename XT, typename YT, int E, int VPT, int T>
cudaError_t run_fwd(const NormArgs& a, const NormShape& n, int blocks, cudaStream_t s) {
  constexpr int U = kFwdU<XT, E, VPT>, kPieces = kFwdPieces<XT, VPT, U>;
  constexpr size_t kThread = E > 1 ? 16 * ring_depth(kPieces, T * per_sm(VPT, T, false, E)) * kPieces : 0;
  return start<norm_fwd_kernel<XT, YT, E, VPT, U, T, per_sm(VPT, T, false, E)>>(a, blocks, n.threads, kThread * n.threads,
                                                                        kThread * T, s);
}
template <typename XT, typename YT, int E, int VPT, int T>
cudaError_t run_bwd(const NormArgs& a, const NormShape& n, int blocks, cudaStream_t s) {
  constexpr int U = kBwdU<E, VPT>, kPieces = kBwdPieces<XT, YT, VPT, U>;
  constexpr size_t kThread = E > 1 ? 16 * ring_depth(kPieces, T * per_sm(VPT, T, true, E)) * kPieces : 0;
  const size_t acc = n.tpr < n.threads && a.part ? 2 * sizeof(float) * a.C : 0;      // rows of at most 512
  return start<norm_bwd_kernel<XT, YT, E, VPT, U, T, per_sm(VPT, T, true, E)>>(
      a, blocks, n.threads, kThread * n.threads + acc, kThread * T + 2 * sizeof(float) * 512, s);
}

template <typename XT, typename YT, int E, int VPT, int T>
cudaError_t run_either(const NormArgs& a, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  return bwd ? run_bwd<XT, YT, E, VPT, T>(a, n, blocks, s) : run_fwd<XT, YT, E, VPT, T>(a, n, blocks, s);
}
template <typename XT, typename YT, int E>
cudaError_t run_norm(const NormArgs& a, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  // what norm_shape gives for these rows, and nothing else
  if constexpr (E == 1) {
    if (n.built == 640) return run_either<XT, YT, E, 1, 640>(a, bwd, n, blocks, s);
  } else {
    if (n.vpt == 2 && n.built == 256) return run_either<XT, YT, E, 2, 256>(a, bwd, n, blocks, s);
    if (n.built == 320) return run_either<XT, YT, E, 2, 320>(a, bwd, n, blocks, s);
    if constexpr (E >= 4 && sizeof(XT) == 2)        // forward only: the backward pass has 4 slots past 256 threads
      if (n.vpt == 4 && n.built == 256) return run_fwd<XT, YT, E, 4, 256>(a, n, blocks, s);
  }
  if (n.vpt == 1) return run_either<XT, YT, E, 1, 256>(a, bwd, n, blocks, s);
  if (n.vpt == 2) return run_either<XT, YT, E, 2, 512>(a, bwd, n, blocks, s);
  return run_either<XT, YT, E, 4, 512>(a, bwd, n, blocks, s);
}

NormArgs norm_args(const bsa_norm_shape& f) {
  NormArgs a = {};
  a.rows = f.rows;
  a.C = f.C;
  a.per = f.w_per_item ? f.rows / f.items : f.rows;
  a.w_bf16 = f.w_type == BSA_BF16;
  a.w_items = f.w_per_item != 0;
  a.offset = f.weight_offset;
  a.eps = f.eps;
  return a;
}

template <typename XT, typename YT>
cudaError_t run_any(const NormArgs& a, int run, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  constexpr int kWide = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
  if (run == 2) return run_norm<XT, YT, 2>(a, bwd, n, blocks, s);
  return run == 1 ? run_norm<XT, YT, 1>(a, bwd, n, blocks, s) : run_norm<XT, YT, kWide>(a, bwd, n, blocks, s);
}

cudaError_t dispatch(const bsa_norm_shape& f, NormArgs& a, bool bwd, cudaStream_t s, int* blocks_out = nullptr) {
  const bool xb = f.x_type == BSA_BF16, yb = f.y_type == BSA_BF16;
  // x, and in the backward pass dx, are of one type, y or dy of the other; all rows start alike
  // where the width is a multiple of the run
  auto allows = [&](int run) {
    auto at = [run](const void* p, bool bf16) {
      const uintptr_t bytes = (uintptr_t)run * (bf16 ? 2 : 4);
      return (reinterpret_cast<uintptr_t>(p) & ((bytes < 16 ? bytes : 16) - 1)) == 0;
    };
    return f.C % run == 0 && at(a.x, xb) && at(a.y, bwd ? xb : yb) && at(a.dy, yb);
  };
  const int run = allows(8) ? 8 : allows(2) ? 2 : 1;
  const NormShape n = norm_shape(f.C, bwd, !xb, run);
  const int blocks = norm_blocks(n, f.rows, bwd, run);
  a.tpr = n.tpr;
  a.slots = blocks + (a.w_items ? f.items : 1);
  if (blocks_out) *blocks_out = blocks;
  if (xb && yb) return run_any<__nv_bfloat16, __nv_bfloat16>(a, run, bwd, n, blocks, s);
  if (xb) return run_any<__nv_bfloat16, float>(a, run, bwd, n, blocks, s);
  if (yb) return run_any<float, __nv_bfloat16>(a, run, bwd, n, blocks, s);
  return run_any<float, float>(a, run, bwd, n, blocks, s);
}

}  // namespace

size_t norm_workspace(const bsa_norm_shape& f) {
  int blocks = 0;                 // whatever the addresses allow of what the width does
  for (const int run : {1, 2, 8}) {
    if (f.C % run != 0) continue;
    const int n = norm_blocks(norm_shape(f.C, true, f.x_type == BSA_FP32, run), f.rows, true, run);
    if (n > blocks) blocks = n;
  }
  return align256((size_t)(blocks + (f.w_per_item ? f.items : 1)) * f.C * 2 * sizeof(float));
}

cudaError_t launch_norm_fwd(const bsa_norm_shape& f, const void* x, const void* w, const void* b, void* y,
                            float* mean, float* rstd, cudaStream_t s) {
  NormArgs a = norm_args(f);
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return dispatch(f, a, false, s);
}

cudaError_t launch_norm_bwd(const bsa_norm_shape& f, const void* x, const void* dy, const float* mean,
                            const float* rstd, const void* w, void* dx, float* dw, float* db, void* ws,
                            cudaStream_t s) {
  NormArgs a = norm_args(f);
  a.x = x;
  a.dy = dy;
  a.w = w;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = dw || db ? static_cast<float*>(ws) : nullptr;
  int blocks = 0;
  const cudaError_t e = dispatch(f, a, true, s, &blocks);
  if (e != cudaSuccess || !a.part) return e;
  const dim3 grid(ceil_div(f.C, 32), a.w_items ? f.items : 1, 2);
  norm_reduce_kernel<<<grid, dim3(32, 32), 0, s>>>(a.part, a.slots, a.rows, a.per, blocks, f.C, dw, db);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace bsa
