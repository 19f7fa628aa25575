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
// flight cost no registers and no barrier. Rows whose width or address does not
// allow 16-byte loads take the same kernels with single-element, coalesced loads.
// The grid is persistent: each block takes one contiguous range of rows and in the backward pass
// keeps the column sums of the rows it has seen. It writes them as one partial row for each item that its range meets; a second kernel adds
// the partials of an item in the order of the blocks. No atomics: repeated calls give
// identical bits.
#include "common.cuh"

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

// Column of element j of slot k of thread t: runs of E neighbouring elements a thread, E = 8 (16
// bytes of bf16) or, where one side is fp32, 4 (16 bytes of that), or 1 where rows do not allow
// wide accesses; neighbouring threads on neighbouring runs.
template <int E>
__device__ __forceinline__ int column(int t, int k, int j, int tpr) {
  return ((k * (8 / E) + j / E) * tpr + t) * E + j % E;
}
template <typename XT, typename YT, bool VEC>
constexpr int kRun = !VEC ? 1 : sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;

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
    if (sizeof(T) == 2 && E == 4) {                 // two runs of 8 bytes in one 16-byte place
      const uint2 a = reinterpret_cast<const uint2*>(p)[0], b = reinterpret_cast<const uint2*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = p[i * plane];
        v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
      }
    }
  }
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
    const int c = column<E>(t, k, i * E, tpr);
    const bool in = ok && c < C;
    const T* src = in ? row + c : row;
    if (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 16 * i * plane), "l"(src), "r"(in ? 16 : 0)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + 8 * i), "l"(src), "r"(in ? 8 : 0) : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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
      *reinterpret_cast<float4*>(row + c) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(o[E * i + 2 * h], o[E * i + 2 * h + 1]);
        u[h] = *reinterpret_cast<const uint32_t*>(&p);
      }
      if (E == 8) *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
      else *reinterpret_cast<uint2*>(row + c) = make_uint2(u[0], u[1]);
    }
  }
}

// (offset +) w or b of the columns of one slot, or `absent`; zero past C. Held in registers for an
// item: read again for every group of rows they cost as much L2 traffic as the rows.
template <int E>
__device__ __forceinline__ void load_affine(const void* p, bool bf16, long long at, float add, float absent, int t,
                                            int k, int tpr, int C, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = column<E>(t, k, j, tpr);
    float v = absent;
    if (p && c < C)
      v = add + (bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at + c])
                      : static_cast<const float*>(p)[at + c]);
    o[j] = c < C ? v : 0.f;
  }
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
// shared memory while one is at work (VEC). Four groups, fewer where T threads' pieces of them
// are over 200 KB.
template <typename XT, int VPT, int U>
constexpr int kFwdPieces = U* VPT* kPieces<XT>;
template <typename XT, typename YT, int VPT, int U>
constexpr int kBwdPieces = U* VPT*(kPieces<XT> + kPieces<YT>);
constexpr int ring_depth(int pieces, int T) {
  const int d = 204800 / (16 * pieces * T);
  return d < 1 ? 1 : d > 4 ? 4 : d;
}

template <typename XT, typename YT, bool VEC, int VPT, int U, int T, int kPerSm>
__global__ void __launch_bounds__(T, kPerSm) norm_fwd_kernel(NormArgs a) {
  __shared__ float red[2][U * 32];
  extern __shared__ uint4 ring[];         // [kDepth][piece][thread]
  constexpr int E = kRun<XT, YT, VEC>;
  constexpr int P = kPieces<XT>, kDepth = ring_depth(kFwdPieces<XT, VPT, U>, T);
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const int plane = blockDim.x;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  YT* y = static_cast<YT*>(a.y);
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  const long long step = (long long)rpb * U;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per), wat = a.w_items ? item * C : 0;
    float w[VPT][8], b[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      load_affine<E>(a.w, a.w_bf16, wat, a.offset, 1.f, t, k, tpr, C, w[k]);
      load_affine<E>(a.b, a.w_bf16, wat, 0.f, 0.f, t, k, tpr, C, b[k]);
    }
    int put = 0, got = 0;                 // ring stages
    auto request = [&](long long base) {
      if (VEC) {
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
      if constexpr (VEC) {
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
        m[u] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) m[u] += xs[u][k].get(j);
      }
      row_sum<U>(m, tpr, red[0]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        m[u] *= inv_c;
        v[u] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = xs[u][k].get(j) - m[u];
            v[u] += column<E>(t, k, j, tpr) < C ? d * d : 0.f;
          }
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
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = (xs[u][k].get(j) - m[u]) * v[u] * w[k][j] + b[k][j];
          if (r < end) store_slot<E>(y + r * C, t, k, tpr, C, o);
        }
      }
    }
    r0 = end;
  }
}

template <typename XT, typename YT, bool VEC, int VPT, int U, int T, int kPerSm>
__global__ void __launch_bounds__(T, kPerSm) norm_bwd_kernel(NormArgs a) {
  __shared__ float red[2][2 * U * 32];
  extern __shared__ uint4 ring[];         // [kDepth][piece][thread]
  constexpr int E = kRun<XT, YT, VEC>;
  constexpr int PX = kPieces<XT>, PY = kPieces<YT>, kDepth = ring_depth(kBwdPieces<XT, YT, VPT, U>, T);
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const int plane = blockDim.x;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  const YT* dy = static_cast<const YT*>(a.dy);
  XT* dx = static_cast<XT*>(a.y);
  // several rows a block: their column sums [2][C] meet here, behind the ring
  float* acc = reinterpret_cast<float*>(ring + (VEC ? kDepth * kBwdPieces<XT, YT, VPT, U> * plane : 0));
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  const long long step = (long long)rpb * U;
  int flip = 0;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per), wat = a.w_items ? item * C : 0;
    float w[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) load_affine<E>(a.w, a.w_bf16, wat, a.offset, 1.f, t, k, tpr, C, w[k]);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.f;
    int put = 0, got = 0;                 // ring stages
    auto request = [&](long long base) {
      if (VEC) {
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
        m[u] = a.mean[q];
        rs[u] = a.rstd[q];
        s[2 * u] = s[2 * u + 1] = 0.f;
      }
      if constexpr (VEC) {
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
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = base + u * rpb + sub < end;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // past the row's end dy is zero, so none of the sums sees the element
            const float d = gs[u][k].get(j), h = (xs[u][k].get(j) - m[u]) * rs[u], g = d * w[k][j];
            s[2 * u] += g;
            s[2 * u + 1] += g * h;
            dw[k][j] += in ? d * h : 0.f;
            db[k][j] += d;
          }
        }
      }
      row_sum<2 * U>(s, tpr, red[flip]);
      flip ^= 1;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long r = base + u * rpb + sub;
          const float c1 = s[2 * u] * inv_c, c2 = s[2 * u + 1] * inv_c;
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float h = (xs[u][k].get(j) - m[u]) * rs[u];
            o[j] = rs[u] * (gs[u][k].get(j) * w[k][j] - c1 - h * c2);
          }
          if (r < end) store_slot<E>(dx + r * C, t, k, tpr, C, o);
        }
      }
    }
    if (a.part) {
      // this block's partial row of the item: block + item counts up along the blocks' ranges,
      // so no two (block, item) pairs share it
      float* pw = a.part + (blockIdx.x + (a.w_items ? item : 0)) * C;
      float* pb = pw + a.slots * C;
      if (rpb == 1) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = column<E>(t, k, j, tpr);
            if (c < C) pw[c] = dw[k][j], pb[c] = db[k][j];
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
                  acc[c] = g == 0 ? dw[k][j] : acc[c] + dw[k][j];
                  acc[C + c] = g == 0 ? db[k][j] : acc[C + c] + db[k][j];
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
struct NormShape {
  int tpr, vpt, threads;
};
NormShape norm_shape(int C, bool bwd, bool fp32, bool vec) {
  const int slots = ceil_div(C, 8), most = !vec ? 1 : bwd || fp32 ? 2 : 4;
  NormShape n;
  if (slots <= 32 * most) {                         // a warp or less
    n.vpt = slots <= 32 ? 1 : slots <= 64 ? 2 : 4;
    n.tpr = slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
    n.threads = 256;
    return n;
  }
  if (!vec) {                                       // no copies ahead: as many threads as go
    n.vpt = slots <= 640 ? 1 : slots <= 1024 ? 2 : 4;
  } else {                                          // the fewest lanes without work, then the fewest threads
    n.vpt = most == 4 && 128 * ceil_div(slots, 128) <= 64 * ceil_div(slots, 64) ? 4 : 2;
    if (slots > 1024) n.vpt = 4;
  }
  n.threads = n.tpr = 32 * ceil_div(slots, 32 * n.vpt);
  return n;
}

constexpr int kNormSms = 148;     // SMs of the part; the workspace is sized without asking the device

// Rows that a lane group takes together: more make fewer reductions, fewer leave registers.
template <typename XT, bool VEC, int VPT>
constexpr int kFwdU = !VEC ? 1 : VPT == 1 ? 8 / sizeof(XT) : VPT == 2 ? 4 / sizeof(XT) : 1;
template <bool VEC, int VPT>
constexpr int kBwdU = VEC && VPT == 1 ? 2 : 1;

// Blocks an SM that a kernel is built for: registers to hold everything (what does not fit goes
// through L2, since the copies ahead leave L1 little: a backward pass with 216 bytes of it a
// thread took twice as long).
constexpr int per_sm(int vpt, int T) { return T > 256 ? 1 : vpt == 1 ? 3 : 2; }

// Blocks of a launch: enough to fill the device, never more than there are rows for one each of a
// block's lane groups.
int norm_blocks(const NormShape& n, long long rows) {
  const long long step = n.threads / n.tpr, need = (rows + step - 1) / step;
  const int T = n.threads > 256 ? n.threads : 256;
  const long long full = (long long)kNormSms * (per_sm(n.vpt, T) * T / n.threads);
  return (int)(need < full ? need : full);
}

// `most`: the largest shared memory that a launch of this kernel takes (it needs leave above 48 KB,
// static arrays included).
template <auto kKernel>
cudaError_t start(const NormArgs& a, int blocks, int threads, size_t smem, size_t most, cudaStream_t s) {
  if (most > 40 * 1024) {
    static OncePerDevice once;
    const cudaError_t e =
        once([most] { return cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most); });
    if (e != cudaSuccess) return e;
  }
  kKernel<<<blocks, threads, smem, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename XT, typename YT, bool VEC, int VPT, int T>
cudaError_t run_fwd(const NormArgs& a, const NormShape& n, int blocks, cudaStream_t s) {
  constexpr int U = kFwdU<XT, VEC, VPT>, kPieces = kFwdPieces<XT, VPT, U>;
  constexpr size_t kThread = VEC ? 16 * ring_depth(kPieces, T) * kPieces : 0;
  return start<norm_fwd_kernel<XT, YT, VEC, VPT, U, T, per_sm(VPT, T)>>(a, blocks, n.threads, kThread * n.threads,
                                                                        kThread * T, s);
}
template <typename XT, typename YT, bool VEC, int VPT, int T>
cudaError_t run_bwd(const NormArgs& a, const NormShape& n, int blocks, cudaStream_t s) {
  constexpr int U = kBwdU<VEC, VPT>, kPieces = kBwdPieces<XT, YT, VPT, U>;
  constexpr size_t kThread = VEC ? 16 * ring_depth(kPieces, T) * kPieces : 0;
  const size_t acc = n.tpr < n.threads && a.part ? 2 * sizeof(float) * a.C : 0;      // rows of at most 512
  return start<norm_bwd_kernel<XT, YT, VEC, VPT, U, T, per_sm(VPT, T)>>(
      a, blocks, n.threads, kThread * n.threads + acc, kThread * T + 2 * sizeof(float) * 512, s);
}

template <typename XT, typename YT, bool VEC, int VPT, int T>
cudaError_t run_either(const NormArgs& a, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  return bwd ? run_bwd<XT, YT, VEC, VPT, T>(a, n, blocks, s) : run_fwd<XT, YT, VEC, VPT, T>(a, n, blocks, s);
}
template <typename XT, typename YT, bool VEC>
cudaError_t run_norm(const NormArgs& a, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  const bool wide = n.threads > 256;
  if (n.vpt == 1 && wide) return run_either<XT, YT, false, 1, 640>(a, bwd, n, blocks, s);   // rows without wide accesses only
  if (n.vpt == 1) return run_either<XT, YT, VEC, 1, 256>(a, bwd, n, blocks, s);
  if (n.vpt == 2 && wide) return run_either<XT, YT, VEC, 2, 512>(a, bwd, n, blocks, s);
  if (n.vpt == 2) return run_either<XT, YT, VEC, 2, 256>(a, bwd, n, blocks, s);
  if (wide) return run_either<XT, YT, VEC, 4, 512>(a, bwd, n, blocks, s);
  return run_fwd<XT, YT, VEC, 4, 256>(a, n, blocks, s);       // the backward pass has 4 slots only past 256 threads
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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

cudaError_t dispatch(const bsa_norm_shape& f, NormArgs& a, bool bwd, cudaStream_t s, int* blocks_out = nullptr) {
  const bool vec = f.C % 8 == 0 && at16(a.x) && at16(a.y) && at16(a.dy);
  const NormShape n = norm_shape(f.C, bwd, f.x_type == BSA_FP32, vec);
  const int blocks = norm_blocks(n, f.rows);
  a.tpr = n.tpr;
  a.slots = blocks + (a.w_items ? f.items : 1);
  if (blocks_out) *blocks_out = blocks;
  const bool xb = f.x_type == BSA_BF16, yb = f.y_type == BSA_BF16;
  if (xb && yb) return vec ? run_norm<__nv_bfloat16, __nv_bfloat16, true>(a, bwd, n, blocks, s) : run_norm<__nv_bfloat16, __nv_bfloat16, false>(a, bwd, n, blocks, s);
  if (xb) return vec ? run_norm<__nv_bfloat16, float, true>(a, bwd, n, blocks, s) : run_norm<__nv_bfloat16, float, false>(a, bwd, n, blocks, s);
  if (yb) return vec ? run_norm<float, __nv_bfloat16, true>(a, bwd, n, blocks, s) : run_norm<float, __nv_bfloat16, false>(a, bwd, n, blocks, s);
  return vec ? run_norm<float, float, true>(a, bwd, n, blocks, s) : run_norm<float, float, false>(a, bwd, n, blocks, s);
}

}  // namespace

size_t norm_workspace(const bsa_norm_shape& f) {
  int blocks = 0;                 // whatever the addresses allow
  for (const bool vec : {false, true}) {
    const int n = norm_blocks(norm_shape(f.C, true, f.x_type == BSA_FP32, vec), f.rows);
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
