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
// block of its own (1 slot a thread to C = 5120, then 2 and 4). U rows a block are read before
// the first is reduced, to keep enough bytes in flight. Rows whose width or address does not
// allow 16-byte loads take the same kernels with single-element, coalesced loads.
// The grid is persistent: each block takes one contiguous range of rows, keeps w and b of the
// item in registers, and in the backward pass the column sums of the rows it has seen. It
// writes them as one partial row for each item that its range meets; a second kernel adds
// the partials of an item in the order of the blocks. No atomics: repeated calls give
// identical bits.
#include "common.cuh"

namespace bsa {
namespace {

constexpr int kMaxVpt = 4;

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

// Column of element j of slot k of thread t: 8 neighbours a thread with 16-byte loads, else
// neighbouring threads on neighbouring elements.
template <bool VEC>
__device__ __forceinline__ int column(int t, int k, int j, int tpr) {
  return VEC ? (t + k * tpr) * 8 + j : t + (k * 8 + j) * tpr;
}

// Eight elements of a row, as loaded.
template <typename T, bool VEC>
struct Slot {
  T v[8];
  __device__ __forceinline__ void load(const T* row, int t, int k, int tpr, int C, bool ok) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<VEC>(t, k, j, tpr);
      v[j] = (ok && c < C) ? row[c] : T(0.f);
    }
  }
  __device__ __forceinline__ float get(int j) const { return to_f(v[j]); }
};
template <>
struct Slot<__nv_bfloat16, true> {
  uint32_t v[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int t, int k, int tpr, int C, bool ok) {
    const int c = column<true>(t, k, 0, tpr);
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (ok && c < C) u = *reinterpret_cast<const uint4*>(row + c);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float((j & 1) ? (v[j >> 1] & 0xffff0000u) : (v[j >> 1] << 16));
  }
};
template <>
struct Slot<float, true> {
  float v[8];
  __device__ __forceinline__ void load(const float* row, int t, int k, int tpr, int C, bool ok) {
    const int c = column<true>(t, k, 0, tpr);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (ok && c < C) {
      a = *reinterpret_cast<const float4*>(row + c);
      b = *reinterpret_cast<const float4*>(row + c + 4);
    }
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_slot(T* row, int t, int k, int tpr, int C, const float (&o)[8]) {
  if (VEC) {
    const int c = column<true>(t, k, 0, tpr);
    if (c >= C) return;
    if (sizeof(T) == 2) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
      *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float4* d = reinterpret_cast<float4*>(row + c);
      d[0] = make_float4(o[0], o[1], o[2], o[3]);
      d[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(t, k, j, tpr);
      if (c < C) put(row + c, o[j]);
    }
  }
}

// (offset +) w or b of this thread's columns, zero past C.
template <bool VEC, int VPT>
__device__ __forceinline__ void load_affine(const void* p, bool bf16, long long at, float add, float absent, int t,
                                            int tpr, int C, float (&o)[VPT][8]) {
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<VEC>(t, k, j, tpr);
      float v = absent;
      if (p && c < C)
        v = add + (bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at + c])
                        : static_cast<const float*>(p)[at + c]);
      o[k][j] = c < C ? v : 0.f;
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

template <typename XT, typename YT, bool VEC, int VPT, int U, int T>
__global__ void __launch_bounds__(T) norm_fwd_kernel(NormArgs a) {
  __shared__ float red[2][U * 32];
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  YT* y = static_cast<YT*>(a.y);
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per);
    float w[VPT][8], b[VPT][8];
    load_affine<VEC, VPT>(a.w, a.w_bf16, a.w_items ? item * C : 0, a.offset, 1.f, t, tpr, C, w);
    load_affine<VEC, VPT>(a.b, a.w_bf16, a.w_items ? item * C : 0, 0.f, 0.f, t, tpr, C, b);
    for (long long base = r0; base < end; base += (long long)rpb * U) {
      Slot<XT, VEC> xs[U][VPT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub;
#pragma unroll
        for (int k = 0; k < VPT; ++k) xs[u][k].load(x + (r < end ? r : base) * C, t, k, tpr, C, r < end);
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
            v[u] += column<VEC>(t, k, j, tpr) < C ? d * d : 0.f;
          }
      }
      row_sum<U>(v, tpr, red[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub;
        if (r >= end) continue;
        const float rs = 1.0f / sqrtf(v[u] * inv_c + a.eps);
        if (t == 0) {
          if (a.mean) a.mean[r] = m[u];
          if (a.rstd) a.rstd[r] = rs;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = (xs[u][k].get(j) - m[u]) * rs * w[k][j] + b[k][j];
          store_slot<VEC>(y + r * C, t, k, tpr, C, o);
        }
      }
    }
    r0 = end;
  }
}

template <typename XT, typename YT, bool VEC, int VPT, int U, int T>
__global__ void __launch_bounds__(T) norm_bwd_kernel(NormArgs a) {
  __shared__ float red[2][2 * U * 32];
  extern __shared__ float acc[];          // several rows a block: their column sums, [2][C]
  const int tpr = a.tpr, t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr, C = a.C;
  const float inv_c = 1.0f / (float)C;
  const XT* x = static_cast<const XT*>(a.x);
  const YT* dy = static_cast<const YT*>(a.dy);
  XT* dx = static_cast<XT*>(a.y);
  const long long lo = a.rows * blockIdx.x / gridDim.x, hi = a.rows * (blockIdx.x + 1) / gridDim.x;
  int flip = 0;
  for (long long r0 = lo; r0 < hi;) {
    const long long item = r0 / a.per, end = min(hi, (item + 1) * a.per);
    float w[VPT][8], dw[VPT][8], db[VPT][8];
    load_affine<VEC, VPT>(a.w, a.w_bf16, a.w_items ? item * C : 0, a.offset, 1.f, t, tpr, C, w);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.f;
    for (long long base = r0; base < end; base += (long long)rpb * U) {
      Slot<XT, VEC> xs[U][VPT];
      Slot<YT, VEC> gs[U][VPT];
      float m[U], rs[U], s[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub, q = r < end ? r : base;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          xs[u][k].load(x + q * C, t, k, tpr, C, r < end);
          gs[u][k].load(dy + q * C, t, k, tpr, C, r < end);
        }
        m[u] = a.mean[q];
        rs[u] = a.rstd[q];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[2 * u] = s[2 * u + 1] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // past the row's end dy is zero, so none of the sums sees the element
            const float d = gs[u][k].get(j), h = (xs[u][k].get(j) - m[u]) * rs[u], g = d * w[k][j];
            s[2 * u] += g;
            s[2 * u + 1] += g * h;
            const bool in = base + u * rpb + sub < end;
            dw[k][j] += in ? d * h : 0.f;
            db[k][j] += d;
          }
      }
      row_sum<2 * U>(s, tpr, red[flip]);
      flip ^= 1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = base + u * rpb + sub;
        if (r >= end) continue;
        const float c1 = s[2 * u] * inv_c, c2 = s[2 * u + 1] * inv_c;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float h = (xs[u][k].get(j) - m[u]) * rs[u];
            o[j] = rs[u] * (gs[u][k].get(j) * w[k][j] - c1 - h * c2);
          }
          store_slot<VEC>(dx + r * C, t, k, tpr, C, o);
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
            const int c = column<VEC>(t, k, j, tpr);
            if (c < C) pw[c] = dw[k][j], pb[c] = db[k][j];
          }
      } else {
        for (int g = 0; g < rpb; ++g) {     // the rows' sums one after the other, in a fixed order
          if (sub == g)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int c = column<VEC>(t, k, j, tpr);
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

// Threads of a row, slots a thread and threads of a block for a row of C elements.
struct NormShape {
  int tpr, vpt, threads;
};
NormShape norm_shape(int C) {
  const int slots = ceil_div(C, 8);
  NormShape n;
  n.vpt = 1;
  if (slots <= 32) {
    n.tpr = slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
    n.threads = 256;
    return n;
  }
  n.vpt = slots <= 640 ? 1 : slots <= 1280 ? 2 : 4;
  n.threads = n.tpr = 32 * ceil_div(slots, 32 * n.vpt);
  return n;
}

constexpr int kNormU = 2;
constexpr int kNormSms = 148;     // SMs of the part; the workspace is sized without asking the device

// Blocks of a launch: enough to fill the device, never more than the rows give.
int norm_blocks(const NormShape& n, long long rows) {
  const long long step = (long long)(n.threads / n.tpr) * kNormU;
  const long long need = (rows + step - 1) / step;
  const long long full = (long long)kNormSms * (1280 / n.threads > 1 ? 1280 / n.threads : 1);
  return (int)(need < full ? need : full);
}

template <typename XT, typename YT, bool VEC, int VPT, int T>
cudaError_t run_norm(const NormArgs& a, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  if (bwd) {
    const size_t acc = n.tpr < n.threads && a.part ? 2 * sizeof(float) * a.C : 0;
    norm_bwd_kernel<XT, YT, VEC, VPT, kNormU, T><<<blocks, n.threads, acc, s>>>(a);
  } else {
    norm_fwd_kernel<XT, YT, VEC, VPT, kNormU, T><<<blocks, n.threads, 0, s>>>(a);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename XT, typename YT>
cudaError_t run_norm_v(const NormArgs& a, bool vec, bool bwd, const NormShape& n, int blocks, cudaStream_t s) {
  if (n.vpt == 1)
    return vec ? run_norm<XT, YT, true, 1, 640>(a, bwd, n, blocks, s) : run_norm<XT, YT, false, 1, 640>(a, bwd, n, blocks, s);
  if (n.vpt == 2)
    return vec ? run_norm<XT, YT, true, 2, 640>(a, bwd, n, blocks, s) : run_norm<XT, YT, false, 2, 640>(a, bwd, n, blocks, s);
  return vec ? run_norm<XT, YT, true, 4, 512>(a, bwd, n, blocks, s) : run_norm<XT, YT, false, 4, 512>(a, bwd, n, blocks, s);
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
  const NormShape n = norm_shape(f.C);
  const int blocks = norm_blocks(n, f.rows);
  a.tpr = n.tpr;
  a.slots = blocks + (a.w_items ? f.items : 1);
  if (blocks_out) *blocks_out = blocks;
  const bool vec = f.C % 8 == 0 && at16(a.x) && at16(a.y) && at16(a.dy);
  const bool xb = f.x_type == BSA_BF16, yb = f.y_type == BSA_BF16;
  if (xb && yb) return run_norm_v<__nv_bfloat16, __nv_bfloat16>(a, vec, bwd, n, blocks, s);
  if (xb) return run_norm_v<__nv_bfloat16, float>(a, vec, bwd, n, blocks, s);
  if (yb) return run_norm_v<float, __nv_bfloat16>(a, vec, bwd, n, blocks, s);
  return run_norm_v<float, float>(a, vec, bwd, n, blocks, s);
}

}  // namespace

size_t norm_workspace(const bsa_norm_shape& f) {
  const long long slots = norm_blocks(norm_shape(f.C), f.rows) + (f.w_per_item ? f.items : 1);
  return align256((size_t)slots * f.C * 2 * sizeof(float));
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
