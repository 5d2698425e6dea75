// Root-mean-square norm with the residual's addition and an 8-bit output, and its backward.
//
//   h = x + residual,  rs = (mean h^2 + eps)^-1/2,  v = h rs w;   codes = e4m3(v / s), s = amax|v| / 448
//   backward, g = dy w:  dh = rs (g - h rs^2 mean(g h)) + dresidual,  dw = sum_rows dy h rs
//
// Everything is held in fp32 from the loads to the one rounding of each output (h is normalised
// unrounded, and the 8-bit codes come from the unrounded v).
//
// HBM-bound: a row is read once and kept in registers (as fp32 h) between the sum of squares, the
// maximum of its codes and the writes.  A row belongs to one CTA, or, up to 1024 columns, to one
// warp (no block barrier; eight rows per CTA).  Rows that are not made of aligned 8-element pieces
// take the general kernels: a CTA per row with scalar accesses that reads the row again for each
// pass (from L1 / L2).
#pragma once

#include "elem.cuh"
#include "quantize.cuh"

namespace dsa {

struct NormParams {
  const void* x;
  const void* res;
  const void* w;
  int64_t ld_x, ld_res, ld_y, ld_ro;
  int64_t rows;
  int32_t cols;
  float eps;
  void* y;
  void* res_out;
  uint8_t* codes;
  float* scale;
  int32_t groups;  // scales per row of the grouped form; 0: one scale per row
  float* rstd;
};

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dres;
  int64_t ld_dy, ld_h, ld_dres, ld_dh;
  int64_t rows;
  int32_t cols;
  void* dh;
  float* part;  // [gridDim.x, cols] partial sums of dw
};

namespace norm {

constexpr int kGroup = DSA_QUANT_GROUP;
constexpr int kWarpRows = 8;       // rows per CTA of the warp-per-row kernels
constexpr int kWarpCols = 1024;    // widest row of one warp: 4 pieces of 8 elements per lane
constexpr int kGeneralThreads = 256;

__device__ __forceinline__ float scale_of(float amax) { return amax > 0.f ? __fdiv_rn(amax, quant::kE4m3Max) : 1.f; }

__device__ __forceinline__ uint2 encode8(const float* v, float s) {
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = quant::to_e4m3x2(__fdiv_rn(v[4 * i], s), __fdiv_rn(v[4 * i + 1], s));
    const uint32_t hi = quant::to_e4m3x2(__fdiv_rn(v[4 * i + 2], s), __fdiv_rn(v[4 * i + 3], s));
    out[i] = lo | (hi << 16);
  }
  return make_uint2(out[0], out[1]);
}

// Block-wide sum / maximum; every thread calls it and gets the result.  red holds one float per
// warp; consecutive calls use different arrays, so one barrier each is enough.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
  if constexpr (MAX) {
    v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));  // non-negative: bit order
  } else {
    v = elem::warp_sum(v);
  }
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = lane < nw ? red[lane] : 0.f;
  if constexpr (MAX) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r)));
  else return elem::warp_sum(r);
}

}  // namespace norm

// CH pieces of 8 elements per thread; piece i of thread t covers columns 8 (t + i * threads per row).
template <typename T, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? norm::kWarpRows * 32 : 1024) rmsnorm_kernel(const NormParams p) {
  using elem::Raw8;
  __shared__ float red[2][32];
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = WARP ? 32 : blockDim.x;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * norm::kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.rows) return;
  const int pieces = p.cols >> 3;
  const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + row * p.ld_res : nullptr;
  float h[CH][8];
  float ss = 0.f;
  {
    Raw8<T> a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      a[i].zero();
      b[i].zero();
      if (c < pieces) {
        a[i].load(x + 8 * c);
        if (res != nullptr) b[i].load(res + 8 * c);
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      a[i].get(h[i]);
      if (res != nullptr) {
        float r[8];
        b[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  const T* w = static_cast<const T*>(p.w);
  Raw8<T> wr[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * nt;
    wr[i].zero();
    if (c < pieces) wr[i].load(w + 8 * c);
  }
  ss = WARP ? elem::warp_sum(ss) : norm::block_reduce<false>(ss, red[0]);
  const float rs = __fdiv_rn(1.f, sqrtf(__fdiv_rn(ss, static_cast<float>(p.cols)) + p.eps));
  if (p.rstd != nullptr && t == 0) p.rstd[row] = rs;
  T* ro = p.res_out != nullptr ? static_cast<T*>(p.res_out) + row * p.ld_ro : nullptr;
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + row * p.ld_y : nullptr;
  float amax[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * nt;
    if (ro != nullptr && c < pieces) {
      Raw8<T> o;
      o.set(h[i]);
      o.store(ro + 8 * c);
    }
    float g[8];
    wr[i].get(g);
    amax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * rs * g[j];
      amax[i] = fmaxf(amax[i], fabsf(h[i][j]));  // a NaN never wins fmaxf
    }
    if (y != nullptr && c < pieces) {
      Raw8<T> o;
      o.set(h[i]);
      o.store(y + 8 * c);
    }
  }
  if (p.codes == nullptr) return;
  uint8_t* codes = p.codes + row * p.cols;
  if (p.groups == 0) {
    float m = amax[0];
#pragma unroll
    for (int i = 1; i < CH; ++i) m = fmaxf(m, amax[i]);
    m = WARP ? __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))) : norm::block_reduce<true>(m, red[1]);
    const float s = norm::scale_of(m);
    if (t == 0) p.scale[row] = s;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      if (c < pieces) *reinterpret_cast<uint2*>(codes + 8 * c) = norm::encode8(h[i], s);
    }
  } else {
    // a group of 128 columns is 16 pieces: 16 neighbouring lanes (threads per row are whole warps)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      float m = amax[i];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = norm::scale_of(m);
      if (c < pieces) {
        if ((c & 15) == 0) p.scale[row * p.groups + (c >> 4)] = s;
        *reinterpret_cast<uint2*>(codes + 8 * c) = norm::encode8(h[i], s);
      }
    }
  }
}

// General form: any cols, strides and element alignment.  Outputs are written in the last pass
// over an element only, by the thread that reads it there, so they may be x or residual itself.
template <typename T>
__global__ void __launch_bounds__(norm::kGeneralThreads) rmsnorm_general_kernel(const NormParams p) {
  using elem::from_f32;
  using elem::to_f32;
  __shared__ float red[2][32];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + row * p.ld_res : nullptr;
  const T* w = static_cast<const T*>(p.w);
  T* ro = p.res_out != nullptr ? static_cast<T*>(p.res_out) + row * p.ld_ro : nullptr;
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + row * p.ld_y : nullptr;
  uint8_t* codes = p.codes != nullptr ? p.codes + row * p.cols : nullptr;
  auto h_of = [&](int c) { return res != nullptr ? to_f32(x[c]) + to_f32(res[c]) : to_f32(x[c]); };
  float ss = 0.f;
  for (int c = t; c < p.cols; c += norm::kGeneralThreads) {
    const float h = h_of(c);
    ss = fmaf(h, h, ss);
  }
  ss = norm::block_reduce<false>(ss, red[0]);
  const float rs = __fdiv_rn(1.f, sqrtf(__fdiv_rn(ss, static_cast<float>(p.cols)) + p.eps));
  if (p.rstd != nullptr && t == 0) p.rstd[row] = rs;
  if (codes != nullptr && p.groups > 0) {  // a warp per group: 4 elements per lane
    const int lane = t & 31;
    for (int g = t >> 5; g < p.groups; g += norm::kGeneralThreads / 32) {
      float h[4], v[4], m = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = g * norm::kGroup + lane + 32 * i;
        h[i] = c < p.cols ? h_of(c) : 0.f;
        v[i] = c < p.cols ? h[i] * rs * to_f32(w[c]) : 0.f;
        m = fmaxf(m, fabsf(v[i]));
      }
      const float s = norm::scale_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
      if (lane == 0) p.scale[row * p.groups + g] = s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = g * norm::kGroup + lane + 32 * i;
        if (c >= p.cols) continue;
        if (ro != nullptr) ro[c] = from_f32<T>(h[i]);
        if (y != nullptr) y[c] = from_f32<T>(v[i]);
        codes[c] = static_cast<uint8_t>(quant::to_e4m3x2(__fdiv_rn(v[i], s), 0.f));
      }
    }
    return;
  }
  float s = 1.f;
  if (codes != nullptr) {
    float m = 0.f;
    for (int c = t; c < p.cols; c += norm::kGeneralThreads) m = fmaxf(m, fabsf(h_of(c) * rs * to_f32(w[c])));
    s = norm::scale_of(norm::block_reduce<true>(m, red[1]));
    if (t == 0) p.scale[row] = s;
  }
  for (int c = t; c < p.cols; c += norm::kGeneralThreads) {
    const float h = h_of(c);
    const float v = h * rs * to_f32(w[c]);
    if (ro != nullptr) ro[c] = from_f32<T>(h);
    if (y != nullptr) y[c] = from_f32<T>(v);
    if (codes != nullptr) codes[c] = static_cast<uint8_t>(quant::to_e4m3x2(__fdiv_rn(v, s), 0.f));
  }
}

// Backward: a persistent grid; each row group (a CTA, or each warp of it) keeps its columns' weights
// and its partial sums of dw in registers over all of its rows.
template <typename T, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? norm::kWarpRows * 32 : 512) rmsnorm_backward_kernel(const NormBwdParams p) {
  using elem::Raw8;
  __shared__ float red[2][32];
  __shared__ float4 dwx[WARP ? norm::kWarpRows * 64 : 1];
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = WARP ? 32 : blockDim.x;
  const int pieces = p.cols >> 3;
  const T* dyp = static_cast<const T*>(p.dy);
  const T* hp = static_cast<const T*>(p.h);
  const T* rp = static_cast<const T*>(p.dres);
  float dw[CH][8];
  Raw8<T> w[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * nt;
    w[i].zero();
    if (c < pieces) w[i].load(static_cast<const T*>(p.w) + 8 * c);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (WARP ? norm::kWarpRows : 1);
  int it = 0;
  for (int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * norm::kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
       row < p.rows; row += step, ++it) {
    Raw8<T> a[CH], b[CH], d[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      a[i].zero();
      b[i].zero();
      d[i].zero();
      if (c < pieces) {
        a[i].load(dyp + row * p.ld_dy + 8 * c);
        b[i].load(hp + row * p.ld_h + 8 * c);
        if (rp != nullptr) d[i].load(rp + row * p.ld_dres + 8 * c);
      }
    }
    const float rs = p.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float dy[8], h[8], wf[8];
      a[i].get(dy);
      b[i].get(h);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = dy[j] * h[j];
        dot = fmaf(u, wf[j], dot);
        dw[i][j] = fmaf(u, rs, dw[i][j]);
      }
    }
    dot = WARP ? elem::warp_sum(dot) : norm::block_reduce<false>(dot, red[it & 1]);
    const float k = dot * inv_cols * rs * rs;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      if (c >= pieces) continue;
      float dy[8], h[8], wf[8], r[8], o[8];
      a[i].get(dy);
      b[i].get(h);
      w[i].get(wf);
      d[i].get(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, fmaf(-h[j], k, dy[j] * wf[j]), r[j]);
      Raw8<T> out;
      out.set(o);
      out.store(static_cast<T*>(p.dh) + row * p.ld_dh + 8 * c);
    }
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if constexpr (WARP) {
    // the eight warps' sums, added in warp order
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float4* mine = dwx + (threadIdx.x >> 5) * 64 + 2 * t;
      __syncthreads();
      mine[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      mine[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      __syncthreads();
      const int col = 256 * i + static_cast<int>(threadIdx.x);  // 256 columns per i, one per thread
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < norm::kWarpRows; ++v) s += reinterpret_cast<const float*>(dwx)[v * 256 + threadIdx.x];
      if (col < p.cols) part[col] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * nt;
      if (c >= pieces) continue;
      reinterpret_cast<float4*>(part)[2 * c] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      reinterpret_cast<float4*>(part)[2 * c + 1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// General form (any cols, strides and element alignment): the CTA's row of the workspace holds its
// partial sums of dw; each column is read and written by one thread.
template <typename T>
__global__ void __launch_bounds__(norm::kGeneralThreads) rmsnorm_backward_general_kernel(const NormBwdParams p) {
  using elem::to_f32;
  __shared__ float red[2][32];
  const T* w = static_cast<const T*>(p.w);
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.cols;
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  int it = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.ld_dy;
    const T* h = static_cast<const T*>(p.h) + row * p.ld_h;
    const T* r = p.dres != nullptr ? static_cast<const T*>(p.dres) + row * p.ld_dres : nullptr;
    T* dh = static_cast<T*>(p.dh) + row * p.ld_dh;
    const float rs = p.rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += norm::kGeneralThreads)
      dot = fmaf(to_f32(dy[c]) * to_f32(h[c]), to_f32(w[c]), dot);
    dot = norm::block_reduce<false>(dot, red[it & 1]);
    const float k = dot * inv_cols * rs * rs;
    for (int c = threadIdx.x; c < p.cols; c += norm::kGeneralThreads) {
      const float g = to_f32(dy[c]), hv = to_f32(h[c]);
      const float u = g * hv * rs;
      part[c] = it == 0 ? u : part[c] + u;
      dh[c] = elem::from_f32<T>(fmaf(rs, fmaf(-hv, k, g * to_f32(w[c])), r != nullptr ? to_f32(r[c]) : 0.f));
    }
  }
}

// dw[c] = sum of the n partial rows, in a fixed order: 32 columns per CTA, 8 threads per column.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* __restrict__ part, int n, int cols,
                                                         float* __restrict__ dw) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < cols)
    for (int i = k; i < n; i += 8) acc += part[static_cast<int64_t>(i) * cols + c];
  s[k][lane] = acc;
  __syncthreads();
  if (k == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][lane];
    dw[c] = acc;
  }
}

}  // namespace dsa
