// Root-mean-square norm with the residual's addition and an 8-bit output, and its backward.
//
//   h = x + residual,  rs = (mean h^2 + eps)^-1/2,  v = h rs w;   codes = e4m3(v / s), s = amax|v| / 448
//   backward, g = dy w:  dh = rs (g - h rs^2 mean(g h)) + dresidual,  dw = sum_rows dy h rs
//
// Everything is held in fp32 from the loads to the one rounding of each output (h is normalised
// unrounded, and the 8-bit codes come from the unrounded v).
//
// HBM-bound: a row is read once and kept in registers (as fp32 h) between the sum of squares, the
// maximum of its codes and the writes.  A row belongs to one CTA, or, up to 1024 columns (512 in
// pieces smaller than 8), to one warp or a half or quarter of one (no block barrier).  Rows that are not made of aligned pieces of 8
// elements use the same kernels with pieces of 4, 2 or 1.  Rows too wide for the registers of a CTA take
// the general kernels, which read a row again for each pass (from L1 / L2).
// Measured on the device alone (calls in a captured graph): 32768 x 4096 bf16 with residual, y and codes 180 us
// (6.7 TB/s, 1.02 of measured HBM's copy rate; 200 a call among others, from Python; 193 us with a division per code, 185 with
// 2 pieces per thread); 65536 x 128 bf16 9.3 us on one set of buffers (half a warp per row; a warp, half of it idle: 14.9).
#pragma once

#include "elem.cuh"
#include "e4m3.cuh"
#include "ring.cuh"

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
constexpr int kWarps = 8;          // warps per CTA where a row is part of a warp's work
constexpr int kGeneralThreads = 256;
constexpr int kRingMax = 8;        // stages of the backward's ring
constexpr int kRingBytes = 200 * 1024;  // shared memory for the rings of an SM's CTAs

// Writes the codes of V values, at a multiple of V bytes.
template <int V>
__device__ __forceinline__ void encode(uint8_t* dst, const float* v, float s) {
  const float inv = quant::inverse_of(s);
  auto q = [&](int i) { return quant::over(v[i], s, inv); };
  if constexpr (V == 1) {
    *dst = static_cast<uint8_t>(quant::to_e4m3x2(q(0), 0.f));
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint16_t*>(dst) = quant::to_e4m3x2(q(0), q(1));
  } else {
    uint32_t out[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint32_t lo = quant::to_e4m3x2(q(4 * i), q(4 * i + 1));
      const uint32_t hi = quant::to_e4m3x2(q(4 * i + 2), q(4 * i + 3));
      out[i] = lo | (hi << 16);
    }
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(dst) = out[0];
    else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  }
}

// First column of piece i of thread t of a row's nt threads.  Pieces of 8: the row's piece t + i nt;
// smaller ones: a warp has 32 CH V consecutive columns, 32 V to a piece index, so that the 128 columns
// of a group belong to one warp.
template <int V, int CH>
__device__ __forceinline__ int column(int t, int nt, int i) {
  return V == 8 ? 8 * (t + i * nt) : (t >> 5) * (32 * V * CH) + 32 * V * i + V * (t & 31);
}

// Sum / maximum over the LANES lanes of a row (LANES = 8, 16 or 32 neighbours).
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {  // of non-negative values
  if constexpr (LANES == 32) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

// CH pieces of V elements per thread; a row belongs to LANES lanes of a warp (8, 16 or 32), or to the
// CTA (LANES = 0).
template <typename T, int V, int CH, int LANES>
__global__ void __launch_bounds__(LANES > 0 ? norm::kWarps * 32 : 1024) rmsnorm_kernel(const NormParams p) {
  using elem::Piece;
  constexpr bool kCta = LANES == 0;
  constexpr int kLanes = kCta ? 32 : LANES;
  __shared__ float red[2][32];
  const int t = kCta ? threadIdx.x : threadIdx.x % kLanes;
  const int nt = kCta ? blockDim.x : kLanes;
  const int64_t row = kCta ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (norm::kWarps * 32 / kLanes) + threadIdx.x / kLanes;
  const bool live = kCta || row < p.rows;
  auto col = [&](int i) { return norm::column<V, CH>(t, nt, i); };
  auto has = [&](int i) { return live && col(i) < p.cols; };
  const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + row * p.ld_res : nullptr;
  float h[CH][V];
  float ss = 0.f;
  {
    Piece<T, V> a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      a[i].zero();
      b[i].zero();
      if (has(i)) {
        a[i].load(x + col(i));
        if (res != nullptr) b[i].load(res + col(i));
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      a[i].get(h[i]);
      if (res != nullptr) {
        float r[V];
        b[i].get(r);
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  const T* w = static_cast<const T*>(p.w);
  Piece<T, V> wr[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    wr[i].zero();
    if (col(i) < p.cols) wr[i].load(w + col(i));
  }
  ss = kCta ? norm::block_reduce<false>(ss, red[0]) : norm::lanes_sum<kLanes>(ss);
  const float rs = __fdiv_rn(1.f, sqrtf(__fdiv_rn(ss, static_cast<float>(p.cols)) + p.eps));
  if (p.rstd != nullptr && t == 0 && live) p.rstd[row] = rs;
  T* ro = p.res_out != nullptr ? static_cast<T*>(p.res_out) + row * p.ld_ro : nullptr;
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + row * p.ld_y : nullptr;
  float amax[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (ro != nullptr && has(i)) {
      Piece<T, V> o;
      o.set(h[i]);
      o.store(ro + col(i));
    }
    float g[V];
    wr[i].get(g);
    amax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[i][j] = h[i][j] * rs * g[j];
      amax[i] = fmaxf(amax[i], fabsf(h[i][j]));  // a NaN never wins fmaxf
    }
    if (y != nullptr && has(i)) {
      Piece<T, V> o;
      o.set(h[i]);
      o.store(y + col(i));
    }
  }
  if (p.codes == nullptr) return;
  uint8_t* codes = p.codes + row * p.cols;
  if (p.groups == 0) {
    float m = amax[0];
#pragma unroll
    for (int i = 1; i < CH; ++i) m = fmaxf(m, amax[i]);
    m = kCta ? norm::block_reduce<true>(m, red[1]) : norm::lanes_max<kLanes>(m);
    const float s = quant::scale_of(m);
    if (t == 0 && live) p.scale[row] = s;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (has(i)) norm::encode<V>(codes + col(i), h[i], s);
  } else {
    // a group of 128 columns: 16 neighbouring lanes of one piece index (V = 8), or all lanes of kPer of them
    constexpr int kPer = V >= 4 ? 1 : 4 / V;
    static_assert(CH % kPer == 0, "groups do not cross threads' ranges");
#pragma unroll
    for (int i = 0; i < CH; i += kPer) {
      float m = amax[i];
#pragma unroll
      for (int j = i + 1; j < i + kPer; ++j) m = fmaxf(m, amax[j]);
      const float s = quant::scale_of(norm::lanes_max<V == 8 ? (kLanes < 16 ? kLanes : 16) : 32>(m));
      if (has(i) && col(i) % norm::kGroup == 0) p.scale[row * p.groups + col(i) / norm::kGroup] = s;
#pragma unroll
      for (int j = i; j < i + kPer; ++j)
        if (has(j)) norm::encode<V>(codes + col(j), h[j], s);
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
      const float s = quant::scale_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
      if (lane == 0) p.scale[row * p.groups + g] = s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = g * norm::kGroup + lane + 32 * i;
        if (c >= p.cols) continue;
        if (ro != nullptr) ro[c] = from_f32<T>(h[i]);
        if (y != nullptr) y[c] = from_f32<T>(v[i]);
        norm::encode<1>(codes + c, &v[i], s);
      }
    }
    return;
  }
  float s = 1.f;
  if (codes != nullptr) {
    float m = 0.f;
    for (int c = t; c < p.cols; c += norm::kGeneralThreads) m = fmaxf(m, fabsf(h_of(c) * rs * to_f32(w[c])));
    s = quant::scale_of(norm::block_reduce<true>(m, red[1]));
    if (t == 0) p.scale[row] = s;
  }
  for (int c = t; c < p.cols; c += norm::kGeneralThreads) {
    const float h = h_of(c);
    const float v = h * rs * to_f32(w[c]);
    if (ro != nullptr) ro[c] = from_f32<T>(h);
    if (y != nullptr) y[c] = from_f32<T>(v);
    if (codes != nullptr) norm::encode<1>(codes + c, &v, s);
  }
}

// Backward: a persistent grid; each row group (a CTA, or LANES lanes of a warp) keeps its columns'
// weights and its partial sums of dw in registers over all of its rows, and issues a row's loads before
// it reduces and writes the row before.
template <typename T, int V, int CH, int LANES>
__global__ void __launch_bounds__(LANES > 0 ? norm::kWarps * 32 : 1024) rmsnorm_backward_kernel(const NormBwdParams p) {
  using elem::Piece;
  constexpr bool kCta = LANES == 0;
  constexpr int kLanes = kCta ? 32 : LANES;
  __shared__ float red[2][32];
  __shared__ float dwx[kCta ? 1 : norm::kWarps * 256];
  const int t = kCta ? threadIdx.x : threadIdx.x % kLanes;
  const int nt = kCta ? blockDim.x : kLanes;
  auto col = [&](int i) { return norm::column<V, CH>(t, nt, i); };
  const T* dyp = static_cast<const T*>(p.dy);
  const T* hp = static_cast<const T*>(p.h);
  const T* rp = static_cast<const T*>(p.dres);
  float dw[CH][V];
  Piece<T, V> w[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    w[i].zero();
    if (col(i) < p.cols) w[i].load(static_cast<const T*>(p.w) + col(i));
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  }
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  constexpr int kRows = kCta ? 1 : norm::kWarps * 32 / kLanes;  // of a CTA
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  Piece<T, V> a[CH], b[CH], d[CH];
  float rs = 0.f;
  auto load_row = [&](int64_t row, Piece<T, V>* pa, Piece<T, V>* pb, Piece<T, V>* pd, float& r) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      pa[i].zero();
      pb[i].zero();
      pd[i].zero();
      if (row < p.rows && col(i) < p.cols) {
        pa[i].load(dyp + row * p.ld_dy + col(i));
        pb[i].load(hp + row * p.ld_h + col(i));
        if (rp != nullptr) pd[i].load(rp + row * p.ld_dres + col(i));
      }
    }
    if (row < p.rows) r = p.rstd[row];
  };
  int it = 0;
  // base: the first row of the CTA's step, the same for all lanes of a warp
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const int mine = kCta ? 0 : threadIdx.x / kLanes;
  load_row(base + mine, a, b, d, rs);
  for (; base < p.rows; base += step, ++it) {
    const int64_t row = base + mine;
    Piece<T, V> na[CH], nb[CH], nd[CH];
    float nrs = 0.f;
    load_row(row + step, na, nb, nd, nrs);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float dy[V], h[V], wf[V];
      a[i].get(dy);
      b[i].get(h);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float u = dy[j] * h[j];
        dot = fmaf(u, wf[j], dot);
        dw[i][j] = fmaf(u, rs, dw[i][j]);
      }
    }
    dot = kCta ? norm::block_reduce<false>(dot, red[it & 1]) : norm::lanes_sum<kLanes>(dot);
    const float k = dot * inv_cols * rs * rs;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (row < p.rows && col(i) < p.cols) {
        float dy[V], h[V], wf[V], r[V], o[V];
        a[i].get(dy);
        b[i].get(h);
        w[i].get(wf);
        d[i].get(r);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = fmaf(rs, fmaf(-h[j], k, dy[j] * wf[j]), r[j]);
        Piece<T, V> out;
        out.set(o);
        out.store(static_cast<T*>(p.dh) + row * p.ld_dh + col(i));
      }
      a[i] = na[i];
      b[i] = nb[i];
      d[i] = nd[i];
    }
    rs = nrs;
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if constexpr (!kCta) {
    // the warp's row groups, then the eight warps in their order, 256 columns at a time
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) dw[i][j] += __shfl_xor_sync(0xffffffffu, dw[i][j], o);
    constexpr int kStep = 256 / (32 * V) < 1 ? 1 : 256 / (32 * V);  // piece indexes that make 256 columns
#pragma unroll
    for (int i0 = 0; i0 < CH; i0 += kStep) {
      __syncthreads();
      if ((threadIdx.x & 31) < kLanes) {
#pragma unroll
        for (int i = i0; i < i0 + kStep && i < CH; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) dwx[(threadIdx.x >> 5) * 256 + (col(i) + j) % 256] = dw[i][j];
      }
      __syncthreads();
      const int c = 32 * V * i0 + static_cast<int>(threadIdx.x);
      if (c < p.cols && c < kLanes * V * CH) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < norm::kWarps; ++v) s += dwx[v * 256 + threadIdx.x];
        part[c] = s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (col(i) < p.cols) {
#pragma unroll
        for (int j = 0; j < V; ++j) part[col(i) + j] = dw[i][j];
      }
  }
}

// Backward for CTA-wide rows of whole 8-element pieces: one piece per thread, and the rows (dy, h and
// the residual's gradient) come through a ring of shared-memory stages filled by bulk copies, several
// rows ahead, so that the bytes in flight do not depend on registers or on the reduction's barrier.
// Measured on the device alone, 16384 x 5120 bf16 with the residual's gradient: 129 us with one row ahead in
// registers (above), 109.9 us with the ring (6.1 TB/s, 0.93 of measured HBM; 120 a call among others, from Python); 128 us while
// rstd was not read a row ahead too.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_backward_ring_kernel(const NormBwdParams p, int stages) {
  using elem::Raw8;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][32];
  __shared__ uint64_t full[norm::kRingMax];
  const int t = threadIdx.x, c = 8 * t;
  const bool in = c < p.cols;
  const uint32_t row_bytes = static_cast<uint32_t>(p.cols) * sizeof(T);
  const int parts = p.dres != nullptr ? 3 : 2;
  const uint32_t stage_bytes = parts * row_bytes;
  const T* dyp = static_cast<const T*>(p.dy);
  const T* hp = static_cast<const T*>(p.h);
  const T* rp = static_cast<const T*>(p.dres);
  auto issue = [&](int64_t row, int s) {
    uint8_t* dst = ring + s * stage_bytes;
    dev::mbar_arrive_expect_tx(&full[s], stage_bytes);
    elem::bulk_load(dst, dyp + row * p.ld_dy, row_bytes, &full[s]);
    elem::bulk_load(dst + row_bytes, hp + row * p.ld_h, row_bytes, &full[s]);
    if (rp != nullptr) elem::bulk_load(dst + 2 * row_bytes, rp + row * p.ld_dres, row_bytes, &full[s]);
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) dev::mbar_init(&full[s], 1);
    dev::fence_mbar_init();
    dev::fence_proxy_async_smem();
    for (int s = 0; s < stages; ++s) {
      const int64_t row = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (row < p.rows) issue(row, s);
    }
  }
  float dw[8], wf[8];
  {
    Raw8<T> w;
    w.zero();
    if (in) w.load(static_cast<const T*>(p.w) + c);
    w.get(wf);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  __syncthreads();
  bool ok = true;  // a copy that does not land within the limit is reported, and not waited for again
  int landed = 0;  // rows whose copies this thread has seen land
  int s = 0;
  uint32_t phase = 0;
  int it = 0;
  float next_rs = p.rstd[blockIdx.x];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    const float rs = next_rs;
    if (row + gridDim.x < p.rows) next_rs = p.rstd[row + gridDim.x];
    if (ok) ok = dev::mbar_wait(&full[s], phase);
    if (ok) ++landed;
    const uint8_t* src = ring + s * stage_bytes;
    Raw8<T> a, b, d;
    a.zero();
    b.zero();
    d.zero();
    if (in) {
      a.load(reinterpret_cast<const T*>(src) + c);
      b.load(reinterpret_cast<const T*>(src + row_bytes) + c);
      if (parts == 3) d.load(reinterpret_cast<const T*>(src + 2 * row_bytes) + c);
    }
    float dy[8], h[8];
    a.get(dy);
    b.get(h);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = dy[j] * h[j];
      dot = fmaf(u, wf[j], dot);
      dw[j] = fmaf(u, rs, dw[j]);
    }
    dot = norm::block_reduce<false>(dot, red[it & 1]);
    // every thread has read the stage (the barrier of the reduction): refill it
    if (t == 0 && ok) {
      const int64_t next = row + static_cast<int64_t>(stages) * gridDim.x;
      if (next < p.rows) issue(next, s);
    }
    const float k = dot * inv_cols * rs * rs;
    if (in) {
      float r[8], o[8];
      d.get(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, fmaf(-h[j], k, dy[j] * wf[j]), r[j]);
      Raw8<T> out;
      out.set(o);
      out.store(static_cast<T*>(p.dh) + row * p.ld_dh + c);
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {
    record_device_error(DSA_ERR_TIMEOUT);
    // copies still in flight must not outlive the CTA's shared memory.  Thread 0 issues them, and issues none
    // once its own wait has run out; when only another thread's has, it has seen them all land.
    if (t == 0) {
      const int copies = static_cast<int>((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);  // the CTA's rows
      for (int n = landed; n < ring_end(landed, stages, copies); ++n)
        dev::mbar_wait(&full[ring_stage(n, stages)], ring_parity(n, stages));
    }
  }
  if (in) {
    float4* part = reinterpret_cast<float4*>(p.part + static_cast<int64_t>(blockIdx.x) * p.cols + c);
    part[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
    part[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
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

// dw[c] = sum of the n partial rows, in a fixed order: 32 columns per CTA, 32 threads per column.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* __restrict__ part, int n, int cols,
                                                          float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < cols)
    for (int i = k; i < n; i += 32) acc += part[static_cast<int64_t>(i) * cols + c];
  s[k][lane] = acc;
  __syncthreads();
  const float sum = elem::warp_sum(s[lane][k]);  // warp k: column k of the CTA
  if (lane == 0 && blockIdx.x * 32 + k < cols) dw[blockIdx.x * 32 + k] = sum;
}

}  // namespace dsa
