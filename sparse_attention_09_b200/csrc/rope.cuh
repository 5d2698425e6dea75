// Rotary positions on a range of each head's dims.
//
//   angle = position * freq_i;  (a, b) -> (a c - b s, a s + b c),  c = mscale cos, s = mscale sin
//   (transposed, the backward pass: s with the opposite sign)
//
// At position 10^6 an fp32 angle is off by up to 0.03 rad, so the angle is formed in fp64, as turns
// (position * freq / 2 pi); its fraction of a turn, in [-1/2, 1/2], is exact enough in fp32 (2^-26
// turns).  The sine and cosine of that fraction: sincospif for fp32 tensors (about 2^-23); for 16-bit
// ones the hardware's approximation (2^-21 absolute on [-pi, pi], far below the 2^-9 or 2^-12 of
// the output's rounding), 5 instructions instead of about 45.
//
// HBM-bound: x is read and out written once.  A CTA takes one row, a few rows, or a range of one
// row's heads.  Its threads form groups of one thread per piece of a head (8 elements: 16 or 32
// bytes; fewer where the pointers, strides or the rotated range do not allow that), so
// a thread's piece, and its place in the cos / sin table, stay the same for all the (row, head)
// pairs that its group walks through.  The loads of the first batch are issued before the table of
// the CTA's rows is made (it serves every head of a row).
// Measured on the device alone: 16384 x 64 heads x 128 bf16, half layout, 94.2 us (5.7 TB/s, 0.87 of measured HBM; 100 a
// call among others, from Python; 122 us with items dealt out singly and sincospif); 6001 x 64 x 128 fp32 62.9 us (0.95);
// 12000 x 64 x 128 bf16 with 6 rotated dims 85 to 89 us (0.68 to 0.71; 354 us by pairs and single elements alone).
#pragma once

#include "elem.cuh"

namespace dsa {

struct RopeParams {
  const void* x;
  void* out;
  int64_t xr, xh, orow, oh;  // row and head strides, elements
  int64_t rows;
  int32_t heads, dim, rot0, rot;
  int32_t half_layout;
  const int32_t* pos;
  const double* freqs;
  float mscale;
  int32_t transpose;
  int32_t copy_rest;      // out != x: the dims outside the range are copied
  int32_t rows_per_cta;   // > 1 only when a CTA has all heads of its rows
  int32_t heads_per_cta;
  int32_t items;          // pieces of a head that are moved; the first ones are the rotated ones
  int32_t lanes;          // threads of a group
  int32_t groups;         // groups of a CTA
};

namespace rope {

constexpr int kThreads = 256;  // most threads of a CTA
constexpr int kMaxPairs = 512;
constexpr int kTable = 1024;   // cos / sin entries of a CTA's rows

// (row, head) pairs whose loads a group issues together: 64 bytes per thread in flight (128 for pairs of
// pieces, where three CTAs per SM with room for them in registers measured 94.2 us on the case
// above, four 97.5; two pairs at a time and more CTAs 106 to 112).
template <typename T>
constexpr int unroll() { return sizeof(T) == 2 ? 4 : 2; }

// (mscale cos, mscale sin) of position * freq; s negated for the transposed rotation.
template <bool PRECISE>
__device__ __forceinline__ float2 cos_sin(int pos, double freq, float mscale, bool transpose) {
  const double turns = static_cast<double>(pos) * (freq * 0.15915494309189535);
  const float f = static_cast<float>(turns - rint(turns));
  float s, c;
  if constexpr (PRECISE) sincospif(2.f * f, &s, &c);
  else __sincosf(6.2831853f * f, &s, &c);
  return make_float2(mscale * c, transpose ? -mscale * s : mscale * s);
}

// One rounding order, so that every form of the kernel gives the same bits.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float u = fmaf(a, c, -__fmul_rn(b, s));
  b = fmaf(b, c, __fmul_rn(a, s));
  a = u;
}

}  // namespace rope

// The rotated range (in the half layout each of its halves) is made of whole pieces of V: a rotated item is
// a piece, or two of them half of the range apart (HALF); the others are copied.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(rope::kThreads, HALF && sizeof(T) == 2 ? 3 : 4) rope_kernel(const RopeParams p) {
  using elem::Piece;
  constexpr int kU = rope::unroll<T>();
  constexpr int kLog = V == 8 ? 3 : 2;
  __shared__ __align__(16) float2 table[rope::kTable];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.rows - row0));
  const int head0 = blockIdx.y * p.heads_per_cta;
  const int nheads = min(p.heads_per_cta, p.heads - head0);
  const int pairs = p.rot >> 1, units = nrows * nheads;
  const int rot_items = p.rot >> (HALF ? kLog + 1 : kLog);
  const int g = threadIdx.x / p.lanes, k0 = threadIdx.x - g * p.lanes;
  const T* x = static_cast<const T*>(p.x) + row0 * p.xr + head0 * p.xh;
  T* out = static_cast<T*>(p.out) + row0 * p.orow + head0 * p.oh;
  Piece<T, V> a[kU], b[kU];
  int d = 0, second = 0, cs = 0;  // of item k: its first dim, the distance to its second piece, its table entry
  bool rot = false;
  auto item = [&](int k) {
    rot = k < rot_items;
    if (rot) {
      d = p.rot0 + (k << kLog);
      second = pairs;
      cs = k << (HALF ? kLog : kLog - 1);
    } else {
      d = (k - rot_items) << kLog;
      if (d >= p.rot0) d += p.rot;  // the copied pieces skip the rotated range
    }
  };
  auto row_of = [&](int u) { return nrows == 1 ? 0 : u / nheads; };
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = u0 + i * p.groups;
      if (u >= units) break;
      const int r = row_of(u);
      const T* src = x + r * p.xr + (u - r * nheads) * p.xh + d;
      a[i].load(src);
      if (HALF && rot) b[i].load(src + second);
    }
  };
  const bool first = g < p.groups && k0 < p.items;
  if (first) {
    item(k0);
    load(g);
  }
  for (int i = threadIdx.x; i < nrows * pairs; i += blockDim.x) {
    const int r = i / pairs;
    table[i] = rope::cos_sin<sizeof(T) == 4>(p.pos[row0 + r], p.freqs[i - r * pairs], p.mscale, p.transpose != 0);
  }
  __syncthreads();
  if (!first) return;
  for (int k = k0; k < p.items; k += p.lanes) {
    if (k != k0) item(k);
    for (int u0 = g; u0 < units; u0 += kU * p.groups) {
      if (k != k0 || u0 != g) load(u0);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = u0 + i * p.groups;
        if (u >= units) break;
        const int r = row_of(u);
        T* dst = out + r * p.orow + (u - r * nheads) * p.oh + d;
        if (rot) {
          const float2* t = table + r * pairs + cs;
          float f[V];
          a[i].get(f);
          if constexpr (HALF) {
            float h[V];
            b[i].get(h);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
              const float4 q = *reinterpret_cast<const float4*>(t + j);
              rope::turn(f[j], h[j], q.x, q.y);
              rope::turn(f[j + 1], h[j + 1], q.z, q.w);
            }
            b[i].set(h);
          } else {
#pragma unroll
            for (int j = 0; j < V / 2; j += 2) {
              const float4 q = *reinterpret_cast<const float4*>(t + j);
              rope::turn(f[2 * j], f[2 * j + 1], q.x, q.y);
              rope::turn(f[2 * j + 2], f[2 * j + 3], q.z, q.w);
            }
          }
          if constexpr (HALF) b[i].store(dst + second);
          a[i].set(f);
        }
        a[i].store(dst);
      }
    }
  }
}

// Any rotated range: an item is a pair of elements of the range (items 0 .. rot/2 - 1 of a head), or an
// element outside it that shares a piece with it, or a whole piece of V copied elements.  In place only the
// pairs are moved.
template <typename T, int V>
__global__ void __launch_bounds__(rope::kThreads, 4) rope_pairs_kernel(const RopeParams p) {
  using elem::Piece;
  constexpr int kU = rope::unroll<T>();
  __shared__ float2 table[rope::kTable];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.rows - row0));
  const int head0 = blockIdx.y * p.heads_per_cta;
  const int nheads = min(p.heads_per_cta, p.heads - head0);
  const int pairs = p.rot >> 1, units = nrows * nheads;
  const int g = threadIdx.x / p.lanes, k0 = threadIdx.x - g * p.lanes;
  const T* x = static_cast<const T*>(p.x) + row0 * p.xr + head0 * p.xh;
  T* out = static_cast<T*>(p.out) + row0 * p.orow + head0 * p.oh;
  const int from = p.rot0 / V * V, to = (p.rot0 + p.rot + V - 1) / V * V;  // the pieces that hold the range
  const int singles = to - from - p.rot;
  Piece<T, V> piece[kU];
  T a[kU], b[kU];
  int d = 0, second = 0, kind = 0;  // of item k: its first dim, the distance to its second element; 0 pair, 1 element, 2 piece
  auto item = [&](int k) {
    if (k < pairs) {
      kind = 0;
      d = p.rot0 + (p.half_layout ? k : 2 * k);
      second = p.half_layout ? pairs : 1;
    } else if (k < pairs + singles) {
      kind = 1;
      d = from + k - pairs;
      if (d >= p.rot0) d += p.rot;
    } else {
      kind = 2;
      d = V * (k - pairs - singles);
      if (d >= from) d += to - from;
    }
  };
  auto row_of = [&](int u) { return nrows == 1 ? 0 : u / nheads; };
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = u0 + i * p.groups;
      if (u >= units) break;
      const int r = row_of(u);
      const T* src = x + r * p.xr + (u - r * nheads) * p.xh + d;
      if (kind == 2) {
        piece[i].load(src);
      } else {
        a[i] = src[0];
        if (kind == 0) b[i] = src[second];
      }
    }
  };
  const bool first = g < p.groups && k0 < p.items;
  if (first) {
    item(k0);
    load(g);
  }
  for (int i = threadIdx.x; i < nrows * pairs; i += blockDim.x) {
    const int r = i / pairs;
    table[i] = rope::cos_sin<sizeof(T) == 4>(p.pos[row0 + r], p.freqs[i - r * pairs], p.mscale, p.transpose != 0);
  }
  __syncthreads();
  if (!first) return;
  for (int k = k0; k < p.items; k += p.lanes) {
    if (k != k0) item(k);
    for (int u0 = g; u0 < units; u0 += kU * p.groups) {
      if (k != k0 || u0 != g) load(u0);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = u0 + i * p.groups;
        if (u >= units) break;
        const int r = row_of(u);
        T* dst = out + r * p.orow + (u - r * nheads) * p.oh + d;
        if (kind == 2) {
          piece[i].store(dst);
        } else if (kind == 1) {
          dst[0] = a[i];
        } else {
          const float2 q = table[r * pairs + k];
          float f = elem::to_f32(a[i]), h = elem::to_f32(b[i]);
          rope::turn(f, h, q.x, q.y);
          dst[0] = elem::from_f32<T>(f);
          dst[second] = elem::from_f32<T>(h);
        }
      }
    }
  }
}

}  // namespace dsa
