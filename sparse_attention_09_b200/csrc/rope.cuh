// Rotary positions on a range of each head's dims.
//
//   angle = position * freq_i;  (a, b) -> (a c - b s, a s + b c),  c = mscale cos, s = mscale sin
//   (transposed, the backward pass: s with the opposite sign)
//
// At position 10^6 an fp32 angle is off by up to 0.03 rad, so the angle is formed in fp64, as turns
// (position * freq / 2 pi); its fraction of a turn, in [-1/2, 1/2], is then exact enough in fp32 for
// sincospif (error about 2e-7 rad).
//
// HBM-bound: x is read and out written once.  A CTA takes a few rows (or a range of one row's
// heads), issues its loads, computes the rows' cos / sin table once into shared memory (it serves
// every head of the row) and rotates.  Pieces of 8 elements (16 or 32 bytes) where the pointers,
// strides and the rotated range allow; else one pair or element at a time.
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
  int32_t copy_rest;       // out != x: the dims outside the range are copied
  int32_t rows_per_cta;    // > 1 only with head_parts == 1
  int32_t heads_per_cta;
  int32_t items_per_head;  // pieces (or pairs and elements) of a head that are moved
};

namespace rope {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // pieces whose loads a thread issues together
constexpr int kMaxPairs = 512;
constexpr int kTable = 1024;  // cos / sin entries of a CTA's rows

// (mscale cos, mscale sin) of position * freq; s negated for the transposed rotation.
__device__ __forceinline__ float2 cos_sin(int pos, double freq, float mscale, bool transpose) {
  const double turns = static_cast<double>(pos) * (freq * 0.15915494309189535);
  const float f = static_cast<float>(turns - rint(turns));
  float s, c;
  sincospif(2.f * f, &s, &c);
  return make_float2(mscale * c, transpose ? -mscale * s : mscale * s);
}

__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float u = a * cs.x - b * cs.y;
  b = a * cs.y + b * cs.x;
  a = u;
}

}  // namespace rope

template <typename T, bool HALF>
__global__ void __launch_bounds__(rope::kThreads) rope_kernel(const RopeParams p) {
  using elem::Raw8;
  __shared__ float2 table[rope::kTable];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.rows - row0));
  const int head0 = blockIdx.y * p.heads_per_cta;
  const int nheads = min(p.heads_per_cta, p.heads - head0);
  const int pairs = p.rot >> 1;
  const int rot_items = HALF ? p.rot >> 4 : p.rot >> 3;  // of a head; the first items are the rotated ones
  const int hp = p.rot >> 1;
  const int per_row = nheads * p.items_per_head, total = nrows * per_row;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  bool ready = false;
  for (int base = 0; base < total; base += rope::kThreads * rope::kUnroll) {
    Raw8<T> a[rope::kUnroll], b[rope::kUnroll];
    int64_t at[rope::kUnroll];
    int cs[rope::kUnroll];  // first table entry of a rotated piece; -1: copied; -2: none
#pragma unroll
    for (int u = 0; u < rope::kUnroll; ++u) {
      const int i = base + u * rope::kThreads + static_cast<int>(threadIdx.x);
      cs[u] = -2;
      if (i >= total) continue;
      const int r = i / per_row, j = i - r * per_row;
      const int h = j / p.items_per_head, k = j - h * p.items_per_head;
      int d;
      if (k < rot_items) {
        d = p.rot0 + 8 * k;
        cs[u] = r * pairs + (HALF ? 8 * k : 4 * k);
      } else {
        d = 8 * (k - rot_items);
        if (d >= p.rot0) d += p.rot;  // the copied pieces skip the rotated range
        cs[u] = -1;
      }
      const T* src = x + (row0 + r) * p.xr + (head0 + h) * p.xh + d;
      a[u].load(src);
      if (HALF && k < rot_items) b[u].load(src + hp);
      at[u] = (row0 + r) * p.orow + (head0 + h) * p.oh + d;
    }
    if (!ready) {
      for (int i = threadIdx.x; i < nrows * pairs; i += rope::kThreads) {
        const int r = i / pairs;
        table[i] = rope::cos_sin(p.pos[row0 + r], p.freqs[i - r * pairs], p.mscale, p.transpose != 0);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < rope::kUnroll; ++u) {
      if (cs[u] == -2) continue;
      if (cs[u] >= 0) {
        float f[8];
        a[u].get(f);
        if constexpr (HALF) {
          float g[8];
          b[u].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) rope::turn(f[j], g[j], table[cs[u] + j]);
          b[u].set(g);
          b[u].store(out + at[u] + hp);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) rope::turn(f[2 * j], f[2 * j + 1], table[cs[u] + j]);
        }
        a[u].set(f);
      }
      a[u].store(out + at[u]);
    }
  }
}

// General form: an item is a pair (items 0 .. rot/2 - 1 of a head) or one copied element.
template <typename T>
__global__ void __launch_bounds__(rope::kThreads) rope_general_kernel(const RopeParams p) {
  using elem::from_f32;
  using elem::to_f32;
  __shared__ float2 table[rope::kTable];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.rows - row0));
  const int head0 = blockIdx.y * p.heads_per_cta;
  const int nheads = min(p.heads_per_cta, p.heads - head0);
  const int pairs = p.rot >> 1;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  for (int i = threadIdx.x; i < nrows * pairs; i += rope::kThreads) {
    const int r = i / pairs;
    table[i] = rope::cos_sin(p.pos[row0 + r], p.freqs[i - r * pairs], p.mscale, p.transpose != 0);
  }
  __syncthreads();
  const int per_row = nheads * p.items_per_head, total = nrows * per_row;
  for (int i = threadIdx.x; i < total; i += rope::kThreads) {
    const int r = i / per_row, j = i - r * per_row;
    const int h = j / p.items_per_head, k = j - h * p.items_per_head;
    const T* src = x + (row0 + r) * p.xr + (head0 + h) * p.xh;
    T* dst = out + (row0 + r) * p.orow + (head0 + h) * p.oh;
    if (k < pairs) {
      const int d0 = p.rot0 + (p.half_layout ? k : 2 * k), d1 = d0 + (p.half_layout ? pairs : 1);
      float a = to_f32(src[d0]), b = to_f32(src[d1]);
      rope::turn(a, b, table[r * pairs + k]);
      dst[d0] = from_f32<T>(a);
      dst[d1] = from_f32<T>(b);
    } else {
      int d = k - pairs;
      if (d >= p.rot0) d += p.rot;
      dst[d] = src[d];
    }
  }
}

}  // namespace dsa
