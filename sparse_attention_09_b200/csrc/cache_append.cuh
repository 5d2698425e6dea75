// Appends tokens to the latent cache and to the indexer-key cache, in one pass: the latent's 512
// dims RMS-normalised and its 64 rope dims rotated, the indexer key rotated on 64 of its dims and
// quantised to e4m3 with one scale per token, each written to its slot of a paged or contiguous
// cache.
//
// One warp per token: 512 dims are two 16-byte pieces per lane, and 64 rotated dims are one pair
// per lane, so the cos / sin of a lane's pair serve the latent and the key.  All of a token's loads
// are issued before the first reduction.  HBM-bound for a prompt (1152 + 2 d_I bytes read, 1152 +
// d_I + 4 written per token), launch-bound for a decode batch.
#pragma once

#include "elem.cuh"
#include "quantize.cuh"
#include "rope.cuh"

namespace dsa {

struct AppendCache {
  void* data;           // null: this half is left out
  float* scale;
  const int32_t* cu;    // contiguous
  const int32_t* table; // paged
  int64_t rows;         // contiguous: rows of the array; paged: pages of the pool
  int32_t max_blocks;
  int32_t max_seqlen;
};

struct AppendParams {
  const __nv_bfloat16* kv;
  const __nv_bfloat16* w;
  const __nv_bfloat16* key;
  int64_t ld_kv, ld_key;
  float eps;
  const int32_t* seq;  // null: row r is sequence r
  const int32_t* pos;
  int64_t rows;
  int32_t B;
  const double* freqs;
  float mscale;
  int32_t half, key_half, key_rot0;
  AppendCache latent, keys;
};

namespace append {

constexpr int kWarps = 4;  // tokens per CTA

// The cache row of position pos of sequence b, or -1 if it lies outside the cache.
__device__ __forceinline__ int64_t slot_of(const AppendCache& c, int b, int pos) {
  if (pos < 0 || pos >= c.max_seqlen) return -1;
  if (c.cu != nullptr) {
    const int64_t row = static_cast<int64_t>(c.cu[b]) + pos;
    return row >= 0 && row < c.cu[b + 1] && row < c.rows ? row : -1;
  }
  if ((pos >> 6) >= c.max_blocks) return -1;
  const int blk = c.table[static_cast<int64_t>(b) * c.max_blocks + (pos >> 6)];
  return blk >= 0 && blk < c.rows ? static_cast<int64_t>(blk) * 64 + (pos & 63) : -1;
}

// A lane's rotated pair of a row's 64 rope dims: (2 lane, 2 lane + 1) or (lane, lane + 32).
__device__ __forceinline__ void load_pair(const __nv_bfloat16* rope, bool half, int lane, float& a, float& b) {
  if (half) {
    a = __bfloat162float(rope[lane]);
    b = __bfloat162float(rope[lane + 32]);
  } else {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(rope + 2 * lane));
    a = f.x;
    b = f.y;
  }
}

}  // namespace append

template <int D_I>
__global__ void __launch_bounds__(append::kWarps * 32) cache_append_kernel(const AppendParams p) {
  using elem::Raw8;
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * append::kWarps + (threadIdx.x >> 5);
  if (r >= p.rows) return;
  const bool with_kv = p.latent.data != nullptr, with_key = p.keys.data != nullptr;
  const int64_t b = p.seq != nullptr ? p.seq[r] : r;
  if (b == -1) return;  // padding
  const int pos = p.pos[r];
  Raw8<__nv_bfloat16> c0, c1, w0, w1;
  float ra = 0.f, rb = 0.f, ka = 0.f, kb = 0.f, kc = 0.f, kd = 0.f;
  if (with_kv) {
    const __nv_bfloat16* kv = p.kv + r * p.ld_kv;
    c0.load(kv + 8 * lane);
    c1.load(kv + 256 + 8 * lane);
    append::load_pair(kv + 512, p.half != 0, lane, ra, rb);
    w0.load(p.w + 8 * lane);
    w1.load(p.w + 256 + 8 * lane);
  }
  // the dims of a 128-d key outside its rotated range: d = 2 lane, 2 lane + 1, shifted past it
  const int rest = 2 * lane >= p.key_rot0 ? 2 * lane + 64 : 2 * lane;
  if (with_key) {
    const __nv_bfloat16* key = p.key + r * p.ld_key;
    append::load_pair(key + p.key_rot0, p.key_half != 0, lane, ka, kb);
    if constexpr (D_I == 128) append::load_pair(key + rest - 2 * lane, false, lane, kc, kd);
  }
  const bool in_batch = b >= 0 && b < p.B;
  const int64_t ls = with_kv && in_batch ? append::slot_of(p.latent, static_cast<int>(b), pos) : -1;
  const int64_t ks = with_key && in_batch ? append::slot_of(p.keys, static_cast<int>(b), pos) : -1;
  if (lane == 0 && ((with_kv && ls < 0) || (with_key && ks < 0))) record_device_error(DSA_ERR_DEVICE_CHECK);
  const float2 cs = rope::cos_sin(pos, p.freqs[lane], p.mscale, false);
  if (with_kv) {
    float f[16], g[16];
    c0.get(f);
    c1.get(f + 8);
    w0.get(g);
    w1.get(g + 8);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(f[j], f[j], ss);
    ss = elem::warp_sum(ss);
    const float rs = __fdiv_rn(1.f, sqrtf(ss * (1.f / 512.f) + p.eps));
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = f[j] * rs * g[j];
    rope::turn(ra, rb, cs);
    if (ls >= 0) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.latent.data) + ls * 576;
      c0.set(f);
      c1.set(f + 8);
      c0.store(dst + 8 * lane);
      c1.store(dst + 256 + 8 * lane);
      if (p.half != 0) {
        dst[512 + lane] = __float2bfloat16_rn(ra);
        dst[544 + lane] = __float2bfloat16_rn(rb);
      } else {
        *reinterpret_cast<__nv_bfloat162*>(dst + 512 + 2 * lane) = __floats2bfloat162_rn(ra, rb);
      }
    }
  }
  if (with_key) {
    rope::turn(ka, kb, cs);
    const float m = fmaxf(fmaxf(fabsf(ka), fabsf(kb)), fmaxf(fabsf(kc), fabsf(kd)));  // a NaN never wins fmaxf
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    const float s = amax > 0.f ? __fdiv_rn(amax, quant::kE4m3Max) : 1.f;
    if (ks >= 0) {
      uint8_t* dst = static_cast<uint8_t*>(p.keys.data) + ks * D_I;
      const uint16_t ab = quant::to_e4m3x2(__fdiv_rn(ka, s), __fdiv_rn(kb, s));
      if (p.key_half != 0) {
        dst[p.key_rot0 + lane] = static_cast<uint8_t>(ab);
        dst[p.key_rot0 + 32 + lane] = static_cast<uint8_t>(ab >> 8);
      } else {
        *reinterpret_cast<uint16_t*>(dst + p.key_rot0 + 2 * lane) = ab;
      }
      if constexpr (D_I == 128)
        *reinterpret_cast<uint16_t*>(dst + rest) = quant::to_e4m3x2(__fdiv_rn(kc, s), __fdiv_rn(kd, s));
      if (lane == 0) p.keys.scale[ks] = s;
    }
  }
}

}  // namespace dsa
