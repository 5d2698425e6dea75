// Appends tokens to the latent cache and to the indexer-key cache, in one pass: the latent's 512
// dims RMS-normalised and its 64 rope dims rotated, the indexer key rotated on 64 of its dims and
// quantised to e4m3 with one scale per token, each written to its slot of a paged or contiguous
// cache.
//
// One warp per token: 512 dims are two 16-byte pieces per lane, and 64 rotated dims are one pair
// per lane, so the cos / sin of a lane's pair serve the latent and the key.  HBM-bound for a prompt
// (1152 + 2 d_I bytes read, 1152 + d_I + 4 written per token), launch-bound for a decode batch.
//
// A token's chain of dependent loads (its position, its page, its data) is longer than its work, and
// what is the same for all lanes costs as much to compute as what is not.  So a warp takes tokens
// in blocks of 32: lane j finds the slots of the block's token j, and the rows of the next three
// tokens are always on their way into a ring of the warp's own in shared memory (asynchronous
// copies).  Measured on the device alone, 65536 tokens, d_I = 128: 48.9 us with a token's loads issued together and
// no look-ahead, 41.3 us with the ring and each token's slots found by all lanes, 33.2 us with both
// (5.3 TB/s, 0.81 of measured HBM).
#pragma once

#include "elem.cuh"
#include "e4m3.cuh"
#include "rope.cuh"

namespace dsa {

struct AppendCache {
  void* data;           // null: this half is left out
  float* scale;
  const int32_t* cu;    // contiguous
  const int32_t* table; // paged
  int32_t rows;         // contiguous: rows of the array; paged: pages of the pool (rows of either < 2^31)
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

constexpr int kWarps = 4;   // per CTA, each with tokens of its own
constexpr int kStages = 4;  // tokens of a warp's ring
constexpr int kCtas = 8;    // per SM (6, with more registers: 34.6 us)

// The cache row of position pos of sequence b, or -1 if it lies outside the cache.
__device__ __forceinline__ int slot_of(const AppendCache& c, int b, int pos) {
  if (pos < 0 || pos >= c.max_seqlen) return -1;
  if (c.cu != nullptr) {
    const int64_t row = static_cast<int64_t>(c.cu[b]) + pos;
    return row >= 0 && row < c.cu[b + 1] && row < c.rows ? static_cast<int>(row) : -1;
  }
  if ((pos >> 6) >= c.max_blocks) return -1;
  const int blk = c.table[static_cast<int64_t>(b) * c.max_blocks + (pos >> 6)];
  return blk >= 0 && blk < c.rows ? blk * 64 + (pos & 63) : -1;
}

__device__ __forceinline__ void cp_async4(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem), "l"(src) : "memory");
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

// D_I = 0: no indexer keys.
template <bool KV, int D_I>
__global__ void __launch_bounds__(append::kWarps * 32, append::kCtas) cache_append_kernel(const AppendParams p) {
  using elem::Raw8;
  using append::kStages;
  constexpr int kStageElems = 576 + D_I;
  __shared__ __align__(16) __nv_bfloat16 ring[append::kWarps][kStages][kStageElems];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * append::kWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * append::kWarps + warp;
  // each lane's part of the row that is copied next
  int64_t ir = first;
  const __nv_bfloat16* kv = KV ? p.kv + first * p.ld_kv + 8 * lane : nullptr;
  const __nv_bfloat16* kx = D_I > 0 ? p.key + first * p.ld_key + 2 * lane : nullptr;
  const int64_t kv_step = step * p.ld_kv, kx_step = step * p.ld_key;
  auto issue = [&](int s) {  // one group per token, empty past the last
    if (ir < p.rows) {
      const uint32_t dst = dev::smem_addr(ring[warp][s]);
      if constexpr (KV) {
        dev::cp_async16(dst + 16 * lane, kv);
        dev::cp_async16(dst + 512 + 16 * lane, kv + 256);
        if (lane < 8) dev::cp_async16(dst + 1024 + 16 * lane, kv + 512);
        kv += kv_step;
      }
      if constexpr (D_I > 0) {  // keys are 4-byte aligned
#pragma unroll
        for (int i = 0; i < D_I / 64; ++i) append::cp_async4(dst + 1152 + 4 * (lane + 32 * i), kx + 64 * i);
        kx += kx_step;
      }
    }
    ir += step;
    dev::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  const double freq = p.freqs[lane];
  Raw8<__nv_bfloat16> w0, w1;
  w0.zero();
  w1.zero();
  if constexpr (KV) {
    w0.load(p.w + 8 * lane);
    w1.load(p.w + 256 + 8 * lane);
  }
  // the dims of a 128-d key outside its rotated range: d = 2 lane, 2 lane + 1, shifted past it
  const int rest = 2 * lane >= p.key_rot0 ? 2 * lane + 64 : 2 * lane;
  int st = 0;
  for (int64_t base = first; base < p.rows; base += 32 * step) {
    int ls = -1, ks = -1, pos = 0;  // of the block's token `lane`
    {
      const int64_t r = base + lane * step;
      int64_t b = -1;
      if (r < p.rows) {
        b = p.seq != nullptr ? p.seq[r] : r;
        pos = p.pos[r];
      }
      if (b >= 0 && b < p.B) {
        if constexpr (KV) ls = append::slot_of(p.latent, static_cast<int>(b), pos);
        if constexpr (D_I > 0) ks = append::slot_of(p.keys, static_cast<int>(b), pos);
      }
      if (b != -1 && ((KV && ls < 0) || (D_I > 0 && ks < 0))) record_device_error(DSA_ERR_DEVICE_CHECK);  // -1: padding
    }
    const int count = static_cast<int>(min(static_cast<int64_t>(32), (p.rows - base + step - 1) / step));
    for (int j = 0; j < count; ++j) {
      issue(st == 0 ? kStages - 1 : st - 1);  // into the stage read last
      const int cls = __shfl_sync(0xffffffffu, ls, j), cks = __shfl_sync(0xffffffffu, ks, j);
      const int cpos = __shfl_sync(0xffffffffu, pos, j);
      dev::cp_async_wait<kStages - 1>();
      __syncwarp();
      const __nv_bfloat16* row = ring[warp][st];
      if (++st == kStages) st = 0;
      const float2 cs = rope::cos_sin<false>(cpos, freq, p.mscale, false);
      if (KV && cls >= 0) {
        Raw8<__nv_bfloat16> c0, c1;
        float ra, rb;
        c0.load(row + 8 * lane);
        c1.load(row + 256 + 8 * lane);
        append::load_pair(row + 512, p.half != 0, lane, ra, rb);
        float f[16], g[16];
        c0.get(f);
        c1.get(f + 8);
        w0.get(g);
        w1.get(g + 8);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss = fmaf(f[j], f[j], ss);
        ss = elem::warp_sum(ss);
        const float rs = rsqrtf(ss * (1.f / 512.f) + p.eps);  // 2 units in the last place, rounded to bf16 below
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = f[j] * rs * g[j];
        rope::turn(ra, rb, cs.x, cs.y);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.latent.data) + static_cast<int64_t>(cls) * 576;
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
      if (D_I > 0 && cks >= 0) {
        const __nv_bfloat16* key = row + 576;
        float ka, kb, kc = 0.f, kd = 0.f;
        append::load_pair(key + p.key_rot0, p.key_half != 0, lane, ka, kb);
        if constexpr (D_I == 128) append::load_pair(key + rest - 2 * lane, false, lane, kc, kd);
        rope::turn(ka, kb, cs.x, cs.y);
        const float m = fmaxf(fmaxf(fabsf(ka), fabsf(kb)), fmaxf(fabsf(kc), fabsf(kd)));  // a NaN never wins fmaxf
        const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        const float s = quant::scale_of(amax), inv = quant::inverse_of(s);
        uint8_t* dst = static_cast<uint8_t*>(p.keys.data) + static_cast<int64_t>(cks) * D_I;
        const uint16_t ab = quant::to_e4m3x2(quant::over(ka, s, inv), quant::over(kb, s, inv));
        if (p.key_half != 0) {
          dst[p.key_rot0 + lane] = static_cast<uint8_t>(ab);
          dst[p.key_rot0 + 32 + lane] = static_cast<uint8_t>(ab >> 8);
        } else {
          *reinterpret_cast<uint16_t*>(dst + p.key_rot0 + 2 * lane) = ab;
        }
        if constexpr (D_I == 128)
          *reinterpret_cast<uint16_t*>(dst + rest) = quant::to_e4m3x2(quant::over(kc, s, inv), quant::over(kd, s, inv));
        if (lane == 0) p.keys.scale[cks] = s;
      }
      __syncwarp();  // every lane has read the stage before it is refilled
    }
  }
  dev::cp_async_wait<0>();
}

}  // namespace dsa
