// MLA attention (MQA mode) under a sliding window with sinks, on a CTA pair that splits the heads.
//
//   out[t,h,:] = sum_s softmax_s(sm_scale * q[t,h,:] . c_s) * c_s[0:512],  s <= t and (s > t - window or s < sinks)
//
// The two products and their split over the pair are those of the sparse kernel (sparse_mla_pair.cuh):
// CTA r owns heads [64r, 64r + 64); S = Q.K^T and O += P.V are pair MMAs (M = 128) issued from CTA 0, K
// split by keys and V by value dims.  What differs:
//   * the keys are not selected but numbered: entry e < ns is position e, entry e >= ns position
//     e + (lo - ns), with lo = max(0, t + 1 - window) and ns = min(sinks, lo).  So every chunk but a
//     query's last is full, nothing is masked but that chunk's tail (its logits are set to -inf in a
//     branch of its own), and a row outside the window is never loaded: entries past the last are
//     written as zeros, so that a NaN in an unused slot cannot reach P.V as 0 * NaN;
//   * a chunk is 128 keys: Q.K^T with N = 128 reads Q from shared memory half as often per key as with
//     64 (32 cycles of tensor work on 4 KB of operands, where N = 64 has 16 on 3 KB).  The room comes from
//     staging one chunk of own rows by groups of 192 dims, each refilled as soon as its MMAs are done,
//     and P and V by halves of 64 keys.  With 64-key chunks, two of them staged: 979 us against 871 on 3984
//     tokens with a window of 1024, 2099 against 1833 on 5008 with 2048 (bursts), 90 against 80 for
//     three decode sequences up to 128K; equal at windows of 128, and one key block of 64 or less costs
//     1 % more in prefill, 1.3 us more (11.5) in a decode launch.  A last chunk of at most 64 keys
//     has no second half: CTA r then stages keys [32r, 32r + 32) and the upper rows keep what they held,
//     which reaches only columns of S that are masked;
//   * the row sum is that of the unrounded fp32 probabilities (lse is an fp32 result of its own);
//   * each issuing or relaying warp follows one stream of operands and waits for each barrier in turn;
//   * a wait that runs out is remembered: the warp goes on without waiting (on whatever the buffers
//     hold, all within them) and reports it at the end, so that no two warps have to agree on leaving;
//   * decode: a cluster takes a share of all sequences' chunks (below).
//
// Bound: shared-memory bandwidth.  Per chunk and SM the MMAs read 240 KB (Q 72, K 72, P 32, V 64) and
// the copies write 136 KB: 2.9K cycles at 128 B per cycle, against about 3.4K measured (2.2K of tensor work).
// On 5008 tokens with a window of 2048: 1.83 to 1.91 ms in a burst (1.2 PFLOP/s), 2.12 to 2.16 under the power cap
// (1.06, 0.77 of measured sustained bf16).
// The instruction cache comes next: the roles' loops run side by side, and as a form of the sparse
// kernel the same work (by 64 keys) took 2.57 ms with that kernel's unstaged epilogue and 3.41 with the staged
// one inline in the softmax loop, against 2.16 ms on its own, so loops are small and what is rare is
// out of line.  N of Q.K^T is the same for every chunk: chosen per chunk (64 for a last one
// without a second half) the whole kernel took 2.01 ms instead of 1.91.
#pragma once

#include "common.cuh"
#include "mla_common.cuh"
#include "sm100.cuh"
#include "sparse_mla_pair.cuh"

namespace dsa {

struct WinParams {
  const int32_t* cu_seqlens;    // prefill [B+1]
  const int32_t* block_table;   // decode [B, max_blocks]
  const int32_t* context_lens;  // decode [B]
  int32_t max_blocks, num_blocks;
  int32_t max_len;              // decode: contexts are clamped to this
  int32_t B, H, window, sinks;
  int64_t rows;                 // prefill: rows of q
  float scale_log2;             // sm_scale * log2(e)
  __nv_bfloat16* out;           // [rows, H, 512]
  float* lse;                   // [rows, H] natural log (nullable)
  int32_t shared;               // decode: the clusters share out the chunks of all sequences
  float* part_o;                // shared: [2 * clusters, H, 512] unnormalised
  float* part_ml;               // shared: [2 * clusters, H, 2] (M in log2 units, l)
  int2* plan;                   // shared: [B] first and last cluster that hold chunks of a sequence
};

namespace win {

using mlap::kColO;
using mlap::kColS;
using mlap::kFirstProducerWarp;
using mlap::kHeads;
using mlap::kMmaWarp;
using mlap::kOffKQ;
using mlap::kOffP;
using mlap::kOffQ;
using mlap::kOffV;
using mlap::kPBytes;
using mlap::kPvWarp;
using mlap::kQBlockBytes;
using mlap::kQBytes;
using mlap::kQWarp;
using mlap::kSmemBytes;
using mlap::kSoftmaxWarps;
using mlap::kTau;
using mlap::kThreads;
using mlap::kVBlockBytes;
using mlap::kVBytes;
using mlap::kVWarp0;

constexpr int kChunk = 128;                         // entries per pipeline step, in two halves of 64
constexpr int kHalf = 64;
constexpr int kKQBlockBytes = kHalf * 128;          // a CTA's 64 own rows x 64 dims
constexpr int kGroups = 3;                          // own rows are staged by groups of 192 dims
constexpr int kGroupBlocks = 3;
constexpr int kGroupBytes = kGroupBlocks * kKQBlockBytes;
static_assert(kOffKQ + kGroups * kGroupBytes == kOffV, "one chunk of own rows");

// What a query costs beside its chunks (its Q, the pipeline's fill, the readout of O), in chunks:
// measured 3 to 4 us against 1.7 to 1.9 per chunk in prefill (1 and 3 share as evenly; decode's chunks take 2.0 with
// the pages in L2, 2.25 without).
constexpr int kUnitCost = 2;
// Decode: pages are brought into L2 this many chunks ahead of their copies.  Fitted on shared-out sequences only
// (one of 128K 54.5 / 57.0 / 62.6 us with 1 / 2 / 4, three up to 128K 78 / 79.5 / 88), used for whole ones too.
constexpr int kAhead = 1;

// The entries of a query that has `len` keys up to its own: entry e < ns is position e, a later one
// below `end` position e + shift.
struct Visible {
  int ns, shift, end;
  __device__ __forceinline__ int chunks() const { return max(1, (end - 1) / kChunk + 1); }  // 0 keys: one, masked whole
  // Whether chunk c has keys in its second half; all but the last have.
  __device__ __forceinline__ bool second(int c) const { return c * kChunk + kHalf < end; }
};
__device__ __forceinline__ Visible visible(const WinParams& p, int len) {
  len = max(len, 0);
  const int lo = max(0, len - p.window);
  Visible v;
  v.ns = min(p.sinks, lo);
  v.shift = lo - v.ns;
  v.end = len - v.shift;
  return v;
}
__device__ __forceinline__ int context_of(const WinParams& p, int b) { return min(p.context_lens[b], p.max_len); }

// A piece of work: chunks [c0, c1) of a query.
struct Work {
  int64_t qrow;   // row of q, out and lse
  int seq, start; // its sequence; prefill: the latent row of its position 0
  Visible v;
  int c0, c1;
  int part;       // row of part_o / part_ml, or -1: the whole query, straight to out
};

// The pieces of one cluster, in order; every role walks the same ones.
//   prefill: every ncl-th query;  decode, not shared: every ncl-th sequence;
//   decode, shared: sequence b stands for cost units [base_b, base_b + chunks_b + kUnitCost), the first
//   chunks_b of them its chunks, and the cluster takes the chunks in its range [lo, hi).  A cluster has
//   at most two pieces that are not whole: its first and its last.
template <bool DECODE>
struct Walk {
  int64_t u, base, lo, hi, limit;
  int step;
  __device__ __forceinline__ bool next(const WinParams& p, int cid, Work& w) {
    if constexpr (!DECODE) {
      if (u >= limit) return false;
      int a = 0, b = p.B;  // the sequence of packed token u
      while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (p.cu_seqlens[mid] <= u) a = mid;
        else b = mid;
      }
      w.seq = a;
      w.start = p.cu_seqlens[a];
      w.qrow = u;
      w.v = visible(p, static_cast<int>(u + 1 - w.start));
      w.c0 = 0;
      w.c1 = w.v.chunks();
      w.part = -1;
      u += step;
      return true;
    } else {
      w.start = 0;
      while (u < limit && base < hi) {
        w.seq = static_cast<int>(u);
        w.qrow = u;
        w.v = visible(p, context_of(p, w.seq));
        const int chunks = w.v.chunks();
        const int64_t from = base;
        u += step;
        if (!p.shared) {
          w.c0 = 0;
          w.c1 = chunks;
          w.part = -1;
          return true;
        }
        base += chunks + kUnitCost;
        w.c0 = static_cast<int>(max(lo - from, static_cast<int64_t>(0)));
        w.c1 = static_cast<int>(min(hi - from, static_cast<int64_t>(chunks)));
        if (w.c1 > w.c0) {
          w.part = w.c0 > 0 ? 2 * cid : w.c1 < chunks ? 2 * cid + 1 : -1;
          return true;
        }
      }
      return false;
    }
  }
};

// One warp: this cluster's range of cost units and the sequence it begins in (shared decode).
__device__ __forceinline__ void plan_walk(const WinParams& p, int cid, int ncl, bool write, Walk<true>& out) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  for (int b = lane; b < p.B; b += 32) total += visible(p, context_of(p, b)).chunks() + kUnitCost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int n = static_cast<int>(min(static_cast<int64_t>(ncl), total));  // clusters: each has a cost unit at least
  out.lo = cid < n ? total * cid / n : total;
  out.hi = cid < n ? total * (cid + 1) / n : total;
  out.u = p.B;
  out.base = total;
  int64_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int cost = b < p.B ? visible(p, context_of(p, b)).chunks() + kUnitCost : 0;
    const int64_t mine = base + warp_inclusive_scan(cost) - cost;  // 32 costs fit an int
    if (write && b < p.B) {
      // the clusters of its first and its last chunk: cluster i holds [total i / n, total (i + 1) / n)
      const int64_t last = mine + cost - kUnitCost - 1;
      int64_t i0 = mine * n / total, i1 = last * n / total;
      while (total * (i0 + 1) / n <= mine) ++i0;
      while (total * (i1 + 1) / n <= last) ++i1;
      p.plan[b] = make_int2(static_cast<int>(i0), static_cast<int>(i1));
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, b < p.B && mine <= out.lo && out.lo < mine + cost);
    if (hit != 0) {
      out.u = b0 + __ffs(hit) - 1;
      out.base = __shfl_sync(0xffffffffu, mine, __ffs(hit) - 1);
      if (!write) break;
    }
    base = __shfl_sync(0xffffffffu, mine + cost, 31);
  }
}

// Whether entry e of a piece of work is a key, and its latent row (-1 if not).
template <bool DECODE>
__device__ __forceinline__ int row_of(const WinParams& p, const int32_t* bt, const Work& w, int e, bool& bad) {
  bad = false;
  if (e >= w.v.end) return -1;
  const int pos = e < w.v.ns ? e : e + w.v.shift;
  int row;
  if constexpr (DECODE) {
    const int blk = bt[pos >> 6];
    bad = blk < 0 || blk >= p.num_blocks;
    row = blk * 64 + (pos & 63);
  } else {
    row = w.start + pos;
    bad = row < 0;  // a negative cu_seqlens entry
  }
  return bad ? -1 : row;
}

// ---- small device helpers ----------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Copies 16 bytes of row r, or writes 16 zero bytes without reading (r < 0; base is mapped memory).
__device__ __forceinline__ void copy_piece(uint32_t dst_smem, const __nv_bfloat16* latent, int r, int elem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem),
               "l"(latent + static_cast<int64_t>(max(r, 0)) * 576 + elem), "r"(r >= 0 ? 16 : 0)
               : "memory");
}
// Brings a page of the latent pool into L2.
__device__ __forceinline__ void prefetch_page(const __nv_bfloat16* page) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(page), "r"(64 * 576 * 2) : "memory");
}
// Brings a tile of a tensor map into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1) : "memory");
}

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity) { return dev::mbar_wait(bar, parity); }

// O *= alpha for a warp's 32 heads x 256 columns.
__device__ __noinline__ void rescale_o(uint32_t tmem_o, float alpha) {
  using namespace dev;
#pragma unroll 1
  for (int cc = 0; cc < 256; cc += 32) {
    uint32_t o[32];
    tmem_ld32(tmem_o + cc, o);
    tmem_wait_ld();
    reg_fence(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st32(tmem_o + cc, o);
  }
  tmem_wait_st();
}

// A piece's O: the warp's 32 heads x 256 of the 512 value dims (columns 128m + j of its TMEM lanes are dims
// 256m + j from dst), as T scaled, to global memory through 4 KB of shared memory: written a row per
// lane, read and stored four whole 128-byte rows per instruction.  The 4 KB are the warp's head rows of
// P slot kh: every P.V has completed, and the partner warp writes P of the next piece only after the
// pair's next meeting.  Stored straight from the lanes' rows, every 16-byte store touched 32 of them (per
// query of one chunk 6.27 us, staged 4.80).
template <typename T>
__device__ __noinline__ void store_o(uint32_t tmem_o, float scale, uint8_t* stage, T* dst, int head0, int H) {
  using namespace dev;
  constexpr int kCols = 128 / sizeof(T);  // columns of a 128-byte row
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int cc = 0; cc < 256; cc += kCols) {
#pragma unroll
    for (int part = 0; part < kCols / 32; ++part) {
      uint32_t o[32];
      tmem_ld32(tmem_o + cc + 32 * part, o);
      tmem_wait_ld();
      reg_fence(o);
      constexpr int kPieces = sizeof(T) == 2 ? 4 : 8;  // 16-byte pieces of 32 columns
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint4 v;
        if constexpr (sizeof(T) == 2) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[j] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * j]) * scale, __uint_as_float(o[8 * i + 2 * j + 1]) * scale);
          v = make_uint4(q[0], q[1], q[2], q[3]);
        } else {
          v = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);  // unscaled
        }
        *reinterpret_cast<uint4*>(stage + lane * 128 + (((kPieces * part + i) ^ (lane & 7)) << 4)) = v;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      if (head0 + r < H)
        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(head0 + r) * 512 + 256 * (cc >> 7) + (cc & 127) +
                                  (16 / sizeof(T)) * (lane & 7)) = v;
    }
    __syncwarp();
  }
}

}  // namespace win

template <bool DECODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(win::kThreads, 1)
    window_mla_kernel(const __nv_bfloat16* __restrict__ latent, const WinParams p, const __grid_constant__ CUtensorMap q_map) {
  using namespace dev;
  using namespace win;
  constexpr uint32_t IDESC_QK = idesc_bf16(128, kChunk, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16(128, 256, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + kOffQ;
  uint8_t* sP = smem + kOffP;
  uint8_t* sKQ = smem + kOffKQ;
  uint8_t* sV = smem + kOffV;

  // local to each CTA
  __shared__ uint64_t bar_kq_full[kGroups], bar_v_full[2];  // this CTA's rows of a slot have landed
  __shared__ uint64_t bar_kq_empty[kGroups];            // the MMAs reading a slot are done
  __shared__ uint64_t bar_q_full, bar_q_empty;          // Q staged / the piece's last Q.K^T done
  __shared__ uint64_t bar_s_full[2], bar_pv_done[2];    // S of a slot written / P.V of a half done: its P and V slots are free
  __shared__ uint64_t bar_mma_done;                     // every MMA of the kernel has completed
  // used in CTA 0 only: arrivals from both CTAs, or of CTA 1's staged operands
  __shared__ uint64_t bar_s_free[2], bar_p_full, bar_o_free;
  __shared__ uint64_t bar_kq_peer[kGroups], bar_v_peer[2], bar_q_peer;
  __shared__ uint32_t s_tmem;
  __shared__ float s_red[3][2][kHeads];  // [buffer][key half][head] maxima / sums
  __shared__ Walk<DECODE> s_walk;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(num_clusters_x());

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_v_full[i], 64);  // every thread of the two gathering warps (plus its copies in flight)
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_pv_done[i], 1);
      mbar_init(&bar_s_free[i], 2 * kSoftmaxWarps);
      mbar_init(&bar_v_peer[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&bar_kq_full[i], 64);
      mbar_init(&bar_kq_empty[i], 1);
      mbar_init(&bar_kq_peer[i], 1);
    }
    mbar_init(&bar_p_full, 2 * kSoftmaxWarps);
    mbar_init(&bar_q_full, 1);
    mbar_init(&bar_q_empty, 1);
    mbar_init(&bar_mma_done, 2);
    mbar_init(&bar_o_free, 2 * kSoftmaxWarps);
    mbar_init(&bar_q_peer, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&s_tmem, 512);
    tmem_relinquish_pair();
  }
  if (warp == kFirstProducerWarp) {
    Walk<DECODE> wk;
    wk.u = cid;
    wk.step = ncl;
    wk.base = 0;
    wk.lo = 0;
    wk.hi = 1;
    if constexpr (DECODE) {
      wk.limit = p.B;
      if (p.shared) {
        wk.step = 1;
        plan_walk(p, cid, ncl, cid == 0 && rank == 0, wk);
      }
    } else {
      wk.limit = min(p.rows, static_cast<int64_t>(p.cu_seqlens[p.B]));  // rows behind the last sequence are no queries
    }
    if (lane == 0) s_walk = wk;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto at_leader = [](uint64_t* bar) { return map_to_rank(smem_addr(bar), 0u); };
  bool ok = true;  // per lane: no wait has run out
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_test(smem_addr(bar), parity)) ok = wait_slow(bar, parity);
    __syncwarp();
  };
  Walk<DECODE> walk = s_walk;
  Work w;

  if (warp >= kFirstProducerWarp && warp < kFirstProducerWarp + 2) {
    // ================= own rows, all 576 dims (B of Q.K^T): 32 of this CTA's 64 rows per warp =================
    const int pw = warp - kFirstProducerWarp;
    const int ch = lane & 7;
    uint32_t g = 0;
    while (walk.next(p, cid, w)) {
      const int32_t* bt = DECODE ? p.block_table + static_cast<int64_t>(w.seq) * p.max_blocks : nullptr;
      if (DECODE && pw == 0 && rank == 0 && lane == 0 && w.c0 == 0 &&
          (p.context_lens[w.seq] < 0 || p.context_lens[w.seq] > p.max_len))
        record_device_error(DSA_ERR_DEVICE_CHECK);  // the context is clamped
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        const bool second = w.v.second(c);
        const int own = second ? 32 : 16;  // rows of this warp
        bool bad;
        const int row =
            row_of<DECODE>(p, bt, w, c * kChunk + own * (2 * static_cast<int>(rank) + pw) + (lane & (own - 1)), bad);
        if (bad && lane < own) record_device_error(DSA_ERR_DEVICE_CHECK);  // the key is masked
        if constexpr (DECODE) {
          // the page that the entries kAhead chunks ahead begin in, on its way from HBM in one instruction
          const int e = (c + kAhead) * kChunk + kHalf * static_cast<int>(rank);
          if (pw == 0 && lane == 0 && c + kAhead < w.c1 && e < w.v.end) {
            const int blk = bt[(e < w.v.ns ? e : e + w.v.shift) >> 6];
            if (blk >= 0 && blk < p.num_blocks) prefetch_page(latent + static_cast<int64_t>(blk) * 64 * 576);
          }
        }
#pragma unroll 1
        for (int q = 0; q < kGroups; ++q) {
          wait(&bar_kq_empty[q], (g & 1u) ^ 1u);
          const uint32_t kq = smem_addr(sKQ + q * kGroupBytes) + own * pw * 128;
          const int elem = 64 * kGroupBlocks * q + 8 * ch;
#pragma unroll 1
          for (int j0 = 0; j0 < own; j0 += 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // four rows' 128 bytes of a block per instruction
              const int j = j0 + 4 * i + (lane >> 3);
              const int kr = __shfl_sync(0xffffffffu, row, j);
              const uint32_t dst = kq + j * 128 + ((ch ^ (j & 7)) << 4);
#pragma unroll
              for (int b = 0; b < kGroupBlocks; ++b) copy_piece(dst + b * kKQBlockBytes, latent, kr, elem + 64 * b);
            }
          }
          cp_async_commit();
          cp_async_mbar_arrive(&bar_kq_full[q]);
          mbar_arrive(&bar_kq_full[q]);
        }
      }
    }
    cp_async_wait<0>();
  } else if (warp >= kVWarp0 && warp < kVWarp0 + 2) {
    // ================= all rows, this CTA's value dims (B of P.V): by halves, 32 rows per warp =================
    const int pw = warp - kVWarp0;
    const int seg = lane >> 4, pc = lane & 15;  // segment m: dims 256m + 128 rank + 8 pc
    const int ch = pc & 7, elem = 256 * seg + 128 * static_cast<int>(rank) + 8 * pc;
    uint32_t used[2] = {0, 0};
    while (walk.next(p, cid, w)) {
      const int32_t* bt = DECODE ? p.block_table + static_cast<int64_t>(w.seq) * p.max_blocks : nullptr;
      for (int c = w.c0; c < w.c1; ++c) {
#pragma unroll 1
        for (int s = 0; s <= (w.v.second(c) ? 1 : 0); ++s) {
          bool bad;
          const int row = row_of<DECODE>(p, bt, w, c * kChunk + kHalf * s + 32 * pw + lane, bad);
          const uint32_t n_used = s == 0 ? used[0]++ : used[1]++;
          wait(&bar_pv_done[s], (n_used & 1u) ^ 1u);
          const uint32_t vb = smem_addr(sV + s * kVBytes) + (2 * seg + (pc >> 3)) * kVBlockBytes;
#pragma unroll 8
          for (int j = 0; j < 32; ++j) {
            const int n = 32 * pw + j;
            copy_piece(vb + n * 128 + ((ch ^ (n & 7)) << 4), latent, __shfl_sync(0xffffffffu, row, j), elem);
          }
          cp_async_commit();
          cp_async_mbar_arrive(&bar_v_full[s]);
          mbar_arrive(&bar_v_full[s]);
        }
      }
    }
    cp_async_wait<0>();
  } else if (warp == kQWarp) {
    // ================= Q: this CTA's 64 query rows of each piece, nine TMA tiles =================
    uint32_t tok = 0;
    if (lane == 0) tma_prefetch_desc(&q_map);
    while (walk.next(p, cid, w)) {
      wait(&bar_q_empty, (tok & 1u) ^ 1u);
      if (lane == 0 && ok) {
        mbar_arrive_expect_tx(&bar_q_full, kQBytes);
        const int32_t y = static_cast<int32_t>(w.qrow * p.H + kHeads * static_cast<int64_t>(rank));
#pragma unroll 1
        for (int b = 0; b < 9; ++b) tma_load_2d(sQ + b * kQBlockBytes, &q_map, &bar_q_full, 64 * b, y);
        // the next query's Q into L2, so that its load does not wait for HBM once sQ is free
        if (!DECODE && w.qrow + ncl < p.rows) {
#pragma unroll 1
          for (int b = 0; b < 9; ++b) tma_prefetch_2d(&q_map, 64 * b, y + ncl * p.H);
        }
        ++tok;
      }
      tok = __shfl_sync(0xffffffffu, tok, 0);
    }
    // the last load must have landed before the CTA may exit
    if (lane == 0 && tok > 0 && !mbar_wait(&bar_q_full, (tok - 1) & 1u)) ok = false;
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    uint32_t g = 0, g1 = 0, tok = 0;  // chunks, chunks with a second half, pieces
    if (warp == kMmaWarp && rank == 0) {
      // ================= Q.K^T issuer (for the pair) =================
      const uint64_t ad = make_smem_desc(smem_addr(sQ), 16, 1024, kSwizzle128B);
      const uint64_t bd = make_smem_desc(smem_addr(sKQ), 16, 1024, kSwizzle128B);
      while (walk.next(p, cid, w)) {
        wait(&bar_q_full, tok & 1u);
        wait(&bar_q_peer, tok & 1u);
        ++tok;
        for (int c = w.c0; c < w.c1; ++c, ++g) {
          const int s = static_cast<int>(g & 1u);
          wait(&bar_s_free[s], ((g >> 1) & 1u) ^ 1u);
#pragma unroll 1
          for (int q = 0; q < kGroups; ++q) {
            wait(&bar_kq_full[q], g & 1u);
            wait(&bar_kq_peer[q], g & 1u);
            tc_fence_after();
            if (lane == 0) fence_proxy_async_smem();  // the gathered rows were written through the generic proxy
            __syncwarp();
            const uint64_t aq = ad + ((q * kGroupBlocks * kQBlockBytes) >> 4), bq = bd + ((q * kGroupBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4 * kGroupBlocks; ++kk)
              umma_bf16_ss_pair_warp(tmem + kColS + 64 * s, aq + (((kk >> 2) * kQBlockBytes + (kk & 3) * 32) >> 4),
                                     bq + (((kk >> 2) * kKQBlockBytes + (kk & 3) * 32) >> 4), IDESC_QK, q + kk > 0 ? 1u : 0u);
            if (lane == 0) umma_commit_pair(&bar_kq_empty[q], 3);
            __syncwarp();
          }
          if (lane == 0) {
            umma_commit_pair(&bar_s_full[s], 3);
            if (c == w.c1 - 1) umma_commit_pair(&bar_q_empty, 3);
          }
          __syncwarp();
        }
      }
    } else if (warp == kMmaWarp) {
      // ================= CTA 1: "Q, own rows staged" -> CTA 0 =================
      const uint32_t q_peer = at_leader(&bar_q_peer), kq_peer = at_leader(&bar_kq_peer[0]);
      while (walk.next(p, cid, w)) {
        wait(&bar_q_full, tok & 1u);
        ++tok;
        if (lane == 0) mbar_arrive_peer(q_peer);
        for (int c = w.c0; c < w.c1; ++c, ++g) {
#pragma unroll 1
          for (int q = 0; q < kGroups; ++q) {
            wait(&bar_kq_full[q], g & 1u);
            if (lane == 0) {
              fence_proxy_async_smem();
              mbar_arrive_peer(kq_peer + 8 * q);
            }
          }
        }
      }
    } else if (rank == 0) {
      // ================= P.V issuer (for the pair) =================
      while (walk.next(p, cid, w)) {
        for (int c = w.c0; c < w.c1; ++c, ++g) {
          const bool first = c == w.c0;
          if (first) wait(&bar_o_free, (tok & 1u) ^ 1u);
          wait(&bar_p_full, g & 1u);
#pragma unroll 1
          for (int s = 0; s <= (w.v.second(c) ? 1 : 0); ++s) {
            const uint32_t par = (s == 0 ? g : g1) & 1u;
            wait(&bar_v_full[s], par);
            wait(&bar_v_peer[s], par);
            tc_fence_after();
            if (lane == 0) fence_proxy_async_smem();  // P (st.shared) and the value rows (cp.async): generic proxy
            __syncwarp();
            const uint64_t ad = make_smem_desc(smem_addr(sP + s * kPBytes), 16, 1024, kSwizzle128B);
            const uint64_t bd = make_smem_desc(smem_addr(sV + s * kVBytes), kVBlockBytes, 1024, kSwizzle128B);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int kk = 0; kk < kHalf / 16; ++kk)
                umma_bf16_ss_pair_warp(tmem + kColO + 128 * m, ad + ((kk * 32) >> 4),
                                       bd + ((2 * m * kVBlockBytes + kk * 2048) >> 4), IDESC_PV,
                                       (first && s + kk == 0) ? 0u : 1u);
            if (lane == 0) umma_commit_pair(&bar_pv_done[s], 3);
            __syncwarp();
            if (s == 1) ++g1;
          }
        }
        ++tok;
      }
    } else {
      // ================= CTA 1: "value rows staged" -> CTA 0 =================
      const uint32_t v_peer = at_leader(&bar_v_peer[0]);
      while (walk.next(p, cid, w)) {
        for (int c = w.c0; c < w.c1; ++c, ++g) {
#pragma unroll 1
          for (int s = 0; s <= (w.v.second(c) ? 1 : 0); ++s) {
            wait(&bar_v_full[s], (s == 0 ? g : g1) & 1u);
            if (s == 1) ++g1;
            if (lane == 0) {
              fence_proxy_async_smem();
              mbar_arrive_peer(v_peer + 8 * s);
            }
          }
        }
      }
    }
    if (rank == 0) {
      if (lane == 0) umma_commit_pair(&bar_mma_done, 3);
      __syncwarp();
    }
    // both CTAs: wait for CTA 0's final commits (every MMA that reads this CTA's shared memory or
    // writes its TMEM has completed)
    if (!mbar_wait(&bar_mma_done, 0)) ok = false;
    __syncwarp();
  } else {
    // ================= softmax / epilogue (warps 0-3) =================
    const int kh = warp >> 1;                   // key half of each chunk this warp holds
    const int hl = 32 * (warp & 1) + lane;      // head row within the CTA (TMEM lane 32 warp + lane)
    const int h = kHeads * static_cast<int>(rank) + hl;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const uint32_t s_free_l = at_leader(&bar_s_free[0]), p_full_l = at_leader(&bar_p_full);
    const uint32_t o_free_l = at_leader(&bar_o_free);
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    uint32_t g = 0, g1 = 0;  // chunks, chunks with a second half
    while (walk.next(p, cid, w)) {
      const int32_t* bt = DECODE ? p.block_table + static_cast<int64_t>(w.seq) * p.max_blocks : nullptr;
      float m = -INFINITY, l = 0.f;
      bool bad;
      bool second = w.v.second(w.c0);
      int row[2];
      // of chunk c: column i of this thread's S is key 64 kh + i, or 32 kh + i (i < 32) without a second half
      auto rows_of = [&](int c, bool two) {
        const int e = c * kChunk + (two ? kHalf : 32) * kh + lane;
        row[0] = row_of<DECODE>(p, bt, w, e, bad);
        row[1] = row_of<DECODE>(p, bt, w, two ? e + 32 : w.v.end, bad);
      };
      rows_of(w.c0, second);
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        const int s = static_cast<int>(g & 1u);
        second = w.v.second(c);
        const uint32_t vmask[2] = {__ballot_sync(0xffffffffu, row[0] >= 0), __ballot_sync(0xffffffffu, row[1] >= 0)};
        rows_of(c + 1, w.v.second(c + 1));  // the next chunk's, ahead of its use
        wait(&bar_s_full[s], (g >> 1) & 1u);
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld32(lane_base + kColS + 64 * s, sr[0]);
        tmem_ld32(lane_base + kColS + 64 * s + 32, sr[1]);
        tmem_wait_ld();
        reg_fence(sr[0]);
        reg_fence(sr[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(s_free_l + 8 * s);
        // only a query's last chunk (or a bad page) has masked keys: -inf, so that the maximum, the
        // exponentials and the sums need no masks
        if ((vmask[0] & vmask[1]) != 0xffffffffu) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((vmask[k] >> i) & 1u)) sr[k][i] = 0xff800000u;
        }
        // the row maximum over this half's keys, then with the partner half
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(__uint_as_float(sr[0][j]), __uint_as_float(sr[0][j + 4]));
#pragma unroll
        for (int i = 8; i < 64; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mx[j] = max3(mx[j], __uint_as_float(sr[i >> 5][(i & 31) + j]), __uint_as_float(sr[i >> 5][(i & 31) + j + 4]));
        const float hmax = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        s_red[s][kh][hl] = hmax;
        mlap::pair_sync(warp);
        const float cmax = fmaxf(hmax, s_red[s][kh ^ 1][hl]) * p.scale_log2;  // scale > 0
        bool rescale = false;
        float alpha = 1.f;
        if (c == w.c0) {
          m = cmax;
        } else if (cmax > m + kTau) {
          rescale = m > -INFINITY;  // nothing accumulated yet when every earlier key was masked
          alpha = rescale ? exp2f(m - cmax) : 1.f;
          m = cmax;
        }
        // tcgen05.ld/st are warp-collective: the whole warp runs the rescale if any row needs it
        // (the partner warp decides identically: same heads, same maxima)
        if (__any_sync(0xffffffffu, rescale)) {
          wait(&bar_pv_done[1], (g1 - 1) & 1u);  // the chunk before is whole
          tc_fence_after();
          rescale_o(lane_base + kColO, alpha);
          l *= alpha;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;  // no key seen yet: -inf stays -inf
        const uint64_t neg_m2 = pack2(neg_m, neg_m);
        uint64_t sum2 = 0;
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t* e = &sr[i >> 4][2 * (i & 15)];
          const float2 x = unpack2(fma2(pack2(__uint_as_float(e[0]), __uint_as_float(e[1])), scale2, neg_m2));
          const float a = mla::ex2_approx(x.x), b = mla::ex2_approx(x.y);
          pk[i] = pack_bf16x2(a, b);
          sum2 = add2(sum2, pack2(a, b));
        }
        const float2 sum = unpack2(sum2);
        l += sum.x + sum.y;
        // the P slot is free once its P.V of the chunk before has completed
        const int slot = second ? kh : 0;
        wait(&bar_pv_done[slot], ((slot == 0 ? g : g1) & 1u) ^ 1u);
        uint8_t* prow = sP + slot * kPBytes + hl * 128;
        const int x = (second ? 0 : 4 * kh) ^ (hl & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= 4 && !second) break;
          *reinterpret_cast<uint4*>(prow + ((i ^ x) << 4)) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
        fence_proxy_async_smem();
        if (second) ++g1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(p_full_l);
      }
      // ---- the piece's end: the row sum over both halves, then O ----
      s_red[2][kh][hl] = l;
      mlap::pair_sync(warp);
      const float lt = l + s_red[2][kh ^ 1][hl];
      wait(&bar_pv_done[second ? 1 : 0], ((second ? g1 : g) - 1) & 1u);
      tc_fence_after();
      uint8_t* stage = sP + kh * kPBytes + (warp & 1) * 4096;
      const int head0 = kHeads * static_cast<int>(rank) + 32 * (warp & 1);
      const bool any = lt != 0.f;  // a NaN sum stays a NaN
      if (w.part < 0) {
        store_o<__nv_bfloat16>(lane_base + kColO, any ? 1.f / lt : 0.f, stage, p.out + w.qrow * p.H * 512 + 128 * kh, head0, p.H);
        if (kh == 0 && h < p.H && p.lse != nullptr)
          p.lse[w.qrow * p.H + h] = any ? (m + log2f(lt)) * 0.69314718055994531f : -INFINITY;
      } else {
        const int64_t part = static_cast<int64_t>(w.part) * p.H;
        store_o<float>(lane_base + kColO, 1.f, stage, p.part_o + part * 512 + 128 * kh, head0, p.H);
        if (kh == 0 && h < p.H) {
          p.part_ml[(part + h) * 2] = m;
          p.part_ml[(part + h) * 2 + 1] = lt;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_peer(o_free_l);
    }
  }
  if (!ok) record_device_error(DSA_ERR_TIMEOUT);

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA of the pair still signals or reads the other
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Merges the parts of each split sequence of a shared decode: out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i over the
// clusters that hold chunks of it (the plan tells which).  Parts without a key have l = 0.  A CTA per
// head: its four warps share the parts out, so that few sequences of many parts are merged as fast as
// their parts are read (three sequences of about 25 parts each, whole call: 90 to 98 us with a warp per
// head, 83 to 96 here).
__global__ void __launch_bounds__(128) window_merge_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml,
                                                           const int2* __restrict__ plan, int H,
                                                           __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ float4 s_acc[3][128];
  __shared__ float s_sum[4];
  const int b = blockIdx.y, h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i0 = plan[b].x, i1 = plan[b].y;
  if (i0 == i1) return;  // in one cluster: written there
  // the sequence is the last piece of the cluster it begins in, and the first one of the others
  auto part_of = [&](int i) { return static_cast<int64_t>(2 * i + (i == i0 ? 1 : 0)) * H + h; };
  float M = -INFINITY;
  for (int i = i0 + lane; i <= i1; i += 32) {
    const float2 ml = reinterpret_cast<const float2*>(part_ml)[part_of(i)];
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = i0 + warp; i <= i1; i += 4) {
    const int64_t part = part_of(i);
    const float2 ml = reinterpret_cast<const float2*>(part_ml)[part];
    const float wgt = ml.y == 0.f ? 0.f : exp2f(ml.x - M);
    sum += wgt * ml.y;
    const float4* o = reinterpret_cast<const float4*>(part_o + part * 512) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = o[32 * k];
      acc[k].x = fmaf(wgt, v.x, acc[k].x);
      acc[k].y = fmaf(wgt, v.y, acc[k].y);
      acc[k].z = fmaf(wgt, v.z, acc[k].z);
      acc[k].w = fmaf(wgt, v.w, acc[k].w);
    }
  }
  if (lane == 0) s_sum[warp] = sum;
  if (warp > 0)
#pragma unroll
    for (int k = 0; k < 4; ++k) s_acc[warp - 1][lane + 32 * k] = acc[k];
  __syncthreads();
  if (warp > 0) return;
  sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
  const bool any = sum != 0.f;
  const float inv = any ? 1.f / sum : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(out + (static_cast<int64_t>(b) * H + h) * 512) + lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const float4 v = s_acc[j][lane + 32 * k];
      acc[k].x += v.x;
      acc[k].y += v.y;
      acc[k].z += v.z;
      acc[k].w += v.w;
    }
    dst[32 * k] = make_uint2(dev::pack_bf16x2(acc[k].x * inv, acc[k].y * inv), dev::pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
  }
  if (lse != nullptr && lane == 0)
    lse[static_cast<int64_t>(b) * H + h] = any ? (M + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace dsa
