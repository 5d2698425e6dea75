// Host side of the C ABI declared in include/dsa.h: argument validation, TMA descriptor
// encoding and kernel launches.  Every entry point enqueues on the caller's stream and
// returns without synchronising.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "../../include/dsa.h"
#include "common.cuh"
#include "cache_append.cuh"
#include "indexer.cuh"
#include "quantize.cuh"
#include "attn_probs.cuh"
#include "indexer_bwd.cuh"
#include "indexer_kl.cuh"
#include "selftest.cuh"
#include "mla_common.cuh"
#include "rmsnorm.cuh"
#include "rope.cuh"
#include "sparse_mla_pair.cuh"
#include "topk.cuh"
#include "window_mla.cuh"

namespace dsa {
namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline dsa_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// ---- TMA descriptors (encoded on the host through the driver entry point) -------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D map over a row-major [rows, cols] tensor; box = [box_rows, box_cols].
bool make_map_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t cols, uint64_t rows,
                 uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- lightning indexer -------------------------------------------------------------------
constexpr int kIdxStages = 4;      // key-tile ring depth, scores mode
// Fused top-k mode: the candidate sets need the shared memory.  Up to 128K keys (d_I = 128) the
// key ring has 2 stages and a token holds up to 4608 candidates; longer sequences need the
// third stage for the emission bitmap (which reuses the ring) and hold 4096.  Measured at
// L = 131072: 130.9 ms against 135.4 ms with 3 stages and 4096 (fewer streaming cuts).
constexpr int kIdxStagesTopkShort = 2, kIdxCapShort = 4608, kIdxCapExtraShort = 2560;
constexpr int kIdxStagesTopkLong = 3, kIdxCapLong = 4096, kIdxCapExtraLong = 1024;
constexpr int kIdxTok = 4;            // prefill query tokens per CTA
constexpr int kDecodeTilesPerCta = 32;  // decode: 4096 keys per CTA (measured: 16 -> 32 tiles, -3 % at 64 x ~71K keys, -12 % at 8 x ~127K)

template <int D_I, int H_I, int TOK, int MODE, bool PAGED, int STAGES>
dsa_status launch_indexer_s(const CUtensorMap& qm, const CUtensorMap& km, const IndexerParams& p, dim3 grid,
                            cudaStream_t s) {
  auto kern = indexer_kernel<D_I, H_I, TOK, MODE, PAGED, STAGES>;
  const int smem = indexer_smem_bytes<D_I, H_I, TOK, MODE, STAGES>(p.cap) + 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  kern<<<grid, IdxGroups<TOK>::kThreads, smem, s>>>(qm, km, p);
  return launch_status();
}

// Scores mode: kIdxStages; fused top-k mode: the ring depth `stages` (2 or 3, see above).
template <int D_I, int H_I, int TOK, int MODE, bool PAGED>
dsa_status launch_indexer_t(const CUtensorMap& qm, const CUtensorMap& km, const IndexerParams& p, dim3 grid,
                            cudaStream_t s, int stages) {
  if constexpr (MODE == kIdxTopk) {
    if (stages == kIdxStagesTopkShort)
      return launch_indexer_s<D_I, H_I, TOK, MODE, PAGED, kIdxStagesTopkShort>(qm, km, p, grid, s);
    return launch_indexer_s<D_I, H_I, TOK, MODE, PAGED, kIdxStagesTopkLong>(qm, km, p, grid, s);
  } else {
    return launch_indexer_s<D_I, H_I, TOK, MODE, PAGED, kIdxStages>(qm, km, p, grid, s);
  }
}

// Ring depth and candidate capacity of the fused top-k for sequences of up to max_seqlen keys
// (the final ascending emission uses a bitmap of the causal prefix inside the key ring, half of
// it per epilogue group); DSA_ERR_UNSUPPORTED when the bitmap does not fit three stages.
dsa_status topk_config(int d_I, int max_seqlen, int k, int* stages, int* cap) {
  const int64_t bitmap_bytes = (static_cast<int64_t>(max_seqlen) + 31) / 32 * 4;
  const int64_t stage_bytes = 128 * static_cast<int64_t>(d_I);
  if (max_seqlen > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  int extra, cmax;
  if (bitmap_bytes <= kIdxStagesTopkShort * stage_bytes / 2) {
    *stages = kIdxStagesTopkShort;
    extra = kIdxCapExtraShort;
    cmax = kIdxCapShort;
  } else if (bitmap_bytes <= kIdxStagesTopkLong * stage_bytes / 2) {
    *stages = kIdxStagesTopkLong;
    extra = kIdxCapExtraLong;
    cmax = kIdxCapLong;
  } else {
    return DSA_ERR_UNSUPPORTED;
  }
  *cap = k + extra < 2 * k ? 2 * k : k + extra;
  if (*cap > cmax) *cap = cmax;
  return DSA_OK;
}

template <int MODE, bool PAGED>
dsa_status launch_indexer(int d_I, int H_I, const CUtensorMap& qm, const CUtensorMap& km, const IndexerParams& p,
                          dim3 grid, cudaStream_t s, int stages = 0) {
  constexpr int TOK = PAGED ? 1 : kIdxTok;
  if constexpr (PAGED) {
    if (H_I != 64) return DSA_ERR_UNSUPPORTED;
    if (d_I == 128) return launch_indexer_t<128, 64, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
    if (d_I == 64) return launch_indexer_t<64, 64, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
    return DSA_ERR_UNSUPPORTED;
  } else {
    if (d_I == 128 && H_I == 64) return launch_indexer_t<128, 64, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
  if (d_I == 64 && H_I == 64) return launch_indexer_t<64, 64, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
  if (d_I == 128 && H_I == 4) return launch_indexer_t<128, 4, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
  if (d_I == 64 && H_I == 4) return launch_indexer_t<64, 4, TOK, MODE, PAGED>(qm, km, p, grid, s, stages);
  return DSA_ERR_UNSUPPORTED;
  }
}

bool indexer_shape_ok(int H_I, int d_I) { return (H_I == 4 || H_I == 64) && (d_I == 64 || d_I == 128); }

// Validates the common indexer arguments and builds the Q / K tensor maps.
// q_rows: rows held by the query arrays (prefill: the packed tokens they cover; 0 = all of them)
dsa_status indexer_common(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                          const dsa_kv_desc* keys, int32_t B, int32_t H_I, int32_t d_I, CUtensorMap* qm,
                          CUtensorMap* km, IndexerParams* p, int64_t q_rows = 0) {
  if (q_fp8 == nullptr || q_scale == nullptr || w == nullptr || keys == nullptr || keys->data == nullptr ||
      keys->scale == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (q_scale_heads != 1 && q_scale_heads != H_I) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q_fp8, 16) || !aligned(keys->data, 16)) return DSA_ERR_INVALID_ARGUMENT;
  if (!indexer_shape_ok(H_I, d_I)) return DSA_ERR_UNSUPPORTED;
  const CUtensorMapSwizzle sw = d_I == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  std::memset(p, 0, sizeof(*p));
  p->tok_begin = 0;
  p->tok_end = 0x7FFFFFFF;
  p->q_row0 = 0;
  p->q_scale = q_scale;
  p->q_scale_heads = q_scale_heads;
  p->w = w;
  p->k_scale = keys->scale;
  if (keys->kind == DSA_KV_CONTIGUOUS) {
    if (keys->cu_seqlens == nullptr || keys->total_tokens <= 0 || keys->max_seqlen <= 0) return DSA_ERR_INVALID_ARGUMENT;
    if (keys->total_tokens * H_I > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
    const uint64_t T = static_cast<uint64_t>(keys->total_tokens);
    const uint64_t TQ = q_rows > 0 ? static_cast<uint64_t>(q_rows) : T;
    if (!make_map_2d(qm, q_fp8, CU_TENSOR_MAP_DATA_TYPE_UINT8, d_I, TQ * H_I, d_I, d_I, kIdxTok * H_I, sw) ||
        !make_map_2d(km, keys->data, CU_TENSOR_MAP_DATA_TYPE_UINT8, d_I, T, d_I, d_I, 128, sw))
      return DSA_ERR_INVALID_ARGUMENT;
    p->cu_seqlens = keys->cu_seqlens;
  } else if (keys->kind == DSA_KV_PAGED) {
    if (keys->block_table == nullptr || keys->context_lens == nullptr || keys->num_blocks <= 0 ||
        keys->max_blocks_per_seq <= 0 || keys->max_seqlen <= 0)
      return DSA_ERR_INVALID_ARGUMENT;
    if (keys->block_size != 64 || H_I != 64) return DSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(keys->max_seqlen) > static_cast<int64_t>(keys->max_blocks_per_seq) * 64)
      return DSA_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(keys->num_blocks) * 64 > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
    const uint64_t rows = static_cast<uint64_t>(keys->num_blocks) * 64;
    if (!make_map_2d(qm, q_fp8, CU_TENSOR_MAP_DATA_TYPE_UINT8, d_I, static_cast<uint64_t>(B) * H_I, d_I, d_I, H_I,
                     sw) ||
        !make_map_2d(km, keys->data, CU_TENSOR_MAP_DATA_TYPE_UINT8, d_I, rows, d_I, d_I, 64, sw))
      return DSA_ERR_INVALID_ARGUMENT;
    p->block_table = keys->block_table;
    p->context_lens = keys->context_lens;
    p->max_blocks_per_seq = keys->max_blocks_per_seq;
    p->num_blocks = keys->num_blocks;
    p->max_len = keys->max_seqlen;  // validated above: 0 < max_seqlen <= 64 * max_blocks_per_seq
    p->tiles_per_cta = kDecodeTilesPerCta;
  } else {
    return DSA_ERR_INVALID_ARGUMENT;
  }
  return DSA_OK;
}

// ---- sparse MLA ------------------------------------------------------------------------------
constexpr int kMlaClusters = 74;   // one CTA pair per two SMs of a 148-SM B200
constexpr int kLatentDim = 576, kValueDim = 512;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t decode_partials_bytes(int B, int H, int splits) {
  return align256(static_cast<size_t>(B) * splits * H * kValueDim * 4) + align256(static_cast<size_t>(B) * splits * H * 2 * 4);
}

// Decode divides each sequence's selection into `splits` work units of whole 64-row chunks,
// merged afterwards by a log-sum-exp combine.  Splitting pays only while the units still fit
// one round on the CTA pairs: each unit costs a Q load, an O readout and fp32 partials, and
// every chunk of a unit is one step of the same latency chain.  So splits is the largest power
// of two s with B * s <= the number of CTA pairs (one round) and s <= k / 64 (a chunk per
// unit), at least 1.  With one split the kernel writes out and lse itself (no partials, no
// combine).  Measured on a B200 for 64 sequences, k = 2048 (MLA + combine, the latent-split
// kernel that preceded the head-split pair): 1 split 100 us, 2 splits 117 us, 4 splits 151 us,
// 8 splits 221 us.
int decode_splits(int B, int k) {
  int s = 1;
  while (2 * s <= k / 64 && static_cast<int64_t>(B) * 2 * s <= kMlaClusters) s *= 2;
  return s;
}

// Sparse prefill, masked prefill and decode: the head-split pair kernel.  Q is read by TMA as a
// [q_rows * H, 576] bf16 matrix in 64 x 64 tiles (128-byte swizzle).
template <bool DECODE, bool MASKED = false>
dsa_status launch_mla_pair(const void* latent, const void* q, int64_t q_rows, const MlaParams& p, int64_t units,
                           cudaStream_t s) {
  CUtensorMap qm;
  if (!make_map_2d(&qm, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kLatentDim, static_cast<uint64_t>(q_rows) * p.H,
                   kLatentDim * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_INVALID_ARGUMENT;
  auto kern = sparse_mla_pair_kernel<DECODE, MASKED>;
  const int smem = mlap::kSmemBytes + 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const int clusters = static_cast<int>(units < kMlaClusters ? units : kMlaClusters);
  kern<<<2 * clusters, mlap::kThreads, smem, s>>>(static_cast<const __nv_bfloat16*>(latent), p, qm);
  return launch_status();
}

// ---- window MLA --------------------------------------------------------------------------------
// Whether decode shares the chunks of all sequences out over the clusters (and merges the split
// sequences) instead of giving each cluster whole sequences.  In chunks' times: whole sequences take
// rounds of (chunks + kUnitCost); shared, the even share, an eighth of it and 8 for what splits add (a
// second piece of work per cluster, fp32 partial outputs, the merge).  By the longest context the
// arguments allow: the contexts themselves are on the device, so a batch far below it pays for the sharing.
// Measured (us on the device, contexts at the longest, shared / whole): 8 sequences of 512 keys 16.0 / 16.1; of 1024 keys 8: 18.6 / 23.3, 24:
// 24.8 / 23.7; of 2048 keys 16: 25 / 38, 40: 46 / 40, 96: 85 / 87; of 4096 keys 48: 78 / 81, 64: 101 / 87, 112: 162 / 178,
// 128: 187 / 185; of 8192 keys 56: 149 / 182, 64: 189 / 180.
constexpr int kShareSeqs = 1024;  // a cluster's start is found by a scan of the contexts

bool window_shared(int B, int window, int sinks, int max_ctx) {
  const int64_t keys = std::min<int64_t>(max_ctx, static_cast<int64_t>(window) + sinks);
  const int64_t chunks = (keys + win::kChunk - 1) / win::kChunk;
  if (B > kShareSeqs || chunks < 2) return false;
  const int64_t whole = (B + kMlaClusters - 1) / kMlaClusters * (chunks + win::kUnitCost);
  const int64_t share = B * (chunks + win::kUnitCost) / kMlaClusters;
  return share + share / 8 + 8 < whole;
}

size_t window_plan_bytes(int B) { return align256(static_cast<size_t>(B) * sizeof(int2)); }
size_t window_part_bytes(int H) { return align256(static_cast<size_t>(2 * kMlaClusters) * H * kValueDim * 4); }

template <bool DECODE>
dsa_status launch_window(const void* latent, const void* q, const WinParams& p, int64_t clusters, cudaStream_t s) {
  CUtensorMap qm;
  if (!make_map_2d(&qm, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kLatentDim, static_cast<uint64_t>(p.rows) * p.H, kLatentDim * 2,
                   64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_INVALID_ARGUMENT;
  auto kern = window_mla_kernel<DECODE>;
  const int smem = win::kSmemBytes + 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return DSA_ERR_CUDA;
  kern<<<static_cast<unsigned>(2 * std::min<int64_t>(clusters, kMlaClusters)), win::kThreads, smem, s>>>(
      static_cast<const __nv_bfloat16*>(latent), p, qm);
  return launch_status();
}

bool mla_shape_ok(int H, int k) { return H >= 1 && H <= 128 && k >= 64 && k <= 2048 && k % 64 == 0; }

// ---- row operators: norm, rotary positions, cache append ---------------------------------------
// Times here are of the device alone, calls back to back on one set of buffers (of which L2 keeps a part).
constexpr int kSms = 148;
constexpr int kMostCols = 1 << 30;  // columns of a row: the kernels' column numbers, a step past the row's end, fit an int

bool dtype_ok(int32_t dtype) { return dtype == DSA_BF16 || dtype == DSA_F16 || dtype == DSA_F32; }
size_t dtype_size(int32_t dtype) { return dtype == DSA_F32 ? 4 : 2; }

// Calls f with a null pointer of the element type of `dtype`.
template <typename F>
dsa_status with_dtype(int32_t dtype, F f) {
  if (dtype == DSA_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  if (dtype == DSA_F16) return f(static_cast<__half*>(nullptr));
  return f(static_cast<float*>(nullptr));
}

// The largest piece (8, 4, 2 or 1 elements of `size` bytes) that a row of cols is made of and that every
// operand (null: absent) holds at its alignment.
struct Operand {
  const void* p;
  int64_t ld;
};
int piece_of(int cols, size_t size, std::initializer_list<Operand> operands, const void* codes) {
  for (int v = 8; v > 1; v /= 2) {
    bool ok = cols % v == 0 && aligned(codes, v);
    for (const Operand& o : operands) ok = ok && (o.p == nullptr || (aligned(o.p, std::min<size_t>(v * size, 16)) && o.ld % v == 0));
    if (ok) return v;
  }
  return 1;
}

// An output that is an input itself has its row stride too.
bool same_rows(const void* out, int64_t ld_out, const void* in, int64_t ld_in) {
  return out == nullptr || out != in || ld_out == ld_in;
}

// Threads for a CTA-wide row of cols columns, ch pieces of v per thread.
int row_threads(int cols, int v, int ch) { return (cols + 32 * v * ch - 1) / (32 * v * ch) * 32; }

template <typename T, int V, int CH, int LANES>
dsa_status launch_rmsnorm_v(const NormParams& p, cudaStream_t s) {
  if constexpr (LANES > 0) {
    constexpr int kRows = norm::kWarps * 32 / LANES;
    rmsnorm_kernel<T, V, CH, LANES><<<static_cast<unsigned>((p.rows + kRows - 1) / kRows), norm::kWarps * 32, 0, s>>>(p);
  } else {
    rmsnorm_kernel<T, V, CH, 0><<<static_cast<unsigned>(p.rows), row_threads(p.cols, V, CH), 0, s>>>(p);
  }
  return launch_status();
}

// Pieces of 4, 2 or 1 elements.  Up to 512 columns a warp per row, beyond that a CTA with 16 elements per
// thread (bf16, CTA against warp: 65536 x 1001 64.5 us against 70.4, x 1004 67 against 88; with residual and codes
// 172 against 242; but x 500 45 against 37.  8 per thread: 20000 x 3001 72 against 64, x 7004 337 against 189).  Few
// rows whose codes wait for a group's maximum: 8 elements per thread (64 x 501 with codes by groups 3.1 us against
// 4.7 with a warp, x 3001 3.8 against 4.7 with 16).
template <typename T, int V>
dsa_status launch_rmsnorm_small(const NormParams& p, cudaStream_t s) {
  constexpr int kMin = V == 4 ? 1 : 4 / V;  // pieces per lane that make whole groups of 128 columns
  if (p.cols <= 128) return launch_rmsnorm_v<T, V, kMin, 32>(p, s);
  if (p.cols <= 256) return launch_rmsnorm_v<T, V, 2 * kMin, 32>(p, s);
  if (p.codes != nullptr && p.rows <= 4 * kSms && p.cols <= 8192) return launch_rmsnorm_v<T, V, 2 * kMin, 0>(p, s);
  if (p.cols <= 512) return launch_rmsnorm_v<T, V, 4 * kMin, 32>(p, s);
  if (p.cols <= 16384) return launch_rmsnorm_v<T, V, 4 * kMin, 0>(p, s);
  rmsnorm_general_kernel<T><<<static_cast<unsigned>(p.rows), norm::kGeneralThreads, 0, s>>>(p);
  return launch_status();
}

template <typename T>
dsa_status launch_rmsnorm(const NormParams& p, int piece, cudaStream_t s) {
  if (piece == 1) return launch_rmsnorm_small<T, 1>(p, s);
  if (piece == 2) return launch_rmsnorm_small<T, 2>(p, s);
  if (piece == 4) return launch_rmsnorm_small<T, 4>(p, s);
  const int n = p.cols / 8;
  if (n <= 8) return launch_rmsnorm_v<T, 8, 1, 8>(p, s);
  if (n <= 16) return launch_rmsnorm_v<T, 8, 1, 16>(p, s);
  if (n <= 32) return launch_rmsnorm_v<T, 8, 1, 32>(p, s);
  if (n <= 64) return launch_rmsnorm_v<T, 8, 2, 32>(p, s);
  if (n <= 128) return launch_rmsnorm_v<T, 8, 4, 32>(p, s);
  // Few rows: as many threads as there are pieces.  Many: the loads of a whole row in flight in as few
  // threads as its registers allow, which lets more rows share an SM (16-bit types: 4 pieces per thread,
  // where that fills the last warp: 11502 x 3840 33.5 us against 39.6 with 2, 16384 x 8192 with residual
  // and codes 167 against 202, but 32768 x 1536, 48 of 64 threads, 82 against 74; fp32: 2, 16384 x 4096
  // 177 us against 196).
  if (n <= 1024 && p.rows <= kSms) return launch_rmsnorm_v<T, 8, 1, 0>(p, s);
  const bool four = sizeof(T) == 2 && 10 * n >= 9 * 4 * row_threads(p.cols, 8, 4);
  if (n <= 2 * 1024 && !four) return launch_rmsnorm_v<T, 8, 2, 0>(p, s);
  if (n <= 4 * 1024) return launch_rmsnorm_v<T, 8, 4, 0>(p, s);
  rmsnorm_general_kernel<T><<<static_cast<unsigned>(p.rows), norm::kGeneralThreads, 0, s>>>(p);
  return launch_status();
}

int norm_bwd_per_sm(int cols, size_t size) {
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(16384 / (static_cast<int64_t>(cols) * size), 1), 16));
}
// CTAs of the backward, each of which writes one row of partial sums of dw: enough per SM to hide a
// row's reduction (about 16 KB of rows: 32768 x 2048 bf16 88 us with 4, 100 with 2; 16384 x 4096 fp32 159
// with 1, 172 with 2), at most one per row.
int64_t norm_bwd_ctas(int64_t rows, int cols, size_t size) {
  const int64_t most = static_cast<int64_t>(kSms) * norm_bwd_per_sm(cols, size);
  return rows < most ? rows : most;
}

dsa_status launch_dw(const NormBwdParams& p, int64_t ctas, float* dw, cudaStream_t s) {
  const dsa_status st = launch_status();
  if (st != DSA_OK) return st;
  rmsnorm_dw_kernel<<<(p.cols + 31) / 32, 1024, 0, s>>>(p.part, static_cast<int>(ctas), p.cols, dw);
  return launch_status();
}

template <typename T, int V, int CH, int LANES>
dsa_status launch_rmsnorm_backward_v(const NormBwdParams& p, float* dw, cudaStream_t s) {
  int64_t ctas = norm_bwd_ctas(p.rows, p.cols, sizeof(T));
  if constexpr (LANES > 0) {
    constexpr int kRows = norm::kWarps * 32 / LANES;
    ctas = std::min<int64_t>(std::min<int64_t>(ctas, 4 * kSms), (p.rows + kRows - 1) / kRows);
    rmsnorm_backward_kernel<T, V, CH, LANES><<<static_cast<unsigned>(ctas), norm::kWarps * 32, 0, s>>>(p);
  } else {
    rmsnorm_backward_kernel<T, V, CH, 0><<<static_cast<unsigned>(ctas), row_threads(p.cols, V, CH), 0, s>>>(p);
  }
  return launch_dw(p, ctas, dw, s);
}

template <typename T, int V>
dsa_status launch_rmsnorm_backward_small(const NormBwdParams& p, float* dw, cudaStream_t s) {
  constexpr int kMin = 4 / V;  // pieces of 128 columns
  // a warp per row as long as its registers leave room for many (65536 x 250 bf16 39.4 us against 47 with a CTA
  // per row, 65536 x 201 fp32 41.9 against 51.6; but 65536 x 500 bf16 167 against 90)
  if (p.cols <= 128) return launch_rmsnorm_backward_v<T, V, kMin, 32>(p, dw, s);
  if (p.cols <= 256) return launch_rmsnorm_backward_v<T, V, 2 * kMin, 32>(p, dw, s);
  if (p.cols <= 4096) return launch_rmsnorm_backward_v<T, V, kMin, 0>(p, dw, s);
  if (p.cols <= 8192) return launch_rmsnorm_backward_v<T, V, 2 * kMin, 0>(p, dw, s);
  const int64_t ctas = norm_bwd_ctas(p.rows, p.cols, sizeof(T));
  rmsnorm_backward_general_kernel<T><<<static_cast<unsigned>(ctas), norm::kGeneralThreads, 0, s>>>(p);
  return launch_dw(p, ctas, dw, s);
}

template <typename T>
dsa_status launch_rmsnorm_backward(const NormBwdParams& p, int piece, float* dw, cudaStream_t s) {
  if (piece == 1) return launch_rmsnorm_backward_small<T, 1>(p, dw, s);
  if (piece == 2) return launch_rmsnorm_backward_small<T, 2>(p, dw, s);
  if (piece == 4) return launch_rmsnorm_backward_small<T, 4>(p, dw, s);
  const int n = p.cols / 8;
  if (n <= 8) return launch_rmsnorm_backward_v<T, 8, 1, 8>(p, dw, s);
  if (n <= 16) return launch_rmsnorm_backward_v<T, 8, 1, 16>(p, dw, s);
  if (n <= 32) return launch_rmsnorm_backward_v<T, 8, 1, 32>(p, dw, s);
  const int64_t stage = static_cast<int64_t>(p.cols) * sizeof(T) * (p.dres != nullptr ? 3 : 2);
  const int stages = static_cast<int>(std::min<int64_t>(norm::kRingBytes / norm_bwd_per_sm(p.cols, sizeof(T)) / stage, norm::kRingMax));
  const int64_t ctas = norm_bwd_ctas(p.rows, p.cols, sizeof(T));
  if (n <= 1024 && stages >= 2) {
    const int smem = static_cast<int>(stages * stage);
    // the same limit for every size, so that calls from several host threads do not lower one another's
    if (cudaFuncSetAttribute(rmsnorm_backward_ring_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, norm::kRingBytes) !=
        cudaSuccess)
      return DSA_ERR_CUDA;
    rmsnorm_backward_ring_kernel<T><<<static_cast<unsigned>(ctas), row_threads(p.cols, 8, 1), smem, s>>>(p, stages);
    return launch_dw(p, ctas, dw, s);
  }
  // beyond the ring: registers for two pieces of three operands and the row ahead, with spills at 1024 threads (8192 x
  // 12288 bf16 with the residual's gradient 262 us, 0.47 of measured HBM; x 16384 299, 0.55; x 12288 fp32 661, 0.37)
  if (n <= 2 * 1024) return launch_rmsnorm_backward_v<T, 8, 2, 0>(p, dw, s);
  rmsnorm_backward_general_kernel<T><<<static_cast<unsigned>(ctas), norm::kGeneralThreads, 0, s>>>(p);
  return launch_dw(p, ctas, dw, s);
}

// piece: elements that heads, strides and pointers divide into (8, 4, 2 or 1).
template <typename T>
dsa_status launch_rope(RopeParams p, int piece, cudaStream_t s) {
  const int pairs = p.rot / 2;
  const int rest = p.copy_rest ? p.dim - p.rot : 0;
  // the rotated range (in the half layout each of its halves) made of whole pieces, of 8 or of 4
  auto in_pieces = [&](int v) { return piece >= v && p.rot0 % v == 0 && (p.half_layout ? pairs : p.rot) % v == 0; };
  const int whole = in_pieces(8) ? 8 : in_pieces(4) ? 4 : 0;
  if (whole != 0) {
    p.items = (p.half_layout ? pairs : p.rot) / whole + rest / whole;
  } else if (p.copy_rest) {
    const int from = p.rot0 / piece * piece, to = (p.rot0 + p.rot + piece - 1) / piece * piece;
    p.items = pairs + (to - from - p.rot) + (p.dim - (to - from)) / piece;
  } else {
    p.items = pairs;
    piece = 1;
  }
  p.lanes = std::min(p.items, rope::kThreads);
  // groups per CTA: as many as fit, but a divisor of the heads when that costs less than half
  p.groups = rope::kThreads / p.lanes;
  for (int g = p.groups; 2 * g > p.groups; --g)
    if (p.heads % g == 0) {
      p.groups = g;
      break;
    }
  // A CTA walks one batch of (row, head) pairs, or with small pieces some: several rows when a row has
  // fewer, a range of a row's heads when it has more (each CTA makes its own table of rot / 2 entries per
  // row).
  const int batch = p.groups * rope::unroll<T>() * (whole == 8 ? 1 : 2);
  int64_t parts = 1;
  p.rows_per_cta = 1;
  p.heads_per_cta = p.heads;
  if (p.heads >= 2 * batch) {
    p.heads_per_cta = static_cast<int32_t>(std::max<int64_t>(batch, (p.heads + 65534) / 65535));
    parts = (p.heads + p.heads_per_cta - 1) / p.heads_per_cta;
  } else {
    int64_t r = std::min<int64_t>(batch / p.heads, rope::kTable / pairs);
    r = std::min<int64_t>(r, (p.rows + kSms - 1) / kSms);  // few rows: over the GPU first
    p.rows_per_cta = static_cast<int32_t>(std::max<int64_t>(1, r));
  }
  const int64_t ctas = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(parts));
  const int threads = (p.groups * p.lanes + 31) / 32 * 32;
  auto launch = [&](auto kern) { kern<<<grid, threads, 0, s>>>(p); };
  if (whole == 8) launch(p.half_layout ? rope_kernel<T, 8, true> : rope_kernel<T, 8, false>);
  else if (whole == 4) launch(p.half_layout ? rope_kernel<T, 4, true> : rope_kernel<T, 4, false>);
  else if (piece == 8) launch(rope_pairs_kernel<T, 8>);
  else if (piece == 4) launch(rope_pairs_kernel<T, 4>);
  else if (piece == 2) launch(rope_pairs_kernel<T, 2>);
  else launch(rope_pairs_kernel<T, 1>);
  return launch_status();
}

// One cache of dsa_cache_append from its descriptor.
dsa_status append_cache(const dsa_kv_desc* d, bool with_scale, size_t align, AppendCache* c) {
  if (d->data == nullptr || !aligned(d->data, align) || (with_scale && (d->scale == nullptr || !aligned(d->scale, 4))) ||
      d->max_seqlen <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  c->data = const_cast<void*>(d->data);
  c->scale = const_cast<float*>(d->scale);
  c->max_seqlen = d->max_seqlen;
  if (d->kind == DSA_KV_CONTIGUOUS) {
    if (d->cu_seqlens == nullptr || d->total_tokens <= 0) return DSA_ERR_INVALID_ARGUMENT;
    if (d->total_tokens > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
    c->cu = d->cu_seqlens;
    c->rows = static_cast<int32_t>(d->total_tokens);
    return DSA_OK;
  }
  if (d->kind != DSA_KV_PAGED || d->block_table == nullptr || d->num_blocks <= 0 || d->max_blocks_per_seq <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (d->block_size != 64 || static_cast<int64_t>(d->num_blocks) * 64 > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  c->table = d->block_table;
  c->rows = d->num_blocks;
  c->max_blocks = d->max_blocks_per_seq;
  return DSA_OK;
}

// ---- decode with library-held scratch (no allocation on the call path) ---------------------
// One array per device, in this translation unit.  Host code cannot pass the symbol itself to
// a kernel (on the host it is only a stand-in), so each device's address is looked up once,
// with that device current, and cached.
static __device__ __align__(256) uint8_t g_noalloc_scratch[DSA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 256;

dsa_status noalloc_scratch(void** ptr) {
  static std::mutex mu;
  static void* addr[kMaxDevices] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (addr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return DSA_ERR_CUDA;
    addr[dev] = p;
  }
  *ptr = addr[dev];
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

const char* dsa_status_string(int32_t status) {
  switch (status) {
    case DSA_OK: return "ok";
    case DSA_ERR_INVALID_ARGUMENT: return "invalid argument";
    case DSA_ERR_UNSUPPORTED: return "unsupported shape or configuration";
    case DSA_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case DSA_ERR_CUDA: return "CUDA error";
    case DSA_ERR_TIMEOUT: return "device-side wait timed out";
    case DSA_ERR_DEVICE_CHECK: return "device-side input check failed";
    default: return "unknown status";
  }
}

dsa_status dsa_device_error(int32_t* code, void* stream) {
  if (code == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  cudaStream_t s = as_stream(stream);
  int32_t v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_device_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return DSA_ERR_CUDA;
  const int32_t zero = 0;
  if (cudaMemcpyToSymbolAsync(g_device_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return DSA_ERR_CUDA;
  *code = v;
  return DSA_OK;
}

dsa_status dsa_attn_distribution(const void* q, const dsa_kv_desc* latent, const int32_t* idx, const float* lse,
                                 int32_t B, int32_t H, int32_t k, float sm_scale, float* p_out, void* stream) {
  if (q == nullptr || latent == nullptr || latent->data == nullptr || idx == nullptr || lse == nullptr ||
      p_out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr || latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16)) return DSA_ERR_INVALID_ARGUMENT;
  if (H < 1 || H > 128 || k < 64 || k > 2048 || k % 64 != 0) return DSA_ERR_UNSUPPORTED;
  ProbsParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.idx = idx;
  p.lse = lse;
  p.cu_seqlens = latent->cu_seqlens;
  p.B = B;
  p.H = H;
  p.k = k;
  p.rows = latent->total_tokens;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.p = p_out;
  const int smem = probs::kSmemBytes + 1024;
  if (cudaFuncSetAttribute(attn_probs_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const int64_t grid = p.rows < 148 ? p.rows : 148;
  attn_probs_kernel<false><<<static_cast<unsigned>(grid), probs::kThreads, smem, as_stream(stream)>>>(
      static_cast<const __nv_bfloat16*>(latent->data), p);
  return launch_status();
}

dsa_status dsa_attn_distribution_dense(const void* q, const dsa_kv_desc* latent, const float* lse, int32_t B,
                                       int32_t H, int64_t row_begin, int64_t row_end, float sm_scale, float* p_out,
                                       int64_t ld_p, void* stream) {
  if (latent == nullptr || row_begin < 0 || row_end < row_begin) return DSA_ERR_INVALID_ARGUMENT;
  if (row_end == row_begin) return DSA_OK;
  if (q == nullptr || latent->data == nullptr || lse == nullptr || p_out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr || latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (row_end > latent->total_tokens || ld_p < latent->max_seqlen) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16)) return DSA_ERR_INVALID_ARGUMENT;
  if (H < 1 || H > 128) return DSA_ERR_UNSUPPORTED;
  ProbsParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.lse = lse;
  p.cu_seqlens = latent->cu_seqlens;
  p.B = B;
  p.H = H;
  p.rows = row_end - row_begin;
  p.row0 = row_begin;
  p.ld = ld_p;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.p = p_out;
  const int smem = probs::kSmemBytes + 1024;
  if (cudaFuncSetAttribute(attn_probs_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const int64_t grid = p.rows < 148 ? p.rows : 148;
  attn_probs_kernel<true><<<static_cast<unsigned>(grid), probs::kThreads, smem, as_stream(stream)>>>(
      static_cast<const __nv_bfloat16*>(latent->data), p);
  return launch_status();
}

dsa_status dsa_indexer_backward(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                                const dsa_kv_desc* keys, int32_t B, int32_t H_I, int32_t d_I, const int32_t* idx,
                                const float* grad, int32_t k, float* dw, float* dq, float* dk, void* stream) {
  if (keys == nullptr || k <= 0 || B <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (keys->kind != DSA_KV_CONTIGUOUS) return DSA_ERR_UNSUPPORTED;
  if (q_fp8 == nullptr || q_scale == nullptr || w == nullptr || keys->data == nullptr || keys->scale == nullptr ||
      keys->cu_seqlens == nullptr || keys->total_tokens <= 0 || idx == nullptr || grad == nullptr || dw == nullptr ||
      dq == nullptr || dk == nullptr)
    return DSA_ERR_INVALID_ARGUMENT;
  if (q_scale_heads != 1 && q_scale_heads != H_I) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(keys->data, 4) || !aligned(dk, 16) || !aligned(dq, 16)) return DSA_ERR_INVALID_ARGUMENT;
  if (!indexer_shape_ok(H_I, d_I)) return DSA_ERR_UNSUPPORTED;
  IdxBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.q8 = q_fp8;
  p.q_scale = q_scale;
  p.q_scale_heads = q_scale_heads;
  p.w = w;
  p.k8 = static_cast<const uint8_t*>(keys->data);
  p.k_scale = keys->scale;
  p.cu_seqlens = keys->cu_seqlens;
  p.B = B;
  p.idx = idx;
  p.grad = grad;
  p.k = k;
  p.rows = keys->total_tokens;
  p.dw = dw;
  p.dq = dq;
  p.dk = dk;
  cudaStream_t s = as_stream(stream);
  if (cudaMemsetAsync(dk, 0, static_cast<size_t>(keys->total_tokens) * d_I * sizeof(float), s) != cudaSuccess)
    return DSA_ERR_CUDA;
  auto launch = [&](auto kern, int smem) -> dsa_status {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return DSA_ERR_CUDA;
    const int64_t grid = p.rows < 2 * 148 ? p.rows : 2 * 148;
    kern<<<static_cast<unsigned>(grid), ibwd::kThreads, smem, s>>>(p);
    return launch_status();
  };
  if (H_I == 64 && d_I == 128) return launch(indexer_backward_h64_kernel<128>, ibwd::Layout64<128>::kSmemBytes);
  if (H_I == 64 && d_I == 64) return launch(indexer_backward_h64_kernel<64>, ibwd::Layout64<64>::kSmemBytes);
  if (H_I == 4 && d_I == 128) return launch(indexer_backward_kernel<4, 128>, ibwd::Layout<4, 128>::kSmemBytes);
  return launch(indexer_backward_kernel<4, 64>, ibwd::Layout<4, 64>::kSmemBytes);
}

dsa_status dsa_indexer_kl(const float* p, const float* scores, const int32_t* idx, int64_t rows, int32_t k,
                          float* loss, float* grad, void* stream) {
  if (rows < 0 || k <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA_OK;
  if (p == nullptr || scores == nullptr || idx == nullptr || loss == nullptr || grad == nullptr)
    return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  indexer_kl_kernel<<<static_cast<unsigned>(rows), kl::kThreads, 0, as_stream(stream)>>>(p, scores, idx, k, loss, grad);
  return launch_status();
}

dsa_status dsa_selftest_wait_timeout(int32_t limit_us, void* stream) {
  if (limit_us <= 0 || limit_us > 2000000) return DSA_ERR_INVALID_ARGUMENT;
  wait_timeout_selftest_kernel<<<1, 32, 0, as_stream(stream)>>>(static_cast<uint64_t>(limit_us) * 1000u);
  return launch_status();
}

dsa_status dsa_quantize_fp8(const void* x_bf16, int64_t rows, int32_t cols, uint8_t* codes, float* scale,
                            void* stream) {
  if (rows < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA_OK;
  if (cols <= 0 || (cols % 8) != 0) return DSA_ERR_INVALID_ARGUMENT;
  if (x_bf16 == nullptr || codes == nullptr || scale == nullptr || !aligned(x_bf16, 16) || !aligned(codes, 8))
    return DSA_ERR_INVALID_ARGUMENT;
  if (cols >= 2048 && cols <= quant::kWideThreads * quant::kWideMaxChunks * 8) {
    if (rows > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
    quantize_fp8_wide_kernel<<<static_cast<unsigned>(rows), quant::kWideThreads, 0, as_stream(stream)>>>(
        static_cast<const __nv_bfloat16*>(x_bf16), cols, codes, scale);
    return launch_status();
  }
  const int64_t blocks = (rows + quant::kWarps - 1) / quant::kWarps;
  if (blocks > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  quantize_fp8_rows_kernel<<<static_cast<unsigned>(blocks), quant::kWarps * 32, 0, as_stream(stream)>>>(
      static_cast<const __nv_bfloat16*>(x_bf16), rows, cols, codes, scale);
  return launch_status();
}

dsa_status dsa_topk(const float* scores, int64_t ld_scores, int64_t rows, const int32_t* row_len, int32_t k,
                    int32_t* idx, void* stream) {
  if (rows < 0 || k <= 0 || ld_scores <= 0 || (ld_scores % 4) != 0) return DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA_OK;
  if (scores == nullptr || row_len == nullptr || idx == nullptr || !aligned(scores, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 0x7FFFFFFFLL || ld_scores > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  if (rows * kTopkCluster > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  topk_rows_cluster_kernel<<<static_cast<unsigned>(rows * kTopkCluster), kTopkThreads, 0, as_stream(stream)>>>(
      scores, ld_scores, row_len, k, idx);
  return launch_status();
}

dsa_status dsa_indexer_scores(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                              const dsa_kv_desc* keys, int32_t B, int32_t H_I, int32_t d_I, int64_t row_begin,
                              int64_t row_end, float* scores, int64_t ld_scores, void* stream) {
  if (scores == nullptr || row_begin < 0 || row_end < row_begin) return DSA_ERR_INVALID_ARGUMENT;
  if (keys == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  if (row_end == row_begin) return DSA_OK;
  CUtensorMap qm, km;
  IndexerParams p;
  dsa_status st = indexer_common(q_fp8, q_scale, q_scale_heads, w, keys, B, H_I, d_I, &qm, &km, &p);
  if (st != DSA_OK) return st;
  if (ld_scores < keys->max_seqlen) return DSA_ERR_INVALID_ARGUMENT;
  p.scores = scores;
  p.ld = ld_scores;
  p.row_begin = row_begin;
  p.row_end = row_end;
  if (keys->kind == DSA_KV_CONTIGUOUS) {
    if (row_end > keys->total_tokens) return DSA_ERR_INVALID_ARGUMENT;
    dim3 grid((keys->max_seqlen + kIdxTok - 1) / kIdxTok, B);
    return launch_indexer<kIdxScores, false>(d_I, H_I, qm, km, p, grid, as_stream(stream));
  }
  if (row_end > B) return DSA_ERR_INVALID_ARGUMENT;
  dim3 grid((keys->max_seqlen + 128 * kDecodeTilesPerCta - 1) / (128 * kDecodeTilesPerCta), B);
  return launch_indexer<kIdxScores, true>(d_I, H_I, qm, km, p, grid, as_stream(stream));
}

dsa_status dsa_indexer_topk(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                            const dsa_kv_desc* keys, int32_t B, int32_t H_I, int32_t d_I, int32_t k, int32_t* idx_out,
                            void* stream) {
  if (idx_out == nullptr || keys == nullptr || k <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (keys->kind != DSA_KV_CONTIGUOUS) return DSA_ERR_UNSUPPORTED;
  if (k > 2048) return DSA_ERR_UNSUPPORTED;
  CUtensorMap qm, km;
  IndexerParams p;
  dsa_status st = indexer_common(q_fp8, q_scale, q_scale_heads, w, keys, B, H_I, d_I, &qm, &km, &p);
  if (st != DSA_OK) return st;
  int stages;
  st = topk_config(d_I, keys->max_seqlen, k, &stages, &p.cap);
  if (st != DSA_OK) return st;
  p.idx_out = idx_out;
  p.k = k;
  dim3 grid((keys->max_seqlen + kIdxTok - 1) / kIdxTok, B);
  return launch_indexer<kIdxTopk, false>(d_I, H_I, qm, km, p, grid, as_stream(stream), stages);
}

dsa_status dsa_indexer_topk_rows(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                                 const dsa_kv_desc* keys, int32_t H_I, int32_t d_I, int32_t k, int64_t row_begin,
                                 int64_t row_end, int32_t* idx_out, void* stream) {
  if (keys == nullptr || k <= 0 || row_begin < 0 || row_end < row_begin) return DSA_ERR_INVALID_ARGUMENT;
  if (keys->kind != DSA_KV_CONTIGUOUS) return DSA_ERR_UNSUPPORTED;
  if (k > 2048) return DSA_ERR_UNSUPPORTED;
  if (row_end > keys->total_tokens) return DSA_ERR_INVALID_ARGUMENT;
  if (row_end == row_begin) return DSA_OK;  // an empty block: nothing to read or write
  if (idx_out == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  CUtensorMap qm, km;
  IndexerParams p;
  dsa_status st = indexer_common(q_fp8, q_scale, q_scale_heads, w, keys, 1, H_I, d_I, &qm, &km, &p,
                                 row_end - row_begin);
  if (st != DSA_OK) return st;
  int stages;
  st = topk_config(d_I, keys->max_seqlen, k, &stages, &p.cap);
  if (st != DSA_OK) return st;
  p.idx_out = idx_out;
  p.k = k;
  p.tok_begin = static_cast<int32_t>(row_begin);
  p.tok_end = static_cast<int32_t>(row_end);
  p.q_row0 = row_begin;
  dim3 grid(static_cast<unsigned>((row_end - row_begin + kIdxTok - 1) / kIdxTok), 1);
  return launch_indexer<kIdxTopk, false>(d_I, H_I, qm, km, p, grid, as_stream(stream), stages);
}

size_t dsa_decode_select_workspace_size(int32_t B, int32_t max_ctx) {
  if (B <= 0 || max_ctx <= 0) return 0;
  const int64_t ld = (static_cast<int64_t>(max_ctx) + 3) / 4 * 4;
  const int64_t ld16 = ((static_cast<int64_t>(max_ctx) + kSelGroup - 1) / kSelGroup + 3) / 4 * 4;
  return align256(static_cast<size_t>(B) * ld * 4) + align256(static_cast<size_t>(B) * ld16 * 4);
}

dsa_status dsa_indexer_topk_decode(const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads, const float* w,
                                   const dsa_kv_desc* keys, int32_t B, int32_t H_I, int32_t d_I, int32_t k,
                                   int32_t* idx_out, void* workspace, size_t ws_bytes, void* stream) {
  if (keys == nullptr || idx_out == nullptr || k <= 0 || B <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (keys->kind != DSA_KV_PAGED) return DSA_ERR_UNSUPPORTED;
  if (workspace == nullptr || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(B) * kTopkCluster > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  CUtensorMap qm, km;
  IndexerParams p;
  dsa_status st = indexer_common(q_fp8, q_scale, q_scale_heads, w, keys, B, H_I, d_I, &qm, &km, &p);
  if (st != DSA_OK) return st;
  if (ws_bytes < dsa_decode_select_workspace_size(B, keys->max_seqlen)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  // workspace: [scores B x ld fp32][group maxima B x ld16 u32]
  const int64_t ld = (static_cast<int64_t>(keys->max_seqlen) + 3) / 4 * 4;
  const int64_t ld16 = ((static_cast<int64_t>(keys->max_seqlen) + kSelGroup - 1) / kSelGroup + 3) / 4 * 4;
  p.scores = static_cast<float*>(workspace);
  p.ld = ld;
  p.row_begin = 0;
  p.row_end = B;
  p.gmax = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + align256(static_cast<size_t>(B) * ld * 4));
  p.ld16 = ld16;
  cudaStream_t s = as_stream(stream);
  dim3 grid((keys->max_seqlen + 128 * kDecodeTilesPerCta - 1) / (128 * kDecodeTilesPerCta), B);
  st = launch_indexer<kIdxScores, true>(d_I, H_I, qm, km, p, grid, s);
  if (st != DSA_OK) return st;
  if (cudaFuncSetAttribute(topk_decode_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemBytes) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  topk_decode_select_kernel<<<static_cast<unsigned>(B * kTopkCluster), kTopkThreads, kSelSmemBytes, s>>>(
      p.scores, ld, p.gmax, ld16, keys->context_lens, keys->max_seqlen, k, idx_out);
  return launch_status();
}

dsa_status dsa_sparse_mla_prefill_rows(const void* q, const dsa_kv_desc* latent, const int32_t* idx, int32_t H,
                                       int32_t k, float sm_scale, int64_t row_begin, int64_t row_end, void* out,
                                       float* lse, void* stream) {
  if (latent == nullptr || latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr ||
      latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (row_begin < 0 || row_end < row_begin || row_end > latent->total_tokens) return DSA_ERR_INVALID_ARGUMENT;
  if (row_end == row_begin) return DSA_OK;  // an empty block: nothing to read or write
  if (q == nullptr || latent->data == nullptr || idx == nullptr || out == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16) || !aligned(idx, 16) || !aligned(out, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  if (latent->total_tokens > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  MlaParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.idx = idx;
  p.cu_seqlens = latent->cu_seqlens;
  p.B = 1;
  p.H = H;
  p.k = k;
  p.rows = row_end - row_begin;
  p.unit0 = row_begin;
  p.splits = 1;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return launch_mla_pair<false>(latent->data, q, p.rows, p, p.rows, as_stream(stream));
}

dsa_status dsa_sparse_mla_prefill(const void* q, const dsa_kv_desc* latent, const int32_t* idx, int32_t B, int32_t H,
                                  int32_t k, float sm_scale, void* out, float* lse, void* stream) {
  if (q == nullptr || latent == nullptr || latent->data == nullptr || idx == nullptr || out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr || latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16) || !aligned(idx, 16) || !aligned(out, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  if (latent->total_tokens > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  MlaParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.idx = idx;
  p.cu_seqlens = latent->cu_seqlens;
  p.B = B;
  p.H = H;
  p.k = k;
  p.rows = latent->total_tokens;
  p.splits = 1;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return launch_mla_pair<false>(latent->data, q, p.rows, p, p.rows, as_stream(stream));
}

dsa_status dsa_masked_mla_prefill(const void* q, const dsa_kv_desc* latent, const int32_t* idx, int32_t B, int32_t H,
                                  int32_t k, float sm_scale, void* out, float* lse, void* stream) {
  if (q == nullptr || latent == nullptr || latent->data == nullptr || idx == nullptr || out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr || latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16) || !aligned(idx, 16) || !aligned(out, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  if (latent->total_tokens > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  MlaParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.idx = idx;
  p.cu_seqlens = latent->cu_seqlens;
  p.B = B;
  p.H = H;
  p.k = k;
  p.rows = latent->total_tokens;
  p.splits = 1;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return launch_mla_pair<false, true>(latent->data, q, p.rows, p, p.rows, as_stream(stream));
}

dsa_status dsa_sparse_mla_decode(const void* q, const dsa_kv_desc* latent, const int32_t* idx, int32_t B, int32_t H,
                                 int32_t k, float sm_scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                                 void* stream) {
  if (q == nullptr || latent == nullptr || latent->data == nullptr || idx == nullptr || out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->kind != DSA_KV_PAGED || latent->block_table == nullptr || latent->context_lens == nullptr ||
      latent->num_blocks <= 0 || latent->max_blocks_per_seq <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->block_size != 64) return DSA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(latent->data, 16) || !aligned(idx, 16) || !aligned(out, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(latent->num_blocks) * 64 > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  const int splits = decode_splits(B, k);
  if (workspace == nullptr || ws_bytes < decode_partials_bytes(B, H, splits) || !aligned(workspace, 256))
    return workspace == nullptr ? DSA_ERR_INVALID_ARGUMENT : DSA_ERR_WORKSPACE_TOO_SMALL;
  MlaParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.idx = idx;
  p.block_table = latent->block_table;
  p.context_lens = latent->context_lens;
  p.max_blocks_per_seq = latent->max_blocks_per_seq;
  p.num_blocks = latent->num_blocks;
  p.B = B;
  p.H = H;
  p.k = k;
  p.rows = B;
  p.splits = splits;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                       align256(static_cast<size_t>(B) * splits * H * kValueDim * 4));
  p.out = static_cast<__nv_bfloat16*>(out);  // one split: the kernel writes out / lse itself
  p.lse = lse;
  cudaStream_t s = as_stream(stream);
  dsa_status st = launch_mla_pair<true>(latent->data, q, B, p, static_cast<int64_t>(B) * splits, s);
  if (st != DSA_OK) return st;
  if (splits == 1) return DSA_OK;
  mla_combine_kernel<<<dim3(H, B), 128, 0, s>>>(p.part_o, p.part_ml, splits, H, static_cast<__nv_bfloat16*>(out), lse);
  return launch_status();
}

dsa_status dsa_sparse_mla_decode_noalloc(const void* q, const dsa_kv_desc* latent, const int32_t* idx, int32_t B,
                                         int32_t H, int32_t k, float sm_scale, void* out, float* lse, void* stream) {
  if (B <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  if (decode_partials_bytes(B, H, decode_splits(B, k)) > DSA_NOALLOC_SCRATCH_BYTES) return DSA_ERR_UNSUPPORTED;
  void* scratch = nullptr;
  const dsa_status st = noalloc_scratch(&scratch);
  if (st != DSA_OK) return st;
  return dsa_sparse_mla_decode(q, latent, idx, B, H, k, sm_scale, out, lse, scratch, DSA_NOALLOC_SCRATCH_BYTES,
                               stream);
}

dsa_status dsa_forward(int32_t mode, const uint8_t* q_fp8, const float* q_scale, int32_t q_scale_heads,
                       const float* w, const dsa_kv_desc* keys, const void* q, const dsa_kv_desc* latent, int32_t B,
                       int32_t H_I, int32_t d_I, int32_t H, int32_t k, float sm_scale, void* out, float* lse,
                       int32_t* idx_out, void* workspace, size_t ws_bytes, void* stream) {
  if (keys == nullptr || latent == nullptr || B <= 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!mla_shape_ok(H, k)) return DSA_ERR_UNSUPPORTED;
  const size_t need = dsa_workspace_size(mode, B, keys->total_tokens, keys->max_seqlen, H, k);
  if (mode == DSA_MODE_PREFILL) {
    if (keys->kind != DSA_KV_CONTIGUOUS || latent->kind != DSA_KV_CONTIGUOUS) return DSA_ERR_INVALID_ARGUMENT;
    int32_t* idx = idx_out;
    if (idx == nullptr) {
      if (workspace == nullptr) return DSA_ERR_INVALID_ARGUMENT;
      if (ws_bytes < need) return DSA_ERR_WORKSPACE_TOO_SMALL;
      idx = static_cast<int32_t*>(workspace);
    }
    dsa_status st = dsa_indexer_topk(q_fp8, q_scale, q_scale_heads, w, keys, B, H_I, d_I, k, idx, stream);
    if (st != DSA_OK) return st;
    return dsa_sparse_mla_prefill(q, latent, idx, B, H, k, sm_scale, out, lse, stream);
  }
  if (mode != DSA_MODE_DECODE) return DSA_ERR_INVALID_ARGUMENT;
  if (keys->kind != DSA_KV_PAGED || latent->kind != DSA_KV_PAGED) return DSA_ERR_INVALID_ARGUMENT;
  if (workspace == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need || !aligned(workspace, 256)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  // workspace: [decode partials][selection workspace: scores, group maxima][selection B x k]
  const int splits = decode_splits(B, k);
  const size_t part = decode_partials_bytes(B, H, splits);
  const size_t sel = dsa_decode_select_workspace_size(B, keys->max_seqlen);
  int32_t* idx = idx_out != nullptr ? idx_out
                                    : reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + part + sel);
  dsa_status st = dsa_indexer_topk_decode(q_fp8, q_scale, q_scale_heads, w, keys, B, H_I, d_I, k, idx,
                                          static_cast<uint8_t*>(workspace) + part, sel, stream);
  if (st != DSA_OK) return st;
  return dsa_sparse_mla_decode(q, latent, idx, B, H, k, sm_scale, out, lse, workspace, part, stream);
}

dsa_status dsa_row_partition(int64_t L, int32_t k, int32_t parts, double indexer_cost, double mla_cost,
                             int64_t* bounds) {
  if (bounds == nullptr || L < 1 || k < 1 || parts < 1 || parts > L) return DSA_ERR_INVALID_ARGUMENT;
  if (!(indexer_cost >= 0.0) || !(mla_cost >= 0.0) || !(indexer_cost + mla_cost > 0.0)) return DSA_ERR_INVALID_ARGUMENT;
  // cost of rows [0, n): indexer_cost * C(n) / C(L) + mla_cost * M(n) / M(L), with
  // C(n) = sum_{t<n} (t+1) (the causal prefixes the indexer scans) and
  // M(n) = sum_{t<n} min(t+1, k) (the rows sparse MLA attends to)
  const double kk = static_cast<double>(k);
  auto C = [](double n) { return n * (n + 1.0) / 2.0; };
  auto M = [&](double n) { return n <= kk ? n * (n + 1.0) / 2.0 : kk * (kk + 1.0) / 2.0 + (n - kk) * kk; };
  const double Lf = static_cast<double>(L), CL = C(Lf), ML = M(Lf);
  auto cost = [&](int64_t n) {
    const double x = static_cast<double>(n);
    return indexer_cost * C(x) / CL + mla_cost * M(x) / ML;
  };
  const double total = cost(L);
  bounds[0] = 0;
  for (int32_t r = 1; r < parts; ++r) {
    const double target = total * static_cast<double>(r) / static_cast<double>(parts);
    int64_t lo = bounds[r - 1] + 1, hi = L - (parts - r);  // every block keeps at least one row
    if (lo > hi) return DSA_ERR_INVALID_ARGUMENT;
    while (lo < hi) {  // the first boundary whose cost reaches the target
      const int64_t mid = lo + (hi - lo) / 2;
      if (cost(mid) >= target) hi = mid;
      else lo = mid + 1;
    }
    bounds[r] = lo;
  }
  bounds[parts] = L;
  return DSA_OK;
}

size_t dsa_workspace_size(int32_t mode, int32_t B, int64_t total_tokens, int32_t max_ctx, int32_t H, int32_t k) {
  if (B <= 0 || k <= 0 || H <= 0) return 0;
  if (mode == DSA_MODE_PREFILL) return align256(static_cast<size_t>(total_tokens > 0 ? total_tokens : 0) * k * 4);
  return decode_partials_bytes(B, H, decode_splits(B, k)) + dsa_decode_select_workspace_size(B, max_ctx) +
         align256(static_cast<size_t>(B) * k * 4);
}

dsa_status dsa_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                       int64_t rows, int32_t cols, int32_t dtype, float eps, void* y, int64_t ld_y,
                       void* residual_out, int64_t ld_residual_out, uint8_t* codes, float* scale, int32_t group,
                       float* rstd, void* stream) {
  if (rows < 0 || !dtype_ok(dtype) || cols <= 0 || !(eps >= 0.f) || !std::isfinite(eps)) return DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA_OK;
  if (x == nullptr || weight == nullptr || (y == nullptr && codes == nullptr) || (codes == nullptr) != (scale == nullptr))
    return DSA_ERR_INVALID_ARGUMENT;
  if (group != 0 && group != DSA_QUANT_GROUP) return DSA_ERR_INVALID_ARGUMENT;
  const size_t es = dtype_size(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, es) || !aligned(y, es) || !aligned(residual_out, es) ||
      !aligned(scale, 4) || !aligned(rstd, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  if (ld_x < 0 || (residual != nullptr && ld_residual < 0) || (y != nullptr && ld_y < cols) ||
      (residual_out != nullptr && ld_residual_out < cols))
    return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (!same_rows(y, ld_y, x, ld_x) || !same_rows(y, ld_y, residual, ld_residual) ||
                   !same_rows(residual_out, ld_residual_out, x, ld_x) ||
                   !same_rows(residual_out, ld_residual_out, residual, ld_residual)))
    return DSA_ERR_INVALID_ARGUMENT;
  if (y != nullptr && y == residual_out) return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 0x7FFFFFFFLL || cols > kMostCols) return DSA_ERR_UNSUPPORTED;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.res = residual;
  p.w = weight;
  p.ld_x = ld_x;
  p.ld_res = ld_residual;
  p.ld_y = ld_y;
  p.ld_ro = ld_residual_out;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  p.y = y;
  p.res_out = residual_out;
  p.codes = codes;
  p.scale = scale;
  p.groups = group == 0 ? 0 : cols / DSA_QUANT_GROUP + (cols % DSA_QUANT_GROUP != 0);
  p.rstd = rstd;
  const int piece = piece_of(cols, es, {{x, ld_x}, {residual, ld_residual}, {weight, 0}, {y, ld_y}, {residual_out, ld_residual_out}}, codes);
  return with_dtype(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_rmsnorm<T>(p, piece, as_stream(stream));
  });
}

size_t dsa_rmsnorm_backward_workspace_size(int64_t rows, int32_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  // The CTAs fall as rows widen, so a narrower row can need more: the most of all widths up to cols.  Those with
  // k CTAs per SM reach to 8192 / k columns (norm_bwd_per_sm at 2 bytes); with one there is no limit.
  int64_t most = norm_bwd_ctas(rows, cols, 2) * cols;
  for (int k = 2; k <= 16; ++k) {
    const int widest = std::min(cols, 8192 / k);
    most = std::max(most, norm_bwd_ctas(rows, widest, 2) * widest);
  }
  return align256(static_cast<size_t>(most) * sizeof(float));
}

dsa_status dsa_rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* weight,
                                const float* rstd, const void* dresidual, int64_t ld_dresidual, int64_t rows,
                                int32_t cols, int32_t dtype, void* dh, int64_t ld_dh, float* dw, void* workspace,
                                size_t ws_bytes, void* stream) {
  if (rows < 0 || !dtype_ok(dtype) || cols <= 0 || dw == nullptr || !aligned(dw, 4)) return DSA_ERR_INVALID_ARGUMENT;
  cudaStream_t s = as_stream(stream);
  if (rows == 0)
    return cudaMemsetAsync(dw, 0, static_cast<size_t>(cols) * sizeof(float), s) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dh == nullptr || workspace == nullptr)
    return DSA_ERR_INVALID_ARGUMENT;
  const size_t es = dtype_size(dtype);
  if (!aligned(dy, es) || !aligned(h, es) || !aligned(weight, es) || !aligned(dresidual, es) || !aligned(dh, es) ||
      !aligned(rstd, 4) || !aligned(workspace, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  if (ld_dy < 0 || ld_h < 0 || ld_dh < cols || (dresidual != nullptr && ld_dresidual < 0)) return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (!same_rows(dh, ld_dh, dy, ld_dy) || !same_rows(dh, ld_dh, h, ld_h) || !same_rows(dh, ld_dh, dresidual, ld_dresidual)))
    return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 0x7FFFFFFFLL || cols > kMostCols) return DSA_ERR_UNSUPPORTED;
  if (ws_bytes < dsa_rmsnorm_backward_workspace_size(rows, cols)) return DSA_ERR_WORKSPACE_TOO_SMALL;
  NormBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.dy = dy;
  p.h = h;
  p.w = weight;
  p.rstd = rstd;
  p.dres = dresidual;
  p.ld_dy = ld_dy;
  p.ld_h = ld_h;
  p.ld_dres = ld_dresidual;
  p.ld_dh = ld_dh;
  p.rows = rows;
  p.cols = cols;
  p.dh = dh;
  p.part = static_cast<float*>(workspace);
  const int piece = piece_of(cols, es, {{dy, ld_dy}, {h, ld_h}, {weight, 0}, {dresidual, ld_dresidual}, {dh, ld_dh}}, nullptr);
  return with_dtype(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_rmsnorm_backward<T>(p, piece, dw, s);
  });
}

dsa_status dsa_rope(const void* x, int64_t x_row_stride, int64_t x_head_stride, void* out, int64_t out_row_stride,
                    int64_t out_head_stride, int64_t rows, int32_t heads, int32_t dim, int32_t rot_offset,
                    int32_t rot_dim, int32_t layout, int32_t dtype, const int32_t* positions, const double* freqs,
                    float mscale, int32_t transpose, void* stream) {
  if (rows < 0 || heads < 0 || dim <= 0 || !dtype_ok(dtype) || !std::isfinite(mscale)) return DSA_ERR_INVALID_ARGUMENT;
  if (layout != DSA_ROPE_INTERLEAVED && layout != DSA_ROPE_HALF) return DSA_ERR_INVALID_ARGUMENT;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_offset < 0 || rot_dim > dim || rot_offset > dim - rot_dim)
    return DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0 || heads == 0) return DSA_OK;
  if (x == nullptr || out == nullptr || positions == nullptr || freqs == nullptr) return DSA_ERR_INVALID_ARGUMENT;
  const size_t es = dtype_size(dtype);
  if (!aligned(x, es) || !aligned(out, es) || !aligned(positions, 4) || !aligned(freqs, 8)) return DSA_ERR_INVALID_ARGUMENT;
  if (x_row_stride < 0 || x_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0) return DSA_ERR_INVALID_ARGUMENT;
  // no two (row, head) pieces of out on one another: each row's heads in one stretch, or each head's rows
  const int64_t head_step = heads > 1 ? out_head_stride : dim, row_step = rows > 1 ? out_row_stride : dim;
  const int64_t far = int64_t(1) << 60;  // beyond any tensor; keeps the products in range
  if (head_step < dim || row_step < dim || head_step > far / heads || row_step > far / rows) return DSA_ERR_INVALID_ARGUMENT;
  if (rows > 1 && heads > 1 && row_step < head_step * (heads - 1) + dim && head_step < row_step * (rows - 1) + dim)
    return DSA_ERR_INVALID_ARGUMENT;
  if (out == x && ((rows > 1 && x_row_stride != out_row_stride) || (heads > 1 && x_head_stride != out_head_stride)))
    return DSA_ERR_INVALID_ARGUMENT;
  if (rot_dim > 2 * rope::kMaxPairs || rows > 0x7FFFFFFFLL || static_cast<int64_t>(heads) * dim > kMostCols)
    return DSA_ERR_UNSUPPORTED;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.out = out;
  p.xr = x_row_stride;
  p.xh = x_head_stride;
  p.orow = out_row_stride;
  p.oh = out_head_stride;
  p.rows = rows;
  p.heads = heads;
  p.dim = dim;
  p.rot0 = rot_offset;
  p.rot = rot_dim;
  p.half_layout = layout == DSA_ROPE_HALF;
  p.pos = positions;
  p.freqs = freqs;
  p.mscale = mscale;
  p.transpose = transpose;
  p.copy_rest = out != x;
  int piece = 8;
  auto divides = [&](int v) {
    const size_t bytes = std::min<size_t>(v * es, 16);
    auto ok = [&](int64_t stride, int64_t n) { return n <= 1 || stride % v == 0; };
    return dim % v == 0 && aligned(x, bytes) && aligned(out, bytes) && ok(x_row_stride, rows) && ok(x_head_stride, heads) &&
           ok(out_row_stride, rows) && ok(out_head_stride, heads);
  };
  while (piece > 1 && !divides(piece)) piece /= 2;
  return with_dtype(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_rope<T>(p, piece, as_stream(stream));
  });
}

dsa_status dsa_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, double original_ctx,
                                double beta_fast, double beta_slow, double* freqs, float* mscale) {
  if (freqs == nullptr || mscale == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 1.0) || !std::isfinite(theta))
    return DSA_ERR_INVALID_ARGUMENT;
  if (scaling < DSA_ROPE_PLAIN || scaling > DSA_ROPE_YARN) return DSA_ERR_INVALID_ARGUMENT;
  if (scaling != DSA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return DSA_ERR_INVALID_ARGUMENT;
  if (scaling == DSA_ROPE_NTK && rot_dim < 4) return DSA_ERR_INVALID_ARGUMENT;
  double low = 0.0, span = 1.0;
  if (scaling == DSA_ROPE_YARN) {
    if (!(original_ctx > 0.0) || !std::isfinite(original_ctx) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
        !std::isfinite(beta_fast))
      return DSA_ERR_INVALID_ARGUMENT;
    const double two_pi = 6.283185307179586;
    auto dim_of = [&](double turns) { return rot_dim * std::log(original_ctx / (two_pi * turns)) / (2.0 * std::log(theta)); };
    low = std::max(std::floor(dim_of(beta_fast)), 0.0);
    const double high = std::min(std::ceil(dim_of(beta_slow)), rot_dim - 1.0);
    span = std::max(high - low, 0.001);
  }
  const double base = scaling == DSA_ROPE_NTK ? theta * std::pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == DSA_ROPE_LINEAR) {
      freqs[i] = f / factor;
    } else if (scaling == DSA_ROPE_YARN) {
      const double ramp = std::min(std::max((i - low) / span, 0.0), 1.0);
      freqs[i] = f / factor * ramp + f * (1.0 - ramp);
    } else {
      freqs[i] = f;
    }
  }
  *mscale = scaling == DSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DSA_OK;
}

dsa_status dsa_cache_append(const void* kv, int64_t ld_kv, const void* kv_weight, float eps, const void* key,
                            int64_t ld_key, int32_t d_I, const int32_t* seq, const int32_t* positions, int64_t rows,
                            int32_t B, const double* freqs, float mscale, int32_t layout, int32_t key_layout,
                            int32_t key_rot_offset, const dsa_kv_desc* latent, const dsa_kv_desc* keys, void* stream) {
  if (rows < 0 || B <= 0 || !std::isfinite(mscale)) return DSA_ERR_INVALID_ARGUMENT;
  if ((kv == nullptr) != (latent == nullptr) || (key == nullptr) != (keys == nullptr) || (kv == nullptr && key == nullptr))
    return rows == 0 ? DSA_OK : DSA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA_OK;
  if (positions == nullptr || freqs == nullptr || !aligned(freqs, 8)) return DSA_ERR_INVALID_ARGUMENT;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  if (latent != nullptr) {
    if (kv_weight == nullptr || !aligned(kv, 16) || !aligned(kv_weight, 16) ||
        (rows > 1 && (ld_kv % 8 != 0 || ld_kv < kLatentDim)))
      return DSA_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.f) || !std::isfinite(eps) || (layout != DSA_ROPE_INTERLEAVED && layout != DSA_ROPE_HALF))
      return DSA_ERR_INVALID_ARGUMENT;
    const dsa_status st = append_cache(latent, false, 16, &p.latent);
    if (st != DSA_OK) return st;
  }
  if (keys != nullptr) {
    if (d_I != 64 && d_I != 128) return DSA_ERR_UNSUPPORTED;
    if (!aligned(key, 4) || (rows > 1 && (ld_key % 2 != 0 || ld_key < d_I))) return DSA_ERR_INVALID_ARGUMENT;
    if (key_layout != DSA_ROPE_INTERLEAVED && key_layout != DSA_ROPE_HALF) return DSA_ERR_INVALID_ARGUMENT;
    if (key_rot_offset < 0 || key_rot_offset > d_I - 64 || key_rot_offset % 2 != 0) return DSA_ERR_INVALID_ARGUMENT;
    const dsa_status st = append_cache(keys, true, 2, &p.keys);
    if (st != DSA_OK) return st;
  }
  if (rows > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.w = static_cast<const __nv_bfloat16*>(kv_weight);
  p.key = static_cast<const __nv_bfloat16*>(key);
  p.ld_kv = ld_kv;
  p.ld_key = ld_key;
  p.eps = eps;
  p.seq = seq;
  p.pos = positions;
  p.rows = rows;
  p.B = B;
  p.freqs = freqs;
  p.mscale = mscale;
  p.half = layout == DSA_ROPE_HALF;
  p.key_half = key_layout == DSA_ROPE_HALF;
  p.key_rot0 = key_rot_offset;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((rows + append::kWarps - 1) / append::kWarps, kSms * append::kCtas));
  auto launch = [&](auto kern) { kern<<<grid, append::kWarps * 32, 0, as_stream(stream)>>>(p); };
  if (keys == nullptr) launch(cache_append_kernel<true, 0>);
  else if (latent == nullptr) launch(d_I == 64 ? cache_append_kernel<false, 64> : cache_append_kernel<false, 128>);
  else launch(d_I == 64 ? cache_append_kernel<true, 64> : cache_append_kernel<true, 128>);
  return launch_status();
}

// Arguments common to both window entries; fills what they share.
static dsa_status window_common(const void* q, const dsa_kv_desc* latent, int32_t B, int32_t H, int32_t window,
                                int32_t sinks, float sm_scale, void* out, float* lse, WinParams* p) {
  if (q == nullptr || latent == nullptr || latent->data == nullptr || out == nullptr || B <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(latent->data, 16) || !aligned(out, 16) || !aligned(lse, 4)) return DSA_ERR_INVALID_ARGUMENT;
  if (window < 1 || sinks < 0 || !(sm_scale > 0.f) || !std::isfinite(sm_scale) || latent->max_seqlen <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (H < 1 || H > 128) return DSA_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  p->B = B;
  p->H = H;
  p->window = window;
  p->sinks = sinks;
  p->scale_log2 = sm_scale * 1.4426950408889634f;
  p->out = static_cast<__nv_bfloat16*>(out);
  p->lse = lse;
  return DSA_OK;
}

dsa_status dsa_window_mla_prefill(const void* q, const dsa_kv_desc* latent, int32_t B, int32_t H, int32_t window,
                                  int32_t sinks, float sm_scale, void* out, float* lse, void* stream) {
  WinParams p;
  const dsa_status st = window_common(q, latent, B, H, window, sinks, sm_scale, out, lse, &p);
  if (st != DSA_OK) return st;
  if (latent->kind != DSA_KV_CONTIGUOUS || latent->cu_seqlens == nullptr || latent->total_tokens <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->total_tokens * H > 0x7FFFFFFFLL - 128) return DSA_ERR_UNSUPPORTED;  // row coordinates of 128-row tiles
  p.cu_seqlens = latent->cu_seqlens;
  p.rows = latent->total_tokens;
  return launch_window<false>(latent->data, q, p, p.rows, as_stream(stream));
}

static size_t window_workspace_bytes(int32_t B, int32_t H) {
  return window_plan_bytes(B) + window_part_bytes(H) + align256(static_cast<size_t>(2 * kMlaClusters) * H * 2 * 4);
}

size_t dsa_window_mla_workspace_size(int32_t B, int32_t H, int32_t window, int32_t sinks, int32_t max_ctx) {
  if (B <= 0 || H <= 0 || window < 1 || sinks < 0 || max_ctx <= 0) return 0;
  return window_shared(B, window, sinks, max_ctx) ? window_workspace_bytes(B, H) : 0;
}

size_t dsa_window_mla_workspace_limit(int32_t B, int32_t H, int32_t window, int32_t sinks, int32_t max_ctx) {
  if (B <= 0 || H <= 0 || window < 1 || sinks < 0 || max_ctx <= 0) return 0;
  // One sequence is shared out as soon as any number of them is: that takes whole - share > 8, and whole - share is
  // below (chunks + 2) (rounds - B / 74) + 1 <= (chunks + 2) 73 / 74 + 1, which leaves chunks >= 7, where one is.
  if (!window_shared(1, window, sinks, max_ctx)) return 0;
  return window_workspace_bytes(std::min(B, kShareSeqs), H);
}

dsa_status dsa_window_mla_decode(const void* q, const dsa_kv_desc* latent, int32_t B, int32_t H, int32_t window,
                                 int32_t sinks, float sm_scale, void* out, float* lse, void* workspace,
                                 size_t ws_bytes, void* stream) {
  WinParams p;
  const dsa_status st = window_common(q, latent, B, H, window, sinks, sm_scale, out, lse, &p);
  if (st != DSA_OK) return st;
  if (latent->kind != DSA_KV_PAGED || latent->block_table == nullptr || latent->context_lens == nullptr ||
      latent->num_blocks <= 0 || latent->max_blocks_per_seq <= 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (latent->block_size != 64) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(latent->max_seqlen) > static_cast<int64_t>(latent->max_blocks_per_seq) * 64)
    return DSA_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(latent->num_blocks) * 64 > 0x7FFFFFFFLL || static_cast<int64_t>(B) * H > 0x7FFFFFFFLL - 128)
    return DSA_ERR_UNSUPPORTED;
  if (latent->max_seqlen > 1 << 30) return DSA_ERR_UNSUPPORTED;  // entry numbers, a chunk past the last, fit an int
  p.shared = window_shared(B, window, sinks, latent->max_seqlen);
  if (p.shared) {
    if (workspace == nullptr || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARGUMENT;
    if (ws_bytes < dsa_window_mla_workspace_size(B, H, window, sinks, latent->max_seqlen)) return DSA_ERR_WORKSPACE_TOO_SMALL;
    // workspace: [plan][partial outputs][their maxima and sums]
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.plan = reinterpret_cast<int2*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + window_plan_bytes(B));
    p.part_ml = reinterpret_cast<float*>(ws + window_plan_bytes(B) + window_part_bytes(H));
  }
  p.block_table = latent->block_table;
  p.context_lens = latent->context_lens;
  p.max_blocks = latent->max_blocks_per_seq;
  p.num_blocks = latent->num_blocks;
  p.max_len = latent->max_seqlen;
  p.rows = B;
  cudaStream_t s = as_stream(stream);
  const dsa_status launched = launch_window<true>(latent->data, q, p, p.shared ? kMlaClusters : B, s);
  if (launched != DSA_OK || !p.shared) return launched;
  window_merge_kernel<<<dim3(H, B), 128, 0, s>>>(p.part_o, p.part_ml, p.plan, H, p.out, lse);
  return launch_status();
}

}  // extern "C"
