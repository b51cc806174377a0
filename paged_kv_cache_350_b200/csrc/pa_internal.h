// Internal host/device interface of libpagedattn: kernel parameter blocks and the
// launchers the C ABI (api.cu) dispatches to.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "pa.h"

namespace pa {

// Devices that per-device state is kept for.
constexpr int kMaxDevices = 64;

// Multiprocessors of the current device, asked once per device; 0 if unknown.
int device_sms();

// Grant `kernel` its dynamic shared memory on the current device; `granted` (one per kernel and
// device) holds what it has, so that most launches make no call.
struct SmemGrant {
  std::atomic<int> bytes[kMaxDevices];
  std::mutex mutex;  // a smaller grant of another thread must not follow a larger one
};
template <typename K>
cudaError_t grant_smem(SmemGrant& g, K kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (bytes <= g.bytes[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(g.mutex);
  if (bytes <= g.bytes[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) g.bytes[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

// Launch as a programmatic dependent of the previous kernel on the stream: the kernel calls
// griddepcontrol.wait before it touches global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Parameters of one pa_decode call, as the kernels see them.
struct DecodeParams {
  void* out;                   // [B][Hq][D], dtype of q
  const void* q;               // [B][Hq][D]
  const void* k_pool;          // [NB][BS][Hkv][D]
  const void* v_pool;
  const int32_t* block_tables; // [B][max_blocks]
  const int32_t* seq_lens;     // [B]
  int B, Hq, Hkv, G, D, block_size, max_blocks, num_blocks;
  float scale_log2;            // scale * log2(e): softmax runs in base 2
  int partition_tokens;        // P: tokens per context partition
  int max_parts;               // ceil(max_blocks*block_size / P); 1 = no split
  float* ws_ml;                // [B][Hq][max_parts][2]: (running max, sum), base-2
  float* ws_acc;               // [B][Hq][max_parts][D]: unnormalised output
  int32_t* err;                // nullable device error flag
};

// Parameters of the balanced persistent ("stream") tensor-core kernel.
struct StreamParams {
  DecodeParams d;
  int streams;     // consumer warps in the grid = tile ranges
  int32_t* meta;   // [streams][4]: unit in slot 0, it starts in this stream, unit in slot 1
  float* pml;      // [streams][2][G][2]: (max, sum) of cut-unit pieces, base 2
  float* pacc;     // [streams][2][G][D]: unnormalised outputs of those pieces
  // Fused cache write (pa_decode_append); all null for a plain decode.
  const void* k_new;  // [B][Hkv][D] the step's keys: position seq_lens[b]-1 of row b
  const void* v_new;
  void* k_pool_w;     // the pools of `d`, written at that position
  void* v_pool_w;
};

// One wave of the stream kernel for this shape on the current device (0 if unknown).
int stream_grid(int D, int block_size, int G, int B);
// Streams (warps) per CTA of the stream kernel for this block size:
// streams = grid * stream_warps_per_cta(block_size).
int stream_warps_per_cta(int block_size);
size_t stream_workspace_bytes(int streams, int G, int D);
void stream_carve(StreamParams* sp, void* workspace);
cudaError_t launch_decode_stream(const StreamParams& sp, int grid, cudaStream_t stream);

// Parameters of the shared-prefix decode (decode_prefix.cu).
struct PrefixParams {
  DecodeParams d;
  const int32_t* group_of;       // [B] group of batch row b, or -1
  const int32_t* group_prefix;   // [ngroups] shared tokens (multiple of PA_SHARED_PREFIX_ALIGN)
  const int32_t* group_members;  // [ngroups][max_members] batch rows, -1 padded
  int ngroups, max_members;
  int streams;
  uint64_t epoch;  // this call's tag for the cut-unit flags
  unsigned long long* cut_flag;  // [streams]: = epoch once CTA s has published the partial
                                 // of its first piece (a later piece of a cut unit)
  float* pml;      // [streams][64][2]: (max, sum) of that piece per row, base 2
  float* pacc;     // [streams][64][D]: its unnormalised output per row
  float* pxch;     // [streams][2][2][64][2]: per piece parity and column group, the
                   // (max, sum) the two softmax column groups exchange
};
int prefix_grid(int D, int block_size, int R);
int prefix_warps_per_cta();
size_t prefix_workspace_bytes(int streams, int rows, int D);
void prefix_carve(PrefixParams* pp, void* workspace, int rows);
// A fresh tag for one shared-prefix call (its cut-unit flags).
uint64_t prefix_epoch();
cudaError_t launch_decode_prefix(const PrefixParams& pp, int grid, cudaStream_t stream);

// 4-D TMA view of a bf16 pool [NB][BS][Hkv][D]: box = box_rows rows (BS, or a part of a
// block starting at a row coordinate) x 64 columns of one head.
bool make_pool_map(CUtensorMap* map, const void* pool, int NB, int BS, int Hkv, int D,
                   int box_rows);
// 5-D TMA view of the same pool: box = box_rows rows of one head with all D columns,
// landing as [D / 64][box_rows][64], 128-byte swizzled.
bool make_pool_map_rows(CUtensorMap* map, const void* pool, int NB, int BS, int Hkv, int D,
                        int box_rows);
// Tensor map over q viewed as [B][Hq][D] (bf16): boxes of 64 columns x G heads of one
// batch row, 128-byte swizzled.
bool make_q_map(CUtensorMap* map, const void* q, int B, int Hq, int D, int G);
// The same view of an fp32 pool: box = box_rows rows of one head, all D columns, not swizzled.
bool make_pool_map_f32(CUtensorMap* map, const void* pool, int NB, int BS, int Hkv, int D, int box_rows);
// Tensor map over q as T tokens of [Hq][D], q_stride elements apart: boxes of 64 columns x G
// heads x `tokens` tokens, 128-byte swizzled.
bool make_q_rows_map(CUtensorMap* map, const void* q, int T, int Hq, int D, int64_t q_stride, int G,
                     int tokens);

// Launch the bf16 tensor-core decode kernel (+ reduce when max_parts > 1).
cudaError_t launch_decode_tc(const DecodeParams& p, cudaStream_t stream);
// Launch the CUDA-core decode kernel (+ reduce when max_parts > 1).
cudaError_t launch_decode_generic(const DecodeParams& p, pa_dtype dtype, cudaStream_t stream);
// Launch the split-context reduce kernel.
cudaError_t launch_decode_reduce(const DecodeParams& p, pa_dtype dtype, cudaStream_t stream);

cudaError_t launch_reshape_and_cache(const void* key, const void* value, void* k_pool,
                                     void* v_pool, const int64_t* slot_mapping, int T, int Hkv,
                                     int row_bytes, int64_t num_slots, int32_t* err,
                                     cudaStream_t stream);
// Write k_new/v_new[b] ([B][Hkv][D]) at position seq_lens[b]-1 of row b's block table.
cudaError_t launch_append_kv(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                             const int32_t* block_tables, const int32_t* seq_lens, int B,
                             int max_blocks, int block_size, int num_blocks, int row_bytes,
                             int32_t* err, cudaStream_t stream);
cudaError_t launch_copy_blocks(void* k_pool, void* v_pool, const int32_t* pairs, int n,
                               int64_t block_bytes, int num_blocks, int32_t* err,
                               cudaStream_t stream);

// Rotary positions with the cache write (rope.cu).
struct RopeParams {
  void* q_out;              // [T][Hq][D]
  const void *q, *k, *v;    // [T] tokens of Hq / Hkv / Hkv heads, `*_stride` elements apart
  void *k_pool, *v_pool;
  const int32_t* positions; // [T]
  const int64_t* slots;     // [T]
  const double* inv_freq;   // [R / 2] radians per position
  int64_t q_stride, k_stride, v_stride, num_slots;
  int T, Hq, Hkv, D, R;
  int half;                 // pairs (i, i + R/2), else (2i, 2i + 1)
  float factor;
  int32_t* err;
};
cudaError_t launch_rope(const RopeParams& p, pa_dtype dtype, cudaStream_t stream);

// Attention of ragged query tokens (attention.cu, attention_tc.cu, attention_tokens.cu).
// The formulas for the usual caps are off by up to 6.9e-7 (bf16 prompts' polynomial) of the cap, whatever
// the score: 4.4e-5 here, which is little beside the weights' rounding to bf16, and worse for each wider cap.
constexpr float kWideCap = 64.f;
struct AttnItem;
struct AttnStart;
struct AttnParams {
  void* out;                    // [T][Hq][D]
  const void* q;                // [T] tokens of Hq heads, q_stride elements apart
  const void *k_pool, *v_pool;
  const int32_t* block_tables;  // [B][max_blocks]
  const int32_t* seq_lens;      // [B]
  const int32_t* query_starts;  // [B + 1]
  const int32_t* prefix_lens;   // [B], nullable
  const int32_t* first_keys;    // [T], nullable
  const float* slopes;          // [Hq], nullable
  int64_t q_stride;
  float scale_log2;             // scale * log2(e)
  float cap_in, cap_out;        // with a cap: scale / cap and cap * log2(e); cap_out 0: none
  float cap_poly[5], cap_small; // the tensor-core kernel's polynomial of the cap, and its bound
  int cap_wide;                 // a cap past kWideCap: its error is relative to the score (attention.h)
  float cap_ref;           // reference of capped scores without a bias; inf: their maximum is found
  int window;                   // 0: none
  int T, B, max_query_len, Hq, Hkv, G, D, block_size, max_blocks, num_blocks;
  int32_t* err;
  // the plan (in the workspace): rows per item, keys per tile, CTAs of the main kernel
  int RT, KT, ctas, max_items;
  int extra;                    // what a unit costs beside its tiles, in tiles
  int HR;                       // rows of a softmax group of the tensor-core kernel (RT, or RT / 2)
  int dynamic;                  // units may be taken one by one
  int32_t* header;              // [4]: items, slots (tiles and extra ones, of one KV head), whether
                                // units are taken one by one, the next unit then
  int32_t* seq_items;           // [B] items before the sequence
  AttnItem* items;              // [max_items]
  int32_t* tile_sum;            // [max_items + 1] slots before the item
  AttnStart* starts;            // [ctas]
  int32_t* cuts;                // [ctas] records of the cut units (AttnCut; the tokens kernel has its own)
  int by_unit;                  // tokens kernel: cuts lie by unit
  float* part_ml;               // [ctas][2][RT][2]: (max, sum) of a cut unit's piece, base 2
  float* part_acc;              // [ctas][2][D / 4][RT][4]: its unnormalised output
};
cudaError_t launch_attention_plan(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_attention_generic(const AttnParams& p, pa_dtype dtype, cudaStream_t stream);
cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t stream);
int attention_tc_rows(int G);
int attention_tc_extra();
// (their joins included)
cudaError_t launch_attention_tokens(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_attention_tokens32(const AttnParams& p, cudaStream_t stream);
bool attention_tokens_eligible(int max_query_len, int G, int B);
int attention_tokens_ranges(int sms);
cudaError_t launch_attention_join(const AttnParams& p, pa_dtype dtype, cudaStream_t stream);
int attention_generic_ctas_per_sm(int RT, int D);

// Beam search's selection (beam.cu).
struct BeamParams {
  float* scores;            // [N][k]
  int32_t *parents, *tokens;
  const void* logits;       // [N * W] rows of V, row_stride elements apart
  const float* cum;         // [N][W]
  const uint8_t* finished;  // [N][W], nullable
  int64_t row_stride;
  int N, W, V, k, eos;
  int chunks, chunk_len;    // beam_plan
  double* ws_sum;           // [N * W * chunks]
  float* ws_max;
  float* ws_val;            // [N * W * chunks][k]
  int32_t* ws_idx;
};
void beam_plan(BeamParams* p);
size_t beam_workspace_bytes(const BeamParams& p);
cudaError_t launch_beam_topk(BeamParams p, pa_dtype dtype, void* workspace, cudaStream_t stream);
cudaError_t launch_beam_gather(void* dst, const void* src, const int32_t* parents, int N, int W, int k,
                               int64_t row_bytes, int32_t* err, cudaStream_t stream);

// Tensor-core path eligibility (shape/dtype only; alignment is checked by the caller).
bool tc_eligible(int G, int D, int block_size, pa_dtype dtype);

}  // namespace pa
