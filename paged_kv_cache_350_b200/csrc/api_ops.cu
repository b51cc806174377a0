// C ABI of the operators around the decode: rotary positions, attention of ragged query tokens,
// beam selection.  Argument checks, plans and workspace carving; see include/pa.h for the
// contract of each entry point.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention.h"
#include "pa.h"
#include "pa_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool block_size_ok(int bs) { return bs == 4 || bs == 8 || bs == 16 || bs == 32; }
bool dtype_ok(pa_dtype t) { return t == PA_F32 || t == PA_BF16; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Whether [a, a + an) and [b, b + bn) bytes overlap.
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(bn) && y < x + static_cast<uint64_t>(an);
}

// CTAs assumed per launch when no device can be asked.
constexpr int kSmBound = 256;

// The plan of a pa_attention call on `sms` multiprocessors: rows per item (and per softmax
// group), keys per tile, CTAs.
struct AttnShape {
  int RT, HR, KT, ctas, max_items, extra;
};

// Which kernel a call takes: the tokens kernels (one per type) a few rows per sequence, bound by the
// cache's bytes; the tensor-core kernel bf16 with groups of at most the 128 rows of its M tile (a
// block of 4 tokens is half a swizzle atom: the pattern goes by shared-memory address, so its box
// lands like any other); CUDA cores the rest.
enum AttnKernel { kGeneric, kTensor, kTokens };

AttnKernel attention_kernel(int B, int max_query_len, int G, pa_dtype dtype) {
  if (pa::attention_tokens_eligible(max_query_len, G, B)) return kTokens;
  return dtype == PA_BF16 && G <= 128 ? kTensor : kGeneric;
}

AttnShape attention_shape(int T, int B, int max_query_len, int G, int D, AttnKernel kernel, int sms) {
  AttnShape s{};
  if (kernel == kTokens) {
    s.KT = 8;  // (16 in bf16)
    s.RT = s.HR = max_query_len * G;
    s.ctas = pa::attention_tokens_ranges(sms);
    s.max_items = 0;
    return s;
  }
  if (kernel == kTensor) {
    s.KT = 128;
    s.RT = pa::attention_tc_rows(G);
    s.HR = s.RT / 2;
    s.ctas = sms;
    s.extra = pa::attention_tc_extra();
  } else {
    s.KT = 64;
    s.RT = s.HR = static_cast<int64_t>(max_query_len) * G <= 16 ? 16 : 64;
    s.ctas = sms * pa::attention_generic_ctas_per_sm(s.RT, D);
  }
  s.max_items = static_cast<int>(static_cast<int64_t>(T) * G / s.RT + std::min(B, T));
  return s;
}

// Byte offsets of the plan's arrays and the partials; returns the total.
size_t attention_carve(const AttnShape& s, int B, int D, char* ws, pa::AttnParams* p) {
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += up256(bytes);
    return at;
  };
  const int64_t header = take(16), seq = take(int64_t(B) * 4);
  const int64_t items = take(int64_t(s.max_items) * sizeof(pa::AttnItem));
  const int64_t sums = take((int64_t(s.max_items) + 1) * 4);
  const int64_t starts = take(int64_t(s.ctas) * sizeof(pa::AttnStart)), cuts = take(int64_t(s.ctas) * sizeof(pa::AttnCut));
  const int64_t ml = take(int64_t(s.ctas) * 2 * s.RT * 8);
  const int64_t acc = take(int64_t(s.ctas) * 2 * s.RT * D * 4);
  if (p) {
    p->RT = s.RT;
    p->HR = s.HR;
    p->extra = s.extra;
    p->KT = s.KT;
    p->ctas = s.ctas;
    p->max_items = s.max_items;
    p->header = reinterpret_cast<int32_t*>(ws + header);
    p->seq_items = reinterpret_cast<int32_t*>(ws + seq);
    p->items = reinterpret_cast<pa::AttnItem*>(ws + items);
    p->tile_sum = reinterpret_cast<int32_t*>(ws + sums);
    p->starts = reinterpret_cast<pa::AttnStart*>(ws + starts);
    p->cuts = reinterpret_cast<int32_t*>(ws + cuts);
    p->part_ml = reinterpret_cast<float*>(ws + ml);
    p->part_acc = reinterpret_cast<float*>(ws + acc);
  }
  return static_cast<size_t>(off);
}

bool attention_sizes_ok(int T, int B, int max_query_len, int Hq, int Hkv) {
  return T >= 0 && B >= 0 && max_query_len >= 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 &&
         static_cast<int64_t>(T) * (Hq / Hkv) < (int64_t(1) << 30);
}

}  // namespace

int pa::device_sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool kept = dev >= 0 && dev < kMaxDevices;
  if (kept && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (kept) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

extern "C" {

pa_status pa_rope_frequencies(int rotary_dim, double base, pa_rope_scaling scaling, double factor,
                              int original_len, double fast, double slow, double* inv_freq,
                              float* attn_factor) {
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base) || !inv_freq || !attn_factor)
    return PA_ERR_INVALID_ARG;
  if (scaling < PA_ROPE_SCALE_NONE || scaling > PA_ROPE_SCALE_BANDS) return PA_ERR_INVALID_ARG;
  if (scaling != PA_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return PA_ERR_INVALID_ARG;
  const bool by_turns = scaling == PA_ROPE_SCALE_RAMP || scaling == PA_ROPE_SCALE_BANDS;
  if (by_turns && (original_len <= 0 || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return PA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int half = rotary_dim / 2;
  double b = base;
  if (scaling == PA_ROPE_SCALE_BASE && rotary_dim > 2)
    b = base * std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  // ramp: the (fractional) index of the pair that turns r times in original_len positions
  auto index_of = [&](double r) {
    return rotary_dim * std::log(original_len / (r * two_pi)) / (2.0 * std::log(base));
  };
  double lo = 0.0, hi = 0.0;
  if (scaling == PA_ROPE_SCALE_RAMP) {
    lo = std::max(std::floor(index_of(fast)), 0.0);
    hi = std::min(std::ceil(index_of(slow)), static_cast<double>(rotary_dim - 1));
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(b, -2.0 * i / rotary_dim);
    double keep = 1.0;  // 1: as trained, 0: interpolated
    if (scaling == PA_ROPE_SCALE_LINEAR) keep = 0.0;
    if (scaling == PA_ROPE_SCALE_RAMP)
      keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
    if (scaling == PA_ROPE_SCALE_BANDS)
      keep = std::min(std::max((original_len * f / two_pi - slow) / (fast - slow), 0.0), 1.0);
    inv_freq[i] = keep * f + (1.0 - keep) * (scaling == PA_ROPE_SCALE_NONE ? f : f / factor);
  }
  *attn_factor = scaling == PA_ROPE_SCALE_RAMP && factor > 1.0
                     ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return PA_OK;
}

pa_status pa_rope_and_cache(void* q_out, const void* q, const void* k, const void* v, void* k_pool,
                            void* v_pool, const int32_t* positions, const int64_t* slot_mapping,
                            const double* inv_freq, int T, int Hq, int Hkv, int D, int block_size,
                            int num_blocks, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                            int rotary_dim, pa_rope_layout layout, float attn_factor, pa_dtype dtype,
                            int32_t* dev_err_flag, pa_stream_t stream) {
  if (T < 0 || Hq <= 0 || Hkv <= 0 || num_blocks <= 0 || block_size <= 0 || !dtype_ok(dtype) ||
      rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > D || !std::isfinite(attn_factor) ||
      (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED))
    return PA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (!block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
  const int64_t heads = static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv);
  if (heads * D > 0x3fffffffLL || q_stride < static_cast<int64_t>(Hq) * D ||
      k_stride < static_cast<int64_t>(Hkv) * D || v_stride < static_cast<int64_t>(Hkv) * D)
    return PA_ERR_INVALID_ARG;
  if (T == 0) return PA_OK;
  const int esize = dtype == PA_BF16 ? 2 : 4;
  if (!q_out || !q || !k || !v || !k_pool || !v_pool || !positions || !slot_mapping || !inv_freq)
    return PA_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(q, esize) ||
      !aligned(k, esize) || !aligned(v, esize) || !aligned(positions, 4) || !aligned(slot_mapping, 8) ||
      !aligned(inv_freq, 8) || (dev_err_flag && !aligned(dev_err_flag, 4)))
    return PA_ERR_INVALID_ARG;
  // in place only where every thread reads what it writes
  const int64_t row = static_cast<int64_t>(Hq) * D;
  if (!(q_out == q && (q_stride == row || T == 1)) &&
      overlap(q_out, T * row * esize, q, ((T - 1) * q_stride + row) * esize))
    return PA_ERR_INVALID_ARG;
  pa::RopeParams p{};
  p.q_out = q_out;
  p.q = q;
  p.k = k;
  p.v = v;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.positions = positions;
  p.slots = slot_mapping;
  p.inv_freq = inv_freq;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.R = rotary_dim;
  p.half = layout == PA_ROPE_HALF;
  p.factor = attn_factor;
  p.err = dev_err_flag;
  return pa::launch_rope(p, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_attention_workspace_size(int T, int B, int max_query_len, int Hq, int Hkv, int D,
                                   int block_size, int max_blocks) {
  if (!attention_sizes_ok(T, B, max_query_len, Hq, Hkv) || (D != 64 && D != 128) ||
      !block_size_ok(block_size) || max_blocks <= 0)
    return static_cast<size_t>(-1);
  if (T == 0 || B == 0) return 0;
  const int known = pa::device_sms(), sms = known > 0 ? known : kSmBound;
  size_t n = 0;  // enough for either type
  const int most = std::max(max_query_len, 1), G = Hq / Hkv;
  for (const pa_dtype dtype : {PA_F32, PA_BF16})
    n = std::max(n, attention_carve(attention_shape(T, B, most, G, D, attention_kernel(B, most, G, dtype), sms),
                                    B, D, nullptr, nullptr));
  return n;
}

pa_status pa_attention(void* out, const void* q, const void* k_pool, const void* v_pool,
                       const int32_t* block_tables, const int32_t* seq_lens,
                       const int32_t* query_starts, int T, int B, int max_query_len, int Hq, int Hkv,
                       int D, int block_size, int max_blocks, int num_blocks, int64_t q_stride,
                       float scale, const pa_attention_mods* mods, pa_dtype dtype, void* workspace,
                       size_t workspace_bytes, int32_t* dev_err_flag, pa_stream_t stream) {
  const pa_attention_mods none{};
  const pa_attention_mods& m = mods ? *mods : none;
  if (!attention_sizes_ok(T, B, max_query_len, Hq, Hkv) || max_blocks <= 0 || num_blocks <= 0 ||
      block_size <= 0 || !(std::fabs(scale) <= 1e30f) || !dtype_ok(dtype) || m.window < 0 ||
      !(m.softcap == 0.f || (m.softcap >= 1e-30f && m.softcap <= 1e30f)))
    return PA_ERR_INVALID_ARG;
  // (scale / softcap is held in 32 bits)
  if (m.softcap > 0.f && !(std::fabs(static_cast<double>(scale) / m.softcap) <= 1e30)) return PA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (!block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
  const int64_t max_seq = static_cast<int64_t>(max_blocks) * block_size;
  if (max_seq > 0x7fffff00LL) return PA_ERR_INVALID_ARG;
  const int esize = dtype == PA_BF16 ? 2 : 4;
  if (q_stride < static_cast<int64_t>(Hq) * D || q_stride * esize % 16 != 0) return PA_ERR_INVALID_ARG;
  if (T == 0 || B == 0 || max_query_len == 0) return PA_OK;
  if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !query_starts || !workspace)
    return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_starts, 4) ||
      !aligned(workspace, 256) || (dev_err_flag && !aligned(dev_err_flag, 4)) ||
      (m.alibi_slopes && !aligned(m.alibi_slopes, 4)) || (m.prefix_lens && !aligned(m.prefix_lens, 4)) ||
      (m.first_keys && !aligned(m.first_keys, 4)))
    return PA_ERR_INVALID_ARG;
  // (a unit's output may be written before another one has read its queries)
  const int64_t row = static_cast<int64_t>(Hq) * D;
  if (overlap(out, T * row * esize, q, ((T - 1) * q_stride + row) * esize)) return PA_ERR_INVALID_ARG;
  const int sms = pa::device_sms();
  if (sms <= 0) return PA_ERR_CUDA;
  const int G = Hq / Hkv;
  const AttnKernel kernel = attention_kernel(B, max_query_len, G, dtype);
  const AttnShape sh = attention_shape(T, B, max_query_len, G, D, kernel, sms);
  // tile counts are summed in 32 bits: of one KV head, or of all in the tokens kernel
  const int64_t rows = kernel == kTokens ? static_cast<int64_t>(B) * Hkv : sh.max_items;
  if (rows * (max_seq / sh.KT + 2 + sh.extra) >= (int64_t(1) << 31)) return PA_ERR_UNSUPPORTED;
  pa::AttnParams p{};
  if (workspace_bytes < attention_carve(sh, B, D, static_cast<char*>(workspace), &p)) return PA_ERR_INVALID_ARG;
  const double log2e = 1.4426950408889634;
  p.out = out;
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_starts = query_starts;
  p.prefix_lens = m.prefix_lens;
  p.first_keys = m.first_keys;
  p.slopes = m.alibi_slopes;
  p.q_stride = q_stride;
  p.scale_log2 = static_cast<float>(scale * log2e);
  p.cap_in = m.softcap > 0.f ? static_cast<float>(static_cast<double>(scale) / m.softcap) : 0.f;
  p.cap_out = m.softcap > 0.f ? static_cast<float>(m.softcap * log2e) : 0.f;
  {
    // tanh(t) / t in powers of t^2 (attention_tc.cu), of t = cap_in * x and times cap_out; where the
    // powers of cap_in leave the range of 32 bits the polynomial is not used (a bound of inf)
    static const double kTanh[5] = {0.9999918341636658, -0.3330950140953064, 0.13136771321296692,
                                    -0.04714450612664223, 0.01063788216561079};
    const double ci = m.softcap > 0.f ? static_cast<double>(scale) / m.softcap : 0.0;
    for (int k = 0; k < 5; ++k) p.cap_poly[k] = static_cast<float>(kTanh[k] * m.softcap * log2e * std::pow(ci, 2 * k + 1));
    p.cap_wide = m.softcap > pa::kWideCap;
    const bool usable = std::fabs(ci) >= 1e-3 && std::fabs(ci) <= 1e3 && m.softcap >= 1e-6f && !p.cap_wide;
    p.cap_small = usable ? static_cast<float>(std::fabs(ci)) : INFINITY;
    // One reference for all scores within +-cap_out: their weights lie in 2^(top - 2 cap_out) ..
    // 2^top, so top is as low as keeps the smallest above 2^-80, at most 40; inf: none would keep it
    // above 2^-105 (products with V and their sums are to stay normal numbers).
    const float top = std::min(std::max(2.f * p.cap_out - 80.f, 8.f), 40.f);
    p.cap_ref = 2.f * p.cap_out - top <= 105.f ? p.cap_out - top : INFINITY;
  }
  p.window = m.window;
  p.T = T;
  p.B = B;
  p.max_query_len = max_query_len;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.D = D;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.err = dev_err_flag;
  p.dynamic = kernel == kTensor;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (kernel == kTokens) {
    e = dtype == PA_BF16 ? pa::launch_attention_tokens(p, s) : pa::launch_attention_tokens32(p, s);
  } else {
    e = pa::launch_attention_plan(p, s);
    if (e == cudaSuccess)
      e = kernel == kTensor ? pa::launch_attention_tc(p, s) : pa::launch_attention_generic(p, dtype, s);
    if (e == cudaSuccess) e = pa::launch_attention_join(p, dtype, s);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

static bool beam_sizes_ok(int N, int W, int V, int k) {
  return N >= 0 && W > 0 && V > 0 && V <= (1 << 30) && k > 0 &&
         static_cast<int64_t>(W) * V < (int64_t(1) << 31) && k <= static_cast<int64_t>(W) * V;
}

size_t pa_beam_topk_workspace_size(int N, int W, int V, int k) {
  if (!beam_sizes_ok(N, W, V, k) || k > 32) return static_cast<size_t>(-1);
  if (N == 0) return 0;
  pa::BeamParams p{};
  p.N = N;
  p.W = W;
  p.V = V;
  p.k = k;
  pa::beam_plan(&p);
  return pa::beam_workspace_bytes(p);
}

pa_status pa_beam_topk(float* scores, int32_t* parents, int32_t* tokens, const void* logits,
                       const float* cum_scores, const uint8_t* finished, int eos_token, int N, int W,
                       int V, int k, int64_t row_stride, pa_dtype dtype, void* workspace,
                       size_t workspace_bytes, pa_stream_t stream) {
  if (!beam_sizes_ok(N, W, V, k) || !dtype_ok(dtype) || row_stride < V ||
      (finished && (eos_token < 0 || eos_token >= V)))
    return PA_ERR_INVALID_ARG;
  if (k > 32) return PA_ERR_UNSUPPORTED;
  if (N == 0) return PA_OK;
  if (!scores || !parents || !tokens || !logits || !cum_scores || !workspace) return PA_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(parents, 4) || !aligned(tokens, 4) ||
      !aligned(logits, dtype == PA_BF16 ? 2 : 4) || !aligned(cum_scores, 4) || !aligned(workspace, 256))
    return PA_ERR_INVALID_ARG;
  // a request's scores so far are read before its new ones are written
  if (!(scores == cum_scores && k == W) &&
      overlap(scores, static_cast<int64_t>(N) * k * 4, cum_scores, static_cast<int64_t>(N) * W * 4))
    return PA_ERR_INVALID_ARG;
  pa::BeamParams p{};
  p.scores = scores;
  p.parents = parents;
  p.tokens = tokens;
  p.logits = logits;
  p.cum = cum_scores;
  p.finished = finished;
  p.row_stride = row_stride;
  p.N = N;
  p.W = W;
  p.V = V;
  p.k = k;
  p.eos = eos_token;
  pa::beam_plan(&p);
  if (static_cast<int64_t>(N) * W * p.chunks > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  if (workspace_bytes < pa::beam_workspace_bytes(p)) return PA_ERR_INVALID_ARG;
  return pa::launch_beam_topk(p, dtype, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_beam_gather(void* dst, const void* src, const int32_t* parents, int N, int W, int k,
                         int64_t row_bytes, int32_t* dev_err_flag, pa_stream_t stream) {
  if (N < 0 || W <= 0 || k <= 0 || row_bytes < 0 || static_cast<int64_t>(N) * k > 0x7fffffffLL)
    return PA_ERR_INVALID_ARG;
  if (N == 0 || row_bytes == 0) return PA_OK;
  if (!dst || !src || !parents || !aligned(parents, 4) || (dev_err_flag && !aligned(dev_err_flag, 4)))
    return PA_ERR_INVALID_ARG;
  if (overlap(dst, static_cast<int64_t>(N) * k * row_bytes, src, static_cast<int64_t>(N) * W * row_bytes))
    return PA_ERR_INVALID_ARG;
  return pa::launch_beam_gather(dst, src, parents, N, W, k, row_bytes, dev_err_flag,
                                reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
