// Beam search's selection over beams and vocabulary, and the reordering of per-beam states
// (sm_100a).
//
// A candidate (w, v) of request n scores cum[n][w] + x[n][w][v] - lse(x[n][w]); the best k of
// the W * V candidates are wanted, in order of (score, then lowest w * V + v).  Within a beam
// the order is that of the logits, so one pass over the logits keeps a running (max, sum of
// exponentials) and the k largest logits, and the scores are formed for those alone.
//
// Bound by reading the logits once.  Row chunks go to one CTA each; a warp walks its part
// of the chunk in 16-byte vectors (rows may begin anywhere: a row's positions are counted from the
// 16-byte boundary before it) and keeps the k best so far sorted across its lanes (lane i holds
// the i-th).  A batch none of whose values reaches the k-th best costs one comparison of its
// maximum, which the softmax needs anyway; the first batch is filtered by the k-th largest of
// the lanes' maxima, so few values are ever inserted.  A second, small kernel forms the scores of
// the W * chunks * k values kept, spread over its warps, and keeps the best k of them.  Lists are
// merged by bitonic steps across the lanes.  64 requests of 4 beams over 131072 fp32 logits: 31 us
// (4.3 TB/s) and 5 us for the join; an exponential and six more operations a logit, issue at 56 % on
// average but from 42 to 74 % by SM: 512 CTAs are three or four for each, for the whole time.
// One request of 4 x 32000: 11 us with the gather, which is launches.
//
// lse and scores are 64-bit from the chunk sums on: the chosen indices compare scores of
// different beams, which a 32-bit subtraction would round into ties.

#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// The k best (value, index) pairs, sorted over the lanes of a warp: lane i holds the i-th;
// ranked by value, then by lower index.  Empty places hold (-inf, INT_MAX).
template <typename F>
struct TopList {
  F v;
  int idx;
  F thr_v;    // the k-th entry
  int thr_i;

  __device__ __forceinline__ void init() {
    v = thr_v = static_cast<F>(-CUDART_INF);
    idx = thr_i = INT_MAX;
  }
  __device__ __forceinline__ static bool before(F a, int ia, F b, int ib) {
    return a > b || (a == b && ia < ib);
  }
  // Insert one pair, the same in every lane.
  __device__ __forceinline__ void insert(F nv, int ni, int k, int lane) {
    const int pos = __popc(__ballot_sync(kFull, before(v, idx, nv, ni)));
    const F pv = __shfl_up_sync(kFull, v, 1);
    const int pi = __shfl_up_sync(kFull, idx, 1);
    if (lane > pos) {
      v = pv;
      idx = pi;
    } else if (lane == pos) {
      v = nv;
      idx = ni;
    }
    thr_v = __shfl_sync(kFull, v, k - 1);
    thr_i = __shfl_sync(kFull, idx, k - 1);
  }
  // Exchange with the lane `off` away (a power of two): the lower one of the two keeps the better
  // pair where `down`, else the worse.
  __device__ __forceinline__ static void step(F& v, int& i, int off, bool down, int lane) {
    const F ov = __shfl_xor_sync(kFull, v, off);
    const int oi = __shfl_xor_sync(kFull, i, off);
    const bool first = ((lane & off) == 0) == down;  // this lane wants the better pair
    if (before(ov, oi, v, i) == first) {
      v = ov;
      i = oi;
    }
  }
  // Merge a list that is sorted over the lanes: the better of this list's i-th and that one's
  // (31 - i)-th are the 32 best of both, and bitonic.
  __device__ __forceinline__ void merge_sorted(F nv, int ni, int k, int lane) {
    const F rv = __shfl_sync(kFull, nv, 31 - lane);
    const int ri = __shfl_sync(kFull, ni, 31 - lane);
    if (before(rv, ri, v, idx)) {
      v = rv;
      idx = ri;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) step(v, idx, off, true, lane);
    thr_v = __shfl_sync(kFull, v, k - 1);
    thr_i = __shfl_sync(kFull, idx, k - 1);
  }
  // Offer one pair per lane (`have`: the lane has one): inserted one by one where few can enter,
  // else sorted and merged.
  __device__ __forceinline__ void offer(F nv, int ni, bool have, int k, int lane) {
    unsigned m = __ballot_sync(kFull, have && before(nv, ni, thr_v, thr_i));
    if (__popc(m) > 8) {
      if (!(m >> lane & 1)) {
        nv = static_cast<F>(-CUDART_INF);
        ni = INT_MAX;
      }
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int off = size >> 1; off > 0; off >>= 1) step(nv, ni, off, (lane & size) == 0, lane);
      merge_sorted(nv, ni, k, lane);
      return;
    }
    while (m) {
      const int src = __ffs(m) - 1;
      insert(__shfl_sync(kFull, nv, src), __shfl_sync(kFull, ni, src), k, lane);
      m &= m - 1;
      m &= __ballot_sync(kFull, have && before(nv, ni, thr_v, thr_i));
    }
  }
};

// Floats as integers of the same order (-0 below 0), and back.
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(v);
  return i < 0 ? i ^ 0x7fffffff : i;
}
__device__ __forceinline__ float unordered(int i) {
  return i == INT_MIN ? -INFINITY : __int_as_float(i < 0 ? i ^ 0x7fffffff : i);
}

// The k-th largest of the lanes' values.
__device__ __forceinline__ float kth_of_lanes(float v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off > 0; off >>= 1) {
      const float o = __shfl_xor_sync(kFull, v, off);
      v = ((lane & off) == 0) == ((lane & size) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl_sync(kFull, v, k - 1);
}

// Join the warps' lists of a CTA in pairs; warp 0 ends with the k best.  Every thread calls it.
template <typename F>
__device__ __forceinline__ void join_lists(TopList<F>& top, F (*sm_v)[32], int (*sm_i)[32], int k, int warp,
                                           int lane) {
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
      sm_v[warp][lane] = lane < k ? top.v : static_cast<F>(-CUDART_INF);
      sm_i[warp][lane] = lane < k ? top.idx : INT_MAX;
    }
    __syncthreads();
    if (warp < half) top.merge_sorted(sm_v[warp + half][lane], sm_i[warp + half][lane], k, lane);
  }
}

// 16 bytes of logits, kept as loaded until they are used.
template <typename T>
struct Load;
template <>
struct Load<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  __device__ static void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  // word w of a vector of which elements [from, to) are loaded, the others -inf
  __device__ static uint32_t word(const float* p, int w, int from, int to) {
    return w >= from && w < to ? __float_as_uint(p[w]) : kNone;
  }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xff80u;  // -inf
  __device__ static void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ static uint32_t word(const __nv_bfloat16* p, int w, int from, int to) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    const uint32_t lo = 2 * w >= from && 2 * w < to ? q[2 * w] : kNone;
    const uint32_t hi = 2 * w + 1 >= from && 2 * w + 1 < to ? q[2 * w + 1] : kNone;
    return lo | hi << 16;
  }
};

// Running (max, sum of 2^((x - max) log2 e)) of one lane.  NaN and +inf in a row end in a
// NaN sum, which marks the row as one without candidates.
struct Sum {
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ void raise(float mx) {
    if (mx > m) {
      s = m == -INFINITY ? s : s * exp2f((m - mx) * kLog2e);
      m = mx;
    }
  }
  // what add subtracts: a lane that has seen nothing but -inf keeps the reference 0 (2^-inf = 0,
  // NaN stays)
  __device__ __forceinline__ float ref() const { return m == -INFINITY ? 0.f : m; }
  __device__ __forceinline__ void add(float x, float ref) {
    // the difference first: it is exact next to the maximum, where the sum's weight lies (a
    // product with log2 e of each term would shift the whole sum by its rounding)
    s += ex2_approx((x - ref) * kLog2e);
  }
};

// One chunk of one row per CTA: blockIdx.x = row * chunks + chunk.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const BeamParams p) {
  constexpr int N = Load<T>::N;
  constexpr int U = 32 / N / 2;  // vectors in flight per lane
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(p.logits) + static_cast<int64_t>(row) * p.row_stride;
  // positions from the 16-byte boundary at or before the row: the row is [skip, skip + V)
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
  x -= skip;
  const int beg = chunk * p.chunk_len;
  const int end = static_cast<int>(min(static_cast<int64_t>(p.V) + skip, static_cast<int64_t>(beg) + p.chunk_len));
  const int k = p.k;

  // No value below `filter` is among the CTA's k best: the k-th largest of the lanes' maxima of a
  // warp's first batch, then the best of the warps' k-th values (shared as ordered integers).
  __shared__ int shared_filter;
  if (threadIdx.x == 0) shared_filter = INT_MIN;
  __syncthreads();
  float filter = -INFINITY;
  auto raise_filter = [&](float v) {
    if (v > filter) {
      filter = v;
      if (lane == 0) atomicMax(&shared_filter, ordered(v));
    }
  };

  TopList<float> top;
  top.init();
  Sum sum;
  // warps interleave: batch i of the chunk (32 * N * U values) goes to warp i % kWarps; a batch is
  // loaded while the one before it is worked on
  constexpr int BATCH = 32 * N * U, STEP = kWarps * BATCH;
  auto load = [&](int b0, uint4 (&raw)[U]) {
    if (b0 >= skip && b0 + BATCH <= end) {
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = __ldcs(reinterpret_cast<const uint4*>(x + b0 + (u * 32 + lane) * N));
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = b0 + (u * 32 + lane) * N;
      const T* q = x + at;
      if (at >= skip && at + N <= end) {
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(q));
      } else {
        const int from = skip - at, to = end - at;
        raw[u] = make_uint4(Load<T>::word(q, 0, from, to), Load<T>::word(q, 1, from, to),
                            Load<T>::word(q, 2, from, to), Load<T>::word(q, 3, from, to));
      }
    }
  };
  __shared__ float2 cand_sh[kWarps][BATCH];
  float2* cand = cand_sh[warp];
  bool first = true;
  auto work = [&](int b0, const uint4 (&raw)[U]) {
    float e[U * N];
#pragma unroll
    for (int u = 0; u < U; ++u) Load<T>::unpack(raw[u], e + u * N);
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < U * N; ++j) mx = fmaxf(mx, e[j]);
    sum.raise(mx);
    const float ref = sum.ref();
#pragma unroll
    for (int j = 0; j < U * N; ++j) sum.add(e[j], ref);
    if (first) raise_filter(kth_of_lanes(mx, k, lane));
    first = false;
    filter = fmaxf(filter, unordered(*const_cast<volatile int*>(&shared_filter)));
    const float least = fmaxf(filter, top.thr_v);
    if (!__any_sync(kFull, mx >= least)) return;
    // the candidates side by side in shared memory, then 32 at a time
    int n = 0;
#pragma unroll
    for (int j = 0; j < U * N; ++j) {
      const bool in = e[j] >= least;
      const unsigned m = __ballot_sync(kFull, in);
      if (m) {
        if (in)
          cand[n + __popc(m & ((1u << lane) - 1))] = make_float2(e[j], __int_as_float(b0 + (j / N * 32 + lane) * N + j % N));
        n += __popc(m);
      }
    }
    __syncwarp();
    for (int c = lane; c - lane < n; c += 32) {
      const float2 o = cand[min(c, n - 1)];
      const int at = __float_as_int(o.y);
      top.offer(o.x, at - skip, c < n && at >= skip && at < end, k, lane);
    }
    __syncwarp();
    raise_filter(top.thr_v);
  };
  uint4 ea[U], eb[U];
  int b0 = beg + warp * BATCH;
  if (b0 < end) load(b0, ea);
  for (; b0 < end; b0 += 2 * STEP) {
    if (b0 + STEP < end) load(b0 + STEP, eb);
    work(b0, ea);
    if (b0 + STEP >= end) break;
    if (b0 + 2 * STEP < end) load(b0 + 2 * STEP, ea);
    work(b0 + STEP, eb);
  }

  // join the lanes' sums, then the warps'
  __shared__ float sm_m[kWarps];
  __shared__ double sm_s[kWarps];
  __shared__ float sm_v[kWarps][32];
  __shared__ int sm_i[kWarps][32];
  float m = sum.m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  double s = sum.s;
  if (sum.m != -INFINITY) s *= exp2(static_cast<double>(sum.m - m) * 1.4426950408889634);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
  if (lane == 0) {
    sm_m[warp] = m;
    sm_s[warp] = s;
  }
  join_lists(top, sm_v, sm_i, k, warp, lane);  // (its barriers order the sums as well)
  if (warp != 0) return;
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  double S = 0.0;
  for (int w = 0; w < kWarps; ++w)
    S += sm_m[w] == -INFINITY ? sm_s[w]
                              : sm_s[w] * exp2(static_cast<double>(sm_m[w] - M) * 1.4426950408889634);
  const int64_t at = static_cast<int64_t>(blockIdx.x);
  if (lane == 0) {
    p.ws_max[at] = M;
    p.ws_sum[at] = S;
  }
  if (lane < k) {
    p.ws_val[at * k + lane] = top.v;
    p.ws_idx[at * k + lane] = top.idx;
  }
}

// One request per CTA.  First the beams' log-sum-exp (a warp each, kept in shared memory for up to
// kBeams at a time), then all the values kept of these beams, 32 at a time and warp.
constexpr int kBeams = 64;

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = p.k;
  __shared__ double sm_v[kWarps][32];
  __shared__ int sm_i[kWarps][32];
  __shared__ double lse_sh[kBeams];  // NaN: the beam has no ordinary candidate
  __shared__ float cum_sh[kBeams];
  __shared__ float kth_sh[kWarps];
  TopList<double> best;
  best.init();
  for (int w0 = 0; w0 < p.W; w0 += kBeams) {
    const int beams = min(kBeams, p.W - w0);
    __syncthreads();  // (the round before has read them)
    for (int w = warp; w < beams; w += kWarps) {
      const int row = n * p.W + w0 + w;
      const int64_t c0 = static_cast<int64_t>(row) * p.chunks;
      const float cum = __ldg(p.cum + row);
      const bool done = p.finished && __ldg(p.finished + row) != 0;
      float m = -INFINITY;
      for (int c = lane; c < p.chunks; c += 32) m = fmaxf(m, p.ws_max[c0 + c]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
      double s = 0.0;
      for (int c = lane; c < p.chunks; c += 32) {
        const float mc = p.ws_max[c0 + c];
        s += mc == -INFINITY ? p.ws_sum[c0 + c]
                             : p.ws_sum[c0 + c] * exp2(static_cast<double>(mc - m) * 1.4426950408889634);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
      const double lse = static_cast<double>(m) + log(s);
      const bool ordinary = !done && isfinite(lse) && isfinite(cum);
      if (lane == 0) {
        lse_sh[w] = ordinary ? lse : CUDART_NAN;
        cum_sh[w] = cum;
      }
      if (ordinary) continue;
      // a beam without an ordinary candidate: finished (its score stays, at the end token), dead
      // (score -inf) or with a sum that is not finite.  All its other candidates score -inf and
      // rank by index.
      const int base = (w0 + w) * p.V;
      if (done && isfinite(cum)) best.offer(static_cast<double>(cum), base + p.eos, lane == 0, k, lane);
      const bool skip = done && isfinite(cum) && lane == p.eos;
      // k + 1 of them: one may be the end token, ranked above already
      best.offer(-CUDART_INF, base + lane, lane < p.V && !skip, k, lane);
      if (done && k == 32) best.offer(-CUDART_INF, base + 32, lane == 0 && 32 < p.V && p.eos != 32, k, lane);
    }
    __syncthreads();
    const int per = p.chunks * k, total = beams * per;  // (W * V < 2^31 bounds it)
    const int64_t first = (static_cast<int64_t>(n) * p.W + w0) * per;
    auto candidate = [&](int e, double& score, int& at) {
      if (e >= total) return false;
      const int w = e / per, i = p.ws_idx[first + e];
      const double lse = lse_sh[w];
      if (i == INT_MAX || lse != lse) return false;
      at = (w0 + w) * p.V + i;
      score = static_cast<double>(cum_sh[w]) + (static_cast<double>(p.ws_val[first + e]) - lse);
      return true;
    };
    // as above, no score below the k-th largest of a warp's lanes' maxima is among the k best
    // (rounded down, so that it is a bound)
    double score = 0.0;
    int at = INT_MAX;
    float mx = -INFINITY;
    for (int e0 = warp * 32; e0 < total; e0 += kThreads)
      if (candidate(e0 + lane, score, at)) mx = fmaxf(mx, __double2float_rd(score));
    if (lane == 0) kth_sh[warp] = -INFINITY;
    if (warp * 32 < total) {
      const float kth = kth_of_lanes(mx, k, lane);
      if (lane == 0) kth_sh[warp] = kth;
    }
    __syncthreads();
    float filter = kth_sh[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) filter = fmaxf(filter, kth_sh[i]);
    for (int e0 = warp * 32; e0 < total; e0 += kThreads) {
      const bool have = candidate(e0 + lane, score, at) && score >= filter;
      best.offer(score, at, have, k, lane);
    }
  }
  __syncthreads();
  join_lists(best, sm_v, sm_i, k, warp, lane);
  if (warp == 0 && lane < k) {
    const int64_t at = static_cast<int64_t>(n) * k + lane;
    p.scores[at] = static_cast<float>(best.v);
    p.parents[at] = best.idx / p.V;
    p.tokens[at] = best.idx % p.V;
  }
}

// dst[n][i] = src[n][parents[n][i]], rows of `row_bytes`; one CTA row per (n, i).
template <typename V>
__global__ void __launch_bounds__(kThreads) beam_gather_kernel(V* __restrict__ dst, const V* __restrict__ src,
                                                               const int32_t* __restrict__ parents, int W, int k,
                                                               int64_t vecs, int32_t* err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  const int par = __ldg(parents + row);
  if (par < 0 || par >= W) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(err, PA_DEVERR_BAD_PARENT);
    return;
  }
  const V* s = src + (row / k * W + par) * vecs;
  V* d = dst + row * vecs;
  const int64_t step = static_cast<int64_t>(gridDim.y) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; i < vecs; i += step) d[i] = s[i];
}

template <typename T>
cudaError_t launch_rows(const BeamParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.N * p.W * p.chunks));
  return launch_pdl(beam_rows_kernel<T>, grid, kThreads, 0, stream, p);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Chunks per row: as many as keep the CTAs within four per SM, which all run at once (the few CTAs
// past one wave doubled the time of 256 rows of 131072), none below 4096 values, a
// batch for each warp (a shorter chunk is all reduction); a multiple of 8 values, so that chunks start on vector boundaries.  A row's
// positions begin up to 7 before it.
void beam_plan(BeamParams* p) {
  const int64_t rows = static_cast<int64_t>(p->N) * p->W, V = static_cast<int64_t>(p->V) + 7;
  const int64_t fit = 148 * 4 / (rows > 0 ? rows : 1), want = fit > 0 ? fit : 1;
  int64_t len = (V + want - 1) / want;
  if (len < 4096) len = 4096;
  len = (len + 7) / 8 * 8;
  p->chunk_len = static_cast<int>(len < V ? len : (V + 7) / 8 * 8);
  p->chunks = static_cast<int>((V + p->chunk_len - 1) / p->chunk_len);
}

size_t beam_workspace_bytes(const BeamParams& p) {
  const int64_t n = static_cast<int64_t>(p.N) * p.W * p.chunks;
  return static_cast<size_t>(up256(n * 8) + up256(n * 4) + 2 * up256(n * p.k * 4));
}

cudaError_t launch_beam_topk(BeamParams p, pa_dtype dtype, void* workspace, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.N) * p.W * p.chunks;
  char* ws = static_cast<char*>(workspace);
  p.ws_sum = reinterpret_cast<double*>(ws);
  p.ws_max = reinterpret_cast<float*>(ws + up256(n * 8));
  p.ws_val = reinterpret_cast<float*>(ws + up256(n * 8) + up256(n * 4));
  p.ws_idx = reinterpret_cast<int32_t*>(ws + up256(n * 8) + up256(n * 4) + up256(n * p.k * 4));
  cudaError_t e = dtype == PA_BF16 ? launch_rows<__nv_bfloat16>(p, stream) : launch_rows<float>(p, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_join_kernel, dim3(static_cast<unsigned>(p.N)), kThreads, 0, stream, p);
}

cudaError_t launch_beam_gather(void* dst, const void* src, const int32_t* parents, int N, int W, int k,
                               int64_t row_bytes, int32_t* err, cudaStream_t stream) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src) |
                      static_cast<uintptr_t>(row_bytes);
  auto go = [&](auto* type) {
    using V = std::remove_pointer_t<decltype(type)>;
    const int64_t vecs = row_bytes / static_cast<int64_t>(sizeof(V));
    int64_t gy = (vecs + kThreads * 4 - 1) / (kThreads * 4);
    if (gy > 64) gy = 64;
    return launch_pdl(beam_gather_kernel<V>, dim3(static_cast<unsigned>(N * k), static_cast<unsigned>(gy)), kThreads, 0, stream,
                  static_cast<V*>(dst), static_cast<const V*>(src), parents, W, k, vecs, err);
  };
  if (a % 16 == 0) return go(static_cast<uint4*>(nullptr));
  if (a % 4 == 0) return go(static_cast<uint32_t*>(nullptr));
  return go(static_cast<uint8_t*>(nullptr));
}

}  // namespace pa
