// What the kernels for a few query tokens per sequence share (device code): a sequence's keys, the
// scan of the units' tile counts that every CTA makes for itself, scores, and the join of units
// that are cut between ranges.
#pragma once

#include <climits>

#include "attention.h"

namespace pa {

namespace {

// Query tokens of sequence b ([q0, q0 + n); none where the span is malformed or longer than the
// caller said), its length, and the keys [lo, hi) that any of them sees.
struct Seq {
  int q0, n, L, lo, hi;
};

__device__ __forceinline__ Seq sequence(const AttnParams& p, int b, bool flag) {
  Seq s;
  s.n = attn_query_span(p, b, flag, s.q0);
  s.L = attn_len(p, b, flag);
  const int pre = p.prefix_lens ? __ldg(p.prefix_lens + b) : 0;
  s.lo = INT_MAX;
  s.hi = 0;
  for (int t = 0; t < s.n; ++t) {
    int l, h;
    attn_visible(p, s.L - s.n + t, s.L, pre, p.first_keys ? __ldg(p.first_keys + s.q0 + t) : 0, l, h);
    if (l < h) {
      s.lo = min(s.lo, l);
      s.hi = max(s.hi, h);
    }
  }
  if (s.hi == 0) s.lo = 0;
  return s;
}

__device__ __forceinline__ int upper_bound(const int* P, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (P[mid] > v) hi = mid; else lo = mid + 1;
  }
  return lo;
}

struct TilePos {
  int b, kvh, j, nt;
};

__device__ __forceinline__ TilePos locate(const int* P, int B, int Hkv, int g) {
  TilePos t;
  const int v = g / Hkv;
  t.b = upper_bound(P, B + 1, v) - 1;
  t.nt = P[t.b + 1] - P[t.b];
  const int off = g - Hkv * P[t.b];
  t.kvh = off / t.nt;
  t.j = off - t.kvh * t.nt;
  return t;
}

// Tiles (of `tile` keys) before each sequence into P[B + 1] and first keys into LO[B], by every CTA;
// rows of sequences that see nothing are zeroed, by one CTA each.
template <typename T, int THREADS>
__device__ __forceinline__ void scan_units(const AttnParams& p, int tile, int* P, int* LO, int* warp_sum) {
  const int B = p.B, Hkv = p.Hkv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr unsigned kFull = 0xffffffffu;
  T* out = static_cast<T*>(p.out);
  for (int b = threadIdx.x; b < B; b += THREADS) {
    const Seq q = sequence(p, b, blockIdx.x == 0);
    P[b] = q.hi > 0 ? (q.hi - 1) / tile - q.lo / tile + 1 : 0;
    LO[b] = q.lo;
  }
  __syncthreads();
  // sequences whose rows see nothing have no tile: their rows are zero (one CTA each)
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    if (P[b] != 0) continue;
    if (p.by_unit)
      for (int h = threadIdx.x; h < Hkv; h += THREADS)
        reinterpret_cast<int4*>(p.cuts)[b * Hkv + h] = make_int4(0, 0, 0, 0);
    int q0;
    const int n = attn_query_span(p, b, false, q0);
    uint4* o = reinterpret_cast<uint4*>(out + static_cast<int64_t>(q0) * p.Hq * p.D);
    for (int i = threadIdx.x; i < n * p.Hq * p.D * static_cast<int>(sizeof(T)) / 16; i += THREADS) o[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  {
    const int chunk = (B + THREADS - 1) / THREADS;
    const int lo = min(B, static_cast<int>(threadIdx.x) * chunk), hi = min(B, lo + chunk);
    int sum = 0;
    for (int b = lo; b < hi; ++b) sum += P[b];
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_sum[w];
    for (int b = lo; b < hi; ++b) {
      const int n = P[b];
      P[b] = run;
      run += n;
    }
    if (threadIdx.x == THREADS - 1) P[B] = run;
  }
  __syncthreads();
}

struct Row {
  int lo, hi;  // visible keys
  int pos;
  float slope;
};

// Scores of one tile for N rows of a lane.  EXACT (fp32): the cap holds to 32 bits (a few ulp of the
// score); else to 2^-22 of the cap, or to 2^-20 of the score where the cap is wide.
template <int N, bool EXACT>
struct TileScores {
  float sl2, cap_in, cap_out;
  bool biased, wide;
  int key0;
  Row row[N];
  __device__ __forceinline__ void init(const AttnParams& p) {
    sl2 = p.scale_log2;
    cap_in = p.cap_in;
    cap_out = p.cap_out;
    biased = p.slopes != nullptr;
    wide = p.cap_wide;
  }
  // row `which` is row r of unit (sequence s of batch row b, KV head kvh)
  __device__ __forceinline__ void set(const AttnParams& p, int which, const Seq& s, int b, int kvh, int r) {
    const int pre = p.prefix_lens ? __ldg(p.prefix_lens + b) : 0, tok = r / p.G;
    Row& w = row[which];
    attn_visible(p, s.L - s.n + tok, s.L, pre, p.first_keys ? __ldg(p.first_keys + s.q0 + tok) : 0, w.lo, w.hi);
    w.pos = s.L - s.n + tok;
    w.slope = p.slopes ? __ldg(p.slopes + kvh * p.G + (r - tok * p.G)) * kLog2e : 0.f;
  }
  __device__ __forceinline__ float operator()(float s, int k, int which) const {
    const Row& r = row[which];
    const int key = key0 + k;
    float x = s * sl2;
    if (cap_out > 0.f) {
      const float t = s * cap_in;
      if constexpr (EXACT) {
        x = cap_out * tanhf(t);
      } else {
        x = cap_score(t, cap_out);
        if (__builtin_expect(wide, 0) && fabsf(t) < kNearTanh) x = cap_score_near(s, t, sl2);
      }
    }
    // (the positions' difference in whole numbers: past 2^24 a float does not tell neighbours apart)
    if (biased) x = fmaf(-r.slope, fabsf(static_cast<float>(r.pos - key0) - static_cast<float>(k)), x);
    return key >= r.lo && key < r.hi ? x : -INFINITY;
  }
};

// Merge the pieces of a unit that is cut: piece i is in slot 0 of range s + i, but the first in the
// slot recorded.  Records lie by unit where units are fewer than ranges (most blocks would find
// none), else by the range the unit begins in; no pieces: not cut.  PS groups of BT threads (one per
// row and 4 columns) take pieces k, k + PS, .., kBatch of them at a time (one round trip), and are
// then combined in order.
template <typename T, int D>
__global__ void __launch_bounds__(1024) tokens_join_kernel(const AttnParams p, int BT, int PS) {
  constexpr int kBatch = 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = reinterpret_cast<const int4*>(p.cuts)[blockIdx.x];
  const int n = cut.x;
  if (n == 0) return;
  const int kvh = cut.z >> 8, rows = cut.z & 255;
  // a record that a warp which gave up (flagged) left unwritten is not followed out of range
  if (n < 0 || cut.y < 0 || (cut.y >> 1) + n > p.ctas || kvh < 0 || kvh >= p.Hkv || rows < 1 || rows > p.RT ||
      cut.w < 0 || cut.w + (rows - 1) / p.G >= p.T)
    return;
  const int grp = threadIdx.x / BT, idx = threadIdx.x - grp * BT;
  const int r = idx / (D / 4), c = idx % (D / 4) * 4;
  const bool live = r < rows;
  float M = -INFINITY, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  // scale what there is to the maximum `m`; a maximum of -inf stands for no key at all
  auto rescale = [&](float m) {
    const float w = m == -INFINITY ? 0.f : exp2f(M - m);
    l *= w;
    a.x *= w;
    a.y *= w;
    a.z *= w;
    a.w *= w;
    M = m;
  };
  auto add = [&](float w, float l2, const float4& o) {
    l = fmaf(l2, w, l);
    a.x = fmaf(o.x, w, a.x);
    a.y = fmaf(o.y, w, a.y);
    a.z = fmaf(o.z, w, a.z);
    a.w = fmaf(o.w, w, a.w);
  };
  if (live) {
    for (int i0 = grp; i0 < n; i0 += PS * kBatch) {
      float2 ml[kBatch];
      float4 o[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * PS;
        ml[b] = make_float2(-INFINITY, 0.f);
        o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          const int64_t row = (static_cast<int64_t>(i == 0 ? cut.y : (cut.y & ~1) + 2 * i)) * p.RT + r;
          ml[b] = reinterpret_cast<const float2*>(p.part_ml)[row];
          o[b] = *reinterpret_cast<const float4*>(p.part_acc + row * D + c);
        }
      }
      float top = M;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) top = fmaxf(top, ml[b].x);
      rescale(top);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) add(top == -INFINITY ? 0.f : exp2f(ml[b].x - top), ml[b].y, o[b]);
    }
  }
  if (PS > 1) {
    extern __shared__ float red[];  // [PS][BT][6]
    float* mine = red + (grp * BT + idx) * 6;
    mine[0] = M;
    mine[1] = l;
    mine[2] = a.x;
    mine[3] = a.y;
    mine[4] = a.z;
    mine[5] = a.w;
    __syncthreads();
    if (grp != 0) return;
    for (int k = 1; k < PS; ++k) {
      const float* o = red + (k * BT + idx) * 6;
      const float top = fmaxf(M, o[0]);
      rescale(top);
      add(top == -INFINITY ? 0.f : exp2f(o[0] - top), o[1], make_float4(o[2], o[3], o[4], o[5]));
    }
  }
  if (!live) return;
  const int t = r / p.G;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  T* o = static_cast<T*>(p.out) + (static_cast<int64_t>(cut.w + t) * p.Hq + kvh * p.G + (r - t * p.G)) * D + c;
  const float4 y = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  else
    *reinterpret_cast<float4*>(o) = y;
}

template <typename T, int D>
cudaError_t launch_tokens_join(const AttnParams& p, cudaStream_t stream) {
  const int BT = (p.RT * D / 4 + 31) / 32 * 32;
  // several pieces per unit are the rule where units are fewer than ranges
  const int PS = p.by_unit ? (1024 / BT < 1 ? 1 : 1024 / BT < 4 ? 1024 / BT : 4) : 1;
  return launch_pdl(tokens_join_kernel<T, D>, dim3(static_cast<unsigned>(p.by_unit ? p.B * p.Hkv : p.ctas)), BT * PS,
                    PS > 1 ? static_cast<size_t>(PS) * BT * 24 : 0, stream, p, BT, PS);
}

}  // namespace

}  // namespace pa
