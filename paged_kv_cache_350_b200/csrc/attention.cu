// Attention of ragged query tokens over the paged cache (sm_100a): the work plan, the CUDA-core
// kernel and the join of units that are cut between CTAs.
//
// For query token i of a sequence of L cached tokens with n query tokens, at position
// p = L - n + i, and head h:
//   x_j = scale * q.k_j;  c * tanh(x_j / c) with a cap c;  x_j - slope_h |p - j| with a bias;
//   out = softmax over the visible j of x_j, times v_j;  0 where nothing is visible.
// The visible keys of a token are one interval [lo, hi) (attention.h), so a mask is two numbers
// per row, and tiles of keys outside an item's interval are never read.
//
// Work plan.  An item is RT consecutive rows ((token, head of the group) pairs) of a sequence;
// with one KV head it is a unit of nt = tiles of KT keys that its rows may see.  All units lie
// end to end (item, then KV head, then tile) and every CTA of one wave takes an equal contiguous
// range, whatever mixture of lengths and masks the batch is: a long axis with few rows is split
// and a short one is not by the same rule.  Before its tiles a unit counts `extra` more, which
// stand for its loads of Q and its output, so that ranges of many short units are not the last
// to end.  A unit cut by a range's end leaves partials (max, sum, unnormalised output; base 2)
// that attention_join_kernel merges by log-sum-exp.  Where there are many units for a CTA (the
// tensor-core kernel, from kDynamicUnits on) they are not cut but taken one by one, the longest of
// a sequence first: CTAs with equal shares were up to 30 % apart in time, and the partials and their
// join are saved (8 prompts of 2048 tokens: 381 -> 341 us).  Each unit is computed in the same way
// whichever CTA takes it.
//
// CUDA-core kernel: fp32 inputs (no TF32) and bf16 with more than 128 query heads per KV head, from 17
// rows per sequence on.  A CTA holds a tile of RT rows of Q, and K and V tiles of 64 keys as fp32
// in shared memory; a thread computes MR x 4 scores and MR x D/16 outputs in registers.  Bound by the
// products' shared-memory reads (17 TFLOP/s for 8 prompts of 512 tokens).  The 16-row variant is
// for batches of more sequences than the kernels for few rows scan.

#include <cuda_bf16.h>
#include <limits.h>

#include "attention.h"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlanThreads = 1024;
constexpr int kPlanKept = 4096;  // sequences, items
constexpr int kDynamicUnits = 8;  // units a CTA

// ---- plan --------------------------------------------------------------------------------

// Exclusive scan over the CTA's threads; returns the total too.
template <typename I>
__device__ __forceinline__ I block_scan(I v, I* warp_sums, I& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const I o = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const I w = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
    I s = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const I o = __shfl_up_sync(kFull, s, off);
      if (lane >= off) s += o;
    }
    warp_sums[lane] = s - w;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  const I r = warp_sums[warp] + incl - v;
  total = warp_sums[32];
  __syncthreads();
  return r;
}

// One CTA.  Sequences' item counts are scanned, then each item's interval and tile count,
// then the tile counts; last, where each CTA of the main kernel begins.
__global__ void __launch_bounds__(kPlanThreads) attention_plan_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int sums[33];
  // what the searches below read, in shared memory where it fits (each step of a search is a
  // round trip)
  __shared__ int seq_sh[kPlanKept], sum_sh[kPlanKept];
  int* seq_items = p.B <= kPlanKept ? seq_sh : p.seq_items;
  int* slots_before = p.max_items < kPlanKept ? sum_sh : p.tile_sum;
  // overlapping spans (malformed) could exceed the host's bound, and 32 bits
  __shared__ int64_t wide_sums[33];
  int64_t counted = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0, total;
    int q0;
    if (b < p.B) n = (static_cast<int64_t>(attn_query_span(p, b, true, q0)) * p.G + p.RT - 1) / p.RT;
    const int64_t at = block_scan(n, wide_sums, total);
    if (b < p.B) seq_items[b] = static_cast<int>(min(counted + at, static_cast<int64_t>(INT_MAX)));
    counted += total;
  }
  if (counted > p.max_items && threadIdx.x == 0) flag_error(p.err, PA_DEVERR_BAD_SEQ_LEN);
  const int items = static_cast<int>(min(counted, static_cast<int64_t>(p.max_items)));
  __syncthreads();
  __shared__ int filled;  // items with tiles
  if (threadIdx.x == 0) filled = 0;
  __syncthreads();
  int tiles = 0;
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int nt = 0;
    if (i < items) {
      int a = 0, z = p.B;  // the last sequence whose items begin at or before i
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (seq_items[mid] <= i) a = mid; else z = mid;
      }
      AttnItem it;
      it.b = a;
      const int n = attn_query_span(p, a, false, it.q0);
      const int nrows = n * p.G;
      it.row0 = (i - seq_items[a]) * p.RT;
      it.rows = min(p.RT, nrows - it.row0);
      it.L = attn_len(p, a, true);
      it.pos0 = it.L - n;
      const int pre = p.prefix_lens ? __ldg(p.prefix_lens + a) : 0;
      it.lo = INT_MAX;
      it.hi = 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int r0 = it.row0 + g * p.HR, r1 = min(r0 + p.HR, it.row0 + it.rows);
        int lo = INT_MAX, hi = 0;
        if (r0 < r1) {
          const int t0 = r0 / p.G, t1 = (r1 - 1) / p.G;
          auto take = [&](int t, int first) {
            int l, h;
            attn_visible(p, it.pos0 + t, it.L, pre, first, l, h);
            if (l < h) {
              lo = min(lo, l);
              hi = max(hi, h);
            }
          };
          if (p.first_keys) {
            for (int t = t0; t <= t1; t += 32) {  // (one round trip for the usual item)
              int first[32];
#pragma unroll
              for (int u = 0; u < 32; ++u) first[u] = __ldg(p.first_keys + it.q0 + min(t + u, t1));
#pragma unroll
              for (int u = 0; u < 32; ++u) take(min(t + u, t1), first[u]);
            }
          } else {  // both ends are monotone in the token (from position 0 on, which sees key 0)
            take(max(t0, min(-it.pos0, t1)), 0);
            take(t1, 0);
          }
        }
        it.glo[g] = hi > 0 ? lo : 0;
        it.ghi[g] = hi;
        it.lo = min(it.lo, lo);
        it.hi = max(it.hi, hi);
      }
      if (it.hi == 0) it.lo = 0;
      p.items[i] = it;
      nt = it.hi > 0 ? (it.hi - 1) / p.KT - it.lo / p.KT + 1 + p.extra : 0;
    }
    int total;
    const int at = block_scan(nt, sums, total);
    if (nt > 0) atomicAdd(&filled, 1);
    if (i < items) slots_before[i] = p.tile_sum[i] = tiles + at;
    tiles += total;
  }
  if (threadIdx.x == 0) {
    slots_before[items] = p.tile_sum[items] = tiles;
    p.header[0] = items;
    p.header[1] = tiles;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.header[2] = p.dynamic && static_cast<int64_t>(filled) * p.Hkv >= static_cast<int64_t>(kDynamicUnits) * p.ctas;
    p.header[3] = 0;
  }
  const int64_t T = static_cast<int64_t>(tiles) * p.Hkv;
  const int64_t per = (T + p.ctas - 1) / p.ctas;
  for (int s = threadIdx.x; s < p.ctas; s += kPlanThreads) {
    const int64_t beg = min(T, s * per), end = min(T, beg + per);
    AttnStart st{0, 0, 0, static_cast<int>(end - beg)};
    if (beg < end) {
      const int v = static_cast<int>(beg / p.Hkv);
      int a = 0, z = items;  // the last item whose tiles begin at or before v (and has some)
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (slots_before[mid] <= v) a = mid; else z = mid;
      }
      const int nt = slots_before[a + 1] - slots_before[a];
      const int off = static_cast<int>(beg - static_cast<int64_t>(slots_before[a]) * p.Hkv);
      st.item = a;
      st.kvh = off / nt;
      st.tile = off - st.kvh * nt;
    }
    p.starts[s] = st;
  }
}

// ---- CUDA-core kernel -----------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

constexpr int kGenKT = 64;
constexpr int kGenThreads = 256;

template <int D, int MR>
struct GenCfg {
  static constexpr int RT = 16 * MR;
  static constexpr int KS = D + 4;       // row stride of Q and K: 16 rows fall on 16 bank groups
  static constexpr int PS = kGenKT + 4;  // row stride of P
  static constexpr int SMEM = (RT * KS + kGenKT * KS + kGenKT * D + RT * PS) * 4;
};

template <typename T, int D, int MR>
__global__ void __launch_bounds__(kGenThreads) attention_generic_kernel(const AttnParams p) {
  using C = GenCfg<D, MR>;
  constexpr int RT = C::RT, KS = C::KS, PS = C::PS, NC = D / 64;  // NC float4 of output per row
  // the join may launch; it waits for this grid to complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float smem_f[];
  float* Qs = smem_f;
  float* Ks = Qs + RT * KS;
  float* Vs = Ks + kGenKT * KS;
  float* Ps = Vs + kGenKT * D;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int s = blockIdx.x;
  const int items = p.header[0];
  const int64_t tiles = static_cast<int64_t>(p.header[1]) * p.Hkv;
  const int64_t per = (tiles + p.ctas - 1) / p.ctas;
  const AttnStart st = p.starts[s];
  T* out = static_cast<T*>(p.out);
  const T* q = static_cast<const T*>(p.q);
  const T* kp = static_cast<const T*>(p.k_pool);
  const T* vp = static_cast<const T*>(p.v_pool);

  // items whose rows see nothing have no tile: their rows are zero
  for (int i = s; i < items; i += p.ctas) {
    if (p.tile_sum[i + 1] != p.tile_sum[i]) continue;
    const AttnItem it = p.items[i];
    const int n4 = it.rows * D / 4;
    for (int h = 0; h < p.Hkv; ++h)
      for (int e = tid; e < n4; e += kGenThreads) {
        const int r = it.row0 + e / (D / 4);
        store4(out + (static_cast<int64_t>(it.q0 + r / p.G) * p.Hq + h * p.G + r % p.G) * D + e % (D / 4) * 4,
               make_float4(0.f, 0.f, 0.f, 0.f));
      }
  }

  AttnCut own{};
  int left = st.count, item = st.item, kvh = st.kvh, tile = st.tile;
  bool first_piece = true;
  while (left > 0) {
    const AttnItem it = p.items[item];
    const int slots = p.tile_sum[item + 1] - p.tile_sum[item];
    if (slots == 0) {
      ++item;
      continue;
    }
    UnitPart u = unit_part(p, slots, tile, left);
    left -= u.slots;
    if (u.cnt == 0) {  // the range ends before the unit's first tile
      tile = 0;
      continue;
    }
    const int nt = u.nt, cnt = u.cnt;
    tile = u.tile;
    const int pre = p.prefix_lens ? __ldg(p.prefix_lens + it.b) : 0;
    __syncthreads();  // the last piece's reads of Q are done
    for (int e = tid; e < RT * (D / 4); e += kGenThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < it.rows) {
        const int f = it.row0 + r;
        v = load4(q + static_cast<int64_t>(it.q0 + f / p.G) * p.q_stride +
                  static_cast<int64_t>(kvh * p.G + f % p.G) * D + c);
      }
      *reinterpret_cast<float4*>(Qs + r * KS + c) = v;
    }
    // this thread's rows
    int lo[MR], hi[MR], pos[MR];
    float slope[MR], m[MR], l[MR];
    float4 acc[MR][NC];
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const int r = ty * MR + i, f = it.row0 + min(r, it.rows - 1);
      const int t = f / p.G;
      pos[i] = it.pos0 + t;
      attn_visible(p, pos[i], it.L, pre, p.first_keys ? __ldg(p.first_keys + it.q0 + t) : 0, lo[i], hi[i]);
      slope[i] = p.slopes ? __ldg(p.slopes + kvh * p.G + f % p.G) * kLog2e : 0.f;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int32_t* tab = p.block_tables + static_cast<int64_t>(it.b) * p.max_blocks;
    const int kt0 = it.lo / kGenKT;
    for (int j = 0; j < cnt; ++j) {
      const int k0 = (kt0 + tile + j) * kGenKT;
      __syncthreads();  // the tile before is consumed (and Q is written)
      for (int e = tid; e < kGenKT * (D / 4); e += kGenThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        const int key = k0 + r;
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (key >= it.lo && key < it.hi) {
          int phys = __ldg(tab + key / p.block_size);
          if (phys < 0 || phys >= p.num_blocks) {
            flag_error(p.err, PA_DEVERR_BAD_BLOCK_ID);
            phys = 0;
          }
          const int64_t at = ((static_cast<int64_t>(phys) * p.block_size + key % p.block_size) * p.Hkv + kvh) * D + c;
          kv = load4(kp + at);
          vv = load4(vp + at);
        }
        *reinterpret_cast<float4*>(Ks + r * KS + c) = kv;
        *reinterpret_cast<float4*>(Vs + r * D + c) = vv;
      }
      __syncthreads();
      // scores of rows ty*MR + i and keys tx + 16 * u
      float x[MR][4];
#pragma unroll
      for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[MR], b[4];
#pragma unroll
        for (int i = 0; i < MR; ++i) a[i] = *reinterpret_cast<const float4*>(Qs + (ty * MR + i) * KS + d);
#pragma unroll
        for (int u = 0; u < 4; ++u) b[u] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * u) * KS + d);
#pragma unroll
        for (int i = 0; i < MR; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            x[i][u] = fmaf(a[i].x, b[u].x, x[i][u]);
            x[i][u] = fmaf(a[i].y, b[u].y, x[i][u]);
            x[i][u] = fmaf(a[i].z, b[u].z, x[i][u]);
            x[i][u] = fmaf(a[i].w, b[u].w, x[i][u]);
          }
      }
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = k0 + tx + 16 * u;
          float y = p.cap_out > 0.f ? p.cap_out * tanhf(x[i][u] * p.cap_in) : x[i][u] * p.scale_log2;
          y -= slope[i] * fabsf(static_cast<float>(pos[i] - key));
          x[i][u] = key >= lo[i] && key < hi[i] ? y : -INFINITY;
          mx = fmaxf(mx, x[i][u]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // no key yet: every p is 0
        const float alpha = exp2f(m[i] - ref);
        m[i] = mn;
        l[i] *= alpha;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float e = exp2f(x[i][u] - ref);
          l[i] += e;
          Ps[(ty * MR + i) * PS + tx + 16 * u] = e;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          acc[i][c].x *= alpha;
          acc[i][c].y *= alpha;
          acc[i][c].z *= alpha;
          acc[i][c].w *= alpha;
        }
      }
      __syncwarp();  // a row's P is written and read by one half-warp
#pragma unroll 2
      for (int k = 0; k < kGenKT; k += 4) {
        float4 a[MR];
#pragma unroll
        for (int i = 0; i < MR; ++i) a[i] = *reinterpret_cast<const float4*>(Ps + (ty * MR + i) * PS + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(Vs + (k + kk) * D + c * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < MR; ++i) {
              const float w = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
              acc[i][c].x = fmaf(w, v.x, acc[i][c].x);
              acc[i][c].y = fmaf(w, v.y, acc[i][c].y);
              acc[i][c].z = fmaf(w, v.z, acc[i][c].z);
              acc[i][c].w = fmaf(w, v.w, acc[i][c].w);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(kFull, l[i], off);
    const bool whole = tile == 0 && cnt == nt;
    const int slot = first_piece ? 0 : 1;
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const int r = ty * MR + i;
      if (r >= it.rows) continue;
      if (whole) {
        const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // NaN stays
        const int f = it.row0 + r;
        T* o = out + (static_cast<int64_t>(it.q0 + f / p.G) * p.Hq + kvh * p.G + f % p.G) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          store4(o + c * 64 + tx * 4, make_float4(acc[i][c].x * inv, acc[i][c].y * inv, acc[i][c].z * inv,
                                                  acc[i][c].w * inv));
      } else {
        const int64_t base = static_cast<int64_t>(s) * 2 + slot;
        if (tx == 0) reinterpret_cast<float2*>(p.part_ml)[base * RT + r] = make_float2(m[i], l[i]);
#pragma unroll
        for (int c = 0; c < NC; ++c)
          reinterpret_cast<float4*>(p.part_acc)[(base * (D / 4) + c * 16 + tx) * RT + r] = acc[i][c];
      }
    }
    if (!whole && tile == 0) {  // the unit begins here: its pieces follow in the next CTAs
      const int64_t ubeg = static_cast<int64_t>(p.tile_sum[item]) * p.Hkv + static_cast<int64_t>(kvh) * slots;
      own = AttnCut{static_cast<int>((ubeg + slots - 1) / per) - s + 1, slot, kvh, it.q0, it.row0, it.rows, 0, 0};
    }
    first_piece = false;
    tile = 0;
    if (++kvh == p.Hkv) {
      kvh = 0;
      ++item;
    }
  }
  if (tid == 0) reinterpret_cast<AttnCut*>(p.cuts)[s] = own;
}

// ---- join -----------------------------------------------------------------------------------

// Merge the pieces of the unit that begins in CTA s and continues in the next ones: piece 0 in
// the slot that CTA recorded, the others in slot 0.  32 rows per block (lanes), warps over the
// columns; partials lie [D/4][RT] so that a warp reads 512 consecutive bytes.
template <typename T, int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kBatch = 4;
  const int s = blockIdx.x;
  const AttnCut cut = reinterpret_cast<const AttnCut*>(p.cuts)[s];
  if (cut.pieces == 0) return;
  const int RT = p.RT;
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  if (r >= cut.rows) return;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const float4* acc = reinterpret_cast<const float4*>(p.part_acc);
  auto base = [&](int i) { return static_cast<int64_t>(s + i) * 2 + (i == 0 ? cut.slot : 0); };
  constexpr int NC = D / 4 / 8;
  float M = -INFINITY, l = 0.f;
  float4 a[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  // kBatch pieces at a time: their loads are one round trip
  for (int i0 = 0; i0 < cut.pieces; i0 += kBatch) {
    float2 v[kBatch];
    float4 o[kBatch][NC];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool in = i0 + b < cut.pieces;
      v[b] = in ? ml[base(i0 + b) * RT + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        o[b][c] = in ? acc[(base(i0 + b) * (D / 4) + warp + 8 * c) * RT + r] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = M;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) top = fmaxf(top, v[b].x);
    const float ref = top == -INFINITY ? 0.f : top;  // no key yet: every weight is 0
    const float old = exp2f(M - ref);
    M = top;
    l *= old;
#pragma unroll
    for (int c = 0; c < NC; ++c) a[c] = make_float4(a[c].x * old, a[c].y * old, a[c].z * old, a[c].w * old);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float w = exp2f(v[b].x - ref);
      l = fmaf(v[b].y, w, l);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        a[c].x = fmaf(o[b][c].x, w, a[c].x);
        a[c].y = fmaf(o[b][c].y, w, a[c].y);
        a[c].z = fmaf(o[b][c].z, w, a[c].z);
        a[c].w = fmaf(o[b][c].w, w, a[c].w);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const int f = cut.row0 + r;
  T* o = static_cast<T*>(p.out) +
         (static_cast<int64_t>(cut.q0 + f / p.G) * p.Hq + cut.kvh * p.G + f % p.G) * D;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    store4(o + (warp + 8 * c) * 4, make_float4(a[c].x * inv, a[c].y * inv, a[c].z * inv, a[c].w * inv));
}

template <typename T, int D, int MR>
cudaError_t run_generic(const AttnParams& p, cudaStream_t stream) {
  using C = GenCfg<D, MR>;
  static SmemGrant granted;
  const cudaError_t e = grant_smem(granted, attention_generic_kernel<T, D, MR>, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(attention_generic_kernel<T, D, MR>, dim3(static_cast<unsigned>(p.ctas)), kGenThreads, C::SMEM,
                stream, p);
}

template <typename T>
cudaError_t run_generic_t(const AttnParams& p, cudaStream_t stream) {
  if (p.RT == 16) return p.D == 64 ? run_generic<T, 64, 1>(p, stream) : run_generic<T, 128, 1>(p, stream);
  return p.D == 64 ? run_generic<T, 64, 4>(p, stream) : run_generic<T, 128, 4>(p, stream);
}

}  // namespace

cudaError_t launch_attention_plan(const AttnParams& p, cudaStream_t stream) {
  return launch_pdl(attention_plan_kernel, dim3(1), kPlanThreads, 0, stream, p);
}

cudaError_t launch_attention_generic(const AttnParams& p, pa_dtype dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? run_generic_t<__nv_bfloat16>(p, stream) : run_generic_t<float>(p, stream);
}

cudaError_t launch_attention_join(const AttnParams& p, pa_dtype dtype, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.ctas), static_cast<unsigned>((p.RT + 31) / 32));
  if (dtype == PA_BF16)
    return p.D == 64 ? launch_pdl(attention_join_kernel<__nv_bfloat16, 64>, grid, 256, 0, stream, p)
                     : launch_pdl(attention_join_kernel<__nv_bfloat16, 128>, grid, 256, 0, stream, p);
  return p.D == 64 ? launch_pdl(attention_join_kernel<float, 64>, grid, 256, 0, stream, p)
                   : launch_pdl(attention_join_kernel<float, 128>, grid, 256, 0, stream, p);
}

// By shared memory (228 KB per SM, 1 KB reserved per CTA), at most 4.
int attention_generic_ctas_per_sm(int RT, int D) {
  const int bytes = D == 64 ? (RT == 16 ? GenCfg<64, 1>::SMEM : GenCfg<64, 4>::SMEM)
                            : (RT == 16 ? GenCfg<128, 1>::SMEM : GenCfg<128, 4>::SMEM);
  const int n = 228 * 1024 / (bytes + 1024);
  return n < 4 ? n : 4;
}

}  // namespace pa
