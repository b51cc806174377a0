// Attention of a few query tokens per sequence over the paged cache in fp32 (sm_100a): at most 16
// rows, scheduled as attention_tokens.cu is.  The products run on the CUDA cores (no TF32).
//
// A warp takes a tile of 8 keys.  Lane l holds columns [l D/32, (l + 1) D/32) of every row of q and
// of the outputs, so that K and V rows are read from shared memory once, whole and without
// conflicts, for all rows.  The lanes' partial scores, 8 R of them, are summed by a butterfly
// that halves the values at every step (31 shuffles for 32 sums where 32 reductions would take
// 160) and leaves lane l with the score of row l / 8 (+ 4, + 8, ..), key l % 8; weights go back by
// shuffles.  With R = 4 that is about 60 instructions a key and warp for its 1024 bytes (D = 128).
// 256 tokens with 1000 cached, 8 KV heads of 128: 6.0 TB/s with up to 4 rows, 5.1 with 8, 2.6 with 16,
// where the rows' own products and shuffles take longer than the memory; with heads of 64, where the
// butterfly is the same for half the bytes, 3.9 TB/s with up to 4 rows, 3.1 and 1.9.  With cap and
// window, lengths from 63 to 4095, heads of 128 and 4 rows: 220 us, 5.4 TB/s.

#include "attention_ranges.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 2, kTile = 8, kMinTiles = 4;

template <int D_, int BS_, int R_>
struct Tokens32 {
  static constexpr int D = D_, BS = BS_, R = R_;
  static constexpr int VEC = D / 32;                      // columns of a lane
  static constexpr int NV = R / 4;                        // scores of a lane per tile
  static constexpr int BOXR = BS < kTile ? BS : kTile;    // rows of a TMA box
  static constexpr int BPS = kTile / BOXR;                // boxes of a stage
  static constexpr int PART = kTile * D * 4, STAGE = 2 * PART;
  static constexpr int FIXED = kWarps * kStages * STAGE;
};

template <int N>
struct Cols {
  float v[N];
};

__device__ __forceinline__ Cols<4> load_cols(const float* p, Cols<4>) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  return Cols<4>{{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ Cols<2> load_cols(const float* p, Cols<2>) {
  const float2 x = *reinterpret_cast<const float2*>(p);
  return Cols<2>{{x.x, x.y}};
}
__device__ __forceinline__ void store_cols(float* p, const Cols<4>& c, float k) {
  *reinterpret_cast<float4*>(p) = make_float4(c.v[0] * k, c.v[1] * k, c.v[2] * k, c.v[3] * k);
}
__device__ __forceinline__ void store_cols(float* p, const Cols<2>& c, float k) {
  *reinterpret_cast<float2*>(p) = make_float2(c.v[0] * k, c.v[1] * k);
}

// Sum each of 32 values over the lanes; lane l gets the sum of value l.
__device__ __forceinline__ float transpose_sum(float (&a)[32], int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float send = up ? a[i] : a[i + off];
      const float keep = up ? a[i + off] : a[i];
      a[i] = keep + __shfl_xor_sync(kFull, send, off);
    }
  }
  return a[0];
}

template <class C>
__global__ void __launch_bounds__(kThreads, 2)
    attention_tokens32_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                              const AttnParams p) {
  constexpr int D = C::D, R = C::R, NV = C::NV, VEC = C::VEC;
  const int B = p.B, Hkv = p.Hkv, G = p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  int* P = reinterpret_cast<int*>(smem + C::FIXED);  // [B + 1] tiles before sequence b
  int* LO = P + B + 1;                               // [B]
  __shared__ __align__(8) uint64_t full_bar[kWarps * kStages];
  __shared__ int warp_sum[kWarps];

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_addr(&full_bar[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  scan_units<float, kThreads>(p, kTile, P, LO, warp_sum);

  const int T = Hkv * P[B];
  const int S = static_cast<int>(gridDim.x) * kWarps;
  const int per = max((T + S - 1) / S, kMinTiles);
  const int s = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int beg = min(T, s * per), end = min(T, beg + per), cnt = end - beg;
  const uint64_t policy = l2_policy_evict_first();

  // A tile's boxes, resolved by one lane: KV head, row within the block, ids (-1: not loaded).
  struct Boxes {
    int kvh, row0, id[C::BPS];
  };
  auto resolve = [&](int g) {
    Boxes r{0, 0, {}};
#pragma unroll
    for (int k = 0; k < C::BPS; ++k) r.id[k] = INT_MIN;
    if (g >= end) return r;
    const TilePos t = locate(P, B, Hkv, g);
    r.kvh = t.kvh;
    const int L = attn_len(p, t.b, false), lo = LO[t.b];
    const int tok0 = (lo / kTile + t.j) * kTile, blk = tok0 / C::BS;
    r.row0 = tok0 % C::BS;
    const int32_t* tab = p.block_tables + static_cast<int64_t>(t.b) * p.max_blocks + blk;
#pragma unroll
    for (int k = 0; k < C::BPS; ++k)
      if ((blk + k) * C::BS < L && (blk + k + 1) * C::BS > lo) r.id[k] = max(__ldg(tab + k), -1);
    return r;
  };
  Boxes cur = resolve(beg + lane), nxt = resolve(beg + 32 + lane);
  int batch = 0;
  auto issue = [&](int k) {
    if ((k >> 5) != batch) {
      cur = nxt;
      ++batch;
      nxt = resolve(beg + 32 * (batch + 1) + lane);
    }
    const int src = k & 31;
    const int kv = __shfl_sync(kFull, cur.kvh, src), row0 = __shfl_sync(kFull, cur.row0, src);
    int ids[C::BPS], live = 0;
#pragma unroll
    for (int q = 0; q < C::BPS; ++q) {
      ids[q] = __shfl_sync(kFull, cur.id[q], src);
      live += ids[q] != INT_MIN;
    }
    if (lane == 0) {
      const int stage = warp * kStages + k % kStages;
      const uint32_t fb = smem_addr(&full_bar[stage]);
      const uint32_t kt = smem_addr(smem + stage * C::STAGE), vt = kt + C::PART;
      fence_proxy_async_smem();  // this stage's earlier generic reads and writes come first
      mbar_arrive_expect_tx(fb, static_cast<uint32_t>(live * C::BOXR * D * 4 * 2));
#pragma unroll
      for (int q = 0; q < C::BPS; ++q) {
        if (ids[q] == INT_MIN) continue;
        int phys = ids[q];
        if (phys < 0 || phys >= p.num_blocks) {
          flag_error(p.err, PA_DEVERR_BAD_BLOCK_ID);
          phys = 0;
        }
        tma_load_4d(kt + q * C::BOXR * D * 4, &tmk, 0, kv, row0, phys, fb, policy);
        tma_load_4d(vt + q * C::BOXR * D * 4, &tmv, 0, kv, row0, phys, fb, policy);
      }
    }
    __syncwarp();
  };
  for (int k = 0; k < kStages && k < cnt; ++k) issue(k);

  float* out = static_cast<float*>(p.out);
  const float* qp = static_cast<const float*>(p.q);
  TileScores<NV, true> score;
  score.init(p);
  int4 own = make_int4(0, 0, 0, 0);  // as in attention_tokens.cu
  int i = 0, gpos = beg;
  bool ok = true;
  while (gpos < end && ok) {
    const TilePos t = locate(P, B, Hkv, gpos);
    const Seq sq = sequence(p, t.b, false);
    const int rows = sq.n * G;
    const int ubeg = Hkv * P[t.b] + t.kvh * t.nt, uend = ubeg + t.nt, pend = min(end, uend);
    Cols<VEC> q[R], o[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tok = r / G;
      q[r] = o[r] = Cols<VEC>{};
      if (r < rows)
        q[r] = load_cols(qp + static_cast<int64_t>(sq.q0 + tok) * p.q_stride +
                             static_cast<int64_t>(t.kvh * G + (r - tok * G)) * D + lane * VEC, Cols<VEC>{});
    }
    float m[NV], l[NV];  // of this lane's rows: lane / 8 + 4 v
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      score.set(p, v, sq, t.b, t.kvh, min((lane >> 3) + 4 * v, rows - 1));
      m[v] = -INFINITY;
      l[v] = 0.f;
    }
    const int first = sq.lo / kTile, jend = t.j + (pend - gpos);
    for (int j = t.j; j < jend; ++j, ++i) {
      const int stage = warp * kStages + i % kStages;
      if (!mbar_wait_warp(smem_addr(&full_bar[stage]), (i / kStages) & 1, p.err)) {
        ok = false;  // the same in every lane
        break;
      }
      float* K = reinterpret_cast<float*>(smem + stage * C::STAGE);
      float* V = K + kTile * D;
      score.key0 = (first + j) * kTile;
      // keys that no row sees may hold anything (0 * Inf is NaN): they are not read
      const int a = max(sq.lo - score.key0, 0), z = min(sq.hi - score.key0, kTile);
      float x[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float part[32];  // rows 4v .. 4v + 3, 8 keys each
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
          Cols<VEC> c{};
          if (k >= a && k < z) c = load_cols(K + k * D + lane * VEC, Cols<VEC>{});
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) d = fmaf(q[4 * v + r].v[e], c.v[e], d);
            part[r * 8 + k] = d;
          }
        }
        x[v] = score(transpose_sum(part, lane), lane & 7, v);
      }
      float alpha[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float mx = x[v];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
        const float mn = fmaxf(m[v], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // no key yet: every weight is 0
        alpha[v] = exp2f(m[v] - ref);
        m[v] = mn;
        x[v] = exp2f(x[v] - ref);
        l[v] = l[v] * alpha[v] + x[v];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float al = __shfl_sync(kFull, alpha[r / 4], r % 4 * 8);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[r].v[e] *= al;
      }
#pragma unroll
      for (int k = 0; k < kTile; ++k) {
        Cols<VEC> c{};
        if (k >= a && k < z) c = load_cols(V + k * D + lane * VEC, Cols<VEC>{});
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float w = __shfl_sync(kFull, x[r / 4], r % 4 * 8 + k);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[r].v[e] = fmaf(w, c.v[e], o[r].v[e]);
        }
      }
      __syncwarp();
      if (i + kStages < cnt) issue(i + kStages);  // refill the stage just consumed
    }
    if (!ok) break;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) l[v] += __shfl_xor_sync(kFull, l[v], off);
    const bool whole = gpos == ubeg && pend == uend;
    const int slot = gpos == beg ? 0 : 1;  // a cut piece is the range's first or last
    const int64_t row0 = (static_cast<int64_t>(s) * 2 + slot) * p.RT;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float lr = __shfl_sync(kFull, l[r / 4], r % 4 * 8), mr = __shfl_sync(kFull, m[r / 4], r % 4 * 8);
      if (r >= rows) continue;
      if (whole) {
        const int tok = r / G;
        store_cols(out + (static_cast<int64_t>(sq.q0 + tok) * p.Hq + t.kvh * G + (r - tok * G)) * D + lane * VEC, o[r],
                   lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr));  // NaN stays
      } else {
        if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[row0 + r] = make_float2(mr, lr);
        store_cols(p.part_acc + (row0 + r) * D + lane * VEC, o[r], 1.f);
      }
    }
    if (whole) {
      if (p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[t.b * Hkv + t.kvh] = make_int4(0, 0, 0, 0);
    } else if (ubeg >= beg) {
      own = make_int4((uend - 1) / per - s + 1, 2 * s + slot, t.kvh << 8 | rows, sq.q0);
      if (p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[t.b * Hkv + t.kvh] = own;
    }
    gpos = pend;
  }
  if (!ok) {  // wait (bounded) for the loads still in flight
    for (int k = i; k < cnt && k < i + kStages; ++k)
      mbar_wait(smem_addr(&full_bar[warp * kStages + k % kStages]), (k / kStages) & 1, p.err);
  }
  if (!p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[s] = own;
}

template <class C>
cudaError_t run(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap tmk, tmv;
  if (!make_pool_map_f32(&tmk, p.k_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR) ||
      !make_pool_map_f32(&tmv, p.v_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR))
    return cudaErrorInvalidValue;
  const size_t smem = C::FIXED + 128 + (2 * static_cast<size_t>(p.B) + 1) * 4;
  static SmemGrant granted;
  cudaError_t e = grant_smem(granted, attention_tokens32_kernel<C>, static_cast<int>(smem));
  if (e == cudaSuccess)
    e = launch_pdl(attention_tokens32_kernel<C>, dim3(static_cast<unsigned>(p.ctas / kWarps)), kThreads, smem, stream,
                   tmk, tmv, p);
  if (e != cudaSuccess) return e;
  return launch_tokens_join<float, C::D>(p, stream);
}

template <int D, int BS>
cudaError_t run_rows(const AttnParams& p, cudaStream_t stream) {
  if (p.RT <= 4) return run<Tokens32<D, BS, 4>>(p, stream);
  return p.RT <= 8 ? run<Tokens32<D, BS, 8>>(p, stream) : run<Tokens32<D, BS, 16>>(p, stream);
}

}  // namespace

cudaError_t launch_attention_tokens32(const AttnParams& params, cudaStream_t stream) {
  AttnParams p = params;
  p.by_unit = static_cast<int64_t>(p.B) * p.Hkv < p.ctas;
  switch (p.D * 100 + p.block_size) {
    case 6404: return run_rows<64, 4>(p, stream);
    case 6408: return run_rows<64, 8>(p, stream);
    case 6416: return run_rows<64, 16>(p, stream);
    case 6432: return run_rows<64, 32>(p, stream);
    case 12804: return run_rows<128, 4>(p, stream);
    case 12808: return run_rows<128, 8>(p, stream);
    case 12816: return run_rows<128, 16>(p, stream);
    case 12832: return run_rows<128, 32>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
