// Attention of a few query tokens per sequence over the paged cache (sm_100a, bf16): at most 16
// rows, a row being a (query token, head of the group) pair; single tokens above all.  The formula
// and the masks are attention.cu's.
//
// Bound by reading K and V once, so it is scheduled as the balanced decode is: each (sequence, KV
// head) is a unit of the 16-key tiles that any of its rows sees (the interval of attention.h: a
// window's unit begins at the window); units lie end to end and every warp of one persistent wave
// takes an equal contiguous range, feeding itself with TMA loads through its own ring of stages.
// A tile is one m16n8k16 product chain over the rows (tc_tile.cuh), whose scores the Modified
// functor caps, biases and masks; P enters P.V as two bf16 parts, so it keeps ~16 bits.  Caps
// and biases cost about 20 instructions a tile and lane beside ~150, which the loads hide: 256
// tokens with 1000 cached, 32/8 heads of 128, take 171 us (6.15 TB/s) capped and plain; 8
// contexts of 32K to 128K with a bias 312 us (6.5 TB/s, the rate of a copy).  With heads of 64 a tile has
// half the bytes and nearly the same instructions outside its products: 135 us, 3.9 TB/s.
//
// Every CTA scans the units' tile counts itself (B loads), so there is no plan kernel: for a
// single request the launches are most of the time.  Units cut by a range boundary leave partials
// that tokens_join_kernel merges by log-sum-exp, in the order of the pieces.

#include "attention_ranges.cuh"
#include "tc_tile.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 2;  // per CTA; ring stages per warp
constexpr int kMinTiles = 2;

template <int D_, int BS_, bool ROWS16_>
struct TokensCfg : TileCfg<D_, BS_, ROWS16_, 16, true> {
  static constexpr int RING = kWarps * kStages * TokensCfg::STAGE_BYTES;
  static constexpr int Q_BYTES = WarpAcc<TokensCfg, true>::Q_BYTES;
  static constexpr int FIXED = RING + kWarps * 2 * Q_BYTES;
};

// The sequences' tiles before each one [B + 1] and first keys [B].
template <class C>
size_t tokens_smem(int B) {
  return C::FIXED + 1024 + (2 * static_cast<size_t>(B) + 1) * 4;
}

// Scores of one tile for this lane's two rows (tc_tile.cuh).
struct Modified : TileScores<2, false> {
  static constexpr bool kEmptyRows = true;
};

// KV head, first block of the stage and the ones to load of one tile, resolved by one lane.
struct TileIds {
  int kvh, row0;
  uint32_t live;
  int id[4];
};

template <class C>
__device__ __forceinline__ TileIds resolve(const AttnParams& p, const int* P, const int* LO, int g, int end) {
  TileIds r{0, 0, 0u, {0, 0, 0, 0}};
  if (g >= end) return r;
  const TilePos t = locate(P, p.B, p.Hkv, g);
  r.kvh = t.kvh;
  const int L = attn_len(p, t.b, false);
  const int lo = LO[t.b];
  const int tok0 = (lo / C::TILE_T + t.j) * C::TILE_T;
  const int blk = tok0 / C::BS;
  r.row0 = tok0 % C::BS;  // non-zero only where a stage holds part of a block
  const int32_t* tab = p.block_tables + static_cast<int64_t>(t.b) * p.max_blocks + blk;
#pragma unroll
  for (int k = 0; k < C::BPS; ++k)
    if ((blk + k) * C::BS < L && (blk + k + 1) * C::BS > lo) {  // a block with a key of the unit
      r.live |= 1u << k;
      r.id[k] = __ldg(tab + k);
    }
  return r;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 2)
    attention_tokens_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                            const AttnParams p) {
  constexpr int D = C::D, TILE_T = C::TILE_T;
  const int B = p.B, Hkv = p.Hkv, G = p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
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
  // the join may launch; it waits for this grid to complete.  Nothing before the wait reads
  // global memory.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
  scan_units<__nv_bfloat16, kThreads>(p, TILE_T, P, LO, warp_sum);

  const int T = Hkv * P[B];
  const int S = static_cast<int>(gridDim.x) * kWarps;
  // (no range below kMinTiles: where a single request leaves each warp less, a piece more costs
  // the join as much as the tiles)
  const int per = max((T + S - 1) / S, kMinTiles);
  const int s = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int beg = min(T, s * per), end = min(T, beg + per), cnt = end - beg;
  const uint64_t policy = l2_policy_evict_first();

  // Block ids of this warp's tiles, 32 at a time (lane j holds tile 32 * batch + j); the next
  // batch's table reads are issued one batch ahead.
  TileIds cur = resolve<C>(p, P, LO, beg + lane, end), nxt = resolve<C>(p, P, LO, beg + 32 + lane, end);
  int batch = 0;
  auto issue = [&](int k) {
    if ((k >> 5) != batch) {
      cur = nxt;
      ++batch;
      nxt = resolve<C>(p, P, LO, beg + 32 * (batch + 1) + lane, end);
    }
    const int src = k & 31;
    const int kv = __shfl_sync(kFull, cur.kvh, src), row0 = __shfl_sync(kFull, cur.row0, src);
    const uint32_t live = __shfl_sync(kFull, cur.live, src);
    int ids[C::BPS];
#pragma unroll
    for (int q = 0; q < C::BPS; ++q) ids[q] = __shfl_sync(kFull, cur.id[q], src);
    if (lane == 0) {
      const int stage = warp * kStages + k % kStages;
      const uint32_t fb = smem_addr(&full_bar[stage]);
      const uint32_t kt = smem_addr(smem + stage * C::STAGE_BYTES), vt = kt + C::TILE_BYTES;
      fence_proxy_async_smem();  // this stage's earlier generic reads and writes come first
      mbar_arrive_expect_tx(fb, static_cast<uint32_t>(__popc(live) * C::BOXR * D * 2 * 2));
#pragma unroll
      for (int sub = 0; sub < C::BPS; ++sub) {
        if (!(live >> sub & 1)) continue;
        int phys = ids[sub];
        if (phys < 0 || phys >= p.num_blocks) {
          flag_error(p.err, PA_DEVERR_BAD_BLOCK_ID);
          phys = 0;
        }
        if constexpr (C::BPS == 1) {
          tma_load_5d(kt, &tmk, 0, row0, 0, kv, phys, fb, policy);
          tma_load_5d(vt, &tmv, 0, row0, 0, kv, phys, fb, policy);
        } else {
#pragma unroll
          for (int c = 0; c < C::DCH; ++c) {
            tma_load_4d(kt + c * C::CHUNK_BYTES + sub * C::BOXR * 128, &tmk, c * 64, kv, row0, phys, fb, policy);
            tma_load_4d(vt + c * C::CHUNK_BYTES + sub * C::BOXR * 128, &tmv, c * 64, kv, row0, phys, fb, policy);
          }
        }
      }
    }
    __syncwarp();
  };
  for (int k = 0; k < kStages && k < cnt; ++k) issue(k);

  const int g = lane >> 2, tig = lane & 3;
  const int r0 = C::ROWS16 ? g : 2 * tig, r1 = C::ROWS16 ? g + 8 : 2 * tig + 1;  // score rows of this lane
  int4 own = make_int4(0, 0, 0, 0);  // the cut unit that begins here: pieces, first partial, KV head and rows, token
  int i = 0;  // tiles consumed (ring position)
  bool ok = true;
  using Acc = WarpAcc<C, true>;
  Acc acc;
  uint8_t* my_q = smem + C::RING + warp * 2 * C::Q_BYTES;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  // copy the rows of a unit into a Q tile (rows past them are zero); returns its first token
  auto prefetch_q = [&](const TilePos& u, uint8_t* tile) {
    int q0;
    const int rows = attn_query_span(p, u.b, false, q0) * G;
    constexpr int CPR = Acc::QROW_BYTES / 16;
    for (int e = lane; e < C::ROWS * CPR; e += 32) {
      const int r = e / CPR, c = e - r * CPR;
      const bool live = r < rows;
      const int t = live ? r / G : 0, h = live ? r - t * G : 0;
      cp_async_16_zfill(smem_addr(tile + Acc::q_off(r, c)),
                        q + static_cast<int64_t>(q0 + t) * p.q_stride + static_cast<int64_t>(u.kvh * G + h) * D + c * 8,
                        live ? 16 : 0);
    }
    cp_async_commit();
  };
  Modified score;
  score.init(p);

  int gpos = beg, qb = 0;
  TilePos t{};
  if (gpos < end) {
    t = locate(P, B, Hkv, gpos);
    prefetch_q(t, my_q);
  }
  while (gpos < end && ok) {
    const Seq sq = sequence(p, t.b, false);
    const int rows = sq.n * G;
    const int ubeg = Hkv * P[t.b] + t.kvh * t.nt, uend = ubeg + t.nt, pend = min(end, uend);
    score.set(p, 0, sq, t.b, t.kvh, min(r0, rows - 1));
    score.set(p, 1, sq, t.b, t.kvh, min(r1, rows - 1));
    // the next unit's Q rows are copied while this unit streams
    TilePos tn{};
    if (pend < end) tn = locate(P, B, Hkv, pend);
    acc.use_q(my_q + qb * C::Q_BYTES);
    if (pend < end) prefetch_q(tn, my_q + (qb ^ 1) * C::Q_BYTES);
    qb ^= 1;
    acc.reset();
    const int first = sq.lo / TILE_T;
    const int jend = t.j + (pend - gpos);
    for (int j = t.j; j < jend; ++j, ++i) {
      const int stage = warp * kStages + i % kStages;
      if (!mbar_wait_warp(smem_addr(&full_bar[stage]), (i / kStages) & 1, p.err)) {
        ok = false;  // the same in every lane
        break;
      }
      uint8_t* st = smem + stage * C::STAGE_BYTES;
      score.key0 = (first + j) * TILE_T;
      // V rows of keys that no row sees may hold anything (0 * Inf is NaN)
      const int a = sq.lo - score.key0, z = min(sq.hi - score.key0, TILE_T);
      if (a > 0) zero_rows<C>(st, 0, a, lane);
      if (z < TILE_T) zero_rows<C>(st, z, TILE_T, lane);
      acc.tile_scores(smem_addr(st), z, score, lane);
      __syncwarp();
      if (i + kStages < cnt) issue(i + kStages);  // refill the stage just consumed
    }
    if (!ok) break;
    acc.reduce_l();
    auto row_out = [&](int r) {
      const int tok = r / G;
      return out + (static_cast<int64_t>(sq.q0 + tok) * p.Hq + t.kvh * G + (r - tok * G)) * D;
    };
    if (gpos == ubeg && pend == uend) {
      if (p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[t.b * Hkv + t.kvh] = make_int4(0, 0, 0, 0);
      auto inverse = [](float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); };  // NaN stays
      if (g < rows) {
        const float inv = inverse(acc.l_lo);
        __nv_bfloat16* o = row_out(g);
#pragma unroll
        for (int jn = 0; jn < C::NT; ++jn)
          *reinterpret_cast<uint32_t*>(o + 8 * jn + 2 * tig) =
              pack_bf16x2(acc.o_lo[jn][0] * inv, acc.o_lo[jn][1] * inv);
      }
      if (C::ROWS16 && g + 8 < rows) {
        const float inv = inverse(acc.l_hi);
        __nv_bfloat16* o = row_out(g + 8);
#pragma unroll
        for (int jn = 0; jn < C::NT; ++jn)
          *reinterpret_cast<uint32_t*>(o + 8 * jn + 2 * tig) =
              pack_bf16x2(acc.o_hi[jn][0] * inv, acc.o_hi[jn][1] * inv);
      }
    } else {
      const int slot = gpos == beg ? 0 : 1;  // a cut piece is the range's first or last
      const int64_t row0 = (static_cast<int64_t>(s) * 2 + slot) * p.RT;
      if (tig == 0) {
        float2* ml = reinterpret_cast<float2*>(p.part_ml) + row0;
        if (g < rows) ml[g] = make_float2(acc.m_lo, acc.l_lo);
        if (C::ROWS16 && g + 8 < rows) ml[g + 8] = make_float2(acc.m_hi, acc.l_hi);
      }
#pragma unroll
      for (int jn = 0; jn < C::NT; ++jn) {
        float* o = p.part_acc + (row0 + g) * D + 8 * jn + 2 * tig;
        if (g < rows) *reinterpret_cast<float2*>(o) = make_float2(acc.o_lo[jn][0], acc.o_lo[jn][1]);
        if (C::ROWS16 && g + 8 < rows)
          *reinterpret_cast<float2*>(o + 8 * D) = make_float2(acc.o_hi[jn][0], acc.o_hi[jn][1]);
      }
      if (ubeg >= beg) {  // the unit begins here: its pieces are those of s .. (uend - 1) / per
        own = make_int4((uend - 1) / per - s + 1, 2 * s + slot, t.kvh << 8 | rows, sq.q0);
        if (p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[t.b * Hkv + t.kvh] = own;
      }
    }
    gpos = pend;
    t = tn;
  }
  cp_async_wait_all();
  if (!ok) {  // wait (bounded) for the loads still in flight
    for (int k = i; k < cnt && k < i + kStages; ++k)
      mbar_wait(smem_addr(&full_bar[warp * kStages + k % kStages]), (k / kStages) & 1, p.err);
  }
  if (!p.by_unit && lane == 0) reinterpret_cast<int4*>(p.cuts)[s] = own;
}

template <class C>
cudaError_t run(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap tmk, tmv;
  // a stage of one block (or of part of one): one box of all D columns; else one per block and
  // 64-column chunk
  const bool maps = C::BPS == 1 ? make_pool_map_rows(&tmk, p.k_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR) &&
                                      make_pool_map_rows(&tmv, p.v_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR)
                                : make_pool_map(&tmk, p.k_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR) &&
                                      make_pool_map(&tmv, p.v_pool, p.num_blocks, C::BS, p.Hkv, C::D, C::BOXR);
  if (!maps) return cudaErrorInvalidValue;
  const size_t smem = tokens_smem<C>(p.B);
  static SmemGrant granted;
  cudaError_t e = grant_smem(granted, attention_tokens_kernel<C>, static_cast<int>(smem));
  if (e == cudaSuccess)
    e = launch_pdl(attention_tokens_kernel<C>, dim3(static_cast<unsigned>(p.ctas / kWarps)), kThreads, smem, stream, tmk,
                   tmv, p);
  if (e != cudaSuccess) return e;
  return launch_tokens_join<__nv_bfloat16, C::D>(p, stream);
}

template <int D, int BS>
cudaError_t run_rows(const AttnParams& p, cudaStream_t stream) {
  return p.RT > 8 ? run<TokensCfg<D, BS, true>>(p, stream) : run<TokensCfg<D, BS, false>>(p, stream);
}

}  // namespace

// Whether a call is for this kernel: its rows fit a tile, and the scan of the batch fits
// shared memory with two CTAs per SM.
bool attention_tokens_eligible(int max_query_len, int G, int B) {
  return static_cast<int64_t>(max_query_len) * G <= 16 && B <= 2048;
}

int attention_tokens_ranges(int sms) { return sms * 2 * kWarps; }

cudaError_t launch_attention_tokens(const AttnParams& params, cudaStream_t stream) {
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
