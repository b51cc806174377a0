// Attention of ragged query tokens over the paged cache on the 5th-generation tensor cores
// (sm_100a, bf16).  The formula, the masks and the work plan are attention.cu's; a CTA of one
// wave walks its range of (item, KV head, tile of 128 keys), or takes unit after unit.
//
// An item is two M tiles of whole tokens, HR = floor(128 / G) * G rows each.  Softmax group g
// serves M tile g; both read the same K and V tiles, so a tile of 128 keys is loaded once for up to
// 256 rows.  Group g skips the tiles that none of its rows sees.
//
// Warps: 0-7 softmax (group g = warps 4g .. 4g + 3, a thread per row), 8 and 11 the products of
// group 0 and 1, 9 K/V loads, 10 schedule and Q loads.  The schedule warp writes records of the
// CTA's pieces (a piece is the part of a unit in the range) into a small ring that all others
// follow.  K and V tiles share a ring of slots in load order (K0 V0 K1 V1 ..), one TMA box per
// block and 64-column chunk.
//
// Tensor memory: S_g at column 128 g in two halves of 64 keys, each overwritten by its P (bf16
// pairs, 32 columns); O_g at column 256 + 128 g.  Products are issued by one thread and run in
// order, so the next tile's half of S_g is issued right behind the P.V that reads the same half of
// P_g, and is computed while the softmax works on the other half (S of whole tiles, behind both
// halves of P.V: 327 us for 305).  While group 0 works on its S, the products of group 1 run and the
// other way round.
//
// Bound by latencies: the exponentials take as long as the products (2048 cycles for a pair of M tiles
// and 128 keys, at 16 a cycle and SM), but no pipe is busy half of the time (8 x 2048 plain: tensor 46 %,
// exponentials 48, issue 42; capped: 39, 40, 48, and FMA 38).  With two softmax warps a scheduler each
// group's chain S, weights, P.V, S is not hidden by the other group's.  A prompt of 8192 tokens, 32/8
// heads of 128, with a prefix mask: 615 us, 1127 TFLOP/s; 8 of 2048, causal: 305 us, 902; with capped
// scores 370 us, 744 (caps past 50, whose maximum is found: 620 us; past 64: 815 us); with a bias 450 us.
// (Sustained, at the 1000 W limit, the prompt takes 710 us at 1.65 GHz.)
//
// P is rounded to bf16 (half a step, 2^-8 of each weight, as the output is); row sums, maxima and
// O stay in 32 bits.  The reference maximum moves lazily, by more than 2^8 only; capped scores have
// a fixed one (api_ops.cu), which saves the search for a maximum (8 x 2048: 514 us for 413).
//
// Every wait is bounded in time; on expiry the kernel records PA_DEVERR_TIMEOUT, every role
// stops, loads and products in flight are drained (bounded) and the tensor memory is freed.

#include "attention.h"
#include "tc05.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kKT = 128;        // keys per tile
constexpr int kHalf = kKT / 2;  // and per S, P and their barriers
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kPlanWarp = 10;  // and 11: the other group's products
// Registers of a softmax thread and of another one: together what 384 threads are launched with.
constexpr int kSoftRegs = 208, kOtherRegs = 88;
constexpr int kPieces = 4;      // records in flight
constexpr int kMaxSlots = 10;
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kColS = 0, kColO = 256, kGroupCols = 128, kTmemCols = 512;
// released by the two MMA warps, the K/V load warp and each softmax warp
constexpr int kPieceUsers = 3 + kSoftWarps;

// CAP, BIAS: what is done to the scores, fixed at compile time so that the loop of a call is short
// straight code (instruction fetches bound the kernel that decided at run time).  WIDE: the cap is one
// past kWideCap (with CAP and BIAS).
template <int D_, bool CAP_, bool BIAS_, bool WIDE_ = false>
struct TcAttn {
  static constexpr int D = D_;
  static constexpr bool CAP = CAP_, BIAS = BIAS_, WIDE = WIDE_;
  static constexpr int MT = 2;                        // M tiles of an item
  static constexpr int DCH = D / 64;
  static constexpr int CHUNK = kKT * 128;             // one 64-column chunk of 128 rows
  static constexpr int SLOT = DCH * CHUNK;            // a K or V tile; an M tile of Q
  static constexpr int BUDGET = 227 * 1024 - 1024 - 1536;  // alignment, static shared memory
  static constexpr int FIT = (BUDGET - MT * SLOT) / SLOT;
  static constexpr int NST = FIT < kMaxSlots ? FIT : kMaxSlots;
  static constexpr int SMEM = 1024 + MT * SLOT + NST * SLOT;
  static_assert(NST >= 5, "K and V of two tiles and one more");
  static_assert(SMEM > 114 * 1024, "one CTA per SM: it holds all of the SM's tensor memory");
};

// A piece: tiles [0, cnt) of it are tiles kt0 .. of the sequence's keys.
struct Piece {
  int cnt;             // 0: no more pieces
  int kt0;
  int kvh;
  int b, q0, row0, rows, pos0, L, lo, hi;
  int ga[2], gb[2];    // group g's tiles
  int whole, slot;     // the whole unit; else the slot of its partial
};

struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t qfull, qempty;
  uint64_t sfull[2][2], pfull[2][2], ofull[2];  // per group; S and P in two halves
  uint64_t half_done[2];  // a group's product with the first half of a tile's P
  uint64_t pc_full[kPieces], pc_empty[kPieces];
  uint64_t drain_bar[2];
  uint64_t turn[2][4];  // warp w of group g has done its exponentials of a tile
  Piece pc[kPieces];
  uint32_t tmem;
  volatile int abort_flag;
};

// What most tiles do not take is kept out of the way of the instructions that they do.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// What a row of a piece sees and how its scores are biased.
struct Row {
  int lo, hi;      // visible keys
  int pos;
  float slope;     // times log2 e
};

// What a row reads from global memory, loaded while the piece before ends.
struct RowLoads {
  int prefix, first;
  float slope;
};

__device__ __forceinline__ RowLoads load_row(const AttnParams& p, const Piece& pc, int f) {
  const int t = f / p.G;
  RowLoads r;
  r.prefix = p.prefix_lens ? __ldg(p.prefix_lens + pc.b) : 0;
  r.first = p.first_keys ? __ldg(p.first_keys + pc.q0 + t) : 0;
  r.slope = p.slopes ? __ldg(p.slopes + pc.kvh * p.G + (f - t * p.G)) : 0.f;
  return r;
}

__device__ __forceinline__ Row row_of(const AttnParams& p, const Piece& pc, int f, const RowLoads& in) {
  Row r;
  r.pos = pc.pos0 + f / p.G;
  attn_visible(p, r.pos, pc.L, in.prefix, in.first, r.lo, r.hi);
  r.slope = in.slope * kLog2e;
  return r;
}

// One operation per element costs a warp 128 cycles a tile, two warps share a sub-partition and the
// products of a pair of tiles take 2048: operations are counted here.  So are instructions: once
// the loop of all roles is larger than the 32 KB that instructions are kept in, each takes three
// times as long.  Two-element forms take as long as two scalar ones, but half the instructions.

// Whether the polynomial below holds for raw scores of up to `top` in any lane of the warp.
__device__ __forceinline__ bool cap_is_small(const AttnParams& p, float top) {
  return __all_sync(kFull, top * p.cap_small <= 0.85f);  // (NaN: no)
}

// cap * tanh(scale * x / cap) log2(e) + add of N raw scores, in place: tanh(t) / t as a polynomial in
// t^2 (iterated reweighted least squares on |t| <= 0.85, where |t P(t^2) - tanh t| < 6.9e-7 in 32
// bits): on the FMA pipe alone, the exponentials need the other.  Scale and cap are in the
// coefficients.
template <int N>
__device__ __forceinline__ void cap_polynomial(float (&x)[N], const AttnParams& p, float add) {
  constexpr int E = 8;  // elements taken step by step, so that the steps of one do not wait
  const float2 c4 = splat(p.cap_poly[4]), c3 = splat(p.cap_poly[3]), c2 = splat(p.cap_poly[2]),
               c1 = splat(p.cap_poly[1]), c0 = splat(p.cap_poly[0]), last = splat(add);
#pragma unroll
  for (int j = 0; j < N; j += E) {
    float2 t[E / 2], u[E / 2], y[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) t[e] = make_float2(x[j + 2 * e], x[j + 2 * e + 1]);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) u[e] = __fmul2_rn(t[e], t[e]);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) y[e] = __ffma2_rn(u[e], c4, c3);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) y[e] = __ffma2_rn(y[e], u[e], c2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) y[e] = __ffma2_rn(y[e], u[e], c1);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) y[e] = __ffma2_rn(y[e], u[e], c0);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      y[e] = __ffma2_rn(y[e], t[e], last);
      x[j + 2 * e] = y[e].x;
      x[j + 2 * e + 1] = y[e].y;
    }
  }
}

// The same by the formula that `small` allows.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], const AttnParams& p, bool small, float add) {
  constexpr int E = 8;
  if (__builtin_expect(small, 1)) {
    cap_polynomial(x, p, add);
  } else {
    // tanh t = 1 - 2 / (1 + e^2t)
    const float c2 = p.cap_in * (2.f * kLog2e), m2 = -2.f * p.cap_out, last = p.cap_out + add;
#pragma unroll
    for (int j = 0; j < N; j += E) {
      float u[E];
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = ex2_approx(x[j + e] * c2);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = rcp_approx(1.f + u[e]);
#pragma unroll
      for (int e = 0; e < E; ++e) x[j + e] = fmaf(m2, u[e], last);
    }
  }
}

// Largest and smallest of a row's scores; NaN are passed over.
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < N; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(x[j + 2 * e], x[j + 2 * e + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <int N>
__device__ __forceinline__ float smallest(const float (&x)[N]) {
  float m[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
  for (int j = 0; j < N; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fminf(m[e], fminf(x[j + 2 * e], x[j + 2 * e + 1]));
  return fminf(fminf(m[0], m[1]), fminf(m[2], m[3]));
}

template <int N>
__device__ __forceinline__ float largest_magnitude(const float (&x)[N]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < N; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(fabsf(x[j + 2 * e]), fabsf(x[j + 2 * e + 1])));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Elements of columns outside [a, b) become `v`.
template <int N>
__device__ __forceinline__ void mask_scores(float (&x)[N], int a, int b, float v) {
#pragma unroll
  for (int j = 0; j < N; ++j) x[j] = j >= a && j < b ? x[j] : v;
}

// Turn the N raw scores of a row (keys key0 ..) into log2-domain scores in place and return their
// maximum.  The plain case keeps raw scores, so that the scale and the subtraction of the maximum
// become one operation.  `ahead`: some of the keys may lie behind the row's position and count.
template <bool CAP, bool BIAS, bool WIDE, int N>
__device__ __forceinline__ float modify_scores(float (&x)[N], const AttnParams& p, const Row& r, int key0,
                                               bool masked, bool ahead) {
  constexpr int E = 8;
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < N; ++j) {  // (both, and a choice: branches in this loop take 1138 us for 8 x 2048, not 813)
      const float t = x[j] * p.cap_in, near = cap_score_near(x[j], t, p.scale_log2), far = cap_score(t, p.cap_out);
      x[j] = fabsf(t) < kNearTanh ? near : far;
    }
  } else if constexpr (CAP) {
    if (rare(masked)) mask_scores(x, r.lo - key0, r.hi - key0, 0.f);  // what lies there must not choose the formula
    cap_scores(x, p, cap_is_small(p, fmaxf(largest(x), -smallest(x))), 0.f);
  }
  if constexpr (BIAS) {
    const float d0 = static_cast<float>(r.pos - key0);
    if (rare(ahead)) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float y = CAP ? x[j] : x[j] * p.scale_log2;
        x[j] = fmaf(-r.slope, fabsf(d0 - static_cast<float>(j)), y);
      }
    } else {  // |pos - key| = d0 - j
      const float c0 = -r.slope * d0;
#pragma unroll
      for (int j = 0; j < N; j += E) {
        float d[E];
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = fmaf(r.slope, static_cast<float>(j + e), c0);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = make_float2(x[j + e], x[j + e + 1]), w = make_float2(d[e], d[e + 1]);
          const float2 y = CAP ? __fadd2_rn(v, w) : __ffma2_rn(v, splat(p.scale_log2), w);
          x[j + e] = y.x;
          x[j + e + 1] = y.y;
        }
      }
    }
  }
  if (rare(masked)) mask_scores(x, r.lo - key0, r.hi - key0, -INFINITY);
  return largest(x);
}

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const __grid_constant__ CUtensorMap tmq, const AttnParams p) {
  constexpr int D = C::D, DCH = C::DCH, NST = C::NST;
  const int BS = p.block_size;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + C::MT * C::SLOT;
  __shared__ __align__(16) Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x;
  const int HR = p.HR;  // rows of an M tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 2);  // both groups' products have read it
    }
    mbar_init(smem_addr(&sh.qfull), 1);
    mbar_init(smem_addr(&sh.qempty), 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.sfull[i][0]), 1);
      mbar_init(smem_addr(&sh.sfull[i][1]), 1);
      mbar_init(smem_addr(&sh.half_done[i]), 1);
      mbar_init(smem_addr(&sh.pfull[i][0]), 128);
      mbar_init(smem_addr(&sh.pfull[i][1]), 128);
      mbar_init(smem_addr(&sh.ofull[i]), 1);
      mbar_init(smem_addr(&sh.drain_bar[i]), 1);
      for (int w = 0; w < 4; ++w) mbar_init(smem_addr(&sh.turn[i][w]), 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(smem_addr(&sh.pc_full[i]), 1);
      mbar_init(smem_addr(&sh.pc_empty[i]), kPieceUsers);
    }
    sh.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) tc05::alloc(smem_addr(&sh.tmem), kTmemCols);
  // rows of the Q tiles that no load covers: finite scores for them (their P is never used)
  for (int e = threadIdx.x; e < C::MT * DCH * 128 * 8; e += kThreads) {
    const int row = (e >> 3) & 127;
    if (row >= HR) *reinterpret_cast<uint4*>(smem + e * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (threadIdx.x == kLoadWarp * 32) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    prefetch_tensormap(&tmq);
  }
  // the join may launch; it waits for this grid to complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = __reduce_max_sync(kFull, sh.tmem);
  volatile int* abort_flag = &sh.abort_flag;
  // nothing above reads global memory; the plan is written by the kernel before
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto piece_wait = [&](int n) {  // record n is there; false: give up
    return wait_warp(smem_addr(&sh.pc_full[n % kPieces]), (n / kPieces) & 1, p.err, abort_flag);
  };
  auto piece_done = [&](int n) {  // this warp will not read record n again
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.pc_empty[n % kPieces]));
  };

  static_assert(256 * kSoftRegs + 128 * kOtherRegs <= kThreads * 168, "the launch's registers");
  if (warp >= kSoftWarps) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kPlanWarp) {
      // ============================ schedule, Q tiles ============================
      if (lane == 0) {
        const uint64_t policy = l2_policy_evict_normal();
        const int ht = HR / p.G;  // tokens of an M tile
        const uint32_t box = static_cast<uint32_t>(HR) * 128;
        bool ok = true;
        const int64_t per =
            (static_cast<int64_t>(p.header[1]) * p.Hkv + p.ctas - 1) / p.ctas;
        const AttnStart st = p.starts[s];
        int left = st.count, item = st.item, kvh = st.kvh, at = st.tile, n = 0;
        int loaded = 0;  // Q loads issued
        // many units: each CTA takes the next one when it has room for it, else its own range (attention.cu)
        const bool dynamic = p.header[2] != 0;
        const int units = p.header[0] * p.Hkv;
        AttnCut cut{};
        AttnItem it{};
        int sum = 0, slots = 0;
        auto load_item = [&] {  // the item at or after `item` that has tiles
          sum = p.tile_sum[item];
          while ((slots = p.tile_sum[item + 1] - sum) == 0) ++item;
          it = p.items[item];
        };
        if (!dynamic && left > 0) load_item();
        for (;; ++n) {
          const int slot = n % kPieces;
          if (n >= kPieces &&
              !(ok = wait_or_abort(smem_addr(&sh.pc_empty[slot]), (n / kPieces - 1) & 1, p.err, abort_flag)))
            break;
          UnitPart u{0, 0, 0, 0};
          if (dynamic) {
            left = -1;
            for (int next; left < 0 && (next = atomicAdd(p.header + 3, 1)) < units;) {
              item = units / p.Hkv - 1 - next / p.Hkv;  // the last items of a sequence see the most
              kvh = next % p.Hkv;
              slots = p.tile_sum[item + 1] - p.tile_sum[item];
              if (slots == 0) continue;
              it = p.items[item];
              u = unit_part(p, slots, 0, slots);
              left = 1;
            }
          } else {
            if (left > 0) u = unit_part(p, slots, at, left);
            left -= u.slots;
            if (u.cnt == 0) left = -1;  // (the range ends before the unit's first tile)
          }
          at = 0;
          Piece* pc = &sh.pc[slot];
          if (left < 0) {
            pc->cnt = 0;
            mbar_arrive(smem_addr(&sh.pc_full[slot]));
            break;
          }
          const int cnt = u.cnt;
          const int first = it.lo / kKT + u.tile;
          pc->cnt = cnt;
          pc->kt0 = first;
          pc->kvh = kvh;
          pc->b = it.b;
          pc->q0 = it.q0;
          pc->row0 = it.row0;
          pc->rows = it.rows;
          pc->pos0 = it.pos0;
          pc->L = it.L;
          pc->lo = it.lo;
          pc->hi = it.hi;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int a = it.glo[g] / kKT - first, z = (it.ghi[g] + kKT - 1) / kKT - first;
            pc->ga[g] = it.ghi[g] > 0 ? max(a, 0) : 0;
            pc->gb[g] = it.ghi[g] > 0 ? min(z, cnt) : 0;
          }
          pc->whole = cnt == u.nt;
          pc->slot = n == 0 ? 0 : 1;
          mbar_arrive(smem_addr(&sh.pc_full[slot]));
          if (u.tile == 0 && cnt != u.nt) {  // the unit begins here and goes on in the next CTAs
            const int64_t ubeg = static_cast<int64_t>(sum) * p.Hkv + static_cast<int64_t>(kvh) * slots;
            cut = AttnCut{static_cast<int>((ubeg + slots - 1) / per) - s + 1, n == 0 ? 0 : 1, kvh, it.q0, it.row0,
                          it.rows, 0, 0};
          }
          // its Q, once the products of the piece before have read theirs
          if (n > 0 && !(ok = wait_or_abort(smem_addr(&sh.qempty), (n - 1) & 1, p.err, abort_flag))) break;
          const uint32_t bar = smem_addr(&sh.qfull), q = smem_addr(smem);
          const int tiles = it.rows > HR ? 2 : 1, tok = it.q0 + it.row0 / p.G;
          mbar_arrive_expect_tx(bar, box * DCH * tiles);
          for (int m = 0; m < tiles; ++m)
#pragma unroll
            for (int c = 0; c < DCH; ++c)
              tma_load_3d(q + m * C::SLOT + c * C::CHUNK, &tmq, c * 64, kvh * p.G, tok + m * ht, bar, policy);
          ++loaded;
          if (!dynamic && ++kvh == p.Hkv) {
            kvh = 0;
            ++item;
            if (left > 0) load_item();
          }
        }
        reinterpret_cast<AttnCut*>(p.cuts)[s] = cut;
        if (!ok && loaded > 0) mbar_wait(smem_addr(&sh.qfull), (loaded - 1) & 1, nullptr);
      }
    } else if (warp == kLoadWarp) {
      // ============================ K and V tiles ============================
      const int BPT = kKT / BS;  // blocks per tile, at most 32: a lane each
      const uint64_t policy = l2_policy_evict_normal();
      bool ok = true;
      int slot = 0;
      uint32_t phase = 0, used = 0;  // of the next load; slots in use (bits) once round
      auto next_slot = [&] {
        used |= 1u << slot;
        if (++slot == NST) {
          slot = 0;
          phase ^= 1;
        }
      };
      for (int i = 0; ok; ++i) {
        if (!(ok = piece_wait(i))) break;
        const Piece& pc = sh.pc[i % kPieces];
        const int cnt = pc.cnt;
        if (cnt == 0) break;
        const int kt0 = pc.kt0, lo = pc.lo, hi = pc.hi, kvh = pc.kvh;
        const int32_t* tab = p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks;
        piece_done(i);
        // this lane's block of a tile; ids are read one tile ahead
        auto live_at = [&](int j) {
          const int k = (kt0 + j) * kKT + lane * BS;
          return lane < BPT && j < cnt && k < hi && k + BS > lo;
        };
        auto id_at = [&](int j) { return live_at(j) ? __ldg(tab + (kt0 + j) * BPT + lane) : 0; };
        int next = id_at(0);
        for (int j = 0; j < cnt && ok; ++j) {
          int phys = next;
          const bool live = live_at(j);
          next = id_at(j + 1);
          if (phys < 0 || phys >= p.num_blocks) {
            flag_error(p.err, PA_DEVERR_BAD_BLOCK_ID);
            phys = 0;
          }
          const uint32_t bytes = __popc(__ballot_sync(kFull, live)) * BS * D * 2;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if ((used >> slot & 1) &&
                !(ok = wait_warp(smem_addr(&sh.empty[slot]), phase ^ 1, p.err, abort_flag)))
              break;
            const uint32_t bar = smem_addr(&sh.full[slot]);
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (live) {
              const uint32_t dst = smem_addr(ring + slot * C::SLOT) + lane * BS * 128;
#pragma unroll
              for (int c = 0; c < DCH; ++c)
                tma_load_4d(dst + c * C::CHUNK, kv ? &tmv : &tmk, c * 64, kvh, 0, phys, bar, policy);
            }
            __syncwarp();
            next_slot();
          }
        }
      }
      if (!ok)  // loads issued but perhaps never waited for: the last of each slot
        for (int k = 0; k < NST; ++k)
          if (used >> k & 1) mbar_wait(smem_addr(&sh.full[k]), k < slot ? phase : phase ^ 1, nullptr);
    } else {
      // ============================ products ============================
      // A warp per softmax group: what one does between products overlaps the other's products, and
      // neither waits for the other group's P.  This loop is the latency between a group's P and its
      // next S, so it is kept short: what it needs of a piece lies in (uniform) registers and ring
      // slots are counted.
      constexpr uint32_t id_s = tc05::instr_desc_bf16(128, kHalf, 0);
      constexpr uint32_t id_pv = tc05::instr_desc_bf16(128, D, 1);
      // (a reduction over the warp tells the compiler that a value is the same in all lanes)
      auto uni = [](int v) { return __reduce_max_sync(kFull, v); };
      const int g = uni(warp == kMmaWarp ? 0 : 1);
      const uint32_t q_base = smem_addr(smem) + g * C::SLOT, ring_base = smem_addr(ring);
      const uint32_t full0 = smem_addr(&sh.full[0]), empty0 = smem_addr(&sh.empty[0]);
      const uint32_t ts = tmem + kColS + g * kGroupCols, to = tmem + kColO + g * kGroupCols;
      const uint32_t sfull = smem_addr(&sh.sfull[g][0]), ofull = smem_addr(&sh.ofull[g]);
      const uint32_t pfull = smem_addr(&sh.pfull[g][0]), half_done = smem_addr(&sh.half_done[g]);
      bool ok = true;
      int kslot = 0, vslot = 1;
      uint32_t kphase = 0, vphase = 0, ppar = 0;  // parities of K's and V's slots, and of P
      auto next_slot = [](int& slot, uint32_t& phase) {
        slot += 2;
        if (slot >= NST) {
          slot -= NST;
          phase ^= 1;
        }
      };
      auto issue_s = [&](int h) {  // of 64 keys
        const uint64_t dq = tc05::smem_desc(q_base, 16, 1024);
        const uint64_t dk = tc05::smem_desc(ring_base + kslot * C::SLOT + h * (kHalf * 128), 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * C::CHUNK + (k & 3) * 32;
          tc05::mma_ss_warp(ts + h * (kHalf), dq + (off >> 4), dk + (off >> 4), id_s, k > 0);
        }
        tc05::commit_warp(sfull + 8 * h);
      };
      for (int n = 0; ok; ++n) {
        if (!(ok = piece_wait(n))) break;
        const Piece& pc = sh.pc[n % kPieces];
        const int cnt = uni(pc.cnt);
        if (cnt == 0) break;
        const int k00 = uni(pc.kt0) * kKT, lo = uni(pc.lo) - k00, hi = uni(pc.hi) - k00;
        const int ga = uni(pc.ga[g]), gb = uni(pc.gb[g]);
        piece_done(n);
        // S of the first tile
        if (!(ok = wait_warp(smem_addr(&sh.qfull), n & 1, p.err, abort_flag) &&
                   wait_warp(full0 + 8 * kslot, kphase, p.err, abort_flag)))
          break;
        tc05::fence_after_sync();
        if (ga == 0 && gb > 0) {
          issue_s(0);
          issue_s(1);
        }
        tc05::commit_warp(empty0 + 8 * kslot);
        if (cnt == 1) tc05::commit_warp(smem_addr(&sh.qempty));
        next_slot(kslot, kphase);
        for (int j = 0; j < cnt; ++j) {
          // all that can be waited for before P is
          const bool more = j + 1 < cnt, mine = j >= ga && j < gb, next = more && j + 1 >= ga && j + 1 < gb;
          if (!(ok = wait_warp(full0 + 8 * vslot, vphase, p.err, abort_flag))) break;
          const int a = max(lo - j * kKT, 0), z = min(hi - j * kKT, kKT);  // the item's keys within the tile
          if (rare(a > 0 || z < kKT)) {
            // V rows outside them may hold anything (0 * Inf is NaN): zero those that the product
            // reads, up to the 16-key steps (both warps write the same zeros)
            const int na = a & 15, nz = -z & 15;
            uint8_t* v = ring + vslot * C::SLOT;
            for (int e = lane; e < (na + nz) * DCH * 8; e += 32) {
              const int r = e / (DCH * 8), q = e % (DCH * 8);
              const int row = r < na ? a - na + r : z + r - na;
              *reinterpret_cast<uint4*>(v + (q >> 3) * C::CHUNK + row * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (more && !(ok = wait_warp(full0 + 8 * kslot, kphase, p.err, abort_flag))) break;
          if (mine) {
            const uint64_t dv = tc05::smem_desc(ring_base + vslot * C::SLOT, C::CHUNK, 1024);
            const int s0 = a >> 4, s1 = (z + 15) >> 4;
            uint32_t acc = j != ga;  // the group's first tile of the piece overwrites O
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // P comes in two halves, and the next S takes their places
              if (!(ok = wait_warp(pfull + 8 * h, ppar, p.err, abort_flag))) break;
              tc05::fence_after_sync();
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k) {
                if (k >= s0 && k < s1) {
                  tc05::mma_ts_warp(to, ts + h * (kHalf) + 8 * (k - 4 * h), dv + (k * 2048 >> 4), id_pv, acc);
                  acc = 1;
                }
              }
              if (h == 0) tc05::commit_warp(half_done);
              if (next) issue_s(h);
            }
            if (!ok) break;
            ppar ^= 1;
            if (j == gb - 1) tc05::commit_warp(ofull);
          } else if (next) {
            issue_s(0);
            issue_s(1);
          }
          tc05::commit_warp(empty0 + 8 * vslot);
          next_slot(vslot, vphase);
          if (more) {
            tc05::commit_warp(empty0 + 8 * kslot);
            if (j + 2 == cnt) tc05::commit_warp(smem_addr(&sh.qempty));
            next_slot(kslot, kphase);
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // every product issued has completed before the memory is freed
      __syncwarp();
      tc05::commit_warp(smem_addr(&sh.drain_bar[g]));
      mbar_wait(smem_addr(&sh.drain_bar[g]), 0, p.err);
    }
  } else {
    // ============================ softmax ============================
    setmaxnreg_inc<kSoftRegs>();
    const int g = warp >> 2, w = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(32 * w) << 16;
    const uint32_t ts = tmem + kColS + g * kGroupCols + lane_addr;
    const uint32_t to = tmem + kColO + g * kGroupCols + lane_addr;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    constexpr bool CAP_ONLY = C::CAP && !C::BIAS;
    constexpr bool PLAIN = !C::CAP && !C::BIAS;  // (with a positive scale: it commutes with the maximum)
    constexpr bool kTurns = PLAIN;
    const float mul = PLAIN ? p.scale_log2 : 1.f;
    const bool wide_out = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    const int r = 32 * w + lane;  // row of the M tile

    // items whose rows see nothing have no tile: their rows are zero
    const int items = p.header[0];
    for (int i0 = 0; s + i0 * p.ctas < items; i0 += kSoftWarps * 32) {
      const int64_t mine = s + static_cast<int64_t>(i0 + threadIdx.x) * p.ctas;
      unsigned empty = __ballot_sync(kFull, mine < items && p.tile_sum[mine + 1] == p.tile_sum[mine]);
      while (empty) {
        const int i = s + (i0 + 32 * warp + __ffs(empty) - 1) * p.ctas;
        empty &= empty - 1;
        const int rows = p.items[i].rows, row0 = p.items[i].row0, q0 = p.items[i].q0;
        for (int h = 0; h < p.Hkv; ++h)
          for (int e = lane; e < rows * (D / 8); e += 32) {
            const int f = row0 + e / (D / 8);
            *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(q0 + f / p.G) * p.Hq + h * p.G + f % p.G) * D +
                                      e % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
          }
      }
    }

    int done = 0, pieces = 0, turns = 0;  // phases of sfull, ofull and turn
    // rows of this group in a piece's M tile, and this thread's row of the sequence
    auto rows_of = [&](const Piece& pc) { return min(HR, pc.rows - g * HR); };
    auto mine = [&](const Piece& pc) { return pc.row0 + g * HR + min(r, max(rows_of(pc), 1) - 1); };
    // Warps w of the two groups share a sub-partition and its exponentials: they take turns at them,
    // group 0 first, so that one group's products run while the other computes.  (Left alone they
    // fall into step, compute at half the rate each and wait for their products together: 645 us
    // against 618 for a prompt of 8192 tokens.  Where scores are capped or biased the groups' other
    // arithmetic overlaps the exponentials better without turns: 366 us against 463 for 8 x 2048.)
    // Tiles that one of the groups skips have no turn.
    auto my_turn = [&] {
      if (g == 0 && turns == 0) return true;
      return wait_warp(smem_addr(&sh.turn[g ^ 1][w]), (g ? turns : turns - 1) & 1, p.err, abort_flag);
    };
    auto turn_over = [&] {
      ++turns;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.turn[g][w]));
    };
    RowLoads next{0, 0, 0.f};
    bool ok = piece_wait(0);
    if (ok && sh.pc[0].cnt != 0 && rows_of(sh.pc[0]) > 0) next = load_row(p, sh.pc[0], mine(sh.pc[0]));
    for (int i = 0; ok; ++i) {
      const Piece& pc = sh.pc[i % kPieces];  // (waited for)
      const int cnt = pc.cnt;
      if (cnt == 0) break;
      const int rows = rows_of(pc), f = mine(pc);
      Row row{0, 0, 0, 0.f};
      if (rows > 0) row = row_of(p, pc, f, next);
      const int ja = pc.ga[g], jb = pc.gb[g];
      const bool active = ja < jb;
      const int turn_lo = max(pc.ga[0], pc.ga[1]), turn_hi = min(pc.gb[0], pc.gb[1]);
      // keys that every row of the warp sees, and its first position
      int all_lo = row.lo, all_hi = row.hi, all_pos = row.pos;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(kFull, all_lo, off));
        all_hi = min(all_hi, __shfl_xor_sync(kFull, all_hi, off));
        all_pos = min(all_pos, __shfl_xor_sync(kFull, all_pos, off));
      }
      // (capped scores lie within the cap: their reference is fixed, with no maximum to be found)
      float m_ref = CAP_ONLY ? p.cap_ref : -INFINITY, l = 0.f;
      for (int j = ja; j < jb && ok; ++j, ++done) {
        const bool turn = kTurns && j >= turn_lo && j < turn_hi;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t sfull = smem_addr(&sh.sfull[g][0]);
          if (!(ok = wait_warp(sfull + 8 * h, done & 1, p.err, abort_flag))) break;
          tc05::fence_after_sync();
          const uint32_t tsh = ts + h * kHalf;
          if (rare(32 * w >= rows)) {  // none of the warp's rows is a row of the item
            if (turn) {
              if (!(ok = my_turn())) break;
              turn_over();
            }
            tc05::fence_before_sync();
            mbar_arrive(smem_addr(&sh.pfull[g][h]));
            continue;
          }
          const int key0 = (pc.kt0 + j) * kKT + h * kHalf;
          uint32_t raw[2][32];
          tc05::ld32(tsh, raw[0]);
          tc05::ld32(tsh + 32, raw[1]);
          tc05::wait_ld(raw[0], raw[1]);
          float x[kHalf];
#pragma unroll
          for (int e = 0; e < kHalf; ++e) x[e] = __uint_as_float(raw[e / 32][e % 32]);
          const bool masked = key0 < all_lo || key0 + kHalf > all_hi;
          float mt = m_ref;
          bool small = false;
          if constexpr (CAP_ONLY) {
            if (rare(masked)) mask_scores(x, row.lo - key0, row.hi - key0, 0.f);
            small = cap_is_small(p, largest_magnitude(x));
          } else {
            mt = modify_scores<C::CAP, C::BIAS, C::WIDE>(x, p, row, key0, masked, p.prefix_lens && key0 + kHalf - 1 > all_pos) *
                 mul;
          }
          const bool raise = mt > m_ref + kRescaleLog2;
          if (!CAP_ONLY && rare(__any_sync(kFull, raise))) {
            const float alpha = raise ? ex2_approx(m_ref - mt) : 1.f;
            if (j > ja || h > 0) {
              // the group's earlier P.V must be complete: the second half's S is issued behind those
              // of the tile before
              if (!(ok = wait_warp(h ? smem_addr(&sh.half_done[g]) : sfull + 8, done & 1, p.err, abort_flag))) break;
              tc05::fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t v[16];
                tc05::ld16(to + c, v);
                tc05::wait_ld(v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                tc05::st16(to + c, v);
              }
            }
            l *= alpha;
            if (raise) m_ref = mt;
          }
          if (turn && !(ok = my_turn())) break;
          const float2 mul2 = splat(mul), ref2 = splat(!CAP_ONLY && m_ref == -INFINITY ? 0.f : -m_ref);
          float2 l0 = make_float2(0.f, 0.f), l1 = l0;
          uint32_t v[32];
          auto weigh = [&](int e, float2 y) {
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
            if (e & 1) l1 = __fadd2_rn(l1, y); else l0 = __fadd2_rn(l0, y);
            v[e] = pack_bf16x2(y.x, y.y);
          };
          if (CAP_ONLY && __builtin_expect(small && !masked, 1)) {
            // caps and exponentials in one block: the caps of some scores run on the FMA pipe while
            // the exponentials of others have theirs (one after the other: 418 us for 370)
#pragma unroll
            for (int c = 0; c < kHalf; c += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = x[c + e];
              cap_polynomial(y, p, ref2.x);
#pragma unroll
              for (int e = 0; e < 4; ++e) weigh(c / 2 + e, make_float2(y[2 * e], y[2 * e + 1]));
            }
          } else {
            if constexpr (CAP_ONLY) {
              cap_scores(x, p, small, ref2.x);
              if (rare(masked)) mask_scores(x, row.lo - key0, row.hi - key0, -INFINITY);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 y = make_float2(x[2 * e], x[2 * e + 1]);
              // (cap_scores has added the reference)
              weigh(e, CAP_ONLY ? y : PLAIN ? __ffma2_rn(y, mul2, ref2) : __fadd2_rn(y, ref2));
            }
          }
          tc05::st32(tsh, v);
          tc05::wait_st();
          tc05::fence_before_sync();
          mbar_arrive(smem_addr(&sh.pfull[g][h]));
          if (turn) turn_over();
          l += (l0.x + l0.y) + (l1.x + l1.y);
        }
      }
      if (!ok) break;

      // ---- the piece's output, or its partial ----
      if (!(ok = piece_wait(i + 1))) break;
      {
        const Piece& np = sh.pc[(i + 1) % kPieces];
        if (np.cnt != 0 && rows_of(np) > 0) next = load_row(p, np, mine(np));
      }
      const bool whole = pc.whole;
      const int64_t base = static_cast<int64_t>(s) * 2 + pc.slot;
      if (active) {
        if (!(ok = wait_warp(smem_addr(&sh.ofull[g]), pieces & 1, p.err, abort_flag))) break;
        ++pieces;
        tc05::fence_after_sync();
      }
      if (rows > 0) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
        const int t = f / p.G;
        __nv_bfloat16* o =
            out + (static_cast<int64_t>(pc.q0 + t) * p.Hq + pc.kvh * p.G + (f - t * p.G)) * D;
        const int pr = g * HR + r;  // row of the partial
        if (!whole && r < rows) reinterpret_cast<float2*>(p.part_ml)[base * p.RT + pr] = make_float2(m_ref, l);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          if (active) {
            tc05::ld32(to + c, v);
            tc05::wait_ld(v);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (r < rows) {
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                uint32_t u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  u[k] = pack_bf16x2(__uint_as_float(v[e + 2 * k]) * inv, __uint_as_float(v[e + 2 * k + 1]) * inv);
                if (wide_out) {  // whole 32-byte sectors: every lane writes a line of its own
                  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + c + e), "r"(u[0]),
                               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                               : "memory");
                } else {
                  *reinterpret_cast<uint4*>(o + c + e) = make_uint4(u[0], u[1], u[2], u[3]);
                  *reinterpret_cast<uint4*>(o + c + e + 8) = make_uint4(u[4], u[5], u[6], u[7]);
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                reinterpret_cast<float4*>(p.part_acc)[(base * (D / 4) + (c + e) / 4) * p.RT + pr] =
                    make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]),
                                __uint_as_float(v[e + 3]));
            }
          }
          __syncwarp();
        }
      }
      tc05::fence_before_sync();  // the reads of O come before the next piece's products
      piece_done(i);
    }
    if (!ok) *abort_flag = 1;
  }

  // ---- exit: every role is done; free the tensor memory ----
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  if (warp == kMmaWarp) tc05::dealloc(tmem, kTmemCols);
}

template <class C>
cudaError_t run(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap tmk, tmv, tmq;
  const int tokens = p.HR / p.G;
  if (!make_pool_map(&tmk, p.k_pool, p.num_blocks, p.block_size, p.Hkv, C::D, p.block_size) ||
      !make_pool_map(&tmv, p.v_pool, p.num_blocks, p.block_size, p.Hkv, C::D, p.block_size) ||
      !make_q_rows_map(&tmq, p.q, p.T, p.Hq, C::D, p.q_stride, p.G, tokens))
    return cudaErrorInvalidValue;
  static SmemGrant granted;
  const cudaError_t e = grant_smem(granted, attention_tc_kernel<C>, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(attention_tc_kernel<C>, dim3(static_cast<unsigned>(p.ctas)), kThreads, C::SMEM, stream, tmk, tmv,
                    tmq, p);
}

}  // namespace

// What a unit costs beside its tiles, in tiles.
int attention_tc_extra() { return 2; }

// Rows per item: two M tiles of whole tokens.
int attention_tc_rows(int G) { return 2 * (128 / G) * G; }

template <int D>
static cudaError_t run_modified(const AttnParams& p, cudaStream_t stream) {
  // a cap too wide for one reference is the general case, as a negative scale is
  const bool cap = p.cap_out > 0.f, bias = p.slopes != nullptr || (cap ? !(p.cap_ref < INFINITY) : !(p.scale_log2 > 0.f));
  if (p.cap_wide) return run<TcAttn<D, true, true, true>>(p, stream);
  if (cap) return bias ? run<TcAttn<D, true, true>>(p, stream) : run<TcAttn<D, true, false>>(p, stream);
  return bias ? run<TcAttn<D, false, true>>(p, stream) : run<TcAttn<D, false, false>>(p, stream);
}

cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t stream) {
  return p.D == 64 ? run_modified<64>(p, stream) : run_modified<128>(p, stream);
}

}  // namespace pa
