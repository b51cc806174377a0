// Attention of ragged query tokens over the paged cache: the parameter block, the work plan
// and the visibility rule that its kernels share (device code).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// One item: RT consecutive rows of a sequence, for one KV head.  A row is a (query token, head
// of the group) pair, numbered token * G + head, so a tile is full whatever G is.
struct AttnItem {
  int b, q0;         // sequence; its first query token (row of q and out)
  int row0, rows;    // first row of the item within the sequence, rows
  int L, pos0;       // cached tokens; position of the sequence's first query token (L - n)
  int lo, hi;        // keys that any row may see: [lo, hi)
  int glo[2], ghi[2];  // the same of its rows [0, HR) and [HR, 2 HR)
};

// The cut unit that begins in a CTA's range: its pieces (0: none), the slot of the first one's
// partial, and where its rows go.
struct __align__(16) AttnCut {
  int pieces, slot, kvh, q0, row0, rows, pad0, pad1;
};

// Where a CTA's range begins: the slot (extra ones, then tiles) of a unit, and the range's slots.
struct AttnStart {
  int item, kvh, tile, count;
};

// The part of a unit of `slots` slots that a range with `left` slots to go takes from slot
// `slot` on: its slots, and its tiles [tile, tile + cnt) of nt.  A range that begins among the
// unit's extra slots begins with its first tile; one that ends there takes none.
struct UnitPart {
  int slots, nt, tile, cnt;
};

__device__ __forceinline__ UnitPart unit_part(const AttnParams& p, int slots, int slot, int left) {
  UnitPart u;
  u.slots = min(left, slots - slot);
  u.nt = slots - p.extra;
  u.tile = max(slot - p.extra, 0);
  u.cnt = max(slot + u.slots - p.extra - u.tile, 0);
  return u;
}

__device__ __forceinline__ int attn_len(const AttnParams& p, int b, bool flag) {
  const int L = __ldg(p.seq_lens + b);
  const int most = p.max_blocks * p.block_size;
  if (L < 0 || L > most) {
    if (flag) flag_error(p.err, PA_DEVERR_BAD_SEQ_LEN);
    return L < 0 ? 0 : most;
  }
  return L;
}

// Query tokens of sequence b: [q0, q0 + n); none where the span is malformed or longer than
// the caller said.
__device__ __forceinline__ int attn_query_span(const AttnParams& p, int b, bool flag, int& q0) {
  const int s0 = __ldg(p.query_starts + b), s1 = __ldg(p.query_starts + b + 1);
  const bool bad = s0 < 0 || s1 < s0 || s1 > p.T || s1 - s0 > p.max_query_len;
  if (bad && flag) flag_error(p.err, PA_DEVERR_BAD_SEQ_LEN);
  q0 = s0;
  return bad ? 0 : s1 - s0;
}

// cap * tanh(scale * s / cap) * log2 e of a raw score s, by tanh t = 1 - 2 / (1 + e^2t) of t = s * cap_in:
// the error is absolute, 2^-22 of the cap, as this cancels for small t.
__device__ __forceinline__ float cap_score(float t, float cap_out) {
  return fmaf(-2.f * cap_out, rcp_approx(1.f + ex2_approx(t * (2.f * kLog2e))), cap_out);
}

// The same below |t| = kNearTanh: scale * s times the series of tanh(t) / t up to t^8 (the next term is
// 2.4e-7 there).  With the other one above it the error is 2^-20 of the result, whatever the cap.
constexpr float kNearTanh = 0.35f;
__device__ __forceinline__ float cap_score_near(float s, float t, float scale_log2) {
  const float u = t * t;
  float y = fmaf(u, 62.f / 2835.f, -17.f / 315.f);
  y = fmaf(y, u, 2.f / 15.f);
  y = fmaf(y, u, -1.f / 3.f);
  y = fmaf(y, u, 1.f);
  return s * scale_log2 * y;
}

// Keys visible to the query token at position pos of a sequence of L tokens: [lo, hi) with
//   key j visible iff j < L, (j <= pos or j < prefix), j > pos - window (if any), j >= first.
// A position below 0 (more query tokens than cached ones) sees nothing.
__device__ __forceinline__ void attn_visible(const AttnParams& p, int pos, int L, int prefix,
                                             int first, int& lo, int& hi) {
  hi = min(max(pos + 1, prefix), L);
  lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  lo = max(lo, first);
  if (pos < 0 || lo >= hi) lo = hi = 0;
}

}  // namespace pa
