// Rotary positions fused with the paged cache write (sm_100a).
//
// For token t at position p and rotated pair i the angle is theta = p * inv_freq[i], and the
// pair (a, b) becomes f * (a cos theta - b sin theta, a sin theta + b cos theta): pairs are
// elements (i, i + R/2) of the head (half layout) or (2i, 2i + 1) (interleaved), elements
// R .. D-1 pass through.  q goes to q_out, k to its slot of the key pool, v unchanged to its
// slot of the value pool ("什么是 LLM 中的分页注意力", 块表: slot s is row s of the pool viewed
// as [NB*BS][Hkv][D]).
//
// The angle is formed and reduced in 64 bits (turns = p * inv_freq / 2 pi, minus the nearest
// whole number): at position 10^5 a 32-bit product is off by up to 2^-24 * 10^5 = 0.006 rad.
// The fraction of a turn is then below 1/2 and 32 bits hold it to 2^-25; sincospif takes it
// from there.  One CTA serves one token, so a token's R/2 sines and cosines are computed once
// for all its Hq + Hkv heads.
//
// Bound by memory: q, k and v are read once and written once, in 16-byte vectors.  A thread keeps
// its place within a head and walks over the heads, so that its sines and cosines stay in
// registers and no index is divided (where every vector's place was computed for itself the
// instructions took as long as the memory).  The loads of its first kAhead heads come before
// anything else: the latencies of the data, of the token's position and slot, and of the angles
// overlap.  Three forms by where a pair lies: in two vectors R / 2 apart (half layout, R / 2 a
// whole number of vectors), within one vector (interleaved), or anywhere (half layout otherwise:
// the token's rows pass through shared memory).  Where a stride is not a multiple of 16 bytes a
// scalar form runs.  16384 tokens, 32/8 heads of 128 in bf16: 65 us (6.2 TB/s) with 64 elements
// interleaved, 61 us with whole heads in halves, 95 us with 50 elements in halves (staged: each
// element's partner is read by itself from shared memory, and a barrier stands between the loads and the
// stores), 206 us with whole heads in the scalar form; 256 tokens: 3 us.

#include <cuda_bf16.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;

template <typename T>
struct Vec;  // 16 bytes of T
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  // the one rounding: each rotated element to nearest bf16
  __device__ static uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

template <typename T>
__device__ __forceinline__ float as_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// cos and sin (times the factor) of this token's pairs into cs[R/2]; positions are exact in
// 64 bits, so far ones lose nothing.
__device__ __forceinline__ void angles(const RopeParams& p, int pos, float2* cs) {
  for (int i = threadIdx.x; i < p.R / 2; i += kThreads) {
    const double turns = static_cast<double>(pos) * __ldg(p.inv_freq + i) * 0.15915494309189535;
    const float frac = static_cast<float>(turns - rint(turns));
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs[i] = make_float2(c * p.factor, s * p.factor);
  }
}

enum Form { kHalf, kInterleaved, kStaged };

// 1 << shift threads share a head of q, k or v (its place: w); in the kHalf form place w < R/2/N
// takes the vectors at wN and wN + R/2, and the next ones the vectors from R on.
template <typename T, Form FORM>
__global__ void __launch_bounds__(kThreads, 8) rope_vec_kernel(const RopeParams p, int shift) {
  constexpr int N = Vec<T>::N;
  constexpr bool HALF = FORM == kHalf;
  constexpr int kAhead = HALF ? 3 : 6;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float2 cs[];
  T* staged = reinterpret_cast<T*>(cs + (p.R / 2 + 1) / 2 * 2);  // kStaged: [Hq + Hkv][D]
  const int64_t t = blockIdx.x;
  const int D = p.D, R = p.R, half = R / 2;
  const int w = threadIdx.x & ((1 << shift) - 1), step = kThreads >> shift;
  const bool pair = HALF && w * N < half;  // two vectors
  const int lead = !HALF || pair ? w * N : R + w * N - half;
  const bool turns = HALF ? pair : lead < R;  // of a head of q or k
  const int rotated = p.Hq + p.Hkv;
  const int heads = lead < D ? rotated + p.Hkv : 0;  // (places past the head are idle)
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride + lead;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride + lead;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride + lead;
  auto load = [&](int h, uint4& a, uint4& b) {
    const T* src = h < p.Hq ? q + h * D : h < rotated ? k + (h - p.Hq) * D : v + (h - rotated) * D;
    a = *reinterpret_cast<const uint4*>(src);
    if (pair) b = *reinterpret_cast<const uint4*>(src + half);
  };

  const int h0 = threadIdx.x >> shift;
  uint4 a[kAhead], b[kAhead];
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    if (h0 + s * step < heads) load(h0 + s * step, a[s], b[s]);
  const int64_t slot = __ldg(p.slots + t);
  angles(p, __ldg(p.positions + t), cs);
  const bool bad = slot >= p.num_slots;
  if (bad && threadIdx.x == 0) flag_error(p.err, PA_DEVERR_BAD_SLOT);
  const bool write = slot >= 0 && !bad;
  T* qo = static_cast<T*>(p.q_out) + t * p.Hq * D + lead;
  T* kp = static_cast<T*>(p.k_pool) + (write ? slot : 0) * p.Hkv * D + lead;
  T* vp = static_cast<T*>(p.v_pool) + (write ? slot : 0) * p.Hkv * D + lead;
  if (FORM == kStaged) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
      if (h0 + s * step < min(heads, rotated))
        *reinterpret_cast<uint4*>(staged + (h0 + s * step) * D + lead) = a[s];
    for (int h = h0 + kAhead * step; h < min(heads, rotated); h += step) {
      uint4 x, none;
      load(h, x, none);
      *reinterpret_cast<uint4*>(staged + h * D + lead) = x;
    }
  }
  __syncthreads();
  float2 c[N];  // of this place's elements (pairs)
  if (turns) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = lead + j;
      if (HALF) c[j] = cs[e];
      if (FORM == kInterleaved && j % 2 == 0) c[j] = e < R ? cs[e / 2] : make_float2(1.f, 0.f);
      if (FORM == kStaged) c[j] = e < half ? cs[e] : e < R ? cs[e - half] : make_float2(1.f, 0.f);
    }
  }
  auto store = [&](int h, const uint4& a0, const uint4& b0) {
    if (h >= p.Hq && !write) return;
    T* dst = h < p.Hq ? qo + h * D : h < rotated ? kp + (h - p.Hq) * D : vp + (h - rotated) * D;
    if (!turns || h >= rotated) {
      *reinterpret_cast<uint4*>(dst) = a0;
      if (pair) *reinterpret_cast<uint4*>(dst + half) = b0;
      return;
    }
    float x[N];
    Vec<T>::unpack(a0, x);
    if (HALF) {
      float y[N];
      Vec<T>::unpack(b0, y);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float xr = x[j] * c[j].x - y[j] * c[j].y;
        y[j] = x[j] * c[j].y + y[j] * c[j].x;
        x[j] = xr;
      }
      *reinterpret_cast<uint4*>(dst + half) = Vec<T>::pack(y);
    } else if (FORM == kInterleaved) {
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        if (lead + j >= R) break;  // (what is not rotated stays as it is: exact both ways)
        const float xr = x[j] * c[j].x - x[j + 1] * c[j].y;
        x[j + 1] = x[j] * c[j].y + x[j + 1] * c[j].x;
        x[j] = xr;
      }
    } else {
      const T* row = staged + h * D;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = lead + j;
        if (e >= R) break;
        const bool second = e >= half;
        const float other = as_f(row[second ? e - half : e + half]);
        x[j] = second ? other * c[j].y + x[j] * c[j].x : x[j] * c[j].x - other * c[j].y;
      }
    }
    *reinterpret_cast<uint4*>(dst) = Vec<T>::pack(x);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    if (h0 + s * step < heads) store(h0 + s * step, a[s], b[s]);
  for (int h = h0 + kAhead * step; h < heads; h += step) {
    uint4 x, y;
    load(h, x, y);
    store(h, x, y);
  }
}

// The same, one pair (or one unrotated element) at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(const RopeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float2 cs[];
  const int64_t t = blockIdx.x;
  const int D = p.D, R = p.R;
  const int64_t slot = __ldg(p.slots + t);
  const bool bad = slot >= p.num_slots;
  if (bad && threadIdx.x == 0) flag_error(p.err, PA_DEVERR_BAD_SLOT);
  const bool write = slot >= 0 && !bad;
  angles(p, __ldg(p.positions + t), cs);
  __syncthreads();
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  T* qo = static_cast<T*>(p.q_out) + t * p.Hq * D;
  T* kp = static_cast<T*>(p.k_pool) + (write ? slot : 0) * p.Hkv * D;
  T* vp = static_cast<T*>(p.v_pool) + (write ? slot : 0) * p.Hkv * D;
  const int uph = R / 2 + (D - R);
  const int units = (write ? p.Hq + p.Hkv : p.Hq) * uph;
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const int h = i / uph, w = i - h * uph;
    const T* src = h < p.Hq ? q + h * D : k + (h - p.Hq) * D;
    T* dst = h < p.Hq ? qo + h * D : kp + (h - p.Hq) * D;
    if (w >= R / 2) {
      const int e = R + (w - R / 2);
      dst[e] = src[e];
      continue;
    }
    const int ea = p.half ? w : 2 * w, eb = p.half ? w + R / 2 : 2 * w + 1;
    const float a = as_f(src[ea]), b = as_f(src[eb]);
    const float2 c = cs[w];
    dst[ea] = from_f<T>(a * c.x - b * c.y);
    dst[eb] = from_f<T>(a * c.y + b * c.x);
  }
  if (write)
    for (int i = threadIdx.x; i < p.Hkv * D; i += kThreads) vp[i] = v[i];
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  auto mult = [](int64_t a) { return a % N == 0; };
  const bool vec = mult(p.q_stride) && mult(p.k_stride) && mult(p.v_stride) &&
                   (reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                    reinterpret_cast<uintptr_t>(p.v)) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(p.T));
  const size_t smem = static_cast<size_t>((p.R / 2 + 1) / 2 * 2) * sizeof(float2);
  const size_t rows = static_cast<size_t>(p.Hq + p.Hkv) * p.D * sizeof(T);
  int shift = 0;  // threads of a head: a power of two, at least its places
  const int places = p.half && mult(p.R / 2) ? (p.D - p.R / 2) / N : p.D / N;
  while ((1 << shift) < places) ++shift;
  if (vec && !p.half) return launch_pdl(rope_vec_kernel<T, kInterleaved>, grid, kThreads, smem, stream, p, shift);
  if (vec && mult(p.R / 2)) return launch_pdl(rope_vec_kernel<T, kHalf>, grid, kThreads, smem, stream, p, shift);
  // (in the shared memory that needs no grant)
  if (vec && smem + rows <= 48 * 1024)
    return launch_pdl(rope_vec_kernel<T, kStaged>, grid, kThreads, smem + rows, stream, p, shift);
  return launch_pdl(rope_scalar_kernel<T>, grid, kThreads, smem, stream, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, pa_dtype dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace pa
