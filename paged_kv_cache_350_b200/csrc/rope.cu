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
// Bound by memory: q, k and v are read once and written once, in 16-byte vectors.  Each
// thread issues the loads of its first pairs before the angles are computed, so that the two
// latencies overlap.  Where a layout's pairs do not fall into whole 16-byte vectors, or a
// stride is not a multiple of 16 bytes, a scalar variant runs.

#include <cuda_bf16.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

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

// A token's work in units of 16-byte vectors.  Rotated heads (q, then k): in the half layout a
// unit is the vector pair (u, u + R/2/N); in the interleaved one a single vector; past R
// a unit is a plain copy of one vector.  Then v's vectors.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(const RopeParams p) {
  constexpr int N = Vec<T>::N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float2 cs[];
  const int64_t t = blockIdx.x;
  const int D = p.D, R = p.R;
  const int rot = HALF ? R / 2 / N : R / N;  // rotating units of a head
  const int uph = rot + (D - R) / N;         // units of a rotated head
  const int units = (p.Hq + p.Hkv) * uph;
  const int total = units + p.Hkv * (D / N);
  const int64_t slot = __ldg(p.slots + t);
  const bool bad = slot >= p.num_slots;
  if (bad && threadIdx.x == 0) flag_error(p.err, PA_DEVERR_BAD_SLOT);
  const bool write = slot >= 0 && !bad;
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  T* qo = static_cast<T*>(p.q_out) + t * p.Hq * D;
  T* kp = static_cast<T*>(p.k_pool) + (write ? slot : 0) * p.Hkv * D;
  T* vp = static_cast<T*>(p.v_pool) + (write ? slot : 0) * p.Hkv * D;

  struct Unit {
    const T* src;
    T* dst;
    int lead;  // first element within the head
    bool rotates;
  };
  auto unit = [&](int i) -> Unit {
    Unit u;
    if (i < units) {
      const int h = i / uph, w = i - h * uph;
      u.rotates = w < rot;
      u.lead = u.rotates ? w * N : R + (w - rot) * N;
      if (h < p.Hq) {
        u.src = q + h * D + u.lead;
        u.dst = qo + h * D + u.lead;
      } else {
        u.src = write ? k + (h - p.Hq) * D + u.lead : nullptr;
        u.dst = kp + (h - p.Hq) * D + u.lead;
      }
    } else {
      const int w = i - units;
      u.rotates = false;
      u.lead = 0;
      u.src = write ? v + w * N : nullptr;
      u.dst = vp + w * N;
    }
    return u;
  };
  auto load = [&](const Unit& u, uint4& a, uint4& b) {
    if (!u.src) return;
    a = *reinterpret_cast<const uint4*>(u.src);
    if (HALF && u.rotates) b = *reinterpret_cast<const uint4*>(u.src + R / 2);
  };
  auto store = [&](const Unit& u, const uint4& a, const uint4& b) {
    if (!u.src) return;
    if (!u.rotates) {
      *reinterpret_cast<uint4*>(u.dst) = a;
      return;
    }
    if (HALF) {
      float x[N], y[N];
      Vec<T>::unpack(a, x);
      Vec<T>::unpack(b, y);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 c = cs[u.lead + j];
        const float xr = x[j] * c.x - y[j] * c.y;
        y[j] = x[j] * c.y + y[j] * c.x;
        x[j] = xr;
      }
      *reinterpret_cast<uint4*>(u.dst) = Vec<T>::pack(x);
      *reinterpret_cast<uint4*>(u.dst + R / 2) = Vec<T>::pack(y);
    } else {
      float x[N];
      Vec<T>::unpack(a, x);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 c = cs[(u.lead + j) / 2];
        const float xr = x[j] * c.x - x[j + 1] * c.y;
        x[j + 1] = x[j] * c.y + x[j + 1] * c.x;
        x[j] = xr;
      }
      *reinterpret_cast<uint4*>(u.dst) = Vec<T>::pack(x);
    }
  };

  Unit u0{}, u1{};
  uint4 a0{}, b0{}, a1{}, b1{};
  const int i0 = threadIdx.x, i1 = threadIdx.x + kThreads;
  if (i0 < total) load(u0 = unit(i0), a0, b0);
  if (i1 < total) load(u1 = unit(i1), a1, b1);
  angles(p, __ldg(p.positions + t), cs);
  __syncthreads();
  if (i0 < total) store(u0, a0, b0);
  if (i1 < total) store(u1, a1, b1);
  for (int i = i1 + kThreads; i < total; i += kThreads) {
    const Unit u = unit(i);
    uint4 a{}, b{};
    load(u, a, b);
    store(u, a, b);
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
  const bool vec = (p.half ? mult(p.R / 2) : mult(p.R)) && mult(p.R) && mult(p.q_stride) &&
                   mult(p.k_stride) && mult(p.v_stride) &&
                   (reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                    reinterpret_cast<uintptr_t>(p.v)) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(p.T));
  const size_t smem = static_cast<size_t>(p.R / 2) * sizeof(float2);
  if (!vec) return launch_pdl(rope_scalar_kernel<T>, grid, kThreads, smem, stream, p);
  return p.half ? launch_pdl(rope_vec_kernel<T, true>, grid, kThreads, smem, stream, p)
                : launch_pdl(rope_vec_kernel<T, false>, grid, kThreads, smem, stream, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, pa_dtype dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace pa
