// optim.cu -- AdamW over many tensors, with full or 8-bit states, and the
// global gradient norm.
//
// One step, for every element of every tensor (t counts the steps taken):
//   g = c * grad                      c: the caller's scale times the clipping factor
//   m = beta1 m + (1 - beta1) g
//   v = beta2 v + (1 - beta2) g^2
//   p = p - lr w p - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// The arithmetic is fp32 (fp64 for fp64 parameters); the update uses m and v
// before any rounding to 8 bits.
//
// 8-bit states.  256 consecutive elements of a tensor share a scale, s =
// max|x| / 448, and hold x / s as e4m3 codes: x = m for the first moment, x =
// r = sqrt(v) for the second, so that both moments cover the same range of
// gradient magnitudes.  One step moves v by 0.1 % (beta2 = 0.999), far less
// than the codes' spacing (6-12 %), so rounding to nearest would freeze them:
// both moments round at random between the two neighbouring codes, with the
// chance that keeps the mean of m, and of v = r^2 (to 2^-16 of the codes'
// spacing, the random numbers' own).  With k d the lower
// neighbour, (k + 1) d the upper one and f = x / (s d) - k, the upper one is
// taken with chance f for m and f (2 k + f) / (2 k + 1) for r.  The random
// bits are a hash of (seed, step, tensor, element), so a step is reproducible
// whatever its launch shape.  A positive r never rounds to 0: the smallest
// code is taken, which makes the update smaller, never m / eps; where r is 0
// m is stored as 0, too.
#include "optim.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "launch.cuh"
#include "qml.h"

namespace qml {

namespace {

constexpr int kThreadsOpt = 256;

// ---------------------------------------------------------------- wide loads

// Eight consecutive values of T as 32-bit words.
template <class T>
struct Raw {
  uint32_t w[8 * sizeof(T) / 4];
};

struct E4m3 {
  uint8_t x;
};

template <int W>
__device__ __forceinline__ void ld_words(uint32_t* w, const void* p) {
  if constexpr (W >= 8) {
#pragma unroll
    for (int i = 0; i < W; i += 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(static_cast<const char*>(p) + 4 * i));
  } else if constexpr (W == 4) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  } else {
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  }
}

template <int W>
__device__ __forceinline__ void st_words(const uint32_t* w, void* p) {
  if constexpr (W >= 8) {
#pragma unroll
    for (int i = 0; i < W; i += 8)
      asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]),
                   "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7]),
                   "l"(static_cast<char*>(p) + 4 * i)
                   : "memory");
  } else if constexpr (W == 4) {
    asm volatile("st.global.v4.b32 [%4], {%0,%1,%2,%3};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "l"(p)
                 : "memory");
  } else {
    asm volatile("st.global.v2.b32 [%2], {%0,%1};" ::"r"(w[0]), "r"(w[1]), "l"(p) : "memory");
  }
}

template <class T>
__device__ __forceinline__ Raw<T> ld8(const T* p) {
  Raw<T> r;
  ld_words<8 * sizeof(T) / 4>(r.w, p);
  return r;
}

// Values of one type in the arithmetic type C and back (to nearest even: the
// rounding of every store of a bf16 / fp16 parameter).
template <class C>
__device__ __forceinline__ C up(float x) { return (C)x; }
template <class C>
__device__ __forceinline__ C up(double x) { return (C)x; }
template <class C>
__device__ __forceinline__ C up(__nv_bfloat16 x) { return (C)__bfloat162float(x); }
template <class C>
__device__ __forceinline__ C up(__half x) { return (C)__half2float(x); }
template <class C>
__device__ __forceinline__ C up(E4m3 x) { return (C)__half2float(__half(__nv_cvt_fp8_to_halfraw(x.x, __NV_E4M3))); }
template <class T, class C>
__device__ __forceinline__ T down(C x);
template <>
__device__ __forceinline__ float down<float, float>(float x) { return x; }
template <>
__device__ __forceinline__ double down<double, double>(double x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16, float>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half down<__half, float>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ E4m3 down<E4m3, float>(float x) {
  return E4m3{(uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3)};
}

template <class C, class T>
__device__ __forceinline__ void unpack(const Raw<T>& r, C (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 1) {
      if (j % 2 == 0) {
        const uint32_t two = r.w[j / 4] >> (8 * (j % 4));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
        x[j] = f.x, x[j + 1] = f.y;
      }
    } else if constexpr (sizeof(T) == 2) {
      if (j % 2 == 0) {
        const uint32_t two = r.w[j / 2];
        float2 f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          f = make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
        } else {
          f = __half22float2(*reinterpret_cast<const __half2*>(&two));
        }
        x[j] = f.x, x[j + 1] = f.y;
      }
    } else if constexpr (sizeof(T) == 4) {
      x[j] = __uint_as_float(r.w[j]);
    } else {
      x[j] = __hiloint2double((int)r.w[2 * j + 1], (int)r.w[2 * j]);
    }
  }
}

template <class T, class C>
__device__ __forceinline__ void st8(T* p, const C (&x)[8]) {
  Raw<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 1) {
      if (j % 4 == 0) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[j], x[j + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[j + 2], x[j + 3]), __NV_SATFINITE, __NV_E4M3);
        r.w[j / 4] = lo | hi << 16;
      }
    } else if constexpr (sizeof(T) == 2) {
      if (j % 2 == 0) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const __nv_bfloat162 two = __floats2bfloat162_rn(x[j], x[j + 1]);
          r.w[j / 2] = *reinterpret_cast<const uint32_t*>(&two);
        } else {
          const __half2 two = __floats2half2_rn(x[j], x[j + 1]);
          r.w[j / 2] = *reinterpret_cast<const uint32_t*>(&two);
        }
      }
    } else if constexpr (sizeof(T) == 4) {
      r.w[j] = __float_as_uint(x[j]);
    } else {
      r.w[2 * j] = (uint32_t)__double2loint(x[j]), r.w[2 * j + 1] = (uint32_t)__double2hiint(x[j]);
    }
  }
  st_words<8 * sizeof(T) / 4>(r.w, p);
}

// ------------------------------------------------------------ random rounding

// 32-bit integer mixer: xorshifts and two odd multipliers, whose constants C.
// Wellons published in 2018 as the result of a search for low bias.  An element's two
// random numbers are the low and the high half of mix(): from the value before
// its last step, y, these are the low half xor the high half, and the high half.
__device__ __forceinline__ uint32_t mix_most(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  return x * 0x846ca68bu;
}
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = mix_most(x);
  return x ^ (x >> 16);
}

// Packed fp32 arithmetic: one instruction for two elements.  A packed product
// and the packed sum that takes it are compiled into one multiply-add, with or
// without the _rn names; where that would change a result, the sum is apart().
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 apart(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Rounding of a >= 0 (x in units of its block's scale) to a neighbouring e4m3
// value, upwards where the element's 16-bit uniform number u is below the
// chance; what reaches 480 is taken down to 448 by the saturating conversion.
// y: the random bits, see mix_most().
//
// First moment, chance f.  A positive float's bits beyond e4m3's three
// fraction bits are f in units of 2^-20: adding 2^20 - 1 - 16 u carries into
// the kept bits exactly where f > u.  Below 2^-6 the spacing is 2^-9, which a +
// 2^-6 has as its float's third fraction bit; the sum is rounded upwards, to a
// multiple of 2^-20 spacings, so f > u (u a multiple of 2^-16) holds after it
// exactly where it held before.  The sign is x's.
__device__ __forceinline__ float2 round_first(float2 x, float2 inv, const uint32_t (&y)[2]) {
  const float2 a = mul2(x, inv);
  auto below = [](float t) {
    float one;
    asm("set.lt.f32.f32 %0, %1, %2;" : "=f"(one) : "f"(fabsf(t)), "f"(0.015625f));
    return one;
  };
  auto carry = [](float t, float off, uint32_t w) {
    const uint32_t r = ~((w << 4 | w >> 28) ^ (w << 20 | w >> 12)) & 0xffff0u;  // 16 (2^16 - 1 - u)
    return __uint_as_float((__float_as_uint(__fadd_ru(fabsf(t), off)) + r + 15u) & 0xfff00000u);
  };
  const float2 off = mul2(make_float2(below(a.x), below(a.y)), both(0.015625f));
  const float2 q = add2(make_float2(carry(a.x, off.x, y[0]), carry(a.y, off.y, y[1])), neg2(off));
  return make_float2(copysignf(q.x, x.x), copysignf(q.y, x.y));
}

// Second moment: a lies between lo and lo + d (d the spacing of its binade, 2^-9
// below 2^-6); up where (a - lo) (a + lo) > u d (2 lo + d), the chance that
// keeps the mean of a^2.  The right side is exact (16 + 5 bits), the left one
// rounded twice.  Where lo = 0 the right side is taken as -a: the left one may
// underflow to 0, but every positive r rounds up and none vanishes.
__device__ __forceinline__ float2 round_second(float2 r, float2 inv, const uint32_t (&y)[2]) {
  const float2 a = mul2(r, inv);
  auto binade = [](float t) { return __uint_as_float(max(__float_as_uint(t) & 0x7f800000u, 121u << 23)); };
  const float2 e = make_float2(binade(a.x), binade(a.y));  // 2^floor(log2 a), at least 2^-6; d = e / 8
  const float2 d = mul2(e, both(0.125f)), m = mul2(e, both(1048576.f));
  const float2 lo = add2(__fadd2_rd(a, m), neg2(m));  // the unit of m's last place is d
  const float2 left = mul2(add2(a, neg2(lo)), add2(a, lo));
  auto uniform = [](uint32_t w) { return __uint_as_float(__byte_perm(w, 0x41800000u, 0x7632)); };  // 16 + u / 8
  const float2 u = add2(make_float2(uniform(y[0]), uniform(y[1])), both(-16.f));
  const float2 right = mul2(mul2(u, e), fma2(lo, both(2.f), d)), most = fma2(lo, both(0x1p40f), neg2(a));
  auto above = [](float l, float r0, float r1) {
    float one;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(one) : "f"(l), "f"(fminf(r0, r1)));
    return one;
  };
  return fma2(make_float2(above(left.x, right.x, most.x), above(left.y, right.y, most.y)), d, lo);
}

// Block maximum as the bits of a float: NaN is the largest.
__device__ __forceinline__ uint32_t block_max(const float2 (&x)[4]) {
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(fabsf(x[j].x)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(fabsf(x[j].y)));
  }
  return __reduce_max_sync(0xffffffffu, __float_as_uint(t));
}

// The scale of a block.  One with a NaN or infinity gets the scale NaN.
__device__ __forceinline__ float block_scale(uint32_t top, float base) {
  const float s = __fmul_rn(base, 1.f / kE4m3Max);
  return top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : top ? s : 0.f;
}

// r = sqrt(v) and the quotient of the update.
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ double root(double v) { return sqrt(v); }
// 1 / x for x in the normal range (x >= eps).
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float quotient(float a, float b) { return a * inverse(b); }
__device__ __forceinline__ double quotient(double a, double b) { return a / b; }

// ------------------------------------------------------------------- the step

template <class C>
struct Coef {
  C step, decay, b1, omb1, b2, omb2, eps, isb2, clip;
};

// What one warp holds of a block of 256 elements before the arithmetic: lane l
// the elements 8 l .. 8 l + 7, as loaded.
template <class WT, class GT, class ST>
struct Loaded {
  Raw<GT> g;
  Raw<WT> p;
  Raw<ST> m, v;
};

// Pointers of a unit of work, by type.
template <class PT, class GT, class C, bool MASTER, bool S8>
struct Unit {
  using ST = typename std::conditional<S8, E4m3, C>::type;
  using WT = typename std::conditional<MASTER, float, PT>::type;
  const GT* g;
  WT* w;   // the weights that the step updates
  PT* p;   // their rounded copy (MASTER)
  ST *m, *v;
  float *m_scale, *v_scale;
};

// The arithmetic of eight elements; m and v leave as the values to store.
template <class C>
__device__ __forceinline__ void step_eight(C (&p)[8], const C (&q)[8], C (&m)[8], C (&v)[8], const Coef<C>& k) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const C g = q[j] * k.clip;
    m[j] = k.b1 * m[j] + k.omb1 * g;
    v[j] = k.b2 * v[j] + k.omb2 * (g * g);
    p[j] -= k.decay * p[j];
    p[j] -= quotient(k.step * m[j], root(v[j]) * k.isb2 + k.eps);
  }
}

// The same with 8-bit states: m and v come and leave as e4m3 values, the scales
// as the old and the new ones.  WIDE: which elements the lane holds.
// Each operation that m and r go through is rounded by itself (no fused
// multiply-add), so that the codes follow from plain fp32 arithmetic.
template <bool WIDE>
__device__ __forceinline__ void step_eight8(float (&pf)[8], const float (&qf)[8], float (&mf)[8], float (&vf)[8],
                                            float* ms, float* vs, const Coef<float>& k, uint32_t key, int lane) {
  float2 m[4], v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 g = mul2(make_float2(qf[2 * j], qf[2 * j + 1]), both(k.clip));
    const float2 r0 = mul2(make_float2(vf[2 * j], vf[2 * j + 1]), both(*vs));
    m[j] = apart(mul2(mul2(make_float2(mf[2 * j], mf[2 * j + 1]), both(*ms)), both(k.b1)), mul2(g, both(k.omb1)));
    const float2 v1 = apart(mul2(mul2(r0, r0), both(k.b2)), mul2(mul2(g, g), both(k.omb2)));
    v[j] = make_float2(__fsqrt_rn(v1.x), __fsqrt_rn(v1.y));
    float2 p = make_float2(pf[2 * j], pf[2 * j + 1]);
    p = fma2(both(-k.decay), p, p);
    const float2 den = fma2(v[j], both(k.isb2), both(k.eps));
    p = fma2(mul2(m[j], both(-k.step)), make_float2(inverse(den.x), inverse(den.y)), p);
    pf[2 * j] = p.x, pf[2 * j + 1] = p.y;
  }
  const uint32_t top1 = block_max(m), top2 = block_max(v);
  float least = v[0].x;
#pragma unroll
  for (int j = 0; j < 4; ++j) least = fminf(least, fminf(v[j].x, v[j].y));
  // half of the warp inverts one scale, half the other
  const float base = __uint_as_float(max(lane < 16 ? top1 : top2, __float_as_uint(kOptFloor)));
  const float inv = __fmul_rn(__frcp_rn(base), kE4m3Max), scale = block_scale(lane < 16 ? top1 : top2, base);
  *ms = __shfl_sync(0xffffffffu, scale, 0);
  *vs = __shfl_sync(0xffffffffu, scale, 16);
  const float2 inv1 = both(__shfl_sync(0xffffffffu, inv, 0)), inv2 = both(__shfl_sync(0xffffffffu, inv, 16));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      y[i] = mix_most(key + (uint32_t)(WIDE ? 8 * lane + 2 * j + i : lane + 32 * (2 * j + i)) * 0x9e3779b9u);
    const float2 a = round_first(m[j], inv1, y), b = round_second(v[j], inv2, y);
    mf[2 * j] = a.x, mf[2 * j + 1] = a.y;
    vf[2 * j] = b.x, vf[2 * j + 1] = b.y;
  }
  // Where g^2 underflows (|g| < 8.4e-22 with beta2 = 0.999) r is 0, and no m is
  // kept there: at the random number 0 the smallest m rounds up to a code, which
  // the next step would divide by eps alone.  (1.2 % of the time at 128M elements;
  // as a factor of 0 or 1 an element 2.2 %.)
  if (least == 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (vf[j] == 0.f) mf[j] = 0.f;
  }
}

template <class C, bool S8, bool WIDE>
__device__ __forceinline__ void step_any(C (&p)[8], const C (&q)[8], C (&m)[8], C (&v)[8], float* ms, float* vs,
                                         const Coef<C>& k, uint32_t key, int lane) {
  if constexpr (S8) step_eight8<WIDE>(p, q, m, v, ms, vs, k, key, lane);
  else step_eight(p, q, m, v, k);
}

// A warp's landing buffer for one block with 8-bit states, filled by 16-byte
// asynchronous copies in the order of memory (a lane's own 32 bytes in two
// copies would fetch every sector twice: 15 % more time at 128M elements).  The
// loads ahead then cost no registers; held in registers, as the full states'
// kernel holds them, they take 3 % more time and spill.
template <class WT, class GT>
struct Landing {
  uint4 g[sizeof(GT) / 2 * 32];
  uint4 p[sizeof(WT) / 2 * 32];
  uint2 m[32], v[32];
};

__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t t = (uint32_t)__cvta_generic_to_shared(to);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(t), "l"(from) : "memory");
}

__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All copies but those after the last copies_issued() but one.
__device__ __forceinline__ void copies_landed_but_last() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <class U, class B>
__device__ __forceinline__ void land(const U& u, int base, int lane, B* to) {
  constexpr int NG = sizeof(to->g) / 512, NP = sizeof(to->p) / 512;
#pragma unroll
  for (int i = 0; i < NG; ++i) copy_async(&to->g[32 * i + lane], reinterpret_cast<const uint4*>(u.g + base) + 32 * i + lane);
#pragma unroll
  for (int i = 0; i < NP; ++i) copy_async(&to->p[32 * i + lane], reinterpret_cast<const uint4*>(u.w + base) + 32 * i + lane);
  copy_async(lane < 16 ? &to->m[2 * lane] : &to->v[2 * (lane - 16)], (lane < 16 ? u.m : u.v) + base + 16 * (lane & 15));
}

template <class T>
__device__ __forceinline__ Raw<T> landed(const uint4* x, int lane) {
  Raw<T> r;
  constexpr int N = sizeof(T) / 2;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint4 w = x[N * lane + i];
    r.w[4 * i] = w.x, r.w[4 * i + 1] = w.y, r.w[4 * i + 2] = w.z, r.w[4 * i + 3] = w.w;
  }
  return r;
}
template <class T>
__device__ __forceinline__ Raw<T> landed(const uint2 (&x)[32], int lane) {
  Raw<T> r;
  const uint2 w = x[lane];
  r.w[0] = w.x, r.w[1] = w.y;
  return r;
}

template <class U, class L>
__device__ __forceinline__ void load_wide(const U& u, int e, L* r) {
  r->g = ld8(u.g + e);
  r->p = ld8(u.w + e);
  r->m = ld8(u.m + e);
  r->v = ld8(u.v + e);
}

// The elements of a block that is not whole or not aligned: lane l takes l, l +
// 32, ... of its first n.
template <class T, class C>
__device__ __forceinline__ void load_ragged(const T* x, int n, int lane, C (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = lane + 32 * j < n ? up<C>(x[lane + 32 * j]) : C(0);
}
template <class T, class C>
__device__ __forceinline__ void store_ragged(T* x, int n, int lane, const C (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (lane + 32 * j < n) x[lane + 32 * j] = down<T>(y[j]);
}

template <class PT, class GT, class C, bool MASTER, bool S8>
__device__ __forceinline__ void step_ragged(const Unit<PT, GT, C, MASTER, S8>& u, int base, int n, int lane,
                                            const Coef<C>& k, uint32_t key) {
  C p[8], q[8], m[8], v[8];
  float ms = 0.f, vs = 0.f;
  if (S8) ms = u.m_scale[base / kOptBlock], vs = u.v_scale[base / kOptBlock];
  load_ragged(u.g + base, n, lane, q);
  load_ragged(u.w + base, n, lane, p);
  load_ragged(u.m + base, n, lane, m);
  load_ragged(u.v + base, n, lane, v);
  step_any<C, S8, false>(p, q, m, v, &ms, &vs, k, key, lane);
  store_ragged(u.w + base, n, lane, p);
  if (MASTER) store_ragged(u.p + base, n, lane, p);
  store_ragged(u.m + base, n, lane, m);
  store_ragged(u.v + base, n, lane, v);
  if (S8 && lane == 0) u.m_scale[base / kOptBlock] = ms, u.v_scale[base / kOptBlock] = vs;
}

// Random key of a step.
__device__ __forceinline__ uint32_t step_key(unsigned long long seed, long long t) {
  uint32_t key = mix(mix((uint32_t)seed) ^ (uint32_t)(seed >> 32));
  return mix(mix(key ^ (uint32_t)t) ^ (uint32_t)((unsigned long long)t >> 32));
}

// The counter, and the factors and key of the step after it.  1 - beta^t as
// -expm1(t log beta): within a few roundings for every t, where 1 - beta^t
// loses 1 / (1 - beta) of them to the difference.
__device__ __forceinline__ void set_counter(OptCtrl* c, long long t, double log_b1, double log_b2,
                                            unsigned long long seed) {
  const double next = (double)(t + 1);
  c->t = t;
  c->inv_bc1 = 1.0 / -expm1(next * log_b1);
  c->inv_sbc2 = 1.0 / sqrt(-expm1(next * log_b2));
  c->inv_bc1_f = (float)c->inv_bc1;
  c->inv_sbc2_f = (float)c->inv_sbc2;
  c->key = step_key(seed, t + 1);
}

template <class C>
__device__ __forceinline__ C pick(double d, float f) {
  return sizeof(C) == 8 ? (C)d : (C)f;
}

// The pointers of a unit of work (the scales' are the unit's in global memory).
template <class U, class PT, class GT>
__device__ __forceinline__ U unit_of(const OptChunk& c, const GT* g, bool master) {
  U u;
  u.g = g + c.first;
  u.w = static_cast<typename U::WT*>(master ? c.master : c.p);
  u.p = static_cast<PT*>(c.p);
  u.m = static_cast<typename U::ST*>(c.m);
  u.v = static_cast<typename U::ST*>(c.v);
  u.m_scale = c.m_scale;
  u.v_scale = c.v_scale;
  return u;
}

// The factors of a step for a tensor; clip is set by the caller.
template <class C>
__device__ __forceinline__ Coef<C> coef_of(const OptStepArgs<C>& a, const OptCtrl* ctrl, const OptChunk& c) {
  Coef<C> k;
  const C lr = (a.lr_dev ? *a.lr_dev : a.lr) * pick<C>(c.lr_scale, c.lr_scale_f);
  k.step = lr * pick<C>(ctrl->inv_bc1, ctrl->inv_bc1_f);
  k.decay = lr * pick<C>(c.decay, c.decay_f);
  k.b1 = a.b1, k.omb1 = a.omb1, k.b2 = a.b2, k.omb2 = a.omb2, k.eps = a.eps;
  k.isb2 = pick<C>(ctrl->inv_sbc2, ctrl->inv_sbc2_f);
  k.clip = a.grad_scale;
  return k;
}

// Wide accesses, else element by element (32M fp32 elements: full states 138
// against 179 us, 8-bit 88 against 120).
template <class GT>
__device__ __forceinline__ bool takes_wide(const OptChunk& c, const GT* g) {
  constexpr unsigned long long kGradAlign = 8 * sizeof(GT) < 32 ? 8 * sizeof(GT) : 32;
  return c.aligned && (unsigned long long)g % kGradAlign == 0;
}

// The general step: a block a unit of work, a warp a block of 256 elements a
// round.  Full states are bound by memory (128M fp32 elements, 28 bytes each:
// 526 us, 6.8 TB/s, above the rate of a plain copy).  8-bit states are bound by
// the instructions they issue, some 72 an element of which the rounding takes
// 26, its random bits 9 and the exactly rounded root 10 (128M: 385 us, 5.3 TB/s;
// 315 us without these three).  Three blocks an SM: 80 registers.  fp64 takes 178
// registers, one block an SM, and waits for memory (48M elements 442 us, 6.1 TB/s).
template <class PT, class GT, class C, bool MASTER, bool S8, int CAP>
__global__ void __launch_bounds__(kThreadsOpt, sizeof(C) == 4 ? 3 : 1)
    adamw_kernel(const __grid_constant__ OptStepArgs<C> a, const __grid_constant__ GradPtrs<CAP> gp) {
  using U = Unit<PT, GT, C, MASTER, S8>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the table does not change: a record is read before the previous kernel ends
  const bool some = (int)blockIdx.x < a.n_chunks;
  const OptChunk c = some ? a.chunks[blockIdx.x] : OptChunk{};
  after_previous();
  if (some && !(a.clipped && a.ctrl->skip)) {
    const GT* g = static_cast<const GT*>(gp.p[c.slot - a.slot0]);
    if (g) {
      U u = unit_of<U, PT>(c, g, MASTER);
      const int count = c.count, blocks = (count + kOptBlock - 1) / kOptBlock;
      __shared__ float scales[2][kOptMaxRounds * (kOptChunk / kOptBlock)];
      if (S8) {
        // the unit's scales in one piece: written by each warp for itself they
        // are partial writes of a sector (a third more time at 128M elements)
        u.m_scale = scales[0], u.v_scale = scales[1];
        for (int i = threadIdx.x; i < blocks; i += kThreadsOpt)
          scales[0][i] = c.m_scale[i], scales[1][i] = c.v_scale[i];
        __syncthreads();
      }
      const uint32_t block0 = (uint32_t)(c.first / kOptBlock);
      Coef<C> k = coef_of(a, a.ctrl, c);
      if (a.clipped) k.clip = pick<C>(a.ctrl->clip, a.ctrl->clip_f);
      const uint32_t key = S8 ? mix(a.ctrl->key ^ c.tensor) : 0u;
      const int whole = takes_wide(c, u.g) ? count / kOptBlock * kOptBlock : 0;
      int base = warp * kOptBlock;
      if constexpr (S8) {
        __shared__ Landing<typename U::WT, GT> pool[kThreadsOpt / 32][2];
        if (base < whole) land(u, base, lane, &pool[warp][0]);
        copies_issued();
        for (int i = 0; base < whole; base += kOptChunk, i ^= 1) {
          // the next round's copies are in flight during this one's arithmetic
          __syncwarp();  // every lane has read the buffer that they fill
          if (base + kOptChunk < whole) land(u, base + kOptChunk, lane, &pool[warp][i ^ 1]);
          copies_issued();
          copies_landed_but_last();
          __syncwarp();
          const auto& now = pool[warp][i];
          C p[8], q[8], m[8], v[8];
          float ms = u.m_scale[base / kOptBlock], vs = u.v_scale[base / kOptBlock];
          unpack(landed<GT>(now.g, lane), q);
          unpack(landed<typename U::WT>(now.p, lane), p);
          unpack(landed<E4m3>(now.m, lane), m);
          unpack(landed<E4m3>(now.v, lane), v);
          step_eight8<true>(p, q, m, v, &ms, &vs, k, mix(key ^ (block0 + base / kOptBlock)), lane);
          const int e = base + 8 * lane;
          st8(u.w + e, p);
          if (MASTER) st8(u.p + e, p);
          st8(u.m + e, m);
          st8(u.v + e, v);
          if (lane == 0) u.m_scale[base / kOptBlock] = ms, u.v_scale[base / kOptBlock] = vs;
        }
      } else if (base < whole) {
        Loaded<typename U::WT, GT, typename U::ST> now;
        load_wide(u, base + 8 * lane, &now);
        while (true) {
          // the next round's loads are in flight during this one's arithmetic
          const int next = base + kOptChunk;
          auto ahead = now;
          if (next < whole) load_wide(u, next + 8 * lane, &ahead);
          C p[8], q[8], m[8], v[8];
          unpack(now.g, q);
          unpack(now.p, p);
          unpack(now.m, m);
          unpack(now.v, v);
          step_eight(p, q, m, v, k);
          const int e = base + 8 * lane;
          st8(u.w + e, p);
          if (MASTER) st8(u.p + e, p);
          st8(u.m + e, m);
          st8(u.v + e, v);
          base = next;
          if (next >= whole) break;
          now = ahead;
        }
      }
      for (; base < count; base += kOptChunk)
        step_ragged<PT, GT, C, MASTER, S8>(u, base, min(count - base, kOptBlock), lane, k,
                                           S8 ? mix(key ^ (block0 + base / kOptBlock)) : 0u);
      if (S8) {
        __syncthreads();
        for (int i = threadIdx.x; i < blocks; i += kThreadsOpt)
          c.m_scale[i] = scales[0][i], c.v_scale[i] = scales[1][i];
      }
    }
  }
  // The last block to finish advances the counter; every block has read it by then.
  if (a.last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(&a.ctrl->ticket_step, 1u) == gridDim.x - 1) {
        a.ctrl->ticket_step = 0;
        if (!(a.clipped && a.ctrl->skip)) set_counter(a.ctrl, a.ctrl->t + 1, a.log_b1, a.log_b2, a.seed);
      }
    }
  }
}

// ------------------------------------------------------------- small handles

// The clipping factor of a norm, and whether the step is taken.
__device__ __forceinline__ double clip_factor(double norm, double max_norm, double grad_scale) {
  return norm > max_norm ? grad_scale * (max_norm / norm) : grad_scale;
}

// The whole step of a handle with few blocks in one launch of one cluster: a
// warp a block of 256 elements, which it holds in registers from the norm to
// the update.  The thread blocks exchange their sums of squares through
// distributed shared memory; the cluster's barrier stands in for the two
// launches and the ticket of the general kernels.  Latency is all that counts
// here (figures at kSmallBlocks in optim_api.cu).
template <class PT, class GT, class C, bool MASTER, bool S8, int CAP>
__global__ void __launch_bounds__(kOptSmallWarps * 32)
    adamw_small_kernel(const __grid_constant__ OptStepArgs<C> a, const __grid_constant__ OptClipArgs clip,
                       const __grid_constant__ GradPtrs<CAP> gp) {
  namespace cg = cooperative_groups;
  using U = Unit<PT, GT, C, MASTER, S8>;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double warp_sums[kOptSmallWarps];
  __shared__ double block_sums[kOptSmallCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * (blockDim.x >> 5) + warp;
  // (a block writes into the others' shared memory only once all of them run)
  cg::cluster_group::arrival_token all_run;
  if (a.clipped) all_run = cluster.barrier_arrive();
  // the table does not change: a record is read before the previous kernel ends
  const OptChunk c = i < a.n_chunks ? a.chunks[i] : OptChunk{};
  after_previous();
  const GT* g = i < a.n_chunks ? static_cast<const GT*>(gp.p[c.slot]) : nullptr;
  const OptCtrl now = *a.ctrl;
  U u;
  Coef<C> k;
  bool wide = false;
  C p[8], q[8], m[8], v[8];
  float ms = 0.f, vs = 0.f;
  if (g) {
    u = unit_of<U, PT>(c, g, MASTER);
    k = coef_of(a, &now, c);
    wide = c.count == kOptBlock && takes_wide(c, u.g);
    if (S8) ms = *u.m_scale, vs = *u.v_scale;
    if (wide) {
      Loaded<typename U::WT, GT, typename U::ST> r;
      load_wide(u, 8 * lane, &r);
      unpack(r.g, q);
      unpack(r.p, p);
      unpack(r.m, m);
      unpack(r.v, v);
    } else {
      load_ragged(u.g, c.count, lane, q);
      load_ragged(u.w, c.count, lane, p);
      load_ragged(u.m, c.count, lane, m);
      load_ragged(u.v, c.count, lane, v);
    }
  }
  bool taken = true;
  if (a.clipped) {
    double s = 0.0;
    if (g) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)q[j], (double)q[j], s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) warp_sums[warp] = s;
    __syncthreads();
    cluster.barrier_wait(std::move(all_run));
    if (threadIdx.x < cluster.num_blocks()) {  // this block's sum into every block's list
      s = 0.0;
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += warp_sums[w];
      cluster.map_shared_rank(block_sums, threadIdx.x)[cluster.block_rank()] = s;
    }
    cluster.sync();
    s = 0.0;
    for (int b = 0; b < (int)cluster.num_blocks(); ++b) s += block_sums[b];
    const double norm = sqrt(s) * fabs(clip.grad_scale);
    taken = norm - norm == 0.0;
    k.clip = (C)clip_factor(norm, clip.max_norm, clip.grad_scale);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      if (clip.norm && clip.norm64) *static_cast<double*>(clip.norm) = norm;
      else if (clip.norm) *static_cast<float*>(clip.norm) = (float)norm;
      if (!taken) a.ctrl->status |= 1u << QML_ERR_NUMERIC;
    }
  } else {
    cluster.sync();  // every block has read the counter's state
  }
  if (taken && blockIdx.x == 0 && threadIdx.x == blockDim.x - 1)
    set_counter(a.ctrl, now.t + 1, a.log_b1, a.log_b2, a.seed);
  if (!g || !taken) return;
  const uint32_t key = S8 ? mix(mix(now.key ^ c.tensor) ^ (uint32_t)(c.first / kOptBlock)) : 0u;
  if (wide) {
    step_any<C, S8, true>(p, q, m, v, &ms, &vs, k, key, lane);
    st8(u.w + 8 * lane, p);
    if (MASTER) st8(u.p + 8 * lane, p);
    st8(u.m + 8 * lane, m);
    st8(u.v + 8 * lane, v);
  } else {
    step_any<C, S8, false>(p, q, m, v, &ms, &vs, k, key, lane);
    store_ragged(u.w, c.count, lane, p);
    if (MASTER) store_ragged(u.p, c.count, lane, p);
    store_ragged(u.m, c.count, lane, m);
    store_ragged(u.v, c.count, lane, v);
  }
  if (S8 && lane == 0) *u.m_scale = ms, *u.v_scale = vs;
}

// ------------------------------------------------------------------- the norm

__device__ __forceinline__ double block_sum(double x, double* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreadsOpt / 32; ++w) s += part[w];
  return s;  // thread 0's
}

// Sum of the squares of eight gradients in fp64.  Converting every one to fp64
// would bound the kernel (some 6 conversions a clock and SM: 100M bf16 in 47 us,
// of which 31 are the memory's), so two fp32 (four bf16 / fp16, whose squares
// are exact) are summed in fp32 first: 2 roundings, so the norm is off by one
// part in 2^24 at most.  Where the largest of the eight is outside 2^-55 ..
// 2^60, a square could overflow or lose bits to underflow: all eight in fp64.
template <class GT>
__device__ __forceinline__ double eight_squares(const Raw<GT>& r) {
  if constexpr (sizeof(GT) == 8) {
    double x[8], s = 0.0;
    unpack(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma(x[j], x[j], s);
    return s;
  } else {
    float x[8], top = 0.f;
    unpack(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
    if ((top >= 0x1p-55f && top < 0x1p60f) || top == 0.f) {  // (a NaN among them makes the sum NaN)
      float2 s[2];  // two pairs each
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = make_float2(x[4 * j], x[4 * j + 1]), b = make_float2(x[4 * j + 2], x[4 * j + 3]);
        s[j] = fma2(b, b, mul2(a, a));
      }
      if (sizeof(GT) == 2) return (double)(s[0].x + s[0].y) + (double)(s[1].x + s[1].y);
      return ((double)s[0].x + (double)s[0].y) + ((double)s[1].x + (double)s[1].y);
    }
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma((double)x[j], (double)x[j], s);
    return s;
  }
}

// Sum of squares of a unit's gradients (this thread's part): four wide loads a
// thread in flight.
template <class GT>
__device__ __forceinline__ double chunk_squares(const GT* g, int count) {
  constexpr int kFlight = 4;
  double s[kFlight] = {};
  constexpr unsigned long long kGradAlign = 8 * sizeof(GT) < 32 ? 8 * sizeof(GT) : 32;
  const int whole = (unsigned long long)g % kGradAlign == 0 ? count / 8 * 8 : 0;
  for (int e0 = threadIdx.x * 8; e0 < whole; e0 += kFlight * kOptChunk) {
    Raw<GT> r[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (e0 + i * kOptChunk < whole) {
        r[i] = ld8(g + e0 + i * kOptChunk);
      } else {
#pragma unroll
        for (uint32_t& w : r[i].w) w = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) s[i] += eight_squares(r[i]);
  }
  for (int i = whole + threadIdx.x; i < count; i += kThreadsOpt) {
    const double x = up<double>(g[i]);
    s[0] = fma(x, x, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum of squares in a fixed order: per thread over the block's chunks (eight at
// a time, see eight_squares(); element by element in fp64, where an fp32
// gradient's square neither overflows nor underflows, if the wide loads cannot
// take them), the block, then all blocks' partials by the block that finishes last.
template <int CAP>
__global__ void __launch_bounds__(kThreadsOpt)
    grad_norm_kernel(const __grid_constant__ OptNormArgs a, const __grid_constant__ GradPtrs<CAP> gp) {
  __shared__ double part[kThreadsOpt / 32];
  __shared__ int is_last;
  double s = 0.0;
  after_previous();
  let_next_start();  // the step's blocks, as these exit; they wait for this kernel's results themselves
  for (int i = blockIdx.x; i < a.n_chunks; i += gridDim.x) {
    const OptChunk* c = a.chunks + i;
    const void* g = gp.p[c->slot - a.slot0];
    if (!g) continue;
    if (a.grad_type == OPT_F32) s += chunk_squares(static_cast<const float*>(g) + c->first, c->count);
    else if (a.grad_type == OPT_BF16) s += chunk_squares(static_cast<const __nv_bfloat16*>(g) + c->first, c->count);
    else if (a.grad_type == OPT_F16) s += chunk_squares(static_cast<const __half*>(g) + c->first, c->count);
    else s += chunk_squares(static_cast<const double*>(g) + c->first, c->count);
  }
  s = block_sum(s, part);
  if (threadIdx.x == 0) {
    a.partials[a.part0 + blockIdx.x] = s;
    is_last = 0;
    if (a.last) {
      __threadfence();
      is_last = atomicAdd(&a.ctrl->ticket_norm, 1u) == gridDim.x - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!is_last) return;
  s = 0.0;
  for (int i = threadIdx.x; i < a.n_part; i += kThreadsOpt) s += __ldcg(a.partials + i);
  s = block_sum(s, part);
  if (threadIdx.x == 0) {
    a.ctrl->ticket_norm = 0;
    const double norm = sqrt(s) * fabs(a.grad_scale);
    const bool finite = norm - norm == 0.0;
    if (a.norm && a.norm64) *static_cast<double*>(a.norm) = norm;
    else if (a.norm) *static_cast<float*>(a.norm) = (float)norm;
    if (a.set_clip) {
      a.ctrl->clip = clip_factor(norm, a.max_norm, a.grad_scale);
      a.ctrl->clip_f = (float)a.ctrl->clip;
      a.ctrl->skip = finite ? 0 : 1;
      if (!finite) a.ctrl->status |= 1u << QML_ERR_NUMERIC;
    }
  }
}

__global__ void opt_set_kernel(OptCtrl* c, long long t, double log_b1, double log_b2, unsigned long long seed) {
  after_previous();
  set_counter(c, t, log_b1, log_b2, seed);
}

// Kernel parameters of the smallest size that holds the gradient pointers.
template <class F>
cudaError_t with_ptrs(const void* const* grads, int n, F&& f) {
  auto fill = [&](auto& gp) {
    for (int i = 0; i < n; ++i) gp.p[i] = grads[i];
    return f(gp);
  };
  if (n <= kOptCaps[0]) {
    GradPtrs<kOptCaps[0]> gp;
    return fill(gp);
  }
  if (n > kOptCaps[1]) return cudaErrorInvalidValue;
  static thread_local GradPtrs<kOptCaps[1]> gp;
  return fill(gp);
}

template <class P, class G, bool M>
struct Types {
  using Param = P;
  using Grad = G;
  static constexpr bool master = M;
};

// f(Types) for a combination of types.
template <class F>
cudaError_t for_combo(const OptCombo& c, F&& f) {
  using bf16 = __nv_bfloat16;
  const bool same = c.param == c.grad;
  switch (c.param) {
    case OPT_F32: return f(Types<float, float, false>{});
    case OPT_F64: return f(Types<double, double, false>{});
    case OPT_BF16:
      if (c.master) return same ? f(Types<bf16, bf16, true>{}) : f(Types<bf16, float, true>{});
      return same ? f(Types<bf16, bf16, false>{}) : f(Types<bf16, float, false>{});
    case OPT_F16:
      if (c.master) return same ? f(Types<__half, __half, true>{}) : f(Types<__half, float, true>{});
      return same ? f(Types<__half, __half, false>{}) : f(Types<__half, float, false>{});
  }
  return cudaErrorInvalidValue;
}

template <class PT, class GT, bool MASTER>
cudaError_t step_combo(bool bits8, const OptSettings& t, const OptClipArgs* small, const void* const* grads, int n,
                       cudaStream_t s) {
  using C = typename std::conditional<sizeof(PT) == 8, double, float>::type;
  OptStepArgs<C> a{};
  a.chunks = t.chunks;
  a.ctrl = t.ctrl;
  a.n_chunks = t.n_chunks;
  a.slot0 = t.slot0;
  a.lr = (C)t.lr;
  a.b1 = (C)t.beta1, a.omb1 = (C)(1.0 - t.beta1);
  a.b2 = (C)t.beta2, a.omb2 = (C)(1.0 - t.beta2);
  a.eps = (C)t.eps;
  a.grad_scale = (C)t.grad_scale;
  a.lr_dev = static_cast<const C*>(t.lr_dev);
  a.log_b1 = std::log(t.beta1);  // beta = 0: -infinity, a correction of 1
  a.log_b2 = std::log(t.beta2);
  a.seed = t.seed;
  a.clipped = t.clipped;
  a.last = t.last;
  const int grid = a.n_chunks > 0 ? a.n_chunks : 1;
  return with_ptrs(grads, n, [&](auto& gp) {
    constexpr int CAP = sizeof(gp.p) / sizeof(gp.p[0]);
    if constexpr (CAP == kOptCaps[0]) {
      if (small) {
        // as many thread blocks as the cluster takes, the warps spread evenly
        const int blocks = std::min(grid, small->cluster), warps = (grid + blocks - 1) / blocks;
        if constexpr (sizeof(PT) < 8) {
          if (bits8) {
            return launch_after(adamw_small_kernel<PT, GT, C, MASTER, true, CAP>, blocks, warps * 32, blocks, s, a, *small,
                                gp);
          }
        }
        return launch_after(adamw_small_kernel<PT, GT, C, MASTER, false, CAP>, blocks, warps * 32, blocks, s, a, *small,
                            gp);
      }
    }
    if constexpr (sizeof(PT) < 8) {
      if (bits8) {
        return launch_after(adamw_kernel<PT, GT, C, MASTER, true, CAP>, grid, kThreadsOpt, 1, s, a, gp);
      }
    }
    return launch_after(adamw_kernel<PT, GT, C, MASTER, false, CAP>, grid, kThreadsOpt, 1, s, a, gp);
  });
}

}  // namespace

cudaError_t launch_opt_step(const OptCombo& c, const OptSettings& a, const OptClipArgs* small,
                            const void* const* grads, int n, cudaStream_t s) {
  return for_combo(c, [&](auto types) {
    using T = decltype(types);
    return step_combo<typename T::Param, typename T::Grad, T::master>(c.bits8, a, small, grads, n, s);
  });
}

int opt_cluster_limit(const OptCombo& c) {
  int limit = 8;
  for_combo(c, [&](auto types) {
    using T = decltype(types);
    using P = typename T::Param;
    auto probe = [&](auto kernel) {
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = kOptSmallCluster, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(kOptSmallCluster);
      cfg.blockDim = dim3(kOptSmallWarps * 32);
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
          cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0)
        limit = kOptSmallCluster;
      else
        cudaGetLastError();
    };
    if constexpr (sizeof(P) == 8) {
      probe(adamw_small_kernel<P, typename T::Grad, double, false, false, kOptCaps[0]>);
    } else {
      if (c.bits8) probe(adamw_small_kernel<P, typename T::Grad, float, T::master, true, kOptCaps[0]>);
      else probe(adamw_small_kernel<P, typename T::Grad, float, T::master, false, kOptCaps[0]>);
    }
    return cudaSuccess;
  });
  return limit;
}

cudaError_t launch_opt_norm(const OptNormArgs& a, const void* const* grads, int n, int grid, cudaStream_t s) {
  return with_ptrs(grads, n, [&](auto& gp) {
    constexpr int CAP = sizeof(gp.p) / sizeof(gp.p[0]);
    return launch_after(grad_norm_kernel<CAP>, grid, kThreadsOpt, 1, s, a, gp);
  });
}

cudaError_t launch_opt_set(OptCtrl* ctrl, long long t, double beta1, double beta2, unsigned long long seed,
                           cudaStream_t s) {
  return launch_after(opt_set_kernel, 1, 1, 1, s, ctrl, t, std::log(beta1), std::log(beta2), seed);
}

}  // namespace qml
