// ckpt8.cu -- checkpoint slots in 8 bits (QML_STORE_INT8).
//
// A slot keeps a state as int8 codes, every block of 16 consecutive amplitudes
// (32 real numbers; the whole state of fewer qubits) sharing a power of two:
//   k = floor(log2 max|x|) - 6 (at least -127),  code = clamp(rint(x 2^-k), -127, 127),  x' = code 2^k
// The scale is a power of two, so 2^-k x and code 2^k are exact and the only
// rounding is rint's: half a step 2^k, a step where max|x| lies within half a
// step of 2^(k+7) and its code is held at 127.  The exponent is stored as the
// byte k + 127; 255 marks a block with a NaN or infinity, which reads back as
// NaN.  2 1/16 bytes an amplitude, against 8 (fp32) and 4 (bf16).
//
// Blocks follow the working-state order (plan.hpp, addr_of: the index order up
// to 20 qubits), so that the passes' slots are written from and restored to the
// working state in runs.
#include <cstdint>

#include "kernels.cuh"
#include "launch.cuh"

namespace qml {

namespace {

constexpr int kBlockAmps = 16;
constexpr int kThreads8 = 256;

// Bit b of a working-state address is bit to[b] of the standard index (cb
// lowest bits; the others are the same).
struct BitMap {
  int cb;
  int to[kTileBits];
};

__device__ __forceinline__ long long std_index(const BitMap& m, long long a) {
  long long i = a & ~((1ll << m.cb) - 1);
  for (int b = 0; b < m.cb; ++b) i |= ((a >> b) & 1) << m.to[b];
  return i;
}

// Exponent byte of a block from the largest |x| in it (as the bits of a float).
__device__ __forceinline__ uint32_t exponent_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : e < 6u ? 0u : e - 6u;
}

// 2^-k and 2^k of an exponent byte.
__device__ __forceinline__ float inverse_scale(uint32_t e) { return e == 255u ? 0.f : __uint_as_float((254u - e) << 23); }
__device__ __forceinline__ float scale_of(uint32_t e) {
  if (e == 255u) return __uint_as_float(0x7fffffffu);
  return e ? __uint_as_float(e << 23) : __uint_as_float(0x00400000u);  // 2^-127 is a subnormal number
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ int code_of(float x, float inv) {
  return __float2int_rn(fminf(fmaxf(x * inv, -127.f), 127.f));  // (NaN * 0: some code, unused)
}

// Eight values as eight bytes.
__device__ __forceinline__ uint2 pack8(const float (&x)[8], float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j / 4] |= (uint32_t)(code_of(x[j], inv) & 255) << (8 * (j % 4));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8(uint2 w, float s, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j % 4))) * s;
}

// Largest of a block: four neighbouring lanes hold 8 of its 32 values each.
__device__ __forceinline__ uint32_t quad_max(const float (&x)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = max(t, abs_bits(x[j]));
  t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
  return max(t, __shfl_xor_sync(0xffffffffu, t, 2));
}

// A warp's share of a state of 2^n >= 16 amplitudes: kRuns runs of 128
// amplitudes, four a lane.  All runs' loads are in flight together, and the 32
// exponent bytes go out as one sector.  Bound by memory: a save and a restore of
// 85 states of 20 qubits take 266 us (6.7 TB/s); with one run a warp, 16-byte
// accesses and the exponents a byte at a time (partial writes of sectors), 309.
constexpr int kRuns = 4;
constexpr int kWarpAmps = 128 * kRuns;

__device__ __forceinline__ long long warp_first() {
  return ((long long)blockIdx.x * (kThreads8 / 32) + (threadIdx.x >> 5)) * kWarpAmps;
}

// Lane l's exponent byte for the warp's store: of block l % 8 of run l / 8,
// which lane 4 (l % 8) holds.
__device__ __forceinline__ uint32_t gather_exponent(const uint32_t (&e)[kRuns], int lane) {
  uint32_t mine = 0;
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const uint32_t x = __shfl_sync(0xffffffffu, e[r], (lane & 7) * 4);
    if (lane >> 3 == r) mine = x;
  }
  return mine;
}
// The reverse: the exponent byte of a lane's block in run r.
__device__ __forceinline__ uint32_t spread_exponent(uint32_t mine, int r, int lane) {
  return __shfl_sync(0xffffffffu, mine, r * 8 + (lane >> 2));
}

__device__ __forceinline__ void ld8f(const float* p, float (&x)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}
__device__ __forceinline__ void st8f(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "l"(p)
               : "memory");
}

// Whether four amplitudes from a multiple of 4 are one aligned piece of the
// state: it starts on 32 bytes and its order keeps the two lowest bits (plans of
// three or more qubit sets do).  20 qubits x 32: save 50, restore 53 us; from
// and to a state that is off by 8 bytes 50 and 113; 21 qubits x 16 (same bytes): 67 and
// 63, amplitude by amplitude 168 and 174.
template <bool PERM>
__device__ __forceinline__ bool takes_wide(const float2* psi, const BitMap& map) {
  return ((uintptr_t)psi & 31) == 0 && (!PERM || (map.to[0] == 0 && map.to[1] == 1));
}

// State (standard order) to its slot and back.  count: amplitudes, a multiple of 16.
template <bool PERM>
__global__ void __launch_bounds__(kThreads8)
    slot8_save_kernel(const float2* psi, int8_t* codes, uint8_t* exps, long long count, BitMap map) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long first = warp_first();
  if (first >= count) return;
  const bool wide = takes_wide<PERM>(psi, map);
  float x[kRuns][8];
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const long long a = first + 128 * r + 4 * lane;
    if (a < count && wide) {
      ld8f(reinterpret_cast<const float*>(psi + (PERM ? std_index(map, a) : a)), x[r]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = a < count ? psi[PERM ? std_index(map, a + j) : a + j] : make_float2(0.f, 0.f);
        x[r][2 * j] = v.x, x[r][2 * j + 1] = v.y;
      }
    }
  }
  uint32_t e[kRuns];
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const long long a = first + 128 * r + 4 * lane;
    e[r] = exponent_byte(quad_max(x[r]));
    if (a < count) *reinterpret_cast<uint2*>(codes + 2 * a) = pack8(x[r], inverse_scale(e[r]));
  }
  const uint32_t mine = gather_exponent(e, lane);
  if (first + kBlockAmps * lane < count) exps[first / kBlockAmps + lane] = (uint8_t)mine;
}

template <bool PERM>
__global__ void __launch_bounds__(kThreads8)
    slot8_load_kernel(float2* psi, const int8_t* codes, const uint8_t* exps, long long count, BitMap map) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long first = warp_first();
  if (first >= count) return;
  const bool wide = takes_wide<PERM>(psi, map);
  const uint32_t mine = first + kBlockAmps * lane < count ? exps[first / kBlockAmps + lane] : 0u;
  uint2 w[kRuns];
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const long long a = first + 128 * r + 4 * lane;
    w[r] = a < count ? *reinterpret_cast<const uint2*>(codes + 2 * a) : make_uint2(0u, 0u);
  }
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const long long a = first + 128 * r + 4 * lane;
    float x[8];
    unpack8(w[r], scale_of(spread_exponent(mine, r, lane)), x);
    if (a < count && wide) {
      st8f(reinterpret_cast<float*>(psi + (PERM ? std_index(map, a) : a)), x);
    } else if (a < count) {
#pragma unroll
      for (int j = 0; j < 4; ++j) psi[PERM ? std_index(map, a + j) : a + j] = make_float2(x[2 * j], x[2 * j + 1]);
    }
  }
}

// A slot from the forward pass's working layout: unit u = samples 2u, 2u + 1
// keeps (Re, Re) of the two at sample 2u's positions and (Im, Im) at sample
// 2u + 1's (an odd batch's last unit: in `partner`).  Four addresses of a unit
// a lane; grid.y: units.  Bound by memory with one run a warp: 20 qubits x 32 54
// us, where the save kernel with its four takes 51 (ncu).
__global__ void __launch_bounds__(kThreads8)
    slot8_from_planes_kernel(const float2* buf, const float2* partner, int8_t* codes, uint8_t* exps, int B,
                             long long N) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long a0 = ((long long)blockIdx.x * (kThreads8 / 32) + (threadIdx.x >> 5)) * 128;
  if (a0 >= N) return;
  const long long a = a0 + 4 * lane;
  const bool in = a < N;
  for (int u = blockIdx.y; 2 * u < B; u += gridDim.y) {
    const bool two = 2 * u + 1 < B;
    float x[8] = {}, y[8] = {};
    if (in) {
      const float4* p0 = reinterpret_cast<const float4*>(buf + (size_t)(2 * u) * N + a);
      const float4* p1 = reinterpret_cast<const float4*>(two ? buf + (size_t)(2 * u + 1) * N + a : partner + a);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 re = p0[h], im = p1[h];
        x[4 * h] = re.x, x[4 * h + 1] = im.x, x[4 * h + 2] = re.z, x[4 * h + 3] = im.z;
        y[4 * h] = re.y, y[4 * h + 1] = im.y, y[4 * h + 2] = re.w, y[4 * h + 3] = im.w;
      }
    }
    const uint32_t e0 = exponent_byte(quad_max(x)), e1 = exponent_byte(quad_max(y));
    const uint32_t out0 = __shfl_sync(0xffffffffu, e0, (lane & 7) * 4), out1 = __shfl_sync(0xffffffffu, e1, (lane & 7) * 4);
    const long long o0 = (long long)(2 * u) * N;
    if (lane < 8 && a0 + kBlockAmps * lane < N) {
      exps[(o0 + a0) / kBlockAmps + lane] = (uint8_t)out0;
      if (two) exps[(o0 + N + a0) / kBlockAmps + lane] = (uint8_t)out1;
    }
    if (in) {
      *reinterpret_cast<uint2*>(codes + 2 * (o0 + a)) = pack8(x, inverse_scale(e0));
      if (two) *reinterpret_cast<uint2*>(codes + 2 * (o0 + N + a)) = pack8(y, inverse_scale(e1));
    }
  }
}

// The psi lanes of the backward planes from a slot, times *rscale (null: 1):
// plane0[i].x = Re, plane1[i].x = Im.  The planes are read and written whole, 34
// bytes an amplitude: 20 qubits x 32 185 us (ncu), 6.2 TB/s.
__global__ void __launch_bounds__(kThreads8)
    slot8_to_planes_kernel(float2* plane0, float2* plane1, const int8_t* codes, const uint8_t* exps,
                           const float* rscale, long long count) {
  after_previous();
  const long long a = ((long long)blockIdx.x * kThreads8 + threadIdx.x) * 4;
  if (a >= count) return;
  const float rs = rscale ? __ldg(rscale) : 1.f;
  float x[8];
  unpack8(*reinterpret_cast<const uint2*>(codes + 2 * a), scale_of(exps[a / kBlockAmps]), x);
  float4* p0 = reinterpret_cast<float4*>(plane0 + a);
  float4* p1 = reinterpret_cast<float4*>(plane1 + a);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float4 re = p0[h], im = p1[h];
    re.x = x[4 * h] * rs, im.x = x[4 * h + 1] * rs;
    re.z = x[4 * h + 2] * rs, im.z = x[4 * h + 3] * rs;
    p0[h] = re, p1[h] = im;
  }
}

// States of fewer than 16 amplitudes: a sample is one block, one thread each.
// OP 0: state to slot, 1: slot to state, 2: working layout to slot, 3: slot to
// the backward planes.
template <int OP>
__global__ void slot8_small_kernel(float2* buf0, float2* buf1, int8_t* codes, uint8_t* exps, const float* rscale,
                                   int B, int N) {
  after_previous();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  int8_t* c = codes + (size_t)b * N * 2;
  float2* p0 = buf0 + (size_t)(OP == 2 ? b & ~1 : b) * N;
  float2* p1 = OP == 2 ? ((b | 1) < B ? buf0 + (size_t)(b | 1) * N : buf1) : OP == 3 ? buf1 + (size_t)b * N : nullptr;
  auto value = [&](int i) {
    if (OP == 0) return p0[i];
    return b & 1 ? make_float2(p0[i].y, p1[i].y) : make_float2(p0[i].x, p1[i].x);
  };
  if (OP == 0 || OP == 2) {
    uint32_t top = 0;
    for (int i = 0; i < N; ++i) top = max(top, max(abs_bits(value(i).x), abs_bits(value(i).y)));
    const uint32_t e = exponent_byte(top);
    exps[b] = (uint8_t)e;
    for (int i = 0; i < N; ++i) {
      c[2 * i] = (int8_t)code_of(value(i).x, inverse_scale(e));
      c[2 * i + 1] = (int8_t)code_of(value(i).y, inverse_scale(e));
    }
  } else {
    const float s = scale_of(exps[b]), rs = rscale ? *rscale : 1.f;
    for (int i = 0; i < N; ++i) {
      const float re = (float)c[2 * i] * s, im = (float)c[2 * i + 1] * s;
      if (OP == 1) p0[i] = make_float2(re, im);
      else p0[i].x = re * rs, p1[i].x = im * rs;
    }
  }
}

BitMap bit_map(int cb, const int* to) {
  BitMap m{};
  m.cb = cb;
  for (int b = 0; b < cb; ++b) m.to[b] = to[b];
  return m;
}

unsigned blocks_for(long long count) { return (unsigned)((count / 4 + kThreads8 - 1) / kThreads8); }

}  // namespace

size_t slot8_blocks(int n) { return n >= 4 ? (size_t)1 << (n - 4) : 1; }

cudaError_t launch_slot8_copy(bool save, float2* psi, int8_t* codes, uint8_t* exps, int B, int n, int cb,
                              const int* to, cudaStream_t s) {
  const long long count = (long long)B << n;
  if (n < 4) {
    const unsigned g = (unsigned)((B + 63) / 64);
    if (save) return launch_after(slot8_small_kernel<0>, g, 64, 1, s, psi, nullptr, codes, exps, nullptr, B, 1 << n);
    return launch_after(slot8_small_kernel<1>, g, 64, 1, s, psi, nullptr, codes, exps, nullptr, B, 1 << n);
  }
  if (cb > kTileBits) return cudaErrorInvalidValue;
  const BitMap m = bit_map(cb, to);
  const unsigned g = (unsigned)((count + (long long)kWarpAmps * (kThreads8 / 32) - 1) / ((long long)kWarpAmps * (kThreads8 / 32)));
  if (save) {
    if (cb) return launch_after(slot8_save_kernel<true>, g, kThreads8, 1, s, psi, codes, exps, count, m);
    return launch_after(slot8_save_kernel<false>, g, kThreads8, 1, s, psi, codes, exps, count, m);
  }
  if (cb) return launch_after(slot8_load_kernel<true>, g, kThreads8, 1, s, psi, codes, exps, count, m);
  return launch_after(slot8_load_kernel<false>, g, kThreads8, 1, s, psi, codes, exps, count, m);
}

cudaError_t launch_slot8_from_planes(const float2* buf, const float2* partner, int8_t* codes, uint8_t* exps, int B,
                                     int n, cudaStream_t s) {
  if (n < 4) {
    return launch_after(slot8_small_kernel<2>, (unsigned)((B + 63) / 64), 64, 1, s, const_cast<float2*>(buf),
                        const_cast<float2*>(partner), codes, exps, nullptr, B, 1 << n);
  }
  const dim3 g(blocks_for(1ll << n), (unsigned)((B + 1) / 2 < 32768 ? (B + 1) / 2 : 32768));
  return launch_after(slot8_from_planes_kernel, g, kThreads8, 1, s, buf, partner, codes, exps, B, 1ll << n);
}

cudaError_t launch_slot8_to_planes(float2* plane0, float2* plane1, const int8_t* codes, const uint8_t* exps,
                                   const float* rscale, int B, int n, cudaStream_t s) {
  if (n < 4) {
    return launch_after(slot8_small_kernel<3>, (unsigned)((B + 63) / 64), 64, 1, s, plane0, plane1,
                        const_cast<int8_t*>(codes), const_cast<uint8_t*>(exps), rscale, B, 1 << n);
  }
  const long long count = (long long)B << n;
  return launch_after(slot8_to_planes_kernel, blocks_for(count), kThreads8, 1, s, plane0, plane1, codes, exps, rscale, count);
}

}  // namespace qml
