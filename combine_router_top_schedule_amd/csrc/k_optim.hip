// The optimizer step: the squared norm of all gradients, and AdamW over many tensors with moments
// in fp32 or in MXFP8 (E4M3 codes, one UE8M0 scale per 32 elements).
//
// Both stream their tensors once and do little arithmetic per byte, so HBM bounds them: the norm reads 6.8
// TB/s (178 M fp32 gradients, 105 us), the step moves 5.8 TB/s with fp32 moments (the same tensors and a bf16
// copy, 30 bytes a parameter, 927 us) and 6.2 TB/s with 8-bit ones (267 M parameters, 18.1 bytes, 777 us), where
// a large copy reaches 4.7 TB/s and a large fill 6.8 TB/s. Tensors are
// described in kernel arguments (no device table to upload, so a call can be captured); a workgroup finds its
// tensor by searching the prefix sums of their chunk counts.
#include <algorithm>
#include <cmath>

#include "mok_internal.h"
#include "mok_device.h"

// Every product and sum is rounded on its own: contracted into fused multiply-adds, results would
// depend on what the compiler chose to fuse in each of the variants below.
#pragma clang fp contract(off)

namespace mok {
namespace {

// ---- sum of squares -------------------------------------------------------------------------
constexpr int kSqTensors = 160;      // tensors a launch takes (kernel arguments hold 4 KB)
constexpr int kSqThreads = 512;
constexpr int kSqBlocks = 512;       // workgroups of a launch; fixed, so sums do not depend on the device
constexpr int kSqChunk = 8192;       // elements of a chunk: 4 loads of 16 bytes a thread in flight

struct SqArgs {
  const void* g[kSqTensors];
  int64_t n[kSqTensors];
  int32_t first[kSqTensors + 1];     // chunks before tensor t
  int32_t count;
  double* part;
  uint32_t* ticket;                  // of the last launch: workgroups that have written their sum (else null)
  int64_t parts;                     // sums of all launches
  double* out;
};

// The tensor of chunk c: the last t with first[t] <= c. Every lane looks at one prefix sum (a binary search
// took 6 dependent loads, each some 0.3 us).
template <int CAP>
__device__ __forceinline__ int find_tensor(const int32_t (&first)[CAP], int count, int c) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll
  for (int i = 0; i < CAP; i += 64) {
    const bool in = i + lane < count && first[min(i + lane, CAP - 1)] <= c;
    before += __popcll(__ballot(in));
  }
  return before - 1;
}

// Sum over a workgroup, in a fixed order; the result in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kSqThreads / 64];
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();   // (an earlier call's readers)
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0;
  for (int w = 0; w < kSqThreads / 64; ++w) sum += s[w];
  return sum;
}

// Four consecutive elements from i on, as they lie in memory, those past n as zero. (Converted behind all loads:
// in the branches each load would be waited for before the next.)
__device__ __forceinline__ f32x4 load_sq(const float* g, int64_t i, int64_t n) {
  if (i + 4 <= n) return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(g + i));
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < 4; ++j)
    if (i + j < n) v[j] = g[i + j];
  return v;
}
__device__ __forceinline__ uint64_t load_sq(const uint16_t* g, int64_t i, int64_t n) {
  if (i + 4 <= n) return __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(g + i));
  uint64_t v = 0;
  for (int j = 0; j < 4; ++j)
    if (i + j < n) v |= uint64_t(g[i + j]) << (16 * j);
  return v;
}
__device__ __forceinline__ float element(const f32x4& v, int j) { return v[j]; }
__device__ __forceinline__ float element(uint64_t v, int j) { return bf2f(uint16_t(v >> (16 * j))); }

template <bool BF16>
__global__ __launch_bounds__(kSqThreads) void k_sumsq(SqArgs a) {
  double sum = 0;
  for (int c = blockIdx.x; c < a.first[a.count]; c += gridDim.x) {
    const int t = __builtin_amdgcn_readfirstlane(find_tensor(a.first, a.count, c));
    const int64_t i0 = int64_t(c - a.first[t]) * kSqChunk + threadIdx.x * 4, n = a.n[t];
    constexpr int U = kSqChunk / (4 * kSqThreads);
    using Elem = std::conditional_t<BF16, uint16_t, float>;
    std::conditional_t<BF16, uint64_t, f32x4> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_sq(static_cast<const Elem*>(a.g[t]), i0 + u * 4 * kSqThreads, n);
#pragma unroll
    for (int u = 0; u < U; ++u)
      for (int j = 0; j < 4; ++j) {
        const double x = element(v[u], j);
        sum = fma(x, x, sum);
      }
  }
  sum = block_sum(sum);
  // The sums of all workgroups are joined, in the order of their numbers, by the one that comes last; a
  // second launch for that took 4 us. Sums and ticket go through agent-scope accesses, which are coherent
  // across XCDs: a sum has arrived (the wait) before its workgroup is counted.
  __shared__ bool s_last;
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.part + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    s_last = a.ticket && __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                             gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  double all = 0;
  const double* first = a.part + gridDim.x - a.parts;   // this launch's sums are the last ones
  for (int64_t i = threadIdx.x; i < a.parts; i += kSqThreads)
    all += __hip_atomic_load(first + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  all = block_sum(all);
  if (threadIdx.x == 0) {
    *a.out = all;
    st_relaxed_u(a.ticket, 0u);   // ready for the next call
  }
}

// ---- AdamW ------------------------------------------------------------------------------------
constexpr int kAdTensors = 48;       // tensors a launch takes
constexpr int kAdChunk = 1024;       // elements a workgroup updates, 4 a thread (8 a thread, or 4 times 4, are
                                     // 2 to 9 % slower at 100 M elements and more)

struct AdamArgs {
  void* p[kAdTensors];
  uint16_t* copy[kAdTensors];
  const void* g[kAdTensors];
  void* m[kAdTensors];
  void* v[kAdTensors];
  uint8_t* ms[kAdTensors];
  uint8_t* vs[kAdTensors];
  int64_t n[kAdTensors];
  int32_t first[kAdTensors + 1];
  int32_t count, number0;            // number0: position of this launch's first tensor in the call
  uint32_t seed;
  float b1, c1, b2, c2, eps;         // c = 1 - b
  float rbc2;                        // 1 / sqrt(1 - beta2^step)
  float decay, rate;                 // 1 - lr weight_decay, lr / (1 - beta1^step)
  const double* sumsq;
  const double* lr_dev;
  const int64_t* step_dev;
  double max_norm, lr, beta1, beta2, weight_decay;
  int64_t step;
};

// Random bits: a hash by xor-shifts and odd multiplications (the fractional bits of sqrt 2 and
// sqrt 3), which map 32 bits one to one.
__host__ __device__ inline uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x6A09E667u;
  h ^= h >> 15;
  h *= 0xBB67AE85u;
  return h ^ (h >> 16);
}

// 2^e, e in [-127, 127]
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __uint_as_float(uint32_t(e + 127) << 23) : __uint_as_float(1u << 22);
}

// Exponent code of a run whose largest magnitude has these fp32 bits: the smallest power of two 2^(c-127)
// that keeps it at most 448 = 1.75 * 2^8; 0 for a run of zeros, 0xFF if it is not finite.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  if (amax >= 0x7F800000u) return 0xFFu;
  const int c = int(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax < 0x800000u || c < 0 ? 0u : uint32_t(c);
}

// The largest of 8 consecutive lanes: exchanges within 4 lanes, then with the mirrored lane of the other 4.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true)));
  v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true)));
  return max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x141, 0xF, 0xF, true)));
}

// Four values of a run held by 8 consecutive lanes -> their codes, and the run's scale code. `u` holds 16
// random bits in its upper half. The conversion adds the upper 20 bits of its seed below the kept
// mantissa and cuts: |x| goes to floor(|x| / step + u / 2^16) steps, subnormal codes too. POSITIVE: what is above
// zero does not become zero, as one step (2^-9) stays one step.
template <bool POSITIVE>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], const uint32_t (&u)[4], uint32_t* scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  amax = max8(amax);
  const uint32_t c = scale_code(amax);
  *scale = c;
  const float inv = pow2(127 - int(min(c, 254u)));
  float r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = x[j] * inv;
    if (POSITIVE) r[j] = r[j] > 0.f ? fmaxf(r[j], 0x1p-9f) : r[j];
  }
  int code = __builtin_amdgcn_cvt_sr_fp8_f32(r[0], int(u[0]), 0, 0);
  code = __builtin_amdgcn_cvt_sr_fp8_f32(r[1], int(u[1]), code, 1);
  code = __builtin_amdgcn_cvt_sr_fp8_f32(r[2], int(u[2]), code, 2);
  code = __builtin_amdgcn_cvt_sr_fp8_f32(r[3], int(u[3]), code, 3);
  return c == 0xFFu ? 0u : uint32_t(code);
}

__device__ __forceinline__ void decode4(uint32_t code, uint32_t scale, float (&x)[4]) {
  const float s = scale == 0xFFu ? NAN : pow2(int(scale) - 127);
  x[0] = __builtin_amdgcn_cvt_f32_fp8(int(code), 0) * s;
  x[1] = __builtin_amdgcn_cvt_f32_fp8(int(code), 1) * s;
  x[2] = __builtin_amdgcn_cvt_f32_fp8(int(code), 2) * s;
  x[3] = __builtin_amdgcn_cvt_f32_fp8(int(code), 3) * s;
}

// Four consecutive elements from i on; without FULL (a chunk that ends inside, n > 0), those past n read as
// zero and are not written, and the others are loaded one by one from clamped addresses: with branches around
// whole and single loads each load would be waited for before the next. Every byte is used once, so whole
// accesses pass the caches by (927 us instead of 985 us for 178 M elements with fp32 states, 777 us instead of
// 868 us for 267 M with 8-bit ones).
template <bool FULL>
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t n, float (&x)[4]) {
  if constexpr (FULL) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = p[min(i + j, n - 1)];
      x[j] = i + j < n ? v : 0.f;
    }
  }
}
template <bool FULL>
__device__ __forceinline__ void load4(const uint16_t* p, int64_t i, int64_t n, float (&x)[4]) {
  if constexpr (FULL) {
    const uint64_t v = __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(p + i));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = bf2f(uint16_t(v >> (16 * j)));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = bf2f(p[min(i + j, n - 1)]);
      x[j] = i + j < n ? v : 0.f;
    }
  }
}
template <bool FULL>
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int64_t i, int64_t n) {
  if constexpr (FULL) {
    return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + i));
  } else {
    uint32_t x = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = p[min(i + j, n - 1)];
      x |= (i + j < n ? v : 0u) << (8 * j);
    }
    return x;
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, const float (&x)[4]) {
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = x[j];
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint16_t* p, int64_t i, int64_t n, uint2 x) {
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(uint64_t(x.x) | uint64_t(x.y) << 32, reinterpret_cast<uint64_t*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = uint16_t((j & 2 ? x.y : x.x) >> (16 * (j & 1)));
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint8_t* p, int64_t i, int64_t n, uint32_t x) {
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(x, reinterpret_cast<uint32_t*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = uint8_t(x >> (8 * j));
  }
}

// fp32 -> BF16 bits by adding 16 random bits below the kept ones (infinities and NaN as they are).
__device__ __forceinline__ uint32_t bf16_random(float x, uint32_t u) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7F800000u) == 0x7F800000u) return f2bf(x);
  return (b + u) >> 16;
}

// The step of 4 elements a thread, from i on, of tensor t.
template <bool GBF, bool PBF, bool MX8, bool FULL>
__device__ __forceinline__ void adamw4(const AdamArgs& a, int t, int64_t i, int64_t n, uint32_t seed, float clip,
                                       float decay, float rate, float rbc2) {
  float g[4], p[4], m[4], v[4], r[4];
  load4<FULL>(static_cast<const std::conditional_t<GBF, uint16_t, float>*>(a.g[t]), i, n, g);
  load4<FULL>(static_cast<const std::conditional_t<PBF, uint16_t, float>*>(a.p[t]), i, n, p);
  if constexpr (MX8) {
    const uint32_t cm = load4<FULL>(static_cast<const uint8_t*>(a.m[t]), i, n);
    const uint32_t cv = load4<FULL>(static_cast<const uint8_t*>(a.v[t]), i, n);
    const int64_t run = (FULL ? i : min(i, n - 1)) >> 5;
    const uint32_t sm = a.ms[t][run], sv = a.vs[t][run];
    decode4(cm, sm, m);
    decode4(cv, sv, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * v[j];
  } else {
    load4<FULL>(static_cast<const float*>(a.m[t]), i, n, m);
    load4<FULL>(static_cast<const float*>(a.v[t]), i, n, v);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gj = g[j] * clip;
    m[j] = m[j] * a.b1 + gj * a.c1;
    v[j] = v[j] * a.b2 + (gj * gj) * a.c2;
    r[j] = sqrtf(v[j]);
    p[j] = p[j] * decay - (m[j] / (r[j] * rbc2 + a.eps)) * rate;
  }
  uint32_t h[4], u[4];
  if constexpr (MX8 || PBF) {
    const uint32_t salt = mix(seed + uint32_t(a.number0 + t) * 0x9E3779B1u);
    const uint32_t base = mix(salt + uint32_t(i >> 32));
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = mix((uint32_t(i) + j) ^ base);
  }
  if constexpr (PBF) {
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = bf16_random(p[j], mix(h[j] ^ 0x3C6EF372u) & 0xFFFFu);
    store4<FULL>(static_cast<uint16_t*>(a.p[t]), i, n, uint2{u[0] | u[1] << 16, u[2] | u[3] << 16});
  } else {
    store4<FULL>(static_cast<float*>(a.p[t]), i, n, p);
    if (a.copy[t]) store4<FULL>(a.copy[t], i, n, uint2{pack_bf2(p[0], p[1]), pack_bf2(p[2], p[3])});
  }
  if constexpr (MX8) {
    uint32_t sm, sv;
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = h[j] << 16;
    const uint32_t cm = encode4<false>(m, u, &sm);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = h[j] & 0xFFFF0000u;
    const uint32_t cv = encode4<true>(r, u, &sv);
    store4<FULL>(static_cast<uint8_t*>(a.m[t]), i, n, cm);
    store4<FULL>(static_cast<uint8_t*>(a.v[t]), i, n, cv);
    if ((threadIdx.x & 7) == 0 && (FULL || i < n)) {
      a.ms[t][i >> 5] = uint8_t(sm);
      a.vs[t][i >> 5] = uint8_t(sv);
    }
  } else {
    store4<FULL>(static_cast<float*>(a.m[t]), i, n, m);
    store4<FULL>(static_cast<float*>(a.v[t]), i, n, v);
  }
}

template <bool GBF, bool PBF, bool MX8>
__global__ __launch_bounds__(256) void k_adamw(AdamArgs a) {
  float clip = 1.f;
  if (a.sumsq) {
    const double sq = *a.sumsq;
    if (!(sq < INFINITY)) return;   // NaN, too
    const double norm = sqrt(sq);
    clip = norm > a.max_norm ? float(a.max_norm / norm) : 1.f;
  }
  float decay = a.decay, rate = a.rate, rbc2 = a.rbc2;
  uint32_t seed = a.seed;
  // Formed again by every thread: 926 us instead of 899 us for 178 M elements with fp32 moments, 1,374 us instead of
  // 778 us for 267 M with 8-bit ones, which have more arithmetic in their way already.
  if (a.lr_dev || a.step_dev) {
    const double lr = a.lr_dev ? *a.lr_dev : a.lr;
    const int64_t number = a.step_dev ? *a.step_dev : a.step;
    if (!(lr >= 0.0 && lr < INFINITY) || number < 1) return;   // what the host refuses: NaN, too
    // replays of a captured step differ in their step alone, and with the same bits in each of them
    // an element's small updates would be dropped in all of them, or in none
    if (a.step_dev) seed += uint32_t(number);
    const double step = double(number);
    decay = float(1.0 - lr * a.weight_decay);
    rate = float(lr / (1.0 - pow(a.beta1, step)));
    rbc2 = float(1.0 / sqrt(1.0 - pow(a.beta2, step)));
  }
  const int c = blockIdx.x;
  const int t = __builtin_amdgcn_readfirstlane(find_tensor(a.first, a.count, c));
  const int64_t n = a.n[t], i0 = int64_t(c - a.first[t]) * kAdChunk, i = i0 + threadIdx.x * 4;
  if (i0 + kAdChunk <= n) adamw4<GBF, PBF, MX8, true>(a, t, i, n, seed, clip, decay, rate, rbc2);
  else adamw4<GBF, PBF, MX8, false>(a, t, i, n, seed, clip, decay, rate, rbc2);
}

template <bool GBF, bool PBF>
void adamw_kernel(bool mx, const AdamArgs& a, int blocks, hipStream_t s) {
  if (mx) hipLaunchKernelGGL((k_adamw<GBF, PBF, true>), dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_adamw<GBF, PBF, false>), dim3(blocks), dim3(256), 0, s, a);
}

}  // namespace

// The ticket (64 bytes), then a sum per workgroup of every launch.
int64_t sumsq_ws_bytes(int count) {
  return 64 + 8 * int64_t(kSqBlocks) * std::max<int64_t>(1, cdiv(count, kSqTensors));
}

hipError_t launch_sumsq(int count, const mok_sumsq_tensor* t, bool bf16, double* out, uint8_t* ws,
                        hipStream_t s) {
  SqArgs a;
  a.out = out;
  a.parts = 0;
  int t0 = 0;
  do {   // (without an element, one launch writes 0)
    a.count = 0;
    int64_t chunks = 0;
    a.first[0] = 0;
    // (chunk numbers stay within 31 bits: a tensor of at most 2^33 elements has 2^20)
    for (; t0 < count && a.count < kSqTensors; ++t0) {
      if (t[t0].n == 0) continue;
      a.g[a.count] = t[t0].g;
      a.n[a.count] = t[t0].n;
      chunks += cdiv(t[t0].n, kSqChunk);
      a.first[++a.count] = int32_t(chunks);
    }
    while (t0 < count && t[t0].n == 0) ++t0;
    const int blocks = int(std::max<int64_t>(1, std::min<int64_t>(chunks, kSqBlocks)));
    a.part = reinterpret_cast<double*>(ws + 64) + a.parts;
    a.parts += blocks;
    a.ticket = t0 < count ? nullptr : reinterpret_cast<uint32_t*>(ws);
    if (bf16) hipLaunchKernelGGL(k_sumsq<true>, dim3(blocks), dim3(kSqThreads), 0, s, a);
    else hipLaunchKernelGGL(k_sumsq<false>, dim3(blocks), dim3(kSqThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (t0 < count);
  return hipSuccess;
}

hipError_t launch_adamw(int count, const mok_adamw_tensor* t, const mok_adamw_config& c, hipStream_t s) {
  AdamArgs a;
  a.seed = c.seed;
  a.b1 = float(c.beta1);
  a.c1 = float(1.0 - c.beta1);
  a.b2 = float(c.beta2);
  a.c2 = float(1.0 - c.beta2);
  a.eps = float(c.eps);
  a.lr = c.lr;
  a.beta1 = c.beta1;
  a.beta2 = c.beta2;
  a.weight_decay = c.weight_decay;
  a.max_norm = c.max_norm;
  a.step = c.step;
  a.sumsq = c.sumsq_dev;
  a.lr_dev = c.lr_dev;
  a.step_dev = c.step_dev;
  const double step = double(c.step);
  a.decay = float(1.0 - c.lr * c.weight_decay);
  a.rate = float(c.lr / (1.0 - std::pow(c.beta1, step)));
  a.rbc2 = float(1.0 / std::sqrt(1.0 - std::pow(c.beta2, step)));
  const bool mx = c.state == MOK_STATE_MX8, gbf = c.grad_elem == MOK_ELEM_BF16,
             pbf = c.param_elem == MOK_ELEM_BF16;
  for (int t0 = 0; t0 < count;) {
    a.count = 0;
    a.number0 = t0;
    int64_t chunks = 0;
    a.first[0] = 0;
    for (; t0 < count && a.count < kAdTensors; ++t0) {
      // a launch has fewer than 2^32 threads
      const int64_t more = cdiv(t[t0].n, kAdChunk);
      if (a.count > 0 && chunks + more >= (int64_t(1) << 24)) break;
      const int k = a.count++;
      a.p[k] = t[t0].p;
      a.copy[k] = static_cast<uint16_t*>(t[t0].copy);
      a.g[k] = t[t0].g;
      a.m[k] = t[t0].m;
      a.v[k] = t[t0].v;
      a.ms[k] = t[t0].m_scale;
      a.vs[k] = t[t0].v_scale;
      a.n[k] = t[t0].n;
      chunks += more;   // (an empty tensor has no chunk, so no workgroup finds it)
      a.first[a.count] = int32_t(chunks);
    }
    if (chunks == 0) continue;
    const int blocks = int(chunks);
    if (gbf) {
      if (pbf) adamw_kernel<true, true>(mx, a, blocks, s);
      else adamw_kernel<true, false>(mx, a, blocks, s);
    } else {
      if (pbf) adamw_kernel<false, true>(mx, a, blocks, s);
      else adamw_kernel<false, false>(mx, a, blocks, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mok
