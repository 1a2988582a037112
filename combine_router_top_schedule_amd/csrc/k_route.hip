// Expert routing with scores, balancing bias, groups and renormalised weights, and its gradient.
//
// Forward, per token: s = sigmoid(x) or softmax(x); keys s + b (or x); the best groups; the K largest
// keys; weights from s. The choice has to be that of exact arithmetic, and among a few million scores
// many pairs are closer than fp32 rounding, so keys are compared in fp64.
// Backward: the chosen weights are q = softmax over the chosen of f(x), f = x or log sigmoid(x), so
// dx_k = scale q_k (dw_k - sum_j dw_j q_j) f'(x_k) with f' = 1 or sigmoid(-x_k), zero elsewhere; without
// renormalisation the scores' own derivatives.
#include "mok_internal.h"
#include "mok_device.h"

namespace mok {
namespace {

constexpr int kWaves = 4;   // waves per workgroup

struct RouteArgs {
  const void* x;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* w;
  int32_t* load;
  int64_t N, ld;
  int E, K, G, Kg, gs;   // gs: experts per group
  int sigmoid, top2, renorm;
  float scale;
};

template <bool BF16>
__device__ __forceinline__ float logit(const void* x, int64_t at) {
  if constexpr (BF16) return bf2f(static_cast<const uint16_t*>(x)[at]);
  else return static_cast<const float*>(x)[at];
}

// Orders LDS accesses of the lanes of one wave (which runs them in order) for the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// x -> log sigmoid(x); the form that neither overflows nor cancels.
__device__ __forceinline__ float log_sigmoid(float x) {
  return fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
}

// ---- one token by a whole wave, keys in fp64 -----------------------------------------------------
// key: LDS, one double per expert, private to the wave. Returns the expert chosen by slot `lane`
// (lane < K), -1 where none is left.
template <bool BF16>
__device__ __forceinline__ int choose_wave(const RouteArgs& a, int64_t n, int lane, double* key) {
  const double kNone = -INFINITY;
  const int64_t row = n * a.ld;
  double top = kNone, sum = 0;
  if (!a.sigmoid && (a.bias || (a.G > 1 && a.top2))) {
    for (int e = lane; e < a.E; e += 64) top = fmax(top, double(logit<BF16>(a.x, row + e)));
    for (int off = 32; off; off >>= 1) top = fmax(top, __shfl_xor(top, off, 64));
    for (int e = lane; e < a.E; e += 64) sum += exp(double(logit<BF16>(a.x, row + e)) - top);
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  auto score = [&](double x) { return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum; };
  for (int e = lane; e < a.E; e += 64) {
    const double x = logit<BF16>(a.x, row + e);
    const double k = a.bias ? score(x) + double(a.bias[e]) : x;
    key[e] = x > kNone && k > kNone ? k : kNone;
  }
  wave_sync();
  if (a.G > 1) {
    // lane g < G: the group's score, then its place among all groups
    double best = kNone, second = kNone;
    if (lane < a.G) {
      for (int i = 0; i < a.gs; ++i) {
        double k = key[lane * a.gs + i];
        if (a.top2 && !a.bias && k > kNone) k = score(k);
        if (k > best) { second = best; best = k; }
        else if (k > second) second = k;
      }
      if (a.top2 && second > kNone) best += second;
    }
    int place = 0;
    for (int g = 0; g < a.G; ++g) {
      const double other = __shfl(best, g, 64);
      place += other > best || (other == best && g < lane);
    }
    const uint64_t stay = __ballot(lane < a.G && place < a.Kg);
    wave_sync();
    for (int e = lane; e < a.E; e += 64)
      if (!((stay >> (e / a.gs)) & 1)) key[e] = kNone;
    wave_sync();
  }
  int mine = -1;
  for (int k = 0; k < a.K; ++k) {
    double best = kNone;
    int at = a.E;
    for (int e = lane; e < a.E; e += 64)
      if (key[e] > best) { best = key[e]; at = e; }
    for (int off = 32; off; off >>= 1) {
      const double b = __shfl_xor(best, off, 64);
      const int i = __shfl_xor(at, off, 64);
      if (b > best || (b == best && i < at)) { best = b; at = i; }
    }
    if (!(best > kNone)) break;   // the same in every lane
    if (lane == k) mine = at;
    if ((at & 63) == lane) key[at] = kNone;
    wave_sync();
  }
  wave_sync();
  return mine;
}

// Weight of the expert in slot `lane` (lane < K; e < 0: none), by a whole wave.
template <bool BF16>
__device__ __forceinline__ float weight_wave(const RouteArgs& a, int64_t n, int lane, int e) {
  const int64_t row = n * a.ld;
  const bool some = lane < a.K && e >= 0;
  const float x = some ? logit<BF16>(a.x, row + e) : -INFINITY;
  float w;
  if (a.renorm) {
    const float f = a.sigmoid ? log_sigmoid(x) : x;
    float top = f;
    for (int off = 8; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 16));
    const float q = some ? expf(f - top) : 0.f;
    float sum = q;
    for (int off = 8; off; off >>= 1) sum += __shfl_xor(sum, off, 16);
    w = q / sum;
  } else if (a.sigmoid) {
    w = 1.f / (1.f + expf(-x));
  } else {
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < a.E; i += 64) top = fmaxf(top, logit<BF16>(a.x, row + i));
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    for (int i = lane; i < a.E; i += 64) sum += expf(logit<BF16>(a.x, row + i) - top);
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
    w = expf(x - top) / sum;
  }
  return some ? w * a.scale : 0.f;
}

template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_route_fwd(RouteArgs a) {
  extern __shared__ double s_key[];   // [kWaves][E], then int [E]
  int* s_load = reinterpret_cast<int*>(s_key + kWaves * a.E);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (a.load) {
    for (int e = threadIdx.x; e < a.E; e += 64 * kWaves) s_load[e] = 0;
    __syncthreads();
  }
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < a.N; n += int64_t(gridDim.x) * kWaves) {
    int e = -1;
    float w = 0.f;
    if (!a.mask || a.mask[n]) {
      e = choose_wave<BF16>(a, n, lane, s_key + wave * a.E);
      w = weight_wave<BF16>(a, n, lane, e);
    }
    if (lane < a.K) {
      a.idx[n * a.K + lane] = e;
      a.w[n * a.K + lane] = w;
      if (a.load && e >= 0) atomicAdd(&s_load[e], 1);
    }
  }
  if (a.load) {
    // integer sums: their order changes nothing
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 64 * kWaves) {
      if (gridDim.x == 1) a.load[e] = s_load[e];
      else if (s_load[e]) atomicAdd(&a.load[e], s_load[e]);
    }
  }
}

// ---- backward -----------------------------------------------------------------------------------
struct RouteBwdArgs {
  const void* x;
  const int32_t* idx;
  const float* dw;
  void* dx;
  int64_t N, ld;
  int E, K;
  int sigmoid, renorm;
  float scale;
};

// Expert of slot k of a token; -1 if it names none, or one that an earlier slot named.
template <int KP>
__device__ __forceinline__ int slot_expert(const RouteBwdArgs& a, int64_t n, int k, bool live) {
  int e = live && k < a.K ? a.idx[n * a.K + k] : -1;
  if (e >= a.E) e = -1;
  bool again = false;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    const int o = __shfl(e, j, KP);
    again |= j < k && o == e;
  }
  return again ? -1 : e;
}

template <int KP>
__device__ __forceinline__ float slots_sum(float v) {
#pragma unroll
  for (int off = KP / 2; off; off >>= 1) v += __shfl_xor(v, off, KP);
  return v;
}

// Stores `count` consecutive values (fp32 in LDS) at a 16-byte aligned place, by a wave.
template <bool BF16>
__device__ __forceinline__ void store_run(void* dst, int64_t at, const float* s, int count, int lane) {
  if constexpr (BF16) {
    uint16_t* d = static_cast<uint16_t*>(dst) + at;
    int i = lane * 8;
    for (; i + 8 <= count; i += 512) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(s + i), q = *reinterpret_cast<const f32x4*>(s + i + 4);
      *reinterpret_cast<u32x4*>(d + i) =
          u32x4{pack_bf2(p[0], p[1]), pack_bf2(p[2], p[3]), pack_bf2(q[0], q[1]), pack_bf2(q[2], q[3])};
    }
    for (int j = i; j < count && j < i + 8; ++j) d[j] = f2bf(s[j]);
  } else {
    float* d = static_cast<float*>(dst) + at;
    int i = lane * 4;
    for (; i + 4 <= count; i += 256) *reinterpret_cast<f32x4*>(d + i) = *reinterpret_cast<const f32x4*>(s + i);
    for (int j = i; j < count && j < i + 4; ++j) d[j] = s[j];
  }
}

// Gradients that reach the chosen logits only: every weight but the plain softmax's. A wave takes 8
// tokens: their K slots in KP lanes each, the results scattered into 8 zeroed rows in LDS, and
// the rows (consecutive in memory) stored with 16 bytes a lane. LDS goes back to zero by the same
// scatter.
template <bool BF16, int KP>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd(RouteBwdArgs a) {
  extern __shared__ __attribute__((aligned(16))) float s_row[];   // [waves][8][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  float* s = s_row + wave * 8 * a.E;
  for (int i = lane; i < 8 * a.E; i += 64) s[i] = 0.f;
  wave_sync();
  constexpr int kPass = KP / 8;   // passes of 64 / KP tokens
  for (int64_t n0 = (int64_t(blockIdx.x) * waves + wave) * 8; n0 < a.N;
       n0 += int64_t(gridDim.x) * waves * 8) {
    int at[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int t = p * (64 / KP) + lane / KP, k = lane % KP;
      const int64_t n = n0 + t;
      const int e = slot_expert<KP>(a, n, k, n < a.N);
      const bool some = e >= 0;
      const float x = some ? logit<BF16>(a.x, n * a.ld + e) : -INFINITY;
      const float dw = some ? a.dw[n * a.K + k] : 0.f;
      float d;
      if (a.renorm) {
        const float f = a.sigmoid ? log_sigmoid(x) : x;
        float top = f;
#pragma unroll
        for (int off = KP / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, KP));
        const float u = some ? expf(f - top) : 0.f;
        const float q = u / slots_sum<KP>(u);
        d = a.scale * q * (dw - slots_sum<KP>(some ? dw * q : 0.f));
        if (a.sigmoid) d /= 1.f + expf(x);
      } else {
        const float sg = 1.f / (1.f + expf(-x));
        d = a.scale * dw * sg / (1.f + expf(x));
      }
      at[p] = some ? t * a.E + e : -1;
      if (some) s[at[p]] = d;
    }
    wave_sync();
    const int64_t left = a.N - n0;
    store_run<BF16>(a.dx, n0 * a.E, s, int(left < 8 ? left : 8) * a.E, lane);
    wave_sync();
#pragma unroll
    for (int p = 0; p < kPass; ++p)
      if (at[p] >= 0) s[at[p]] = 0.f;
    wave_sync();
  }
}

// The plain softmax's weights reach every logit: dx_e = scale s_e ([e chosen] dw_e - sum_j dw_j s_j).
// One wave per token.
template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd_dense(RouteBwdArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < a.N; n += int64_t(gridDim.x) * kWaves) {
    const int64_t row = n * a.ld;
    const int e = slot_expert<16>(a, n, lane & 15, true);
    const bool some = e >= 0;
    const bool any = __ballot(some) != 0;
    const float x = some ? logit<BF16>(a.x, row + e) : -INFINITY;
    const float dw = some ? a.dw[n * a.K + (lane & 15)] : 0.f;
    float top = -INFINITY, sum = 0.f;
    if (any) {
      for (int i = lane; i < a.E; i += 64) top = fmaxf(top, logit<BF16>(a.x, row + i));
      for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
      for (int i = lane; i < a.E; i += 64) sum += expf(logit<BF16>(a.x, row + i) - top);
      for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
    }
    const float back = slots_sum<16>(some ? dw * (expf(x - top) / sum) : 0.f);
    for (int i0 = 0; i0 < a.E; i0 += 64) {
      const int i = i0 + lane;
      float g = -back;
      for (int k = 0; k < a.K; ++k) {
        const int ek = __shfl(e, k, 64);
        const float dk = __shfl(dw, k, 64);
        if (ek == i) g += dk;
      }
      if (i < a.E) {
        const float v = any ? a.scale * (expf(logit<BF16>(a.x, row + i) - top) / sum) * g : 0.f;
        if constexpr (BF16) static_cast<uint16_t*>(a.dx)[n * a.E + i] = f2bf(v);
        else static_cast<float*>(a.dx)[n * a.E + i] = v;
      }
    }
  }
}

int grid_of(int64_t items, int per, int cap) {
  const int64_t b = cdiv(items, per);
  return int(b < 1 ? 1 : (b > cap ? cap : b));
}

}  // namespace

hipError_t launch_route_fwd(const mok_route_desc& d, const void* x, const float* bias,
                            const uint8_t* mask, int32_t* idx, float* w, int32_t* load, hipStream_t s) {
  RouteArgs a{x, bias, mask, idx, w, load, d.num_tokens, d.logits_stride, d.num_experts, d.top_k,
              d.num_groups, d.top_groups, d.num_experts / d.num_groups, d.score == MOK_SCORE_SIGMOID,
              d.group_score == MOK_GROUP_TOP2, d.renorm, d.scale};
  const int cus = device_cus() > 0 ? device_cus() : 256;
  const int grid = grid_of(a.N, kWaves, 8 * cus);
  if (load && (grid > 1 || a.N == 0)) {
    const hipError_t e = launch_fill_u32(reinterpret_cast<uint32_t*>(load), 0u, a.E, s);
    if (e != hipSuccess) return e;
  }
  if (a.N == 0) return hipSuccess;
  const size_t lds = size_t(kWaves) * a.E * 8 + size_t(a.E) * 4;   // at most 36 KB
  if (d.elem == MOK_ELEM_BF16)
    hipLaunchKernelGGL(k_route_fwd<true>, dim3(grid), dim3(64 * kWaves), lds, s, a);
  else
    hipLaunchKernelGGL(k_route_fwd<false>, dim3(grid), dim3(64 * kWaves), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const mok_route_desc& d, const void* x, const int32_t* idx, const float* dw,
                            void* dx, hipStream_t s) {
  RouteBwdArgs a{x, idx, dw, dx, d.num_tokens, d.logits_stride, d.num_experts, d.top_k,
                 d.score == MOK_SCORE_SIGMOID, d.renorm, d.scale};
  if (a.N == 0) return hipSuccess;
  const int cus = device_cus() > 0 ? device_cus() : 256;
  const bool bf = d.elem == MOK_ELEM_BF16;
  if (!a.sigmoid && !a.renorm) {
    const int grid = grid_of(a.N, kWaves, 8 * cus);
    if (bf) hipLaunchKernelGGL(k_route_bwd_dense<true>, dim3(grid), dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL(k_route_bwd_dense<false>, dim3(grid), dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
  }
  // 32 E bytes of LDS per wave, within the 64 KB that a workgroup has without asking for more
  const int waves = a.E <= 512 ? 4 : 2;
  const int grid = grid_of(a.N, 8 * waves, 8 * cus);
  const size_t lds = size_t(waves) * 8 * a.E * 4;
  const dim3 t(64 * waves);
  if (a.K <= 8) {
    if (bf) hipLaunchKernelGGL((k_route_bwd<true, 8>), dim3(grid), t, lds, s, a);
    else hipLaunchKernelGGL((k_route_bwd<false, 8>), dim3(grid), t, lds, s, a);
  } else {
    if (bf) hipLaunchKernelGGL((k_route_bwd<true, 16>), dim3(grid), t, lds, s, a);
    else hipLaunchKernelGGL((k_route_bwd<false, 16>), dim3(grid), t, lds, s, a);
  }
  return hipGetLastError();
}

}  // namespace mok
