// Expert routing with scores, balancing bias, groups and renormalised weights, and its gradient.
//
// Forward, per token: s = sigmoid(x) or softmax(x); keys s + b (or x); the best groups; the K largest
// keys; weights from s. The choice must not depend on fp32 rounding, and among a few million scores
// many pairs are closer than that. k_route_fwd compares all keys in fp64, one token a wave (131,072 tokens,
// top 8: 293 us for 256 experts, sigmoid, bias, 16 groups; 282 us for 8 groups of 31; 665 us for 384 experts in 12
// groups); k_route_fast lets fp32 decide what it can and takes 60 us for 256 experts in 8 groups: 1,390 vector
// instructions for 8 tokens, issued in 70 % of its cycles, bound it; reading the logits would take 22 us at
// 6.2 TB/s. 131,072 x 384 in bf16 (no groups): 57 us. More experts or choices: 113 us for 256 with top 16, 114 us
// for 512 in 16 groups (154 us with top 16), 229 us for 1024 in 32 groups, 289 us for 1024 in bf16 with top 16.
// Backward: the chosen weights are q = softmax over the chosen of f(x), f = x or log sigmoid(x), so
// dx_k = scale q_k (dw_k - sum_j dw_j q_j) f'(x_k) with f' = 1 or sigmoid(-x_k), zero elsewhere; without
// renormalisation the scores' own derivatives. It is bound by the store of the gradient: 35 us for
// 131,072 x 256 fp32 (134 MB written; 64 bytes fetched around each chosen logit are another 67 MB), 8.6 us
// for plain softmax weights, 20,011 x 384 bf16 (31 MB).
#include <cfloat>
#include <type_traits>

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
  int vec;               // rows allow loads of 4 logits
  uint32_t chunk_magic;  // ceil(2^16 / (gs / 4)): a chunk's group is (chunk * magic) >> 16 (chunks < 256)
  uint32_t group_magic;  // ceil(2^32 / gs), gs > 1: an expert's group is (expert * magic) >> 32
  float scale;
};

template <bool BF16>
__device__ __forceinline__ float logit(const void* x, int64_t at) {
  if constexpr (BF16) return bf2f(static_cast<const uint16_t*>(x)[at]);
  else return static_cast<const float*>(x)[at];
}

// Four consecutive logits, aligned for one load.
template <bool BF16>
__device__ __forceinline__ void load_logits4(const void* x, int64_t at, float* v) {
  if constexpr (BF16) {
    const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + at);
    v[0] = bf2f(uint16_t(b.x));
    v[1] = bf2f(uint16_t(b.x >> 16));
    v[2] = bf2f(uint16_t(b.y));
    v[3] = bf2f(uint16_t(b.y >> 16));
  } else {
    const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at);
    v[0] = b[0];
    v[1] = b[1];
    v[2] = b[2];
    v[3] = b[3];
  }
}

// Orders LDS accesses of the lanes of one wave (which runs them in order) for the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// x -> log sigmoid(x), to a few units of 2^-23 of max(1, |result|): it goes into exponentials. The form
// does not overflow.
__device__ __forceinline__ float log_sigmoid(float x) {
  return fminf(x, 0.f) - __logf(1.f + __expf(-fabsf(x)));
}

// ---- exchanges between lanes
template <int OFF>
__device__ __forceinline__ float lane_xor(float v) {
  const int x = __float_as_int(v);
  // (after the steps below it, a partner in the mirrored place of the other half holds what the xor-ed
  // lane holds)
  if constexpr (OFF == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));
  else if constexpr (OFF == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));
  else if constexpr (OFF == 4) return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));
  else if constexpr (OFF == 8) return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true));
  else return __shfl_xor(v, OFF, 64);
}
template <int CTRL>   // a permutation of every 4 lanes
__device__ __forceinline__ int quad(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true); }
template <int CTRL>
__device__ __forceinline__ float quad(float v) { return __int_as_float(quad<CTRL>(__float_as_int(v))); }
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, lane_xor<1>(v));
  v = fmaxf(v, lane_xor<2>(v));
  v = fmaxf(v, lane_xor<4>(v));
  if constexpr (L > 8) v = fmaxf(v, lane_xor<8>(v));
  if constexpr (L > 16) v = fmaxf(v, lane_xor<16>(v));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  if constexpr (L > 8) v += lane_xor<8>(v);
  if constexpr (L > 16) v += lane_xor<16>(v);
  return v;
}

// ---- one token by a whole wave, keys in fp64 -----------------------------------------------------
// Largest of the wave's values, in every lane: shifts within rows of 16 lanes, then broadcasts of a row's
// last lane to the next rows; lanes without a source keep their own value.
template <int CTRL>
__device__ __forceinline__ double max_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int lo = int(uint32_t(b)), hi = int(uint32_t(b >> 32));
  const uint32_t l = uint32_t(__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, false));
  const uint32_t h = uint32_t(__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, false));
  const double o = __builtin_bit_cast(double, uint64_t(h) << 32 | l);
  return o > v ? o : v;
}
__device__ __forceinline__ double wave_max(double v) {
  v = max_dpp<0x111>(v);   // row_shr:1
  v = max_dpp<0x112>(v);   // row_shr:2
  v = max_dpp<0x114>(v);   // row_shr:4
  v = max_dpp<0x118>(v);   // row_shr:8
  v = max_dpp<0x142>(v);   // row_bcast:15
  v = max_dpp<0x143>(v);   // row_bcast:31
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b)), 63));
  const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b >> 32)), 63));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// key: LDS, 64 Q doubles (Q = experts / 64, rounded up), private to the wave; bias: in LDS or memory. Returns
// the expert chosen by slot `lane` (lane < K), -1 where none is left. Written for a short way through few
// instructions: where a token in some thousands needs it, all but latency and the fetching of its
// code is hidden.
template <bool BF16, int Q>
__device__ __forceinline__ int choose_wave(const RouteArgs& a, const float* bias, int64_t n, int lane,
                                           double* key) {
  const double kNone = -INFINITY;
  const int64_t row = n * a.ld;
  const bool top2 = a.G > 1 && a.top2, scored = bias || top2;
  float x[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) x[q] = lane + 64 * q < a.E ? logit<BF16>(a.x, row + lane + 64 * q) : -INFINITY;
#pragma unroll
  for (int q = 0; q < Q; ++q) key[lane + 64 * q] = x[q];
  if (scored) {
    float most = 0.f;
    double sum = 0;
    if (!a.sigmoid) {
      most = x[0];
#pragma unroll
      for (int q = 1; q < Q; ++q) most = fmaxf(most, x[q]);
#pragma unroll 1
      for (int off = 32; off; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    }
    // exp(-x), or exp(x - largest), and the score with its bias; a softmax needs its sum before
#pragma unroll 1
    for (int pass = a.sigmoid; pass < 2; ++pass) {
#pragma unroll 1
      for (int e = lane; e < a.E; e += 64) {
        const double v = key[e];
        const double t = exp(a.sigmoid ? -v : v - double(most));
        if (pass == 0) {
          sum += t;
        } else {
          const double k = (a.sigmoid ? 1.0 : t) / (a.sigmoid ? 1.0 + t : sum) + (bias ? double(bias[e]) : 0.0);
          key[e] = v > kNone && k > kNone ? k : kNone;
        }
      }
      if (pass == 0)
#pragma unroll 1
        for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
    }
  }
  wave_sync();
  uint64_t stay = ~0ull;
  int P = 64;   // lanes a group
  if (a.G > 1) {
    while (P * a.G > 64) P >>= 1;
    // each lane the two largest of its experts, then those of the P lanes
    const int g = lane / P;
    double best = kNone, second = kNone;
    if (g < a.G)
#pragma unroll 2
      for (int i = lane % P; i < a.gs; i += P) {
        const double k = key[g * a.gs + i];
        const bool able = k > kNone;   // (NaN is not)
        const double low = k < best ? k : best;
        second = able && low > second ? low : second;
        best = able && k > best ? k : best;
      }
#pragma unroll 1
    for (int off = P >> 1; off; off >>= 1) {
      const double b = __shfl_xor(best, off, 64), c = __shfl_xor(second, off, 64);
      const double low = b < best ? b : best;
      second = c > second ? c : second;
      second = low > second ? low : second;
      best = b > best ? b : best;
    }
    if (a.top2 && second > kNone) best += second;
    int place = 0;
    for (int o = 0; o < a.G; ++o) {
      const double other = __shfl(best, o * P, 64);
      place += other > best || (other == best && o < g);
    }
    stay = __ballot(g < a.G && place < a.Kg);
  }
  // From here on in registers. Without a bias the logits decide (groups may have gone by scores).
  double k[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    const int g = a.gs > 1 ? int(__umulhi(uint32_t(e), a.group_magic)) : e;
    const double v = e < a.E ? key[e] : kNone;
    const bool in = e < a.E && v > kNone && (a.G == 1 || ((stay >> (g * P & 63)) & 1));
    k[q] = in ? (bias ? v : double(x[q])) : kNone;
  }
  int mine = -1;
#pragma unroll 1
  for (int slot = 0; slot < a.K; ++slot) {
    double best = k[0];
    int at = lane;
#pragma unroll
    for (int q = 1; q < Q; ++q) {
      at = k[q] > best ? lane + 64 * q : at;
      best = k[q] > best ? k[q] : best;
    }
    const double all = wave_max(best);
    if (!(all > kNone)) break;   // the same in every lane
    uint64_t who = __ballot(best == all);
    if (who & (who - 1)) {       // several: the lowest expert
      int first = best == all ? at : a.E;
#pragma unroll 1
      for (int off = 32; off; off >>= 1) first = min(first, __shfl_xor(first, off, 64));
      who = __ballot(best == all && at == first);
    }
    const int first = __builtin_amdgcn_readlane(at, __builtin_ctzll(who));
    mine = lane == slot ? first : mine;
#pragma unroll
    for (int q = 0; q < Q; ++q) k[q] = first == lane + 64 * q ? kNone : k[q];
  }
  wave_sync();
  return mine;
}

// Weight from a chosen expert's logit v: a softmax over the chosen of v or log sigmoid(v) among the `W` lanes
// of its token, or the score itself (top, sum: the row's largest logit and the sum of its
// exponentials).
template <int W>
__device__ __forceinline__ float slot_weight(const RouteArgs& a, bool some, float v, float top, float sum) {
  float w;
  if (a.renorm) {
    const float f = a.sigmoid ? log_sigmoid(v) : v;
    const float top_f = lanes_max<W>(f);   // (every lane takes part in the exchanges)
    const float q = some ? __expf(f - top_f) : 0.f;
    w = q / lanes_sum<W>(q);
  } else {
    w = a.sigmoid ? 1.f / (1.f + __expf(-v)) : __expf(v - top) / sum;
  }
  return some ? w * a.scale : 0.f;
}

// Weight of the expert in slot `lane` (lane < K; e < 0: none), by a whole wave.
template <bool BF16>
__device__ __forceinline__ float weight_wave(const RouteArgs& a, int64_t n, int lane, int e) {
  const int64_t row = n * a.ld;
  const bool some = lane < a.K && e >= 0;
  float top = 0.f, sum = 1.f;
  if (!a.sigmoid && !a.renorm) {
    top = -INFINITY;
    sum = 0.f;
    for (int i = lane; i < a.E; i += 64) top = fmaxf(top, logit<BF16>(a.x, row + i));
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    for (int i = lane; i < a.E; i += 64) sum += __expf(logit<BF16>(a.x, row + i) - top);
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  return slot_weight<16>(a, some, some ? logit<BF16>(a.x, row + e) : -INFINITY, top, sum);
}

template <bool BF16, int Q>
__global__ __launch_bounds__(64 * kWaves) void k_route_fwd(RouteArgs a) {
  __shared__ double s_key[kWaves][64 * Q];
  __shared__ int s_load[64 * Q];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (a.load) {
    for (int e = threadIdx.x; e < a.E; e += 64 * kWaves) s_load[e] = 0;
    __syncthreads();
  }
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < a.N; n += int64_t(gridDim.x) * kWaves) {
    int e = -1;
    float w = 0.f;
    if (!a.mask || a.mask[n]) {
      e = choose_wave<BF16, Q>(a, a.bias, n, lane, s_key[wave]);
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

// ---- many tokens per wave ---------------------------------------------------------------------
// L lanes share a token, each with V of its experts in registers (lane j holds experts 4 (j + L i) + c), so
// a wave reads whole rows of 64 / L tokens and keeps enough loads in flight. Comparing every key in
// fp64 would cost 256 exponentials in fp64 a token; instead
//   1. keys are formed in fp32 with an error of at most eps (0 without a bias: the logits themselves);
//   2. the groups are ranked by their fp32 scores; a token whose border between staying and leaving groups
//      is not wider than the error goes to choose_wave;
//   3. tau, the K-th largest fp32 key, comes from sorting networks: each lane's V keys to a sorted list of
//      KM, then the lists of the L lanes merged pairwise. The K best in exact arithmetic all have an fp32
//      key of at least tau - 2 eps (of the keys above kappa + eps, kappa the exact K-th, fewer than K exist, so
//      tau <= kappa + eps; and theirs are at least kappa - eps);
//   4. those few candidates (nearly always exactly K) are ranked by counting. Two whose fp32 keys are
//      further apart than 2 eps are in that order; two of the same logit and bias are tied; else
//      the candidates are compared by fp64 keys. A token with more than 2 KM candidates goes to choose_wave
//      (choose_apart), and so does one of softmax scores whose fp32 keys do not decide.
// Larger value to a, smaller to b.
__device__ __forceinline__ void order(float& a, float& b) {
  const float hi = fmaxf(a, b), lo = fminf(a, b);
  a = hi;
  b = lo;
}

// Sorts v[0..M) downwards: Batcher's odd-even merge network (M a power of two).
template <int M>
__device__ __forceinline__ void sort_down(float* v) {
#pragma unroll
  for (int p = 1; p < M; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < M; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < M && (i + j) / (p * 2) == (i + j + k) / (p * 2)) order(v[i + j], v[i + j + k]);
}

// The M largest of two lists sorted downwards, sorted: the larger of v[i] and w[M-1-i] form a bitonic
// sequence, which log2 M half-cleaners sort.
template <int M>
__device__ __forceinline__ void merge_down(float* v, const float* w) {
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = fmaxf(v[i], w[M - 1 - i]);
#pragma unroll
  for (int k = M / 2; k >= 1; k /= 2)
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (!(i & k)) order(v[i], v[i + k]);
}
template <int OFF, int M>
__device__ __forceinline__ void merge_lanes(float* v) {
  float w[M];
#pragma unroll
  for (int i = 0; i < M; ++i) w[i] = lane_xor<OFF>(v[i]);
  merge_down<M>(v, w);
}
// The least of the M largest of two lanes' lists.
template <int OFF, int M>
__device__ __forceinline__ float merged_least(const float* v) {
  float least = fmaxf(v[0], lane_xor<OFF>(v[M - 1]));
#pragma unroll
  for (int i = 1; i < M; ++i) least = fminf(least, fmaxf(v[i], lane_xor<OFF>(v[M - 1 - i])));
  return least;
}

// The tokens n0 + b / L for the set bits b of `left`, one after the other. Not inlined: the constants of its
// fp64 exponentials would be kept in 80 registers throughout the tile loop (70 us instead of 61 us for
// 131,072 tokens of 256 experts). Called from the loop and not behind it, so that the 4 to 10 us which a
// token takes, nearly all of it latency, are filled by the other waves.
template <bool BF16, int Q>
__device__ __attribute__((noinline)) void choose_apart(const RouteArgs* args, const float* bias, double* key,
                                                       int* load, int64_t n0, uint64_t left, int L) {
  // the same in every lane, and so in scalar registers
  RouteArgs a;
  {
    const int* from = reinterpret_cast<const int*>(args);
    int* to = reinterpret_cast<int*>(&a);
    static_assert(sizeof(RouteArgs) % 4 == 0, "copied by words");
#pragma unroll
    for (int i = 0; i < int(sizeof(RouteArgs) / 4); ++i) to[i] = __builtin_amdgcn_readfirstlane(from[i]);
  }
  const int lane = threadIdx.x & 63;
  for (; left; left &= left - 1) {
    const int64_t n = n0 + __builtin_ctzll(left) / L;
    const int e = choose_wave<BF16, Q>(a, bias, n, lane, key);
    const float w = weight_wave<BF16>(a, n, lane, e);
    if (lane < a.K) {
      a.idx[n * a.K + lane] = e;
      a.w[n * a.K + lane] = w;
      if (a.load && e >= 0) atomicAdd(&load[e], 1);
    }
  }
}

// (Not inlined for the same reason.)
__device__ __attribute__((noinline)) double sigmoid64(float x) { return 1.0 / (1.0 + exp(-double(x))); }

// The fp64 number in the first two components.
__device__ __forceinline__ double pair64(const f32x4& v) {
  return __builtin_bit_cast(double, uint64_t(__float_as_uint(v[1])) << 32 | __float_as_uint(v[0]));
}

template <int L, int V, int KM>
struct FastLds {   // of one wave
  static constexpr int T = 64 / L, CAP = 2 * KM, CH = L * V / 4;
  union {
    float2 pair[T][CH + 1];       // the two largest of every 4 experts
    f32x4 cand[T][CAP];           // key, logit, bias, expert
    struct {
      double key[L * V];
      RouteArgs args;
    } slow;
  };
  float group[T][L];
  int2 out[T][KM];              // expert and logit (its bits) of each slot
};

// What a kernel forms scores of: of nothing (keys are the logits), of nothing but the softmax's sum (for plain
// softmax weights), or of every expert, for keys with a bias or for groups ranked by their two largest.
enum ScoreMode { kLogits, kLogitsAndSum, kSigmoidBias, kSoftmaxBias, kSigmoidTop2, kSoftmaxTop2 };

template <bool BF16, int L, int V, int KM, int MODE>
__global__ __launch_bounds__(64 * kWaves, L * V >= 1024 || V > 32 ? 3 : 4) void k_route_fast(RouteArgs a) {
  using Lds = FastLds<L, V, KM>;
  constexpr int T = Lds::T, CAP = Lds::CAP, SL = CAP > L ? CAP / L : 1;
  constexpr bool kBias = MODE == kSigmoidBias || MODE == kSoftmaxBias;
  constexpr bool kTop2 = MODE == kSigmoidTop2 || MODE == kSoftmaxTop2;   // scores for the groups only
  constexpr bool kSigmoid = MODE == kSigmoidBias || MODE == kSigmoidTop2;
  constexpr bool kSum = MODE == kLogitsAndSum || MODE == kSoftmaxBias || MODE == kSoftmaxTop2;
  __shared__ Lds s_wave[kWaves];
  __shared__ __attribute__((aligned(16))) float s_bias[kBias ? L * V : 4];
  __shared__ int s_load[L * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane % L, t = lane / L;
  Lds& s = s_wave[wave];
  for (int e = threadIdx.x; e < L * V; e += 64 * kWaves) {
    if constexpr (kBias) {
      const float b = e < a.E ? a.bias[e] : 0.f;
      s_bias[e] = b == b ? b : -INFINITY;   // NaN bars the expert, as -inf does
    }
    s_load[e] = 0;
  }
  __syncthreads();
  float big = 0.f;   // largest finite bias
  if constexpr (kBias) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const float b = fabsf(s_bias[e]);
      big = fmaxf(big, b < INFINITY ? b : 0.f);
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
  }
  const int per = a.gs >> 2;   // chunks of 4 experts per group
  // group of each of the lane's chunks, a byte each (31: none that can stay)
  uint32_t of_group[(V + 15) / 16] = {};
  if (a.G > 1)
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      of_group[i >> 2] |= min(((j + L * i) * a.chunk_magic) >> 16, 31u) << (8 * (i & 3));
  const uint64_t here = ((1ull << L) - 1) << (t * L);   // the token's lanes
  const int64_t tiles = (a.N + T - 1) / T;
  const int64_t stride = int64_t(gridDim.x) * kWaves;
  for (int64_t tile = int64_t(blockIdx.x) * kWaves + wave; tile < tiles; tile += stride) {
    const int64_t n = tile * T + t;
    const bool live = n < a.N && (!a.mask || a.mask[n]);
    // experts past E, and all of a masked token, are barred and not read: expert 4 (j + L i) + c of
    // this lane if 4 L i + c >= lim
    const int lim = live ? a.E - 4 * j : 0;
    const int64_t at = n * a.ld + 4 * j;
    float x[V];
    if (a.vec && a.E == L * V && __all(live)) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) load_logits4<BF16>(a.x, at + 4 * L * i, x + 4 * i);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) x[u] = -INFINITY;
      if (a.vec) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
          if (4 * L * i < lim) load_logits4<BF16>(a.x, at + 4 * L * i, x + 4 * i);
      } else {
#pragma unroll
        for (int u = 0; u < V; ++u)
          if (4 * L * (u >> 2) + (u & 3) < lim) x[u] = logit<BF16>(a.x, at + 4 * L * (u >> 2) + (u & 3));
      }
    }
    float top = 0.f, sum = 1.f, rsum = 1.f;
    if constexpr (kSum) {
      top = x[0];
#pragma unroll
      for (int u = 1; u < V; ++u) top = fmaxf(top, x[u]);
      top = lanes_max<L>(top);
      if (top == -INFINITY) top = 0.f;
      sum = 0.f;
#pragma unroll
      for (int u = 0; u < V; ++u) sum += __expf(x[u] - top);
      sum = lanes_sum<L>(sum);
      rsum = 1.f / sum;
    }
    // eps, in units u = 2^-24. Sigmoid: t = e^-v is off by 1.5 u |v| (two roundings of the exponent) and
    // 2 u (the instruction) of itself, which moves s by s (1 - s) <= 1/4 times that, and s (1 - s) |v| <= 0.23:
    // under 0.9 u; 1 + t and the reciprocal by another 1 u each (the last place of a number below 1). Softmax:
    // exponentials and the sum of at most 1024 positive terms (V in a row, then a tree) by 100 u of the
    // largest score, 1 / sum. The sum with the bias is rounded once more, to 1 u of at most 1 + |b|.
    const float eps = (kSigmoid ? 3.f : 100.f * rsum) * 0x1p-24f + (1.f + big) * 0x1p-24f;
    const float key_eps = kBias ? eps : 0.f;
    // Groups by their largest key: two fp32 scores are off by eps each, 2 eps apart, and a third takes up the
    // rounding of score -+ gap (up to half a unit, below eps) ahead of a comparison for less or more. By their two
    // largest: a sum of two keys is off by 2 eps and its own rounding of (up to 2 (1 + big)) u, two of them by 4 eps
    // and 4 (1 + big) u; score -+ gap, again a number of that size, by another 2 (1 + big) u; the seventh is slack.
    const float group_gap = kTop2 || (kBias && a.top2) ? 4.f * eps + 7.f * 0x1p-24f * (1.f + big) : 3.f * key_eps;
    auto score32 = [&](float v) {
      return kSigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-v)) : __expf(v - top) * rsum;
    };
    bool slow = false;
    // keys (in x from here on) and, through LDS, the groups' scores
    auto form_keys = [&](auto checked) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        float g[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float v = x[4 * i + c];
          float k = v;
          if constexpr (kBias) k = score32(v) + s_bias[4 * (j + L * i) + c];
          bool able = !checked || v > -INFINITY;                // NaN is not
          if constexpr (MODE == kSoftmaxBias) able = able && k > -INFINITY;   // (the row's sum may be NaN)
          if constexpr (kTop2) g[c] = score32(v);
          // (here too: without scores no group is better than another, and none stays)
          if constexpr (MODE == kSoftmaxTop2) able = able && (!checked || g[c] > -INFINITY);
          x[4 * i + c] = able ? k : -INFINITY;
          g[c] = able ? (kTop2 ? g[c] : k) : -INFINITY;
        }
        if (a.G > 1) {
          const float h0 = fmaxf(g[0], g[1]), l0 = fminf(g[0], g[1]);
          const float h1 = fmaxf(g[2], g[3]), l1 = fminf(g[2], g[3]);
          s.pair[t][j + L * i] = float2{fmaxf(h0, h1), fmaxf(fminf(h0, h1), fmaxf(l0, l1))};
        }
      }
    };
    // Two instructions an expert bar those of -inf and NaN; one an expert finds that a wave's rows hold none
    // (131,072 x 384 bf16: 58.9 us, so 56.8 us; x 256: 61.0 us, 60.2 us).
    float size = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) size += fabsf(x[u]);
    if (__any(!(size < INFINITY))) form_keys(std::true_type{});
    else form_keys(std::false_type{});
    if (a.G > 1) {
      wave_sync();
      float best = -INFINITY, second = -INFINITY;
      if (j < a.G) {
        int q = j;   // (lanes begin at different chunks of their groups: fewer bank conflicts)
        while (q >= per) q -= per;
        for (int r = 0; r < per; ++r, q = q + 1 == per ? 0 : q + 1) {
          const float2 p = s.pair[t][j * per + q];
          second = fmaxf(fmaxf(second, p.y), fminf(best, p.x));
          best = fmaxf(best, p.x);
        }
        if ((kBias || kTop2) && a.top2 && second > -INFINITY) best += second;
      }
      s.group[t][j] = best;
      wave_sync();
      // groups that certainly, or possibly, come before this one (places past G hold -inf)
      int above = 0, maybe = 0;
#pragma unroll
      for (int g = 0; g < L; ++g) {
        const float o = s.group[t][g];
        if constexpr (kBias || kTop2) {
          above += o > best + group_gap;
          maybe += o > best - group_gap;   // (this one counts itself)
        } else {
          above += o > best || (o == best && g < j);
        }
      }
      if constexpr (kBias || kTop2) maybe -= best > best - group_gap;
      else maybe = above;
      const bool in = j < a.G && above < a.Kg;
      const bool unsure = j < a.G && best > -INFINITY &&
                          ((in && maybe >= a.Kg) || ((kBias || kTop2) && !(best < INFINITY)));
      slow = (__ballot(unsure) & here) != 0;
      const uint32_t stay = uint32_t((__ballot(in) & here) >> (t * L));
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const bool keep = (stay >> ((of_group[i >> 2] >> (8 * (i & 3))) & 31)) & 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * i + c] = keep ? x[4 * i + c] : -INFINITY;
      }
    }
    // tau
    float list[KM], next[KM];
#pragma unroll
    for (int u = 0; u < KM; ++u) list[u] = x[u];
    sort_down<KM>(list);
#pragma unroll
    for (int i = KM; i < V; i += KM) {
#pragma unroll
      for (int u = 0; u < KM; ++u) next[u] = x[i + u];
      sort_down<KM>(next);
      merge_down<KM>(list, next);
    }
    merge_lanes<1, KM>(list);
    merge_lanes<2, KM>(list);
    if constexpr (L > 8) merge_lanes<4, KM>(list);
    if constexpr (L > 16) merge_lanes<8, KM>(list);
    float tau;
    if (a.K == KM) {   // (the last two lists then need no sorting: 60 us for 131,072 x 256, 61 us with it)
      tau = merged_least<L / 2, KM>(list);
    } else {
      merge_lanes<L / 2, KM>(list);
      tau = list[0];
#pragma unroll
      for (int i = 1; i < KM; ++i) tau = i < a.K ? list[i] : tau;
    }
    const float cut = fmaxf(tau - 2.f * key_eps, -FLT_MAX);
    // a bit per expert of the lane: shifted in with the comparison's carry
    constexpr int W = (V + 31) / 32;
    uint32_t mine[W] = {};
#pragma unroll
    for (int u = V - 1; u >= 0; --u)
      asm("v_cmp_ge_f32 vcc, %1, %2\n\tv_addc_co_u32 %0, vcc, %0, %0, vcc" : "+v"(mine[u / 32]) : "v"(x[u]), "v"(cut) : "vcc");
    int upto = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) upto += __popc(mine[i]);
    const int own = upto;
#pragma unroll
    for (int off = 1; off < L; off *= 2) {
      const int o = __shfl_up(upto, off, L);
      if (j >= off) upto += o;
    }
    const int count = __shfl(upto, L - 1, L);
    slow = slow || count > CAP;
    const int have = slow ? 0 : count;
    if (!slow) {
      int slot = upto - own;
#pragma unroll
      for (int i = 0; i < W; ++i)
        while (mine[i]) {
          const int u = 32 * i + __builtin_ctz(mine[i]);
          mine[i] &= mine[i] - 1;
          s.cand[t][slot++][3] = __int_as_float(4 * (j + L * (u >> 2)) + (u & 3));
        }
    }
    wave_sync();
    f32x4 me[SL];
    float logit_of[SL];
    int rank[SL];
    const bool more = SL > 1 && __any(have > L);
#pragma unroll
    for (int q = 0; q < SL; ++q) {
      const int c = j + L * q;
      me[q] = f32x4{0.f, 0.f, 0.f, __int_as_float(-1)};
      rank[q] = 0;
      logit_of[q] = 0.f;
      if (q > 0 && !more) break;
      if (c < have) {
        const int e = __float_as_int(s.cand[t][c][3]);
        const float v = logit<BF16>(a.x, n * a.ld + e);
        float k = v, b = 0.f;
        if constexpr (kBias) {
          b = s_bias[e];
          k = score32(v) + b;
        }
        me[q] = f32x4{k, v, b, __int_as_float(e)};
        logit_of[q] = v;
        s.cand[t][c] = me[q];
      }
    }
    // At most 8 candidates, all in the token's first 8 lanes: each meets the other 7 by lane exchanges. If all
    // keys are further apart than the error, or exact, that is their order; else, and for more candidates,
    // the loop below looks at logits and biases too.
    bool unsure = false, again = __any(have > 8);
    if (!again) {
      const float k0 = j < have ? me[0][0] : -INFINITY;
      const int e0 = __float_as_int(me[0][3]);
      const float k7 = lane_xor<4>(k0);   // (lane 7 - j)
      const int e7 = __float_as_int(lane_xor<4>(__int_as_float(e0)));
      bool near = false;
      auto meet = [&](float ko, int eo) {
        rank[0] += ko > k0 || (ko == k0 && eo < e0);
        if constexpr (kBias) near |= fabsf(ko - k0) <= 2.f * key_eps;
      };
      meet(quad<0xB1>(k0), quad<0xB1>(e0));
      meet(quad<0x4E>(k0), quad<0x4E>(e0));
      meet(quad<0x1B>(k0), quad<0x1B>(e0));
      meet(k7, e7);
      meet(quad<0xB1>(k7), quad<0xB1>(e7));
      meet(quad<0x4E>(k7), quad<0x4E>(e7));
      meet(quad<0x1B>(k7), quad<0x1B>(e7));
      // (two +inf: their difference is not a number)
      if constexpr (kBias) again = __any(j < have && (near || k0 == INFINITY));
      if (again) rank[0] = 0;
    }
    if (again) {
      wave_sync();
      for (int c = 0; __ballot(c < have) != 0; ++c) {
        if (c < have) {
          const f32x4 o = s.cand[t][c];
#pragma unroll
          for (int q = 0; q < SL; ++q) {
            if (q > 0 && !more) break;
            const bool lower = __float_as_int(o[3]) < __float_as_int(me[q][3]);
            const bool same = o[1] == me[q][1] && o[2] == me[q][2];
            rank[q] += same ? lower : o[0] > me[q][0];
            // (keys of -inf and NaN are no candidates; with +inf the difference is not a number)
            if constexpr (kBias)
              unsure |= !same && !(fabsf(o[0] - me[q][0]) > 2.f * key_eps) && j + L * q < have;
          }
        }
      }
    }
    if constexpr (MODE == kSigmoidBias) {
      if (__any(unsure)) {
        // the candidates' keys in fp64, in the place of their fp32 key and logit
        wave_sync();
#pragma unroll
        for (int q = 0; q < SL; ++q) {
          const int c = j + L * q;
          rank[q] = 0;
          if (q > 0 && !more) break;
          const uint64_t k = __builtin_bit_cast(uint64_t, sigmoid64(me[q][1]) + double(me[q][2]));
          me[q][0] = __uint_as_float(uint32_t(k));
          me[q][1] = __uint_as_float(uint32_t(k >> 32));
          if (c < have) s.cand[t][c] = me[q];
        }
        wave_sync();
        for (int c = 0; __ballot(c < have) != 0; ++c) {
          if (c < have) {
            const f32x4 o = s.cand[t][c];
#pragma unroll
            for (int q = 0; q < SL; ++q) {
              if (q > 0 && !more) break;
              const double ko = pair64(o), km = pair64(me[q]);
              rank[q] += ko > km || (ko == km && __float_as_int(o[3]) < __float_as_int(me[q][3]));
            }
          }
        }
        unsure = false;
      }
    }
    slow = slow || (kBias && (__ballot(unsure) & here) != 0);
#pragma unroll
    for (int q = 0; q < SL; ++q)
      if (j + L * q < have && rank[q] < a.K)
        s.out[t][rank[q]] = int2{__float_as_int(me[q][3]), __float_as_int(logit_of[q])};
    // (a token that leaves here may have ranks that do not fill its slots)
    const int filled = slow ? 0 : have < a.K ? have : a.K;
    wave_sync();
    // weights of the slots, one a lane
    const int2 slot = j < filled ? s.out[t][j] : int2{-1, __float_as_int(-INFINITY)};
    const int e = slot.x;
    const bool some = e >= 0;
    const float v = __int_as_float(slot.y);
    const float w = slot_weight<L>(a, some, v, top, sum);
    if (n < a.N && j < a.K && !slow) {
      a.idx[n * a.K + j] = e;
      a.w[n * a.K + j] = w;
      if (a.load && some) atomicAdd(&s_load[e], 1);
    }
    wave_sync();
    if (const uint64_t apart = __ballot(slow && j == 0)) {
      if (lane == 0) s.slow.args = a;
      wave_sync();
      choose_apart<BF16, L * V / 64>(&s.slow.args, kBias ? s_bias : nullptr, s.slow.key, s_load, tile * T,
                                     apart, L);
      wave_sync();
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
  int vec;   // rows allow loads of 4 logits
  float scale;
};

// Expert of slot k of a token; -1 if it names none, or one that an earlier slot named. The token's KP
// slots are in KP consecutive lanes.
template <int KP>
__device__ __forceinline__ int slot_expert(const RouteBwdArgs& a, int64_t n, int k, bool live) {
  int e = live && k < a.K ? a.idx[n * a.K + k] : -1;
  if (e >= a.E) e = -1;
  bool again = false;
  if constexpr (KP == 8) {
    auto meet = [&](int o, int other) { again |= other < k && o == e; };
    const int m = __float_as_int(lane_xor<4>(__int_as_float(e)));   // (slot 7 - k)
    meet(quad<0xB1>(e), k ^ 1);
    meet(quad<0x4E>(e), k ^ 2);
    meet(quad<0x1B>(e), k ^ 3);
    meet(m, 7 - k);
    meet(quad<0xB1>(m), 7 - (k ^ 1));
    meet(quad<0x4E>(m), 7 - (k ^ 2));
    meet(quad<0x1B>(m), 7 - (k ^ 3));
  } else {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int o = __shfl(e, j, KP);
      again |= j < k && o == e;
    }
  }
  return again ? -1 : e;
}

// Stores `count` consecutive values (fp32 in LDS) at a 16-byte aligned place, by a wave.
template <bool BF16>
__device__ __forceinline__ void store_run(void* dst, int64_t at, const float* s, int count, int lane) {
  if constexpr (BF16) {
    uint16_t* d = static_cast<uint16_t*>(dst) + at;
    int i = lane * 8;
    for (; i + 8 <= count; i += 512) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(s + i), q = *reinterpret_cast<const f32x4*>(s + i + 4);
      __builtin_nontemporal_store(
          u32x4{pack_bf2(p[0], p[1]), pack_bf2(p[2], p[3]), pack_bf2(q[0], q[1]), pack_bf2(q[2], q[3])},
          reinterpret_cast<u32x4*>(d + i));
    }
    for (int j = i; j < count && j < i + 8; ++j) d[j] = f2bf(s[j]);
  } else {
    float* d = static_cast<float*>(dst) + at;
    int i = lane * 4;
    for (; i + 4 <= count; i += 256)
      __builtin_nontemporal_store(*reinterpret_cast<const f32x4*>(s + i), reinterpret_cast<f32x4*>(d + i));
    for (int j = i; j < count && j < i + 4; ++j) d[j] = s[j];
  }
}

// Gradients that reach the chosen logits only: every weight but the plain softmax's. A wave takes 8
// tokens: their K slots in KP lanes each, the results scattered into `rows` (4 or 8) zeroed rows in LDS at a
// time, and the rows (consecutive in memory) stored with 16 bytes a lane. LDS goes back to zero by the
// same scatter.
template <bool BF16, int KP>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd(RouteBwdArgs a, int rows) {
  extern __shared__ __attribute__((aligned(16))) float s_row[];   // [waves][rows][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  float* s = s_row + wave * rows * a.E;
  for (int i = lane; i < rows * a.E; i += 64) s[i] = 0.f;
  wave_sync();
  constexpr int kPass = KP / 8;   // passes of 64 / KP tokens
  for (int64_t n0 = (int64_t(blockIdx.x) * waves + wave) * 8; n0 < a.N;
       n0 += int64_t(gridDim.x) * waves * 8) {
    int ex[kPass];
    float dx[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int t = p * (64 / KP) + lane / KP, k = lane % KP;
      const int64_t n = n0 + t;
      const bool in = n < a.N && k < a.K;
      const float dw_in = in ? a.dw[n * a.K + k] : 0.f;
      const int e = slot_expert<KP>(a, n, k, n < a.N);
      const bool some = e >= 0;
      const float x = some ? logit<BF16>(a.x, n * a.ld + e) : -INFINITY;
      const float dw = some ? dw_in : 0.f;
      float d;
      if (a.renorm) {
        const float f = a.sigmoid ? log_sigmoid(x) : x;
        const float top = lanes_max<KP>(f);
        const float u = some ? __expf(f - top) : 0.f;
        const float q = u / lanes_sum<KP>(u);
        d = a.scale * q * (dw - lanes_sum<KP>(some ? dw * q : 0.f));
        if (a.sigmoid) d /= 1.f + __expf(x);
      } else {
        const float sg = 1.f / (1.f + __expf(-x));
        d = a.scale * dw * sg / (1.f + __expf(x));
      }
      ex[p] = e;
      dx[p] = d;
    }
    for (int r0 = 0; r0 < 8 && n0 + r0 < a.N; r0 += rows) {
      int at[kPass];
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const int t = p * (64 / KP) + lane / KP - r0;
        at[p] = ex[p] >= 0 && t >= 0 && t < rows ? t * a.E + ex[p] : -1;
        if (at[p] >= 0) s[at[p]] = dx[p];
      }
      wave_sync();
      const int64_t left = a.N - n0 - r0;
      store_run<BF16>(a.dx, (n0 + r0) * a.E, s, int(left < rows ? left : rows) * a.E, lane);
      wave_sync();
#pragma unroll
      for (int p = 0; p < kPass; ++p)
        if (at[p] >= 0) s[at[p]] = 0.f;
      wave_sync();
    }
  }
}

// The plain softmax's weights reach every logit: dx_e = scale s_e ([e chosen] dw_e - sum_j dw_j s_j). As in the
// forward, L lanes share a token, each with V of its experts in registers; the weights' gradients come to
// their experts through a row in LDS, zero but for them.
template <bool BF16, int L, int V>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd_dense(RouteBwdArgs a) {
  constexpr int T = 64 / L, SL = L < 16 ? 16 / L : 1;
  __shared__ __attribute__((aligned(16))) float s_row[kWaves][T][L * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane % L, t = lane / L;
  float* s = s_row[wave][t];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) *reinterpret_cast<f32x4*>(s + 4 * (j + L * i)) = f32x4{0.f, 0.f, 0.f, 0.f};
  wave_sync();
  const uint64_t here = ((1ull << L) - 1) << (t * L);   // the token's lanes
  const int64_t tiles = (a.N + T - 1) / T;
  for (int64_t tile = int64_t(blockIdx.x) * kWaves + wave; tile < tiles; tile += int64_t(gridDim.x) * kWaves) {
    const int64_t n = tile * T + t;
    const bool live = n < a.N;
    int ex[SL];
    float dw[SL], xk[SL];
    bool some = false;
#pragma unroll
    for (int p = 0; p < SL; ++p) {
      const int k = j + L * p;
      ex[p] = live && k < a.K ? a.idx[n * a.K + k] : -1;
      dw[p] = live && k < a.K ? a.dw[n * a.K + k] : 0.f;
      if (ex[p] >= a.E) ex[p] = -1;
    }
    // an expert that an earlier slot named counts once
    bool again[SL] = {};
    for (int k = 0; k + 1 < a.K; ++k) {
      const int o = SL > 1 && k >= L ? __shfl(ex[SL - 1], k - L, L) : __shfl(ex[0], k % L, L);
#pragma unroll
      for (int p = 0; p < SL; ++p) again[p] |= k < j + L * p && o == ex[p];
    }
#pragma unroll
    for (int p = 0; p < SL; ++p) {
      if (again[p]) ex[p] = -1;
      some |= ex[p] >= 0;
      xk[p] = ex[p] >= 0 ? logit<BF16>(a.x, n * a.ld + ex[p]) : -INFINITY;
    }
    // a row without a chosen expert is zero, whatever its logits hold
    const bool any = (__ballot(some) & here) != 0;
    const int lim = any ? a.E - 4 * j : 0;   // expert 4 (j + L i) + c of this lane exists if 4 L i + c < lim
    const int64_t at = n * a.ld + 4 * j;
    float x[V];
#pragma unroll
    for (int u = 0; u < V; ++u) x[u] = -INFINITY;
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        if (4 * L * i < lim) load_logits4<BF16>(a.x, at + 4 * L * i, x + 4 * i);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (4 * L * (u >> 2) + (u & 3) < lim) x[u] = logit<BF16>(a.x, at + 4 * L * (u >> 2) + (u & 3));
    }
    float top = x[0];
#pragma unroll
    for (int u = 1; u < V; ++u) top = fmaxf(top, x[u]);
    top = lanes_max<L>(top);
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      x[u] = __expf(x[u] - top);
      sum += x[u];
    }
    sum = lanes_sum<L>(sum);
    float back = 0.f;
#pragma unroll
    for (int p = 0; p < SL; ++p)
      if (ex[p] >= 0) {
        back += dw[p] * (__expf(xk[p] - top) / sum);
        s[ex[p]] = dw[p];
      }
    back = lanes_sum<L>(back);
    wave_sync();
    const float f = a.scale / sum;
    const int end = live ? a.E - 4 * j : 0;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      if (4 * L * i < end) {
        const f32x4 g = *reinterpret_cast<const f32x4*>(s + 4 * (j + L * i));
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = any ? x[4 * i + c] * f * (g[c] - back) : 0.f;
        const int64_t to = n * a.E + 4 * (j + L * i);
        if (a.E % 4 == 0) {
          if constexpr (BF16)
            __builtin_nontemporal_store(uint64_t(pack_bf2(o[0], o[1])) | uint64_t(pack_bf2(o[2], o[3])) << 32,
                                        reinterpret_cast<uint64_t*>(static_cast<uint16_t*>(a.dx) + to));
          else
            __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]},
                                        reinterpret_cast<f32x4*>(static_cast<float*>(a.dx) + to));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (4 * L * i + c < end) {
              if constexpr (BF16) static_cast<uint16_t*>(a.dx)[to + c] = f2bf(o[c]);
              else static_cast<float*>(a.dx)[to + c] = o[c];
            }
        }
      }
    }
    wave_sync();
#pragma unroll
    for (int p = 0; p < SL; ++p)
      if (ex[p] >= 0) s[ex[p]] = 0.f;
    wave_sync();
  }
}

int grid_of(int64_t items, int per, int cap) {
  const int64_t b = cdiv(items, per);
  return int(b < 1 ? 1 : (b > cap ? cap : b));
}

template <bool BF16, int L, int V, int KM>
void fast(const RouteArgs& a, int grid, hipStream_t s) {
  const dim3 g(grid), b(64 * kWaves);
  const bool top2 = a.G > 1 && a.top2;
  if (a.bias) {
    if (a.sigmoid) hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kSigmoidBias>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kSoftmaxBias>), g, b, 0, s, a);
  } else if (top2) {
    if (a.sigmoid) hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kSigmoidTop2>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kSoftmaxTop2>), g, b, 0, s, a);
  } else if (a.sigmoid || a.renorm) {
    hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kLogits>), g, b, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_route_fast<BF16, L, V, KM, kLogitsAndSum>), g, b, 0, s, a);
  }
}

template <bool BF16>
void route_fwd(const RouteArgs& a, bool quick, int lanes, int grid, hipStream_t s) {
  if (!quick) {
    if (a.E <= 256) hipLaunchKernelGGL((k_route_fwd<BF16, 4>), dim3(grid), dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((k_route_fwd<BF16, 16>), dim3(grid), dim3(64 * kWaves), 0, s, a);
  } else if (a.K <= 8) {
    if (lanes == 8) {
      if (a.E <= 64) fast<BF16, 8, 8, 8>(a, grid, s);
      else if (a.E <= 128) fast<BF16, 8, 16, 8>(a, grid, s);
      else if (a.E <= 256) fast<BF16, 8, 32, 8>(a, grid, s);
      else fast<BF16, 8, 48, 8>(a, grid, s);
    } else if (lanes == 16) {
      fast<BF16, 16, 32, 8>(a, grid, s);
    } else {
      fast<BF16, 32, 32, 8>(a, grid, s);
    }
  } else {
    if (lanes == 16) {
      if (a.E <= 256) fast<BF16, 16, 16, 16>(a, grid, s);
      else fast<BF16, 16, 32, 16>(a, grid, s);
    } else {
      fast<BF16, 32, 32, 16>(a, grid, s);
    }
  }
}

template <bool BF16>
void route_bwd_dense(const RouteBwdArgs& a, int cus, hipStream_t s) {
  const int lanes = a.E <= 256 ? 8 : a.E <= 512 ? 16 : 32;
  const dim3 g(grid_of(a.N, kWaves * 64 / lanes, 8 * cus)), b(64 * kWaves);
  if (a.E <= 64) hipLaunchKernelGGL((k_route_bwd_dense<BF16, 8, 8>), g, b, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((k_route_bwd_dense<BF16, 8, 16>), g, b, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route_bwd_dense<BF16, 8, 32>), g, b, 0, s, a);
  else if (a.E <= 384) hipLaunchKernelGGL((k_route_bwd_dense<BF16, 16, 24>), g, b, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_route_bwd_dense<BF16, 16, 32>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_route_bwd_dense<BF16, 32, 32>), g, b, 0, s, a);
}

}  // namespace

hipError_t launch_route_fwd(const mok_route_desc& d, const void* x, const float* bias,
                            const uint8_t* mask, int32_t* idx, float* w, int32_t* load, hipStream_t s) {
  RouteArgs a{x, bias, mask, idx, w, load, d.num_tokens, d.logits_stride, d.num_experts, d.top_k,
              d.num_groups, d.top_groups, d.num_experts / d.num_groups, d.score == MOK_SCORE_SIGMOID,
              d.group_score == MOK_GROUP_TOP2, d.renorm, 0, 0, 0, d.scale};
  const bool bf = d.elem == MOK_ELEM_BF16;
  a.vec = a.E % 4 == 0 && a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(x) & (bf ? 7 : 15)) == 0;
  const int cus = device_cus() > 0 ? device_cus() : 256;
  // lanes of a token: as many as its experts need at 32 a lane, and its choices at one a lane
  const int lanes = a.E <= (a.K <= 8 ? 384 : 0) ? 8 : a.E <= 512 ? 16 : 32;
  // groups that are not made of whole runs of 4 experts, or more of them than lanes, go one token a wave (256
  // experts, top 8: 293 us in 16 groups, which 16 lanes a token would hold, against 60 us in 8)
  const bool fast = a.G == 1 || (a.gs % 4 == 0 && a.G <= lanes);
  if (a.gs > 1) a.group_magic = uint32_t(cdiv(int64_t(1) << 32, a.gs));
  if (a.gs >= 4) a.chunk_magic = uint32_t(cdiv(65536, a.gs / 4));
  // One workgroup writes the load by itself; several add to it, which takes a launch that clears it first
  // (1.9 us in a graph, 3.8 us without). What a workgroup does in two steps, of 2 us (64 experts) to 3.7 us
  // (256) each, is left to one: 64 tokens take it 6.2 to 10.2 us in a graph, several 6.0 to 8.5 us, but without
  // a graph the second launch costs more; 128 tokens 10.4 to 17.5 us against 6.4 to 9.0 us. (8 waves in the
  // one, 5.1 to 8.5 us for 64 tokens, need LDS of a size set at launch, which is 0.7 % of every large call.)
  const int per_step = fast ? kWaves * 64 / lanes : kWaves;
  // as many workgroups as are resident: 4 a CU, 3 of the kernels with more registers (131,072 tokens of 384
  // experts: 60 us, with 4 a CU 65 us)
  const int per_cu = !fast ? 8 : a.E > 512 || (lanes == 8 && a.E > 256) ? 3 : 4;
  const int grid = load && a.N <= 2 * per_step ? 1 : grid_of(a.N, per_step, per_cu * cus);
  if (load && (grid > 1 || a.N == 0)) {
    const hipError_t e = launch_fill_u32(reinterpret_cast<uint32_t*>(load), 0u, a.E, s);
    if (e != hipSuccess) return e;
  }
  if (a.N == 0) return hipSuccess;
  if (bf) route_fwd<true>(a, fast, lanes, grid, s);
  else route_fwd<false>(a, fast, lanes, grid, s);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const mok_route_desc& d, const void* x, const int32_t* idx, const float* dw,
                            void* dx, hipStream_t s) {
  RouteBwdArgs a{x, idx, dw, dx, d.num_tokens, d.logits_stride, d.num_experts, d.top_k,
                 d.score == MOK_SCORE_SIGMOID, d.renorm, 0, d.scale};
  if (a.N == 0) return hipSuccess;
  const int cus = device_cus() > 0 ? device_cus() : 256;
  const bool bf = d.elem == MOK_ELEM_BF16;
  a.vec = a.E % 4 == 0 && a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(x) & (bf ? 7 : 15)) == 0;
  if (!a.sigmoid && !a.renorm) {
    if (bf) route_bwd_dense<true>(a, cus, s);
    else route_bwd_dense<false>(a, cus, s);
    return hipGetLastError();
  }
  // 4 rows a wave at a time (16 E bytes of LDS, so that enough waves are resident); 8 where a run of 4
  // bf16 rows would not end on 16 bytes, or where 8 are small. At most the 64 KB that a workgroup has
  // without asking for more.
  const int rows = (bf && a.E % 2) || a.E <= 64 ? 8 : 4;
  const int waves = int64_t(kWaves) * rows * a.E * 4 <= 65536 ? kWaves : 2;
  const int grid = grid_of(a.N, 8 * waves, 16 * cus);
  const size_t lds = size_t(waves) * rows * a.E * 4;
  const dim3 t(64 * waves);
  if (a.K <= 8) {
    if (bf) hipLaunchKernelGGL((k_route_bwd<true, 8>), dim3(grid), t, lds, s, a, rows);
    else hipLaunchKernelGGL((k_route_bwd<false, 8>), dim3(grid), t, lds, s, a, rows);
  } else {
    if (bf) hipLaunchKernelGGL((k_route_bwd<true, 16>), dim3(grid), t, lds, s, a, rows);
    else hipLaunchKernelGGL((k_route_bwd<false, 16>), dim3(grid), t, lds, s, a, rows);
  }
  return hipGetLastError();
}

}  // namespace mok
