// Muon: momentum, and its update orthogonalised by Newton-Schulz products.
//
// For a matrix u (the momentum, or with Nesterov the gradient plus mu times it), with X on its smaller side
// m <= n and X_0 = u / (|u|_F + eps), each step does
//   A = X X^T,   B = b A + c A A,   X <- a X + B X,
// an odd polynomial of X's singular values that takes them all towards 1. A step is three launches of products:
// A and A A are symmetric, so only the tiles on and below the diagonal are computed and both halves written; the last
// step's product ends in the parameters' update instead of X. All matrices of a call go through the same
// launches, whatever their shapes: a workgroup finds its matrix by the prefix sums of their tile counts.
//
// Precision. X is kept in 19 bits, fp16 and a byte for the bits below, times a power of two near sqrt(n) that keeps it in
// fp16's normal range; a X is formed from all of them, the products take X, A and B in fp16 with fp32 sums. Kept in
// fp16 alone, X's rounding drowns the small singular values of a gradient with a few large ones: the result is off by
// 1.3e-2 there (512 x 1792, rank 129 plus 1 % noise), with the byte by 8e-4, with bf16 everywhere by 1e-1. A's and B's
// diagonals hold most of them where singular values are alike: they are kept apart in fp32 (fp16 holds zeros), and their parts
// of the products added to the sums, with the same fp16 as the products take: so a direction that A lacks stays one in A A
// and B X. Random matrices are off by 1e-3 so, by 2e-3 to 4e-3 without. On the matrix cores fp16 is as fast as bf16.
//
// Measured, 12 matrices of 2048 x 7168 and a small one, 5 steps, 8.64 ms: X X^T 410 us (880 TFLOP/s on the half that is
// computed; 433 tiles of 256 x 256 on 256 CUs make two rounds, the second 69 % full), A A 133 us, B X 985 us (730 TFLOP/s; 600 us
// of it the products, the rest X in and out, 2.6 GB through HBM), once a call the norm 447 us and X_0 537 us, both at 4.7 TB/s.
// 256 x 256 tiles have one workgroup a CU, 128 x 128 two: B X takes 1,256 us so, but calls with under 256 large tiles less.
#include <algorithm>
#include <cmath>

#include "k_gemm.h"

// What is fused is written so: left to the compiler, the variants of a kernel would round differently, and a matrix's result
// depend on what else is in the call.
#pragma clang fp contract(off)

namespace mok {
namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

constexpr int kMuItems = 40;       // tensors (or parts of their batches) that a launch takes (of 4 KB of arguments)
constexpr int kMuParts = 256;      // partial sums of a matrix's norm at most
constexpr int kMuPad = 128;        // matrices are padded to multiples of this with zeros, which stay zeros

struct MuItem {
  const void* g;      // gradient, or the source
  float* m;           // momentum; null: orthogonalise g
  void* p;            // parameters, or the bf16 output
  uint16_t* copy;
  uint8_t* ws;        // of the part's first matrix
  int32_t e0, batch;  // the part's matrices: e0 .. e0 + batch - 1 of the tensor
  int32_t rows, cols;
  float adjust;
};

struct MuArgs {
  MuItem item[kMuItems];
  int32_t first[kMuItems + 1];   // tiles (or chunks) before item t
  int32_t count;
  int32_t nesterov, gbf;
  float mu, eps;
  float a, b, c;                 // the step's coefficients
  int32_t flip;                  // the step's number, odd or even: which operand buffer holds X
  double lr, weight_decay, max_norm;
  const double* sumsq;
  const double* lr_dev;
};

// A matrix's buffers in the workspace. `s` is X as its parameters lie ([rows][cols], padded), `t` its transpose. The
// product with B reads `t` (`s` where rows > cols) while its tiles are written, so that one has a second buffer.
struct MuBuffers {
  int64_t plane, gram;           // bytes of X in fp16 and of A
  int rows, cols, m, n;          // padded; m = min, n = max
  __host__ __device__ MuBuffers(int r, int c) {
    rows = int(align_up(r, kMuPad));
    cols = int(align_up(c, kMuPad));
    m = rows < cols ? rows : cols;
    n = rows < cols ? cols : rows;
    plane = int64_t(rows) * cols * 2;
    gram = int64_t(m) * m * 2;
  }
  __host__ __device__ int64_t bytes() const { return parts_at() + kMuParts * 8; }
  __host__ __device__ int64_t parts_at() const { return 3 * plane + plane / 2 + 2 * (gram + m * 4); }
  __device__ bool turned(const MuItem& it) const { return it.rows > it.cols; }
  __device__ _Float16* s(uint8_t* ws, bool turn, int flip) const { return at(ws, turn && flip ? 2 * plane : 0); }
  __device__ _Float16* t(uint8_t* ws, bool turn, int flip) const { return at(ws, !turn && flip ? 2 * plane : plane); }
  __device__ _Float16* a(uint8_t* ws) const { return at(ws, 3 * plane); }
  __device__ _Float16* b(uint8_t* ws) const { return at(ws, 3 * plane + gram); }
  __device__ uint8_t* lo(uint8_t* ws) const { return ws + 3 * plane + 2 * gram; }
  __device__ float* diagonal(uint8_t* ws, bool of_b) const {
    return reinterpret_cast<float*>(lo(ws) + plane / 2) + (of_b ? m : 0);
  }
  __device__ double* parts(uint8_t* ws) const { return reinterpret_cast<double*>(ws + parts_at()); }
  __device__ static _Float16* at(uint8_t* p, int64_t off) { return reinterpret_cast<_Float16*>(p + off); }
};

// x rounded to fp16. The compiler would join this with the sum that gives x in an instruction that rounds once, in some
// variants of a kernel and not in others.
__device__ __forceinline__ _Float16 to_half(float x) {
  asm("" : "+v"(x));
  return _Float16(x);
}

// X's lower bits: what fp16 leaves of x, in 256ths of h's last place (2^-24 for the smallest), one byte.
__device__ __forceinline__ int exponent_of(_Float16 h) {
  return max(int(__float_as_uint(float(h)) >> 23 & 0xFF), 113);   // (2^-14, below which fp16's places stay)
}
__device__ __forceinline__ int low_bits(float x, _Float16 h) {
  const float q = rintf((x - float(h)) * __uint_as_float(uint32_t(272 - exponent_of(h)) << 23));
  return int(fminf(fmaxf(q, -128.f), 127.f));
}
__device__ __forceinline__ float with_low(_Float16 h, int low) {
  return fmaf(float(low), __uint_as_float(uint32_t(exponent_of(h) - 18) << 23), float(h));
}

// The power of two that X is stored with: near sqrt(n), so that the result's elements are near 1.
__host__ __device__ inline float mu_scale(int rows, int cols) {
  int n = rows > cols ? rows : cols, e = 0;
  while (n > 1) n >>= 2, ++e;
  return float(1 << e);
}

// What u is multiplied by before it is divided by `size` = |u| + eps, whose reciprocal is beyond fp32 below some 2^-120: a
// power of two, so nothing is rounded, and nothing overflows as no element of u is larger than `size`.
__device__ __forceinline__ float mu_lift(double size) { return size < 0x1p-100 ? 0x1p100f : 1.f; }

// The item of workgroup c.
__device__ __forceinline__ int find_item(const MuArgs& a, int c) {
  const int lane = threadIdx.x & 63;
  const bool in = lane < a.count && a.first[min(lane, kMuItems)] <= c;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(in)) - 1);
}

// A step whose gradients' norm is not finite, or whose rate on the device is negative or not finite, changes nothing.
__device__ __forceinline__ bool left_out(const MuArgs& a) {
  if (a.sumsq && !isfinite(*a.sumsq)) return true;
  return a.lr_dev && !(*a.lr_dev >= 0.0 && isfinite(*a.lr_dev));
}
__device__ __forceinline__ float clip_factor(const MuArgs& a) {
  return a.sumsq ? float(fmin(1.0, a.max_norm / sqrt(*a.sumsq))) : 1.f;
}

__device__ __forceinline__ float element(const void* p, bool bf, int64_t i) {
  return bf ? bf2f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// ---- momentum and norm --------------------------------------------------------------------------
__host__ __device__ inline int64_t mu_chunk(int64_t size) {   // elements of a partial sum
  const int64_t c = align_up(cdiv(size, kMuParts), 1024);
  return c < 4096 ? 4096 : c;
}

// One partial sum of |u|^2 a workgroup, in fp64; with a momentum, also its update.
__global__ __launch_bounds__(256) void k_muon_norm(MuArgs a) {
  if (left_out(a)) return;
  if (int(blockIdx.x) >= a.first[a.count]) return;
  const int t = find_item(a, blockIdx.x);
  const MuItem& it = a.item[t];
  const int64_t size = int64_t(it.rows) * it.cols, chunk = mu_chunk(size);
  const int per = int(cdiv(size, chunk)), q = blockIdx.x - a.first[t], e = q / per;
  const int64_t base = (it.e0 + e) * size, i0 = base + (q % per) * chunk, i1 = min(i0 + chunk, base + size);
  const float clip = clip_factor(a);
  const bool bf = a.gbf;
  double sum = 0;
  const auto one = [&](float g, float m) {
    g *= clip;
    float u = g;
    if (it.m) {
      m = fmaf(m, a.mu, g);
      u = a.nesterov ? fmaf(a.mu, m, g) : m;
    }
    const double d = u;
    sum = fma(d, d, sum);
    return m;
  };
  for (int64_t i = (i0 & ~int64_t(3)) + threadIdx.x * 4; i < i1; i += 1024) {
    if (i >= i0 && i + 4 <= i1) {
      f32x4 g, m = {0.f, 0.f, 0.f, 0.f};
      if (bf) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(it.g) + i);
        g = f32x4{bf2f(uint16_t(v.x)), bf2f(uint16_t(v.x >> 16)), bf2f(uint16_t(v.y)), bf2f(uint16_t(v.y >> 16))};
      } else {
        g = *reinterpret_cast<const f32x4*>(static_cast<const float*>(it.g) + i);
      }
      if (it.m) m = *reinterpret_cast<const f32x4*>(it.m + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = one(g[j], m[j]);
      if (it.m) *reinterpret_cast<f32x4*>(it.m + i) = m;
    } else {
      for (int j = 0; j < 4; ++j)
        if (i + j >= i0 && i + j < i1) {
          const float m = one(element(it.g, bf, i + j), it.m ? it.m[i + j] : 0.f);
          if (it.m) it.m[i + j] = m;
        }
    }
  }
  __shared__ double s[4];
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    const MuBuffers b(it.rows, it.cols);
    b.parts(it.ws + e * align_up(b.bytes(), 256))[q % per] = s[0] + s[1] + s[2] + s[3];
  }
}

// A window of rows of a tensor's matrix, from element `first` on: buffer accesses whose bounds are the window's, so that
// elements outside read as zero and are not written, without branches (around single loads, each would be waited for
// before the next).
struct MuWindow {
  int64_t first, count;   // elements
  int cols;
  __device__ __forceinline__ MuWindow(const MuItem& it, int64_t first_, int rows)
      : first(first_), count(int64_t(rows) * it.cols), cols(it.cols) {}
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t of(const void* p, int size) const {
    return make_rsrc(static_cast<const uint8_t*>(p) + first * size, count * size);
  }
  // of row r and column c; beyond the window's end where c is beyond its columns
  __device__ __forceinline__ int at(int r, int c) const { return c < cols ? r * cols + c : 1 << 28; }
};
__device__ __forceinline__ float load_f32(__amdgpu_buffer_rsrc_t r, int i) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, i * 4, 0, 0));
}
__device__ __forceinline__ float load_bf16(__amdgpu_buffer_rsrc_t r, int i) {
  return bf2f(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(r, i * 2, 0, 0)));
}
__device__ __forceinline__ void store_f32(__amdgpu_buffer_rsrc_t r, int i, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, i * 4, 0, 0);
}
__device__ __forceinline__ void store_bf16(__amdgpu_buffer_rsrc_t r, int i, float v) {
  __builtin_amdgcn_raw_buffer_store_b16(f2bf(v), r, i * 2, 0, 0);
}

// N gradients (or source elements) of rows r0 + row(v) of column c.
template <int N, class R>
__device__ __forceinline__ void load_gradients(const MuArgs& a, const MuItem& it, const MuWindow& win, int r0, int c, R&& row,
                                               float (&g)[N]) {
  const int at = win.at(r0, c);
  if (a.gbf) {
    const __amdgpu_buffer_rsrc_t r = win.of(it.g, 2);
#pragma unroll
    for (int v = 0; v < N; ++v) g[v] = load_bf16(r, at + row(v) * win.cols);
  } else {
    const __amdgpu_buffer_rsrc_t r = win.of(it.g, 4);
#pragma unroll
    for (int v = 0; v < N; ++v) g[v] = load_f32(r, at + row(v) * win.cols);
  }
}

// The update of parameters (or the output) by results value(v) at rows r0 + row(v) of column c.
template <int N, class R, class V>
__device__ __forceinline__ void store_results(const MuItem& it, const MuWindow& win, int r0, int c, R&& row, V&& value,
                                              float decay, float rate) {
  const int at = win.at(r0, c);
  if (it.m) {
    const __amdgpu_buffer_rsrc_t p = win.of(it.p, 4);
    float y[N];
#pragma unroll
    for (int v = 0; v < N; ++v) y[v] = load_f32(p, at + row(v) * win.cols);
#pragma unroll
    for (int v = 0; v < N; ++v) {
      y[v] = fmaf(-value(v), rate, y[v] * decay);
      store_f32(p, at + row(v) * win.cols, y[v]);
    }
    if (it.copy) {
      const __amdgpu_buffer_rsrc_t q = win.of(it.copy, 2);
#pragma unroll
      for (int v = 0; v < N; ++v) store_bf16(q, at + row(v) * win.cols, y[v]);
    }
  } else {
    const __amdgpu_buffer_rsrc_t q = win.of(it.p, 2);
#pragma unroll
    for (int v = 0; v < N; ++v) store_bf16(q, at + row(v) * win.cols, value(v) * rate);
  }
}

// The same for N rows from r0 on of columns c and c + 1, where rows have an even number of columns and both are inside.
template <int N>
__device__ __forceinline__ void store_pairs(const MuItem& it, const MuWindow& win, int r0, int c, const float (&x)[2][N],
                                            float decay, float rate) {
  const int at = win.at(r0, c);
  if (it.m) {
    const __amdgpu_buffer_rsrc_t p = win.of(it.p, 4);
    float y[2][N];
#pragma unroll
    for (int v = 0; v < N; ++v) {
      const auto t = __builtin_amdgcn_raw_buffer_load_b64(p, (at + v * win.cols) * 4, 0, 0);
      y[0][v] = __uint_as_float(t[0]);
      y[1][v] = __uint_as_float(t[1]);
    }
#pragma unroll
    for (int v = 0; v < N; ++v) {
      for (int j = 0; j < 2; ++j) y[j][v] = fmaf(-x[j][v], rate, y[j][v] * decay);
      decltype(__builtin_amdgcn_raw_buffer_load_b64(p, 0, 0, 0)) t;
      t[0] = __float_as_uint(y[0][v]);
      t[1] = __float_as_uint(y[1][v]);
      __builtin_amdgcn_raw_buffer_store_b64(t, p, (at + v * win.cols) * 4, 0, 0);
    }
    if (it.copy) {
      const __amdgpu_buffer_rsrc_t q = win.of(it.copy, 2);
#pragma unroll
      for (int v = 0; v < N; ++v)
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf2(y[0][v], y[1][v]), q, (at + v * win.cols) * 2, 0, 0);
    }
  } else {
    const __amdgpu_buffer_rsrc_t q = win.of(it.p, 2);
#pragma unroll
    for (int v = 0; v < N; ++v)
      __builtin_amdgcn_raw_buffer_store_b32(pack_bf2(x[0][v] * rate, x[1][v] * rate), q, (at + v * win.cols) * 2, 0, 0);
  }
}

// ---- X_0 ------------------------------------------------------------------------------------------
// 64 x 64 elements a workgroup, written as they lie and turned, zeros in the padding.
__global__ __launch_bounds__(256) void k_muon_start(MuArgs a) {
  if (left_out(a)) return;
  if (int(blockIdx.x) >= a.first[a.count]) return;
  const int t = find_item(a, blockIdx.x);
  const MuItem& it = a.item[t];
  const MuBuffers b(it.rows, it.cols);
  const int tc = b.cols / 64, per = (b.rows / 64) * tc, q = blockIdx.x - a.first[t], e = q / per;
  const int r0 = (q % per) / tc * 64, c0 = (q % per) % tc * 64;
  const int64_t size = int64_t(it.rows) * it.cols;
  uint8_t* ws = it.ws + e * align_up(b.bytes(), 256);
  const int parts = int(cdiv(size, mu_chunk(size)));
  double sum = int(threadIdx.x) < parts ? b.parts(ws)[threadIdx.x] : 0.0;
  __shared__ double s[4];
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double norm = sqrt(s[0] + s[1] + s[2] + s[3]) + a.eps;
  const float clip = clip_factor(a), lift = mu_lift(norm), f = float(double(mu_scale(it.rows, it.cols)) / (norm * lift));
  __shared__ _Float16 tile[64][66];
  const bool turn = b.turned(it);
  _Float16 *hs = b.s(ws, turn, 0), *ht = b.t(ws, turn, 0);
  uint8_t* lo = b.lo(ws);
  const int c = threadIdx.x & 63;
  const int wv = threadIdx.x >> 6;
  const MuWindow win(it, (it.e0 + e) * size + int64_t(r0) * it.cols, min(64, max(0, it.rows - r0)));
  const auto row = [](int k) { return 4 * k; };
  float g[16], m[16];
  load_gradients<16>(a, it, win, wv, c0 + c, row, g);
  if (it.m) {
    const __amdgpu_buffer_rsrc_t rm = win.of(it.m, 4);
#pragma unroll
    for (int k = 0; k < 16; ++k) m[k] = load_f32(rm, win.at(wv, c0 + c) + 4 * k * it.cols);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int r = wv + 4 * k;
    float u = g[k] * clip;
    if (it.m) u = a.nesterov ? fmaf(a.mu, m[k], u) : m[k];
    const float x = u * lift * f;
    const _Float16 h = to_half(x);
    const int64_t at = int64_t(r0 + r) * b.cols + c0 + c;
    hs[at] = h;
    lo[at] = uint8_t(low_bits(x, h));
    tile[r][c] = h;
  }
  __syncthreads();
#pragma unroll 4
  for (int r = threadIdx.x >> 6; r < 64; r += 4) ht[int64_t(c0 + r) * b.rows + r0 + c] = tile[c][r];
}

// ---- products -------------------------------------------------------------------------------------
// WA x WB waves of FA x 2 blocks of 32 x 32; both operands' rows have the sum's axis contiguous.
//
// Which rows of the operands make a block is chosen for the results, which a lane holds as 4 consecutive rows of one
// column in each quarter q of each block. Block j of the second operand takes rows 2 l + j of the wave's 64, so a lane has
// two neighbouring columns, and a row of 32 lanes is a whole cache line of fp16. Block i of the first takes rows
// q 8 FA + h 4 FA + 4 i + u (lane l = 8 q + 4 h + u), so a lane's FA blocks are runs of 4 FA rows, whole 16 bytes of the
// transpose. In LDS a wave's share lies block by block, so that lanes read rows that follow one another: the loads that fill it
// take the rows in that order (in the matrix's order, lanes two rows apart halve the reads' rate: X X^T of 12 matrices of 2048 x
// 7168 took 425 us instead of 410).
template <int WA_, int WB_, int FA_>
struct MuShape {
  static constexpr int WA = WA_, WB = WB_, FA = FA_, FB = 2;
  static constexpr int kRun = 4 * FA;
  static_assert(FA == 2 || FA == 4);
  // First row (in the wave's share) of the results of quarter q in this half of the lanes.
  static __device__ __forceinline__ int result_row(int q, int half) { return q * 2 * kRun + half * kRun; }
  // The rows of a tile that lie in run `run` of 8 rows in LDS: the first one, and the x-th's distance from it.
  static __device__ __forceinline__ int run_a(int run) {
    return run / (4 * FA) * FA * 32 + (run & 3) * 2 * kRun + run / 4 % FA * 4;
  }
  static __device__ __forceinline__ int in_run_a(int x) { return (x >> 2) * kRun + (x & 3); }
  static __device__ __forceinline__ int run_b(int run) { return run / 8 * 64 + (run & 3) * 16 + (run >> 2 & 1); }
  static __device__ __forceinline__ int in_run_b(int x) { return 2 * x; }
  static constexpr int kWaves = WA * WB, kA = WA * FA * 32, kB = WB * FB * 32;
  struct Lds {
    uint8_t a[2][kA * kStageRowBytes];
    uint8_t b[2][kB * kStageRowBytes];
  };
};

// Part `part` of 4 of a wave's share of a stage: run `run` of 8 rows, 128 bytes each. `lane_off` holds the lane's row and
// chunk in an even run, `first` is the run's first row.
__device__ __forceinline__ void issue_f16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int lane_off, int first, int run, int stride,
                                          int kt) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      r, (lds_void*)(lds + run * 8 * kStageRowBytes), 16,
      (lane_off ^ (run & 1) * 16) + (first * stride + kt * kStageRowBytes), 0, 0, 0);
}

// acc = A B^T over k halves (a multiple of 128) of rows of `stride` halves; rows past na, nb count as zeros.
//
// Stages of 64 halves a row are double-buffered in LDS and cut into 4 slices, whose operands are read while the slice
// before is multiplied. The barrier of a stage stands before its last slice's products: then the next stage has
// arrived, and this one's buffer takes the stage after the next, a quarter at a time over four slices (in one run the
// loads hold the waves up).
template <class S>
__device__ __forceinline__ void tile_f16(typename S::Lds& sm, const _Float16* a, int na, const _Float16* b, int nb, int k,
                                         f32x16 (&acc)[S::FA][S::FB]) {
  const int lane = threadIdx.x & 63, w = wave_id(), wa = w / S::WB, wb = w % S::WB, half = lane >> 5, l32 = lane & 31;
#pragma unroll
  for (int i = 0; i < S::FA; ++i)
#pragma unroll
    for (int j = 0; j < S::FB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  const int stride = k * 2, ksteps = stride / kStageRowBytes;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a, int64_t(na) * stride), rb = make_rsrc(b, int64_t(nb) * stride);
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  const int off_a = S::in_run_a(lane >> 3) * stride + chunk, off_b = S::in_run_b(lane >> 3) * stride + chunk;
  static_assert(S::kA == S::kWaves * 32 && S::kB == S::kWaves * 32, "four runs a wave");
  const auto issue = [&](int kt, int part) {   // (past the last stage, the last once more for nothing)
    const int buf = kt & 1, run = w * 4 + part;
    kt = min(kt, ksteps - 1);
    issue_f16(ra, sm.a[buf], off_a, S::run_a(run), run, stride, kt);
    issue_f16(rb, sm.b[buf], off_b, S::run_b(run), run, stride, kt);
  };
  f16x8 fa[2][S::FA], fb[2][S::FB];
  const auto load = [&](int f, int buf, int kk) {
#pragma unroll
    for (int i = 0; i < S::FA; ++i)
      fa[f][i] = *reinterpret_cast<const f16x8*>(sm.a[buf] + swz((wa * S::FA + i) * 32 + l32, kk * 2 + half));
#pragma unroll
    for (int j = 0; j < S::FB; ++j)
      fb[f][j] = *reinterpret_cast<const f16x8*>(sm.b[buf] + swz((wb * 2 + j) * 32 + l32, kk * 2 + half));
  };
#pragma unroll
  for (int q = 0; q < 4; ++q) issue(0, q);
  issue(1, 0);
  issue(1, 1);
  wait_vmem();
  __syncthreads();
  load(0, 0, 0);
  for (int kt = 0; kt < ksteps; ++kt) {
    const int cur = kt & 1;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      __builtin_amdgcn_sched_barrier(0);
      if (kk < 3) {
        load((kk + 1) & 1, cur, kk + 1);
      } else {
        wait_vmem();
        __syncthreads();
        load(0, cur ^ 1, 0);   // (in the last stage what is read is not used)
      }
      if (kk < 2) issue(kt + 1, 2 + kk);
      if (kk == 3) {
        issue(kt + 2, 0);
        issue(kt + 2, 1);
      }
#pragma unroll
      for (int i = 0; i < S::FA; ++i)
#pragma unroll
        for (int j = 0; j < S::FB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[kk & 1][i], fb[kk & 1][j], acc[i][j], 0, 0, 0);
      // one operand read between products
      constexpr int kReads = S::FA + S::FB, kProducts = S::FA * S::FB;
#pragma unroll
      for (int q = 0; q < kReads; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
      }
      if constexpr (kProducts > kReads) __builtin_amdgcn_sched_group_barrier(0x008, kProducts - kReads, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vmem();   // (loads into LDS do not outlive the workgroup)
}

// The tile that a workgroup takes: those of one XCD follow one another (they share operands); -1: none.
__device__ __forceinline__ int xcd_tile(int total) {
  const int run = (total + kXcds - 1) / kXcds, in = blockIdx.x / kXcds, id = blockIdx.x % kXcds * run + in;
  return in < run && id < total ? id : -1;
}

// Tile number q of the lower triangle, rows first: (0,0), (1,0), (1,1), (2,0), ...
__device__ __forceinline__ void triangle(int q, int& i, int& j) {
  i = int((sqrtf(8.f * q + 1.f) - 1.f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= q) ++i;
  while (i * (i + 1) / 2 > q) --i;
  j = q - i * (i + 1) / 2;
}

// SECOND false: A = X X^T; true: B = b A + c A A. Both symmetric: tiles with i >= j, written twice.
template <class S, bool SECOND>
__global__ __launch_bounds__(S::kWaves * 64, 2) void k_muon_gram(MuArgs a) {
  static_assert(S::kA == S::kB, "square tiles");
  if (left_out(a)) return;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  typename S::Lds& sm = *reinterpret_cast<typename S::Lds*>(smem);
  const int id = xcd_tile(a.first[a.count]);
  if (id < 0) return;
  const int t = find_item(a, id);
  const MuItem& it = a.item[t];
  const MuBuffers b(it.rows, it.cols);
  const int T = (b.m + S::kA - 1) / S::kA, per = T * (T + 1) / 2, q = id - a.first[t], e = q / per;
  uint8_t* ws = it.ws + e * align_up(b.bytes(), 256);
  int ti, tj;
  triangle(q % per, ti, tj);
  const bool turn = b.turned(it);
  const int i0 = ti * S::kA, j0 = tj * S::kA, ni = min(S::kA, b.m - i0), nj = min(S::kA, b.m - j0);
  const int k = SECOND ? b.m : b.n;
  const _Float16* x = SECOND ? b.a(ws) : turn ? b.t(ws, turn, a.flip) : b.s(ws, turn, a.flip);
  f32x16 acc[S::FA][S::FB];
  tile_f16<S>(sm, x + int64_t(i0) * k, ni, x + int64_t(j0) * k, nj, k, acc);
  const float scale = mu_scale(it.rows, it.cols), down = 1.f / (scale * scale);
  const _Float16* old = b.a(ws);
  _Float16* out = SECOND ? b.b(ws) : b.a(ws);
  const int tid = tile_tid(), lane = tid & 63, w = tid >> 6, wa = w / S::WB, wb = w % S::WB, half = lane >> 5;
  // (padded sizes are multiples of 128, which a wave's share does not cross)
  if (wa * S::FA * 32 >= ni || wb * 64 >= nj) return;
  const int c = j0 + wb * 64 + 2 * (lane & 31);
  const float* da = b.diagonal(ws, false);
  float* diagonal = b.diagonal(ws, SECOND);
  float dc[2] = {0.f, 0.f};
  if constexpr (SECOND) {
    dc[0] = da[c];
    dc[1] = da[c + 1];
  }
#pragma unroll
  for (int p = 0; p < S::kRun / 2; ++p) {   // 8 rows at a time
    const int v0 = p * 8 % S::kRun, q = p * 8 / S::kRun, r0 = i0 + wa * S::FA * 32 + S::result_row(q, half) + v0;
    const int64_t at = int64_t(r0) * b.m + c;
    f16x2 z[8];
    float dr[8];
    if constexpr (SECOND)
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        z[v] = *reinterpret_cast<const f16x2*>(old + at + v * b.m);
        dr[v] = da[r0 + v];
      }
    _Float16 y[2][8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float g = acc[(v0 + v) >> 2][j][4 * q + (v & 3)];
        const bool on = ti == tj && r0 + v == c + j;   // (where the matrix in fp16 holds zero)
        float f;
        if constexpr (SECOND) {
          const float x = on ? dr[v] : float(z[v][j]);
          f = fmaf(a.c, fmaf(on ? x : dr[v] + dc[j], x, g), a.b * x);
        } else {
          f = g * down;
        }
        y[j][v] = to_half(on ? 0.f : f);
        if (on) diagonal[c + j] = f;
      }
      *reinterpret_cast<f16x2*>(out + at + v * b.m) = f16x2{y[0][v], y[1][v]};
    }
    if (ti != tj)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<f16x8*>(out + int64_t(c + j) * b.m + r0) = *reinterpret_cast<const f16x8*>(y[j]);
  }
}

// X <- a X + B X, as the parameters lie; LAST: the update of the parameters (or the output) by it instead.
template <class S, bool LAST>
__global__ __launch_bounds__(S::kWaves * 64, 2) void k_muon_apply(MuArgs a) {
  if (left_out(a)) return;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  typename S::Lds& sm = *reinterpret_cast<typename S::Lds*>(smem);
  const int id = xcd_tile(a.first[a.count]);
  if (id < 0) return;
  const int t = find_item(a, id);
  const MuItem& it = a.item[t];
  const MuBuffers b(it.rows, it.cols);
  const int tr = (b.rows + S::kA - 1) / S::kA, tc = (b.cols + S::kB - 1) / S::kB, per = tr * tc;
  const int q = id - a.first[t], e = q / per;
  uint8_t* ws = it.ws + e * align_up(b.bytes(), 256);
  int ti, tj;
  tile_coords(q % per, tr, tc, ti, tj);
  const bool turn = b.turned(it);
  const int i0 = ti * S::kA, j0 = tj * S::kB, ni = min(S::kA, b.rows - i0), nj = min(S::kB, b.cols - j0);
  const _Float16* hi = b.s(ws, turn, a.flip);
  // the result's rows times its columns: B X, or X B where X is turned
  const _Float16* left = turn ? hi : b.b(ws);
  const _Float16* right = turn ? b.b(ws) : b.t(ws, turn, a.flip);
  f32x16 acc[S::FA][S::FB];
  tile_f16<S>(sm, left + int64_t(i0) * b.m, ni, right + int64_t(j0) * b.m, nj, b.m, acc);
  const int tid = tile_tid(), lane = tid & 63, w = tid >> 6, wa = w / S::WB, wb = w % S::WB, half = lane >> 5;
  const double lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float decay = float(1.0 - lr * a.weight_decay), scale = mu_scale(it.rows, it.cols);
  const float rate = it.m ? float(lr * it.adjust / scale) : 1.f / scale;
  const MuWindow win(it, (int64_t(it.e0 + e) * it.rows + i0) * it.cols, min(ni, max(0, it.rows - i0)));
  _Float16 *hs = b.s(ws, turn, a.flip ^ 1), *ht = b.t(ws, turn, a.flip ^ 1);
  uint8_t* lo = b.lo(ws);
  if (wa * S::FA * 32 >= ni || wb * 64 >= nj) return;   // (padded sizes are multiples of 128)
  const int wc = wb * 64 + 2 * (lane & 31), c = j0 + wc;
  const bool pairs = j0 + S::kB <= it.cols && it.cols % 2 == 0;
  const float* diagonal = b.diagonal(ws, true);   // along the side of m
  const float dc[2] = {turn ? diagonal[c] : 0.f, turn ? diagonal[c + 1] : 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int wr = wa * S::FA * 32 + S::result_row(q, half), r0 = i0 + wr;
    f16x2 xh[S::kRun];
    float dr[S::kRun];
#pragma unroll
    for (int v = 0; v < S::kRun; ++v) dr[v] = turn ? 0.f : diagonal[r0 + v];
    uint16_t xl[S::kRun];
#pragma unroll
    for (int v = 0; v < S::kRun; ++v) {
      const int64_t at = int64_t(r0 + v) * b.cols + c;
      xh[v] = *reinterpret_cast<const f16x2*>(hi + at);
      xl[v] = *reinterpret_cast<const uint16_t*>(lo + at);
    }
    float x[2][S::kRun];
#pragma unroll
    for (int v = 0; v < S::kRun; ++v)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[j][v] = fmaf(a.a, with_low(xh[v][j], int8_t(xl[v] >> (8 * j))),
                       fmaf(turn ? dc[j] : dr[v], float(xh[v][j]), acc[v >> 2][j][4 * q + (v & 3)]));
    if constexpr (LAST) {
      if (pairs) {
        store_pairs<S::kRun>(it, win, wr, c, x, decay, rate);
      } else {
        const auto row = [](int v) { return v; };
#pragma unroll
        for (int j = 0; j < 2; ++j) store_results<S::kRun>(it, win, wr, c + j, row, [&](int v) { return x[j][v]; }, decay, rate);
      }
    } else {
      _Float16 y[2][S::kRun];
#pragma unroll
      for (int v = 0; v < S::kRun; ++v) {
        const int64_t at = int64_t(r0 + v) * b.cols + c;
        int low[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          y[j][v] = to_half(x[j][v]);
          low[j] = low_bits(x[j][v], y[j][v]);
        }
        *reinterpret_cast<f16x2*>(hs + at) = f16x2{y[0][v], y[1][v]};
        *reinterpret_cast<uint16_t*>(lo + at) = uint16_t((low[0] & 0xFF) | low[1] << 8);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < S::kRun; v += 8)
          *reinterpret_cast<f16x8*>(ht + int64_t(c + j) * b.rows + r0 + v) = *reinterpret_cast<const f16x8*>(&y[j][v]);
    }
  }
}

struct MuSteps {
  int32_t count;
  float coef[16][3];
};

// ---- matrices with up to 32 rows or columns -------------------------------------------------------
// Rounding to fp16 averages out over many directions; of a few, each is off by up to 1e-2. A = u u^T is small here, so
// the steps are taken on it alone, in fp64 on the matrix cores, and u is read twice whatever their number:
//   Q = a + b A + c A A,   P <- Q P,   A <- Q A Q,   X = P u / (|u| + eps),   |u|^2 the trace of the first A.
// Errors of A grow by a^2 a step where X is small: 12^4 in five steps, 1e-12 in fp64. Up to kThinElements, one workgroup
// keeps u in LDS and does it all (8 x 128: 13 us, 32 x 250: 27 us, of which two thirds are the steps, latency); longer ones take
// three launches (32 x 5,000: 46 us, 2 x 50,000: 40 us; the general kernels' 17 take 170 to 200 us there). One workgroup for
// 8,000 columns took 57 us, three launches take 27 us.
constexpr int kThin = 32, kThinRow = kThin + 1, kThinMatrix = kThin * kThinRow;   // doubles
constexpr int kThinElements = 8192, kThinColumns = 1024;                         // of u in one workgroup, at most
constexpr int kThinParts = 128;                                                  // partial sums of A at most
constexpr int kThinChunk = 2048;                                                 // elements of a chunk: 64 to 512 columns

typedef __attribute__((ext_vector_type(4))) double f64x4;

struct ThinShape {
  int m, n, stride;          // rows and columns of u as it lies in LDS, and a row's length there
  int columns, chunks, parts;
  __host__ __device__ ThinShape(int rows, int cols) {
    m = rows < cols ? rows : cols;
    n = rows < cols ? cols : rows;
    columns = kThinChunk / (m < 4 ? 4 : m) & ~15;
    chunks = int(cdiv(n, columns));
    parts = chunks < kThinParts ? chunks : kThinParts;
    stride = columns | 1;
  }
  __host__ __device__ bool thin() const { return m <= kThin; }
  __host__ __device__ bool fits() const { return thin() && n <= kThinColumns && m * n <= kThinElements; }
  __host__ __device__ int64_t bytes() const { return int64_t(parts + 1) * m * m * 8; }   // partial sums, P
  __host__ __device__ int chunk_lds() const { return kThinMatrix * 8 + m * stride * 4; }
};

// Calls use(elements, their places in LDS, how many of them) for the columns j0 .. j0 + cols - 1, 8 elements a
// thread at a time, so that their loads are in flight together. Elements past the last one are the first once more.
template <int THREADS, class U>
__device__ __forceinline__ void thin_elements(const MuItem& it, int64_t base, int m, int stride, int j0, int cols, U&& use) {
  const bool turn = it.rows > it.cols;
  const int inner = turn ? m : cols, total = m * cols, dq = THREADS / inner, dr = THREADS % inner;
  int q = threadIdx.x / inner, r = threadIdx.x % inner;
  for (int e = threadIdx.x; e < total; e += 8 * THREADS) {
    int64_t i[8];
    int at[8], count = 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const bool in = e + v * THREADS < total;
      i[v] = in ? base + (turn ? int64_t(j0) * m + e + v * THREADS : int64_t(q) * it.cols + j0 + r) : base;
      at[v] = turn ? r * stride + q : q * stride + r;
      count += in;
      q += dq;
      r += dr;
      if (r >= inner) r -= inner, ++q;
    }
    use(i, at, count);
  }
}

template <int THREADS, bool UPDATE>
__device__ __forceinline__ void thin_load(const MuArgs& a, const MuItem& it, int64_t base, int m, int stride, int j0, int cols,
                                          float* u) {
  const float clip = clip_factor(a);
  thin_elements<THREADS>(it, base, m, stride, j0, cols, [&](const int64_t (&i)[8], const int (&at)[8], int count) {
    float g[8], mm[8];
    if (a.gbf) {
#pragma unroll
      for (int v = 0; v < 8; ++v) g[v] = element(it.g, true, i[v]);
    } else {
#pragma unroll
      for (int v = 0; v < 8; ++v) g[v] = element(it.g, false, i[v]);
    }
    if (it.m) {
#pragma unroll
      for (int v = 0; v < 8; ++v) mm[v] = it.m[i[v]];
    }
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (v < count) {
        float x = g[v] * clip;
        if (it.m) {
          if constexpr (UPDATE) it.m[i[v]] = mm[v] = fmaf(mm[v], a.mu, x);
          x = a.nesterov ? fmaf(a.mu, mm[v], x) : mm[v];
        }
        u[at[v]] = x;
      }
  });
}

// The update (or the output) by the results in LDS.
template <int THREADS>
__device__ __forceinline__ void thin_store(const MuArgs& a, const MuItem& it, int64_t base, int m, int stride, int j0, int cols,
                                           const float* u) {
  const double lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float decay = float(1.0 - lr * a.weight_decay), rate = float(lr * it.adjust);
  thin_elements<THREADS>(it, base, m, stride, j0, cols, [&](const int64_t (&i)[8], const int (&at)[8], int count) {
    float* p = static_cast<float*>(it.p);
    float y[8];
    if (it.m)
#pragma unroll
      for (int v = 0; v < 8; ++v) y[v] = p[i[v]];
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (v < count) {
        const float x = u[at[v]];
        if (it.m) {
          p[i[v]] = y[v] = fmaf(-x, rate, y[v] * decay);
          if (it.copy) it.copy[i[v]] = f2bf(y[v]);
        } else {
          static_cast<uint16_t*>(it.p)[i[v]] = f2bf(x);
        }
      }
  });
}

// The lane's part of a 16 x 16 product in fp64: operands' row (or column) lane % 16 at k = lane / 16 of 4; element i of
// a result is in row 4 i + lane / 16, column lane % 16.
__device__ __forceinline__ f64x4 thin_mfma(double x, double y, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(x, y, c, 0, 0, 0);
}

// acc += u u^T over the columns in LDS, blocks (0, 0), (1, 0) and (1, 1); each wave takes every WAVES-th 16 columns, in two
// sums, so that neither loads nor instructions wait for one another.
template <int WAVES>
__device__ __forceinline__ void thin_gram(const float* u, int m, int stride, int cols, f64x4 (&acc)[2][3]) {
  const int lane = threadIdx.x & 63, r = lane & 15;
  const float *ur = u + min(r, m - 1) * stride, *ul = u + min(r + 16, m - 1) * stride;
  for (int k0 = wave_id() * 16; k0 < cols; k0 += WAVES * 16) {
    float x[4], y[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = ur[min(k0 + 4 * v + (lane >> 4), cols - 1)];
    if (m > 16) {
#pragma unroll
      for (int v = 0; v < 4; ++v) y[v] = ul[min(k0 + 4 * v + (lane >> 4), cols - 1)];
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const bool in = k0 + 4 * v + (lane >> 4) < cols;
      const double a = in && r < m ? double(x[v]) : 0.0;
      acc[v & 1][0] = thin_mfma(a, a, acc[v & 1][0]);
      if (m > 16) {
        const double b = in && r + 16 < m ? double(y[v]) : 0.0;
        acc[v & 1][1] = thin_mfma(b, a, acc[v & 1][1]);
        acc[v & 1][2] = thin_mfma(b, b, acc[v & 1][2]);
      }
    }
  }
}

// Adds the waves' blocks up in LDS, one wave after another, so that the order is always the same.
template <int WAVES>
__device__ __forceinline__ void thin_gather(const f64x4 (&parts)[2][3], int m, double* sum) {
  const f64x4 acc[3] = {parts[0][0] + parts[1][0], parts[0][1] + parts[1][1], parts[0][2] + parts[1][2]};
  const int lane = threadIdx.x & 63, c = lane & 15, w = wave_id();
  for (int t = 0; t < WAVES; ++t) {
    if (t == w)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 4);
        const auto add = [&](int row, int col, double v) {
          double& d = sum[row * kThinRow + col];
          d = t ? d + v : v;
        };
        add(r, c, acc[0][i]);
        if (m > 16) {
          add(r + 16, c, acc[1][i]);
          add(c, r + 16, acc[1][i]);
          add(r + 16, c + 16, acc[2][i]);
        }
      }
    __syncthreads();
  }
}

// From A = u u^T in LDS: P / (|u| + eps) in `p`. Eight waves; `q` is scratch. The matrices are symmetric (and polynomials of
// one matrix), so an operand's columns are read as its rows. TILES: 16 x 16 blocks along a side.
template <int TILES>
__device__ __forceinline__ void thin_steps(const MuSteps& st, double eps, int m, double* a, double* q, double* p) {
  const int lane = threadIdx.x & 63, c = lane & 15, w = wave_id(), ti = (w & 3) >> 1, tj = w & 1;
  const bool mine = ti < TILES && tj < TILES;
  double norm = lane < m ? a[lane * kThinRow + lane] : 0.0;
  for (int off = 16; off; off >>= 1) norm += __shfl_xor(norm, off, 64);
  norm = 1.0 / (sqrt(__shfl(norm, 0, 64)) + eps);
  __syncthreads();
  for (int i = threadIdx.x; i < TILES * 16 * kThinRow; i += 512) a[i] *= norm * norm;
  __syncthreads();
  const auto product = [&](const double* x, const double* y) {
    const double *xr = x + (ti * 16 + c) * kThinRow + (lane >> 4), *yr = y + (tj * 16 + c) * kThinRow + (lane >> 4);
    double fx[TILES * 4], fy[TILES * 4];
#pragma unroll
    for (int k = 0; k < TILES * 4; ++k) fx[k] = xr[4 * k], fy[k] = yr[4 * k];
    f64x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};   // (two sums: an instruction does not wait for the one before)
#pragma unroll
    for (int k = 0; k < TILES * 4; ++k) s[k & 1] = thin_mfma(fx[k], fy[k], s[k & 1]);
    return s[0] + s[1];
  };
  const auto place = [&](int i) { return (ti * 16 + 4 * i + (lane >> 4)) * kThinRow + tj * 16 + c; };
  const auto put = [&](double* x, const f64x4& s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[place(i)] = s[i];
  };
  f64x4 s;
  for (int k = 0; k < st.count; ++k) {
    const double ca = st.coef[k][0], cb = st.coef[k][1], cc = st.coef[k][2];
    if (mine && w < 4) {
      s = product(a, a);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool diagonal = ti == tj && 4 * i + (lane >> 4) == c;
        s[i] = (diagonal ? ca : 0.0) + cb * a[place(i)] + cc * s[i];
      }
      put(q, s);
    }
    __syncthreads();
    const bool more = k + 1 < st.count;
    if (mine && w < 4 && more) s = product(q, a);
    if (mine && w >= 4) s = k ? product(p, q) : f64x4{q[place(0)], q[place(1)], q[place(2)], q[place(3)]};
    __syncthreads();
    if (mine && w < 4 && more) put(a, s);
    if (mine && w >= 4) put(p, more ? s : s * norm);
    __syncthreads();
    if (more) {
      if (mine && w < 4) s = product(a, q);
      __syncthreads();
      if (mine && w < 4) put(a, s);
      __syncthreads();
    }
  }
}
__device__ __forceinline__ void thin_steps(const MuSteps& st, double eps, int m, double* a, double* q, double* p) {
  if (m > 16) thin_steps<2>(st, eps, m, a, q, p);
  else thin_steps<1>(st, eps, m, a, q, p);
}

// u <- P u, for the columns in LDS; a wave takes 64 at a time, as four operands of 16.
template <int WAVES>
__device__ __forceinline__ void thin_apply(const double* p, float* u, int m, int stride, int cols) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  for (int j0 = wave_id() * 64; j0 < cols; j0 += WAVES * 64) {
    f64x4 s[4][2] = {};
    for (int k = lane >> 4; k < (m + 3 & ~3); k += 4) {
      float x[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) x[g] = u[min(k, m - 1) * stride + min(j0 + 16 * g + c, cols - 1)];
      const double p0 = p[c * kThinRow + k], p1 = p[(c + 16) * kThinRow + k];   // (rows past m are not used)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const double b = k < m ? double(x[g]) : 0.0;   // (P's columns past m are zero but for its diagonal)
        s[g][0] = thin_mfma(p0, b, s[g][0]);
        if (m > 16) s[g][1] = thin_mfma(p1, b, s[g][1]);
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (const int j = j0 + 16 * g + c; j < cols)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 4);
          if (r < m) u[r * stride + j] = float(s[g][i >> 2][i & 3]);
        }
  }
}

// All of it in one workgroup of eight waves.
__device__ __forceinline__ void muon_thin(const MuArgs& a, const MuSteps& st, const MuItem& it, int e) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  double *sum = reinterpret_cast<double*>(smem), *q = sum + kThinMatrix, *p = q + kThinMatrix;
  float* u = reinterpret_cast<float*>(p + kThinMatrix);
  const ThinShape sh(it.rows, it.cols);
  const int64_t base = int64_t(it.e0 + e) * it.rows * it.cols;
  const int stride = sh.n | 1;
  thin_load<512, true>(a, it, base, sh.m, stride, 0, sh.n, u);
  __syncthreads();
  f64x4 acc[2][3] = {};
  thin_gram<8>(u, sh.m, stride, sh.n, acc);
  thin_gather<8>(acc, sh.m, sum);
  thin_steps(st, a.eps, sh.m, sum, q, p);
  thin_apply<8>(p, u, sh.m, stride, sh.n);
  __syncthreads();
  thin_store<512>(a, it, base, sh.m, stride, 0, sh.n, u);
}

// Partial sums of A: part `blockIdx`'s chunks, every parts-th one; with a momentum, also its update.
__global__ __launch_bounds__(256) void k_thin_gram(MuArgs a) {
  if (left_out(a)) return;
  if (int(blockIdx.x) >= a.first[a.count]) return;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  double* sum = reinterpret_cast<double*>(smem);
  float* u = reinterpret_cast<float*>(sum + kThinMatrix);
  const int t = find_item(a, blockIdx.x);
  const MuItem& it = a.item[t];
  const ThinShape sh(it.rows, it.cols);
  const int id = blockIdx.x - a.first[t], e = id / sh.parts, part = id % sh.parts;
  const int64_t base = int64_t(it.e0 + e) * it.rows * it.cols;
  f64x4 acc[2][3] = {};
  for (int c = part; c < sh.chunks; c += sh.parts) {
    const int j0 = c * sh.columns, cols = min(sh.columns, sh.n - j0);
    thin_load<256, true>(a, it, base, sh.m, sh.stride, j0, cols, u);
    __syncthreads();
    thin_gram<4>(u, sh.m, sh.stride, cols, acc);
    __syncthreads();
  }
  thin_gather<4>(acc, sh.m, sum);
  double* out = reinterpret_cast<double*>(it.ws + e * align_up(sh.bytes(), 256)) + int64_t(part) * sh.m * sh.m;
  for (int i = threadIdx.x; i < sh.m * sh.m; i += 256) out[i] = sum[i / sh.m * kThinRow + i % sh.m];
}

// P of each matrix, from its partial sums.
__global__ __launch_bounds__(512) void k_thin_steps(MuArgs a, MuSteps st) {
  if (left_out(a)) return;
  if (int(blockIdx.x) >= a.first[a.count]) return;
  __shared__ double sum[kThinMatrix], q[kThinMatrix], p[kThinMatrix];
  const int t = find_item(a, blockIdx.x), e = blockIdx.x - a.first[t];
  const MuItem& it = a.item[t];
  const ThinShape sh(it.rows, it.cols);
  double* ws = reinterpret_cast<double*>(it.ws + e * align_up(sh.bytes(), 256));
  const int mm = sh.m * sh.m;
  for (int i = threadIdx.x; i < kThinMatrix; i += 512) sum[i] = 0;
  __syncthreads();
  constexpr int kAhead = 16;   // parts loaded together, added in order
  double v[2] = {0, 0};        // of elements threadIdx and threadIdx + 512
  for (int part = 0; part < sh.parts; part += kAhead) {
    double x[2][kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[h][k] = ws[int64_t(min(part + k, sh.parts - 1)) * mm + min(int(threadIdx.x) + 512 * h, mm - 1)];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] += part + k < sh.parts ? x[h][k] : 0.0;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (const int i = threadIdx.x + 512 * h; i < mm) sum[i / sh.m * kThinRow + i % sh.m] = v[h];
  __syncthreads();
  thin_steps(st, a.eps, sh.m, sum, q, p);
  for (int i = threadIdx.x; i < mm; i += 512) ws[int64_t(sh.parts) * mm + i] = p[i / sh.m * kThinRow + i % sh.m];
}

// The results, a chunk a workgroup.
__global__ __launch_bounds__(256) void k_thin_apply(MuArgs a) {
  if (left_out(a)) return;
  if (int(blockIdx.x) >= a.first[a.count]) return;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  double* p = reinterpret_cast<double*>(smem);
  float* u = reinterpret_cast<float*>(p + kThinMatrix);
  const int t = find_item(a, blockIdx.x);
  const MuItem& it = a.item[t];
  const ThinShape sh(it.rows, it.cols);
  const int id = blockIdx.x - a.first[t], e = id / sh.chunks, j0 = id % sh.chunks * sh.columns;
  const int cols = min(sh.columns, sh.n - j0);
  const int64_t base = int64_t(it.e0 + e) * it.rows * it.cols;
  const double* ws = reinterpret_cast<const double*>(it.ws + e * align_up(sh.bytes(), 256)) + int64_t(sh.parts) * sh.m * sh.m;
  for (int i = threadIdx.x; i < kThin * kThin; i += 256) {
    const int r = i / kThin, c = i % kThin;
    p[r * kThinRow + c] = r < sh.m && c < sh.m ? ws[r * sh.m + c] : 0.0;
  }
  thin_load<256, false>(a, it, base, sh.m, sh.stride, j0, cols, u);
  __syncthreads();
  thin_apply<4>(p, u, sh.m, sh.stride, cols);
  __syncthreads();
  thin_store<256>(a, it, base, sh.m, sh.stride, j0, cols, u);
}

// ---- small matrices -----------------------------------------------------------------------------
// A matrix whose X and X^T in fp16 fit the LDS beside A takes one workgroup and one launch for everything: X stays in
// registers in fp32, its fp16 copies, A and then B in LDS. Launches and the way through memory bound the general kernels at
// such sizes (25 matrices of 256 x 128 and less: 222 us in 17 launches, 56 us here).
// Vector instructions bound it (60 % of the cycles of 8 waves): conversions, addresses, and the diagonals' parts.
//
// X is cut into 32 x 32 blocks, 2..4 along its shorter side and up to 16 along the longer one. Wave w takes the
// longer side's blocks w, w + 8, ..., for each of them all of the shorter side's: four slots at most, which share the
// operand of their longer side.
struct SmallShape {
  int shorter, longer;   // blocks along the sides
  bool one_workgroup;
  __host__ __device__ SmallShape(int r, int c) : one_workgroup(ThinShape(r, c).fits()) {
    shorter = ((r < c ? r : c) + 31) / 32;
    longer = ((r < c ? c : r) + 31) / 32;
  }
  __host__ __device__ bool fits() const {
    return shorter == 1 ? one_workgroup : shorter <= 4 && (longer + 7) / 8 * shorter <= 4;
  }
};
// The longest row of the layout in LDS, in halves: that of all rows, so that addresses are constants and a row's base.
constexpr int small_long(int shorter) { return 256 * (4 / shorter); }
constexpr int small_lds(int shorter) { return (2 * 32 * shorter * small_long(shorter) + 1024 * shorter * shorter) * 2; }

// Element (row, col) of a matrix in LDS whose rows have `len` halves (128, 256, 512; 64; 96): 16-byte chunks are swapped by
// the row so that 16 rows of one chunk, which the LDS serves in a cycle, lie in different banks (rows of 256 bytes begin in the same
// one, those of 128 in every other, of 192 in every fourth).
__device__ __forceinline__ int small_turn(int row, int len) {
  return len % 128 == 0 ? row & 15 : len == 64 ? (row & 7) ^ (row >> 3 & 1) : row >> 2 & 3;
}
__device__ __forceinline__ int small_at(int row, int col, int len) {
  return row * len + (((col >> 3) ^ small_turn(row, len)) << 3) + (col & 7);
}
// The same for a lane's elements of a 32 x 32 block of results: rows row + 8 v + u (row: a multiple of 4) of one column. What a
// row adds to an address is a multiple of what turns in it, so one exclusive or and a constant make an element's from the first.
template <int LEN>
struct SmallColumn {
  uint8_t* x;
  int first;
  __device__ __forceinline__ SmallColumn(_Float16* m, int row, int col)
      : x(reinterpret_cast<uint8_t*>(m)), first((row * LEN + col) * 2 ^ small_turn(row, LEN) << 4) {}
  __device__ __forceinline__ _Float16& operator()(int v, int u) const {
    return *reinterpret_cast<_Float16*>(x + (first ^ small_turn(8 * v + u, LEN) << 4) + (8 * v + u) * LEN * 2);
  }
};
// A lane's part of a row as an operand: chunk c of it.
struct SmallRow {
  const _Float16* p;
  int turn;
  __device__ __forceinline__ SmallRow(const _Float16* x, int row, int len) : p(x + row * len), turn(small_turn(row, len)) {}
  __device__ __forceinline__ f16x8 operator()(int c) const { return *reinterpret_cast<const f16x8*>(p + ((c ^ turn) << 3)); }
};

// N results of 32 rows each, a[i] times b[i / EACH] (or in the other order), over `len` halves; the next slice's operands
// are read while one is multiplied.
template <int N, int EACH, bool SWAP>
__device__ __forceinline__ void small_products(const SmallRow* a, const SmallRow* b, int len, f32x16 (&acc)[N]) {
  const int half = (threadIdx.x & 63) >> 5;
  constexpr int M = (N + EACH - 1) / EACH;
  f16x8 fa[2][N], fb[2][M];
  const auto load = [&](int buf, int c) {
#pragma unroll
    for (int j = 0; j < M; ++j) fb[buf][j] = b[j](c + half);
#pragma unroll
    for (int i = 0; i < N; ++i) fa[buf][i] = a[i](c + half);
  };
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0.f;
  const int last = len / 8 - 2;
  load(0, 0);
#pragma unroll 1
  for (int c = 0; c <= last; c += 4)   // (two slices, as len is a multiple of 32)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load(u ^ 1, min(c + 2 * u + 2, last));
#pragma unroll
      for (int i = 0; i < N; ++i)
        acc[i] = SWAP ? __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[u][i / EACH], fa[u][i], acc[i], 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[u][i], fb[u][i / EACH], acc[i], 0, 0, 0);
    }
}

// SHORTER: blocks along the shorter side; TURN: that is the columns' side.
template <int SHORTER, bool TURN>
__device__ __forceinline__ void muon_small(const MuArgs& a, const MuSteps& st, const MuItem& it, int e) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int N = SHORTER == 3 ? 3 : 4;   // slots
  constexpr int kShort = 32 * SHORTER, kLong = small_long(SHORTER);   // rows of the matrices in LDS
  const int longer = SmallShape(it.rows, it.cols).longer, n = longer * 32;
  _Float16 *xs = reinterpret_cast<_Float16*>(smem), *xt = xs + kShort * kLong, *gram = xt + kShort * kLong;
  const int lane = threadIdx.x & 63, w = wave_id(), half = lane >> 5, l32 = lane & 31;
  const MuWindow win(it, int64_t(it.e0 + e) * it.rows * it.cols, it.rows);
  const auto row = [](int v) { return 8 * (v >> 2) + (v & 3); };
  const float scale = mu_scale(it.rows, it.cols), down = 1.f / (scale * scale), clip = clip_factor(a);
  // element v of slot q is row rq(q) + 8 (v / 4) + 4 half + v % 4, column cq(q) + l32
  const auto rq = [&](int q) { return (TURN ? w + 8 * (q / SHORTER) : q % SHORTER) * 32; };
  const auto cq = [&](int q) { return (TURN ? q % SHORTER : w + 8 * (q / SHORTER)) * 32; };
  float x[N][16];
  bool live[N];
  double sum = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    live[q] = w + 8 * (q / SHORTER) < longer;
    const int r0 = rq(q) + 4 * half, c0 = cq(q) + l32;
    float g[16], m[16];
    load_gradients<16>(a, it, win, r0, c0, row, g);
    if (it.m) {
      const __amdgpu_buffer_rsrc_t rm = win.of(it.m, 4);
      const int at = win.at(r0, c0);
#pragma unroll
      for (int v = 0; v < 16; ++v) m[v] = load_f32(rm, at + row(v) * it.cols);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        g[v] *= clip;
        m[v] = fmaf(m[v], a.mu, g[v]);
        store_f32(rm, at + row(v) * it.cols, m[v]);
        x[q][v] = a.nesterov ? fmaf(a.mu, m[v], g[v]) : m[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < 16; ++v) x[q][v] = g[v] * clip;
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) sum = fma(double(x[q][v]), double(x[q][v]), sum);
  }
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  double* sums = reinterpret_cast<double*>(gram);
  if (lane == 0) sums[w] = sum;
  __syncthreads();
  double norm = 0;
  for (int k = 0; k < 8; ++k) norm += sums[k];
  norm = sqrt(norm) + a.eps;
  const float lift = mu_lift(norm), f = float(double(scale) / (norm * lift));
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int v = 0; v < 16; ++v) x[q][v] = x[q][v] * lift * f;
  // A's blocks of the wave, 32 x 32 of SHORTER x SHORTER: number w, and of those from 8 on one in the same column.
  constexpr int G = SHORTER > 2 ? 2 : 1;
  int gr[G], gc[G];
  bool glive[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int b = q == 0 || SHORTER == 4 ? w + 8 * q : w == 8 % SHORTER ? 8 : SHORTER * SHORTER;
    glive[q] = b < SHORTER * SHORTER;
    gr[q] = glive[q] ? b / SHORTER * 32 : 0;
    gc[q] = glive[q] ? b % SHORTER * 32 : 0;
  }
  // (addresses in LDS are formed anew where they are used: hoisted out of the loop they would fill the registers)
  const auto put_gram = [&](const f32x16 (&g)[G]) {
    const int tid = tile_tid(), h = (tid >> 5) & 1, c = tid & 31;
#pragma unroll
    for (int q = 0; q < G; ++q)
      if (glive[q]) {
        const SmallColumn<kShort> column(gram, gr[q] + 4 * h, gc[q] + c);
#pragma unroll
        for (int v = 0; v < 16; ++v) column(v >> 2, v & 3) = to_half(g[q][v]);
      }
  };
  _Float16 *across_rows = TURN ? xt : xs, *along_rows = TURN ? xs : xt;   // rows of n, and of m halves
  // A's and B's diagonals, in place of the former once A is made
  float *diag_a = reinterpret_cast<float*>(across_rows), *diag_b = diag_a + kShort;
  // A wave has one block on the diagonal at most. Its lanes' elements there (of half the lanes), and their places
  int dq = -1;
#pragma unroll
  for (int q = 0; q < G; ++q)
    if (glive[q] && gr[q] == gc[q]) dq = q;
  const auto on_diagonal = [&](const f32x16 (&g)[G]) {
    const int c = tile_tid() & 31, on = (c >> 3) * 4 + (c & 3);
    float f = 0.f;
#pragma unroll
    for (int q = 0; q < G; ++q)
      if (q == dq)
#pragma unroll
        for (int v = 0; v < 16; ++v) f = v == on ? g[q][v] : f;
    return f;
  };
  const auto diagonal_place = [&] { return gc[G - 1 == dq ? G - 1 : 0] + (tile_tid() & 31); };
  const auto put_diagonal = [&](float* d, float f) {
    const int tid = tile_tid();
    if ((tid >> 2 & 1) == (tid >> 5 & 1)) d[diagonal_place()] = f;
  };
  const auto clear_diagonal = [&] {
    const int tid = tile_tid(), c = diagonal_place();
    if ((tid >> 2 & 1) == (tid >> 5 & 1)) gram[small_at(c, c, kShort)] = 0;
  };
  // four of a diagonal's elements, for elements 4 v .. 4 v + 3 of a lane in a block whose first row is r
  const auto four = [&](const float* d, int r, int v) {
    return *reinterpret_cast<const f32x4*>(d + r + 8 * v + 4 * (tile_tid() >> 5 & 1));
  };
#pragma unroll 1
  for (int k = 0; k < st.count; ++k) {
    const float ca = st.coef[k][0], cb = st.coef[k][1], cc = st.coef[k][2];
    {
      const int tid = tile_tid(), h = (tid >> 5) & 1, c = tid & 31;
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (live[q]) {
          const SmallColumn<TURN ? kShort : kLong> column(xs, rq(q) + 4 * h, cq(q) + c);
          // (rows of xt are columns of xs: four runs of 4 elements, a chunk apart)
          uint8_t* turned = reinterpret_cast<uint8_t*>(xt);
          const int first = small_at(cq(q) + c, rq(q) + 4 * h, TURN ? kLong : kShort) * 2;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            f16x4 y;
#pragma unroll
            for (int u = 0; u < 4; ++u) column(v, u) = y[u] = to_half(x[q][4 * v + u]);
            *reinterpret_cast<f16x4*>(turned + (first ^ v << 4)) = y;
          }
        }
    }
    __syncthreads();
    // A, then B in its place: the wave's blocks w and w + 8 of SHORTER x SHORTER
    f32x16 g[G];
    if (glive[0]) {
      const int l = tile_tid() & 31;
      const SmallRow left[2] = {SmallRow(across_rows, gr[0] + l, kLong), SmallRow(across_rows, gr[G - 1] + l, kLong)};
      const SmallRow right[1] = {SmallRow(across_rows, gc[0] + l, kLong)};   // (two blocks of a wave share their column)
      small_products<G, G, false>(left, right, n, g);
#pragma unroll
      for (int q = 0; q < G; ++q) g[q] *= down;
      put_gram(g);
      if (dq >= 0) clear_diagonal();
    }
    __syncthreads();
    f32x16 aa[G];
    float d = 0.f;
    if (dq >= 0) {
      d = on_diagonal(g);
      put_diagonal(diag_a, fmaf(cc, d, 0.5f * cb));   // (two of these make an element's factor)
    }
    if (glive[0]) {
      const int l = tile_tid() & 31;
      const SmallRow left[2] = {SmallRow(gram, gr[0] + l, kShort), SmallRow(gram, gr[G - 1] + l, kShort)};
      const SmallRow right[1] = {SmallRow(gram, gc[0] + l, kShort)};
      small_products<G, G, false>(left, right, kShort, aa);
    }
    __syncthreads();
    if (glive[0]) {
      const int c = tile_tid() & 31;
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const float dc = diag_a[gc[q] + c];
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          const f32x4 dr = four(diag_a, gr[q], v >> 2);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x = float(to_half(g[q][v + u]));
            g[q][v + u] = fmaf(dr[u] + dc, x, cc * aa[q][v + u]);
          }
        }
      }
      put_gram(g);
      if (dq >= 0) {
        clear_diagonal();
        put_diagonal(diag_b, fmaf(cc, fmaf(d, d, on_diagonal(aa)), cb * d));
      }
    }
    __syncthreads();
    if (live[0]) {
      const int l = tile_tid() & 31;
      const auto along = [&](int j) { return SmallRow(along_rows, min(w + 8 * j, longer - 1) * 32 + l, kShort); };
      const auto across = [&](int q) { return SmallRow(gram, q % SHORTER * 32 + l, kShort); };
      const SmallRow ra[4] = {across(0), across(1), across(2), across(3)};
      const SmallRow rb[4] = {along(0), along(1), along(2), along(3)};
      f32x16 y[N];
      small_products<N, SHORTER, TURN>(ra, rb, kShort, y);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const float dc = diag_b[q % SHORTER * 32 + l];
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          const f32x4 dr = TURN ? f32x4{dc, dc, dc, dc} : four(diag_b, q % SHORTER * 32, v >> 2);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            x[q][v + u] = fmaf(ca, x[q][v + u], fmaf(dr[u], float(to_half(x[q][v + u])), y[q][v + u]));
        }
      }
    }
    __syncthreads();
  }
  const double lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float decay = float(1.0 - lr * a.weight_decay), rate = it.m ? float(lr * it.adjust / scale) : 1.f / scale;
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (live[q]) {
      const int r0 = rq(q) + 4 * half, c = cq(q) + l32;
      store_results<16>(it, win, r0, c, row, [&](int v) { return x[q][v]; }, decay, rate);
    }
}

__global__ __launch_bounds__(512) void k_muon_small(MuArgs a, MuSteps st) {
  if (left_out(a)) return;
  const int t = find_item(a, blockIdx.x);
  const MuItem& it = a.item[t];
  const int e = blockIdx.x - a.first[t], shorter = SmallShape(it.rows, it.cols).shorter;
  if (shorter == 1) {
    muon_thin(a, st, it, e);
  } else if (it.rows > it.cols) {
    if (shorter == 2) muon_small<2, true>(a, st, it, e);
    else if (shorter == 3) muon_small<3, true>(a, st, it, e);
    else muon_small<4, true>(a, st, it, e);
  } else {
    if (shorter == 2) muon_small<2, false>(a, st, it, e);
    else if (shorter == 3) muon_small<3, false>(a, st, it, e);
    else muon_small<4, false>(a, st, it, e);
  }
}

using MuMid = MuShape<2, 2, 2>;    // 128 x 128
using MuWide = MuShape<2, 4, 4>;   // 256 x 256

template <class F>
hipError_t allow_lds(F* f, int bytes, std::atomic<bool> (&done)[kMaxDevices]) {
  return once_per_device(done, [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

// Runs `kernel` over the tiles that `tiles` counts for each item.
template <class K, class N, class... More>
hipError_t run(K* kernel, MuArgs& a, int threads, int lds, hipStream_t s, N&& tiles, const More&... more) {
  int64_t sum = 0;
  for (int t = 0; t < a.count; ++t) {
    a.first[t] = int32_t(sum);
    sum += tiles(a.item[t]) * a.item[t].batch;
  }
  a.first[a.count] = int32_t(sum);
  kernel<<<unsigned(align_up(sum, kXcds)), threads, lds, s>>>(a, more...);
  return hipGetLastError();
}

template <class S>
hipError_t steps(MuArgs& a, int count, const float* coef, hipStream_t s) {
  static std::atomic<bool> done[4][kMaxDevices];
  constexpr int lds = int(sizeof(typename S::Lds)), threads = S::kWaves * 64;
  hipError_t e = allow_lds(k_muon_gram<S, false>, lds, done[0]);
  if (e == hipSuccess) e = allow_lds(k_muon_gram<S, true>, lds, done[1]);
  if (e == hipSuccess) e = allow_lds(k_muon_apply<S, false>, lds, done[2]);
  if (e == hipSuccess) e = allow_lds(k_muon_apply<S, true>, lds, done[3]);
  const auto half = [](const MuItem& it) {
    const int64_t T = cdiv(MuBuffers(it.rows, it.cols).m, S::kA);
    return T * (T + 1) / 2;
  };
  const auto full = [](const MuItem& it) {
    const MuBuffers b(it.rows, it.cols);
    return cdiv(b.rows, S::kA) * cdiv(b.cols, S::kB);
  };
  for (int k = 0; k < count && e == hipSuccess; ++k) {
    a.a = coef[3 * k];
    a.b = coef[3 * k + 1];
    a.c = coef[3 * k + 2];
    a.flip = k & 1;
    e = run(k_muon_gram<S, false>, a, threads, lds, s, half);
    if (e == hipSuccess) e = run(k_muon_gram<S, true>, a, threads, lds, s, half);
    if (e == hipSuccess && k + 1 < count) e = run(k_muon_apply<S, false>, a, threads, lds, s, full);
    if (e == hipSuccess && k + 1 == count) e = run(k_muon_apply<S, true>, a, threads, lds, s, full);
  }
  return e;
}

// A run: matrices that go through the launches together, at most kMuItems items and as many matrices as this workspace
// holds (one at least). Tensors are cut between the matrices of their batches where a run is full.
constexpr int64_t kMuWs = int64_t(2) << 30;

struct MuPart {
  int tensor, first, count;   // matrices first .. first + count - 1 of a tensor
  int64_t ws;                 // offset of their buffers
};

enum class MuSize { Small, Thin, General };
MuSize size_of(const mok_muon_tensor& t) {
  if (SmallShape(t.rows, t.cols).fits()) return MuSize::Small;
  return ThinShape(t.rows, t.cols).thin() ? MuSize::Thin : MuSize::General;
}

// (A launch has fewer than 2^32 threads. Small ones need none; counted as 512 bytes, a run has at most 2^22 of them, a
// workgroup each. Long thin ones are counted as 256 bytes a chunk at least: 2^23 workgroups of 256 threads.)
int64_t matrix_bytes(const mok_muon_tensor& t, MuSize size) {
  if (size == MuSize::Small) return 512;
  if (size == MuSize::General) return align_up(MuBuffers(t.rows, t.cols).bytes(), 256);
  const ThinShape sh(t.rows, t.cols);
  return std::max<int64_t>(align_up(sh.bytes(), 256), sh.chunks * int64_t(256));
}

// Calls go(parts, count, bytes) for each run of the tensors of a size; stops at an error.
template <class G>
hipError_t each_run(int count, const mok_muon_tensor* t, MuSize size, G&& go) {
  MuPart part[kMuItems];
  int n = 0;
  int64_t bytes = 0;
  for (int k = 0; k < count; ++k) {
    if (size_of(t[k]) != size) continue;
    const int64_t one = matrix_bytes(t[k], size);
    for (int b = 0; b < t[k].batch;) {
      if (n == kMuItems || (n > 0 && bytes + one > kMuWs)) {
        const hipError_t e = go(part, n, bytes);
        if (e != hipSuccess) return e;
        n = 0;
        bytes = 0;
      }
      const int take = int(std::min<int64_t>(t[k].batch - b, std::max<int64_t>(1, (kMuWs - bytes) / one)));
      part[n++] = MuPart{k, b, take, bytes};
      bytes += take * one;
      b += take;
    }
  }
  return n > 0 ? go(part, n, bytes) : hipSuccess;
}

double adjustment(int rule, int rows, int cols) {
  if (rule == MOK_ADJUST_RMS) return 0.2 * std::sqrt(double(std::max(rows, cols)));
  if (rule == MOK_ADJUST_SPECTRAL) return std::sqrt(std::max(1.0, double(rows) / cols));
  return 1.0;
}

}  // namespace

int64_t muon_ws_bytes(int count, const mok_muon_tensor* t) {
  int64_t most = 0;
  for (const MuSize size : {MuSize::Thin, MuSize::General})
    (void)each_run(count, t, size, [&](const MuPart*, int, int64_t bytes) {
      most = std::max(most, bytes);
      return hipSuccess;
    });
  return std::max<int64_t>(most, 256);
}

hipError_t launch_muon(int count, const mok_muon_tensor* t, const mok_muon_config& c, uint8_t* ws, hipStream_t s) {
  const auto arguments = [&](const MuPart* part, int n) {
    MuArgs a{};
    for (int k = 0; k < n; ++k) {
      const mok_muon_tensor& x = t[part[k].tensor];
      a.item[k] = MuItem{x.g, x.m, x.p, static_cast<uint16_t*>(x.copy), ws + part[k].ws, part[k].first, part[k].count,
                         x.rows, x.cols, float(adjustment(c.adjust, x.rows, x.cols))};
    }
    a.count = n;
    a.nesterov = c.nesterov;
    a.gbf = c.grad_elem == MOK_ELEM_BF16;
    a.mu = float(c.momentum);
    a.eps = float(c.ns.eps);
    a.lr = c.lr;
    a.weight_decay = c.weight_decay;
    a.max_norm = c.max_norm;
    a.sumsq = c.sumsq_dev;
    a.lr_dev = c.lr_dev;
    return a;
  };
  MuSteps st{};
  st.count = c.ns.steps;
  std::copy_n(&c.ns.coefficients[0][0], 3 * st.count, &st.coef[0][0]);
  hipError_t e = each_run(count, t, MuSize::Small, [&](const MuPart* part, int n, int64_t) {
    static std::atomic<bool> done[kMaxDevices];
    const hipError_t e0 = allow_lds(k_muon_small, 160 << 10, done);
    if (e0 != hipSuccess) return e0;
    MuArgs a = arguments(part, n);
    int lds = 0, matrices = 0;
    for (int k = 0; k < n; ++k) {
      const MuItem& it = a.item[k];
      const ThinShape thin(it.rows, it.cols);
      lds = std::max(lds, thin.thin() ? (3 * kThinMatrix * 8 + thin.m * (thin.n | 1) * 4)
                                      : small_lds(SmallShape(it.rows, it.cols).shorter));
      a.first[k] = matrices;
      matrices += a.item[k].batch;
    }
    a.first[n] = matrices;
    k_muon_small<<<matrices, 512, lds, s>>>(a, st);
    return hipGetLastError();
  });
  if (e == hipSuccess)
    e = each_run(count, t, MuSize::Thin, [&](const MuPart* part, int n, int64_t) {
      MuArgs a = arguments(part, n);
      int lds = 0;
      for (int k = 0; k < n; ++k) lds = std::max(lds, ThinShape(a.item[k].rows, a.item[k].cols).chunk_lds());
      hipError_t e1 = run(k_thin_gram, a, 256, lds, s, [](const MuItem& it) { return int64_t(ThinShape(it.rows, it.cols).parts); });
      if (e1 == hipSuccess) e1 = run(k_thin_steps, a, 512, 0, s, [](const MuItem&) { return int64_t(1); }, st);
      if (e1 == hipSuccess)
        e1 = run(k_thin_apply, a, 256, lds, s, [](const MuItem& it) { return int64_t(ThinShape(it.rows, it.cols).chunks); });
      return e1;
    });
  if (e != hipSuccess) return e;
  return each_run(count, t, MuSize::General, [&](const MuPart* part, int n, int64_t) {
    MuArgs a = arguments(part, n);
    hipError_t e1 = run(k_muon_norm, a, 256, 0, s, [](const MuItem& it) {
      const int64_t size = int64_t(it.rows) * it.cols;
      return cdiv(size, mu_chunk(size));
    });
    if (e1 == hipSuccess)
      e1 = run(k_muon_start, a, 256, 0, s, [](const MuItem& it) {
        const MuBuffers b(it.rows, it.cols);
        return int64_t(b.rows / 64) * (b.cols / 64);
      });
    if (e1 != hipSuccess) return e1;
    int64_t tiles = 0;   // of 256 x 256 in a step's last product
    for (int k = 0; k < n; ++k)
      tiles += cdiv(a.item[k].rows, 256) * cdiv(a.item[k].cols, 256) * a.item[k].batch;
    e1 = tiles >= 256 ? steps<MuWide>(a, c.ns.steps, &c.ns.coefficients[0][0], s)
                      : steps<MuMid>(a, c.ns.steps, &c.ns.coefficients[0][0], s);
    return e1;
  });
}

}  // namespace mok
