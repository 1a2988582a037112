// Products of E4M3 operands with one fp32 scale for 128 values along the sum:
//   rows sorted by expert times the experts' weights (scales of 128 x 128 there),
//     out[r][n] = sum_j xs[j][r] ws[g][n / 128][j] sum_{k in block j} x[r][k] w[g][n][k];
//   the weight gradient, both operands with their tokens contiguous and scaled in blocks of 128 tokens,
//     dw[g][n][k] = sum_j dys[j][n] xs[j][k] sum_{t in block j} dy[n][t] x[k][t].
//
// A stage of 128 bytes a row is one block of the sum, so each stage's 32 x 32 product of two
// v_mfma_f32_32x32x64_f8f6f4 starts from zero and is added, times its scales, by one fused multiply-add an element
// (the weight gradient needs one product of two scales more). The first operand's rows (weights; dy) are the rows of
// the MFMA's result, which lie in registers, the second's (tokens; x) its columns, which lie in lanes: a lane has one token
// scale, and a weight scale is the same for a whole wave.
//
// The FP8 instructions cut their products some 20 bits below the largest one of a sum: results are off by 1e-5 to 5e-5 of
// their size, a hundredth of a bf16 result's rounding. fp32 results (the weight gradient among them) are wanted better:
// there the codes are widened to fp16, which holds all of them, and multiplied at half the rate with sums as good as
// fp32.
//
// Measured: 16,384 rows of 4 uneven experts, 4096 x 7168, bf16: 497 us, 1.94 PFLOP/s, the matrix cores busy in 58 % of the cycles
// of a clock that falls to 1.6 GHz (one 256 x 256 tile a CU, four rounds of them and a fifth of 32 tiles; equal experts, four full
// rounds, took 405 us where uneven ones took 479; without the next product beside an addition 872 us). Weight gradient of
// 4 experts of 7168 x 2048 over them: 475 to 610 us by the card, 0.8 to 1.0 PFLOP/s in fp16, 51 % (128 x 128, two on a CU;
// 256 x 128 and products one ahead were equal or slower). 44 rows of 6 experts, 7168 x 2048: 19 us, 74 MB at 3.9 TB/s; one row
// of 4096 x 7168: 7.2 us, 29 MB at 4.1 TB/s, launch included (20 and 9.3 us with weights that are in no cache).
#include <algorithm>
#include <cmath>

#include "k_block.h"
#include "k_gemm.h"

namespace mok {
namespace {

struct ProductArgs {
  const uint8_t* a;      // weights [g][n][stride], or dy columns [n][stride]
  const float* as;       // weights' scales [g][nb][kb], or dy's [..][n]
  const uint8_t* b;      // tokens [rows][stride], or x columns [k][stride]
  const float* bs;       // [kb][rows], or [..][k]
  void* out;
  RowGroups rg;
  int64_t out_stride, stride;   // stride: of a's and b's rows
  int n, k, kb;          // k, kb: columns and blocks of the sum (gradient: columns of x)
  int tiles_n;           // tiles of n
  int tiles_k;           // gradient: tiles of k
  int accumulate, bf16;
};

// WA x WB waves, each FA x FB blocks of 32 x 32.
template <int WA_, int WB_, int FA_, int FB_>
struct Shape {
  static constexpr int WA = WA_, WB = WB_, FA = FA_, FB = FB_;
  static constexpr int kWaves = WA * WB, kA = WA * FA * 32, kB = WB * FB * 32;
  struct Lds {
    uint8_t a[2][kA * kStageRowBytes];
    uint8_t b[2][kB * kStageRowBytes];
    float as[4][kA];   // (a stage's scales are read until its last product, when its codes' buffer takes others)
    float bs[4][kB];
  };
};

// 128 bytes of each of ROWS rows into an LDS stage, swizzled as swz() reads them; a wave takes kEach runs of 8 rows. Rows
// past the resource's end read as zeros. `lane_off` is lane_offset(stride): a lane's row and chunk in an even run; in an odd
// one the chunk's lowest bit turns, which is the offset's bit 4, as strides are multiples of 128.
__device__ __forceinline__ int lane_offset(int stride) {
  const int L = int(threadIdx.x) & 63;
  return (L >> 3) * stride + ((L & 7) ^ (L >> 3)) * 16;
}
template <int ROWS, int WAVES>
__device__ __forceinline__ void issue_rows(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int lane_off, int stride, int col,
                                           int w, int part, int parts) {
  constexpr int kEach = ROWS / 8 / WAVES;
  static_assert(kEach % 2 == 0, "a wave's first run is even");
#pragma unroll
  for (int c = kEach * part / parts; c < kEach * (part + 1) / parts; ++c) {
    const int run = w * kEach + c;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + run * 8 * kStageRowBytes), 16,
                                             (lane_off ^ (c & 1) * 16) + (run * 8 * stride + col), 0, 0, 0);
  }
}

// COUNT scales (consecutive floats, those from `valid` on zero) into LDS, 64 a wave (by several waves the same ones: a
// branch here would cut the stage's code in two, and the compiler then moves products across it).
template <int COUNT>
__device__ __forceinline__ void issue_scales(const float* s, int valid, float* lds, int w) {
  const int L = int(threadIdx.x) & 63, q = w % (COUNT / 64) * 64;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(s, int64_t(valid) * 4), (lds_void*)(lds + q), 4, (q + L) * 4, 0, 0,
                                           0);
}

typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

// A row's 128 codes of a stage: a lane has the 16-byte chunks 2 q + half. (Which of them meet in a product does not matter
// as long as both operands agree.)
struct Codes {
  u32x4 q[4];
};
__device__ __forceinline__ Codes load_codes(const uint8_t* lds, int row, int half) {
  Codes c;
#pragma unroll
  for (int q = 0; q < 4; ++q) c.q[q] = *reinterpret_cast<const u32x4*>(lds + swz(row, 2 * q + half));
  return c;
}

// The codes as operands of the FP8 instructions, or as fp16 values, which hold every E4M3 value.
struct NarrowRow {
  i32x8 v[2];
  __device__ __forceinline__ explicit NarrowRow(const Codes& c) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[h][u] = int(c.q[2 * h][u]);
        v[h][4 + u] = int(c.q[2 * h + 1][u]);
      }
  }
};
struct WideRow {
  f16x8 v[8];
  __device__ __forceinline__ explicit WideRow(const Codes& c) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = widen(c.q[q][0], c.q[q][1]);
      v[2 * q + 1] = widen(c.q[q][2], c.q[q][3]);
    }
  }
  static __device__ __forceinline__ f16x8 widen(uint32_t lo, uint32_t hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(lo), 1.f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(lo), 1.f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(hi), 1.f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(hi), 1.f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
};

__device__ __forceinline__ f32x16 block_product(const NarrowRow& a, const NarrowRow& b) {
  f32x16 p;
#pragma unroll
  for (int v = 0; v < 16; ++v) p[v] = 0.f;
  // (no scales: the codes' products as they are)
  p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v[0], b.v[0], p, 0, 0, 0, 0, 0, 0);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v[1], b.v[1], p, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 block_product(const WideRow& a, const WideRow& b) {
  f32x16 p;
#pragma unroll
  for (int v = 0; v < 16; ++v) p[v] = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) p = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.v[q], b.v[q], p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ void add_scaled(f32x16& sum, const f32x16& part, float s) {
#pragma unroll
  for (int v = 0; v < 16; ++v) sum[v] = fmaf(part[v], s, sum[v]);
}

// The tile's rows, from registers through LDS to out[row0 ..][n0 ..]: `rows` rows of `cols` elements. 16 bytes a lane where
// rows begin at multiples of that, else an element a lane.
template <class S, class T>
__device__ __forceinline__ void store_rows(uint8_t* smem, const f32x16 (&acc)[S::FA][S::FB], const ProductArgs& p,
                                           int64_t row0, int n0, int rows, int cols) {
  constexpr int kPitch = S::kA * int(sizeof(T)) + 16, kChunk = 16 / int(sizeof(T)), kThreads = S::kWaves * 64;
  static_assert(S::kB * kPitch <= int(sizeof(typename S::Lds)));
  const int tid = tile_tid(), lane = tid & 63, w = tid >> 6, wa = w / S::WB, wb = w % S::WB, half = lane >> 5;
  __syncthreads();   // (the other waves' last reads of the stages)
#pragma unroll
  for (int j = 0; j < S::FB; ++j) {
    uint8_t* row = smem + ((wb * S::FB + j) * 32 + (lane & 31)) * kPitch;
#pragma unroll
    for (int i = 0; i < S::FA; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        T* o = reinterpret_cast<T*>(row) + (wa * S::FA + i) * 32 + 8 * q + 4 * half;
        const f32x16& y = acc[i][j];
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(o) = uint2{pack_bf2(y[4 * q], y[4 * q + 1]), pack_bf2(y[4 * q + 2], y[4 * q + 3])};
        else
          *reinterpret_cast<f32x4*>(o) = f32x4{y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
      }
  }
  __syncthreads();
  T* out = static_cast<T*>(p.out) + row0 * p.out_stride + n0;
  if ((reinterpret_cast<uintptr_t>(out) & 15) == 0 && p.out_stride % kChunk == 0) {
    constexpr int kRun = S::kA / kChunk;   // lanes of a row
    for (int r = tid / kRun; r < rows; r += kThreads / kRun) {
      const int c = tid % kRun * kChunk;
      const T* x = reinterpret_cast<const T*>(smem + r * kPitch) + c;
      T* o = out + r * p.out_stride + c;
      if (c + kChunk <= cols) {
        *reinterpret_cast<u32x4*>(o) = *reinterpret_cast<const u32x4*>(x);
      } else {
        for (int u = 0; c + u < cols; ++u) o[u] = x[u];
      }
    }
  } else {
    for (int r = w; r < rows; r += S::kWaves)
      for (int c = lane; c < cols; c += 64) out[r * p.out_stride + c] = reinterpret_cast<const T*>(smem + r * kPitch)[c];
  }
}

// WIDE: the products in fp16 (see the head of the file).
template <class S, bool GRAD, bool WIDE, bool AHEAD = !WIDE>
__global__ __launch_bounds__(S::kWaves * 64, 2) void k_block_product(ProductArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  typename S::Lds& sm = *reinterpret_cast<typename S::Lds*>(smem);
  const int lane = threadIdx.x & 63, w = wave_id(), wa = w / S::WB, wb = w % S::WB, half = lane >> 5, l32 = lane & 31;
  GroupTile gt;
  int n0, k0 = 0, ksteps, valid_b;
  const uint8_t *a, *b;
  const float *as, *bs;
  if constexpr (GRAD) {
    // Every XCD takes an eighth of each group's tiles, which follow one another: groups differ in length, and with whole
    // groups to an XCD the one with the longest would be the last (4 uneven groups, 7168 x 2048: 694 us instead of 608).
    const int per = p.tiles_n * p.tiles_k, run = (per + kXcds - 1) / kXcds, in = blockIdx.x / kXcds;
    const int g = in / run, t = blockIdx.x % kXcds * run + in % run;
    if (t >= per) return;
    gt = find_group(p.rg, g);
    int tn, tk;
    tile_coords(t, p.tiles_n, p.tiles_k, tn, tk);
    n0 = tn * S::kA;
    k0 = tk * S::kB;
    ksteps = (gt.rows + kBlk - 1) / kBlk;
    if (ksteps == 0 && p.accumulate) return;
    valid_b = min(S::kB, p.k - k0);
    a = p.a + n0 * p.stride + gt.pad0;
    b = p.b + k0 * p.stride + gt.pad0;
    as = p.as + (gt.pad0 / kBlk) * p.n + n0;
    bs = p.bs + (gt.pad0 / kBlk) * p.k + k0;
  } else {
    // the tiles there are (not the bound that was launched) in runs of equal length for the XCDs
    const int row_tiles = count_group_tiles(p.rg, S::kB), total = row_tiles * p.tiles_n, run = (total + 7) / 8;
    const int in = blockIdx.x / kXcds, id = blockIdx.x % kXcds * run + in;
    if (in >= run || id >= total) return;
    int tm, tn;
    tile_coords(id, row_tiles, p.tiles_n, tm, tn);
    gt = find_group_tile(p.rg, tm, S::kB);
    n0 = tn * S::kA;
    ksteps = p.kb;
    valid_b = gt.rows;
    a = p.a + (int64_t(gt.group) * p.n + n0) * p.stride;
    b = p.b + gt.row0 * p.stride;
    const int blocks = (p.n + kBlk - 1) / kBlk;
    as = p.as + (int64_t(gt.group) * blocks + min((n0 + wa * S::FA * 32) / kBlk, blocks - 1)) * p.kb;
    bs = p.bs + gt.row0;
  }
  const int valid_a = min(S::kA, p.n - n0);
  // (the last row ends at its own last block, which is all that is read of it)
  const auto span = [&](int rows, int64_t stride) { return (rows - 1) * stride + int64_t(ksteps) * kBlk; };
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a, span(valid_a, p.stride)), rb = make_rsrc(b, span(valid_b, p.stride));
  const int stride = int(p.stride), lane_off = lane_offset(stride);
  const int64_t bs_step = GRAD ? p.k : p.rg.rows;
  // part `part` of `parts` of a stage's loads (scales with the first); past the last stage, the last once more for nothing
  const auto issue = [&](int kt, int part, int parts) {
    const int buf = kt & 1, slot = kt & 3;
    kt = min(kt, ksteps - 1);
    issue_rows<S::kA, S::kWaves>(ra, sm.a[buf], lane_off, stride, kt * kBlk, w, part, parts);
    issue_rows<S::kB, S::kWaves>(rb, sm.b[buf], lane_off, stride, kt * kBlk, w, part, parts);
    if (part > 0) return;
    issue_scales<S::kB>(bs + kt * bs_step, valid_b, sm.bs[slot], w);
    if (GRAD) issue_scales<S::kA>(as + int64_t(kt) * p.n, valid_a, sm.as[slot], w);
  };
  f32x16 acc[S::FA][S::FB];
#pragma unroll
  for (int i = 0; i < S::FA; ++i)
#pragma unroll
    for (int j = 0; j < S::FB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  // One operand's rows of a stage stay in registers (tokens' columns in the gradient, else weights), the other's pass
  // through them.
  using Row = std::conditional_t<WIDE, WideRow, NarrowRow>;
  constexpr int FR = GRAD ? S::FB : S::FA, FT = GRAD ? S::FA : S::FB;
  const int row_r = (GRAD ? wb * S::FB : wa * S::FA) * 32 + l32, row_t = (GRAD ? wa * S::FA : wb * S::FB) * 32 + l32;
  const auto lds_r = [&](int buf) { return GRAD ? sm.b[buf] : sm.a[buf]; };
  const auto lds_t = [&](int buf) { return GRAD ? sm.a[buf] : sm.b[buf]; };
  Codes cr[FR], ct[2];
  float sb[S::FB];
  const auto load_sb = [&](int kt) {
#pragma unroll
    for (int j = 0; j < S::FB; ++j) sb[j] = sm.bs[kt & 3][(wb * S::FB + j) * 32 + l32];
  };
  if (ksteps > 0) {
    issue(0, 0, 1);
    if (AHEAD) {
      issue(1, 0, 4);
      issue(1, 1, 4);
      wait_vmem();
      __syncthreads();
      load_sb(0);
#pragma unroll
      for (int i = 0; i < FR; ++i) cr[i] = load_codes(lds_r(0), row_r + 32 * i, half);
      ct[0] = load_codes(lds_t(0), row_t, half);
    }
  }
  float wscales = 0.f;   // of 64 stages, one a lane
  const auto load_wscales = [&](int kt) {
    wscales = kt + lane < ksteps ? as[kt + lane] : 0.f;
    wait_vmem();   // (here, as the compiler would wait in each stage, for the stage loads, too)
  };
  if (!GRAD) load_wscales(0);
  f32x16 part[2];
  float part_scale = 0.f;
#pragma unroll
  for (int v = 0; v < 16; ++v) part[1][v] = 0.f;
  for (int kt = 0; kt < ksteps; ++kt) {
    const int cur = kt & 1;
    if (!GRAD && kt > 0 && (kt & 63) == 0) load_wscales(kt);
    const float wscale = GRAD ? 1.f : __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wscales), kt & 63));
    const float* asc = sm.as[kt & 3] + wa * S::FA * 32 + 4 * half;
    if constexpr (!AHEAD) {
      wait_vmem();
      __syncthreads();
      issue(kt + 1, 0, 1);
#pragma unroll
      for (int i = 0; i < FR; ++i) cr[i] = load_codes(lds_r(cur), row_r + 32 * i, half);
      ct[0] = load_codes(lds_t(cur), row_t, half);
    }
    if constexpr (!AHEAD) load_sb(kt);
    float scaled[S::FB];
#pragma unroll
    for (int j = 0; j < S::FB; ++j) scaled[j] = sb[j] * wscale;
    Row r[FR] = {Row(cr[0]), Row(cr[1])};
    static_assert(FR == 2, "two resident rows");
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const bool next = AHEAD && t + 1 == FT;   // (in the last stage what is read is not used)
      if (AHEAD) __builtin_amdgcn_sched_barrier(0);
      if (t + 1 < FT) ct[(t + 1) & 1] = load_codes(lds_t(cur), row_t + 32 * (t + 1), half);
      if (next) {
        wait_vmem();
        __syncthreads();
        load_sb(kt + 1);
        ct[(t + 1) & 1] = load_codes(lds_t(cur ^ 1), row_t, half);
      }
      const Row x(ct[t & 1]);
      f32x4 sa[4];
      if constexpr (GRAD)
#pragma unroll
        for (int q = 0; q < 4; ++q) sa[q] = *reinterpret_cast<const f32x4*>(asc + t * 32 + 8 * q);
#pragma unroll
      for (int i = 0; i < FR; ++i) {
        if constexpr (AHEAD) {
          static_assert(!GRAD || !AHEAD);
          // each product's sum is added while the next one runs
          constexpr int U = FR * FT;
          const int u = t * FR + i, before = (u + U - 1) % U;
          part[u & 1] = block_product(r[i], x);
          __builtin_amdgcn_sched_barrier(0);
          // (the loads of a stage are spread over four products: in one run they hold the waves up)
          if (u < 2) issue(kt + 1, 2 + u, 4);
          if (u >= U - 2) issue(kt + 2, u - (U - 2), 4);
          if (next) cr[i] = load_codes(lds_r(cur ^ 1), row_r + 32 * i, half);
          add_scaled(acc[before % FR][before / FR], part[before & 1], part_scale);
          part_scale = scaled[t];
          __builtin_amdgcn_sched_barrier(0);
        } else {
          f32x16& sum = GRAD ? acc[t][i] : acc[i][t];
          const f32x16 prod = GRAD ? block_product(x, r[i]) : block_product(r[i], x);
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[v] = fmaf(prod[v], GRAD ? scaled[i] * sa[v >> 2][v & 3] : scaled[t], sum[v]);
        }
      }
    }
  }
  wait_vmem();   // (loads into LDS do not outlive the workgroup)
  if constexpr (AHEAD) add_scaled(acc[FR - 1][FT - 1], part[1], part_scale);
  if constexpr (GRAD) {
    // (through a buffer that ends with the tile: what is outside reads as zero and is not written, without branches, around
    // which loads would be waited for one by one)
    const int tid = tile_tid(), el = tid & 31, eh = (tid >> 5) & 1;
    float* out = static_cast<float*>(p.out) + (int64_t(gt.group) * p.n + n0) * p.k + k0;
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(out, (int64_t(valid_a - 1) * p.k + valid_b) * 4);
#pragma unroll
    for (int j = 0; j < S::FB; ++j) {
      const int c = (wb * S::FB + j) * 32 + el;
#pragma unroll
      for (int i = 0; i < S::FA; ++i) {
        const int r0 = (wa * S::FA + i) * 32 + 4 * eh, at = c < valid_b ? (r0 * p.k + c) * 4 : 1 << 30;
        if (p.accumulate) {
          float y[16];
#pragma unroll
          for (int v = 0; v < 16; ++v)
            y[v] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ro, at + (8 * (v >> 2) + (v & 3)) * p.k * 4, 0, 0));
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] += y[v];
        }
#pragma unroll
        for (int v = 0; v < 16; ++v)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][v]), ro, at + (8 * (v >> 2) + (v & 3)) * p.k * 4, 0, 0);
      }
    }
  } else {
    // A lane holds 4 consecutive columns of one row: rows come together in LDS and go out in whole runs.
    if constexpr (WIDE) store_rows<S, float>(smem, acc, p, gt.row0, n0, valid_b, valid_a);
    else store_rows<S, uint16_t>(smem, acc, p, gt.row0, n0, valid_b, valid_a);
  }
}

// A dynamic shared memory size above 64 KB has to be allowed once for each kernel and device.
template <class S, bool GRAD, bool WIDE>
hipError_t launch_product(const ProductArgs& p, int64_t tiles, hipStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  const void* f = reinterpret_cast<const void*>(k_block_product<S, GRAD, WIDE>);
  constexpr int bytes = int(sizeof(typename S::Lds));
  const hipError_t e =
      once_per_device(done, [&] { return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  if (e != hipSuccess) return e;
  k_block_product<S, GRAD, WIDE><<<unsigned(tiles), S::kWaves * 64, bytes, s>>>(p);
  return hipGetLastError();
}

// ---- few rows ------------------------------------------------------------------------------------
// Up to 16 FT tokens against 16 FN weight rows a workgroup. The weights' bytes bound it: operands go from memory straight
// into registers, the blocks of the sum are dealt out to the 8 waves in turn (so a workgroup reads runs of 1 KB of a
// weight row) and kAhead blocks of a wave are in flight; the waves' sums join in LDS in their order. One
// v_mfma_f32_16x16x128_f8f6f4 is one block: lane l has 32 codes of row l % 16, from 32 (l / 16) on.
constexpr int kFewWaves = 8;

struct FewCodes {
  u32x4 lo, hi;
};
__device__ __forceinline__ FewCodes load_few(const uint8_t* p) {
  return FewCodes{*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + 16)};
}
template <bool WIDE>
__device__ __forceinline__ f32x4 few_product(const FewCodes& a, const FewCodes& b) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 x = h ? a.hi : a.lo, y = h ? b.hi : b.lo;
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(WideRow::widen(x[0], x[1]), WideRow::widen(y[0], y[1]), p, 0, 0, 0);
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(WideRow::widen(x[2], x[3]), WideRow::widen(y[2], y[3]), p, 0, 0, 0);
    }
    return p;
  } else {
    const auto eight = [](const FewCodes& c) {
      return i32x8{int(c.lo[0]), int(c.lo[1]), int(c.lo[2]), int(c.lo[3]),
                   int(c.hi[0]), int(c.hi[1]), int(c.hi[2]), int(c.hi[3])};
    };
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(eight(a), eight(b), p, 0, 0, 0, 0, 0, 0);
  }
}

template <int FN, int FT, bool WIDE>
__global__ __launch_bounds__(kFewWaves * 64) void k_block_few(ProductArgs p) {
  __shared__ f32x4 sums[kFewWaves][FN * FT][64];
  // (columns first: with rows first 128 rows of 7168 took 43 us instead of 23)
  const GroupTile gt = find_group_tile(p.rg, blockIdx.x / p.tiles_n, 16 * FT);
  if (gt.group < 0) return;
  const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, part = lane >> 4;
  const int n0 = blockIdx.x % p.tiles_n * (16 * FN), blocks = (p.n + kBlk - 1) / kBlk;
  const uint8_t* a[FN];
  const uint8_t* b[FT];
  const float* bs[FT];
  // (rows past the last are the last one's: their results are not stored)
#pragma unroll
  for (int i = 0; i < FN; ++i)
    a[i] = p.a + (int64_t(gt.group) * p.n + min(n0 + 16 * i + l16, p.n - 1)) * p.stride + part * 32;
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t row = gt.row0 + min(16 * j + l16, gt.rows - 1);
    b[j] = p.b + row * p.stride + part * 32;
    bs[j] = p.bs + row;
  }
  const float* as = p.as + (int64_t(gt.group) * blocks + n0 / kBlk) * p.kb;
  f32x4 acc[FN][FT];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = FN + FT <= 3 ? 4 : 2;
  for (int k0 = w; k0 < p.kb; k0 += kFewWaves * kAhead) {
    FewCodes ca[kAhead][FN], cb[kAhead][FT];
    float sa[kAhead], sb[kAhead][FT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u * kFewWaves, at = min(k, p.kb - 1);   // (past the end a block once more, with a scale of zero)
#pragma unroll
      for (int i = 0; i < FN; ++i) ca[u][i] = load_few(a[i] + int64_t(at) * kBlk);
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        cb[u][j] = load_few(b[j] + int64_t(at) * kBlk);
        sb[u][j] = bs[j][int64_t(at) * p.rg.rows];
      }
      sa[u] = as[at];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k0 + u * kFewWaves >= p.kb) break;
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        const float s = sa[u] * sb[u][j];
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const f32x4 y = few_product<WIDE>(ca[u][i], cb[u][j]);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(y[v], s, acc[i][j][v]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) sums[w][i * FT + j][lane] = acc[i][j];
  __syncthreads();
  // lane l of a block: token l % 16, weight rows 4 (l / 16) ..
  for (int q = threadIdx.x; q < FN * FT * 64; q += kFewWaves * 64) {
    const int f = q >> 6, l = q & 63, i = f / FT, j = f % FT;
    f32x4 y = sums[0][f][l];
#pragma unroll
    for (int u = 1; u < kFewWaves; ++u) y += sums[u][f][l];
    const int r = 16 * j + (l & 15), c = n0 + 16 * i + 4 * (l >> 4);
    if (r >= gt.rows) continue;
    const int64_t at = (gt.row0 + r) * p.out_stride + c;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c + v < p.n) {
        if constexpr (WIDE) static_cast<float*>(p.out)[at + v] = y[v];
        else static_cast<uint16_t*>(p.out)[at + v] = f2bf(y[v]);
      }
  }
}

template <int FN, int FT>
hipError_t launch_few(ProductArgs p, hipStream_t s) {
  p.tiles_n = int(cdiv(p.n, 16 * FN));
  const unsigned grid = unsigned(group_tiles_max(p.rg.rows, p.rg.groups, 16 * FT) * p.tiles_n);
  if (p.bf16) k_block_few<FN, FT, false><<<grid, kFewWaves * 64, 0, s>>>(p);
  else k_block_few<FN, FT, true><<<grid, kFewWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

// Weight rows of a workgroup: 64, 32 or 16, the most that leave a workgroup for every CU (the more of them, the less
// often the tokens' codes are read).
template <int FT>
hipError_t launch_few_n(const ProductArgs& p, hipStream_t s) {
  const int64_t tiles = group_tiles_max(p.rg.rows, p.rg.groups, 16 * FT);
  if (cdiv(p.n, 64) * tiles >= 256) return launch_few<4, FT>(p, s);
  return cdiv(p.n, 32) * tiles >= 256 ? launch_few<2, FT>(p, s) : launch_few<1, FT>(p, s);
}

using Mid = Shape<2, 2, 2, 2>;    // 128 x 128
using Wide = Shape<4, 2, 2, 4>;   // 256 x 256

template <class S, bool WIDE>
hipError_t launch_tiles(ProductArgs p, hipStream_t s) {
  p.tiles_n = int(cdiv(p.n, S::kA));
  return launch_product<S, false, WIDE>(p, align_up(group_tiles_max(p.rg.rows, p.rg.groups, S::kB) * p.tiles_n, kXcds), s);
}

constexpr int64_t kMaxFewTiles = int64_t(1) << 23;   // (a launch has fewer than 2^32 threads)

// Which kernel: the one that these estimates call fastest, in microseconds. The tile kernels take so long for a stage of
// the sum (alone on a CU, or beside another workgroup) and for a tile's beginning and end, in rounds of as many tiles as
// run at once; the kernel for few rows is bound by what its workgroups read, at 9.5 TB/s from the L2 caches. Measured, bf16:
// 6 experts of 7168 x 2048: 44 rows 18.9 (few) against 23.4 (128 x 128), 384 rows 23 (128 x 128), 3,000 rows 66 (128 x 128);
// one of 4096 x 7168: 64 rows 20 (few), 512 rows 49 (128 x 128) against 59 (few); 4 experts, 16,384 rows 505 (256 x 256)
// against 610 (128 x 128).
int64_t few_tokens(const mok_block_desc& d) {   // blocks of 16 tokens that a workgroup takes
  const int64_t each = d.rows / d.groups;
  return each <= 16 ? 1 : each <= 32 ? 2 : 4;
}
double few_us(const mok_block_desc& d, int64_t ft) {
  const int64_t tiles = cdiv(d.rows, 16 * ft) + (d.groups > 1 ? std::min<int64_t>(d.rows, d.groups) / 2 : 0);
  const int64_t fn = cdiv(d.n, 64) * tiles >= 256 ? 4 : cdiv(d.n, 32) * tiles >= 256 ? 2 : 1;
  return double(tiles * cdiv(d.n, 16 * fn) * cdiv(d.k, kBlk) * (fn + ft) * 2048) / 9.5e6 + 3.0;
}
template <class S>
double tiles_us(const mok_block_desc& d, int per_cu, double alone, double beside, double tile) {
  // (groups end inside tiles: half a tile each on average)
  const int64_t rows = cdiv(d.rows, S::kB) + (d.groups > 1 ? std::min<int64_t>(d.rows, d.groups) / 2 : 0);
  const int64_t tiles = rows * cdiv(d.n, S::kA);
  const double each = double(cdiv(d.k, kBlk)) * (tiles <= 256 ? alone : beside) + tile;
  return each * (per_cu == 1 ? double(cdiv(tiles, 256)) : std::max(1.0, double(tiles) / (256 * per_cu) + 0.3));
}

}  // namespace

mok_block_kernel block_gemm_kernel(const mok_block_desc& d) {
  const bool bf = d.elem == MOK_ELEM_BF16;
  const int64_t few_ft = few_tokens(d);
  const double few = few_us(d, few_ft), mid = tiles_us<Mid>(d, 2, bf ? 0.77 : 1.1, bf ? 1.1 : 1.5, 3.0),
               wide = bf ? tiles_us<Wide>(d, 1, 1.7, 1.7, 10.0) : INFINITY;
  if (few <= mid && few <= wide && group_tiles_max(d.rows, d.groups, int(16 * few_ft)) * cdiv(d.n, 16) < kMaxFewTiles)
    return MOK_BLOCK_FEW_ROWS;
  return mid <= wide ? MOK_BLOCK_TILES_128 : MOK_BLOCK_TILES_256;
}

hipError_t launch_block_gemm(const mok_block_desc& d, const uint8_t* x, const float* xs, const uint8_t* w,
                             const float* ws, const int32_t* offsets, void* out, hipStream_t s) {
  if (d.rows == 0) return hipSuccess;
  ProductArgs p{};
  p.kb = int(cdiv(d.k, kBlk));
  p.a = w;
  p.as = ws;
  p.b = x;
  p.bs = xs;
  p.out = out;
  p.rg = RowGroups{offsets, d.rows, d.groups};
  p.out_stride = d.stride;
  p.stride = int64_t(p.kb) * kBlk;
  p.n = d.n;
  p.k = d.k;
  p.bf16 = d.elem == MOK_ELEM_BF16;
  switch (block_gemm_kernel(d)) {
    case MOK_BLOCK_FEW_ROWS: {
      const int64_t ft = few_tokens(d);
      return ft == 1 ? launch_few_n<1>(p, s) : ft == 2 ? launch_few_n<2>(p, s) : launch_few_n<4>(p, s);
    }
    case MOK_BLOCK_TILES_128: return p.bf16 ? launch_tiles<Mid, false>(p, s) : launch_tiles<Mid, true>(p, s);
    default: return launch_tiles<Wide, false>(p, s);
  }
}

hipError_t launch_block_wgrad(const mok_block_desc& d, const uint8_t* dy, const float* dys, const uint8_t* x,
                              const float* xs, const int32_t* offsets, float* dw, bool accumulate, hipStream_t s) {
  ProductArgs p{};
  p.a = dy;
  p.as = dys;
  p.b = x;
  p.bs = xs;
  p.out = dw;
  p.rg = RowGroups{offsets, d.rows, d.groups};
  p.stride = block_padded_rows(d.rows, d.groups);
  p.n = d.n;
  p.k = d.k;
  p.accumulate = accumulate;
  using S = Mid;
  p.tiles_n = int(cdiv(d.n, S::kA));
  p.tiles_k = int(cdiv(d.k, S::kB));
  return launch_product<S, true, true>(p, int64_t(d.groups) * align_up(int64_t(p.tiles_n) * p.tiles_k, kXcds), s);
}

}  // namespace mok
