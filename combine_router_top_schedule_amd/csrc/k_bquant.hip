// Quantising to E4M3 with one fp32 scale for 128 values: token rows along the row and along the tokens of each
// expert, weights in blocks of 128 x 128.
//
// For a block x: amax = max(max |x|, 2^-100), scale = amax / 448, code = e4m3(x * (448 / amax)), nearest even. The
// product is at most 448 (1 + 2^-23), which rounds to 448. A NaN stays NaN where it stands (the largest magnitude
// passes over it); an infinity gives its block a scale of infinity and its own code NaN.
//
// HBM bounds all of it: 2 or 4 bytes read and 1 + 4/128 (rows) or 2 + 8/128 (both directions) written for each value. Both
// directions take one pass, a 128 x 128 tile a workgroup (two passes over 16,384 x 7168 bf16 took 168 us, one takes 124 us,
// 3.9 TB/s); weights of 4 x 4096 x 7168 in fp32, both ways, 136 us, 5.2 TB/s; 16,384 x 7168 bf16
// along the row alone, 77 us, 4.6 TB/s; one row of 7168, 6.1 us, a launch and one latency.
#include "k_block.h"

#pragma clang fp contract(off)

namespace mok {
namespace {

struct Q8 {
  float v[8];
};

// Eight values from column c on of a row of k; past its end zero. VEC: 16-byte loads (whole chunks only).
template <bool VEC>
__device__ __forceinline__ Q8 load8(const float* row, int c, int k) {
  Q8 q;
  if (VEC && c + 8 <= k) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(row + c), b = *reinterpret_cast<const f32x4*>(row + c + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) q.v[j] = a[j], q.v[4 + j] = b[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = row[min(c + j, k - 1)];
      q.v[j] = c + j < k ? x : 0.f;
    }
  }
  return q;
}
template <bool VEC>
__device__ __forceinline__ Q8 load8(const uint16_t* row, int c, int k) {
  Q8 q;
  if (VEC && c + 8 <= k) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q.v[2 * j] = __uint_as_float(a[j] << 16);
      q.v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = bf2f(row[min(c + j, k - 1)]);
      q.v[j] = c + j < k ? x : 0.f;
    }
  }
  return q;
}

__device__ __forceinline__ float amax8(const Q8& q) {
  float m = kBlkLeast;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(q.v[j]));
  return m;
}

// The largest over the 16 lanes of a row's block.
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  return m;
}

__device__ __forceinline__ uint32_t code2(float a, float b) {
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xFFFFu;
}

struct RowsArgs {
  const void* x;
  uint8_t* codes;
  float* scales;     // [kb][rows]
  int64_t rows, stride;
  int k, kb;         // columns, blocks of 128 columns
};

// 16 rows x 8 blocks a workgroup: 16 lanes hold a row's block, 8 values each. The scales of a block go out as runs of
// 16 floats.
constexpr int kRowTile = 16, kRowBlocks = 8;

template <class T, bool VEC>
__global__ __launch_bounds__(256) void k_bquant_rows(RowsArgs a) {
  __shared__ float s[kRowBlocks][kRowTile];
  const int tid = threadIdx.x, r = tid >> 4, c = (tid & 15) * 8;
  const int64_t row = int64_t(blockIdx.x) * kRowTile + r;
  const int b0 = blockIdx.y * kRowBlocks, nb = min(kRowBlocks, a.kb - b0);
  const bool live = row < a.rows;
  const T* src = static_cast<const T*>(a.x) + (live ? row : 0) * a.stride;
  Q8 q[kRowBlocks];
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i)
    if (i < nb) q[i] = load8<VEC>(src, (b0 + i) * kBlk + c, a.k);
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i)
    if (i < nb) {
      const float m = max16(amax8(q[i])), f = kBlkTop / m;
      if ((tid & 15) == 0) s[i][r] = m / kBlkTop;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = q[i].v[j] * f;
      if (live)
        *reinterpret_cast<uint2*>(a.codes + row * (int64_t(a.kb) * kBlk) + (b0 + i) * kBlk + c) =
            uint2{code2(y[0], y[1]) | code2(y[2], y[3]) << 16, code2(y[4], y[5]) | code2(y[6], y[7]) << 16};
    }
  __syncthreads();
  const int i = tid >> 4, rr = tid & 15;
  const int64_t out = int64_t(blockIdx.x) * kRowTile + rr;
  if (i < nb && out < a.rows) a.scales[int64_t(b0 + i) * a.rows + out] = s[i][rr];
}

// The tiles behind the groups': rows before the first group and behind the last, which only get row codes.
__device__ __forceinline__ bool find_outside_tile(const RowGroups& rg, int t, GroupTile& gt) {
  if (!rg.offsets) return false;
  const int lane = threadIdx.x & 63;
  int last = clamp_offset(rg.offsets[0], rg.rows);
  const int head = last;
  for (int g = lane; g < rg.groups; g += 64) last = max(last, clamp_offset(rg.offsets[g + 1], rg.rows));
#pragma unroll
  for (int o = 32; o; o >>= 1) last = max(last, __shfl_xor(last, o, 64));
  const int before = (head + kBlk - 1) / kBlk, u = t - count_group_tiles(rg, kBlk);
  const int64_t row0 = u < before ? int64_t(u) * kBlk : last + int64_t(u - before) * kBlk;
  const int64_t end = u < before ? head : rg.rows;
  if (row0 >= end) return false;
  gt.row0 = gt.tile0 = row0;
  gt.rows = int(min(int64_t(kBlk), end - row0));
  return true;
}

struct TileArgs {
  const void* x;
  uint8_t* codes;       // null: not wanted
  float* scales;
  uint8_t* codes_t;     // null: not wanted
  float* scales_t;
  RowGroups rg;         // token rows; weights: rows of one matrix
  int64_t stride, rows_t;   // rows_t: length of a row of codes_t
  int k, kb, row_tiles;
};

// One tile of up to 128 rows (of one group) x 128 columns a workgroup; a thread holds 8 x 8 of them. Rows' largest values
// join over 16 lanes, columns' over the lanes of a wave 16 apart and then over the 4 waves; columns' codes turn
// in LDS, where a thread's 8 rows of a column are 8 consecutive bytes. SQUARE: one scale for the whole tile (weights),
// else one for each row and each column of it.
constexpr int kTurn = kBlk + 8;   // bytes from one column to the next in LDS

template <class T, bool VEC, bool SQUARE>
__global__ __launch_bounds__(256) void k_bquant_tile(TileArgs a) {
  __shared__ float s_col[4][kBlk];
  __shared__ float s_row[kBlk];
  __shared__ __attribute__((aligned(16))) uint8_t turn[kBlk * kTurn];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int jb = blockIdx.x % a.kb, t = blockIdx.x / a.kb;
  const T* x = static_cast<const T*>(a.x);
  uint8_t *codes = a.codes, *codes_t = a.codes_t;
  float *scales = a.scales, *scales_t = a.scales_t;
  GroupTile gt;
  if constexpr (SQUARE) {
    const int e = t / a.row_tiles, it = t % a.row_tiles;
    gt.group = e;
    gt.row0 = gt.tile0 = int64_t(it) * kBlk;
    gt.rows = int(min(int64_t(kBlk), a.rg.rows - gt.row0));
    x += e * a.rg.rows * a.stride;
    codes += e * a.rg.rows * (int64_t(a.kb) * kBlk);
    scales += int64_t(e) * a.row_tiles * a.kb;
    if (codes_t) {
      codes_t += e * (int64_t(a.k) * a.rows_t);
      scales_t += int64_t(e) * a.row_tiles * a.kb;
    }
  } else {
    gt = find_group_tile(a.rg, t, kBlk);
    if (gt.group < 0) {
      if (!codes || !find_outside_tile(a.rg, t, gt)) return;
      codes_t = nullptr;
    }
  }
  const int r0 = (tid >> 4) * 8, c = (tid & 15) * 8, col = jb * kBlk + c;
  Q8 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (rows past the tile's last are loaded from it and taken as zero: no branches around the loads)
    const int64_t row = gt.row0 + min(r0 + i, gt.rows - 1);
    q[i] = load8<VEC>(x + row * a.stride, col, a.k);
    if (r0 + i >= gt.rows)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[i].v[j] = 0.f;
  }
  float fr[8], fc[8];
  if constexpr (SQUARE) {
    float m = kBlkLeast;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(q[i]));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if (lane == 0) s_row[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_row[0], s_row[1]), fmaxf(s_row[2], s_row[3]));
    const float f = kBlkTop / m;
#pragma unroll
    for (int i = 0; i < 8; ++i) fr[i] = fc[i] = f;
    if (tid == 0) {
      const int it = int(gt.row0 / kBlk);
      scales[int64_t(it) * a.kb + jb] = m / kBlkTop;
      if (codes_t) scales_t[int64_t(jb) * a.row_tiles + it] = m / kBlkTop;
    }
  } else {
    if (codes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = max16(amax8(q[i]));
        fr[i] = kBlkTop / m;
        if ((tid & 15) == 0) s_row[r0 + i] = m / kBlkTop;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = kBlkLeast;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(q[i].v[j]));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      if (lane < 16) s_col[wave][c + j] = m;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fmaxf(fmaxf(s_col[0][c + j], s_col[1][c + j]), fmaxf(s_col[2][c + j], s_col[3][c + j]));
      fc[j] = kBlkTop / m;
      if (codes_t && tid < 16 && col + j < a.k) scales_t[(gt.tile0 / kBlk) * int64_t(a.k) + col + j] = m / kBlkTop;
    }
    if (codes && tid < gt.rows) scales[int64_t(jb) * a.rg.rows + gt.row0 + tid] = s_row[tid];
  }
  if (codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* v = q[i].v;
      if (r0 + i < gt.rows)
        *reinterpret_cast<uint2*>(codes + (gt.row0 + r0 + i) * (int64_t(a.kb) * kBlk) + col) =
            uint2{code2(v[0] * fr[i], v[1] * fr[i]) | code2(v[2] * fr[i], v[3] * fr[i]) << 16,
                  code2(v[4] * fr[i], v[5] * fr[i]) | code2(v[6] * fr[i], v[7] * fr[i]) << 16};
    }
  }
  if (!codes_t) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = fc[j];
    *reinterpret_cast<uint2*>(turn + (c + j) * kTurn + r0) =
        uint2{code2(q[0].v[j] * f, q[1].v[j] * f) | code2(q[2].v[j] * f, q[3].v[j] * f) << 16,
              code2(q[4].v[j] * f, q[5].v[j] * f) | code2(q[6].v[j] * f, q[7].v[j] * f) << 16};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int idx = tid + 256 * i, cc = idx >> 3, ch = idx & 7;
    const uint2 lo = *reinterpret_cast<const uint2*>(turn + cc * kTurn + ch * 16);
    const uint2 hi = *reinterpret_cast<const uint2*>(turn + cc * kTurn + ch * 16 + 8);
    if (jb * kBlk + cc < a.k)
      *reinterpret_cast<u32x4*>(codes_t + int64_t(jb * kBlk + cc) * a.rows_t + gt.tile0 + ch * 16) =
          u32x4{lo.x, lo.y, hi.x, hi.y};
  }
}

template <class T>
bool whole16(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * int64_t(sizeof(T))) % 16 == 0;
}

template <class T>
hipError_t rows_typed(const RowsArgs& a, hipStream_t s) {
  const dim3 grid(unsigned(cdiv(a.rows, kRowTile)), unsigned(cdiv(a.kb, kRowBlocks)));
  if (whole16<T>(a.x, a.stride)) k_bquant_rows<T, true><<<grid, 256, 0, s>>>(a);
  else k_bquant_rows<T, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <class T, bool SQUARE>
hipError_t tile_typed(const TileArgs& a, int64_t tiles, hipStream_t s) {
  const unsigned grid = unsigned(tiles * a.kb);
  if (whole16<T>(a.x, a.stride)) k_bquant_tile<T, true, SQUARE><<<grid, 256, 0, s>>>(a);
  else k_bquant_tile<T, false, SQUARE><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quantize(const mok_block_desc& d, const void* x, const int32_t* offsets, uint8_t* codes,
                                 float* scales, uint8_t* codes_t, float* scales_t, hipStream_t s) {
  if (d.rows == 0) return hipSuccess;
  const bool bf = d.elem == MOK_ELEM_BF16;
  const int kb = int(cdiv(d.k, kBlk));
  if (!codes_t) {
    const RowsArgs a{x, codes, scales, d.rows, d.stride, d.k, kb};
    return bf ? rows_typed<uint16_t>(a, s) : rows_typed<float>(a, s);
  }
  const TileArgs a{x, codes, scales, codes_t, scales_t, RowGroups{offsets, d.rows, d.groups}, d.stride,
                   block_padded_rows(d.rows, d.groups), d.k, kb, 0};
  const int64_t tiles = group_tiles_max(d.rows, d.groups, kBlk) + (codes && offsets ? 2 : 0);
  return bf ? tile_typed<uint16_t, false>(a, tiles, s) : tile_typed<float, false>(a, tiles, s);
}

hipError_t launch_block_quantize_weights(const mok_block_desc& d, const void* w, uint8_t* codes, float* scales,
                                         uint8_t* codes_t, float* scales_t, hipStream_t s) {
  const int row_tiles = int(cdiv(d.n, kBlk));
  const TileArgs a{w, codes, scales, codes_t, scales_t, RowGroups{nullptr, d.n, 1}, d.k, int64_t(row_tiles) * kBlk,
                   d.k, int(cdiv(d.k, kBlk)), row_tiles};
  const int64_t tiles = int64_t(d.groups) * row_tiles;
  return d.elem == MOK_ELEM_BF16 ? tile_typed<uint16_t, true>(a, tiles, s) : tile_typed<float, true>(a, tiles, s);
}

}  // namespace mok
