// Shared by the block-scaled FP8 kernels (k_bquant.hip, k_bgemm.hip): the blocks' size and the way from a
// workgroup's number to its group of rows.
//
// Rows come sorted by group (expert): group g is [offsets[g], offsets[g + 1]). The offsets are on the device, so
// the host launches for a bound and every wave finds its tile itself, 64 groups a step by a prefix sum over lanes;
// no table has to be written before. Offsets outside 0..rows are clamped and one that is smaller than an earlier
// one counts as that, so no offsets lead outside the buffers.
#pragma once

#include "mok_device.h"
#include "mok_internal.h"

namespace mok {

constexpr int kBlk = 128;               // values with one scale
constexpr float kBlkTop = 448.f;        // largest E4M3 value
constexpr float kBlkLeast = 0x1p-100f;  // a block's largest magnitude counts as at least this
constexpr int kMaxGroups = 1024;

struct RowGroups {
  const int32_t* offsets;   // [groups + 1], or null: one group of all rows
  int64_t rows;
  int32_t groups;
};

struct GroupTile {
  int group;        // -1: no such tile
  int64_t row0;     // first row of the tile
  int rows;         // rows of the tile
  int64_t pad0;     // multiple of 128: where the group's rows begin when each group is padded to 128
  int64_t tile0;    // first row of the tile in that numbering
};

__device__ __forceinline__ int wave_scan_max(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v = max(v, u);
  }
  return v;
}
__device__ __forceinline__ int wave_scan_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ int clamp_offset(int v, int64_t rows) {
  return v < 0 ? 0 : (int64_t(v) > rows ? int(rows) : v);
}

// Tile t of the groups cut into tiles of `tile` rows (the last of a group may have fewer). Uniform over the
// wave, every lane of which must call it.
__device__ __forceinline__ GroupTile find_group_tile(const RowGroups& rg, int t, int tile) {
  GroupTile r;
  r.group = -1;
  r.rows = 0;
  r.row0 = r.pad0 = r.tile0 = 0;
  if (!rg.offsets) {
    const int64_t a = int64_t(t) * tile;
    if (a < rg.rows) {
      r.group = 0;
      r.row0 = r.tile0 = a;
      r.rows = int(min(int64_t(tile), rg.rows - a));
    }
    return r;
  }
  const int lane = threadIdx.x & 63;
  int prev = clamp_offset(rg.offsets[0], rg.rows), tiles = 0, pads = 0;
  for (int g0 = 0; g0 < rg.groups; g0 += 64) {
    const int g = g0 + lane;
    int end = g < rg.groups ? clamp_offset(rg.offsets[g + 1], rg.rows) : 0;
    end = wave_scan_max(max(end, prev), lane);
    int start = __shfl_up(end, 1, 64);
    if (lane == 0) start = prev;
    const int cnt = end - start;   // (0 in the lanes past the last group)
    const int nt = (cnt + tile - 1) / tile, np = (cnt + kBlk - 1) / kBlk;
    const int st = wave_scan_sum(nt, lane), sp = wave_scan_sum(np, lane);
    const uint64_t hit = __ballot(tiles + st > t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int first = tiles + __shfl(st - nt, l, 64), begin = __shfl(start, l, 64);
      const int in = (t - first) * tile;
      r.group = __builtin_amdgcn_readfirstlane(g0 + l);
      r.row0 = __builtin_amdgcn_readfirstlane(begin + in);
      r.rows = __builtin_amdgcn_readfirstlane(min(tile, __shfl(cnt, l, 64) - in));
      r.pad0 = int64_t(__builtin_amdgcn_readfirstlane(pads + __shfl(sp - np, l, 64))) * kBlk;
      r.tile0 = r.pad0 + __builtin_amdgcn_readfirstlane(in);
      return r;
    }
    tiles += __shfl(st, 63, 64);
    pads += __shfl(sp, 63, 64);
    prev = __shfl(end, 63, 64);
  }
  return r;
}

// Number of tiles that find_group_tile knows. Uniform over the wave.
__device__ __forceinline__ int count_group_tiles(const RowGroups& rg, int tile) {
  if (!rg.offsets) return int((rg.rows + tile - 1) / tile);
  const int lane = threadIdx.x & 63;
  int prev = clamp_offset(rg.offsets[0], rg.rows), tiles = 0;
  for (int g0 = 0; g0 < rg.groups; g0 += 64) {
    const int g = g0 + lane;
    int end = g < rg.groups ? clamp_offset(rg.offsets[g + 1], rg.rows) : 0;
    end = wave_scan_max(max(end, prev), lane);
    int start = __shfl_up(end, 1, 64);
    if (lane == 0) start = prev;
    int sum = (end - start + tile - 1) / tile;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
    tiles += sum;
    prev = __shfl(end, 63, 64);
  }
  return __builtin_amdgcn_readfirstlane(tiles);
}

// Group g: its rows, and where they begin when each group is padded to 128. Uniform over the wave.
__device__ __forceinline__ GroupTile find_group(const RowGroups& rg, int g) {
  GroupTile r;
  r.group = g;
  r.row0 = r.pad0 = r.tile0 = 0;
  r.rows = int(rg.rows);
  if (!rg.offsets) return r;
  const int lane = threadIdx.x & 63;
  int prev = clamp_offset(rg.offsets[0], rg.rows), pads = 0;
  for (int g0 = 0;; g0 += 64) {
    const int i = g0 + lane;
    int end = i < rg.groups ? clamp_offset(rg.offsets[i + 1], rg.rows) : 0;
    end = wave_scan_max(max(end, prev), lane);
    int start = __shfl_up(end, 1, 64);
    if (lane == 0) start = prev;
    const int np = (end - start + kBlk - 1) / kBlk;
    const int sp = wave_scan_sum(np, lane);
    if (g < g0 + 64) {
      const int l = g - g0;
      r.row0 = __builtin_amdgcn_readfirstlane(__shfl(start, l, 64));
      r.rows = __builtin_amdgcn_readfirstlane(__shfl(end, l, 64)) - int(r.row0);
      r.pad0 = r.tile0 = int64_t(__builtin_amdgcn_readfirstlane(pads + __shfl(sp - np, l, 64))) * kBlk;
      return r;
    }
    pads += __shfl(sp, 63, 64);
    prev = __shfl(end, 63, 64);
  }
}

// Tiles of `tile` rows that `rows` rows in `groups` groups have at most.
inline int64_t group_tiles_max(int64_t rows, int groups, int tile) {
  return rows / tile + (rows < groups ? rows : int64_t(groups));
}

}  // namespace mok
