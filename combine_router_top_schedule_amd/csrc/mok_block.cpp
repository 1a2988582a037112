// Host side of the block-scaled FP8 calls of include/mok.h: checks arguments, then enqueues kernels on
// the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mok_internal.h"

using namespace mok;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 27;            // 16 rows a workgroup of 256, fewer than 2^32 threads
constexpr int64_t kMaxColumnRows = int64_t(1) << 22;      // 256 rows of column codes within 32-bit offsets
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxTiles = (int64_t(1) << 22) - 1;     // workgroups of up to 512 threads in a launch

// Tiles that the rows of d have at most.
int64_t row_tiles(const mok_block_desc& d) { return d.rows / 128 + d.groups; }
bool product_fits(const mok_block_desc& d) { return row_tiles(d) * cdiv(d.n, 128) <= kMaxTiles; }

bool width_ok(int32_t v) { return v >= 1 && v <= kMaxWidth; }
bool elem_ok(int32_t e) { return e == MOK_ELEM_F32 || e == MOK_ELEM_BF16; }
uintptr_t elem_size(int32_t e) { return e == MOK_ELEM_BF16 ? 2 : 4; }

bool rows_ok(const mok_block_desc& d, bool columns) {
  return d.rows >= 0 && d.rows <= (columns ? kMaxColumnRows : kMaxRows) && d.groups >= 1 && d.groups <= 1024 &&
         width_ok(d.k);
}

// Rows, groups and offsets, common to all calls on rows.
mok_status check_rows(const mok_block_desc* d, const int32_t* offsets, bool columns) {
  if (!d) return MOK_ERR_NULL;
  if (!rows_ok(*d, columns)) return MOK_ERR_SHAPE;
  if (!offsets && d->groups != 1) return MOK_ERR_NULL;
  return aligned(offsets, 4) ? MOK_OK : MOK_ERR_ALIGN;
}

mok_status hip_status(hipError_t e) { return e == hipSuccess ? MOK_OK : MOK_ERR_HIP; }

}  // namespace

extern "C" {

int64_t mok_block_padded_rows(int64_t rows, int32_t groups) {
  if (rows < 0 || rows > kMaxRows || groups < 1 || groups > 1024) return -1;
  return block_padded_rows(rows, groups);
}

mok_status mok_block_quantize(const mok_block_desc* desc, const void* x_dev, const int32_t* offsets_dev,
                              uint8_t* codes_dev, float* scales_dev, uint8_t* codes_t_dev, float* scales_t_dev,
                              void* stream) {
  const mok_status st = check_rows(desc, offsets_dev, codes_t_dev != nullptr);
  if (st != MOK_OK) return st;
  if (!elem_ok(desc->elem)) return MOK_ERR_DTYPE;
  if (desc->stride < desc->k || desc->stride > (int64_t(1) << 31)) return MOK_ERR_SHAPE;
  if (desc->rows == 0) return MOK_OK;
  if (!x_dev || (!codes_dev && !codes_t_dev) || !codes_dev != !scales_dev || !codes_t_dev != !scales_t_dev)
    return MOK_ERR_NULL;
  if (!aligned(x_dev, elem_size(desc->elem)) || !aligned(codes_dev, 16) || !aligned(codes_t_dev, 16) ||
      !aligned(scales_dev, 4) || !aligned(scales_t_dev, 4))
    return MOK_ERR_ALIGN;
  if (codes_t_dev && (row_tiles(*desc) + 2) * cdiv(desc->k, 128) > kMaxTiles) return MOK_ERR_SHAPE;
  return hip_status(launch_block_quantize(*desc, x_dev, offsets_dev, codes_dev, scales_dev, codes_t_dev, scales_t_dev,
                                          static_cast<hipStream_t>(stream)));
}

mok_status mok_block_quantize_weights(const mok_block_desc* desc, const void* w_dev, uint8_t* codes_dev,
                                      float* scales_dev, uint8_t* codes_t_dev, float* scales_t_dev, void* stream) {
  if (!desc) return MOK_ERR_NULL;
  if (desc->groups < 1 || desc->groups > 1024 || !width_ok(desc->n) || !width_ok(desc->k)) return MOK_ERR_SHAPE;
  if (!elem_ok(desc->elem)) return MOK_ERR_DTYPE;
  if (!w_dev || !codes_dev || !scales_dev || !codes_t_dev != !scales_t_dev) return MOK_ERR_NULL;
  if (!aligned(w_dev, elem_size(desc->elem)) || !aligned(codes_dev, 16) || !aligned(codes_t_dev, 16) ||
      !aligned(scales_dev, 4) || !aligned(scales_t_dev, 4))
    return MOK_ERR_ALIGN;
  if (desc->groups * cdiv(desc->n, 128) * cdiv(desc->k, 128) > kMaxTiles * 2) return MOK_ERR_SHAPE;
  return hip_status(launch_block_quantize_weights(*desc, w_dev, codes_dev, scales_dev, codes_t_dev, scales_t_dev,
                                                  static_cast<hipStream_t>(stream)));
}

mok_status mok_block_gemm(const mok_block_desc* desc, const uint8_t* x_dev, const float* x_scales_dev,
                          const uint8_t* w_dev, const float* w_scales_dev, const int32_t* offsets_dev, void* out_dev,
                          void* stream) {
  const mok_status st = check_rows(desc, offsets_dev, false);
  if (st != MOK_OK) return st;
  if (!width_ok(desc->n)) return MOK_ERR_SHAPE;
  if (!elem_ok(desc->elem)) return MOK_ERR_DTYPE;
  if (desc->stride < desc->n || desc->stride > (int64_t(1) << 31)) return MOK_ERR_SHAPE;
  if (desc->rows == 0) return MOK_OK;
  if (!x_dev || !x_scales_dev || !w_dev || !w_scales_dev || !out_dev) return MOK_ERR_NULL;
  if (!aligned(x_dev, 16) || !aligned(w_dev, 16) || !aligned(x_scales_dev, 4) || !aligned(w_scales_dev, 4) ||
      !aligned(out_dev, elem_size(desc->elem)))
    return MOK_ERR_ALIGN;
  if (!product_fits(*desc)) return MOK_ERR_SHAPE;
  return hip_status(launch_block_gemm(*desc, x_dev, x_scales_dev, w_dev, w_scales_dev, offsets_dev, out_dev,
                                      static_cast<hipStream_t>(stream)));
}

int32_t mok_block_gemm_kernel(const mok_block_desc* desc) {
  if (!desc || !rows_ok(*desc, false) || !width_ok(desc->n) || !elem_ok(desc->elem) || !product_fits(*desc)) return -1;
  return block_gemm_kernel(*desc);
}

mok_status mok_block_wgrad(const mok_block_desc* desc, const uint8_t* dy_t_dev, const float* dy_scales_dev,
                           const uint8_t* x_t_dev, const float* x_scales_dev, const int32_t* offsets_dev,
                           float* dw_dev, int32_t accumulate, void* stream) {
  const mok_status st = check_rows(desc, offsets_dev, true);
  if (st != MOK_OK) return st;
  if (!width_ok(desc->n) || (accumulate != 0 && accumulate != 1)) return MOK_ERR_SHAPE;
  if (!dw_dev || (desc->rows > 0 && (!dy_t_dev || !dy_scales_dev || !x_t_dev || !x_scales_dev))) return MOK_ERR_NULL;
  if (!aligned(dy_t_dev, 16) || !aligned(x_t_dev, 16) || !aligned(dy_scales_dev, 4) || !aligned(x_scales_dev, 4) ||
      !aligned(dw_dev, 4))
    return MOK_ERR_ALIGN;
  if (desc->groups * cdiv(desc->n, 128) * cdiv(desc->k, 128) > kMaxTiles) return MOK_ERR_SHAPE;
  return hip_status(launch_block_wgrad(*desc, dy_t_dev, dy_scales_dev, x_t_dev, x_scales_dev, offsets_dev, dw_dev,
                                       accumulate != 0, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
