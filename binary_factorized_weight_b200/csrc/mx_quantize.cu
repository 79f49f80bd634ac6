// Microscaled quantisation (OCP Microscaling Formats, MX v1.0) and its inverse.
//
//   s = clamp(floor(log2(max |x|)) - top, -127, 127) over each block of 32
//   code = round_to_nearest_even(x 2^-s), saturating;  value = code 2^s
//
// Both read every input once and write every output once, so DRAM bounds them.
#include <algorithm>

#include "dbf_internal.h"
#include "mx_device.cuh"

namespace dbf {
namespace {

constexpr int kThreads = 256;

// One warp item: 256 neighbouring columns of one row, eight per lane.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) dbf_mx_quantize_kernel(const T* __restrict__ src, int64_t rows,
                                                                   int64_t cols, int64_t pitch,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per_row = (pitch + 255) >> 8;
  const int64_t items = rows * per_row;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t r = it / per_row;
    const int64_t c = (it - r * per_row) * 32 + lane;
    const Pack8<T> p = load8<VEC>(src + r * cols, 8 * c, cols);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(p.e[j]);
    mx_store_row8<FMT>(v, r, c, pitch, codes, scales);
  }
}

// The transpose: output row = source column, blocks of 32 run down the source's
// rows.  A CTA takes 128 source rows x 64 source columns through shared memory
// (fp32); thread (column, block) then holds a whole block of 32 values.  The
// four blocks of a column are neighbouring lanes: their codes are one
// contiguous run and their scale bytes one word.  Each 32-row block is shifted
// by 8 words in shared memory, so the warp's 4 blocks x 8 columns of one read
// lie in 32 banks.
constexpr int kTRows = 128, kTCols = 64, kTLd = kTCols + 1;
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) dbf_mx_quantize_t_kernel(const T* __restrict__ src, int64_t rows,
                                                                     int64_t cols, int64_t pitch,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  __shared__ float tile[kTRows * kTLd + 3 * 8];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t col_tiles = (cols + kTCols - 1) / kTCols;
  const int64_t items = col_tiles * (pitch >> 7);
  const int tid = threadIdx.x;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t k4 = it / col_tiles;  // 128 source rows
    const int64_t c0 = (it - k4 * col_tiles) * kTCols;
    for (int i = tid; i < kTRows * kTCols; i += kThreads) {
      const int rr = i / kTCols, cc = i % kTCols;
      const int64_t r = k4 * kTRows + rr, c = c0 + cc;
      tile[rr * kTLd + (rr >> 5) * 8 + cc] = r < rows && c < cols ? to_f32(src[r * cols + c]) : 0.f;
    }
    __syncthreads();
    const int blk = tid & 3, cc = tid >> 2;
    const float* base = tile + blk * (32 * kTLd + 8) + cc;
    float v[32];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = base[j * kTLd];
      amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    const uint32_t byte = mx_scale_byte<FMT>(amax);
    uint32_t word = byte << (8 * blk);
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const float inv = mx_inverse_scale(min(byte, 253u));
    uint32_t q[FMT == kMx4 ? 4 : 8];
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = byte == 255 ? 0.f : v[j + i] * inv;
      if constexpr (FMT == kMx4) {
        q[j / 8] = mx_encode_e2m1(u);
      } else {
        q[j / 4] = mx_encode_e4m3(u[0], u[1], u[2], u[3]);
        q[j / 4 + 1] = mx_encode_e4m3(u[4], u[5], u[6], u[7]);
      }
    }
    const int64_t r = c0 + cc;  // output row
    if (r < cols) {
      const int64_t at = r * pitch + k4 * 128 + blk * 32;
      uint4* dst = reinterpret_cast<uint4*>(codes + (FMT == kMx4 ? at >> 1 : at));
      dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
      if constexpr (FMT == kMx8) dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
      if (blk == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(r, k4, pitch >> 7)) = word;
    }
    __syncthreads();
  }
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) dbf_mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                     const uint8_t* __restrict__ scales, int64_t rows,
                                                                     int64_t cols, int64_t pitch, T* __restrict__ dst) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per_row = (cols + 255) >> 8;
  const int64_t items = rows * per_row;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t r = it / per_row;
    const int64_t c = (it - r * per_row) * 32 + lane;
    if (8 * c >= cols) continue;
    float v[8];
    if constexpr (FMT == kMx4) {
      mx_decode_e2m1(*reinterpret_cast<const uint32_t*>(codes + (r * pitch >> 1) + 4 * c), v);
    } else {
      mx_decode_e4m3(*reinterpret_cast<const uint2*>(codes + r * pitch + 8 * c), v);
    }
    const float s = mx_scale(scales[mx_scale_word(r, c >> 4, pitch >> 7) + ((c >> 2) & 3)]);
    Pack8<T> p;
#pragma unroll
    for (int j = 0; j < 8; ++j) p.e[j] = from_f32<T>(v[j] * s);
    store8<VEC>(dst + r * cols, 8 * c, cols, p);
  }
}

unsigned grid_for(int64_t items, int64_t per_block, const DeviceInfo& dev) {
  return static_cast<unsigned>(std::min<int64_t>((items + per_block - 1) / per_block, int64_t{dev.num_sms} * 8));
}

template <typename T, int FMT>
dbf_status quantize_typed(const void* src, int64_t rows, int64_t cols, bool transpose, uint8_t* codes, uint8_t* scales,
                          const DeviceInfo& dev, cudaStream_t stream) {
  const T* s = static_cast<const T*>(src);
  if (transpose) {
    const int64_t pitch = mx_pitch(rows);
    const int64_t items = (cols + kTCols - 1) / kTCols * (pitch >> 7);
    return launch_pdl(dbf_mx_quantize_t_kernel<T, FMT>, dim3(grid_for(items, 1, dev)), dim3(kThreads), 0, stream, s,
                      rows, cols, pitch, codes, scales);
  }
  const int64_t pitch = mx_pitch(cols);
  const int64_t items = rows * ((pitch + 255) >> 8);
  const bool vec = cols % 8 == 0 && aligned_to(src, 16);
  const dim3 grid(grid_for(items, kThreads / 32, dev));
  return vec ? launch_pdl(dbf_mx_quantize_kernel<T, FMT, true>, grid, dim3(kThreads), 0, stream, s, rows, cols, pitch,
                          codes, scales)
             : launch_pdl(dbf_mx_quantize_kernel<T, FMT, false>, grid, dim3(kThreads), 0, stream, s, rows, cols, pitch,
                          codes, scales);
}

template <typename T, int FMT>
dbf_status dequantize_typed(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst,
                            const DeviceInfo& dev, cudaStream_t stream) {
  T* d = static_cast<T*>(dst);
  const int64_t pitch = mx_pitch(cols);
  const int64_t items = rows * ((cols + 255) >> 8);
  const dim3 grid(grid_for(items, kThreads / 32, dev));
  const bool vec = cols % 8 == 0 && aligned_to(dst, 16);
  return vec ? launch_pdl(dbf_mx_dequantize_kernel<T, FMT, true>, grid, dim3(kThreads), 0, stream, codes, scales, rows,
                          cols, pitch, d)
             : launch_pdl(dbf_mx_dequantize_kernel<T, FMT, false>, grid, dim3(kThreads), 0, stream, codes, scales, rows,
                          cols, pitch, d);
}

}  // namespace
}  // namespace dbf

using namespace dbf;

extern "C" {

int64_t dbf_mx_code_bytes(int64_t rows, int64_t cols, dbf_mx_format fmt) {
  if (!mx_shape_ok(rows, cols) || !mx_format_ok(fmt)) return 0;
  return fmt == DBF_MX_E2M1 ? rows * mx_pitch(cols) / 2 : rows * mx_pitch(cols);
}

int64_t dbf_mx_scale_bytes(int64_t rows, int64_t cols) {
  if (!mx_shape_ok(rows, cols)) return 0;
  return (rows + 127) / 128 * (mx_pitch(cols) / 128) * 512;
}

dbf_status dbf_mx_quantize(const void* src, dbf_dtype src_t, int64_t rows, int64_t cols, dbf_mx_format fmt,
                           uint32_t flags, uint8_t* codes, uint8_t* scales, struct CUstream_st* stream) {
  if (!src || !codes || !scales || !float_dtype_ok(src_t) || !mx_format_ok(fmt)) return DBF_ERR_INVALID_ARG;
  if ((flags & ~static_cast<uint32_t>(DBF_MX_TRANSPOSE)) != 0 || rows < 1 || cols < 1) return DBF_ERR_INVALID_ARG;
  if (!mx_shape_ok(rows, cols) || !mx_shape_ok(cols, rows)) return DBF_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(codes, 32) || !aligned_to(scales, 16) || !aligned_to(src, dtype_size(src_t)))
    return DBF_ERR_MISALIGNED;
  DeviceInfo dev;
  const dbf_status st = current_device(&dev);
  if (st != DBF_OK) return st;
  const bool t = (flags & DBF_MX_TRANSPOSE) != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool four = fmt == DBF_MX_E2M1;
  switch (src_t) {
    case DBF_F16:
      return four ? quantize_typed<__half, kMx4>(src, rows, cols, t, codes, scales, dev, s)
                  : quantize_typed<__half, kMx8>(src, rows, cols, t, codes, scales, dev, s);
    case DBF_BF16:
      return four ? quantize_typed<__nv_bfloat16, kMx4>(src, rows, cols, t, codes, scales, dev, s)
                  : quantize_typed<__nv_bfloat16, kMx8>(src, rows, cols, t, codes, scales, dev, s);
    default:
      return four ? quantize_typed<float, kMx4>(src, rows, cols, t, codes, scales, dev, s)
                  : quantize_typed<float, kMx8>(src, rows, cols, t, codes, scales, dev, s);
  }
}

dbf_status dbf_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                             dbf_mx_format fmt, void* dst, dbf_dtype dst_t, struct CUstream_st* stream) {
  if (!dst || !codes || !scales || !float_dtype_ok(dst_t) || !mx_format_ok(fmt)) return DBF_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1) return DBF_ERR_INVALID_ARG;
  if (!mx_shape_ok(rows, cols)) return DBF_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(codes, 32) || !aligned_to(scales, 16) || !aligned_to(dst, dtype_size(dst_t)))
    return DBF_ERR_MISALIGNED;
  DeviceInfo dev;
  const dbf_status st = current_device(&dev);
  if (st != DBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool four = fmt == DBF_MX_E2M1;
  switch (dst_t) {
    case DBF_F16:
      return four ? dequantize_typed<__half, kMx4>(codes, scales, rows, cols, dst, dev, s)
                  : dequantize_typed<__half, kMx8>(codes, scales, rows, cols, dst, dev, s);
    case DBF_BF16:
      return four ? dequantize_typed<__nv_bfloat16, kMx4>(codes, scales, rows, cols, dst, dev, s)
                  : dequantize_typed<__nv_bfloat16, kMx8>(codes, scales, rows, cols, dst, dev, s);
    default:
      return four ? dequantize_typed<float, kMx4>(codes, scales, rows, cols, dst, dev, s)
                  : dequantize_typed<float, kMx8>(codes, scales, rows, cols, dst, dev, s);
  }
}

}  // extern "C"
