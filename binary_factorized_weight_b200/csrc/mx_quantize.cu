// Microscaled quantisation (OCP Microscaling Formats, MX v1.0) and its inverse.
//
//   s = clamp(floor(log2(max |x|)) - top, -127, 127) over each block of 32
//   code = round_to_nearest_even(x 2^-s), saturating;  value = code 2^s
//
// Both read every input once and write every output once, so DRAM bounds them;
// what keeps them from its rate are the instructions (about 90 for the sixteen
// elements of a thread).  14336 x 4096 bf16 into 4 bits 29.2 us (5.1 TB/s, 78% of
// the copy rate), back 26.4 us (5.6 TB/s, 86%), its transpose into 4 bits 31.0 us
// (4.8 TB/s, 74%).
#include <algorithm>

#include "dbf_internal.h"
#include "mx_device.cuh"

namespace dbf {
namespace {

constexpr int kThreads = 256;

// How a block's warps share out rows: 2^lg warps to a row, each with 512
// neighbouring columns at a time (sixteen per lane), so that no item needs a
// division to find its row.
struct Share {
  int64_t row, row_step;  // this warp's first row, and the distance to its next
  int group, group_step;  // its first group of 512 columns of a row, and the distance to the next
};
__device__ __forceinline__ Share share_of(int lg) {
  const int warp = threadIdx.x >> 5;
  const int rows = (kThreads / 32) >> lg;  // of a block
  return {static_cast<int64_t>(blockIdx.x) * rows + (warp >> lg), static_cast<int64_t>(gridDim.x) * rows,
          warp & ((1 << lg) - 1), 1 << lg};
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) dbf_mx_quantize_kernel(const T* __restrict__ src, int64_t rows,
                                                                   int64_t cols, int64_t pitch, int lg,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
  __shared__ alignas(32) T stage[VEC ? 1 : kThreads * kChunk];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = static_cast<int>((pitch + 511) >> 9);
  const Share w = share_of(lg);
  for (int64_t r = w.row; r < rows; r += w.row_step) {
    for (int g = w.group; g < groups; g += w.group_step) {
      const int c = g * 32 + lane;
      const Pack16<T> p = load16<VEC>(src + r * cols, c, cols, stage + (VEC ? 0 : warp * 32 * kChunk));
      float v[kChunk];
      unpack16(p, v);
      mx_store_row16<FMT>(v, r, c, pitch, codes, scales);
    }
  }
}

// The transpose: output row = source column, blocks of 32 run down the source's
// rows.  A CTA takes 128 source rows x 128 (fp32: 64) source columns through
// shared memory; a thread then holds two neighbouring columns' blocks of 32
// (each read of shared memory brings both).  The four blocks of a column are
// neighbouring lanes: their codes are one contiguous run and their scale bytes
// one word.  Each 32-row block is shifted by 8 words, so a warp's read of 4
// blocks x 8 column pairs lies in 32 banks.
constexpr int kTRows = 128;
template <typename T>
constexpr int kTCols = sizeof(T) == 2 ? 128 : 64;
template <typename T>
constexpr int kTThreads = 2 * kTCols<T>;

template <typename T>
struct alignas(2 * sizeof(T)) Pair {
  T a, b;
};

template <int FMT>
__device__ __forceinline__ void mx_store_block(const float (&v)[32], int64_t r, int64_t k4, int blk, int64_t pitch,
                                               bool valid, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 2) m = max_abs3(m, v[j], v[j + 1]);
  const uint32_t byte = mx_scale_byte<FMT>(__float_as_uint(m) & 0x7FFFFFFFu);
  uint32_t word = byte << (8 * blk);
  word |= __shfl_xor_sync(0xffffffffu, word, 1);
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  if (!valid) return;
  const float inv = mx_inverse_scale(min(byte, 253u));
  uint32_t q[FMT == kMx4 ? 4 : 8];
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[j + i] * inv;
    if constexpr (FMT == kMx4) {
      q[j / 8] = byte == 255 ? 0u : mx_encode_e2m1(u);
    } else {
      q[j / 4] = byte == 255 ? 0u : mx_encode_e4m3(u[0], u[1], u[2], u[3]);
      q[j / 4 + 1] = byte == 255 ? 0u : mx_encode_e4m3(u[4], u[5], u[6], u[7]);
    }
  }
  const int64_t at = r * pitch + k4 * 128 + blk * 32;
  uint4* dst = reinterpret_cast<uint4*>(codes + (FMT == kMx4 ? at >> 1 : at));
  dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
  if constexpr (FMT == kMx8) dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
  if (blk == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(r, k4, pitch >> 7)) = word;
}

// (16-bit elements: three blocks to an SM, 31.0 us for 4096 x 14336 where the 107
// registers of two took 37.6)
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kTThreads<T>, sizeof(T) == 2 ? 3 : 1) dbf_mx_quantize_t_kernel(const T* __restrict__ src, int64_t rows,
                                                                         int64_t cols, int64_t pitch,
                                                                         uint8_t* __restrict__ codes,
                                                                         uint8_t* __restrict__ scales) {
  constexpr int kCols = kTCols<T>, kPad = 32 / sizeof(T), kVec = 16 / sizeof(T);
  __shared__ alignas(16) T tile[kTRows * kCols + 3 * kPad];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t col_tiles = (cols + kCols - 1) / kCols;
  const int64_t items = col_tiles * (pitch >> 7);
  const int tid = threadIdx.x;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t k4 = it / col_tiles;  // 128 source rows
    const int64_t c0 = (it - k4 * col_tiles) * kCols;
    if constexpr (VEC) {  // cols a multiple of 16 bytes: whole vectors lie inside or outside
#pragma unroll
      for (int i = 0; i < kTRows * kCols / kVec / kTThreads<T>; ++i) {
        const int at = i * kTThreads<T> + tid, rr = at / (kCols / kVec), cc = at % (kCols / kVec) * kVec;
        const int64_t r = k4 * kTRows + rr, c = c0 + cc;
        const uint4 v = r < rows && c < cols ? *reinterpret_cast<const uint4*>(src + r * cols + c) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(&tile[rr * kCols + (rr >> 5) * kPad + cc]) = v;
      }
    } else {
      // sixteen loads under way together
#pragma unroll 1
      for (int i0 = tid; i0 < kTRows * kCols; i0 += 16 * kTThreads<T>) {
        T v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int i = i0 + k * kTThreads<T>;
          const int64_t r = k4 * kTRows + i / kCols, c = c0 + i % kCols;
          v[k] = r < rows && c < cols ? src[r * cols + c] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int i = i0 + k * kTThreads<T>, rr = i / kCols;
          tile[rr * kCols + (rr >> 5) * kPad + i % kCols] = v[k];
        }
      }
    }
    __syncthreads();
    const int blk = tid & 3, cc = 2 * (tid >> 2);
    const T* base = tile + blk * (32 * kCols + kPad) + cc;
    Pair<T> t[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = *reinterpret_cast<const Pair<T>*>(base + j * kCols);
    const int64_t r = c0 + cc;  // output row
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = to_f32(t[j].a);
    mx_store_block<FMT>(v, r, k4, blk, pitch, r < cols, codes, scales);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = to_f32(t[j].b);
    mx_store_block<FMT>(v, r + 1, k4, blk, pitch, r + 1 < cols, codes, scales);
    __syncthreads();
  }
}

// kUnroll rows of a warp are under way together: a row's codes are few bytes.
constexpr int kUnroll = 2;
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) dbf_mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                     const uint8_t* __restrict__ scales, int64_t rows,
                                                                     int64_t cols, int64_t pitch, int lg,
                                                                     T* __restrict__ dst) {
  __shared__ alignas(32) T stage[VEC ? 1 : kThreads * kChunk];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = static_cast<int>((cols + 511) >> 9);
  const Share w = share_of(lg);
  for (int64_t r0 = w.row; r0 < rows; r0 += kUnroll * w.row_step) {
    for (int g = w.group; g < groups; g += w.group_step) {
      const int c = g * 32 + lane;
      uint32_t q[kUnroll][FMT == kMx4 ? 2 : 4];
      uint32_t byte[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = r0 + u * w.row_step;
        if (r >= rows || kChunk * static_cast<int64_t>(c) >= cols) continue;
        if constexpr (FMT == kMx4) {
          *reinterpret_cast<uint2*>(q[u]) = *reinterpret_cast<const uint2*>(codes + (r * pitch >> 1) + 8 * static_cast<int64_t>(c));
        } else {
          *reinterpret_cast<uint4*>(q[u]) = *reinterpret_cast<const uint4*>(codes + r * pitch + 16 * static_cast<int64_t>(c));
        }
        byte[u] = scales[mx_scale_word(r, c >> 3, pitch >> 7) + ((c >> 1) & 3)];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = r0 + u * w.row_step;
        if (r >= rows) break;
        Pack16<T> p;
        if (kChunk * static_cast<int64_t>(c) < cols) {
          float v[kChunk];
          float(&lo)[8] = *reinterpret_cast<float(*)[8]>(&v[0]);
          float(&hi)[8] = *reinterpret_cast<float(*)[8]>(&v[8]);
          if constexpr (FMT == kMx4) {
            mx_decode_e2m1(q[u][0], lo);
            mx_decode_e2m1(q[u][1], hi);
          } else {
            mx_decode_e4m3(make_uint2(q[u][0], q[u][1]), lo);
            mx_decode_e4m3(make_uint2(q[u][2], q[u][3]), hi);
          }
          const float s = mx_scale(byte[u]);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) v[j] *= s;
          p = pack16<T>(v);
        }
        store16<VEC>(dst + r * cols, c, cols, p, stage + (VEC ? 0 : warp * 32 * kChunk));
      }
    }
  }
}

// Warps to a row (as a power of two) for so many groups of 512 columns, and the
// blocks that cover `rows`, `per` of them at a time in a warp.
int warps_lg(int64_t groups) { return groups <= 1 ? 0 : groups <= 2 ? 1 : groups <= 4 ? 2 : 3; }
unsigned row_blocks(int64_t rows, int lg, int per, const DeviceInfo& dev) {
  const int64_t of_block = static_cast<int64_t>(per) * ((kThreads / 32) >> lg);
  return static_cast<unsigned>(std::min<int64_t>((rows + of_block - 1) / of_block, int64_t{dev.num_sms} * 8));
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
    const int64_t items = (cols + kTCols<T> - 1) / kTCols<T> * (pitch >> 7);
    const dim3 grid(grid_for(items, 1, dev)), block(kTThreads<T>);
    return cols * sizeof(T) % 16 == 0 && aligned_to(src, 16)
               ? launch_pdl(dbf_mx_quantize_t_kernel<T, FMT, true>, grid, block, 0, stream, s, rows, cols, pitch, codes,
                            scales)
               : launch_pdl(dbf_mx_quantize_t_kernel<T, FMT, false>, grid, block, 0, stream, s, rows, cols, pitch, codes,
                            scales);
  }
  const int64_t pitch = mx_pitch(cols);
  const int lg = warps_lg((pitch + 511) >> 9);
  const bool vec = cols % kChunk == 0 && aligned_to(src, 32);
  const dim3 grid(row_blocks(rows, lg, 1, dev));
  return vec ? launch_pdl(dbf_mx_quantize_kernel<T, FMT, true>, grid, dim3(kThreads), 0, stream, s, rows, cols, pitch, lg,
                          codes, scales)
             : launch_pdl(dbf_mx_quantize_kernel<T, FMT, false>, grid, dim3(kThreads), 0, stream, s, rows, cols, pitch, lg,
                          codes, scales);
}

template <typename T, int FMT>
dbf_status dequantize_typed(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst,
                            const DeviceInfo& dev, cudaStream_t stream) {
  T* d = static_cast<T*>(dst);
  const int64_t pitch = mx_pitch(cols);
  const int lg = warps_lg((cols + 511) >> 9);
  const dim3 grid(row_blocks(rows, lg, kUnroll, dev));
  const bool vec = cols % kChunk == 0 && aligned_to(dst, 32);
  return vec ? launch_pdl(dbf_mx_dequantize_kernel<T, FMT, true>, grid, dim3(kThreads), 0, stream, codes, scales, rows,
                          cols, pitch, lg, d)
             : launch_pdl(dbf_mx_dequantize_kernel<T, FMT, false>, grid, dim3(kThreads), 0, stream, codes, scales, rows,
                          cols, pitch, lg, d);
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
