// Device helpers of the microscaled (MX) formats and of the kernels that read
// or write 16-bit and fp32 rows eight elements at a time.
//
// OCP Microscaling Formats (MX) v1.0: 32 neighbouring elements share a power of
// two 2^(s - 127), s one byte (255: NaN).  The layouts are those of
// include/dbf.h: codes in rows of ceil(cols/128)*128 elements, scales in
// 512-byte tiles of 128 rows x 4 blocks.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dbf_device.cuh"

namespace dbf {

constexpr int kMx4 = 0;  // DBF_MX_E2M1
constexpr int kMx8 = 1;  // DBF_MX_E4M3

// Largest exponent of an element: 6 = 1.5 * 2^2, 448 = 1.75 * 2^8.
template <int FMT>
constexpr int kMxTop = FMT == kMx4 ? 2 : 8;

// Byte offset of the scale word (4 blocks) of row r, blocks 4 k4 .. 4 k4 + 3;
// k4s = ceil(cols / 128) words per row.
__host__ __device__ __forceinline__ int64_t mx_scale_word(int64_t r, int64_t k4, int64_t k4s) {
  return ((r >> 7) * k4s + k4) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// The scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign cleared): floor(log2(amax)) - top, clamped to the byte's range.  An
// infinity or NaN among the 32 values has the all-ones exponent, which is the
// largest as an integer too, and makes the block NaN.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - kMxTop<FMT>, 0));
}

// 2^(127 - byte): what the elements are multiplied by before rounding (exact;
// byte <= 252 here).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127) as fp32 (byte 0 is a subnormal, 255 is NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Eight values -> eight e2m1 codes (round to nearest even, saturating), the
// even element in the low half of each byte.
__device__ __forceinline__ uint32_t mx_encode_e2m1(const float (&v)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

// Four values -> four e4m3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t mx_encode_e4m3(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}

__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight e2m1 codes -> values.
__device__ __forceinline__ void mx_decode_e2m1(uint32_t w, float (&v)[8]) {
  uint32_t h0, h1, h2, h3;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
  const float2 a = half2_bits_to_float2(h0), b = half2_bits_to_float2(h1), c = half2_bits_to_float2(h2),
               d = half2_bits_to_float2(h3);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

// Eight e4m3 codes (two words) -> values.
__device__ __forceinline__ void mx_decode_e4m3(uint2 w, float (&v)[8]) {
  uint32_t h0, h1, h2, h3;
  asm("{\n\t.reg .b16 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1}, %4;\n\t"
      "mov.b32 {b2, b3}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, b3;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w.x), "r"(w.y));
  const float2 a = half2_bits_to_float2(h0), b = half2_bits_to_float2(h1), c = half2_bits_to_float2(h2),
               d = half2_bits_to_float2(h3);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

// ---------------------------------------------------------------- eight elements of a row
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// Eight elements as they lie in memory.
template <typename T>
struct alignas(16) Pack8 {
  T e[8];
};

// Elements i .. i+7 of a row of `cols`; those behind the end read as zero.
// VEC: i + 8 <= cols wherever i < cols, and the row starts on 16 bytes.
template <bool VEC, typename T>
__device__ __forceinline__ Pack8<T> load8(const T* row, int64_t i, int64_t cols) {
  Pack8<T> p;
  if constexpr (VEC) {
    if (i < cols) {
      const uint4* src = reinterpret_cast<const uint4*>(row + i);
      uint4* dst = reinterpret_cast<uint4*>(&p);
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(p) / 16); ++j) dst[j] = src[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.e[j] = from_f32<T>(0.f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p.e[j] = i + j < cols ? row[i + j] : from_f32<T>(0.f);
  }
  return p;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int64_t i, int64_t cols, const Pack8<T>& p) {
  if constexpr (VEC) {
    if (i < cols) {
      uint4* dst = reinterpret_cast<uint4*>(row + i);
      const uint4* src = reinterpret_cast<const uint4*>(&p);
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(p) / 16); ++j) dst[j] = src[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < cols) row[i + j] = p.e[j];
  }
}

// A warp's 256 neighbouring columns of one row -> codes and scales: lane l holds
// columns 8 l .. 8 l + 7, a block is four neighbouring lanes, a scale word
// sixteen.  c = column / 8 of this lane; nothing is written from pitch on
// (pitch: the padded row length, a multiple of 128).
template <int FMT>
__device__ __forceinline__ void mx_store_row8(const float (&v)[8], int64_t r, int64_t c, int64_t pitch,
                                              uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t byte = mx_scale_byte<FMT>(amax);
  const int lane = threadIdx.x & 31;
  uint32_t word = byte << (8 * ((lane >> 2) & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
  float u[8];
  const float inv = mx_inverse_scale(min(byte, 253u));
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = byte == 255 ? 0.f : v[j] * inv;
  if (8 * c >= pitch) return;
  if constexpr (FMT == kMx4) {
    *reinterpret_cast<uint32_t*>(codes + (r * pitch >> 1) + 4 * c) = mx_encode_e2m1(u);
  } else {
    *reinterpret_cast<uint2*>(codes + r * pitch + 8 * c) =
        make_uint2(mx_encode_e4m3(u[0], u[1], u[2], u[3]), mx_encode_e4m3(u[4], u[5], u[6], u[7]));
  }
  if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(r, c >> 4, pitch >> 7)) = word;
}

// Sum of one value per thread over the block (every thread gets it).  `red`:
// 33 floats of shared memory, free to be reused after the next __syncthreads.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = lane < warps ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

}  // namespace dbf
