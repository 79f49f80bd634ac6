// Device helpers of the microscaled (MX) formats and of the kernels that read
// or write 16-bit and fp32 rows sixteen elements at a time.
//
// OCP Microscaling Formats (MX) v1.0: 32 neighbouring elements share a power of
// two 2^(s - 127), s one byte (255: NaN).  The layouts are those of
// include/dbf.h: codes in rows of ceil(cols/128)*128 elements, scales in
// 512-byte tiles of 128 rows x 4 blocks.
#pragma once

#include <cstdint>
#include <type_traits>
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

// ---------------------------------------------------------------- sixteen elements of a row
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

// Sixteen elements as they lie in memory: what a thread holds of a row.
constexpr int kChunk = 16;
template <typename T>
struct alignas(32) Pack16 {
  T e[kChunk];
};

// Whole packs at a time: the conversions of two values run at several times the
// rate of single ones.
__device__ __forceinline__ void unpack16(const Pack16<float>& p, float (&v)[kChunk]) {
#pragma unroll
  for (int j = 0; j < kChunk; ++j) v[j] = p.e[j];
}
__device__ __forceinline__ void unpack16(const Pack16<__half>& p, float (&v)[kChunk]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
  for (int j = 0; j < kChunk / 2; ++j) {
    const float2 f = half2_bits_to_float2(w[j]);
    v[2 * j] = f.x, v[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack16(const Pack16<__nv_bfloat16>& p, float (&v)[kChunk]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
  for (int j = 0; j < kChunk / 2; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
}
template <typename T>
__device__ __forceinline__ Pack16<T> pack16(const float (&v)[kChunk]) {
  Pack16<T> p;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) p.e[j] = v[j];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 t = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&t);
      } else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
  }
  return p;
}

// Two fp32 values side by side, for the instructions that work on both.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
constexpr int kPairs = kChunk / 2;
template <typename T>
__device__ __forceinline__ void unpack16(const Pack16<T>& p, F2 (&v)[kPairs]) {
  float t[kChunk];
  unpack16(p, t);
#pragma unroll
  for (int j = 0; j < kPairs; ++j) v[j] = f2(t[2 * j], t[2 * j + 1]);
}
template <typename T>
__device__ __forceinline__ Pack16<T> pack16(const F2 (&v)[kPairs]) {
  float t[kChunk];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const float2 a = f2_get(v[j]);
    t[2 * j] = a.x, t[2 * j + 1] = a.y;
  }
  return pack16<T>(t);
}

// 32-byte accesses (global memory, 32-byte aligned).
__device__ __forceinline__ void ldg_32(const void* p, uint32_t* r) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void stg_32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Elements 16 c .. 16 c + 15 of a row of `cols` (c consecutive over the warp's
// lanes); those behind the end read as zero and are not written.
// VEC: cols is a multiple of 16 and the row starts on 32 bytes.  Else the warp's
// 512 columns pass through its 512 elements of shared memory, so that
// neighbouring lanes touch neighbouring elements in memory.
template <bool VEC, typename T>
__device__ __forceinline__ Pack16<T> load16(const T* row, int64_t c, int64_t cols, T* stage) {
  Pack16<T> p;
  if constexpr (VEC) {
    uint32_t* r = reinterpret_cast<uint32_t*>(&p);
    if (kChunk * c < cols) {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(p) / 32); ++j) ldg_32(row + kChunk * c + j * (32 / sizeof(T)), r + 8 * j);
    } else {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(p) / 4); ++j) r[j] = 0u;
    }
  } else {
    const int lane = threadIdx.x & 31;
    const int64_t first = kChunk * (c - lane) + lane;
    const int left = static_cast<int>(min(cols - first, int64_t{32 * kChunk}));
    T v[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] = 32 * j < left ? row[first + 32 * j] : from_f32<T>(0.f);
    __syncwarp();  // earlier readers of the stage
#pragma unroll
    for (int j = 0; j < kChunk; ++j) stage[32 * j + lane] = v[j];
    __syncwarp();
    const uint4* src = reinterpret_cast<const uint4*>(stage + kChunk * lane);
    uint4* dst = reinterpret_cast<uint4*>(&p);
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(p) / 16); ++j) dst[j] = src[j];
  }
  return p;
}

// The same of one row that starts on 32 bytes, whatever its length (a weight
// vector): whole chunks in vectors, the last one by elements.
template <typename T>
__device__ __forceinline__ Pack16<T> load16_aligned(const T* row, int64_t c, int64_t cols) {
  if (kChunk * (c + 1) <= cols) return load16<true>(row, c, cols, static_cast<T*>(nullptr));
  Pack16<T> p;
#pragma unroll
  for (int j = 0; j < kChunk; ++j) p.e[j] = kChunk * c + j < cols ? row[kChunk * c + j] : from_f32<T>(0.f);
  return p;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store16(T* row, int64_t c, int64_t cols, const Pack16<T>& p, T* stage) {
  if constexpr (VEC) {
    if (kChunk * c < cols) {
      const uint32_t* r = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(p) / 32); ++j) stg_32(row + kChunk * c + j * (32 / sizeof(T)), r + 8 * j);
    }
  } else {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    uint4* dst = reinterpret_cast<uint4*>(stage + kChunk * lane);
    const uint4* src = reinterpret_cast<const uint4*>(&p);
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(p) / 16); ++j) dst[j] = src[j];
    __syncwarp();
    const int64_t first = kChunk * (c - lane) + lane;
    const int left = static_cast<int>(min(cols - first, int64_t{32 * kChunk}));
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (32 * j < left) row[first + 32 * j] = stage[32 * j + lane];
  }
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A warp's 512 neighbouring columns of one row -> codes and scales: the lane of
// chunk c holds columns 16 c .., a block is two neighbouring lanes (the even one
// stores its scale byte).  Nothing is written from pitch on (pitch: the padded row length, a
// multiple of 128).
template <int FMT>
__device__ __forceinline__ void mx_store_row16(const float (&v)[kChunk], int64_t r, int64_t c, int64_t pitch,
                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int j = 0; j < kChunk; j += 4) {
    m0 = max_abs3(m0, v[j], v[j + 1]);
    m1 = max_abs3(m1, v[j + 2], v[j + 3]);
  }
  const float m = max_abs3(m0, m1, 0.f);
  uint32_t amax = __float_as_uint(m) & 0x7FFFFFFFu;
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t byte = mx_scale_byte<FMT>(amax);
  if (kChunk * c >= pitch) return;
  const bool bad = byte == 255;
  const float inv = mx_inverse_scale(min(byte, 253u));
  float u[kChunk];
#pragma unroll
  for (int j = 0; j < kChunk; j += 2) {
    const float2 t = f2_get(f2_mul(f2(v[j], v[j + 1]), f2(inv, inv)));
    u[j] = t.x, u[j + 1] = t.y;
  }
  const float(&lo)[8] = *reinterpret_cast<const float(*)[8]>(&u[0]);
  const float(&hi)[8] = *reinterpret_cast<const float(*)[8]>(&u[8]);
  if constexpr (FMT == kMx4) {
    const uint2 q = make_uint2(mx_encode_e2m1(lo), mx_encode_e2m1(hi));
    *reinterpret_cast<uint2*>(codes + (r * pitch >> 1) + 8 * c) = bad ? make_uint2(0u, 0u) : q;
  } else {
    const uint4 q = make_uint4(mx_encode_e4m3(u[0], u[1], u[2], u[3]), mx_encode_e4m3(u[4], u[5], u[6], u[7]),
                               mx_encode_e4m3(u[8], u[9], u[10], u[11]), mx_encode_e4m3(u[12], u[13], u[14], u[15]));
    *reinterpret_cast<uint4*>(codes + r * pitch + 16 * c) = bad ? make_uint4(0u, 0u, 0u, 0u) : q;
  }
  if ((c & 1) == 0) scales[mx_scale_word(r, c >> 3, pitch >> 7) + ((c >> 1) & 3)] = static_cast<uint8_t>(byte);
}

}  // namespace dbf
