// Root-mean-square norm with the residual's addition, dense or microscaled
// output, and its gradients.
//
//   h = round(x + residual)            (h = x without a residual)
//   y = h rstd weight,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd g - h rstd^3 mean(g h) + dh,  g = dy weight;  dweight = sum_rows dy h rstd
//
// The sums are fp32.  Every operand is read once where a row fits the block's
// registers, so DRAM bounds all of it; few rows are bound by latency.
#include <algorithm>

#include "dbf_internal.h"
#include "mx_device.cuh"

namespace dbf {
namespace {

constexpr int kDense = 2;  // output kinds: kMx4, kMx8, kDense

struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;
  void* h;  // or null (no residual)
  void* y;  // dense output
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols, pitch;  // pitch: columns padded to 128 (MX output) or 8 (dense)
  float eps;
};

// One block per row (persistent over rows); thread t owns the eight columns of
// chunks t, t + threads, .. (NV of them, held in registers).  NV = 0: any
// number of chunks, the second pass reads h (or x) again.
template <typename T, int OUT, int NV, bool VEC>
__global__ void __launch_bounds__(1024) dbf_rmsnorm_kernel(const NormArgs p) {
  __shared__ float red[2][33];
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  const T* weight = static_cast<const T*>(p.weight);
  const int64_t chunks = p.pitch >> 3;
  int flip = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1) {
    const T* xr = x + r * p.cols;
    const T* rr = res ? res + r * p.cols : nullptr;
    T* hr = res ? static_cast<T*>(p.h) + r * p.cols : nullptr;
    float sum = 0.f;
    auto fetch = [&](int64_t c) {
      Pack8<T> a = load8<VEC>(xr, 8 * c, p.cols);
      if (rr) {
        const Pack8<T> b = load8<VEC>(rr, 8 * c, p.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.e[j] = from_f32<T>(to_f32(a.e[j]) + to_f32(b.e[j]));
        store8<VEC>(hr, 8 * c, p.cols, a);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(to_f32(a.e[j]), to_f32(a.e[j]), sum);
      return a;
    };
    auto finish = [&](int64_t c, const Pack8<T>& a, const Pack8<T>& w, float rstd) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f32(a.e[j]) * rstd * to_f32(w.e[j]);
      if constexpr (OUT == kDense) {
        Pack8<T> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.e[j] = from_f32<T>(v[j]);
        store8<VEC>(static_cast<T*>(p.y) + r * p.cols, 8 * c, p.cols, o);
      } else {
        mx_store_row8<OUT>(v, r, c, p.pitch, p.codes, p.scales);
      }
    };
    const float inv_cols = 1.f / static_cast<float>(p.cols);
    if constexpr (NV > 0) {
      Pack8<T> a[NV], w[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
        a[i] = fetch(c);
        w[i] = load8<VEC>(weight, 8 * c, p.cols);
      }
      const float rstd = 1.f / sqrtf(block_sum(sum, red[flip]) * inv_cols + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) finish(threadIdx.x + static_cast<int64_t>(i) * blockDim.x, a[i], w[i], rstd);
    } else {
      // a whole number of rounds for every thread: the MX store is a warp's work
      const int64_t rounds = (chunks + blockDim.x - 1) / blockDim.x;
      for (int64_t i = 0; i < rounds; ++i) fetch(threadIdx.x + i * blockDim.x);
      const float rstd = 1.f / sqrtf(block_sum(sum, red[flip]) * inv_cols + p.eps);
      const T* again = rr ? hr : xr;
      for (int64_t i = 0; i < rounds; ++i) {
        const int64_t c = threadIdx.x + i * blockDim.x;
        finish(c, load8<VEC>(again, 8 * c, p.cols), load8<VEC>(weight, 8 * c, p.cols), rstd);
      }
    }
  }
}

template <typename T, int OUT, bool VEC>
dbf_status launch_norm(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t chunks = (a.pitch + 7) / 8;
  const int nv = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 0;
  const int64_t want = nv ? (chunks + nv - 1) / nv : 1024;
  const int threads = static_cast<int>((want + 31) / 32 * 32);
  const int per_sm = std::max(1, 2048 / threads);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t{dev.num_sms} * std::min(per_sm, 16))));
  const dim3 block(threads);
  if (nv == 1) return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 1, VEC>, grid, block, 0, stream, a);
  if (nv == 2) return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 2, VEC>, grid, block, 0, stream, a);
  return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 0, VEC>, grid, block, 0, stream, a);
}

template <typename T, int OUT>
dbf_status norm_typed(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.residual, 16) && aligned_to(a.weight, 16) &&
                   aligned_to(a.h, 16) && aligned_to(a.y, 16);
  return vec ? launch_norm<T, OUT, true>(a, dev, stream) : launch_norm<T, OUT, false>(a, dev, stream);
}

template <int OUT>
dbf_status norm_any(const NormArgs& a, dbf_dtype t, const DeviceInfo& dev, cudaStream_t stream) {
  if (t == DBF_F16) return norm_typed<__half, OUT>(a, dev, stream);
  if (t == DBF_BF16) return norm_typed<__nv_bfloat16, OUT>(a, dev, stream);
  return norm_typed<float, OUT>(a, dev, stream);
}

// ---------------------------------------------------------------- gradients
struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* weight;
  const void* dh;  // or null
  void* dx;
  float* dweight;
  float* part;  // blocks x cols fp32: each block's sum over its rows
  int64_t rows, cols;
  int blocks;
  float eps;
};

// Sums of two values per thread over the block; red: 66 floats.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  if (lane == 0) {
    red[warp] = a;
    red[33 + warp] = b;
  }
  __syncthreads();
  float s = lane < warps ? red[lane] : 0.f, t = lane < warps ? red[33 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  return make_float2(s, t);
}

// One block per row at a time, eight columns per thread (cols <= 8192); the
// block's sum of dweight over its rows stays in registers and goes to its row
// of `part`.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) dbf_rmsnorm_grad_kernel(const NormGradArgs p) {
  __shared__ float red[2][66];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = 8 * static_cast<int64_t>(threadIdx.x);
  const Pack8<T> w = load8<VEC>(static_cast<const T*>(p.weight), i, p.cols);
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  float dw[8] = {};
  int flip = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1) {
    const Pack8<T> h = load8<VEC>(static_cast<const T*>(p.h) + r * p.cols, i, p.cols);
    const Pack8<T> dy = load8<VEC>(static_cast<const T*>(p.dy) + r * p.cols, i, p.cols);
    Pack8<T> dh;
    if (p.dh) dh = load8<VEC>(static_cast<const T*>(p.dh) + r * p.cols, i, p.cols);
    float hh = 0.f, gh = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = to_f32(h.e[j]);
      hh = fmaf(a, a, hh);
      gh = fmaf(to_f32(dy.e[j]) * to_f32(w.e[j]), a, gh);
    }
    const float2 s = block_sum2(hh, gh, red[flip]);
    const float rstd = 1.f / sqrtf(s.x * inv_cols + p.eps);
    const float c = rstd * rstd * rstd * (s.y * inv_cols);
    Pack8<T> o;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = to_f32(h.e[j]), d = to_f32(dy.e[j]);
      float v = rstd * (d * to_f32(w.e[j])) - a * c;
      if (p.dh) v += to_f32(dh.e[j]);
      o.e[j] = from_f32<T>(v);
      dw[j] = fmaf(d * a, rstd, dw[j]);
    }
    store8<VEC>(static_cast<T*>(p.dx) + r * p.cols, i, p.cols, o);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < p.cols) p.part[blockIdx.x * p.cols + i + j] = dw[j];
}

// Rows wider than a block: the row's two sums first (from a first reading),
// then dx and the block's dweight row in `part`, accumulated there by the
// thread that owns the column.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) dbf_rmsnorm_grad_wide_kernel(const NormGradArgs p) {
  __shared__ float red[2][66];
  pdl_wait();
  pdl_launch_dependents();
  const T* weight = static_cast<const T*>(p.weight);
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  float* part = p.part + blockIdx.x * p.cols;
  int flip = 0;
  bool first = true;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1, first = false) {
    const T* hr = static_cast<const T*>(p.h) + r * p.cols;
    const T* dyr = static_cast<const T*>(p.dy) + r * p.cols;
    const T* dhr = p.dh ? static_cast<const T*>(p.dh) + r * p.cols : nullptr;
    float hh = 0.f, gh = 0.f;
    for (int64_t i = 8 * static_cast<int64_t>(threadIdx.x); i < p.cols; i += 8 * blockDim.x) {
      const Pack8<T> h = load8<VEC>(hr, i, p.cols), dy = load8<VEC>(dyr, i, p.cols), w = load8<VEC>(weight, i, p.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = to_f32(h.e[j]);
        hh = fmaf(a, a, hh);
        gh = fmaf(to_f32(dy.e[j]) * to_f32(w.e[j]), a, gh);
      }
    }
    const float2 s = block_sum2(hh, gh, red[flip]);
    const float rstd = 1.f / sqrtf(s.x * inv_cols + p.eps);
    const float c = rstd * rstd * rstd * (s.y * inv_cols);
    for (int64_t i = 8 * static_cast<int64_t>(threadIdx.x); i < p.cols; i += 8 * blockDim.x) {
      const Pack8<T> h = load8<VEC>(hr, i, p.cols), dy = load8<VEC>(dyr, i, p.cols), w = load8<VEC>(weight, i, p.cols);
      Pack8<T> dh, o;
      if (dhr) dh = load8<VEC>(dhr, i, p.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = to_f32(h.e[j]), d = to_f32(dy.e[j]);
        float v = rstd * (d * to_f32(w.e[j])) - a * c;
        if (dhr) v += to_f32(dh.e[j]);
        o.e[j] = from_f32<T>(v);
        if (i + j < p.cols) part[i + j] = fmaf(d * a, rstd, first ? 0.f : part[i + j]);
      }
      store8<VEC>(static_cast<T*>(p.dx) + r * p.cols, i, p.cols, o);
    }
  }
}

// dweight[c] = sum over the blocks' rows of `part`, in their order.  32 columns
// and 8 runs of rows per block.
__global__ void __launch_bounds__(256) dbf_rmsnorm_grad_sum_kernel(const NormGradArgs p) {
  __shared__ float tile[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t c = 32 * static_cast<int64_t>(blockIdx.x) + lane;
  float s = 0.f;
  if (c < p.cols)
    for (int b = run; b < p.blocks; b += 8) s += p.part[b * p.cols + c];
  tile[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < p.cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += tile[k][lane];
    p.dweight[c] = s;
  }
}

constexpr int64_t kGradRowCols = 8192;  // eight columns for each of 1024 threads
constexpr int kGradBlocks = 2 * 148;    // rows of `part` at most

template <typename T, bool VEC>
dbf_status launch_grad(NormGradArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  a.blocks = static_cast<int>(std::min<int64_t>(a.rows, kGradBlocks));
  dbf_status st;
  if (a.cols <= kGradRowCols) {
    const int threads = static_cast<int>(((a.cols + 7) / 8 + 31) / 32 * 32);
    st = launch_pdl(dbf_rmsnorm_grad_kernel<T, VEC>, dim3(a.blocks), dim3(threads), 0, stream, a);
  } else {
    st = launch_pdl(dbf_rmsnorm_grad_wide_kernel<T, VEC>, dim3(a.blocks), dim3(1024), 0, stream, a);
  }
  if (st != DBF_OK) return st;
  return launch_pdl(dbf_rmsnorm_grad_sum_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32)), dim3(256), 0, stream,
                    a);
}

template <typename T>
dbf_status grad_typed(const NormGradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && aligned_to(a.dy, 16) && aligned_to(a.h, 16) && aligned_to(a.weight, 16) &&
                   aligned_to(a.dh, 16) && aligned_to(a.dx, 16);
  return vec ? launch_grad<T, true>(a, dev, stream) : launch_grad<T, false>(a, dev, stream);
}

constexpr int64_t kMaxNormCols = int64_t{1} << 20;

bool norm_shape_ok(int64_t rows, int64_t cols) { return mx_shape_ok(rows, cols) && cols <= kMaxNormCols; }

dbf_status check_norm(const NormArgs& a, dbf_dtype t) {
  if (!a.x || !a.weight || (a.residual != nullptr) != (a.h != nullptr) || !float_dtype_ok(t)) return DBF_ERR_INVALID_ARG;
  if (a.rows < 1 || a.cols < 1 || !(a.eps >= 1.17549435e-38f) || !(a.eps <= 3.402823466e38f)) return DBF_ERR_INVALID_ARG;
  if (!norm_shape_ok(a.rows, a.cols)) return DBF_ERR_UNSUPPORTED_SHAPE;
  const size_t e = dtype_size(t);
  if (!aligned_to(a.x, e) || !aligned_to(a.weight, e) || !aligned_to(a.residual, e) || !aligned_to(a.h, e))
    return DBF_ERR_MISALIGNED;
  return DBF_OK;
}

}  // namespace
}  // namespace dbf

using namespace dbf;

extern "C" {

dbf_status dbf_rmsnorm_forward(const void* x, const void* residual, const void* weight, dbf_dtype t, int64_t rows,
                               int64_t cols, float eps, void* h, void* y, struct CUstream_st* stream) {
  NormArgs a{x, residual, weight, h, y, nullptr, nullptr, rows, cols, cols, eps};
  if (!y) return DBF_ERR_INVALID_ARG;
  dbf_status st = check_norm(a, t);
  if (st != DBF_OK) return st;
  if (!aligned_to(y, dtype_size(t))) return DBF_ERR_MISALIGNED;
  a.pitch = (cols + 7) / 8 * 8;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != DBF_OK) return st;
  return norm_any<kDense>(a, t, dev, reinterpret_cast<cudaStream_t>(stream));
}

dbf_status dbf_rmsnorm_mx_forward(const void* x, const void* residual, const void* weight, dbf_dtype t, int64_t rows,
                                  int64_t cols, float eps, dbf_mx_format fmt, void* h, uint8_t* codes, uint8_t* scales,
                                  struct CUstream_st* stream) {
  NormArgs a{x, residual, weight, h, nullptr, codes, scales, rows, cols, cols, eps};
  if (!codes || !scales || !mx_format_ok(fmt)) return DBF_ERR_INVALID_ARG;
  dbf_status st = check_norm(a, t);
  if (st != DBF_OK) return st;
  if (!aligned_to(codes, 32) || !aligned_to(scales, 16)) return DBF_ERR_MISALIGNED;
  a.pitch = mx_pitch(cols);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != DBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return fmt == DBF_MX_E2M1 ? norm_any<kMx4>(a, t, dev, s) : norm_any<kMx8>(a, t, dev, s);
}

size_t dbf_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (!norm_shape_ok(rows, cols)) return 0;
  return static_cast<size_t>(std::min<int64_t>(rows, kGradBlocks)) * static_cast<size_t>(cols) * 4;
}

dbf_status dbf_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh, dbf_dtype t,
                                int64_t rows, int64_t cols, float eps, void* dx, float* dweight, void* workspace,
                                size_t ws_bytes, struct CUstream_st* stream) {
  if (!dy || !dx || !dweight) return DBF_ERR_INVALID_ARG;
  NormArgs check{h, nullptr, weight, nullptr, nullptr, nullptr, nullptr, rows, cols, cols, eps};
  dbf_status st = check_norm(check, t);
  if (st != DBF_OK) return st;
  const size_t e = dtype_size(t);
  if (!aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(dx, e) || !aligned_to(dweight, 4))
    return DBF_ERR_MISALIGNED;
  if (!workspace || !aligned_to(workspace, 16) || ws_bytes < dbf_rmsnorm_backward_workspace_bytes(rows, cols))
    return DBF_ERR_WORKSPACE;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != DBF_OK) return st;
  const NormGradArgs a{dy, h, weight, dh, dx, dweight, static_cast<float*>(workspace), rows, cols, 0, eps};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (t == DBF_F16) return grad_typed<__half>(a, dev, s);
  if (t == DBF_BF16) return grad_typed<__nv_bfloat16>(a, dev, s);
  return grad_typed<float>(a, dev, s);
}

}  // extern "C"
