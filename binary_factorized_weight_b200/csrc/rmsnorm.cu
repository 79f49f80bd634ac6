// Root-mean-square norm with the residual's addition, dense or microscaled
// output, and its gradients.
//
//   h = round(x + residual)            (h = x without a residual)
//   y = h rstd weight,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd g - h rstd^3 mean(g h) + dh,  g = dy weight;  dweight = sum_rows dy h rstd
//      = rstd g - x (rstd mean(g x)) + dh with x = h rstd, as it is computed
//
// The sums are fp32.  Every operand is read once where a row fits the block's
// registers, so DRAM bounds all of it; few rows are bound by latency.  2048 x 4096
// bf16 with residual: into 8 bits 11.4 us (5.2 TB/s, 79% of the copy rate), dense
// 13.5 us (76%), gradients with dh 16.7 us (4.0 TB/s, 61%: the second kernel, which
// adds the blocks' dweight, is about 3 us of it).  One row of 4096: 2.0 us.
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
  int weight_aligned;  // to 32 bytes
};

// Sum of one value per thread over the row's threads (every thread gets it):
// the warp's where a row is a warp's work, else the block's.  `red`: 32 floats
// of shared memory, free to be reused two calls later.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = lane < warps ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

constexpr int kWarpRows = 8;          // rows of a block whose warps take a row each
constexpr int kStagedThreads = 512;   // threads of a block that stages its rows in shared memory, at most

// A row is the work of one warp (WARP: up to 1024 columns, eight rows to a
// block) or of a block; persistent over rows.  Thread t of the row owns the
// sixteen columns of chunks t, t + threads, .. (NV of them, held in registers,
// so everything is read once; of two chunks in aligned blocks of up to 1024 threads,
// 16385 to 32768 columns, 128 bytes a thread in 16 bits and some 500 in fp32
// are spilled).  NV = 0: any number of chunks, the second pass reads h (or x) again.
template <typename T, int OUT, int NV, bool VEC, bool WARP>
__global__ void __launch_bounds__(VEC && !WARP ? 1024 : kStagedThreads) dbf_rmsnorm_kernel(const NormArgs p) {
  __shared__ float red[2][32];
  __shared__ alignas(32) T stages[VEC ? 1 : (WARP ? 32 * kWarpRows : kStagedThreads) * kChunk];
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  const T* weight = static_cast<const T*>(p.weight);
  T* stage = stages + (VEC ? 0 : (threadIdx.x >> 5) * 32 * kChunk);
  const int me = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * (WARP ? kWarpRows : 1);
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  auto load_weight = [&](int64_t c) {
    if (!VEC && p.weight_aligned) return load16_aligned(weight, c, p.cols);
    return load16<VEC>(weight, c, p.cols, stage);
  };
  int flip = 0;
  for (int64_t r = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x; r < p.rows;
       r += row_step, flip ^= 1) {
    const T* xr = x + r * p.cols;
    const T* rr = res ? res + r * p.cols : nullptr;
    T* hr = res ? static_cast<T*>(p.h) + r * p.cols : nullptr;
    F2 sums = f2(0.f, 0.f);
    auto add = [&](int64_t c, Pack16<T> a, const Pack16<T>& b) {
      F2 v[kPairs];
      unpack16(a, v);
      if (rr) {
        F2 u[kPairs];
        unpack16(b, u);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = f2_add(v[j], u[j]);
        a = pack16<T>(v);
        store16<VEC>(hr, c, p.cols, a, stage);
        unpack16(a, v);
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) sums = f2_fma(v[j], v[j], sums);
      return a;
    };
    auto rstd_of = [&]() {
      const float2 t = f2_get(sums);
      return 1.f / sqrtf(row_sum<WARP>(t.x + t.y, red[flip]) * inv_cols + p.eps);
    };
    auto finish = [&](int64_t c, const Pack16<T>& a, const Pack16<T>& w, float rstd) {
      F2 v[kPairs], g[kPairs];
      unpack16(a, v);
      unpack16(w, g);
      // A NaN rstd would make NaN of the zeros behind the last column, and with them
      // of blocks that hold nothing.  (A block that holds a column is NaN then.)
      if (OUT != kDense && kChunk * c >= p.cols) rstd = 0.f;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) v[j] = f2_mul(f2_mul(v[j], f2(rstd, rstd)), g[j]);
      if constexpr (OUT == kDense) {
        store16<VEC>(static_cast<T*>(p.y) + r * p.cols, c, p.cols, pack16<T>(v), stage);
      } else {
        float t[kChunk];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 e = f2_get(v[j]);
          t[2 * j] = e.x, t[2 * j + 1] = e.y;
        }
        mx_store_row16<OUT>(t, r, c, p.pitch, p.codes, p.scales);
      }
    };
    if constexpr (NV > 0) {
      // all loads before the first use
      Pack16<T> a[NV], b[NV], w[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = me + i * threads;
        a[i] = load16<VEC>(xr, c, p.cols, stage);
        if (rr) b[i] = load16<VEC>(rr, c, p.cols, stage);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i] = load_weight(me + i * threads);
#pragma unroll
      for (int i = 0; i < NV; ++i) a[i] = add(me + i * threads, a[i], b[i]);
      const float rstd = rstd_of();
#pragma unroll
      for (int i = 0; i < NV; ++i) finish(me + i * threads, a[i], w[i], rstd);
    } else {
      // a whole number of rounds for every thread: staging and the MX store are a warp's work
      const int64_t rounds = ((p.pitch + kChunk - 1) / kChunk + threads - 1) / threads;
      for (int64_t i = 0; i < rounds; ++i) {
        const int64_t c = me + i * threads;
        const Pack16<T> a = load16<VEC>(xr, c, p.cols, stage);
        add(c, a, rr ? load16<VEC>(rr, c, p.cols, stage) : a);
      }
      const float rstd = rstd_of();
      const T* again = rr ? hr : xr;
      for (int64_t i = 0; i < rounds; ++i) {
        const int64_t c = me + i * threads;
        finish(c, load16<VEC>(again, c, p.cols, stage), load_weight(c), rstd);
      }
    }
  }
}

// With few rows (less than one to an SM) a row gets as many threads as it has
// chunks; else up to 1024 columns are one warp's work.
template <typename T, int OUT, bool VEC>
dbf_status launch_norm(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t chunks = (a.pitch + kChunk - 1) / kChunk;
  if (chunks <= 64 && (chunks <= 32 || a.rows >= dev.num_sms)) {
    const dim3 grid(static_cast<unsigned>(
        std::min<int64_t>((a.rows + kWarpRows - 1) / kWarpRows, int64_t{dev.num_sms} * 8)));
    const dim3 block(32 * kWarpRows);
    if (chunks <= 32) return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 1, VEC, true>, grid, block, 0, stream, a);
    return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 2, VEC, true>, grid, block, 0, stream, a);
  }
  const int most = VEC ? 1024 : kStagedThreads;
  const int nv = chunks <= most ? 1 : chunks <= 2 * most ? 2 : 0;
  const int64_t want = nv ? (chunks + nv - 1) / nv : most;
  const int threads = static_cast<int>((want + 31) / 32 * 32);
  const dim3 grid(
      static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t{dev.num_sms} * std::min(std::max(1, 2048 / threads), 16))));
  const dim3 block(threads);
  if (nv == 1) return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 1, VEC, false>, grid, block, 0, stream, a);
  if (nv == 2) return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 2, VEC, false>, grid, block, 0, stream, a);
  return launch_pdl(dbf_rmsnorm_kernel<T, OUT, 0, VEC, false>, grid, block, 0, stream, a);
}

template <typename T, int OUT>
dbf_status norm_typed(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  NormArgs args = a;
  args.weight_aligned = aligned_to(a.weight, 32);
  const bool vec = a.cols % kChunk == 0 && aligned_to(a.x, 32) && aligned_to(a.residual, 32) &&
                   aligned_to(a.weight, 32) && aligned_to(a.h, 32) && aligned_to(a.y, 32);
  return vec ? launch_norm<T, OUT, true>(args, dev, stream) : launch_norm<T, OUT, false>(args, dev, stream);
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

// Sums of M values per thread over the row's threads; red: 32 M floats.
template <bool WARP, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  }
  if (WARP) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane < M) {
    float mine = v[0];
#pragma unroll
    for (int m = 1; m < M; ++m) mine = lane == m ? v[m] : mine;
    red[warp * M + lane] = mine;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = lane < warps ? red[lane * M + m] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  }
}

// A row is the work of one warp (SPAN 0, eight rows to a block), of a block
// (SPAN 1) or of a cluster of blocks (SPAN 2, which exchange their sums through
// distributed shared memory); sixteen columns per thread, whose sums of dweight
// over the rows stay in registers and go to the row of `part`.  Few rows (SPAN 3):
// one cluster of blocks takes the rows in turn and adds dweight itself, each
// block an eighth of the columns, so that no second launch is needed.
// VEC: a thread owns sixteen neighbouring columns (32-byte accesses); else every
// 32nd of its warp's 512 columns.  PRE: the next row is loaded while this one is reduced (16-
// bit elements: more does not fit the registers; the unaligned forms spill 32 to 48
// bytes of it).
constexpr int kGradThreads = 512;
constexpr int kFewBlocks = 8;  // SPAN 3: the blocks of the cluster
template <typename T, bool VEC, int SPAN>
__global__ void __launch_bounds__(SPAN == 0 ? 32 * kWarpRows : kGradThreads, SPAN == 0 ? 2 : 1)
    dbf_rmsnorm_grad_kernel(const NormGradArgs p) {
  constexpr bool PRE = sizeof(T) == 2, WARP = SPAN == 0;
  __shared__ float red[2][64];
  __shared__ float sums[WARP ? kWarpRows * kChunk * 32 : 1];
  __shared__ float2 ranks[SPAN == 2 ? 2 : 1][8];  // the cluster's sums of a row
  __shared__ float slices[SPAN == 3 ? kChunk * 256 + kFewBlocks * kChunk : 1];  // the cluster's sums of this block's columns
  pdl_wait();
  pdl_launch_dependents();
  const int ks = SPAN == 2 ? static_cast<int>(cluster_size()) : 1;
  const int rank = SPAN == 2 ? static_cast<int>(cluster_rank()) : 0;
  if constexpr (SPAN >= 2) {  // peers write here once every block has started
    cluster_arrive_relaxed();
    cluster_wait_acquire();
  }
  const int me = WARP ? threadIdx.x & 31 : rank * blockDim.x + threadIdx.x;
  const int group = WARP ? threadIdx.x >> 5 : 0;
  const int block = blockIdx.x / ks, blocks = gridDim.x / ks;  // a cluster counts as one
  const int64_t row0 = static_cast<int64_t>(block) * (WARP ? kWarpRows : 1) + group;
  const int64_t row_step = static_cast<int64_t>(blocks) * (WARP ? kWarpRows : 1);
  // this thread's first column, the distance between its columns, and how far the row goes from there
  const int first = VEC ? kChunk * me : kChunk * (me & ~31) + (me & 31);
  constexpr int kStride = VEC ? 1 : 32;
  const int left = static_cast<int>(min(p.cols - first, int64_t{kStride * kChunk}));
  // this thread's elements of a row (zero behind the last column)
  auto load = [&](const void* base, int64_t r) {
    const T* row = static_cast<const T*>(base) + r * p.cols;
    if constexpr (VEC) {
      return load16<true>(row, me, p.cols, static_cast<T*>(nullptr));
    } else {
      Pack16<T> a;
#pragma unroll
      for (int j = 0; j < kChunk; ++j) a.e[j] = kStride * j < left ? row[first + kStride * j] : from_f32<T>(0.f);
      return a;
    }
  };
  struct Row {
    Pack16<T> h, dy, dh;
  };
  auto load_row = [&](int64_t r, Row& a) {
    a.h = load(p.h, r);
    a.dy = load(p.dy, r);
    if (p.dh) a.dh = load(p.dh, r);
  };
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  Row a;
  if (row0 < p.rows) load_row(row0, a);
  const Pack16<T> w = load(p.weight, 0);
  F2 dw[kPairs];
#pragma unroll
  for (int n = 0; n < kPairs; ++n) dw[n] = f2(0.f, 0.f);
  int flip = 0;
  for (int64_t r = row0; r < p.rows; r += row_step, flip ^= 1) {
    Row next;
    if (PRE && r + row_step < p.rows) load_row(r + row_step, next);
    F2 hh = f2(0.f, 0.f), gh = hh;
    {
      F2 h[kPairs], dy[kPairs], g[kPairs];
      unpack16(a.h, h);
      unpack16(a.dy, dy);
      unpack16(w, g);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        hh = f2_fma(h[j], h[j], hh);
        gh = f2_fma(f2_mul(dy[j], g[j]), h[j], gh);
      }
    }
    const float2 th = f2_get(hh), tg = f2_get(gh);
    float s[2] = {th.x + th.y, tg.x + tg.y};
    row_sums<WARP, 2>(s, red[flip]);
    if constexpr (SPAN == 2) {
      if (threadIdx.x < ks) {
        const uint32_t to = map_to_rank(&ranks[flip][rank], threadIdx.x);
        st_cluster_f32(to, s[0]);
        st_cluster_f32(to + 4, s[1]);
      }
      cluster_arrive_release();
      cluster_wait_acquire();
      s[0] = s[1] = 0.f;
      for (int k = 0; k < ks; ++k) {
        s[0] += ranks[flip][k].x;
        s[1] += ranks[flip][k].y;
      }
    }
    // x = h rstd is of ordinary size whatever h and eps are, and rstd mean(g x) of dx's.
    // A power of rstd by itself is not: its cube leaves fp32 at |h| about 1e13, or
    // with eps below 2e-26 and a row of zeros.
    const float rstd = 1.f / sqrtf(s[0] * inv_cols + p.eps);
    const float m = -(rstd * (rstd * (s[1] * inv_cols)));
    const F2 rstd2 = f2(rstd, rstd), m2 = f2(m, m);
    T* dx = static_cast<T*>(p.dx) + r * p.cols;
    F2 h[kPairs], dy[kPairs], g[kPairs];
    unpack16(a.h, h);
    unpack16(a.dy, dy);
    unpack16(w, g);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const F2 x = f2_mul(h[j], rstd2), t = f2_mul(dy[j], rstd2);
      dw[j] = f2_fma(dy[j], x, dw[j]);
      h[j] = f2_fma(x, m2, f2_mul(t, g[j]));
    }
    if (p.dh) {
      unpack16(a.dh, g);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) h[j] = f2_add(h[j], g[j]);
    }
    const Pack16<T> o = pack16<T>(h);
    if constexpr (VEC) {
      store16<true>(dx, me, p.cols, o, static_cast<T*>(nullptr));
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (kStride * j < left) dx[first + kStride * j] = o.e[j];
    }
    if (PRE) a = next;
    else if (r + row_step < p.rows) load_row(r + row_step, a);
  }
  float dws[kChunk];
#pragma unroll
  for (int n = 0; n < kPairs; ++n) {
    const float2 t = f2_get(dw[n]);
    dws[2 * n] = t.x, dws[2 * n + 1] = t.y;
  }
  if constexpr (SPAN == 3) {
    // a block's slice: whole chunks of sixteen columns; blocks in their order
    const int each = static_cast<int>((p.cols + kChunk * kFewBlocks - 1) / (kChunk * kFewBlocks)) * kChunk;
    const int self = static_cast<int>(cluster_rank());
#pragma unroll
    for (int n = 0; n < kChunk; ++n) {
      if (kStride * n >= left) break;
      const int c = first + kStride * n, owner = c / each;
      st_cluster_f32(map_to_rank(&slices[self * each + c - owner * each], owner), dws[n]);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    for (int i = threadIdx.x; i < each; i += blockDim.x) {
      const int64_t c = static_cast<int64_t>(self) * each + i;
      if (c >= p.cols) break;
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kFewBlocks; ++k) t += slices[k * each + i];
      p.dweight[c] = t;
    }
    return;
  }
  float* part = p.part + block * p.cols + first;
  if constexpr (WARP) {
    // the block's warps in their order
#pragma unroll
    for (int n = 0; n < kChunk; ++n) sums[(group * kChunk + n) * 32 + me] = dws[n];
    __syncthreads();
    for (int n = group; n < kChunk; n += kWarpRows) {
      float t = 0.f;
#pragma unroll
      for (int g = 0; g < kWarpRows; ++g) t += sums[(g * kChunk + n) * 32 + me];
      if (kStride * n < left) part[kStride * n] = t;
    }
  } else {
#pragma unroll
    for (int n = 0; n < kChunk; n += 4) {
      if (VEC) {
        if (n < left) *reinterpret_cast<float4*>(part + n) = make_float4(dws[n], dws[n + 1], dws[n + 2], dws[n + 3]);
      } else {
#pragma unroll
        for (int k = n; k < n + 4; ++k)
          if (kStride * k < left) part[kStride * k] = dws[k];
      }
    }
  }
}

// Rows wider than a block's registers: the row's two sums from a first reading,
// then dx and the block's dweight row in `part`, accumulated there by the
// thread that owns the column.  The second reading loads kWide of a thread's columns
// before it stores any (dx may be dy or dh, so the compiler moves no load past a
// store): with the loop left to it the same arithmetic took 260 us for 300 x 70000
// bf16 with dh, so 153 (1.1 TB/s over the four operands).
constexpr int kWide = 4;
template <typename T>
__global__ void __launch_bounds__(1024) dbf_rmsnorm_grad_wide_kernel(const NormGradArgs p) {
  __shared__ float red[2][64];
  pdl_wait();
  pdl_launch_dependents();
  const T* weight = static_cast<const T*>(p.weight);
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  float* part = p.part + blockIdx.x * p.cols;
  int flip = 0;
  bool first = true;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1, first = false) {
    const T* h = static_cast<const T*>(p.h) + r * p.cols;
    const T* dy = static_cast<const T*>(p.dy) + r * p.cols;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + r * p.cols : nullptr;
    T* dx = static_cast<T*>(p.dx) + r * p.cols;
    float hh = 0.f, gh = 0.f;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < p.cols; i += blockDim.x) {
      const float a = to_f32(h[i]);
      hh = fmaf(a, a, hh);
      gh = fmaf(to_f32(dy[i]) * to_f32(weight[i]), a, gh);
    }
    float s[2] = {hh, gh};
    row_sums<false, 2>(s, red[flip]);
    const float rstd = 1.f / sqrtf(s[0] * inv_cols + p.eps);
    const float m = -(rstd * (rstd * (s[1] * inv_cols)));
    auto columns = [&](int64_t i0, auto count) {
      constexpr int kN = decltype(count)::value;
      T hv[kN], dv[kN], wv[kN], ev[kN];
      float sum[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int64_t i = i0 + k * blockDim.x;
        hv[k] = h[i], dv[k] = dy[i], wv[k] = weight[i];
        if (dh) ev[k] = dh[i];
        sum[k] = first ? 0.f : part[i];
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int64_t i = i0 + k * blockDim.x;
        const float x = to_f32(hv[k]) * rstd, d = to_f32(dv[k]);
        float v = fmaf(x, m, rstd * (d * to_f32(wv[k])));
        if (dh) v += to_f32(ev[k]);
        dx[i] = from_f32<T>(v);
        part[i] = fmaf(d, x, sum[k]);
      }
    };
    int64_t i = threadIdx.x;
    for (; i + (kWide - 1) * blockDim.x < p.cols; i += kWide * blockDim.x)
      columns(i, std::integral_constant<int, kWide>());
    for (; i < p.cols; i += blockDim.x) columns(i, std::integral_constant<int, 1>());
  }
}

// dweight[c] = sum over the blocks' rows of `part`, in a fixed order.  A block
// takes COLS columns by RUNS runs of rows.  The loads' latency bounds it: 296
// rows of 4096 columns took 5 us more with 8 runs than with 64.  Narrow rows
// need the runs most (4096 x 64: 7.0 us of the whole call with 32, 5.6 with
// 128), wide ones the whole sectors (2048 x 8192: 27.7 with 32, 29.2 with 64).
template <int COLS, int RUNS>
__global__ void __launch_bounds__(COLS * RUNS) dbf_rmsnorm_grad_sum_kernel(const NormGradArgs p) {
  __shared__ float tile[RUNS][COLS + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int col = threadIdx.x % COLS, run = threadIdx.x / COLS;
  const int64_t c = COLS * static_cast<int64_t>(blockIdx.x) + col;
  float s = 0.f;
  if (c < p.cols) {
    const float* part = p.part + c;
#pragma unroll(RUNS == 32 ? 10 : RUNS == 64 ? 5 : 4)
    for (int b = run; b < p.blocks; b += RUNS) s += part[b * p.cols];
  }
  tile[run][col] = s;
  __syncthreads();
  // warp w adds column w's runs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= COLS) return;
  s = 0.f;
#pragma unroll
  for (int k = lane; k < RUNS; k += 32) s += tile[k][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t out = COLS * static_cast<int64_t>(blockIdx.x) + warp;
  if (lane == 0 && out < p.cols) p.dweight[out] = s;
}

template <int COLS, int RUNS>
dbf_status launch_grad_sum(const NormGradArgs& a, cudaStream_t stream) {
  return launch_pdl(dbf_rmsnorm_grad_sum_kernel<COLS, RUNS>, dim3(static_cast<unsigned>((a.cols + COLS - 1) / COLS)),
                    dim3(COLS * RUNS), 0, stream, a);
}

// How the rows are shared out, from the sizes alone (the workspace's size and
// dweight's order of additions follow from it).  Clusters are counted by the SMs, not
// by how many are resident together: of eight blocks fewer than 18 may be, and the
// rest then run behind them.
constexpr int kGradSms = 148;
constexpr int64_t kFewRows = 16;
struct GradPlan {
  int span;     // a row is the work of 0: a warp, 1: a block, 2: a cluster, 3: a block (one cluster in all), 4: a block, any width
  int ks;       // blocks of a cluster
  int threads;  // of a block
  int blocks;   // rows of `part`
};
GradPlan grad_plan(int64_t rows, int64_t cols) {
  const int64_t chunks = (cols + kChunk - 1) / kChunk;
  auto count = [&](int64_t units, int most) { return static_cast<int>(std::min<int64_t>(units, most)); };
  // Few rows: the second launch costs the host more than two rows in turn cost a
  // block.  A call, wall clock: 8 rows of 4096 bf16 5.7 us, with two launches 7.2;
  // 16 rows 6.6 (1111 fp32: 5.2); 32 rows 8.4; wider rows (8192 fp32) 9.9.
  if (rows <= kFewRows && chunks <= 256)
    return {3, kFewBlocks, static_cast<int>((chunks + 31) / 32 * 32), 1};
  if (chunks <= 32) return {0, 1, 32 * kWarpRows, count((rows + kWarpRows - 1) / kWarpRows, 2 * kGradSms)};
  const int ks = chunks <= kGradThreads ? 1 : chunks <= 2 * kGradThreads ? 2 : chunks <= 4 * kGradThreads ? 4 : 8;
  if (chunks > 8 * kGradThreads) return {4, 1, 1024, count(rows, 2 * kGradSms)};
  const int threads = static_cast<int>(((chunks + ks - 1) / ks + 31) / 32 * 32);
  if (ks > 1) return {2, ks, threads, count(rows, kGradSms / ks)};
  return {1, 1, threads, count(rows, kGradSms * std::min(kGradThreads / threads, 8))};
}

template <typename T, bool VEC>
dbf_status launch_grad(NormGradArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  const GradPlan g = grad_plan(a.rows, a.cols);
  a.blocks = g.blocks;
  const dim3 grid(static_cast<unsigned>(g.blocks * g.ks)), block(g.threads);
  dbf_status st;
  if (g.span == 0) {
    st = launch_pdl(dbf_rmsnorm_grad_kernel<T, VEC, 0>, grid, block, 0, stream, a);
  } else if (g.span == 1) {
    st = launch_pdl(dbf_rmsnorm_grad_kernel<T, VEC, 1>, grid, block, 0, stream, a);
  } else if (g.span == 2) {
    st = launch_pdl_cluster(dbf_rmsnorm_grad_kernel<T, VEC, 2>, grid, block, 0, stream, g.ks, a);
  } else if (g.span == 3) {
    return launch_pdl_cluster(dbf_rmsnorm_grad_kernel<T, VEC, 3>, grid, block, 0, stream, g.ks, a);
  } else {
    st = launch_pdl(dbf_rmsnorm_grad_wide_kernel<T>, grid, block, 0, stream, a);
  }
  if (st != DBF_OK) return st;
  if (a.cols <= 2048) return launch_grad_sum<8, 128>(a, stream);
  return a.cols <= 6144 ? launch_grad_sum<16, 64>(a, stream) : launch_grad_sum<32, 32>(a, stream);
}

template <typename T>
dbf_status grad_typed(const NormGradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const bool vec = a.cols % kChunk == 0 && aligned_to(a.dy, 32) && aligned_to(a.h, 32) && aligned_to(a.dh, 32) &&
                   aligned_to(a.weight, 32) && aligned_to(a.dx, 32);
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
  NormArgs a{x, residual, weight, h, y, nullptr, nullptr, rows, cols, cols, eps, 0};
  if (!y) return DBF_ERR_INVALID_ARG;
  dbf_status st = check_norm(a, t);
  if (st != DBF_OK) return st;
  if (!aligned_to(y, dtype_size(t))) return DBF_ERR_MISALIGNED;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != DBF_OK) return st;
  return norm_any<kDense>(a, t, dev, reinterpret_cast<cudaStream_t>(stream));
}

dbf_status dbf_rmsnorm_mx_forward(const void* x, const void* residual, const void* weight, dbf_dtype t, int64_t rows,
                                  int64_t cols, float eps, dbf_mx_format fmt, void* h, uint8_t* codes, uint8_t* scales,
                                  struct CUstream_st* stream) {
  NormArgs a{x, residual, weight, h, nullptr, codes, scales, rows, cols, cols, eps, 0};
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
  return static_cast<size_t>(grad_plan(rows, cols).blocks) * static_cast<size_t>(cols) * 4;
}

dbf_status dbf_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh, dbf_dtype t,
                                int64_t rows, int64_t cols, float eps, void* dx, float* dweight, void* workspace,
                                size_t ws_bytes, struct CUstream_st* stream) {
  if (!dy || !dx || !dweight) return DBF_ERR_INVALID_ARG;
  NormArgs check{h, nullptr, weight, nullptr, nullptr, nullptr, nullptr, rows, cols, cols, eps, 0};
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
