// engram_layernorm.hip -- layer norm of each row, forward and backward (gfx950).
//
// For a row x of D values, weights w and b [D]:
//   mean = sum x / D,  rstd = (sum (x - mean)^2 / D + eps)^(-1/2),
//   u = (x - mean) rstd,  y = u w + b
// Backward, for the gradient g of y and r of the residual stream that x is:
//   dw = sum over rows of g u,  db = sum over rows of g
//   dx = rstd (g w - mean_j(g w) - u mean_j(g w u)) + r
//
// Every value is read once and written once, so HBM bounds the kernels.  A row
// stays in registers between its two sums (the mean, then the squares around
// it, which keeps the digits that a difference of squares would lose).
//
// Mapping.  A lane has vectors of eight values, those kGroup lanes apart.  Rows
// up to 1024 values belong to 8, 16, 32 or 64 lanes of a wave and need no LDS;
// wider ones to a workgroup, whose waves exchange their sums through LDS.  The
// backward's workgroups take every kBlocks-th row, add up dw and db of their
// rows in registers, and write one fp32 row each, which a second kernel sums in
// a fixed order.
#include "engram_device.h"
#include "engram_launch.h"
#include "engram_values.h"

namespace engram {
namespace {

constexpr int kRowThreads = 256;  // of a workgroup whose rows are a wave or less
constexpr int kMostWaves = 16;

// The sum over kLanes lanes, in each of them.
template <int kLanes>
__device__ __forceinline__ float lane_sum(float v) {
  v += dpp<0xB1, 0xF, 0xF, true>(v);
  v += dpp<0x4E, 0xF, 0xF, true>(v);
  v += dpp<0x141, 0xF, 0xF, true>(v);
  if (kLanes >= 16) v += dpp<0x140, 0xF, 0xF, true>(v);
  if (kLanes >= 32) v += __shfl_xor(v, 16);
  if (kLanes >= 64) v += __shfl_xor(v, 32);
  return v;
}

// Sums over a row, the same values in each of its lanes: kGroup lanes, or the
// whole workgroup (0), its waves in order.  `to` is LDS that no wave reads any more: two sums in a
// row take two places.
template <int kGroup, int kSums>
__device__ __forceinline__ void row_sums(float (&v)[kSums], float (*to)[kMostWaves]) {
#pragma unroll
  for (int i = 0; i < kSums; ++i) v[i] = lane_sum<kGroup ? kGroup : 64>(v[i]);
  if constexpr (kGroup == 0) {
    const int waves = blockDim.x / 64;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < kSums; ++i) to[i][threadIdx.x >> 6] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = 0.0f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int i = 0; i < kSums; ++i) v[i] += to[i][w];
  }
}

struct NormArgs {
  const void *x, *grad_y, *grad_residual;
  void* out;  // y, or the gradient of x
  const float *w, *b;
  float* saved;         // forward: written if not null; backward: read
  float* partial;       // backward: [workgroups][2][D], or null
  int64_t N, ldx, ldgy, ldgr, ldout;
  int D;
  float eps;
};

// Which row of a pass and which of its vectors a thread has.
template <int kGroup>
struct Place {
  int row, rows, lane, lanes;
  __device__ __forceinline__ Place()
      : row(kGroup ? threadIdx.x / (kGroup ? kGroup : 1) : 0),
        rows(kGroup ? kRowThreads / (kGroup ? kGroup : 1) : 1),
        lane(kGroup ? threadIdx.x % (kGroup ? kGroup : 1) : threadIdx.x),
        lanes(kGroup ? kGroup : blockDim.x) {}
};

template <typename T, int kGroup, int kVecs, int kThreads>
__global__ __launch_bounds__(kThreads) void layer_norm_fwd_kernel(NormArgs a) {
  __shared__ float sums[2][1][kMostWaves];
  const Place<kGroup> at;
  const int nv = a.D / 8;
  const float inv = 1.0f / (float)a.D;
  float w[kVecs][8], b[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = at.lane + i * at.lanes;
    unpack8(c < nv ? load_raw(a.w + 8 * c) : zero_raw<float>(), w[i]);
    unpack8(c < nv && a.b ? load_raw(a.b + 8 * c) : zero_raw<float>(), b[i]);
  }
  Raw<T> raw[kVecs];
  const auto fetch = [&](int64_t n) {
    const bool in = n < a.N;
    const T* x = static_cast<const T*>(a.x) + (in ? n : 0) * a.ldx;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      raw[i] = in && c < nv ? load_raw(x + 8 * c) : zero_raw<T>();
    }
  };
  const int64_t step = (int64_t)gridDim.x * at.rows;
  int64_t n = (int64_t)blockIdx.x * at.rows + at.row;
  fetch(n);
  for (int64_t first = (int64_t)blockIdx.x * at.rows; first < a.N; first += step, n += step) {
    float v[kVecs][8], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      unpack8(raw[i], v[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[0] += v[i][k];
    }
    if (first + step < a.N) fetch(n + step);
    row_sums<kGroup>(sum, sums[0]);
    const float mean = sum[0] * inv;
    sum[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const bool mine = at.lane + i * at.lanes < nv;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= mean;
        if (mine) sum[0] = fmaf(v[i][k], v[i][k], sum[0]);
      }
    }
    row_sums<kGroup>(sum, sums[1]);
    const float rstd = 1.0f / sqrtf(sum[0] * inv + a.eps);
    if (n >= a.N) continue;
    if (a.saved && at.lane == 0) *reinterpret_cast<f32x2*>(a.saved + 2 * n) = f32x2{mean, rstd};
    T* y = static_cast<T*>(a.out) + n * a.ldout;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      if (c >= nv) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fmaf(v[i][k] * rstd, w[i][k], b[i][k]);
      store8<true>(y + 8 * c, v[i]);
    }
  }
}

template <typename T, int kGroup, int kVecs, int kThreads>
__global__ __launch_bounds__(kThreads) void layer_norm_bwd_kernel(NormArgs a) {
  __shared__ float sums[2][2][kMostWaves];
  const Place<kGroup> at;
  const int nv = a.D / 8;
  const float inv = 1.0f / (float)a.D;
  float dw[kVecs][8], db[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.0f;
  Raw<T> xr[kVecs], gr[kVecs];
  const auto fetch = [&](int64_t n) {
    const bool in = n < a.N;
    const T* x = static_cast<const T*>(a.x) + (in ? n : 0) * a.ldx;
    const T* g = static_cast<const T*>(a.grad_y) + (in ? n : 0) * a.ldgy;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      const bool mine = in && c < nv;
      xr[i] = mine ? load_raw(x + 8 * c) : zero_raw<T>();
      gr[i] = mine ? load_raw(g + 8 * c) : zero_raw<T>();
    }
  };
  const int64_t step = (int64_t)gridDim.x * at.rows;
  int64_t n = (int64_t)blockIdx.x * at.rows + at.row;
  // The next row's loads on their way, but for two vectors a lane, where the second
  // row is another workgroup's (8192 x 5120: 79 us, 92 with them, both before the
  // residual's loads were sent early).
  constexpr bool kAhead = kGroup != 0 || kVecs == 1;
  if (kAhead) fetch(n);
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * at.rows; first < a.N; first += step, n += step, turn ^= 1) {
    const bool in = n < a.N;
    if (!kAhead) fetch(n);
    const f32x2 saved = in ? *reinterpret_cast<const f32x2*>(a.saved + 2 * n) : f32x2{0.0f, 0.0f};
    const float mean = saved[0], rstd = saved[1];
    float u[kVecs][8], gw[kVecs][8], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      float w[8];
      unpack8(c < nv ? load_raw(a.w + 8 * c) : zero_raw<float>(), w);
      unpack8(xr[i], u[i]);
      unpack8(gr[i], gw[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        u[i][k] = (u[i][k] - mean) * rstd;
        const float g = gw[i][k];
        db[i][k] += g;
        dw[i][k] = fmaf(g, u[i][k], dw[i][k]);
        gw[i][k] = g * w[k];
        sum[0] += gw[i][k];
        sum[1] = fmaf(gw[i][k], u[i][k], sum[1]);
      }
    }
    if (kAhead && first + step < a.N) fetch(n + step);
    Raw<T> rr[kVecs];
    const auto fetch_residual = [&](int i) {
      const int c = at.lane + i * at.lanes;
      rr[i] = in && c < nv ? load_raw(static_cast<const T*>(a.grad_residual) + n * a.ldgr + 8 * c) : zero_raw<T>();
    };
    constexpr bool kLate = kVecs == 2 && sizeof(T) == 4;  // no registers to have these on their way
    if (!kLate && a.grad_residual)
#pragma unroll
      for (int i = 0; i < kVecs; ++i) fetch_residual(i);
    row_sums<kGroup>(sum, sums[turn]);
    const float m0 = sum[0] * inv, m1 = sum[1] * inv;
    T* out = static_cast<T*>(a.out) + (in ? n : 0) * a.ldout;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      if (!in || c >= nv) continue;
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = rstd * (gw[i][k] - m0 - u[i][k] * m1);
      if (a.grad_residual) {
        float r[8];
        if (kLate) fetch_residual(i);
        unpack8(rr[i], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] += r[k];
      }
      store8<true>(out + 8 * c, y);
    }
  }
  if (!a.partial) return;
  float* to = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (kGroup == 0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = at.lane + i * at.lanes;
      if (c >= nv) continue;
      store8<false>(to + 8 * c, dw[i]);
      store8<false>(to + a.D + 8 * c, db[i]);
    }
  } else {
    // the wave's rows in registers, then the four waves' through LDS, dw before db
    __shared__ float lds[kThreads / 64 - 1][kGroup * kVecs * 8];
    const int wave = threadIdx.x >> 6;
    const bool first = (threadIdx.x & 63) < kGroup;
    for (int part = 0; part < 2; ++part) {
      float(&v)[kVecs][8] = part ? db : dw;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int d = kGroup; d < 64; d *= 2) v[i][k] += __shfl_xor(v[i][k], d);
      if (wave > 0 && first)
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) lds[wave - 1][(i * 8 + k) * kGroup + at.lane] = v[i][k];
      __syncthreads();
      if (wave == 0 && first) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const int c = at.lane + i * at.lanes;
          if (c >= nv) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            for (int o = 0; o < kThreads / 64 - 1; ++o) v[i][k] += lds[o][(i * 8 + k) * kGroup + at.lane];
          store8<false>(to + (part ? a.D : 0) + 8 * c, v[i]);
        }
      }
      __syncthreads();
    }
  }
}

// The columns of the workgroups' rows: kRedSlices threads a column, each every
// kRedSlices-th row, eight of them on their way at once, then their sums in halves.
constexpr int kRedCols = 32, kRedSlices = 32, kRedAhead = 8;
__global__ __launch_bounds__(kRedCols * kRedSlices) void layer_norm_reduce_kernel(const float* partial, float* dw, float* db,
                                                                                  int rows, int D) {
  __shared__ float part[kRedSlices][kRedCols];
  const int at = threadIdx.x % kRedCols, slice = threadIdx.x / kRedCols, col = blockIdx.x * kRedCols + at;
  float s = 0.0f;
  if (col < 2 * D)
    for (int r = slice; r < rows; r += kRedSlices * kRedAhead) {
      float v[kRedAhead];
#pragma unroll
      for (int i = 0; i < kRedAhead; ++i)
        v[i] = r + i * kRedSlices < rows ? partial[(int64_t)(r + i * kRedSlices) * 2 * D + col] : 0.0f;
#pragma unroll
      for (int i = 0; i < kRedAhead; ++i) s += v[i];
    }
  part[slice][at] = s;
  __syncthreads();
  for (int half = kRedSlices / 2; half >= 1; half /= 2) {
    if (slice < half) part[slice][at] += part[slice + half][at];
    __syncthreads();
  }
  if (slice == 0 && col < 2 * D) {
    float* to = col < D ? dw : db;
    if (to) to[col < D ? col : col - D] = part[0][at];
  }
}

struct NormKernels {
  const void *fwd, *bwd;
  int threads, rows;  // of a workgroup
};

template <typename T, int kGroup, int kVecs, int kMost>
NormKernels norm_of(int threads) {
  return {(const void*)&layer_norm_fwd_kernel<T, kGroup, kVecs, kMost>,
          (const void*)&layer_norm_bwd_kernel<T, kGroup, kVecs, kMost>, threads, kGroup ? threads / (kGroup ? kGroup : 1) : 1};
}

// The narrowest group of lanes that a row fits, a vector a lane; two vectors where
// that is a workgroup of more than four waves.  (8192 x 5120, 640 threads of one vector:
// forward 33.6 us and backward 83.4 against 29.8 and 79.0 with 320 of two.)
template <typename T>
NormKernels norm_kernels_of(int D) {
  const int nv = D / 8;
  if (nv <= 8) return norm_of<T, 8, 1, kRowThreads>(kRowThreads);
  if (nv <= 16) return norm_of<T, 16, 1, kRowThreads>(kRowThreads);
  if (nv <= 32) return norm_of<T, 32, 1, kRowThreads>(kRowThreads);
  if (nv <= 64) return norm_of<T, 64, 1, kRowThreads>(kRowThreads);
  if (nv <= 128) return norm_of<T, 64, 2, kRowThreads>(kRowThreads);
  if (nv <= 256) return norm_of<T, 0, 1, 256>((nv + 63) / 64 * 64);
  const int threads = ((nv + 1) / 2 + 63) / 64 * 64;
  return norm_of<T, 0, 2, kMostWaves * 64>(threads);
}

NormKernels norm_kernels(int dtype, int D) {
  if (dtype == ENGRAM_BF16) return norm_kernels_of<bf16_t>(D);
  if (dtype == ENGRAM_FP16) return norm_kernels_of<_Float16>(D);
  return norm_kernels_of<float>(D);
}

// Workgroups.  Forward: as many as fit the chip, four a CU with 320 threads (8192 x
// 5120: 27.7 us, 6.1 TB/s; 29.8 with 1536).  Backward: each leaves a row of dw and
// db; two a CU, which all run at once in even shares (8192 x 5120 with residual: 70 us,
// 4.8 TB/s; before the residual's loads were sent ahead of the sums 79, with 448
// workgroups 84.5, 384: 93, and 576 to 768, whose last ones come after the others, 96 to 110).
// Both numbers were set there; as they are, as many values in narrower rows reach (bf16, of the
// forward's and the backward's bytes) 65536 x 512: 6.3 and 4.0 TB/s, 32768 x 1024: 6.2 and 5.0,
// 16384 x 2048: 4.1 backward; and 8192 x 5120 in fp32 4.6 and 5.1.
constexpr int64_t kFwdBlocks = 1024;
constexpr int64_t kBwdBlocks = 512;
int64_t bwd_blocks(int64_t N, int rows) {
  const int64_t all = (N + rows - 1) / rows;
  return all < kBwdBlocks ? all : kBwdBlocks;
}

}  // namespace

size_t layer_norm_bwd_workspace(int64_t N, int64_t D) {
  return (size_t)bwd_blocks(N, norm_kernels(ENGRAM_BF16, (int)D).rows) * 2 * (size_t)D * sizeof(float);
}

hipError_t launch_layer_norm_fwd(const NormCall& c, hipStream_t stream) {
  NormArgs a{};
  a.x = c.x; a.out = c.y; a.w = c.w; a.b = c.b; a.saved = c.saved;
  a.N = c.N; a.ldx = c.ldx; a.ldout = c.ldy; a.D = (int)c.D; a.eps = c.eps;
  const NormKernels k = norm_kernels(c.dtype, a.D);
  void* args[] = {&a};
  const int64_t blocks = (c.N + k.rows - 1) / k.rows;
  return hipLaunchKernel(k.fwd, dim3((unsigned)(blocks < kFwdBlocks ? blocks : kFwdBlocks)), dim3((unsigned)k.threads), args, 0,
                         stream);
}

hipError_t launch_layer_norm_bwd(const NormCall& c, hipStream_t stream) {
  NormArgs a{};
  a.x = c.x; a.grad_y = c.grad_y; a.grad_residual = c.grad_residual; a.out = c.grad_x; a.w = c.w; a.saved = c.saved;
  const bool weights = c.grad_w || c.grad_b;
  a.partial = weights ? static_cast<float*>(c.workspace) : nullptr;
  a.N = c.N; a.ldx = c.ldx; a.ldgy = c.ldgy; a.ldgr = c.ldgr; a.ldout = c.ldgx; a.D = (int)c.D;
  const NormKernels k = norm_kernels(c.dtype, a.D);
  int rows = (int)bwd_blocks(c.N, k.rows), D = a.D;
  void* args[] = {&a};
  const hipError_t e = hipLaunchKernel(k.bwd, dim3((unsigned)rows), dim3((unsigned)k.threads), args, 0, stream);
  if (e != hipSuccess || !weights) return e;
  const float* p = a.partial;
  float *dw = c.grad_w, *db = c.grad_b;
  void* args2[] = {&p, &dw, &db, &rows, &D};
  return hipLaunchKernel(reinterpret_cast<const void*>(&layer_norm_reduce_kernel),
                         dim3((unsigned)((2 * D + kRedCols - 1) / kRedCols)), dim3(kRedCols * kRedSlices), args2, 0, stream);
}

}  // namespace engram
