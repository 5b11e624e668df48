// engram_qknorm.hip -- per-head RMS norms of queries and keys with the
// position rotation in the same pass, forward and backward (gfx950).
//
// For every token n and head, x one head's D values, w [D] the norm's weight
// (one for all query heads, one for all key heads), R rotated values:
//   u = x rstd,  rstd = (mean_j x_j^2 + eps)^(-1/2),  y = u w
//   pair i < R/2 of y turns by phi = positions[n] * freqs[i]:
//     out = (a cos phi - b sin phi, a sin phi + b cos phi)
//   pair i is (y_i, y_{i+R/2}), or (y_2i, y_{2i+1}) when interleaved; values
//   from R on are not rotated.
// Backward, for G the gradient of out: g = the rotation by -phi of G,
//   dw = sum over tokens and heads of g u
//   dx = rstd (g w - u mean_j(g w u))
//
// Angles.  freqs[i] is the pair's turn per position as a 64-bit fraction of a
// whole turn, so positions[n] * freqs[i] modulo 2^64 is the angle's fraction
// of a turn exactly (integer multiplication drops the whole turns): the error
// is the table's, at most 2^-65 turns per position, however far the position.
// The top 32 bits become an fp32 in [-1/2, 1/2) turns; 16-bit outputs use the
// hardware sine and cosine, whose argument is in turns, fp32 outputs the math
// library's.
//
// Mapping.  Each value is read once and written once, so HBM bounds the kernel
// and nothing is staged.  A lane holds two vectors of eight values, vector i
// and its partner at R/2, so both members of every pair are in one lane; D =
// 128 takes 8 lanes a head and a wave 8 heads at once.  A wave's heads are of
// one token, whose sines and cosines it computes once and uses for all of them.
// The weight gradients are sums over all tokens and heads: each workgroup adds
// its rows in registers, writes one fp32 row, and a second kernel sums the
// rows in a fixed order.
#include "engram_device.h"
#include "engram_launch.h"

namespace engram {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;
constexpr float kInv2p32 = 2.3283064365386963e-10f;  // 2^-32

struct bf16_t { uint16_t v; };

// Eight values as they lie in memory.
template <typename T>
struct Raw {
  u32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = load16(reinterpret_cast<const u32x4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> zero_raw() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = u32x4{0, 0, 0, 0};
  return r;
}
__device__ __forceinline__ void unpack8(const Raw<bf16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf_lo(r.w[0][i]);
    v[2 * i + 1] = bf_hi(r.w[0][i]);
  }
}
__device__ __forceinline__ void unpack8(const Raw<_Float16>& r, float (&v)[8]) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const f16x8 h = __builtin_bit_cast(f16x8, r.w[0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
__device__ __forceinline__ void unpack8(const Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i / 4][i % 4]);
}
// kStream: the line is not kept in the caches.
template <bool kStream>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
  if (kStream) store16_stream(p, v);
  else store16(p, v);
}
template <bool kStream>
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  put16<kStream>(p, r);
}
template <bool kStream>
__device__ __forceinline__ void store8(_Float16* p, const float (&v)[8]) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
  put16<kStream>(p, __builtin_bit_cast(u32x4, r));
}
template <bool kStream>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[i + 4]);
  }
  put16<kStream>(p, a);
  put16<kStream>(p + 4, b);
}

// Sum over the kLanes lanes of a row, the same value in each of them.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1, 0xF, 0xF, true>(v);
  v += dpp<0x4E, 0xF, 0xF, true>(v);
  if (kLanes >= 8) v += dpp<0x141, 0xF, 0xF, true>(v);
  if (kLanes >= 16) v += dpp<0x140, 0xF, 0xF, true>(v);
  if (kLanes >= 32) v += __shfl_xor(v, 16);
  return v;
}

// What a lane covers of a head: vector a and vector b, the lanes below R/16 a
// rotated pair of vectors (b at R/2 from a), the next ones two neighbouring
// vectors behind the rotated part.
struct Cover {
  int a, b;      // first values
  bool has_a, has_b, turns;
};

__device__ __forceinline__ Cover cover_of(int j, int D, int R) {
  Cover c;
  const int pairs = R / 16;
  c.turns = j < pairs;
  c.a = c.turns ? 8 * j : R + 16 * (j - pairs);
  c.b = c.turns ? R / 2 + 8 * j : c.a + 8;
  c.has_a = c.a < D;
  c.has_b = c.b < D;
  return c;
}

// The lane's eight rotated pairs: in order (a_i, b_i), or neighbours inside a
// (first four) and inside b.  First pair of each four.
template <bool kInter>
__device__ __forceinline__ int pair_of(const Cover& c, int i) {
  if (!kInter) return c.a + i;
  return i < 4 ? c.a / 2 + i : c.b / 2 + (i - 4);
}

template <typename T, bool kInter>
__device__ __forceinline__ void load_freqs(const uint64_t* freqs, const Cover& c, uint64_t (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = c.turns ? freqs[pair_of<kInter>(c, i)] : 0;
}

template <typename T>
__device__ __forceinline__ void angles(const uint64_t (&f)[8], int64_t pos, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (float)(int32_t)((uint64_t)pos * f[i] >> 32) * kInv2p32;
    if (sizeof(T) == 2) {
      cs[i] = __builtin_amdgcn_cosf(t);
      sn[i] = __builtin_amdgcn_sinf(t);
    } else {
      sincospif(2.0f * t, &sn[i], &cs[i]);
    }
  }
}

// Turn the lane's eight pairs by +phi (kSign 1) or -phi (kSign -1); for the lanes
// that turn only: a turn by nothing would multiply an infinity by a sine of 0.
template <bool kInter, int kSign>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& p = kInter ? (i < 4 ? a[2 * i] : b[2 * (i - 4)]) : a[i];
    float& q = kInter ? (i < 4 ? a[2 * i + 1] : b[2 * (i - 4) + 1]) : b[i];
    const float s = kSign > 0 ? sn[i] : -sn[i];
    const float np = p * cs[i] - q * s, nq = p * s + q * cs[i];
    p = np;
    q = nq;
  }
}

__device__ __forceinline__ void zero8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
}

// One side of a call: the queries or the keys.
struct Side {
  const void* x;      // forward: input; backward: input
  const void* gy;     // backward: gradient of the output
  const float* w;
  void* y;            // forward: output; backward: gradient of x
  int64_t ldx, ldg, ldy;  // values between tokens
  int heads;
  int blocks;         // workgroups on this side
  int passes;         // a token's heads in passes of 64 / lanes
  int share;          // passes of a wave, one behind the other
};

struct QkArgs {
  Side side[2];
  const int64_t* positions;
  const uint64_t* freqs;
  float* partial;     // backward: [blocks of both sides][D]
  int64_t N;
  int D, R;
  float eps;
};

// A wave's share of the passes over all tokens' heads: token after token, the
// passes of each in order, so that shares differ by less than a pass and a
// token's angles are computed once (or again where a share begins inside it).
struct Passes {
  int64_t n;  // token
  int pass, passes, left;
  __device__ __forceinline__ Passes(const Side& s, int64_t tokens, int64_t wave) {
    const int64_t all = tokens * s.passes, first = wave * s.share;
    passes = s.passes;
    left = first < all ? (int)min((int64_t)s.share, all - first) : 0;
    n = first / passes;
    pass = (int)(first - n * passes);
  }
  __device__ __forceinline__ bool next() {
    if (++pass == passes) {
      pass = 0;
      ++n;
    }
    return --left > 0;
  }
};

template <typename T, int kLanes, bool kInter>
__global__ __launch_bounds__(kQkThreads) void qk_norm_rope_fwd_kernel(QkArgs args) {
  const bool keys = (int)blockIdx.x >= args.side[0].blocks;
  const Side s = keys ? args.side[1] : args.side[0];
  const int block = keys ? blockIdx.x - args.side[0].blocks : blockIdx.x;
  constexpr int kRows = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane / kLanes;
  const Cover c = cover_of(lane % kLanes, args.D, args.R);
  const float inv_d = 1.0f / (float)args.D;
  float wa[8], wb[8];
  uint64_t f[8];
  zero8(wa);
  zero8(wb);
  if (c.has_a) unpack8(load_raw(s.w + c.a), wa);
  if (c.has_b) unpack8(load_raw(s.w + c.b), wb);
  load_freqs<T, kInter>(args.freqs, c, f);
  const T* x = static_cast<const T*>(s.x);
  T* y = static_cast<T*>(s.y);
  Passes at(s, args.N, (int64_t)block * kQkWaves + wave);
  const auto fetch = [&](Raw<T>& a, Raw<T>& b) {
    a = zero_raw<T>();
    b = zero_raw<T>();
    const int h = at.pass * kRows + row;
    if (h < s.heads) {
      const T* p = x + at.n * s.ldx + h * args.D;
      if (c.has_a) a = load_raw(p + c.a);
      if (c.has_b) b = load_raw(p + c.b);
    }
  };
  if (at.left == 0) return;
  Raw<T> ra, rb;
  fetch(ra, rb);
  float cs[8], sn[8];
  angles<T>(f, args.R ? args.positions[at.n] : 0, cs, sn);
  for (;;) {
    const int h = at.pass * kRows + row;
    T* yp = y + at.n * s.ldy + h * args.D;
    float a[8], b[8];
    unpack8(ra, a);
    unpack8(rb, b);
    const bool more = at.next(), turned = more && at.pass == 0;
    if (more) fetch(ra, rb);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
    const float rstd = 1.0f / sqrtf(row_sum<kLanes>(ss) * inv_d + args.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= rstd * wa[i];
      b[i] *= rstd * wb[i];
    }
    if (c.turns) rotate<kInter, 1>(a, b, cs, sn);
    if (h < s.heads) {
      if (c.has_a) store8<true>(yp + c.a, a);
      if (c.has_b) store8<true>(yp + c.b, b);
    }
    if (!more) return;
    if (turned) angles<T>(f, args.R ? args.positions[at.n] : 0, cs, sn);
  }
}

template <typename T, int kLanes, bool kInter>
__global__ __launch_bounds__(kQkThreads) void qk_norm_rope_bwd_kernel(QkArgs args) {
  const bool keys = (int)blockIdx.x >= args.side[0].blocks;
  const Side s = keys ? args.side[1] : args.side[0];
  const int block = keys ? blockIdx.x - args.side[0].blocks : blockIdx.x;
  constexpr int kRows = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane / kLanes;
  const Cover c = cover_of(lane % kLanes, args.D, args.R);
  const float inv_d = 1.0f / (float)args.D;
  float wa[8], wb[8], da[8], db[8];
  uint64_t f[8];
  zero8(wa);
  zero8(wb);
  zero8(da);
  zero8(db);
  if (c.has_a) unpack8(load_raw(s.w + c.a), wa);
  if (c.has_b) unpack8(load_raw(s.w + c.b), wb);
  load_freqs<T, kInter>(args.freqs, c, f);
  const T* x = static_cast<const T*>(s.x);
  const T* gy = static_cast<const T*>(s.gy);
  T* dx = static_cast<T*>(s.y);
  Passes at(s, args.N, (int64_t)block * kQkWaves + wave);
  const auto fetch = [&](Raw<T>& a, Raw<T>& b, Raw<T>& ga, Raw<T>& gb) {
    a = b = ga = gb = zero_raw<T>();
    const int h = at.pass * kRows + row;
    if (h < s.heads) {
      const T *p = x + at.n * s.ldx + h * args.D, *q = gy + at.n * s.ldg + h * args.D;
      if (c.has_a) {
        a = load_raw(p + c.a);
        ga = load_raw(q + c.a);
      }
      if (c.has_b) {
        b = load_raw(p + c.b);
        gb = load_raw(q + c.b);
      }
    }
  };
  bool more = at.left != 0;
  if (more) {
    Raw<T> ra, rb, rga, rgb;
    fetch(ra, rb, rga, rgb);
    float cs[8], sn[8];
    angles<T>(f, args.R ? args.positions[at.n] : 0, cs, sn);
    while (more) {
      const int h = at.pass * kRows + row;
      T* dp = dx + at.n * s.ldy + h * args.D;
      float a[8], b[8], ga[8], gb[8];
      unpack8(ra, a);
      unpack8(rb, b);
      unpack8(rga, ga);
      unpack8(rgb, gb);
      more = at.next();
      if (more) fetch(ra, rb, rga, rgb);
      if (c.turns) rotate<kInter, -1>(ga, gb, cs, sn);
      if (more && at.pass == 0) angles<T>(f, args.R ? args.positions[at.n] : 0, cs, sn);
      float ss = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += a[i] * a[i] + b[i] * b[i];
        dot += ga[i] * wa[i] * a[i] + gb[i] * wb[i] * b[i];
      }
      const float norm = 1.0f / sqrtf(row_sum<kLanes>(ss) * inv_d + args.eps);
      const float rstd = h < s.heads ? norm : 0.0f;  // lanes without a head add nothing to dw, whatever eps
      // with u = x rstd: dx = rstd g w - u (rstd mean(g w u)), and mean(g w u) = rstd dot / D
      const float m = row_sum<kLanes>(dot) * inv_d * rstd * rstd;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ua = a[i] * rstd, ub = b[i] * rstd;
        da[i] += ga[i] * ua;
        db[i] += gb[i] * ub;
        a[i] = rstd * (ga[i] * wa[i]) - ua * m;
        b[i] = rstd * (gb[i] * wb[i]) - ub * m;
      }
      if (h < s.heads) {
        if (c.has_a) store8<false>(dp + c.a, a);
        if (c.has_b) store8<false>(dp + c.b, b);
      }
    }
  }
  // the rows of a wave, then the waves, in order
  __shared__ float sums[kQkWaves][16 * kLanes];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = kLanes; off < 64; off *= 2) {
      da[i] += __shfl_xor(da[i], off);
      db[i] += __shfl_xor(db[i], off);
    }
  }
  if (row == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c.has_a) sums[wave][c.a + i] = da[i];
      if (c.has_b) sums[wave][c.b + i] = db[i];
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < args.D; j += kQkThreads) {
    float t = sums[0][j];
#pragma unroll
    for (int w = 1; w < kQkWaves; ++w) t += sums[w][j];
    args.partial[(int64_t)blockIdx.x * args.D + j] = t;
  }
}

// dw[j] = the sum of `rows` partial rows, queries (blockIdx.y 0) or keys: 16
// columns a workgroup, 64 threads a column, joined in a fixed order.
constexpr int kRedCols = 16, kRedSlices = 64;
__global__ __launch_bounds__(kRedCols* kRedSlices) void qk_norm_rope_reduce_kernel(const float* partial, float* dwq,
                                                                                   float* dwk, int rows_q, int rows_k,
                                                                                   int D) {
  __shared__ float part[kRedSlices][kRedCols];
  const bool keys = blockIdx.y != 0;
  const float* p = partial + (keys ? (int64_t)rows_q * D : 0);
  const int rows = keys ? rows_k : rows_q;
  const int col = blockIdx.x * kRedCols + threadIdx.x % kRedCols, slice = threadIdx.x / kRedCols;
  float s = 0.0f;
  if (col < D)
    for (int r = slice; r < rows; r += kRedSlices) s += p[(int64_t)r * D + col];
  part[slice][threadIdx.x % kRedCols] = s;
  __syncthreads();
  for (int half = kRedSlices / 2; half >= 1; half /= 2) {
    if (slice < half) part[slice][threadIdx.x % kRedCols] += part[slice + half][threadIdx.x % kRedCols];
    __syncthreads();
  }
  if (slice == 0 && col < D) (keys ? dwk : dwq)[col] = part[0][threadIdx.x];
}

struct QkKernels {
  const void *fwd, *bwd;
};

template <typename T, bool kInter>
QkKernels qk_kernels_of_lanes(int lanes) {
  switch (lanes) {
    case 4: return {(const void*)&qk_norm_rope_fwd_kernel<T, 4, kInter>, (const void*)&qk_norm_rope_bwd_kernel<T, 4, kInter>};
    case 8: return {(const void*)&qk_norm_rope_fwd_kernel<T, 8, kInter>, (const void*)&qk_norm_rope_bwd_kernel<T, 8, kInter>};
    case 16: return {(const void*)&qk_norm_rope_fwd_kernel<T, 16, kInter>, (const void*)&qk_norm_rope_bwd_kernel<T, 16, kInter>};
    default: return {(const void*)&qk_norm_rope_fwd_kernel<T, 32, kInter>, (const void*)&qk_norm_rope_bwd_kernel<T, 32, kInter>};
  }
}

template <typename T>
QkKernels qk_kernels_of(int lanes, bool inter) {
  return inter ? qk_kernels_of_lanes<T, true>(lanes) : qk_kernels_of_lanes<T, false>(lanes);
}

QkKernels qk_kernels(int dtype, int lanes, bool inter) {
  if (dtype == ENGRAM_BF16) return qk_kernels_of<bf16_t>(lanes, inter);
  if (dtype == ENGRAM_FP16) return qk_kernels_of<_Float16>(lanes, inter);
  return qk_kernels_of<float>(lanes, inter);
}

// Lanes a head takes: R/16 rotated pairs of vectors, then pairs of vectors of the rest.
int qk_lanes(int D, int R) {
  const int need = R / 16 + (D - R + 15) / 16;
  int lanes = 4;
  while (lanes < need) lanes *= 2;
  return lanes;
}

// Workgroups of the two sides: the passes over all heads in even shares, the
// sides by their heads.  Forward: shares of about two passes and streaming
// stores (8192 tokens, 40 + 8 heads of 128: 38.5 us, 5.2 TB/s, against 41.1 with
// as many workgroups as fit the chip and 43.6 with plain stores).  Backward: as
// many workgroups as fit the chip, three a CU, since each leaves a partial row
// of dw, and shares of two passes at least for the same reason (40 + 40 heads:
// 114 us; 124 with 1024 workgroups, 141 with streaming stores).
constexpr int64_t kFwdBlocks = 5120, kBwdBlocks = 768;
void qk_plan(Side (&side)[2], int64_t N, int lanes, int64_t most, int64_t least) {
  const int rows = 64 / lanes;
  int64_t passes[2], all = 0;
  for (int i = 0; i < 2; ++i) {
    side[i].passes = (side[i].heads + rows - 1) / rows;
    passes[i] = N * side[i].passes;
    all += passes[i];
  }
  const int64_t even = (all + most * kQkWaves - 1) / (most * kQkWaves), share = even > least ? even : least;
  for (int i = 0; i < 2; ++i) {
    side[i].share = (int)share;
    side[i].blocks = (int)((passes[i] + share * kQkWaves - 1) / (share * kQkWaves));
  }
}

}  // namespace

size_t qk_norm_rope_bwd_workspace(int64_t D) { return (size_t)(kBwdBlocks + 2) * (size_t)D * sizeof(float); }

hipError_t launch_qk_norm_rope_fwd(const QkCall& q, hipStream_t stream) {
  QkArgs a{};
  const void* x[] = {q.q, q.k};
  void* y[] = {q.q_out, q.k_out};
  const float* w[] = {q.wq, q.wk};
  const int64_t ldx[] = {q.ldq, q.ldk}, ldy[] = {q.ldq_out, q.ldk_out};
  const int64_t heads[] = {q.Hq, q.Hk};
  for (int i = 0; i < 2; ++i) a.side[i] = Side{x[i], nullptr, w[i], y[i], ldx[i], 0, ldy[i], (int)heads[i], 0, 0, 0};
  const int lanes = qk_lanes((int)q.D, (int)q.R);
  qk_plan(a.side, q.N, lanes, kFwdBlocks, 1);
  a.positions = q.positions;
  a.freqs = reinterpret_cast<const uint64_t*>(q.freqs);
  a.N = q.N;
  a.D = (int)q.D;
  a.R = (int)q.R;
  a.eps = q.eps;
  void* args[] = {&a};
  return hipLaunchKernel(qk_kernels(q.dtype, lanes, q.interleaved).fwd,
                         dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)), dim3(kQkThreads), args, 0, stream);
}

hipError_t launch_qk_norm_rope_bwd(const QkCall& q, hipStream_t stream) {
  QkArgs a{};
  const void* x[] = {q.q, q.k};
  const void* gy[] = {q.grad_q_out, q.grad_k_out};
  void* y[] = {q.q_out, q.k_out};
  const float* w[] = {q.wq, q.wk};
  const int64_t ldx[] = {q.ldq, q.ldk}, ldg[] = {q.ldgq, q.ldgk}, ldy[] = {q.ldq_out, q.ldk_out};
  const int64_t heads[] = {q.Hq, q.Hk};
  for (int i = 0; i < 2; ++i) a.side[i] = Side{x[i], gy[i], w[i], y[i], ldx[i], ldg[i], ldy[i], (int)heads[i], 0, 0, 0};
  const int lanes = qk_lanes((int)q.D, (int)q.R);
  qk_plan(a.side, q.N, lanes, kBwdBlocks, 2);
  a.positions = q.positions;
  a.freqs = reinterpret_cast<const uint64_t*>(q.freqs);
  a.partial = static_cast<float*>(q.workspace);
  a.N = q.N;
  a.D = (int)q.D;
  a.R = (int)q.R;
  a.eps = q.eps;
  void* args[] = {&a};
  hipError_t e = hipLaunchKernel(qk_kernels(q.dtype, lanes, q.interleaved).bwd,
                                 dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)), dim3(kQkThreads), args, 0, stream);
  if (e != hipSuccess) return e;
  const float* p = a.partial;
  float *dwq = q.grad_wq, *dwk = q.grad_wk;
  int rq = a.side[0].blocks, rk = a.side[1].blocks, D = a.D;
  void* args2[] = {&p, &dwq, &dwk, &rq, &rk, &D};
  return hipLaunchKernel(reinterpret_cast<const void*>(&qk_norm_rope_reduce_kernel),
                         dim3((unsigned)((D + kRedCols - 1) / kRedCols), 2), dim3(kRedCols * kRedSlices), args2, 0, stream);
}

}  // namespace engram
