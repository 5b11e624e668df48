// engram_linear.hip -- matrix products with a fused epilogue: the projections
// in front of the gate and around the token mixers, forward and backward
// (gfx950).
//
//   z = x W^T + bias,   y = act(z) + residual          x [N][K], W [M][K]
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum_n dz
//
// One tile kernel makes the three products C[i][j] = sum_c A(i, c) B(j, c).
// An operand lies with the contraction c contiguous (x and W in the forward)
// or with i (or j) contiguous (W in dx; dz and x in dW); the second kind is
// turned on its way from LDS to the registers by the transposing LDS load.
// Both operands go from memory straight into LDS, 64 values of c at a time,
// two or four stages deep.  The products are fp32 sums over bf16 or fp16 operands on the matrix cores
// (16x16x32); the one rounding is that of the outputs.  In the backward dz is
// rounded to the operands' type where it differs from dy (an activation), as
// it is an operand of two products; dbias is summed before that rounding.
//
// Single tokens: the weight is read once and bounds the call; a kernel of its
// own takes whole rows of it with plain fp32 products.
#include "engram_device.h"
#include "engram_launch.h"
#include "engram_layers_device.h"
#include "engram_linear_plan.h"

#include <type_traits>

namespace engram {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) void* lds_ptr;

struct Bf16 {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf_hi(w); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
};
struct Fp16 {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f16x2 r = {(_Float16)a, (_Float16)b};  // round to nearest even
    return __builtin_bit_cast(uint32_t, r);
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(u32x4 r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = T::lo(r[i]);
    v[2 * i + 1] = T::hi(r[i]);
  }
}
template <typename T>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = T::pack(v[2 * i], v[2 * i + 1]);
  return r;
}

template <typename T>
__device__ __forceinline__ u32x2 pack4(f32x4 v) {
  return u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
}

// The normal distribution at z; e is exp(-z^2/2), which the gradient needs too.
// At -|z| it is e q(|z|), where q = exp(z^2/2) Phi(-|z|) falls slowly from 1/2
// like 0.4 / |z|; with t = 1 / (1 + 0.3 |z|) a polynomial of degree 8 without a
// constant, fitted to the least relative error on [0, 14.5] (behind which e is
// below fp32), leaves 1.6e-7 of the tail itself and 5e-7 in fp32.  So gelu and
// its slope are far below half a step of the 16-bit types also where they are
// small, which an approximation of erf with a small absolute error is not.
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, fabsf(z), 1.0f));
  float q = fmaf(0.0354237147f, t, -0.156158373f);
  q = fmaf(q, t, 0.204556659f);
  q = fmaf(q, t, -0.0520339124f);
  q = fmaf(q, t, 0.127691716f);
  q = fmaf(q, t, 0.100175962f);
  q = fmaf(q, t, 0.120712131f);
  q = fmaf(q, t, 0.119632006f);
  const float tail = q * t * e;
  return z < 0.0f ? tail : 1.0f - tail;
}
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// act(z); z = -inf gives the limit 0 for silu and gelu, which are below fp32 from kVanished on.
constexpr float kVanished = -104.0f;
__device__ __forceinline__ float act_of(float z, int act) {
  switch (act) {
    case ENGRAM_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case ENGRAM_ACT_SILU: return z < kVanished ? 0.0f : z * sigmoid(z);
    case ENGRAM_ACT_GELU: return z < kVanished ? 0.0f : z * normal_cdf(z, __expf(-0.5f * z * z));
    default: return z;
  }
}
template <int kAct>
__device__ __forceinline__ void act8(float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = act_of(v[k], kAct);
}
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case ENGRAM_ACT_RELU: return z <= 0.0f ? 0.0f : 1.0f;
    case ENGRAM_ACT_SILU: {
      if (fabsf(z) > -kVanished) return z > 0.0f ? 1.0f : 0.0f;
      const float p = sigmoid(z);
      return fmaf(p, z * (1.0f - p), p);
    }
    case ENGRAM_ACT_GELU: {
      if (fabsf(z) > -kVanished) return z > 0.0f ? 1.0f : 0.0f;
      const float e = __expf(-0.5f * z * z);
      return fmaf(z * 0.39894228f, e, normal_cdf(z, e));
    }
    default: return 1.0f;
  }
}

// What happens to a sum before it is stored; all pointers but y may be null.
struct Epilogue {
  const float* bias;
  const void* residual;
  void* z;
  void* y;
  int64_t ldr, ldz, ldy;
  int act;
};

__device__ __forceinline__ u32x4 load_residual(int64_t i, int64_t j, const Epilogue& e) {
  return load16(static_cast<const uint16_t*>(e.residual) + i * e.ldr + j);
}

// Eight neighbouring sums to their end; `residual` is looked at if there is one.
template <typename T>
__device__ __forceinline__ void finish8(float (&v)[8], const float (&bias)[8], u32x4 residual, int64_t i, int64_t j,
                                        const Epilogue& e) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] += bias[k];
  if (e.z) store16(static_cast<uint16_t*>(e.z) + i * e.ldz + j, pack8<T>(v));
  switch (e.act) {
    case ENGRAM_ACT_RELU: act8<ENGRAM_ACT_RELU>(v); break;
    case ENGRAM_ACT_SILU: act8<ENGRAM_ACT_SILU>(v); break;
    case ENGRAM_ACT_GELU: act8<ENGRAM_ACT_GELU>(v); break;
  }
  if (e.residual) {
    float r[8];
    unpack8<T>(residual, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += r[k];
  }
  store16(static_cast<uint16_t*>(e.y) + i * e.ldy + j, pack8<T>(v));
}

__device__ __forceinline__ void load_bias(float (&v)[8], const float* bias, int64_t j) {
  f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  if (bias) {
    a = *reinterpret_cast<const f32x4*>(bias + j);
    b = *reinterpret_cast<const f32x4*>(bias + j + 4);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = a[k];
    v[k + 4] = b[k];
  }
}

// ---------------------------------------------------------------- tiles

// The product's tiles: the first `whole` are made by one workgroup each, the
// contraction of each of the others is cut into `parts`, whose sums go to
// `partial` ([tile][part] tiles of fp32) for the join kernel.
struct GemmArgs {
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int64_t I, J, C;      // rows, columns, contraction
  int ti, tj, whole, parts;
  int64_t c_part;       // contraction values of a part, a multiple of kBk
  float* partial;
  Epilogue e;
};

// Where a tile lies: groups of eight tile rows, column by column, so that
// neighbouring workgroups share operands.
__device__ __forceinline__ void tile_origin(const GemmArgs& g, int tile, int size_i, int size_j, int64_t& i0, int64_t& j0) {
  constexpr int kGroup = 8;
  const int group = tile / (kGroup * g.tj), in_group = tile - group * kGroup * g.tj;
  const int height = min(kGroup, g.ti - group * kGroup);
  i0 = (int64_t)(group * kGroup + in_group % height) * size_i;
  j0 = (int64_t)(in_group / height) * size_j;
}

typedef __attribute__((address_space(3))) const u32x4* lds_u32x4;

// One operand's stage in LDS: kRows rows of the product, 64 contraction values.
//  contraction contiguous (kTurned false): [kRows][64], a line of memory a
//    row, its eight 16-byte pieces in the order piece ^ swizzle(row);
//  rows contiguous (kTurned): [64][kRows], the 64-byte pieces of line c in the
//    order piece ^ (c & kTurns) and their halves changed over in every other eight
//    lines.
// Either way the lanes that LDS serves at once (sixteen of a 16-byte read: rows
// 0-3 and 12-15 of one piece with 4-11 of the next, or the other way round;
// thirty-two of a transposing read) find their values in different banks.
// kPairs (not kTurned): the rows of two neighbouring 16-row fragments
// interleave in fours, which leaves a lane of the product with eight
// neighbouring columns instead of four and four.
// kFrags fragments of 16 rows belong to a wave.
template <int kRows, int kWaves, int kFrags, bool kTurned, bool kPairs>
struct Operand {
  static constexpr int kLoads = kRows * kBk * 2 / (kWaves * 1024);  // 16-byte loads of a lane for a stage
  static constexpr int kReads = kTurned ? 2 : 1;                    // LDS reads of a fragment
  static_assert(kLoads * kWaves * 1024 == kRows * kBk * 2, "the tile is a whole number of loads");

  static __device__ __forceinline__ int swizzle(int row) {
    return kPairs ? ((row >> 3) & 3) << 1 | ((row >> 1) & 1) : (row >> 1) & 7;
  }
  static constexpr int kTurns = kRows >= 128 ? 3 : kRows / 32 - 1;  // a line has at least kTurns + 1 pieces
  static __device__ __forceinline__ int halves(int line) { return ((line >> 3) ^ (line >> 4)) & 1; }

  // The lane's loads of a stage: byte offsets from the stage's first value,
  // and of the first load its contraction value (those of the others: kStep more each).
  static constexpr int kStep = kTurned ? kWaves * 64 / (kRows / 8) : 0;
  struct Loads {
    uint32_t off[kLoads];
    int c;
    __device__ __forceinline__ void set(int64_t ld, int64_t rows, int wave, int lane) {
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        const int at = (q * kWaves + wave) * 64 + lane;
        int line, first;
        if (!kTurned) {
          line = at / 8;
          first = (at % 8 ^ swizzle(line)) * 8;
        } else {
          constexpr int kPieces = kRows / 8;
          line = at / kPieces;
          const int piece = at % kPieces;
          first = ((piece / 4) ^ (line & kTurns)) * 32 + ((piece % 4) ^ 2 * halves(line)) * 8;
        }
        if (q == 0) c = kTurned ? line : first;
        off[q] = (kTurned ? first : line) < rows ? (uint32_t)line * (uint32_t)(ld * 2) + (uint32_t)first * 2 : kBeyond;
      }
    }
    // Into LDS at `to`; contraction values from `left` on are zero.
    __device__ __forceinline__ void fill(uint32_t to, const uint16_t* from, int left, int wave) const {
      const u32x4 src = buffer_words(from);
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
        load_to_lds(to + (q * kWaves + wave) * 1024u, src, c + q * kStep < left ? off[q] : kBeyond);
    }
  };

  // Where the lane finds its part of the wave's fragments in a stage: byte
  // addresses, to which half h of the contraction and the fragment add
  // constants.  Turned: one for each 64-byte piece and half of it.
  static constexpr int kPlaces = kTurned ? (kFrags < 8 ? kFrags : 8) : 2;
  struct Places {
    uint32_t at[kPlaces];
    __device__ __forceinline__ void set(uint32_t lds, int row0, int lane) {
      const int l = lane % 16, g = lane / 16;
      if (!kTurned) {
        const int r = row0 + (kPairs ? 8 * (l / 4) + l % 4 : l);
#pragma unroll
        for (int h = 0; h < 2; ++h) at[h] = lds + 2 * (r * kBk + ((4 * h + g) ^ swizzle(r)) * 8);
      } else {
        const int c = 8 * g + l / 4;
#pragma unroll
        for (int n = 0; n < kPlaces; ++n) {
          const int col = row0 + n * 16 + 4 * (l % 4);
          at[n] = lds + 2 * (c * kRows + ((col / 32) ^ (c & kTurns)) * 32 + (col % 32 ^ 16 * halves(c)));
        }
      }
    }
    template <int kHalf>
    __device__ __forceinline__ u32x4 frag(int n, uint32_t stage) const {
      if constexpr (!kTurned) {
        const int row = kPairs ? n / 2 * 32 + n % 2 * 4 : n * 16;
        return *((lds_u32x4)(uintptr_t)(at[kHalf] + stage) + row * kBk / 8);
      } else {
        const lds_s16x4 p = (lds_s16x4)(uintptr_t)(at[n % kPlaces] + stage) + (n / kPlaces * 16 * kPlaces + 32 * kHalf * kRows) / 4;
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + kRows));
        return u32x4{x[0], x[1], y[0], y[1]};
      }
    }
  };
};

// kI x kJ tiles, kWi x kWj waves.  kDepth stages in LDS, and half a stage's
// fragments ahead in registers: while one half is multiplied, the next half is
// read; in the middle of a stage it is read out, and the stage kDepth further
// on is sent for into its place, kDepth - 1 whole stages of products before its
// use.
template <typename T, int kI, int kJ, int kWi, int kWj, int kDepth, bool kTurnA, bool kTurnB>
__global__ __launch_bounds__(kWi* kWj * 64) void gemm_kernel(GemmArgs g) {
  constexpr int kWaves = kWi * kWj, kMt = kI / kWi / 16, kNt = kJ / kWj / 16;
  using A = Operand<kI, kWaves, kMt, kTurnA, false>;
  using B = Operand<kJ, kWaves, kNt, kTurnB, !kTurnB>;
  constexpr uint32_t kStageBytes = (kI + kJ) * kBk * 2;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDepth][(kI + kJ) * kBk];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroups go round the eight XCDs; each takes a run of neighbouring
  // tiles, whose operands its L2 holds.
  int tile = blockIdx.x, part = 0;
  if (tile < g.whole) {
    const int xcd = tile & 7, per = g.whole / 8, rest = g.whole % 8;
    tile = xcd * per + min(xcd, rest) + (tile >> 3);
  } else {
    part = (tile - g.whole) % g.parts;
    tile = g.whole + (tile - g.whole) / g.parts;
  }
  const bool cut = tile >= g.whole;
  int64_t i0, j0;
  tile_origin(g, tile, kI, kJ, i0, j0);
  const int64_t c0 = cut ? part * g.c_part : 0, c1 = cut ? min(c0 + g.c_part, g.C) : g.C;
  const int stages = (int)((c1 - c0 + kBk - 1) / kBk);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr)&lds[0][0];
  typename A::Loads la;
  typename B::Loads lb;
  la.set(g.lda, g.I - i0, wave, lane);
  lb.set(g.ldb, g.J - j0, wave, lane);
  const uint16_t* pa = g.a + (kTurnA ? c0 * g.lda + i0 : i0 * g.lda + c0);
  const uint16_t* pb = g.b + (kTurnB ? c0 * g.ldb + j0 : j0 * g.ldb + c0);
  int left = (int)(c1 - c0);
  auto fill = [&](uint32_t stage) {  // a stage behind the last is zeros
    la.fill(lds0 + stage, pa, left, wave);
    lb.fill(lds0 + stage + kI * kBk * 2, pb, left, wave);
    pa += kTurnA ? kBk * g.lda : kBk;
    pb += kTurnB ? kBk * g.ldb : kBk;
    left -= kBk;
  };

  f32x4 acc[kMt][kNt];
#pragma unroll
  for (int m = 0; m < kMt; ++m)
#pragma unroll
    for (int n = 0; n < kNt; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
  const int wi = wave / kWj * (kI / kWi), wj = wave % kWj * (kJ / kWj);
  typename A::Places wa;
  typename B::Places wb;
  wa.set(lds0, wi, lane);
  wb.set(lds0 + kI * kBk * 2, wj, lane);
  u32x4 fa[2][kMt], fb[2][kNt];
  auto read = [&](auto half, uint32_t stage) {
    constexpr int h = decltype(half)::value;
#pragma unroll
    for (int n = 0; n < kNt; ++n) fb[h][n] = wb.template frag<h>(n, stage);
#pragma unroll
    for (int m = 0; m < kMt; ++m) fa[h][m] = wa.template frag<h>(m, stage);
  };
  // The products of one half, the LDS reads of the next between them.
  auto multiply = [&](auto half) {
    constexpr int h = decltype(half)::value;
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int n = 0; n < kNt; ++n) acc[m][n] = T::mfma(fb[h][n], fa[h][m], acc[m][n]);
    constexpr int kReads = kNt * B::kReads + kMt * A::kReads, kEach = kMt * kNt / kReads > 0 ? kMt * kNt / kReads : 1;
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // an LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);  // matrix products
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // All but this wave's `newer` youngest loads are in LDS and its reads done; then all waves'.
  auto meet = [&](auto newer) {
    constexpr int n = decltype(newer)::value;
    static_assert(n < 64, "vmcnt counts to 63");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);  // vmcnt n, lgkmcnt 0
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, 1> kSecond{};

  constexpr int kInFlight = A::kLoads + B::kLoads;  // loads of one stage
  const bool plain = !g.e.z && g.e.act == ENGRAM_ACT_NONE;
#pragma unroll
  for (int s = 0; s < kDepth; ++s) fill(s * kStageBytes);
  if (!kTurnB && !cut && plain && g.e.residual) {
    // nothing but a residual to add: the sums begin with it, loaded while the first stages are on
    // their way (4000 x 5120 x 5120: 19 us more than without a residual; 31 when read at the end)
#pragma unroll
    for (int n = 0; n < kNt; n += 2)
#pragma unroll
      for (int m = 0; m < kMt; ++m) {
        // places beyond the result take its last row or columns, which are not stored: no branch, so
        // that all loads are on their way at once
        const int64_t i = min(i0 + wi + m * 16 + lane % 16, g.I - 1);
        const int64_t j = min(j0 + wj + n * 16 + 8 * (lane / 16), g.J - 8);
        float r[8];
        unpack8<T>(load_residual(i, j, g.e), r);
        acc[m][n] = f32x4{r[0], r[1], r[2], r[3]};
        acc[m][n + 1] = f32x4{r[4], r[5], r[6], r[7]};
      }
  }
  meet(std::integral_constant<int, (kDepth - 1) * kInFlight>{});
  read(kFirst, 0);
  uint32_t stage = 0;
#pragma nounroll
  for (int s = 0; s < stages; ++s) {
    read(kSecond, stage);
    multiply(kFirst);
    meet(std::integral_constant<int, (kDepth - 2) * kInFlight>{});  // stage s + 1 is there, stage s read out by all
    fill(stage);
    stage = stage + kStageBytes == kDepth * kStageBytes ? 0 : stage + kStageBytes;
    read(kFirst, stage);
    multiply(kSecond);
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the last fills, of nothing, must not outlive the workgroup's LDS

  // lane: row l of each 16; eight neighbouring columns of each 32 (a turned B: two fours, 16 apart)
  if (cut || kTurnB || plain) {
    float* sums = cut ? g.partial + ((int64_t)(tile - g.whole) * g.parts + part) * kI * kJ : nullptr;
    constexpr int kApart = kTurnB ? 16 : 4;
#pragma unroll
    for (int n = 0; n < kNt; n += 2) {
      const int jj = wj + n * 16 + (kTurnB ? 4 : 8) * (lane / 16);
      float bias[8];
      load_bias(bias, cut || kTurnB || j0 + jj >= g.J ? nullptr : g.e.bias, j0 + jj);
#pragma unroll
      for (int m = 0; m < kMt; ++m) {
        const int ii = wi + m * 16 + lane % 16;
        if (i0 + ii >= g.I) continue;
        if (cut) {
          float* p = sums + ii * kJ + jj;
          *reinterpret_cast<f32x4*>(p) = acc[m][n];
          *reinterpret_cast<f32x4*>(p + kApart) = acc[m][n + 1];
          continue;
        }
        uint16_t* p = static_cast<uint16_t*>(g.e.y) + (i0 + ii) * g.e.ldy + j0;
        if constexpr (kTurnB) {
          // four columns of each of two sixteens become eight neighbours of one: every other sixteen
          // lanes change over (25600 x 4096 x 2560: 450 us against 458 with stores of four)
          const u32x2 x = pack4<T>(acc[m][n]), y = pack4<T>(acc[m][n + 1]);
          const u32x2 u = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
          const u32x2 v = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
          const int j = wj + n * 16 + 16 * (lane / 16 % 2) + 8 * (lane / 32);
          if (j0 + j < g.J) store16(p + j, u32x4{u[0], v[0], u[1], v[1]});
        } else if (j0 + jj < g.J) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = acc[m][n][k] + bias[k];
            v[k + 4] = acc[m][n + 1][k] + bias[k + 4];
          }
          store16(p + jj, pack8<T>(v));
        }
      }
    }
    return;
  }
  // With an activation or z the epilogue is long, and unrolled over
  // the accumulators it would be more code than the instruction cache holds: the
  // sums go through LDS, 32 columns of each wave at a time, and one loop ends them.
  // Piece p (four columns) of row r lies at p ^ (r & 7).
  if constexpr (!kTurnB) {
    __syncthreads();  // the last fragments are read
    constexpr int kRows = kI / kWi;
    float* mine = reinterpret_cast<float*>(&lds[0][0]) + wave * kRows * 32;
    static_assert(kWaves * kRows * 32 * sizeof(float) <= sizeof(lds), "the waves' sums fit");
#pragma unroll
    for (int n = 0; n < kNt; n += 2) {
#pragma unroll
      for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = m * 16 + lane % 16;
          *reinterpret_cast<f32x4*>(mine + r * 32 + ((2 * (lane / 16) + h) ^ (r & 7)) * 4) = acc[m][n + h];
        }
      const int64_t j = j0 + wj + n * 16 + 8 * (lane % 4);
      float bias[8];
      load_bias(bias, j < g.J ? g.e.bias : nullptr, j);
      constexpr int kAhead = 4;  // rows whose residuals are loaded together
#pragma nounroll
      for (int r0 = lane / 4; r0 < kRows; r0 += 16 * kAhead) {
        u32x4 residual[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int64_t i = i0 + wi + r0 + 16 * k;
          if (r0 + 16 * k < kRows && i < g.I && j < g.J && g.e.residual) residual[k] = load_residual(i, j, g.e);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = r0 + 16 * k;
          if (r >= kRows) break;
          const f32x4 a = *reinterpret_cast<const f32x4*>(mine + r * 32 + ((2 * (lane % 4)) ^ (r & 7)) * 4);
          const f32x4 b = *reinterpret_cast<const f32x4*>(mine + r * 32 + ((2 * (lane % 4) + 1) ^ (r & 7)) * 4);
          float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
          const int64_t i = i0 + wi + r;
          if (i < g.I && j < g.J) finish8<T>(v, bias, residual[k], i, j, g.e);
        }
      }
    }
  }
}

// The cut tiles: the sum of each one's parts, in order, and the epilogue.
constexpr int kJoinThreads = 256;
template <typename T, int kI, int kJ>
__global__ __launch_bounds__(kJoinThreads) void gemm_join_kernel(GemmArgs g) {
  const int tile = blockIdx.y, at = (blockIdx.x * kJoinThreads + threadIdx.x) * 8;
  int64_t i0, j0;
  tile_origin(g, g.whole + tile, kI, kJ, i0, j0);
  const int64_t i = i0 + at / kJ, j = j0 + at % kJ;
  if (i >= g.I || j >= g.J) return;
  u32x4 residual = {0, 0, 0, 0};
  if (g.e.residual) residual = load_residual(i, j, g.e);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, bias[8];
  const float* p = g.partial + (int64_t)tile * g.parts * kI * kJ + at;
  for (int s = 0; s < g.parts; ++s, p += kI * kJ) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] += a[k];
      v[k + 4] += b[k];
    }
  }
  load_bias(bias, g.e.bias, j);
  finish8<T>(v, bias, residual, i, j, g.e);
}

// ---------------------------------------------------------------- few rows

template <typename T>
__device__ __forceinline__ float finish1(float v, int64_t i, int64_t j, const Epilogue& e) {
  if (e.bias) v += e.bias[j];
  if (e.z) static_cast<uint16_t*>(e.z)[i * e.ldz + j] = (uint16_t)T::pack(v, 0.0f);
  if (e.act != ENGRAM_ACT_NONE) v = act_of(v, e.act);
  if (e.residual) v += T::lo(static_cast<const uint16_t*>(e.residual)[i * e.ldr + j]);
  return v;
}

// y for N <= kN rows of x.  W is read once, a wave reading whole rows of it, 1 KB
// side by side, kR rows at a time; the products are plain fp32 ones (at N = 1
// a matrix product would leave fifteen of sixteen columns empty).
constexpr int kVecThreads = 256;
template <typename T, int kN, int kR>
__global__ __launch_bounds__(kVecThreads) void vector_kernel(const uint16_t* x, const uint16_t* w, int64_t ldx, int N,
                                                             int64_t K, int64_t M, Epilogue e) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = ((int64_t)blockIdx.x * (kVecThreads / 64) + wave) * kR;
  if (m0 >= M) return;
  float s[kN][kR];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int r = 0; r < kR; ++r) s[n][r] = 0.0f;
  // rows behind the last one read the last one again; their sums are not stored
#pragma unroll 2
  for (int64_t k = 8 * lane; k < K; k += 512) {
    u32x4 fw[kR], fx[kN];
#pragma unroll
    for (int r = 0; r < kR; ++r) fw[r] = load16(w + min(m0 + r, M - 1) * K + k);
#pragma unroll
    for (int n = 0; n < kN; ++n) fx[n] = load16(x + min(n, N - 1) * ldx + k);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float xv[8];
      unpack8<T>(fx[n], xv);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float wv[8];
        unpack8<T>(fw[r], wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[n][r] = fmaf(xv[i], wv[i], s[n][r]);
      }
    }
  }
  // the sum of value (n, r) goes to lane n kR + r
  float mine = 0.0f;
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const float t = read_lane(wave_sum_to_lane63(s[n][r]), 63);
      if (lane == n * kR + r) mine = t;
    }
  const int n = lane / kR;
  const int64_t m = m0 + lane % kR;
  if (n < kN && n < N && m < M)
    static_cast<uint16_t*>(e.y)[n * e.ldy + m] = (uint16_t)T::pack(finish1<T>(mine, n, m, e), 0.0f);
}

// y for N <= 16 rows of x and a small W.  A workgroup has kR rows of W; its waves
// take every kWaves-th piece of 64 contraction values, straight from memory into
// the matrix cores, and join in LDS: one launch, where tiles would need a second
// one to join a split contraction (13 x 5120 x 1368: 9.8 us against 15.5; at
// 131 MB of W the tiles' whole lines win, 33 us against 39).  What a CU can ask
// its cache for bounds it, 64 bytes of a row at a time: lanes whose rows are not
// there load from beyond their buffer, which is zero and asks for nothing.
template <typename T, int kWaves, int kR>
__global__ __launch_bounds__(kWaves * 64) void rows_kernel(const uint16_t* x, const uint16_t* w, int64_t ldx, int N,
                                                           int64_t K, int64_t M, Epilogue e) {
  __shared__ f32x4 part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane % 16, g = lane / 16;
  const int64_t m0 = (int64_t)blockIdx.x * kR;
  const __amdgpu_buffer_rsrc_t wb = buffer_of(w + m0 * K), xb = buffer_of(x);
  const uint32_t wr = l < kR && m0 + l < M ? (uint32_t)(l * (int)K + 8 * g) * 2 : kBeyond;
  const uint32_t xr = l < N ? (uint32_t)(l * (int)ldx + 8 * g) * 2 : kBeyond;
  const auto load = [](__amdgpu_buffer_rsrc_t from, uint32_t at, int k) {  // contraction values from k on
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, (int)at, 2 * k, 0));
  };
  f32x4 acc = {0, 0, 0, 0};
  const int pieces = (int)(K / 64);
  // pieces whose loads are in flight together: as registers allow, or (four waves, more than 16384 rows of a
  // small W) the four at most that a wave has
  constexpr int kAhead = kWaves == 16 ? 6 : 4;
  for (int p = wave; p < pieces; p += kAhead * kWaves) {
    u32x4 fw[kAhead][2], fx[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (p + u * kWaves >= pieces) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fw[u][h] = load(wb, wr, (p + u * kWaves) * 64 + 32 * h);
        fx[u][h] = load(xb, xr, (p + u * kWaves) * 64 + 32 * h);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (p + u * kWaves >= pieces) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = T::mfma(fw[u][h], fx[u][h], acc);
    }
  }
  if (wave == pieces % kWaves) {  // what is left of K, a multiple of 8 below 64
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = pieces * 64 + 32 * h;
      const bool in = at + 8 * g < K;
      acc = T::mfma(load(wb, in ? wr : kBeyond, at), load(xb, in ? xr : kBeyond, at), acc);
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  // lane: row of x l, four neighbouring rows of W; two lanes' fours make eight columns of y
  const int row = threadIdx.x % 16, half = threadIdx.x / 16;
  const int64_t j = m0 + 8 * half;
  if (half >= kR / 8 || row >= N || j >= M) return;
  f32x4 s0 = part[0][row + 32 * half], s1 = part[0][row + 32 * half + 16];
#pragma unroll 4
  for (int v = 1; v < kWaves; ++v) {
    s0 += part[v][row + 32 * half];
    s1 += part[v][row + 32 * half + 16];
  }
  float v[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]}, bias[8];
  load_bias(bias, e.bias, j);
  u32x4 residual = {0, 0, 0, 0};
  if (e.residual) residual = load_residual(row, j, e);
  finish8<T>(v, bias, residual, row, j, e);
}

// ---------------------------------------------------------------- the activation's gradient and dbias

// dz = dy act'(z) and the columns' sums of dz over a slice of the rows.
constexpr int kGradThreads = 256, kGradCols = 256, kGradLines = 8;
template <typename T>
__global__ __launch_bounds__(kGradThreads) void act_grad_kernel(const uint16_t* gy, const uint16_t* z, uint16_t* dz,
                                                                float* partial, int64_t N, int64_t M, int64_t ldgy,
                                                                int64_t ldz, int64_t rows, int act) {
  __shared__ float sums[kGradLines][kGradCols];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int64_t j = (int64_t)blockIdx.x * kGradCols + 8 * tx;
  const int64_t n1 = min((int64_t)(blockIdx.y + 1) * rows, N);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (j < M) {
#pragma unroll 2
    for (int64_t n = (int64_t)blockIdx.y * rows + ty; n < n1; n += kGradLines) {
      float v[8];
      unpack8<T>(load16_stream(gy + n * ldgy + j), v);
      if (act != ENGRAM_ACT_NONE) {
        float zz[8];
        unpack8<T>(load16_stream(z + n * ldz + j), zz);
        // (relu passes nothing on below zero, also of an infinite gradient, whose product with 0 is NaN)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act == ENGRAM_ACT_RELU && zz[k] <= 0.0f ? 0.0f : v[k] * act_slope(zz[k], act);
        store16(dz + n * M + j, pack8<T>(v));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += v[k];
    }
  }
  if (!partial) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sums[ty][8 * tx + k] = s[k];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * kGradCols + threadIdx.x;
  if (col < M) {
    float t = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kGradLines; ++i) t += sums[i][threadIdx.x];
    partial[blockIdx.y * M + col] = t;
  }
}

__global__ __launch_bounds__(256) void bias_grad_kernel(const float* partial, float* db, int64_t M, int slices) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= M) return;
  float s = 0.0f;
#pragma unroll 16  // so many loads on their way (M = 25600: 5 us, 17 one by one)
  for (int i = 0; i < slices; ++i) s += partial[i * M + col];
  db[col] = s;
}

// ---------------------------------------------------------------- launches

size_t plan_bytes(int64_t I, int64_t J, int64_t C) {
  const Plan p = plan_of(I, J, C);
  return (size_t)p.cut * (size_t)p.parts * kShapes[p.shape].i * kShapes[p.shape].j * sizeof(float);
}

template <typename T, bool kTurnA, bool kTurnB, int kI, int kJ, int kWi, int kWj, int kDepth>
hipError_t launch_tiles(const Plan& p, GemmArgs& g, hipStream_t stream) {
  void* args[] = {&g};
  const hipError_t e = hipLaunchKernel((const void*)&gemm_kernel<T, kI, kJ, kWi, kWj, kDepth, kTurnA, kTurnB>,
                                       dim3((unsigned)(p.whole + p.cut * p.parts)), dim3(kWi * kWj * 64), args, 0, stream);
  if (e != hipSuccess || p.cut == 0) return e;
  return hipLaunchKernel((const void*)&gemm_join_kernel<T, kI, kJ>, dim3(kI * kJ / 8 / kJoinThreads, (unsigned)p.cut),
                         dim3(kJoinThreads), args, 0, stream);
}

template <typename T, bool kTurnA, bool kTurnB>
hipError_t launch_gemm(GemmArgs g, hipStream_t stream) {
  const Plan p = plan_of(g.I, g.J, g.C);
  g.ti = p.ti;
  g.tj = p.tj;
  g.whole = p.whole;
  g.parts = p.parts;
  g.c_part = p.c_part;
  switch (p.shape) {
    case 0: return launch_tiles<T, kTurnA, kTurnB, 256, 256, 2, 4, 2>(p, g, stream);
    case 1: return launch_tiles<T, kTurnA, kTurnB, 128, 128, 2, 2, 2>(p, g, stream);
    case 2: return launch_tiles<T, kTurnA, kTurnB, 128, 128, 2, 2, 4>(p, g, stream);
    case 3: return launch_tiles<T, kTurnA, kTurnB, 64, 128, 1, 4, 2>(p, g, stream);
    default: return launch_tiles<T, kTurnA, kTurnB, 32, 128, 1, 4, 2>(p, g, stream);
  }
}

int64_t grad_rows(int64_t N) { return up(up(N, 64), kGradLines) * kGradLines; }  // rows of a slice: at most 64 slices
size_t pad16(size_t n) { return (n + 15) / 16 * 16; }

template <typename T, int kN, int kR>
hipError_t launch_vector(const LinearCall& l, const Epilogue& e, hipStream_t stream) {
  const uint16_t *x = static_cast<const uint16_t*>(l.x), *w = static_cast<const uint16_t*>(l.w);
  int64_t ldx = l.ldx, K = l.K, M = l.M;
  int N = (int)l.N;
  Epilogue ep = e;
  void* args[] = {&x, &w, &ldx, &N, &K, &M, &ep};
  return hipLaunchKernel((const void*)&vector_kernel<T, kN, kR>, dim3((unsigned)up(M, kR * kVecThreads / 64)),
                         dim3(kVecThreads), args, 0, stream);
}

template <typename T, int kWaves, int kR>
hipError_t launch_rows(int64_t M, void** args, hipStream_t stream) {
  return hipLaunchKernel((const void*)&rows_kernel<T, kWaves, kR>, dim3((unsigned)up(M, kR)), dim3(kWaves * 64), args, 0,
                         stream);
}

template <typename T>
hipError_t linear_fwd(const LinearCall& l, hipStream_t stream) {
  const Epilogue e{l.bias, l.residual, l.z, l.y, l.ldr, l.ldz, l.ldy, l.act};
  if (l.N <= kVectorRows) {
    // rows of W a wave has on its way: four, or fewer where that leaves the chip short of waves
    // (1 x 5120 x 5120: 11.2 us with one; 4 x 5120 x 5120: 15.7 us with two, 19.6 with one)
    const bool many = l.M >= 8192;
    if (l.N == 1) return many ? launch_vector<T, 1, 4>(l, e, stream) : launch_vector<T, 1, 1>(l, e, stream);
    if (l.N == 2) return many ? launch_vector<T, 2, 4>(l, e, stream) : launch_vector<T, 2, 1>(l, e, stream);
    return many ? launch_vector<T, 4, 4>(l, e, stream) : launch_vector<T, 4, 2>(l, e, stream);
  }
  if (few_rows(l.N, l.K, l.M)) {
    const uint16_t *x = static_cast<const uint16_t*>(l.x), *w = static_cast<const uint16_t*>(l.w);
    int64_t ldx = l.ldx, K = l.K, M = l.M;
    int N = (int)l.N;
    Epilogue ep = e;
    void* args[] = {&x, &w, &ldx, &N, &K, &M, &ep};
    // waves of a workgroup: enough of them on the chip to keep its memory busy; rows of W: fewer where
    // workgroups with 16 would leave half of the CUs idle (13 x 5120 x 1368: 9.8 us against 11.4)
    if (M > 16 * 1024) return launch_rows<T, 4, 16>(M, args, stream);
    if (M > 16 * 128) return launch_rows<T, 16, 16>(M, args, stream);
    return launch_rows<T, 16, 8>(M, args, stream);
  }
  GemmArgs g{};
  g.a = static_cast<const uint16_t*>(l.x);
  g.b = static_cast<const uint16_t*>(l.w);
  g.lda = l.ldx;
  g.ldb = l.K;
  g.I = l.N;
  g.J = l.M;
  g.C = l.K;
  g.partial = static_cast<float*>(l.workspace);
  g.e = e;
  return launch_gemm<T, false, false>(g, stream);
}

// Workspace of the backward: dz, the slices' column sums, a split contraction's parts.
template <typename T>
hipError_t linear_bwd(const LinearCall& l, hipStream_t stream) {
  char* ws = static_cast<char*>(l.workspace);
  uint16_t* dz = reinterpret_cast<uint16_t*>(ws);
  float* sums = reinterpret_cast<float*>(ws + pad16((size_t)l.N * (size_t)l.M * 2));
  const int64_t rows = grad_rows(l.N);
  const int slices = (int)up(l.N, rows);
  float* parts = sums + pad16((size_t)slices * (size_t)l.M * 4) / 4;
  const uint16_t* gy = static_cast<const uint16_t*>(l.grad_y);
  int64_t N = l.N, M = l.M, ldgy = l.ldgy, ldz = l.ldz;
  if (l.act != ENGRAM_ACT_NONE || l.grad_bias) {
    const uint16_t* z = static_cast<const uint16_t*>(l.z_in);
    float* partial = l.grad_bias ? sums : nullptr;
    int64_t r = rows;
    int act = l.act;
    void* args[] = {&gy, &z, &dz, &partial, &N, &M, &ldgy, &ldz, &r, &act};
    hipError_t e = hipLaunchKernel((const void*)&act_grad_kernel<T>, dim3((unsigned)up(M, kGradCols), (unsigned)slices),
                                   dim3(kGradThreads), args, 0, stream);
    if (e != hipSuccess) return e;
    if (l.grad_bias) {
      const float* p = sums;
      float* db = l.grad_bias;
      int n = slices;
      void* args2[] = {&p, &db, &M, &n};
      e = hipLaunchKernel((const void*)&bias_grad_kernel, dim3((unsigned)up(M, 256)), dim3(256), args2, 0, stream);
      if (e != hipSuccess) return e;
    }
    if (l.act != ENGRAM_ACT_NONE) {
      gy = dz;
      ldgy = M;
    }
  }
  GemmArgs g{};
  g.partial = parts;
  if (l.grad_x) {
    g.a = gy;
    g.lda = ldgy;
    g.b = static_cast<const uint16_t*>(l.w);
    g.ldb = l.K;
    g.I = l.N;
    g.J = l.K;
    g.C = l.M;
    g.e = Epilogue{nullptr, nullptr, nullptr, l.grad_x, 0, 0, l.ldgx, ENGRAM_ACT_NONE};
    const hipError_t e = launch_gemm<T, false, true>(g, stream);
    if (e != hipSuccess) return e;
  }
  if (l.grad_w) {
    g.a = gy;
    g.lda = ldgy;
    g.b = static_cast<const uint16_t*>(l.x);
    g.ldb = l.ldx;
    g.I = l.M;
    g.J = l.K;
    g.C = l.N;
    g.e = Epilogue{nullptr, nullptr, nullptr, l.grad_w, 0, 0, l.K, ENGRAM_ACT_NONE};
    return launch_gemm<T, true, true>(g, stream);
  }
  return hipSuccess;
}

}  // namespace

size_t linear_fwd_workspace(int64_t N, int64_t K, int64_t M) { return few_rows(N, K, M) ? 0 : plan_bytes(N, M, K); }

size_t linear_bwd_workspace(int64_t N, int64_t K, int64_t M) {
  const size_t slices = (size_t)up(N, grad_rows(N)), dx = plan_bytes(N, K, M), dw = plan_bytes(M, K, N);
  return pad16((size_t)N * (size_t)M * 2) + pad16(slices * (size_t)M * 4) + (dx > dw ? dx : dw);
}

hipError_t launch_linear_fwd(const LinearCall& l, hipStream_t stream) {
  return l.dtype == ENGRAM_BF16 ? linear_fwd<Bf16>(l, stream) : linear_fwd<Fp16>(l, stream);
}
hipError_t launch_linear_bwd(const LinearCall& l, hipStream_t stream) {
  return l.dtype == ENGRAM_BF16 ? linear_bwd<Bf16>(l, stream) : linear_bwd<Fp16>(l, stream);
}

}  // namespace engram
