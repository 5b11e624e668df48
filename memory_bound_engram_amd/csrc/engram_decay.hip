// engram_decay.hip -- causal linear attention with a fixed decay for each head:
// the chunked forward over ragged sequences, its backward, and the recurrent
// step of single tokens (gfx950).
//
// For every sequence and head, lam = exp(log_decay[h]), S a Dk x Dv state:
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// and with G_t = scale q_t do_t^T + lam G_{t+1} (G behind the last token: the
// gradient of the final state over lam):
//   dq_t = scale S_t do_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_in = lam G_0
//
// One map does all of it.  For rows a, b (Da values) and c (Dc values) along
// an axis of time and a carried Da x Dc state X,
//   y_t = s_intra sum_{s <= t} lam^(t-s) (a_t . b_s) c_s + s_inter lam^(t+e) X^T a_t
// over a chunk of L rows, after which X becomes
//   lam^L X + s_upd sum_s lam^(L-e-s) b_s c_s^T.
// forward (e = 1):         a, b, c = q, k, v            y = o
// dq (e = 1, X = S^T):     a, b, c = do, v, k           y = dq
// dk (e = 0, time turned): a, b, c = v, do, q           y = dk
// dv (e = 0, time turned): a, b, c = k, q, do           y = dv
//
// Mapping.  The recurrence over tokens becomes matrix products over chunks of
// 64 rows.  A workgroup walks a segment of the token axis for one head with X
// in registers, fp32, wave w the columns of c that belong to it.  Chunks
// start at a sequence's first token, so no product crosses sequences.  Where a
// call has too few heads and sequences to fill the chip, the axis is cut into
// segments: a first kernel walks each segment for its state alone, a second
// joins the states from left to right, and the walk starts each segment from
// its joined state.  The backward's three walks (and its two state passes) are
// one launch each: they read the same rows, which the caches then serve, and
// short calls pay for one launch (300 tokens, 40 heads: 35 us, 66 apart).
//
// Bounds.  The forward of 29623 tokens in 7 sequences, 40 heads of 128 x 128,
// takes 443 us: the state pass 138 for the 0.43 GB that it moves (it reads the
// part of k and v that goes on into another segment), the join 10, the walk 298
// for 1.28 GB.  By the counters nothing bounds the walk alone: 4.3 TB/s are three
// quarters of a copy's rate, the vector ALUs work 56% of the time and the matrix
// cores 26%; a chunk's loads are sent for one chunk ahead, and a workgroup meets
// four times a chunk.  Many sequences of a few tokens are slow, as a workgroup
// walks its segment's one behind the other (64 of 2 tokens, 8 heads: 438 us).
//
// Rounding.  bf16 operands enter the matrix cores as they are; sums are fp32.
// The scores (times their power of the decay) and X are rounded to bf16 where
// they become operands of the products that give y, which is rounded to bf16
// itself.  The products that update X, which all later chunks read and the
// caller gets in fp32, take c times its power of the decay as the sum of three
// bf16 values, 24 bits, to its last one (two leave 2.5e-6 of the state).
#include "engram_device.h"
#include "engram_launch.h"
#include "engram_layers_device.h"

#include <utility>

namespace engram {
namespace {

constexpr int kChunk = 64;
constexpr int kStreamed = 2;  // buffer stores: the line is not kept in the caches

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) const void* lds_ptr;


__device__ __forceinline__ bf16x8 join8(u32x2 lo, u32x2 hi) {
  const u32x4 r = {lo[0], lo[1], hi[0], hi[1]};
  return __builtin_bit_cast(bf16x8, r);
}

// A tile in LDS: rows of kD (64 or 128) values without gaps, the 16-byte pieces
// of row r in the order piece ^ turn(r).  LDS serves sixteen lanes of a 16-byte
// read at once (rows 0-3 and 12-15 of one piece with rows 4-11 of the next, or
// the other way round) and thirty-two of an 8-byte or transposing one (sixteen
// rows of one piece; or rows 0-3 of two eights in different halves of 16); with
// this order the lanes of each kind find their values in different banks (counted:
// no conflicts in the state pass, 9% of the LDS cycles in the walk).
template <int kD>
__device__ __forceinline__ uint32_t turn(uint32_t row) {
  const uint32_t b2 = row >> 2 & 1, b3 = row >> 3 & 1, b4 = row >> 4 & 1;
  return kD == 128 ? (b4 ^ b3 ^ b2) << 3 | (row & 3) << 1 | b3 : (b4 ^ b3 ^ b2) << 2 | (row & 2) | b3;
}
// Value `col` of row `row`; the reads below take 4 or 8 values from a multiple of that.
template <int kD>
__device__ __forceinline__ uint32_t place(uint32_t row, uint32_t col) {
  return row * kD + ((col >> 3) ^ turn<kD>(row)) * 8 + (col & 7);
}

// Operand fragments of the 16x16x32 product: lane l holds row (or column)
// l % 16 and, with g = l / 16, the eight contraction indices 8g .. 8g+7.
// Here the row is a row of the tile.
template <int kD>
__device__ __forceinline__ bf16x8 frag_rows(const uint16_t* tile, uint32_t row0, uint32_t k0, uint32_t lane) {
  return __builtin_bit_cast(bf16x8, load16(tile + place<kD>(row0 + lane % 16, k0 + 8 * (lane / 16))));
}
// The reads of the next two kinds differ from each other by a piece and by rows
// that are constants: kD / 16 bases a lane serve all of them.
//
// The same rows, with the contraction indices in the order of an accumulator's
// rows: 4g .. 4g+3 of the first sixteen, then of the second.  Base j: row
// l % 16, values 16 j + 4 g; sixteen rows further on, bit 4 of the row turns
// the pieces by half of them.
template <int kD>
struct AccOrder {
  uint32_t at[kD / 16];
  __device__ __forceinline__ explicit AccOrder(uint32_t lane) {
    const uint32_t l = lane % 16, g = lane / 16, first = place<kD>(l, 4 * g);
#pragma unroll
    for (int j = 0; j < kD / 16; ++j) at[j] = first ^ 16 * j;
  }
  template <int kTt, int kKk>
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile) const {
    constexpr int kHalf = kTt & 1 ? kD / 32 : 0;
    return join8(*reinterpret_cast<const u32x2*>(tile + at[(2 * kKk) ^ kHalf] + 16 * kTt * kD),
                 *reinterpret_cast<const u32x2*>(tile + at[(2 * kKk + 1) ^ kHalf] + 16 * kTt * kD));
  }
};
// Here the row is a column of the tile and the contraction runs down the
// tile's rows, read through the transposing LDS load: the sixteen lanes of a
// group name four rows of sixteen values and get a column of four each.  Base
// j: row 8 g + l / 4, values 16 j + 4 (l % 4); four rows further on, bit 2 of
// the row turns the pieces by half of them.
template <int kD>
struct Columns {
  uint32_t at[kD / 16];
  __device__ __forceinline__ explicit Columns(uint32_t lane) {
    const uint32_t l = lane % 16, first = place<kD>(8 * (lane / 16) + l / 4, 4 * (l % 4));
#pragma unroll
    for (int j = 0; j < kD / 16; ++j) at[j] = first ^ 16 * j;
  }
  template <int kKt, int kDt>
  __device__ __forceinline__ bf16x8 frag(const uint16_t* tile) const {
    return two(tile + at[kDt] + 32 * kKt * kD, tile + at[kDt ^ (kD / 32)] + (32 * kKt + 4) * kD);
  }
  static __device__ __forceinline__ bf16x8 two(const uint16_t* x, const uint16_t* y) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)x);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)y);
    return join8(__builtin_bit_cast(u32x2, lo), __builtin_bit_cast(u32x2, hi));
  }
};
// The same for one sixteen columns of a wave's own.
template <int kD>
__device__ __forceinline__ bf16x8 frag_cols(const uint16_t* tile, uint32_t k0, uint32_t col0, uint32_t lane) {
  const uint32_t l = lane % 16, row = k0 + 8 * (lane / 16) + l / 4, col = col0 + 4 * (l % 4);
  return Columns<kD>::two(tile + place<kD>(row, col), tile + place<kD>(row + 4, col));
}

template <int... kI, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, kI...>, F f) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kN, typename F>
__device__ __forceinline__ void unrolled(F f) {
  unrolled(std::make_integer_sequence<int, kN>{}, f);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ u32x2 pack4(f32x4 v) {
  const u32x2 r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  return r;
}

// lam^steps for steps >= 0, from the logarithm of lam to base 2 (lam^0 is 1
// also where lam is 0).
__device__ __forceinline__ float decay_power(float log2_decay, int steps) {
  return steps == 0 ? 1.0f : __builtin_amdgcn_exp2f(log2_decay * (float)steps);
}
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

// The power of the decay that a state is multiplied with, chunk after chunk.
// One fp32 value of it is off by up to 3e-8, for every chunk to the same side; so
// what each rounding drops is carried into the next chunk's, and the product of
// all of them stays within 6e-8.  Below 1/2 there is nothing to carry: the
// product vanishes before it would show.  (lam^steps - 1, added to the state in
// place of a factor, would keep the digits near 1 as well, but lose those of a
// small power, a hundredth of 3e-6, and turn an infinite state into NaN.)
struct Power {
  float near, rest, inverse;  // lam^steps rounded, what that dropped and 1 over it
  __device__ __forceinline__ void set(float log2_decay, float steps) {
    const float x = log2_decay * steps, less_one = expm1f(x * kLn2);
    const bool small = !(x >= -1.0f);
    near = small ? __builtin_amdgcn_exp2f(x) : 1.0f + less_one;
    inverse = small ? 0.0f : __builtin_amdgcn_rcpf(near);
    rest = small ? 0.0f : (less_one - (near - 1.0f)) * inverse;  // the difference is exact
  }
  // The factor, given what the factors before it dropped, and what is dropped now (both relative).
  __device__ __forceinline__ float factor(float& dropped) const {
    const float all = dropped + rest, f = fmaf(near, all, near);
    dropped = all - (f - near) * inverse;
    return f;
  }
};

// The lane's number as a value the compiler knows nothing of: what is computed
// from it stays where it is used, instead of moving out of loops and being
// spilled.
__device__ __forceinline__ uint32_t afresh(uint32_t lane) {
  asm volatile("" : "+v"(lane));
  return lane & 63;
}
__device__ __forceinline__ float afresh(float v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A value that all lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }
__device__ __forceinline__ Power uniform(Power p) { return Power{uniform(p.near), uniform(p.rest), uniform(p.inverse)}; }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const int32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | lo);
}

}  // namespace

struct WalkArgs {
  const uint16_t *a, *b, *c;
  uint16_t* y;
  int64_t lda, ldb, ldc, ldy;  // values between tokens
  const float* log_decay;      // [H]
  const int64_t* cu;           // [B + 1]
  const float* state_in;       // [B][H] states, or null (zero)
  float* state_out;            // [B][H] states, or null (not wanted)
  float* carry;                // [segments][H][Da][Dc]: the state a segment starts from
  int64_t N, seg;              // tokens in all and in a segment
  int B, H, Da, Dc;
  bool turned;                 // the axis of time runs against the tokens
  bool state_t, carry_t;       // state_in/state_out, carry are stored [Dc][Da]
  int e;
  float s_intra, s_inter, s_upd;
};

// Walks over the same tokens and heads that one launch makes.
constexpr int kMostWalks = 3;
struct Walks {
  WalkArgs w[kMostWalks];
  int n, pairs;  // walks; segments times heads of each
};

namespace {

// The sequences along the axis of time.  cu is the caller's: bounds are
// clamped to the tokens there are, so that no content of it leads out of the
// arrays.
struct Sequences {
  const int64_t* cu;
  int64_t N;
  int B;
  bool turned;
  __device__ int64_t bound(int i) const {
    const int64_t v = uniform(cu[i]);
    return v < 0 ? 0 : (v > N ? N : v);
  }
  __device__ int index(int i) const { return turned ? B - 1 - i : i; }  // the i-th along the axis
  __device__ int64_t start(int i) const { return turned ? N - bound(B - i) : bound(i); }
  __device__ int64_t end(int i) const { return turned ? N - bound(B - 1 - i) : bound(i + 1); }
  // the first sequence that ends behind pos (B if none does)
  __device__ int first_behind(int64_t pos) const {
    int lo = 0, hi = B;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (end(mid) > pos) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  }
};

// kDa, kDc: the operand widths in LDS (64 or 128; narrower heads are padded
// with zeros).  kStateOnly: the first kernel of a cut axis, which leaves the
// state of the segment's last, unfinished sequence in the next segment's carry.
template <int kDa, int kDc, bool kStateOnly>
struct Walk {
  static constexpr int kWaves = kDc / 16;         // a wave for every sixteen columns of X
  static constexpr int kThreads = kWaves * 64;
  static constexpr int kDt = kDa / 16;            // tiles of state rows
  static constexpr int kSt = 16 / kWaves;         // of the scores' sixteen tiles, those a wave makes

  // b's tile is there twice, as its last reads come at a chunk's end; a's and
  // c's are read out before, and filled again behind that (the state alone is
  // one pass over b and c, and has both twice).
  struct Lds {
    alignas(16) uint16_t a[kStateOnly ? 8 : kChunk * kDa];
    alignas(16) uint16_t b[2][kChunk * kDa];
    alignas(16) uint16_t c[kStateOnly ? 2 : 1][kChunk * kDc];
    alignas(16) uint16_t p[kStateOnly ? 8 : kChunk * kChunk];
    int bad[2];
  };

  // The 16-byte pieces of a tile that a lane moves, kMoves of them: the q-th lies
  // at (q kWaves + wave) 1024 + 16 lane in the tile, and `at` bytes from the
  // chunk's first row in memory (kBeyond if it is no part of it).
  template <int kD>
  struct Pieces {
    static constexpr uint32_t kMoves = kD * kChunk / 8 / kThreads;
    uint32_t at[kMoves];
    __device__ __forceinline__ Pieces(int64_t ld, int d, int L, const WalkArgs& w, uint32_t wave, uint32_t lane) {
      // a lane's rows are kRows apart, a multiple of 32 or of 16, with which the order of the pieces
      // does not (or, at 16, by half of them) change
      constexpr uint32_t kRows = kThreads / (kD / 8);
      const uint32_t line = (uint32_t)ld * 2;
      const uint32_t t0 = (wave * 64 + lane) / (kD / 8), piece = (wave * 64 + lane) % (kD / 8) ^ turn<kD>(t0);
      const uint32_t first = token_of(t0, L, w) * line, step = w.turned ? 0 - kRows * line : kRows * line;
#pragma unroll
      for (uint32_t q = 0; q < kMoves; ++q) {
        const uint32_t col = (piece ^ turn<kD>(q * kRows)) * 8;
        const bool in = (t0 + q * kRows >= kChunk - (uint32_t)L) & (col < (uint32_t)d);
        at[q] = in ? first + q * step + col * 2 : kBeyond;
      }
    }
  };
  // Rows pos .. pos + L - 1 of the head, straight into LDS as the tile's last L
  // rows, the rows before them zero.
  template <int kD>
  static __device__ __forceinline__ void fetch(const uint16_t* tile, const uint16_t* x, int64_t ld, int head, int d,
                                               int64_t pos, int L, const WalkArgs& w, uint32_t wave, uint32_t lane) {
    const u32x4 src = buffer_words(x + (w.turned ? w.N - pos - L : pos) * ld + (int64_t)head * d);
    const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr)tile;
    const Pieces<kD> p(ld, d, L, w, wave, lane);
#pragma unroll
    for (uint32_t q = 0; q < p.kMoves; ++q) load_to_lds(to + (q * kWaves + wave) * 1024, src, p.at[q]);
  }
  // The token of a tile's row t, from the chunk's first token in memory.
  static __device__ __forceinline__ uint32_t token_of(uint32_t t, int L, const WalkArgs& w) {
    return w.turned ? kChunk - 1 - t : t - (uint32_t)(kChunk - L);
  }
  static __device__ __forceinline__ bool not_finite(const bf16x8 (&c)[2]) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 r = __builtin_bit_cast(u32x4, c[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, r[k] & 0x7fff7fffu));
    }
    return (most[0] >= 0x7f80) | (most[1] >= 0x7f80);
  }
  // This wave's loads into LDS (and all else) are done; then all waves'.
  static __device__ __forceinline__ void meet() {
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt 0, lgkmcnt 0
    __syncthreads();
  }

  // X as accumulators: tile dt of a wave holds rows 16 dt + 4 g + r and column
  // 16 wave + lane % 16.
  typedef f32x4 State[kDt];

  // kOut: X to p, else p to X (zero where p is null).
  template <bool kOut, bool kTransposed>
  static __device__ __forceinline__ void move_state(State& X, const float* p, const WalkArgs& w, uint32_t wave, uint32_t lane0) {
    const uint32_t lane = afresh(lane0);
    const __amdgpu_buffer_rsrc_t at = buffer_of(p);
    const uint32_t Da = w.Da, Dc = w.Dc, d = 4 * (lane / 16), n = 16 * wave + lane % 16;
    const uint32_t first = p && n < Dc ? 4 * (kTransposed ? n * Da + d : d * Dc + n) : kBeyond;
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) {
      const int off = (int)(16 * dt + d < Da ? first : kBeyond);
      if constexpr (kTransposed && kOut) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, X[dt]), at, off, 64 * dt, 0);
      } else if constexpr (kTransposed) {
        X[dt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(at, off, 64 * dt, 0));
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int line = 4 * (16 * dt + r) * w.Dc;
          if constexpr (kOut) {
            const float v = X[dt][r];
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), at, off, line, 0);
          } else {
            X[dt][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(at, off, line, 0));
          }
        }
      }
    }
  }
  static __device__ __forceinline__ void load_state(State& X, const float* p, bool transposed, const WalkArgs& w, uint32_t wave,
                                                    uint32_t lane) {
    if (transposed) move_state<false, true>(X, p, w, wave, lane);
    else move_state<false, false>(X, p, w, wave, lane);
  }
  static __device__ __forceinline__ void store_state(State& X, float* p, bool transposed, const WalkArgs& w, uint32_t wave,
                                                     uint32_t lane) {
    if (transposed) move_state<true, true>(X, p, w, wave, lane);
    else move_state<true, false>(X, p, w, wave, lane);
  }

  // The powers of the decay that a lane needs, as products of a factor of its
  // own and one that all lanes share: scores lam^(t-s) with t = 16 tile + l and
  // s = 16 st + 4 g + r, and the rows that go into X, lam^(64-e-s) with
  // s = 32 kt + 8 g + i.  A chunk of fewer rows is the tile's last ones, so these
  // do not depend on its length.
  struct Powers {
    float below;         // s_intra lam^(13+l-4g), times lam^(3-r)
    float tiles[3];      // lam^(16 i)
    float rows[2];       // s_upd lam^(57-e-32kt-8g)
    float eight[8];      // lam^i
    Power chunk;         // lam^64
    __device__ __forceinline__ void set(float ld, const WalkArgs& w, uint32_t lane0) {
      const int lane = (int)lane0, g = lane / 16, l = lane % 16;
      below = w.s_intra * decay_power(ld, 13 + l - 4 * g);
      for (int i = 0; i < 3; ++i) tiles[i] = uniform(decay_power(ld, 16 * i));
      for (int kt = 0; kt < 2; ++kt) rows[kt] = w.s_upd * decay_power(ld, kChunk - 7 - w.e - 32 * kt - 8 * g);
      for (int i = 0; i < 8; ++i) eight[i] = uniform(decay_power(ld, i));
      chunk.set(ld, kChunk);
      chunk = uniform(chunk);
    }
  };

  // Eight values of c times their powers of the decay, each as three bf16
  // values: the upper eight bits of what is left, three times.  What a part
  // leaves is taken 2^-24 of the part too large, an error of at most the last
  // bit, so that all three have one sign and none is 0 beside one that is not:
  // an infinity in b makes the state infinite, not NaN as times 0.  kInf: the
  // values may be infinite, as all three parts then are.
  template <bool kInf>
  static __device__ __forceinline__ void split(bf16x8 (&to)[3], bf16x8 c, float up, const Powers& pw) {
    const u32x4 raw = __builtin_bit_cast(u32x4, c);
    u32x4 part[3];
    const auto left = [](float x) {
      const float r = fmaf(__uint_as_float(__float_as_uint(x) & 0xffff0000u), -0x1.fffffep-1f, x);
      return kInf && r != r ? x : r;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x0 = bf_lo(raw[i]) * (up * pw.eight[7 - 2 * i]), x1 = bf_hi(raw[i]) * (up * pw.eight[6 - 2 * i]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        part[k][i] = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302);
        if (k == 2) break;
        x0 = left(x0);
        x1 = left(x1);
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) to[k] = __builtin_bit_cast(bf16x8, part[k]);
  }

  // Walk the rows [pos, stop) of one sequence, chunk by chunk.
  static __device__ __forceinline__ void rows(Lds& lds, State& X, int64_t pos, int64_t stop, int head, const float ld,
                                              const Powers& pw, int& parity, const WalkArgs& w, uint32_t wave, uint32_t lane0) {
    const Columns<kDa> bs(lane0);
    const AccOrder<kDa> as(lane0);
    int64_t single = pos;  // rows before this one are walked one at a time
    float dropped = 0.0f;  // by the factors of X so far
    int L = (int)(stop - pos < kChunk ? stop - pos : kChunk), at_b = 0;
    auto get_b = [&](int to, int64_t at, int n, uint32_t lane) {
      fetch<kDa>(lds.b[to], w.b, w.ldb, head, w.Da, at, n, w, wave, lane);
    };
    auto get_c = [&](int to, int64_t at, int n, uint32_t lane) {
      fetch<kDc>(lds.c[to], w.c, w.ldc, head, w.Dc, at, n, w, wave, lane);
    };
    auto get_a = [&](int64_t at, int n, uint32_t lane) { fetch<kDa>(lds.a, w.a, w.lda, head, w.Da, at, n, w, wave, lane); };
    get_b(0, pos, L, lane0);
    get_c(0, pos, L, lane0);
    if constexpr (!kStateOnly) get_a(pos, L, lane0);
    while (pos < stop) {
      const uint32_t lane = afresh(lane0), g = lane / 16, l = lane % 16;
      const int64_t next = pos + L;
      const int next_L = next < single ? 1 : (int)(stop - next < kChunk ? stop - next : kChunk);
      meet();
      if constexpr (kStateOnly) {
        if (next < stop) {
          get_b(at_b ^ 1, next, next_L, lane);
          get_c(at_b ^ 1, next, next_L, lane);
        }
      }
      const uint16_t *tb = lds.b[at_b], *tc = lds.c[kStateOnly ? at_b : 0];
      bf16x8 cf[2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) cf[kt] = frag_cols<kDc>(tc, 32 * kt, 16 * wave, lane);
      if constexpr (!kStateOnly) {
        // scores, transposed: the lane has row t = 16 tile + l and four neighbouring s; with eight
        // waves two share the rows of a tile
        const uint32_t tile = wave & 3, st0 = wave / 4 * kSt;
        bf16x8 at[kDa / 32];
#pragma unroll
        for (int kk = 0; kk < kDa / 32; ++kk) at[kk] = frag_rows<kDa>(lds.a, 16 * tile, 32 * kk, lane);
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
          const uint32_t st = st0 + i;
          u32x2 packed = {0, 0};
          if (st <= tile) {
            f32x4 s = {0, 0, 0, 0};
            bf16x8 bt[kDa / 32];
#pragma unroll
            for (int kk = 0; kk < kDa / 32; ++kk) bt[kk] = frag_rows<kDa>(tb, 16 * st, 32 * kk, lane);
#pragma unroll
            for (int kk = 0; kk < kDa / 32; ++kk) s = mfma(bt[kk], at[kk], s);
            if (st == tile) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int steps = (int)l - (int)(4 * g + r);
                s[r] = steps >= 0 ? s[r] * (w.s_intra * decay_power(ld, steps)) : 0.0f;
              }
            } else {
              const float between = pw.below * (tile - st == 1 ? 1.0f : tile - st == 2 ? pw.tiles[1] : pw.tiles[2]);
#pragma unroll
              for (int r = 0; r < 4; ++r) s[r] *= between * pw.eight[3 - r];
            }
            packed = pack4(s);
          }
          *reinterpret_cast<u32x2*>(lds.p + place<kChunk>(16 * tile + l, 16 * st + 4 * g)) = packed;
        }
      }
      if constexpr (!kStateOnly) {
        // An infinity or NaN in a row of c would reach the rows before it too, as
        // 0 * c in the product with the scores: such a chunk is walked row by row.
        if (not_finite(cf)) lds.bad[parity] = 1;
        __syncthreads();  // the scores of all waves, and their word on c
        const bool bad = __builtin_amdgcn_readfirstlane(lds.bad[parity]) != 0;
        parity ^= 1;
        if (threadIdx.x == 0) lds.bad[parity] = 0;
        if (bad && L > 1) {
          single = next;
          L = 1;
          get_b(at_b, pos, 1, lane);
          get_c(0, pos, 1, lane);
          get_a(pos, 1, lane);
          continue;
        }
        if (next < stop) get_b(at_b ^ 1, next, next_L, lane);
        // y^T = X^T a^T, then += c^T scores^T: the lane has row t = 16 tt + l and four neighbouring columns
        f32x4 y[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) y[tt] = f32x4{0, 0, 0, 0};
        unrolled<kDa / 32>([&](auto kk) {
          constexpr int kKk = decltype(kk)::value;
          __builtin_amdgcn_sched_barrier(0);
          const bf16x8 xf = join8(pack4(X[2 * kKk]), pack4(X[2 * kKk + 1]));
          bf16x8 af[4];
          unrolled<4>([&](auto tt) {
            constexpr int kTt = decltype(tt)::value;
            // without this the compiler joins the reads of tt and tt + 2, whose results then need moving
            if constexpr (kTt == 2) asm volatile("" ::: "memory");
            af[kTt] = as.template frag<kTt, kKk>(lds.a);
          });
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) y[tt] = mfma(xf, af[tt], y[tt]);
        });
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) y[tt] *= w.s_inter * decay_power(ld, max((int)(16 * tt + l) - (kChunk - L) + w.e, 0));
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int tt = 2 * kt; tt < 4; ++tt) y[tt] = mfma(cf[kt], frag_rows<kChunk>(lds.p, 16 * tt, 32 * kt, lane), y[tt]);
        // y goes out through c's tile, which is in registers: a wave has sixteen columns, 32 bytes of a
        // row, and whole lines are fewer requests and need not stay in the caches (41444 tokens, 40 heads
        // of 128 x 128: 692 us against 707; backward of 9500 tokens, 32 heads: 307 against 328)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
          *reinterpret_cast<u32x2*>(lds.c[0] + place<kDc>(16 * tt + l, 16 * wave + 4 * g)) = pack4(y[tt]);
        __syncthreads();  // y is there, a read out
        if (next < stop) get_a(next, next_L, lane);
        const Pieces<kDc> out(w.ldy, w.Dc, L, w, wave, lane);
        u32x4 rows[out.kMoves];
#pragma unroll
        for (uint32_t q = 0; q < out.kMoves; ++q) rows[q] = load16(lds.c[0] + (q * kWaves + wave) * 512 + 8 * lane);
        __syncthreads();  // y is read out
        if (next < stop) get_c(0, next, next_L, lane);
        const __amdgpu_buffer_rsrc_t dst =
            buffer_of(w.y + (w.turned ? w.N - pos - L : pos) * w.ldy + (int64_t)head * w.Dc);
#pragma unroll
        for (uint32_t q = 0; q < out.kMoves; ++q)
          __builtin_amdgcn_raw_buffer_store_b128(rows[q], dst, (int)out.at[q], 0, kStreamed);
      }
      // X = lam^L X + s_upd sum_s lam^(L-e-s) b_s c_s^T
      Power power = pw.chunk;
      if (L != kChunk) power.set(ld, (float)L);
      const float keep = uniform(power.factor(dropped));
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) X[dt][r] *= keep;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        bf16x8 cs[3];
        const float up = afresh(pw.rows[kt]);
        if (kStateOnly || L == 1) split<true>(cs, cf[kt], up, pw);
        else split<false>(cs, cf[kt], up, pw);
        unrolled<kDt / 4>([&](auto quarter) {
          constexpr int kD0 = 4 * decltype(quarter)::value;
          __builtin_amdgcn_sched_barrier(0);
          bf16x8 bf[4];
          unrolled<4>([&](auto i) {
            constexpr int kI = decltype(i)::value;
            bf[kI] = kt == 0 ? bs.template frag<0, kD0 + kI>(tb) : bs.template frag<1, kD0 + kI>(tb);
          });
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) X[kD0 + i] = mfma(bf[i], cs[k], X[kD0 + i]);
        });
      }
      at_b ^= 1;
      pos = next;
      L = next_L;
    }
    __syncthreads();  // the tiles are read out
  }

  // pair: the segment and the head
  static __device__ __forceinline__ void run(const WalkArgs& w, int pair) {
    __shared__ __attribute__((aligned(16))) Lds lds;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = pair % w.H;
    const int64_t seg = pair / w.H;
    const float ld = uniform(w.log_decay[head]) * kLog2e;  // to base 2
    const Sequences seqs{w.cu, w.N, w.B, w.turned};
    const int64_t from = seg * w.seg, to = from + w.seg < w.N ? from + w.seg : w.N;
    const size_t state = (size_t)w.Da * w.Dc;
    int parity = 0;
    if (threadIdx.x < 2) lds.bad[threadIdx.x] = 0;
    __syncthreads();
    Powers pw;
    pw.set(ld, w, lane);
    State X;
    int i = seqs.first_behind(kStateOnly ? to - 1 : from);
    if constexpr (kStateOnly) {
      // the sequence of the segment's last row, if it goes on behind it
      if (i >= w.B || seqs.end(i) <= to || seqs.start(i) >= to) return;
    }
    int64_t pos = from;
    for (; i < w.B && pos < to; ++i) {
      const int64_t start = seqs.start(i), end = seqs.end(i);
      if (end <= pos) continue;  // an empty sequence
      if (start >= to) break;
      if (start > pos) pos = start;
      const size_t own = ((size_t)seqs.index(i) * w.H + head) * state;
      const size_t cut = ((size_t)seg * w.H + head) * state;
      if (pos == start) load_state(X, w.state_in ? w.state_in + own : nullptr, w.state_t, w, wave, lane);
      else load_state(X, kStateOnly ? nullptr : w.carry + cut, w.carry_t, w, wave, lane);
      const int64_t stop = end < to ? end : to;
      rows(lds, X, pos, stop, head, ld, pw, parity, w, wave, lane);
      if constexpr (kStateOnly) store_state(X, w.carry + cut + (size_t)w.H * state, w.carry_t, w, wave, lane);
      else if (w.state_out && stop == end) store_state(X, w.state_out + own, w.state_t, w, wave, lane);
      pos = stop;
    }
  }
};

template <int kDa, int kDc, bool kStateOnly>
__global__ __launch_bounds__(kDc * 4, kDc / 32) void decay_walk_kernel(Walks s) {
  // the walks of a pair run on one XCD (workgroups go round the eight) at about the same time
  const int walk = blockIdx.x / 8 % s.n, pair = blockIdx.x / (8 * s.n) * 8 + blockIdx.x % 8;
  if (pair < s.pairs) Walk<kDa, kDc, kStateOnly>::run(s.w[walk], pair);
}

// The states that segments start from: carry[j] holds what segment j - 1 alone
// leaves of the sequence across their border; from left to right,
//   carry[j] += lam^seg carry[j - 1]
// within each sequence.  An empty sequence's state goes through unchanged.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void decay_join_kernel(WalkArgs w) {
  const int head = blockIdx.x % w.H, i = blockIdx.x / w.H;
  const int64_t state = (int64_t)w.Da * w.Dc;
  const int64_t at = ((int64_t)blockIdx.y * kJoinThreads + threadIdx.x) * 4;  // state is a multiple of 64
  if (at >= state) return;
  const Sequences seqs{w.cu, w.N, w.B, w.turned};
  const int64_t start = seqs.start(i), end = seqs.end(i);
  if (start >= end) {
    if (w.state_out) {
      const int64_t own = ((int64_t)seqs.index(i) * w.H + head) * state + at;
      const f32x4 zero = {0, 0, 0, 0};
      *reinterpret_cast<f32x4*>(w.state_out + own) =
          w.state_in ? *reinterpret_cast<const f32x4*>(w.state_in + own) : zero;
    }
    return;
  }
  Power power;
  power.set(w.log_decay[head] * kLog2e, (float)w.seg);
  float dropped = 0.0f;
  const int64_t first = start / w.seg + 1, last = (end - 1) / w.seg;
  f32x4 x = {0, 0, 0, 0};
  for (int64_t j = first; j <= last; ++j) {
    f32x4* p = reinterpret_cast<f32x4*>(w.carry + (j * w.H + head) * state + at);
    f32x4 own = *p;
    if (j > first && (j - 1) * w.seg > start) {
      const float keep = power.factor(dropped);
#pragma unroll
      for (int r = 0; r < 4; ++r) own[r] += keep * x[r];
      *p = own;
    }
    x = own;
  }
}

// The recurrent step: row i of the batch is one token of the sequence whose
// state is slot slots[i]; a state is read and written once, which bounds the
// kernel.  A workgroup has kCols columns of one head's state, a thread four
// columns of every (256 / (kCols / 4))-th row.  Rows with the same slot are
// taken in order by the workgroup of the first of them, which keeps the state
// in registers in between.
constexpr int kStepThreads = 256;

template <int kCols>
__global__ __launch_bounds__(kStepThreads) void decay_step_kernel(const uint16_t* q, const uint16_t* k,
                                                                  const uint16_t* v, const float* log_decay,
                                                                  float* pool, const int64_t* slots, uint16_t* o, int B,
                                                                  int H, int Dk, int Dv, int64_t n_slots, int64_t ldq,
                                                                  int64_t ldk, int64_t ldv, int64_t ldo, float scale) {
  constexpr int kGroups = kCols / 4, kRowsAtOnce = kStepThreads / kGroups, kRows = 128 / kRowsAtOnce;
  __shared__ f32x4 part[kRowsAtOnce][kGroups];
  __shared__ int next_row[2];
  int row = blockIdx.x / H;
  const int head = blockIdx.x % H;
  const int64_t slot = slots[row];
  if (slot < 0 || slot >= n_slots) return;
  const int cg = threadIdx.x % kGroups, r0 = threadIdx.x / kGroups;
  const int col = blockIdx.y * kCols + 4 * cg;
  const bool mine = col < Dv;
  float* state = pool + (slot * H + head) * (int64_t)Dk * Dv + col;
  f32x4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int d = r0 + i * kRowsAtOnce;
    const f32x4 zero = {0, 0, 0, 0};
    S[i] = mine && d < Dk ? *reinterpret_cast<const f32x4*>(state + (int64_t)d * Dv) : zero;
  }
  if (threadIdx.x < 2) next_row[threadIdx.x] = B;
  __syncthreads();
  bool behind = false;
  int next = B;
  for (int i = threadIdx.x; i < B; i += kStepThreads)
    if (i != row && slots[i] == slot) {
      if (i < row) behind = true;
      else if (i < next) next = i;
    }
  if (behind) atomicMin(&next_row[1], 0);
  if (next < B) atomicMin(&next_row[0], next);
  __syncthreads();
  if (next_row[1] == 0) return;  // an earlier row's workgroup takes this one
  const float lam = expf(log_decay[head]);
  for (;;) {
    const uint16_t* qr = q + (int64_t)row * ldq + (int64_t)head * Dk;
    const uint16_t* kr = k + (int64_t)row * ldk + (int64_t)head * Dk;
    const uint16_t* vr = v + (int64_t)row * ldv + (int64_t)head * Dv;
    f32x4 vv = {0, 0, 0, 0}, acc = {0, 0, 0, 0};
    if (mine) {
      const u32x2 raw = *reinterpret_cast<const u32x2*>(vr + col);
      vv = f32x4{bf_lo(raw[0]), bf_hi(raw[0]), bf_lo(raw[1]), bf_hi(raw[1])};
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int d = r0 + i * kRowsAtOnce;
      if (d < Dk) {
        const float kd = __uint_as_float((uint32_t)kr[d] << 16), qd = __uint_as_float((uint32_t)qr[d] << 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          S[i][c] = fmaf(lam, S[i][c], kd * vv[c]);
          acc[c] = fmaf(qd, S[i][c], acc[c]);
        }
      }
    }
    part[r0][cg] = acc;
    __syncthreads();
    for (int half = kRowsAtOnce / 2; half >= 1; half /= 2) {
      if (r0 < half) part[r0][cg] += part[r0 + half][cg];
      __syncthreads();
    }
    if (r0 == 0 && mine) {
      f32x4 y = part[0][cg];
      y *= scale;
      *reinterpret_cast<u32x2*>(o + (int64_t)row * ldo + (int64_t)head * Dv + col) = pack4(y);
    }
    row = next_row[0];
    if (row >= B) break;
    __syncthreads();  // next_row is read
    if (threadIdx.x == 0) next_row[0] = B;
    __syncthreads();
    next = B;
    for (int i = row + 1 + threadIdx.x; i < B; i += kStepThreads)
      if (slots[i] == slot && i < next) next = i;
    if (next < B) atomicMin(&next_row[0], next);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int d = r0 + i * kRowsAtOnce;
    if (mine && d < Dk) __builtin_nontemporal_store(S[i], reinterpret_cast<f32x4*>(state + (int64_t)d * Dv));
  }
}

struct WalkKernel {
  const void* kernel;
  int threads;
};
template <int kDa, int kDc, bool kStateOnly>
WalkKernel walk_of() {
  return {(const void*)&decay_walk_kernel<kDa, kDc, kStateOnly>, Walk<kDa, kDc, kStateOnly>::kThreads};
}
template <bool kStateOnly>
WalkKernel walk_kernel(int Da, int Dc) {
  if (Da <= 64) return Dc <= 64 ? walk_of<64, 64, kStateOnly>() : walk_of<64, 128, kStateOnly>();
  return Dc <= 64 ? walk_of<128, 64, kStateOnly>() : walk_of<128, 128, kStateOnly>();
}

int64_t segments(int64_t N, int64_t seg) { return (N + seg - 1) / seg; }

// The walks of one call; those of the same widths in one launch.
template <bool kStateOnly>
hipError_t launch_walks(const WalkArgs* w, int n, hipStream_t stream) {
  bool done[kMostWalks] = {};
  for (int i = 0; i < n; ++i) {
    if (done[i]) continue;
    const WalkKernel k = walk_kernel<kStateOnly>(w[i].Da, w[i].Dc);
    Walks s{};
    for (int j = i; j < n; ++j)
      if (walk_kernel<kStateOnly>(w[j].Da, w[j].Dc).kernel == k.kernel) {
        done[j] = true;
        s.w[s.n++] = w[j];
      }
    // (the last segment leaves no state to another)
    s.pairs = (int)((segments(w[i].N, w[i].seg) - (kStateOnly ? 1 : 0)) * w[i].H);
    void* args[] = {&s};
    const hipError_t e =
        hipLaunchKernel(k.kernel, dim3((unsigned)((s.pairs + 7) / 8 * 8 * s.n)), dim3((unsigned)k.threads), args, 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
hipError_t launch_join(WalkArgs w, hipStream_t stream) {
  void* args[] = {&w};
  const unsigned parts = (unsigned)((w.Da * w.Dc + 4 * kJoinThreads - 1) / (4 * kJoinThreads));
  return hipLaunchKernel(reinterpret_cast<const void*>(&decay_join_kernel), dim3((unsigned)(w.B * w.H), parts),
                         dim3(kJoinThreads), args, 0, stream);
}
// The states of a cut axis, and the states of empty sequences.
hipError_t launch_carries(const WalkArgs* w, int n, hipStream_t stream) {
  const bool cut = segments(w[0].N, w[0].seg) > 1;
  hipError_t e = cut ? launch_walks<true>(w, n, stream) : hipSuccess;
  for (int i = 0; i < n && e == hipSuccess; ++i)
    if (cut || w[i].state_out) e = launch_join(w[i], stream);
  return e;
}

}  // namespace

// Tokens of a segment: as many segments as fit the chip at once (two
// workgroups a CU, which is what the LDS of the 128 x 128 walk lets in; narrower
// heads are cut alike, though more of their workgroups would fit) for all walks
// of a call, since one more would be a second round (9500 tokens, 32 heads of
// 128 x 128, backward: 337 us with the three walks in one round of 5 segments,
// 367 in three rounds of 15, 385 in three launches; 41444 tokens, 40 heads,
// forward: 710 us with the 12 segments that fit, 774 with 6, 737 with 25; all
// before y went out in whole lines).
int64_t decay_segment(int64_t N, int64_t H, int64_t walks) {
  constexpr int64_t kPlaces = 512;
  const int64_t want = walks * H < kPlaces ? kPlaces / (walks * H) : 1;  // segments
  int64_t seg = (N + want - 1) / want;
  seg = (seg + kChunk - 1) / kChunk * kChunk;
  return seg < 2 * kChunk ? 2 * kChunk : seg;
}

// A state for each segment and head: of the forward, and of one direction of the backward.
size_t carry_bytes(int64_t N, int64_t H, int64_t Dk, int64_t Dv, int64_t walks) {
  return (size_t)segments(N, decay_segment(N, H, walks)) * (size_t)H * (size_t)Dk * (size_t)Dv * sizeof(float);
}
size_t decay_fwd_workspace(int64_t N, int64_t H, int64_t Dk, int64_t Dv) { return carry_bytes(N, H, Dk, Dv, 1); }
size_t decay_bwd_workspace(int64_t N, int64_t H, int64_t Dk, int64_t Dv) { return 2 * carry_bytes(N, H, Dk, Dv, 3); }

hipError_t launch_decay_fwd(const DecayCall& d, hipStream_t stream) {
  WalkArgs w{};
  w.a = d.q; w.b = d.k; w.c = d.v; w.y = d.o;
  w.lda = d.ldq; w.ldb = d.ldk; w.ldc = d.ldv; w.ldy = d.ldo;
  w.log_decay = d.log_decay; w.cu = d.cu; w.state_in = d.state_in; w.state_out = d.state_out;
  w.carry = static_cast<float*>(d.workspace);
  w.N = d.N; w.seg = decay_segment(d.N, d.H, 1);
  w.B = (int)d.B; w.H = (int)d.H; w.Da = (int)d.Dk; w.Dc = (int)d.Dv;
  w.e = 1;
  w.s_intra = w.s_inter = d.scale;
  w.s_upd = 1.0f;
  const hipError_t e = launch_carries(&w, 1, stream);
  return e == hipSuccess ? launch_walks<false>(&w, 1, stream) : e;
}

hipError_t launch_decay_bwd(const DecayCall& d, hipStream_t stream) {
  WalkArgs w{}, all[3];
  w.log_decay = d.log_decay; w.cu = d.cu;
  w.N = d.N; w.seg = decay_segment(d.N, d.H, 3);
  w.B = (int)d.B; w.H = (int)d.H;
  // dq: forward in time, the state transposed
  w.carry = static_cast<float*>(d.workspace);
  w.a = d.grad_o; w.b = d.v; w.c = d.k; w.y = d.grad_q;
  w.lda = d.ldgo; w.ldb = d.ldv; w.ldc = d.ldk; w.ldy = d.ldgq;
  w.Da = (int)d.Dv; w.Dc = (int)d.Dk;
  w.state_in = d.state_in; w.state_t = true;
  w.e = 1;
  w.s_intra = w.s_inter = d.scale;
  w.s_upd = 1.0f;
  all[0] = w;
  // dv: against time; this walk's last states are the gradients of state_in
  w.carry += carry_bytes(d.N, d.H, d.Dk, d.Dv, 3) / sizeof(float);
  w.turned = true;
  w.a = d.k; w.b = d.q; w.c = d.grad_o; w.y = d.grad_v;
  w.lda = d.ldk; w.ldb = d.ldq; w.ldc = d.ldgo; w.ldy = d.ldgv;
  w.Da = (int)d.Dk; w.Dc = (int)d.Dv;
  w.state_in = d.grad_state_out; w.state_out = d.grad_state_in; w.state_t = false;
  w.e = 0;
  w.s_inter = 1.0f;
  w.s_upd = d.scale;
  all[1] = w;
  // dk: the same states, transposed
  w.a = d.v; w.b = d.grad_o; w.c = d.q; w.y = d.grad_k;
  w.lda = d.ldv; w.ldb = d.ldgo; w.ldc = d.ldq; w.ldy = d.ldgk;
  w.Da = (int)d.Dv; w.Dc = (int)d.Dk;
  w.state_out = nullptr; w.state_t = true; w.carry_t = true;
  all[2] = w;
  const hipError_t e = launch_carries(all, 2, stream);
  return e == hipSuccess ? launch_walks<false>(all, 3, stream) : e;
}

hipError_t launch_decay_step(const DecayCall& d, hipStream_t stream) {
  const uint16_t *q = d.q, *k = d.k, *v = d.v;
  uint16_t* o = d.o;
  const float* ld = d.log_decay;
  float* pool = d.pool;
  const int64_t* slots = d.slots;
  int B = (int)d.B, H = (int)d.H, Dk = (int)d.Dk, Dv = (int)d.Dv;
  int64_t n_slots = d.n_slots, ldq = d.ldq, ldk = d.ldk, ldv = d.ldv, ldo = d.ldo;
  float scale = d.scale;
  void* args[] = {&q, &k, &v, &ld, &pool, &slots, &o, &B, &H, &Dk, &Dv, &n_slots, &ldq, &ldk, &ldv, &ldo, &scale};
  // A head's columns over two workgroups, or over four where there are few states (64 x 40 states
  // of 128 x 128: 62.6 us, 5.4 TB/s; with one workgroup a head 80.4, with four 74.3, and 77.1 with
  // stores that stay in the caches).
  const bool few = (int64_t)B * H < 512;
  const int cols = few ? 32 : 64;
  const void* kernel = few ? (const void*)&decay_step_kernel<32> : (const void*)&decay_step_kernel<64>;
  return hipLaunchKernel(kernel, dim3((unsigned)(B * H), (unsigned)((Dv + cols - 1) / cols)), dim3(kStepThreads), args, 0,
                         stream);
}

}  // namespace engram
