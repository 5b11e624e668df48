// engram_window.hip -- softmax attention over a sliding window and the first
// tokens of each sequence: forward and backward over ragged sequences (gfx950).
//
// Token i of a sequence sees token j <= i if i - j < W (the window) or j < S (the
// sinks); query head h reads key head h / G.  With c = scale log2(e):
//   s_ij = q_i . k_j,  lse_i = ln sum_j exp(scale s_ij),  p_ij = exp(scale s_ij - lse_i)
//   o_i = sum_j p_ij v_j
// Backward, with delta_i = do_i . o_i and d_ij = p_ij (do_i . v_j - delta_i):
//   dq_i = scale sum_j d_ij k_j,  dk_j = scale sum_i d_ij q_i,  dv_j = sum_i p_ij do_i
// the sums over i also over the G query heads of the key head.
//
// Mapping.  The rows of a sequence and key head are its (token, query head) pairs,
// token after token, so that a narrow window, a short sequence or a few heads
// still make whole tiles.  A workgroup of four waves takes 128 rows, a wave 32;
// the keys that any of them sees, first the sinks that lie before the window
// and then, without a gap, the window, come through LDS in tiles of 64, straight from
// memory, one tile ahead.  Scores
// are computed transposed, so a lane has one row, and rows and columns of the
// softmax stay where the products leave them: its maximum and sum are a lane's own,
// and the weights, rounded, are the next product's operand without going through
// LDS.
//
// The backward has two such kernels: over the keys of 128 rows for dq (and
// delta, which it leaves for the other), and over the rows of 128 keys for dk and
// dv: seven products where five are the least, but no sums of atomics and no partial
// sums in memory but for the sinks.  These are seen by all rows behind the window as
// well; those rows' part of their dk and dv is summed in pieces of the sequence by
// workgroups of their own, and a last, small launch joins it with the window's part.
//
// What bounds them.  7 sequences up to 8192 tokens, 40 + 8 heads of 128, window 1024: the
// forward takes 595 to 635 us, 0.9 PFLOP/s.  The same call with a window of one token takes
// 159 us, 129 of which are its bytes' at a copy's rate: that much is each workgroup's start (bounds,
// queries, first tiles) and end, which the other workgroup of the CU overlaps only in part.  What
// is beyond goes at 1.2 PFLOP/s (window 4096: 1344 us, 1.05 in all).  Over the call the matrix
// cores are busy 48% of the time, the vector units 52%; a wave issues one instruction at a
// time, of any kind, and a SIMD has two (the registers let in no more).  The
// backward of 5 sequences up to 4096, 32 + 8 heads, takes 620 to 680 us (window 1: 178): dq 250
// (matrix cores 44%, CUs 88%), dk and dv 390 (35%, 83%: 760 workgroups, one a CU at a
// time as their LDS is over 128 KB, so that nothing hides their start and end, and the sinks' behind
// them).  Heads of a size between 64 and 128 take the products of 128 (forward at 80: 568 us,
// at 96: 585, at 64: 361).
// What counted in the loops: a fixed
// number of tiles, in which an operand's place in LDS is a constant behind an
// address in a register (40 us of the forward's 676), few scalar instructions for a
// tile's loads (25), no gap between sinks and window (40).  Tried and slower: 64 rows a wave, one
// wave a SIMD (the products' results then lie where the vector unit cannot
// read them, and registers spill); workgroups that stay and fetch the next
// rows while they work on these, one of eight waves a CU.
//
// Rounding.  Sums, maxima and the softmax are fp32.  p and d are rounded to the
// element type as operands of the second products; the sum of p is taken
// unrounded.  (fp16: p and d are taken times powers of two, so that a weight down to 2^-21 of
// a row's largest keeps its digits, and what a smaller one loses is 2^-32 of the largest
// at most; backward, weights down to 2^-28.)
//
// Where p is 0 because j is not seen, the product with v_j would still be NaN if
// v_j is not finite.  Where results come out not finite, what is seen is looked
// through, for 32 rows or keys at once, for values that leave them infinite or NaN by the
// definition too.  If some column has none, the workgroup goes through its tiles once
// more with such values as 0 in the second products, and what is then finite takes
// the place of those columns alone.  (One infinite value, 8000 tokens that see all of their
// past, 16 + 4 heads of 128, fp16: in grad_o at most 4.0 ms, ordinary
// 1.5, in v 1.0, ordinary 0.36; 714 and 143 when such rows were computed again one by one.)
#include "engram_launch.h"
#include "engram_sequences.h"
#include "engram_window_tiles.h"

#include <type_traits>

namespace engram {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kRows = 128;  // (token, head) pairs, or keys, of a workgroup
constexpr int kKeys = 64;   // of a tile

struct WindowArgs {
  const uint16_t *q, *k, *v, *o, *grad_o;
  const int64_t* cu;
  const float* lse_in;
  uint16_t *out, *grad_k, *grad_v;  // out: o, or the gradient of q
  float* lse;                       // forward: written if not null
  float* delta;                     // backward: [N][Hq]
  float* sums;                      // backward: the sinks' sums over pieces of the sequences
  int64_t N, ldq, ldk, ldv, ldo, ldgo, ldout, ldgk, ldgv;
  int B, Hk, G, D, W, S;
  int tiles;                        // workgroups of a key head
  int piece, pieces, sink_blocks;   // backward: tokens of a piece, pieces there may be, their workgroups (0: no sinks)
  float scale;
  Divide by_G;
};

// The workgroups of all key heads, those of a head neighbours on one XCD
// (workgroups go round the eight), so that its L2 serves the keys they share.
__device__ __forceinline__ int neighbours(int block, int blocks) {
  const int each = blocks / 8, rest = blocks % 8, x = block % 8;
  return x * each + (x < rest ? x : rest) + block / 8;
}

// Which sequence a workgroup is in, and which tile of it: sequence b has the
// numbers from first_tile(start, b) on, as many as its tiles of `unit` rows at
// least (`per` rows a token).
__device__ __forceinline__ int64_t first_tile(int64_t start, int b, uint32_t per, uint32_t unit) {
  return start * per / unit + b;
}
struct Sequence {
  int b;
  int64_t start, length, tile;  // tile: negative before the first sequence
  __device__ __forceinline__ Sequence(const WindowArgs& a, int64_t id, uint32_t per, uint32_t unit) {
    const Sequences seqs{a.cu, a.N, a.B};
    int64_t end;
    b = seqs.last_at_most(id, [&](int64_t at, int i) { return first_tile(at, i, per, unit); }, &start, &end);
    length = end - start;
    tile = id - first_tile(start, b, per, unit);
  }
};

__device__ __forceinline__ bool sees(int t, int j, int W, int S) { return j <= t && (j > t - W || j < S); }

// Of sixteen scores of a row at t, for keys start + 8 (e / 4) + e % 4 below end,
// those of keys that it does not see become `other`.
__device__ __forceinline__ void keep_seen(f32x16& s, int t, int start, int end, int W, int S, float other) {
  asm volatile("" : "+v"(start));  // or what follows moves in front of the branch around it
  const int from = t - W + 1 - start, below = (t < end ? t + 1 : end) - start;
  if (__any(start < S)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int j = 8 * (e / 4) + e % 4;
      s[e] = j < below && (j >= from || j < S - start) ? s[e] : other;
    }
  } else {
    const uint32_t span = below > from ? (uint32_t)(below - from) : 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = (uint32_t)(8 * (e / 4) + e % 4 - from) < span ? s[e] : other;
  }
}
// The softmax's terms may exceed 1: the sum and the outputs are scaled anew only
// where the maximum grows by more than 2^kSlack, which after the first keys hardly
// happens (where it grows at all, they would be in most of the halves of a tile, as one
// of a wave's 32 rows always finds a larger score).  Terms keep their digits, and
// in fp16 are far from its largest value.
constexpr float kSlack = 8.0f;

// Weights as operands in fp16, whose steps below 2^-14 are all 2^-24: the forward's terms
// (2^kSlack at most) and the backward's weights (1 at most) are taken times a power
// of two, which the exponential gives for nothing.
template <typename T>
constexpr float kTermsUp = __is_same(T, _Float16) ? 7.0f : 0.0f;
template <typename T>
constexpr float kWeightsUp = __is_same(T, _Float16) ? 14.0f : 0.0f;

// d as an operand in fp16, whose steps below 2^-14 are all 2^-24: d of ordinary small
// gradients over many keys lies there (3000 keys, heads of 64, grad_o of 1e-4: dq off by 1.2% of
// its norm, 0.25% with this, which is its own rounding), and d itself may pass 65504.  So the kernels hold 2^up d: `up` is a
// lane's own, as its row's (dq) or key's (dk) sums are, and goes down, the sums with
// it, where a value would pass 2^kMostBits.  The largest then lies at 2^4 or more below
// 2^5, so that this is rare, and what is less than 2^-18 of the largest loses digits:
// 2^-29 of the largest at most.  (5 sequences up to 4096, 32 + 8 heads of 128, window
// 1024, fp16: 696 us, 677 without.)
constexpr float kUp = 60.0f;      // where it begins: do . v is below 2^39
constexpr int kMostBits = 15, kAimBits = 5;
template <int kD>
__device__ __forceinline__ void keep_in_range(f32x16& d, f32x16 (&sums)[kD / 32], float& up) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(d[e]));
  if (__any(top > (float)(1 << kMostBits))) {
    top = column_max(top);
    // (an infinite or NaN d stays so, and with it the result)
    const int down = top > (float)(1 << kMostBits) && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) - kAimBits : 0;
    const float times = __builtin_amdgcn_ldexpf(1.0f, -down);
    up -= (float)down;
#pragma unroll
    for (int e = 0; e < 16; ++e) d[e] *= times;
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt) sums[dt] *= times;
  }
}

// The keys of a run of tokens, as tiles of kKeys: first the sinks before the window,
// then the window, without a gap.  So the last sinks may lie in the window's first
// tile: as its first `mixed` rows, which stand for tokens just before the window.
struct KeyTiles {
  int sinks, from, to, full, mixed, n;  // the window is from .. to; `full` tiles hold sinks alone
  __device__ __forceinline__ KeyTiles(int first, int last, int W, int S) {
    from = first - W + 1 > 0 ? first - W + 1 : 0;
    to = last + 1;
    sinks = S < from ? S : from;
    if (sinks == from) sinks = from = 0;  // they meet
    full = sinks / kKeys;
    mixed = sinks % kKeys;
    n = (sinks + to - from + kKeys - 1) / kKeys;
  }
  // The token that a tile's first row is or stands for, and the end of the run that it is in.
  __device__ __forceinline__ int start(int i) const { return i < full ? i * kKeys : from - mixed + (i - full) * kKeys; }
  __device__ __forceinline__ int end(int i) const { return i < full ? sinks : to; }
  __device__ __forceinline__ bool mix(int i) const { return i == full && mixed; }
  // What stands in a tile for tokens before this is seen by all rows.
  __device__ __forceinline__ int below(int i, int S) const { return mix(i) ? from : S; }
  // Halves of tiles, 32 rows each, that rows of the tokens first .. last see all of: `count` from `from` on.
  struct Whole {
    int from;
    uint32_t count;
    __device__ __forceinline__ bool has(int half) const { return (uint32_t)(half - from) < count; }
  };
  __device__ __forceinline__ Whole whole(int first, int last, int W) const {
    const int begin = from - mixed - full * kKeys;  // where the first tile would begin, were the sinks before it the window's
    const int lo = last - W + 1 - begin, hi = first + 1 - begin;
    const int at = lo > 0 ? (lo + 31) / 32 : 0, behind = hi > 0 ? hi / 32 : 0;
    return Whole{at, behind > at ? (uint32_t)(behind - at) : 0u};
  }
  // The token of a tile's row, or -1.
  __device__ __forceinline__ int token(int i, int row) const {
    const int j = start(i) + row;
    return mix(i) && row < mixed ? i * kKeys + row : j < end(i) ? j : -1;
  }
};

// A workgroup's rows of a sequence and key head.
struct RowTile {
  int64_t base;      // the sequence's first token
  int length, head;  // tokens; key head
  int t0;            // the first row's token
  uint32_t x0;       // and head
  int rows;          // there are, kRows at most
  __device__ __forceinline__ uint32_t token(uint32_t row, const WindowArgs& a, uint32_t* g) const {
    const uint32_t x = x0 + row, t = a.by_G(x);
    *g = x - t * (uint32_t)a.G;
    return t;
  }
};

__device__ __forceinline__ bool row_tile(const WindowArgs& a, int block, RowTile* r) {
  const int at = neighbours(block, gridDim.x);
  r->head = at / a.tiles;
  const Sequence s(a, at % a.tiles, a.G, kRows);
  const int64_t all = s.length * a.G;
  if (s.tile < 0 || s.length <= 0 || s.tile * kRows >= all) return false;
  const uint32_t first = (uint32_t)s.tile * kRows;  // N * Hq is below 2^30
  r->base = s.start;
  r->length = (int)s.length;
  r->t0 = (int)(first / (uint32_t)a.G);
  r->x0 = first - (uint32_t)r->t0 * (uint32_t)a.G;
  r->rows = all - first < kRows ? (int)(all - first) : kRows;
  return true;
}

// Of a wave's 32 rows, how many there are.
__device__ __forceinline__ int wave_rows(const RowTile& r, uint32_t wave) {
  const int left = r.rows - 32 * (int)wave;
  return left < 32 ? left : 32;
}

// A lane's row of 8-value pieces, as the operand of kD / 16 products.
template <int kD>
__device__ __forceinline__ void load_row(u32x4 (&to)[kD / 16], const uint16_t* p, bool there, int D, int h) {
#pragma unroll
  for (int kk = 0; kk < kD / 16; ++kk) {
    const u32x4 zero = {0, 0, 0, 0};
    to[kk] = there && 16 * kk + 8 * h < D ? load16(p + 16 * kk + 8 * h) : zero;
  }
}

template <typename T>
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b) {
  float x[8], y[8], s = 0.0f;
  unpack8(Raw<T>{{a}}, x);
  unpack8(Raw<T>{{b}}, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  return s;
}
// Between a wave's writes to LDS and its lanes' reads of each other's.
__device__ __forceinline__ void between_lanes() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Accumulators as rows in LDS: a lane's row is column l % 32 of each, its values
// 32 dt + 8 j + 4 h + 0..3; a wave's 32 rows of kD values.
template <typename T, int kD>
__device__ __forceinline__ void put_rows(uint16_t* to, const f32x16 (&v)[kD / 32], float times, uint32_t lane) {
  const uint32_t row = lane & 31, h = lane >> 5;
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x2 w = {pack2<T>(v[dt][4 * j] * times, v[dt][4 * j + 1] * times),
                       pack2<T>(v[dt][4 * j + 2] * times, v[dt][4 * j + 3] * times)};
      *reinterpret_cast<u32x2*>(to + place<kD>(row, 32 * dt + 8 * j + 4 * h)) = w;
    }
}

// A wave's rows out to memory, whole, sixteen bytes a lane.
template <int kD>
__device__ __forceinline__ void store_rows(const uint16_t* mine, const RowTile& r, uint32_t wave, uint32_t lane,
                                           const WindowArgs& a) {
  between_lanes();
#pragma unroll
  for (int i = 0; i < kD / 16; ++i) {
    const uint32_t at = i * 64 + lane, row = at / (kD / 8), col = at % (kD / 8) * 8;
    uint32_t g;
    const uint32_t t = r.token(32 * wave + row, a, &g);
    if ((int)(32 * wave + row) < r.rows && (int)col < a.D)
      store16(a.out + (r.base + r.t0 + t) * a.ldout + (int64_t)(r.head * a.G + g) * a.D + col,
              load16(mine + place<kD>(row, col)));
  }
}

// The q-th pieces of tile i of the keys (or values) from `src` on, the sequence's
// first, where sinks and window may meet in it.
template <typename P>
__device__ __forceinline__ void fetch_keys(const P& pieces, int q, const uint16_t* tile, const uint16_t* src, int64_t ld,
                                           const KeyTiles& keys, int i, int D, uint32_t at, uint32_t wave) {
  const int start = keys.start(i), n = keys.end(i) - start;
  if (keys.mix(i)) {
    const uint64_t some = __ballot((int)pieces.row + q * pieces.kStep < keys.mixed);
    pieces.move_some(q, tile, src + i * kKeys * ld, ld, keys.mixed, D, at, wave, some);
    pieces.move_some(q, tile, src + start * ld, ld, n, D, at, wave, ~some);
  } else {
    pieces.move(q, tile, src + start * ld, ld, n, D, at, wave);
  }
}

// The tiles from one on that are all of the window (the third at the latest), one after
// the other, with few scalar instructions a tile: where it begins and what is left.
// A wave issues one instruction at a time, of any kind.
template <typename P>
struct Following {
  uint64_t next;
  uint32_t at[P::kMoves];  // of the pieces, in bytes from a tile's first row
  uint32_t row_bytes;
  int left;
  __device__ __forceinline__ Following(const P& pieces, const uint16_t* src, int64_t ld, const KeyTiles& keys, int i, int D)
      : next(reinterpret_cast<uint64_t>(src + (int64_t)keys.start(i) * ld)),
        row_bytes((uint32_t)(ld * 2)),
        left(keys.to - keys.start(i)) {
    const uint32_t first = pieces.offset(ld, D);
#pragma unroll
    for (int q = 0; q < P::kMoves; ++q) at[q] = first == kBeyond ? kBeyond : first + q * P::kStep * row_bytes;
  }
  __device__ __forceinline__ u32x4 words(int D) const {
    u32x4 w = buffer_words(reinterpret_cast<const void*>(next));
    const int n = left < kKeys ? left : kKeys;
    w[2] = n > 0 ? (uint32_t)(n - 1) * row_bytes + (uint32_t)(D * 2) : 0;
    return w;
  }
  __device__ __forceinline__ void go_on() {
    next += kKeys * row_bytes;
    left -= kKeys;
  }
};

// Whether they are all finite (a sum that is not finite has a term that is not).
template <int kD>
__device__ __forceinline__ bool finite_rows(const f32x16 (&v)[kD / 32]) {
  float s = 0.0f;
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) s += v[dt][i] * 0x1p-8f;
  return fabsf(s) < INFINITY;
}

// Which of two values, the lower at bit 15 and the upper at bit 31, are not finite.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t exponents = __is_same(T, bf16_t) ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t one = __is_same(T, bf16_t) ? 0x00800080u : 0x04000400u;
  return ((w & exponents) + one) & 0x80008000u;
}
// Of eight, as eight bits.
template <typename T>
__device__ __forceinline__ uint32_t not_finite8(u32x4 v) {
  uint32_t bits = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t f = not_finite<T>(v[w]);
    bits |= (f >> 15 & 1) << 2 * w | (f >> 31) << (2 * w + 1);
  }
  return bits;
}

// The columns in which rows first .. last - 1 (row(i) says where they are) hold a value that is
// not finite, beside those in `found`, and as far as `wanted` asks: bits of columns
// 8 (l % (kD / 8)) on in lane l.  By a wave.
template <typename T, int kD, typename Row>
__device__ __forceinline__ uint32_t columns_not_finite(int first, int last, int D, uint32_t wanted, uint32_t found, Row row) {
  constexpr int kPieces = kD / 8, kAt = 64 / kPieces, kAhead = 8;
  const int lane = threadIdx.x & 63, col = lane % kPieces * 8, sub = lane / kPieces;
  for (int i = first; i < last && __any(wanted & ~found); i += kAt * kAhead) {
    u32x4 v[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int at = i + n * kAt + sub;
      const u32x4 zero = {0, 0, 0, 0};
      v[n] = at < last && col < D ? load16(row(at) + col) : zero;
    }
    uint32_t bits = 0;
#pragma unroll
    for (int n = 0; n < kAhead; ++n) bits |= not_finite8<T>(v[n]);
#pragma unroll
    for (int d = kPieces; d < 64; d *= 2) bits |= __shfl_xor(bits, d);
    found |= bits;
  }
  return found;
}
// Those of row x of a wave's rows in LDS.
template <typename T, int kD>
__device__ __forceinline__ uint32_t columns_lost(const uint16_t* mine, int x, int D) {
  const int col = (int)(threadIdx.x & 63) % (kD / 8) * 8;
  return col < D ? not_finite8<T>(load16(mine + place<kD>(x, col))) : 0u;
}

// What of a wave's 32 rows (or keys) is to be made again: row x's columns lane and lane + 64 if bit
// x is set.
struct Again {
  uint32_t columns[2] = {0, 0};
  __device__ __forceinline__ bool any() const { return __any(columns[0] | columns[1]); }
  // Row x's columns in `bits`, which lie as columns_not_finite has them.
  template <int kD>
  __device__ __forceinline__ void add(int x, uint32_t bits) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int e = 0; e < kD / 64; ++e) columns[e] |= (__shfl(bits, (lane + 64 * e) / 8) >> lane % 8 & 1) << x;
  }
  // Into `out(x)`, from rows in LDS, the row `first` at the earliest.
  template <int kD, typename F>
  __device__ __forceinline__ void put(const uint16_t* mine, F out, int first = 0) const {
    const int lane = threadIdx.x & 63;
    for (int x = first > 0 ? first : 0; x < 32; ++x) {
      if (!__any((columns[0] | columns[1]) >> x & 1)) continue;
      uint16_t* to = out(x);
#pragma unroll
      for (int e = 0; e < kD / 64; ++e)
        if (columns[e] >> x & 1) to[lane + 64 * e] = mine[place<kD>(x, lane + 64 * e)];
    }
  }
};

// Of a wave's rows in `bad`, which lie in LDS and are not finite, the columns that are to be
// made again: those in which all rows of `src` (keys or values) that they see are finite.
// What the tokens low .. high of the wave's rows all see is looked through once, what
// one of them sees besides for it alone.  `t`: a lane's row's token.
template <typename T, int kD>
__device__ __forceinline__ Again rows_again(uint32_t bad, const uint16_t* mine, const uint16_t* src, int64_t ld, int t,
                                            int low, int high, const WindowArgs& a) {
  const auto row = [&](int i) { return src + i * ld; };
  uint32_t wanted = 0;
  for (uint32_t left = bad; left; left &= left - 1) wanted |= columns_lost<T, kD>(mine, __builtin_ctz(left), a.D);
  const int begin = high - a.W + 1 > 0 ? high - a.W + 1 : 0;  // of the window that all of them have
  const int few = a.S < begin ? a.S : begin, sinks = few < low + 1 ? few : low + 1;
  uint32_t common = columns_not_finite<T, kD>(0, sinks, a.D, wanted, 0, row);
  common = columns_not_finite<T, kD>(begin, low + 1, a.D, wanted, common, row);
  Again again;
  for (uint32_t left = bad; left; left &= left - 1) {
    const int x = __builtin_ctz(left), tx = __shfl(t, x);
    const uint32_t need = columns_lost<T, kD>(mine, x, a.D);
    const int before = begin < tx + 1 ? begin : tx + 1, behind = before > low + 1 ? before : low + 1;
    uint32_t found = columns_not_finite<T, kD>(sinks, a.S < tx + 1 ? a.S : tx + 1, a.D, need, common, row);
    found = columns_not_finite<T, kD>(tx - a.W + 1 > 0 ? tx - a.W + 1 : 0, before, a.D, need, found, row);
    found = columns_not_finite<T, kD>(behind, tx + 1, a.D, need, found, row);
    again.add<kD>(x, need & ~found);
  }
  return again;
}

// Whether `one` holds for some wave of the workgroup, through LDS that no one uses.
template <int kOfWaves>
__device__ __forceinline__ bool any_wave(uint16_t* lds, bool one) {
  uint32_t* const flags = reinterpret_cast<uint32_t*>(lds);
  if ((threadIdx.x & 63) == 0) flags[threadIdx.x >> 6] = one;
  __syncthreads();
  uint32_t some = 0;
#pragma unroll
  for (int w = 0; w < kOfWaves; ++w) some |= flags[w];
  return __builtin_amdgcn_readfirstlane(some) != 0;
}

// A tile's values that are not finite become 0; the n-th of kThreads threads of the workgroup.
template <typename T, int kD, int kTileRows, int kTileThreads>
__device__ __forceinline__ void make_finite(uint16_t* tile) {
#pragma unroll
  for (int n = threadIdx.x; n < kTileRows * kD / 8; n += kTileThreads) {
    u32x4 v = load16(tile + 8 * n);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t f = not_finite<T>(v[w]);
      v[w] &= ~((f >> 15 & 1) * 0xffffu | (f >> 31) * 0xffff0000u);
    }
    store16(tile + 8 * n, v);
  }
}

// A thread and its workgroup as the compiler does not know them: what follows from these is
// worked out anew, for the second way through the tiles, instead of being kept in registers
// along the first, which has none to spare.
struct Afresh {
  int block = blockIdx.x;
  uint32_t thread = threadIdx.x;
  __device__ __forceinline__ Afresh() {
    asm volatile("" : "+s"(block));
    asm volatile("" : "+v"(thread));
  }
};

// A lane's row of a workgroup, and what it needs of the keys.
struct OwnRow {
  RowTile r;
  uint32_t lane, wave, h;
  int t, head;  // t: -1 if there is no such row, which sees nothing
  KeyTiles keys;
  const uint16_t *k0, *v0;
  static __device__ __forceinline__ RowTile tile(const WindowArgs& a, int block) {
    RowTile r;
    row_tile(a, block, &r);
    return r;
  }
  __device__ __forceinline__ int last(const WindowArgs& a) const {
    uint32_t g;
    return r.t0 + (int)r.token(r.rows - 1, a, &g);
  }
  __device__ __forceinline__ OwnRow(const WindowArgs& a, const Afresh& at)
      : r(tile(a, at.block)), lane(at.thread & 63), wave(__builtin_amdgcn_readfirstlane(at.thread >> 6)), h(lane >> 5),
        keys(r.t0, last(a), a.W, a.S), k0(a.k + r.base * a.ldk + (int64_t)r.head * a.D),
        v0(a.v + r.base * a.ldv + (int64_t)r.head * a.D) {
    const int row = 32 * (int)wave + (int)(lane & 31);
    uint32_t g;
    const uint32_t ahead = r.token(row, a, &g);
    t = row < r.rows ? r.t0 + (int)ahead : -1;
    head = r.head * a.G + (int)g;
  }
  __device__ __forceinline__ int64_t token() const { return r.base + (t < 0 ? 0 : t); }
  // A row of queries, or of gradients.
  template <int kD>
  __device__ __forceinline__ void load(u32x4 (&to)[kD / 16], const uint16_t* from, int64_t ld, const WindowArgs& a) const {
    load_row<kD>(to, from + token() * ld + (int64_t)head * a.D, t >= 0, a.D, h);
  }
  // Tile i's keys and values into LDS.
  template <int kD>
  __device__ __forceinline__ void fetch(uint16_t* keys_to, uint16_t* values_to, const Afresh& at, int i,
                                        const WindowArgs& a) const {
    const Pieces<kD, kKeys, kThreads> pieces(at.thread);
    const uint32_t k_at = pieces.offset(a.ldk, a.D), v_at = pieces.offset(a.ldv, a.D);
#pragma unroll
    for (int n = 0; n < pieces.kMoves; ++n) {
      fetch_keys(pieces, n, keys_to, k0, a.ldk, keys, i, a.D, k_at, wave);
      fetch_keys(pieces, n, values_to, v0, a.ldv, keys, i, a.D, v_at, wave);
    }
  }
};

// Half a tile of scores (or of products with values): the half's rows times a lane's row.
template <typename T, int kD>
__device__ __forceinline__ f32x16 products(lds_bytes half, const u32x4 (&row)[kD / 16], uint32_t lane) {
  const RowReader<kD> rows(lane);
  f32x16 s = f32x16{};
#pragma unroll
  for (int x = 0; x < kD / 16; ++x) s = product<T>(rows(half, 0, x), row[x], s);
  return s;
}
// An accumulator's rows, rounded, times the columns of half a tile.
template <typename T, int kD>
__device__ __forceinline__ void add_columns(f32x16 (&to)[kD / 32], lds_bytes half, const f32x16& v, uint32_t lane) {
  const ColumnReader<kD> columns(lane);
  const u32x4 p[2] = {operand<T>(v, 0), operand<T>(v, 1)};
#pragma unroll
  for (int x = 0; x < kD / 16; ++x) {
    const int dt = x % (kD / 32);
    const uint32_t at = (uint32_t)(uintptr_t)half + x / (kD / 32) * 16 * kD * 2;
    to[dt] = product<T>(lds_read_turned(at + columns.at[0][dt], at + columns.at[1][dt]), p[x / (kD / 32)], to[dt]);
  }
}

// The forward's columns in `again`: the weights, as they are known now (lse: of 2), times values
// that are finite.
template <typename T, int kD>
__device__ __forceinline__ void make_rows_again(const WindowArgs& a, uint16_t (*lds)[kKeys * kD], const Again& again,
                                                float lse) {
  const Afresh at;
  const OwnRow own(a, at);
  u32x4 q[kD / 16];
  own.load<kD>(q, a.q, a.ldq, a);
  const float c = a.scale * kLog2e;
  f32x16 o[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) o[dt] = f32x16{};
#pragma unroll 1
  for (int i = 0; i < own.keys.n; ++i) {
    own.fetch<kD>(lds[0], lds[1], at, i, a);
    meet();
    make_finite<T, kD, kKeys, kThreads>(lds[1]);
    meet();
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      f32x16 s = products<T, kD>(lds_of(lds[0]) + u * kKeys * kD, q, own.lane);
      keep_seen(s, own.t, own.keys.start(i) + 32 * u + 4 * (int)own.h, own.keys.end(i), a.W, own.keys.below(i, a.S), -INFINITY);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, kWeightsUp<T> - lse));
      add_columns<T, kD>(o, lds_of(lds[1]) + u * kKeys * kD, s, own.lane);
    }
    meet();
  }
  uint16_t* const mine = lds[0] + own.wave * 32 * kD;
  put_rows<T, kD>(mine, o, __builtin_amdgcn_ldexpf(1.0f, -(int)kWeightsUp<T>), own.lane);
  between_lanes();
  again.template put<kD>(mine, [&](int x) {
    return a.out + __shfl(own.token(), x) * a.ldout + (int64_t)__shfl(own.head, x) * a.D;
  });
}

template <typename T, int kD>
__global__ __launch_bounds__(kThreads, 2) void window_fwd_kernel(WindowArgs a) {
  // keys of two tiles; values of three, since a tile's are read out half a tile after its keys
  __shared__ __attribute__((aligned(16))) uint16_t lds[5][kKeys * kD];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l = lane & 31, h = lane >> 5;
  RowTile r;
  if (!row_tile(a, blockIdx.x, &r)) return;
  const int row = 32 * wave + l;
  uint32_t g;
  const uint32_t dt_ = r.token(row, a, &g);
  const bool there = row < r.rows;
  const int t = there ? r.t0 + (int)dt_ : -1;  // -1 sees nothing
  uint32_t g_last;
  const int first = r.t0, last = r.t0 + (int)r.token(r.rows - 1, a, &g_last);
  const int head = r.head * a.G + (int)g;
  u32x4 q[kD / 16];
  const KeyTiles keys(first, last, a.W, a.S);
  const Pieces<kD, kKeys, kThreads> pieces(threadIdx.x);
  const uint32_t k_at = pieces.offset(a.ldk, a.D), v_at = pieces.offset(a.ldv, a.D);
  const RowReader<kD> rows(lane);
  const ColumnReader<kD> columns(lane);
  const float c = a.scale * kLog2e;
  f32x16 o[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) o[dt] = f32x16{};
  float m = -INFINITY, sum = 0.0f;
  // the x-th of a tile's loads, keys and values in turn (behind the last tile: zeros)
  constexpr int kLoads = 2 * pieces.kMoves;
  // (sinks and window meet in one of the first two, if at all)
  static_assert(ENGRAM_WINDOW_SINKS_MAX <= 2 * kKeys, "");
  const uint16_t* const k0 = a.k + r.base * a.ldk + (int64_t)r.head * a.D;
  const uint16_t* const v0 = a.v + r.base * a.ldv + (int64_t)r.head * a.D;
  const auto fetch_first = [&](int x, int i) {
    if (x % 2 == 0) fetch_keys(pieces, x / 2, lds[i], k0, a.ldk, keys, i, a.D, k_at, wave);
    else fetch_keys(pieces, x / 2, lds[2 + i], v0, a.ldv, keys, i, a.D, v_at, wave);
  };
  Following<Pieces<kD, kKeys, kThreads>> next_k(pieces, k0, a.ldk, keys, 2, a.D), next_v(pieces, v0, a.ldv, keys, 2, a.D);
  const auto whole = keys.whole(first, last, a.W);
  // Operands on their way from LDS: of the next half's scores, and of this half's values.
  constexpr int kX = kD / 16;  // products of a half's scores, and of its values
  u32x4 kf[kX], vf[kX];
  // Tile i's keys lie in place i % 2, its values in place i % 3; the loop goes round
  // both in six steps, so that an operand's place is a constant behind an address
  // that stays in a register.
  constexpr int kRound = 6, kTile = kKeys * kD * 2;
  uint32_t k_from[kX], v_from[2][kD / 32];
#pragma unroll
  for (int x = 0; x < kX; ++x) {
    k_from[x] = (uint32_t)(uintptr_t)lds_of(lds[0]) + rows.at + ((32 * x) ^ rows.swap);
    asm volatile("" : "+v"(k_from[x]));  // or it takes a register for each sum with a constant
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt) {
      v_from[n][dt] = (uint32_t)(uintptr_t)lds_of(lds[2]) + columns.at[n][dt];
      asm volatile("" : "+v"(v_from[n][dt]));
    }
  const auto read_keys = [&](int slot, int u, int x) {
    kf[x] = lds_read(k_from[x] + slot % 2 * kTile + u * kTile / 2);
  };
  const auto read_values = [&](int slot, int u, int x) {
    const uint32_t at = slot % 3 * kTile + (u * 2 + x / (kD / 32)) * kTile / 4;
    vf[x] = lds_read_turned(v_from[0][x % (kD / 32)] + at, v_from[1][x % (kD / 32)] + at);
  };
  const auto largest = [&](const f32x16& s) {
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
    return top;
  };
  // what rows do not see goes; the maximum, and what there is in its terms
  const auto settle = [&](f32x16& s, float top, int i, int u) {
    if (!whole.has(2 * i + u)) {
      const int start = keys.start(i) + 32 * u, end = keys.end(i), below = keys.below(i, a.S);
      keep_seen(s, t, start + 4 * (int)h, end, a.W, below, -INFINITY);
      top = largest(s);
    }
    if (__any((top - m) * c > kSlack)) {
      top = fmaxf(m, column_max(top));
      const float keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * c);
      sum *= keep;
#pragma unroll
      for (int dt = 0; dt < kD / 32; ++dt) o[dt] *= keep;
      m = top;
    }
  };
  // Half u of tile i, whose scores are in s: first the scores of the next half (if
  // there is one), beside which the weights are made, then the weights times the
  // values, beside which the next scores' maximum is found.  Each product is sent
  // with what goes on beside it, in this order: left to itself the compiler reads
  // each operand just before its product and makes the weights in one go.
  const auto step = [&](f32x16& s, f32x16& next, int i, int slot, auto half, auto more) __attribute__((always_inline)) {
    constexpr int u = decltype(half)::value, kEach = 16 / kX;
    constexpr bool kNext = decltype(more)::value;
    static_assert(kLoads == kX, "a load beside each product");
    float less = m == -INFINITY ? 0.0f : -m * c;
    if constexpr (kTermsUp<T> != 0) less += kTermsUp<T>;
    u32x4 p[2];
    next = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
    const auto weigh = [&](int from, int n) {
#pragma unroll
      for (int e = from; e < from + n; ++e) {
        s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, less));
        if (e > 0) sum += s[e - 1];  // not the one just made, which takes a moment
      }
      if ((from + n) % 8 == 0) p[(from + n) / 8 - 1] = operand<T>(s, (from + n) / 8 - 1);
    };
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      if constexpr (kNext) next = product<T>(kf[x], q[x], next);
      read_values(slot, u, x);
      weigh(x * kEach / 2, kEach / 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (u == 0) meet();  // the next tile is there, and this one's keys are read out, the last one's values too
    const u32x4 words_k = next_k.words(a.D), words_v = next_v.words(a.D);
    if constexpr (u == 0) {
      next_k.go_on();
      next_v.go_on();
    }
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      __builtin_amdgcn_sched_barrier(0);
      o[x % (kD / 32)] = product<T>(vf[x], p[x / (kD / 32)], o[x % (kD / 32)]);
      // (behind the last tile these read what lies there, for no one)
      if constexpr (kNext) read_keys(slot + 1, u, x);
      if constexpr (u == 0) {
        if (x % 2 == 0) load_to_lds(pieces.lds_place(x / 2, lds[slot % 2], wave), words_k, next_k.at[x / 2]);
        else load_to_lds(pieces.lds_place(x / 2, lds[2 + (slot + 2) % 3], wave), words_v, next_v.at[x / 2]);
      }
      if (x < kX / 2) weigh(8 + x * kEach, kEach);
      if (x == kX / 2) sum += s[15];
      if (kNext && x >= kX / 2) {
#pragma unroll
        for (int e = (x - kX / 2) * 2 * kEach; e < (x - kX / 2 + 1) * 2 * kEach; ++e) top = fmaxf(top, next[e]);
      }
    }
    asm volatile("" : "+v"(sum), "+v"(top));  // or they move behind the branches, away from the products
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kNext) settle(next, top, i + u, 1 - u);
  };
  constexpr auto first_half = std::integral_constant<int, 0>{};
  constexpr auto second_half = std::integral_constant<int, 1>{};
  // the queries through LDS, whole rows: a wave's own, where the second tile's values come later
  {
    const uint16_t* mine = lds[3] + wave * 32 * kD;
    const Pieces<kD, 32, 64> whole(lane);
    whole.gather(mine, a.q + (r.base + r.t0) * a.ldq + (int64_t)r.head * a.G * a.D, a.D, 0, [&](uint32_t row) {
      uint32_t g;
      const uint32_t t = r.token(32 * wave + row, a, &g);
      return (int)(32 * wave + row) < r.rows ? t * (uint32_t)(a.ldq * 2) + g * (uint32_t)(a.D * 2) : kBeyond;
    });
#pragma unroll
    for (int x = 0; x < kLoads; ++x) fetch_first(x, 0);
#pragma unroll
    for (int x = 0; x < kLoads; x += 2) fetch_first(x, 1);
    meet();
#pragma unroll
    for (int x = 0; x < kX; ++x) q[x] = rows(lds_of(mine), 0, x);
    meet();
#pragma unroll
    for (int x = 1; x < kLoads; x += 2) fetch_first(x, 1);
  }
  f32x16 s0 = f32x16{}, s1;
#pragma unroll
  for (int x = 0; x < kX; ++x) s0 = product<T>(rows(lds_of(lds[0]), 0, x), q[x], s0);
#pragma unroll
  for (int x = 0; x < kX; ++x) read_keys(0, 1, x);
  settle(s0, largest(s0), 0, 0);
  for (int i = 0; i < keys.n;) {
#pragma unroll
    for (int slot = 0; slot < kRound; ++slot) {
      step(s0, s1, i, slot, first_half, std::true_type{});
      if (++i >= keys.n) break;
      step(s1, s0, i - 1, slot, second_half, std::true_type{});
    }
  }
  step(s1, s0, keys.n - 1, (keys.n - 1) % kRound, second_half, std::false_type{});
  sum = column_sum(sum);
  const float inverse = 1.0f / sum;
  if (a.lse && there && h == 0) {
    const float one = kTermsUp<T> == 0 ? sum : __builtin_amdgcn_ldexpf(sum, -(int)kTermsUp<T>);
    a.lse[(r.base + t) * (int64_t)(a.Hk * a.G) + head] = fmaf(m, c, __log2f(one)) * kLn2;
  }

  meet();  // the tiles are read out, and what was fetched behind the last one is there
  uint16_t* mine = lds[0] + wave * 32 * kD;
  put_rows<T, kD>(mine, o, inverse, lane);
  // rows that are not finite though their weights are
  const uint64_t redo = __ballot(there && !finite_rows<kD>(o) && fabsf(m) < INFINITY && sum < INFINITY);
  const uint32_t bad = (uint32_t)redo | (uint32_t)(redo >> 32);
  between_lanes();
  Again again;
  if (bad) again = rows_again<T, kD>(bad, mine, v0, a.ldv, t, __shfl(t, 0), __shfl(t, wave_rows(r, wave) - 1), a);
  store_rows<kD>(mine, r, wave, lane, a);
  if (!any_wave<kWaves>(lds[4], again.any())) return;
  make_rows_again<T, kD>(a, lds, again, fmaf(m, c, __log2f(sum)) - kTermsUp<T>);
}

// dq's columns in `again`: d of what is seen alone, times keys that are finite; half a tile at a time.
template <typename T, int kD>
__device__ __forceinline__ void make_dq_again(const WindowArgs& a, uint16_t (*lds)[kKeys * kD], const Again& again, float lse,
                                              float delta) {
  const Afresh at;
  const OwnRow own(a, at);
  u32x4 q[kD / 16], go[kD / 16];
  own.load<kD>(q, a.q, a.ldq, a);
  own.load<kD>(go, a.grad_o, a.ldgo, a);
  const float c = a.scale * kLog2e;
  constexpr bool kHalf = __is_same(T, _Float16);
  float up = kHalf ? kUp : 0.0f;
  f32x16 dq[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) dq[dt] = f32x16{};
#pragma unroll 1
  for (int n = 0; n < 2 * own.keys.n; ++n) {
    const int i = n / 2, u = n % 2;
    own.fetch<kD>(lds[0], lds[1], at, i, a);
    meet();
    const f32x16 s = products<T, kD>(lds_of(lds[0]) + u * kKeys * kD, q, own.lane);
    f32x16 d = products<T, kD>(lds_of(lds[1]) + u * kKeys * kD, go, own.lane);
#pragma unroll
    for (int e = 0; e < 16; ++e) d[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, kHalf ? up - lse : -lse)) * (d[e] - delta);
    keep_seen(d, own.t, own.keys.start(i) + 32 * u + 4 * (int)own.h, own.keys.end(i), a.W, own.keys.below(i, a.S), 0.0f);
    if constexpr (kHalf) keep_in_range<kD>(d, dq, up);
    meet();
    make_finite<T, kD, kKeys, kThreads>(lds[0]);
    meet();
    add_columns<T, kD>(dq, lds_of(lds[0]) + u * kKeys * kD, d, own.lane);
    meet();
  }
  uint16_t* const mine = lds[0] + own.wave * 32 * kD;
  put_rows<T, kD>(mine, dq, kHalf ? a.scale * __builtin_amdgcn_ldexpf(1.0f, -(int)up) : a.scale, own.lane);
  between_lanes();
  again.template put<kD>(mine, [&](int x) {
    return a.out + __shfl(own.token(), x) * a.ldout + (int64_t)__shfl(own.head, x) * a.D;
  });
}

// dq of 128 rows, and delta.  Half a tile at a time: its scores, its values times the
// rows of grad_o, beside which the weights are made, and d times its keys.  Each
// operand is read four products ahead.
template <typename T, int kD>
__global__ __launch_bounds__(kThreads, 2) void window_dq_kernel(WindowArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][2][kKeys * kD];  // [turn][keys, values]
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l = lane & 31, h = lane >> 5;
  RowTile r;
  if (!row_tile(a, blockIdx.x, &r)) return;
  const int row = 32 * wave + l;
  uint32_t g, g_last;
  const uint32_t ahead = r.token(row, a, &g);
  const bool there = row < r.rows;
  const int t = there ? r.t0 + (int)ahead : -1;  // -1 sees nothing
  const int first = r.t0, last = r.t0 + (int)r.token(r.rows - 1, a, &g_last);
  const int head = r.head * a.G + (int)g;
  const int64_t token = r.base + (there ? t : 0), at_head = token * (a.Hk * a.G) + head;
  const KeyTiles keys(first, last, a.W, a.S);
  const Pieces<kD, kKeys, kThreads> pieces(threadIdx.x);
  const uint32_t k_at = pieces.offset(a.ldk, a.D), v_at = pieces.offset(a.ldv, a.D);
  const uint16_t* const k0 = a.k + r.base * a.ldk + (int64_t)r.head * a.D;
  const uint16_t* const v0 = a.v + r.base * a.ldv + (int64_t)r.head * a.D;
  const auto fetch = [&](int i, int slot) {
#pragma unroll
    for (int q = 0; q < pieces.kMoves; ++q) {
      fetch_keys(pieces, q, lds[slot][0], k0, a.ldk, keys, i, a.D, k_at, wave);
      fetch_keys(pieces, q, lds[slot][1], v0, a.ldv, keys, i, a.D, v_at, wave);
    }
  };
  // (the first tiles before the rows, whose loads are many)
  fetch(0, 0);
  if (keys.n > 1) fetch(1, 1);
  u32x4 q[kD / 16], go[kD / 16];
  load_row<kD>(q, a.q + token * a.ldq + (int64_t)head * a.D, there, a.D, h);
  load_row<kD>(go, a.grad_o + token * a.ldgo + (int64_t)head * a.D, there, a.D, h);
  const float lse = there ? a.lse_in[at_head] * kLog2e : 0.0f;
  float delta = 0.0f;
  {
    u32x4 o[kD / 16];
    load_row<kD>(o, a.o + token * a.ldo + (int64_t)head * a.D, there, a.D, h);
#pragma unroll
    for (int kk = 0; kk < kD / 16; ++kk) delta += dot8<T>(go[kk], o[kk]);
    delta = column_sum(delta);
  }
  const RowReader<kD> rows(lane);
  const ColumnReader<kD> columns(lane);
  const float c = a.scale * kLog2e;
  constexpr bool kHalf = __is_same(T, _Float16);
  float up = kHalf ? kUp : 0.0f;
  f32x16 dq[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) dq[dt] = f32x16{};
  // Places as constants behind addresses that stay in registers, as in the forward; they go
  // to and fro between the two tiles' places.
  constexpr int kX = kD / 16, kEach = 16 / kX, kRing = 4, kTile = kKeys * kD * 2;
  uint32_t by_row[kX], by_column[2][kD / 32];
#pragma unroll
  for (int x = 0; x < kX; ++x) {
    by_row[x] = (uint32_t)(uintptr_t)lds_of(lds[0][0]) + rows.at + ((32 * x) ^ rows.swap);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt) {
      by_column[n][dt] = (uint32_t)(uintptr_t)lds_of(lds[0][0]) + columns.at[n][dt];
    }
  Following<Pieces<kD, kKeys, kThreads>> next_k(pieces, k0, a.ldk, keys, 2, a.D), next_v(pieces, v0, a.ldv, keys, 2, a.D);
  const auto whole = keys.whole(first, last, a.W);
  // Where rows see few keys, do . o is not exact enough: the rounding of o is large
  // against what is left of do . v - delta (sequences of 10 tokens, fp16: it alone moves
  // the gradients by 6e-4 to 9e-4 of their norms; they are off by 3e-4 in all with
  // delta as the weights' mean of do . v).  Where they see many it adds little
  // (window 1024, bf16: 2.5e-3 for 2.3e-3), and two more products for each key would
  // cost a third of the call; here they cost a seventh (10496 tokens, window 48: 237 us, 201 without).
  if (keys.n <= 2) {
    meet();
    float weights = 0.0f, mean = 0.0f;
#pragma unroll 1
    for (int half = 0; half < 2 * keys.n; ++half) {
      const int n = half / 2, u = half % 2;
      const lds_bytes tk = lds_of(lds[n][0]) + u * kTile / 2, tv = lds_of(lds[n][1]) + u * kTile / 2;
      f32x16 s = f32x16{}, d = f32x16{};
#pragma unroll
      for (int x = 0; x < kX; ++x) s = product<T>(rows(tk, 0, x), q[x], s);
#pragma unroll
      for (int x = 0; x < kX; ++x) d = product<T>(rows(tv, 0, x), go[x], d);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lse));
      const int start = keys.start(n) + 32 * u + 4 * (int)h;
      keep_seen(s, t, start, keys.end(n), a.W, keys.below(n, a.S), 0.0f);
      keep_seen(d, t, start, keys.end(n), a.W, keys.below(n, a.S), 0.0f);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        weights += s[e];
        mean = fmaf(s[e], d[e], mean);
      }
    }
    weights = column_sum(weights);
    mean = column_sum(mean);
    // (where the weights do not add up to 1, lse is of other keys, or not finite)
    if (fabsf(weights - 1.0f) <= 0x1p-12f && fabsf(mean) < INFINITY) delta = mean / weights;
  }
  if (there && h == 0) a.delta[at_head] = delta;
  for (int i = 0; i < keys.n; ++i) {
    meet();
    if (i > 0 && i + 1 < keys.n) {
      const u32x4 words_k = next_k.words(a.D), words_v = next_v.words(a.D);
#pragma unroll
      for (int q = 0; q < pieces.kMoves; ++q) {
        load_to_lds(pieces.lds_place(q, lds[(i + 1) & 1][0], wave), words_k, next_k.at[q]);
        load_to_lds(pieces.lds_place(q, lds[(i + 1) & 1][1], wave), words_v, next_v.at[q]);
      }
      next_k.go_on();
      next_v.go_on();
    }
#pragma unroll
    for (int x = 0; x < kX; ++x) asm volatile("" : "+v"(by_row[x]), "+v"(by_column[x / (kD / 32)][x % (kD / 32)]));
    u32x4 f[kRing];
    // the n-th operand of the tile
    const auto read = [&](int n) {
      if (n >= 6 * kX) return;
      const int u = n / (3 * kX), side = n / kX % 3, x = n % kX;
      if (side < 2) {
        f[n % kRing] = lds_read(by_row[x] + side * kTile + u * kTile / 2);
      } else {
        const uint32_t at = (u * 2 + x / (kD / 32)) * kTile / 4;
        f[n % kRing] = lds_read_turned(by_column[0][x % (kD / 32)] + at, by_column[1][x % (kD / 32)] + at);
      }
    };
#pragma unroll
    for (int n = 0; n < kRing; ++n) read(n);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = u * 3 * kX;
      const float less = kHalf ? up - lse : -lse;  // (s is there for d alone)
      f32x16 s = f32x16{}, d = f32x16{};
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        __builtin_amdgcn_sched_barrier(0);
        s = product<T>(f[x % kRing], q[x], s);
        read(at + x + kRing);
      }
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        __builtin_amdgcn_sched_barrier(0);
        d = product<T>(f[x % kRing], go[x], d);
        read(at + kX + x + kRing);
#pragma unroll
        for (int m = x * kEach; m < (x + 1) * kEach; ++m) s[m] = __builtin_amdgcn_exp2f(fmaf(s[m], c, less));
      }
      asm volatile("" : "+v"(s));  // or it moves behind the branch, away from the products
      __builtin_amdgcn_sched_barrier(0);
      if (!whole.has(2 * i + u))
        keep_seen(s, t, keys.start(i) + 32 * u + 4 * (int)h, keys.end(i), a.W, keys.below(i, a.S), 0.0f);
      u32x4 e[2];
      const auto differ = [&](int from, int n) {
#pragma unroll
        for (int m = from; m < from + n; ++m) d[m] = s[m] * (d[m] - delta);
        if ((from + n) % 8 == 0) e[(from + n) / 8 - 1] = operand<T>(d, (from + n) / 8 - 1);
      };
      if constexpr (kHalf) {
#pragma unroll
        for (int m = 0; m < 16; ++m) d[m] = s[m] * (d[m] - delta);
        keep_in_range<kD>(d, dq, up);
        e[0] = operand<T>(d, 0);
        e[1] = operand<T>(d, 1);
      } else {
        differ(0, 8);
      }
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        __builtin_amdgcn_sched_barrier(0);
        dq[x % (kD / 32)] = product<T>(f[x % kRing], e[x / (kD / 32)], dq[x % (kD / 32)]);
        read(at + 2 * kX + x + kRing);
        if (!kHalf && x < kX / 2) differ(8 + x * kEach, kEach);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t turn = i & 1 ? -2 * kTile : 2 * kTile;
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      by_row[x] += turn;
      by_column[x / (kD / 32)][x % (kD / 32)] += turn;
    }
  }

  __syncthreads();  // the tiles are read out
  uint16_t* mine = lds[0][0] + wave * 32 * kD;
  put_rows<T, kD>(mine, dq, kHalf ? a.scale * __builtin_amdgcn_ldexpf(1.0f, -(int)up) : a.scale, lane);
  const uint64_t redo = __ballot(there && !finite_rows<kD>(dq) && fabsf(lse) < INFINITY && fabsf(delta) < INFINITY);
  const uint32_t bad = (uint32_t)redo | (uint32_t)(redo >> 32);
  between_lanes();
  Again again;
  if (bad) again = rows_again<T, kD>(bad, mine, k0, a.ldk, t, __shfl(t, 0), __shfl(t, wave_rows(r, wave) - 1), a);
  store_rows<kD>(mine, r, wave, lane, a);
  if (!any_wave<kWaves>(lds[1][0], again.any())) return;
  make_dq_again<T, kD>(a, lds[0], again, lse, delta);
}

// The sinks' sums, fp32 and unscaled: [piece][key head][dk, dv][S][D], a piece for
// each of the rows that see them as sinks, and then one a sequence for the rows whose
// window they are in.
__device__ __forceinline__ float* piece_sums(const WindowArgs& a, int64_t piece, int head, int which) {
  return a.sums + ((piece * a.Hk + head) * 2 + which) * a.S * a.D;
}

// The columns of dk (which: 0) or dv (1) that rows of the tokens from .. to - 1 leave not finite in
// all tokens that they see, beside those in `found`, and as far as `wanted` asks; bits as those of
// columns_not_finite.  A NaN or -infinite lse makes a row's weights NaN or infinite; an
// infinite or NaN value in grad_o always makes delta so, delta d, and d all of dk; dv takes
// it as it is.
template <typename T, int kD>
__device__ __forceinline__ uint32_t columns_lost(const WindowArgs& a, int64_t base, int head, int from, int to, int which,
                                                 uint32_t wanted, uint32_t found) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 63, Hq = a.Hk * a.G;
  const int last = to * a.G;  // N * Hq is below 2^30
  for (int i = from * a.G; i < last && __any(wanted & ~found); i += 64 * kAhead) {
    float lse[kAhead], delta[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int at = i + 64 * n + lane;
      const int64_t row = at < last ? (base + at / a.G) * Hq + head * a.G + at % a.G : 0;
      lse[n] = at < last ? a.lse_in[row] : 0.0f;
      delta[n] = at < last ? a.delta[row] : 0.0f;
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const bool off = !(fabsf(delta[n]) < INFINITY);
      if (__any(!(lse[n] > -INFINITY) || (which == 0 && off))) return 0xff;
      const int at = i + 64 * n;
      if (__any(off))
        found = columns_not_finite<T, kD>(at, at + 64 < last ? at + 64 : last, a.D, wanted, found, [&](int x) {
          return a.grad_o + (base + x / a.G) * a.ldgo + (int64_t)(head * a.G + x % a.G) * a.D;
        });
    }
  }
  return found;
}

// Whether dk of a token is lost by its value, which is part of every d.
template <typename T>
__device__ __forceinline__ bool lost_by_value(const WindowArgs& a, int64_t base, int head, int j) {
  const int lane = threadIdx.x & 63;
  const uint16_t* v = a.v + (base + j) * a.ldv + (int64_t)head * a.D;
  bool off = false;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 64 * e < a.D) off |= not_finite<T>(v[lane + 64 * e]) != 0;
  return __any(off);
}

// Of a wave's 32 keys from key0 on, in `bad`, whose dk or dv lies in LDS and is not finite, the
// columns that are to be made again, as rows_again: `low(j)` .. `high(j)` - 1 are the tokens
// whose rows' part of key j is in question, both rising with j.
template <typename T, int kD, typename Low, typename High>
__device__ __forceinline__ Again keys_again(uint32_t bad, const uint16_t* mine, const WindowArgs& a, int64_t base, int head,
                                            int key0, int which, Low low, High high) {
  uint32_t wanted = 0;
  for (uint32_t left = bad; left; left &= left - 1) wanted |= columns_lost<T, kD>(mine, __builtin_ctz(left), a.D);
  // the tokens that all of the keys have
  const int begin = low(key0 + 31), most = high(key0), end = most > begin ? most : begin;
  const uint32_t common = columns_lost<T, kD>(a, base, head, begin, end, which, wanted, 0);
  Again again;
  for (uint32_t left = bad; left; left &= left - 1) {
    const int x = __builtin_ctz(left), j = key0 + x, from = low(j), to = high(j);
    const uint32_t need = columns_lost<T, kD>(mine, x, a.D);
    if (which == 0 && from < to && lost_by_value<T>(a, base, head, j)) continue;
    uint32_t found = columns_lost<T, kD>(a, base, head, from, begin < to ? begin : to, which, need, common);
    found = columns_lost<T, kD>(a, base, head, end > from ? end : from, to, which, need, found);
    again.add<kD>(x, need & ~found);
  }
  return again;
}

// A workgroup's keys of a sequence and key head, and the rows whose part of their dk and dv it makes.
struct KeyTile {
  bool sinks;
  int id, b, head, length;
  int64_t base;    // the sequence's first token
  int k0, keys;    // the first key; keys of the sequence, as far as they matter here
  int from, to;    // the rows' tokens
  int near, span;  // how far behind a key those lie that see it: `near` on, fewer than `span` further
  __device__ __forceinline__ bool find(const WindowArgs& a, int block) {
    const int wide_blocks = (int)gridDim.x - a.sink_blocks;
    sinks = block >= wide_blocks;
    const int at = sinks ? block - wide_blocks : neighbours(block, wide_blocks);
    const int per_head = sinks ? a.sink_blocks / a.Hk : a.tiles;
    id = at % per_head;
    head = at / per_head;
    const uint32_t unit = sinks ? (uint32_t)a.piece : (uint32_t)kRows;
    const Sequence seq(a, id, 1, unit);
    const int64_t tile = seq.tile;
    b = seq.b;
    base = seq.start;
    length = (int)seq.length;
    if (tile < 0 || length <= 0 || tile * unit >= length) return false;
    k0 = sinks ? 0 : (int)tile * kRows;
    from = k0;
    to = k0 + kRows - 1 + a.W;
    near = sinks ? a.W : 0;
    if (sinks) {
      from = (int)tile * a.piece > a.W ? (int)tile * a.piece : a.W;
      to = ((int)tile + 1) * a.piece;
    }
    if (to > length) to = length;
    keys = sinks ? (a.S < length ? a.S : length) : length;
    span = sinks ? length : a.W;
    return from < to;  // else no row of the piece sees a sink as one
  }
  // Keys and values of 128 tokens into LDS, values first.
  template <int kD>
  __device__ __forceinline__ void fetch(uint16_t* lds, uint32_t thread, uint32_t wave, const WindowArgs& a) const {
    const Pieces<kD, kRows, 512> wide(thread);
    const int n = keys - k0 < kRows ? keys - k0 : kRows;
    wide.fetch(lds, a.v + (base + k0) * a.ldv + (int64_t)head * a.D, a.ldv, n, a.D, wide.offset(a.ldv, a.D), wave);
    wide.fetch(lds + kRows * kD, a.k + (base + k0) * a.ldk + (int64_t)head * a.D, a.ldk, n, a.D, wide.offset(a.ldk, a.D), wave);
  }
  // Sinks that rows behind their window see too have their sums in fp32, joined by the next launch.
  __device__ __forceinline__ bool part(const WindowArgs& a, int key) const { return sinks || (key < a.S && length > a.W); }
  __device__ __forceinline__ float* to_part(const WindowArgs& a, int key, int which) const {
    return piece_sums(a, sinks ? id : a.pieces + b, head, which) + (int64_t)key * a.D;
  }
  __device__ __forceinline__ uint16_t* out(const WindowArgs& a, int key, int which) const {
    return (which ? a.grad_v + (base + key) * a.ldgv : a.grad_k + (base + key) * a.ldgk) + (int64_t)head * a.D;
  }
  // Keys before this one are the next launch's.
  __device__ __forceinline__ int done(const WindowArgs& a) const { return length > a.W ? a.S : 0; }
  // The tokens whose rows see key j, of those that are looked at here: low(j) .. high(j) - 1.
  __device__ __forceinline__ int low(int j) const {
    const int x = j + near < to ? j + near : to;
    return x > from ? x : from;
  }
  __device__ __forceinline__ int high(int j) const { return to - j < span ? to : j + span; }
};

// The two halves of the rows that two waves have had for the same keys, joined: the first four
// waves then have dk, the others dv.
template <typename T, int kD>
__device__ __forceinline__ void join_halves(f32x16 (&sum)[kD / 32], f32x16 (&dk)[kD / 32], f32x16 (&dv)[kD / 32], float up,
                                            uint16_t* lds, uint32_t lane, uint32_t wave) {
  const uint32_t quarter = wave & 3, half = wave >> 2;
  if constexpr (__is_same(T, _Float16)) {
    const float lowered = __builtin_amdgcn_ldexpf(1.0f, -(int)up);
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt) {
      dk[dt] *= lowered;
      dv[dt] *= __builtin_amdgcn_ldexpf(1.0f, -(int)kWeightsUp<T>);
    }
  }
  // The exchange: the first four waves' dv, then the others' dk, in the order they
  // are there for each lane.
  f32x4* const given = reinterpret_cast<f32x4*>(lds) + quarter * (kD / 8) * 64 + lane;
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    if (half == (uint32_t)turn) {
#pragma unroll
      for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x16& x = turn ? dk[dt] : dv[dt];
          given[(dt * 4 + j) * 64] = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
        }
    }
    __syncthreads();
    if (half != (uint32_t)turn) {
#pragma unroll
      for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 x = given[(dt * 4 + j) * 64];
          f32x16& to = turn ? dk[dt] : dv[dt];
#pragma unroll
          for (int e = 0; e < 4; ++e) to[4 * j + e] += x[e];
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) sum[dt] = half ? dv[dt] : dk[dt];
}

constexpr int kKeyWaves = 8, kKeyThreads = kKeyWaves * 64;

// The columns in `again` of dk (the first four waves) and dv: weights and d of what is seen
// alone, times queries and gradients that are finite.  LDS as the kernel has it.
template <typename T, int kD>
__device__ __forceinline__ void make_keys_again(const WindowArgs& a, uint16_t* lds, float* lses, float* deltas,
                                                const Again& again) {
  const Afresh afresh;
  const uint32_t lane = afresh.thread & 63, wave = __builtin_amdgcn_readfirstlane(afresh.thread >> 6);
  const uint32_t l = lane & 31, h = lane >> 5, quarter = wave & 3, half = wave >> 2;
  KeyTile kt;
  kt.find(a, afresh.block);
  const int key0 = kt.k0 + 32 * (int)quarter, key = key0 + (int)l, which = (int)half;
  const bool there = key < kt.keys;
  uint16_t *const tq = lds + 2 * kRows * kD, *const tg = tq + kKeys * kD;
  const float c = a.scale * kLog2e;
  constexpr bool kHalf = __is_same(T, _Float16);
  float up = kHalf ? kUp : 0.0f;
  f32x16 dk[kD / 32], dv[kD / 32], sum[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) dk[dt] = dv[dt] = f32x16{};
  __syncthreads();  // all waves have their rows out of LDS, and know that they are here
  kt.fetch<kD>(lds, afresh.thread, wave, a);
  const Pieces<kD, kKeys, kKeyThreads> pieces(afresh.thread);
  const int64_t of_head = (int64_t)kt.head * a.G * a.D;
  const int all = (kt.to - kt.from) * a.G;  // rows: N * Hq is below 2^30
#pragma unroll 1
  for (int i = 0; i * kKeys < all; ++i) {
    const int t0 = kt.from + i * kKeys / a.G, x0 = i * kKeys % a.G;  // the first row's
    const int64_t first = kt.base + t0;
#pragma unroll
    for (int j = 0; j < pieces.kMoves; ++j) {
      const int row = (int)pieces.row + j * pieces.kStep;
      const uint32_t t = a.by_G(x0 + row), g = x0 + row - t * a.G;
      const bool in = i * kKeys + row < all && pieces.col < (uint32_t)a.D;
      const uint32_t at = g * (uint32_t)(a.D * 2) + pieces.col * 2;
      load_to_lds(pieces.lds_place(j, tq, wave), buffer_words(a.q + first * a.ldq + of_head),
                  in ? at + t * (uint32_t)(a.ldq * 2) : kBeyond);
      load_to_lds(pieces.lds_place(j, tg, wave), buffer_words(a.grad_o + first * a.ldgo + of_head),
                  in ? at + t * (uint32_t)(a.ldgo * 2) : kBeyond);
    }
    if (wave == 0) {
      const bool in = i * kKeys + (int)lane < all;
      const uint32_t t = a.by_G(x0 + lane), g = x0 + lane - t * a.G;
      const int64_t at = in ? (first + t) * (a.Hk * a.G) + kt.head * a.G + g : 0;
      lses[lane] = in ? fmaf(a.lse_in[at], kLog2e, -kWeightsUp<T>) : INFINITY;
      deltas[lane] = in ? a.delta[at] : 0.0f;
    }
    meet();
    const RowReader<kD> rows(lane);
    const lds_bytes hq = lds_of(tq) + half * kKeys * kD, hg = lds_of(tg) + half * kKeys * kD;
    const lds_bytes hv = lds_of(lds) + quarter * kKeys * kD, hk = hv + kRows * kD * 2;
    f32x16 s = f32x16{}, d = f32x16{};
#pragma unroll
    for (int x = 0; x < kD / 16; ++x) s = product<T>(rows(hq, 0, x), rows(hk, 0, x), s);
#pragma unroll
    for (int x = 0; x < kD / 16; ++x) d = product<T>(rows(hg, 0, x), rows(hv, 0, x), d);
    const float raised = kHalf ? __builtin_amdgcn_ldexpf(1.0f, (int)(up - kWeightsUp<T>)) : 1.0f;
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int row = 32 * (int)half + 8 * (m / 4) + 4 * (int)h + m % 4;
      const int behind = t0 + (int)a.by_G(x0 + row) - key - kt.near;
      // (a row that is not there has an lse of infinity)
      const bool seen = there && (uint32_t)behind < (uint32_t)kt.span && lses[row] != INFINITY;
      const float w = __builtin_amdgcn_exp2f(fmaf(s[m], c, -lses[row]));
      s[m] = seen ? w : 0.0f;
      d[m] = seen ? w * (d[m] - deltas[row]) * raised : 0.0f;
    }
    if constexpr (kHalf) keep_in_range<kD>(d, dk, up);
    meet();
    make_finite<T, kD, 2 * kKeys, kKeyThreads>(tq);  // queries and gradients
    meet();
    add_columns<T, kD>(dk, hq, d, lane);
    add_columns<T, kD>(dv, hg, s, lane);
    meet();
  }
  join_halves<T, kD>(sum, dk, dv, up, lds, lane, wave);
  const bool part = kt.part(a, key);
  float* const to_part = kt.to_part(a, key, which);
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int col = 32 * dt + 8 * (m / 4) + m % 4;  // and 4 h
      const uint32_t lower = __shfl(again.columns[dt / 2], col % 64), upper = __shfl(again.columns[dt / 2], col % 64 + 4);
      if (part && there && ((h ? upper : lower) >> l & 1)) to_part[col + 4 * (int)h] = sum[dt][m];
    }
  uint16_t* const mine = lds + wave * 32 * kD;
  put_rows<T, kD>(mine, sum, which ? 1.0f : a.scale, lane);
  between_lanes();
  if (!kt.sinks)
    again.template put<kD>(mine, [&](int x) { return kt.out(a, key0 + x, which); }, kt.done(a) - key0);
}

// dk and dv of 128 keys, of the rows whose window they are in.  The last
// a.sink_blocks workgroups make the part of the sinks (the first keys of a sequence)
// that comes from the rows of one piece of it that see them as sinks: they are
// short, and so fill the CUs that the last of the others leave free.  Four
// waves have 32 keys each for the first half of a tile of rows, four the same keys for
// the second; at the end they exchange what they have, and the first four leave
// dk, the others dv.  Keys and values stay in LDS: in registers they would leave
// none for operands on their way, and the waits for what is spilled wait for
// the next tile too.
template <typename T, int kD>
__global__ __launch_bounds__(kKeyThreads, 2) void window_dkdv_kernel(WindowArgs a) {
  constexpr int kX = kD / 16;
  // the values and keys; then [turn][queries, gradients of o] of 64 rows; at the end half of it for the exchange
  constexpr int kTile = kKeys * kD;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * kRows * kD + 4 * kTile];
  __shared__ __attribute__((aligned(16))) float lses[2][kKeys], deltas[2][kKeys];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l = lane & 31, h = lane >> 5, quarter = wave & 3, half = wave >> 2;
  KeyTile kt;
  if (!kt.find(a, blockIdx.x)) return;
  const bool sinks = kt.sinks;
  const int64_t base = kt.base;
  const int length = kt.length, head = kt.head, from = kt.from, to = kt.to, near = kt.near, keys = kt.keys;
  const int key0 = kt.k0 + 32 * (int)quarter, key = key0 + (int)l;
  const bool active = key0 < keys, there = key < keys;
  const int span = there ? kt.span : 0;
  kt.fetch<kD>(lds, threadIdx.x, wave, a);
  uint16_t* const tiles = lds + 2 * kRows * kD;

  const Pieces<kD, kKeys, kKeyThreads> pieces(threadIdx.x);
  // Tiles of rows: from the first token that is a multiple of their number on, then what
  // is before it.  Workgroups that run side by side, each 128 keys further, so meet at
  // the same rows at a time, which the XCD's L2 then fetches once for all nine that a window of 1024 reaches.
  const int runs = to - from, ahead = sinks ? 0 : (runs - from % runs) % runs, middle = from + ahead;
  const int n1 = ((to - middle) * a.G + kKeys - 1) / kKeys, n = n1 + (ahead * a.G + kKeys - 1) / kKeys;
  const int Hq = a.Hk * a.G;
  float lse = 0.0f, delta = 0.0f;
  int t0 = middle, behind = to;  // of the next tile to fetch: its first row's token and head, the end of its run
  uint32_t x0 = 0;
  const int64_t of_head = (int64_t)head * a.G * a.D;
  const auto row_at = [&](uint32_t row, uint32_t* t, uint32_t* g) {
    const uint32_t x = x0 + row;
    *t = a.by_G(x);
    *g = x - *t * (uint32_t)a.G;
    return t0 + (int)*t < behind;
  };
  // The j-th pieces of tile i's rows (none behind the last tile: zeros).
  const auto fetch = [&](int i, int j) {
    const int64_t first = base + t0;
    uint32_t t, g;
    const bool in = row_at(pieces.row + j * pieces.kStep, &t, &g) && i < n;
    uint16_t* const to_q = tiles + (i & 1) * 2 * kTile;
    const uint32_t at = in && pieces.col < (uint32_t)a.D ? g * (uint32_t)(a.D * 2) + pieces.col * 2 : kBeyond;
    const uint32_t far = at == kBeyond ? 0 : t;
    static_assert(pieces.kSame, "");
    load_to_lds(pieces.lds_place(j, to_q, wave), buffer_words(a.q + first * a.ldq + of_head), at + far * (uint32_t)(a.ldq * 2));
    load_to_lds(pieces.lds_place(j, to_q + kTile, wave), buffer_words(a.grad_o + first * a.ldgo + of_head),
                at + far * (uint32_t)(a.ldgo * 2));
  };
  // What the first wave keeps of tile i's rows, and on to the next tile.
  const auto fetch_sums = [&](int i) {
    if (wave == 0) {
      uint32_t t, g;
      const bool in = row_at(lane, &t, &g) && i < n;
      const int64_t at = (base + t0 + (in ? t : 0)) * Hq + head * a.G + (in ? g : 0);
      // a row that is not there has weights of 0
      lse = in ? fmaf(a.lse_in[at], kLog2e, -kWeightsUp<T>) : INFINITY;
      delta = in ? a.delta[at] : 0.0f;
    }
    x0 += kKeys;
    t0 += (int)a.by_G(x0);
    x0 -= a.by_G(x0) * (uint32_t)a.G;
    if (i + 1 == n1) {
      t0 = from;
      x0 = 0;
      behind = middle;
    }
  };
  const auto fetch_all = [&](int i) {
#pragma unroll
    for (int j = 0; j < pieces.kMoves; ++j) fetch(i, j);
    fetch_sums(i);
  };
  const RowReader<kD> rows(lane);
  const ColumnReader<kD> columns(lane);
  const float c = a.scale * kLog2e;
  constexpr bool kHalf = __is_same(T, _Float16);
  float up = kHalf ? kUp : 0.0f;
  f32x16 dk[kD / 32], dv[kD / 32];
#pragma unroll
  for (int dt = 0; dt < kD / 32; ++dt) dk[dt] = dv[dt] = f32x16{};
  int t_first = middle;     // of this tile: as t0 and x0
  uint32_t x_first = 0;
  // Places as constants behind addresses that stay in registers and go to and fro
  // between the two tiles' places; those of keys and values in an instruction each.
  constexpr int kBytes = kTile * 2;
  uint32_t by_row[kX], by_column[2][kD / 32];
  const uint32_t of_half = (uint32_t)(uintptr_t)lds_of(tiles) + half * kBytes / 2;
  const uint32_t of_key = (uint32_t)(uintptr_t)lds_of(lds) + rows.at + quarter * kBytes / 2;
#pragma unroll
  for (int x = 0; x < kX; ++x) by_row[x] = of_half + rows.at + ((32 * x) ^ rows.swap);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt) by_column[n][dt] = of_half + columns.at[n][dt];
  fetch_all(0);
  for (int i = 0; i < n; ++i) {
    const uint32_t turn = i == 0 ? 0 : i & 1 ? 2 * kBytes : -2 * kBytes;
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      by_row[x] += turn;
      by_column[x / (kD / 32)][x % (kD / 32)] += turn;
    }
    if (wave == 0) {
      lses[i & 1][lane] = lse;
      deltas[i & 1][lane] = delta;
    }
    meet();
    if (i == n1) {
      t_first = from;
      x_first = 0;
    }
    const uint32_t x = x_first + 32 * half;  // this wave's rows: heads x to x + 31 from token t_first's first on
    const int ta = t_first + (int)a.by_G(x), tb = t_first + (int)a.by_G(x + 31);
    const int t_here = t_first;
    const uint32_t x_here = x;
    x_first += kKeys;
    t_first += (int)a.by_G(x_first);
    x_first -= a.by_G(x_first) * (uint32_t)a.G;
    // rows lie between ta - key0 - 31 and tb - key0 tokens behind the keys
    const int least = ta - key0 - 31, most = tb - key0;
    if (!active || most < near || (!sinks && least >= a.W)) {
      fetch_all(i + 1);
      continue;
    }
    const int r0 = 32 * (int)half;
    // The operands from the tiles of rows, in the order of their products: queries and
    // gradients of o by rows, then gradients and queries by columns; four on their way.
    constexpr int kRing = 4;
    u32x4 f[kRing], kv[kRing], p[2], e[2];
    const auto read = [&](int n) {
      const int x = n % kX, side = n / kX;
      if (side >= 4) return;
      const int tile = side == 0 || side == 3 ? 0 : kBytes;  // queries, gradients
      if (side < 2) {
        f[n % kRing] = lds_read(by_row[x] + tile);
      } else {
        const uint32_t at = tile + x / (kD / 32) * kBytes / 4;
        f[n % kRing] = lds_read_turned(by_column[0][x % (kD / 32)] + at, by_column[1][x % (kD / 32)] + at);
      }
    };
    uint32_t swap = rows.swap;
    asm volatile("" : "+v"(swap));  // or it keeps the addresses for the next tile
    const auto read_key = [&](int n) {
      if (n >= 2 * kX) return;
      kv[n % kRing] = lds_read(of_key + ((32 * (n % kX)) ^ swap) + (n < kX ? kRows * kD * 2 : 0));
    };
    f32x16 s = f32x16{}, d = f32x16{};
    f32x4 row[2];
    const auto read_lse = [&](int j) { row[j & 1] = *reinterpret_cast<const f32x4*>(&lses[i & 1][r0 + 8 * j + 4 * h]); };
    const auto read_delta = [&](int j) { row[j & 1] = *reinterpret_cast<const f32x4*>(&deltas[i & 1][r0 + 8 * j + 4 * h]); };
    constexpr int kEach = 16 / kX;
#pragma unroll
    for (int n = 0; n < kRing; ++n) read(n);
#pragma unroll
    for (int n = 0; n < kRing; ++n) read_key(n);
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      __builtin_amdgcn_sched_barrier(0);
      s = product<T>(f[x % kRing], kv[x % kRing], s);
      read(x + kRing);
      read_key(x + kRing);
      if (x % 2 == 1 && x / 2 < pieces.kMoves) fetch(i + 1, x / 2);
    }
    fetch_sums(i + 1);
    __builtin_amdgcn_sched_barrier(0);
    read_lse(0);
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      __builtin_amdgcn_sched_barrier(0);
      d = product<T>(f[x % kRing], kv[x % kRing], d);
      read(kX + x + kRing);
      read_key(kX + x + kRing);
      if (x * kEach % 4 == 0 && x * kEach < 12) read_lse(x * kEach / 4 + 1);
#pragma unroll
      for (int m = x * kEach; m < (x + 1) * kEach; ++m)
        s[m] = __builtin_amdgcn_exp2f(fmaf(s[m], c, -row[m / 4 & 1][m % 4]));
    }
    asm volatile("" : "+v"(s));  // or the weights move behind the branch, away from the products
    __builtin_amdgcn_sched_barrier(0);
    read_delta(0);
    if (least < near || (!sinks && most >= a.W) || key0 + 31 >= keys) {
      uint32_t xe = x_here + 4 * h;
      asm volatile("" : "+v"(xe));  // or what follows moves in front of the branch
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int behind = t_here + (int)a.by_G(xe + 8 * (m / 4) + m % 4) - key - near;
        s[m] = (uint32_t)behind < (uint32_t)span ? s[m] : 0.0f;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int w = 0; w < 2; ++w) p[w] = operand<T>(s, w);
    const float raised = kHalf ? __builtin_amdgcn_ldexpf(1.0f, (int)(up - kWeightsUp<T>)) : 1.0f;
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      __builtin_amdgcn_sched_barrier(0);
      dv[x % (kD / 32)] = product<T>(f[x % kRing], p[x / (kD / 32)], dv[x % (kD / 32)]);
      read(2 * kX + x + kRing);
      if (x * kEach % 4 == 0 && x * kEach < 12) read_delta(x * kEach / 4 + 1);
#pragma unroll
      for (int m = x * kEach; m < (x + 1) * kEach; ++m) {
        d[m] = s[m] * (d[m] - row[m / 4 & 1][m % 4]);
        if (kHalf) d[m] *= raised;
      }
      if (!kHalf && (x + 1) * kEach % 8 == 0) e[(x + 1) * kEach / 8 - 1] = operand<T>(d, (x + 1) * kEach / 8 - 1);
    }
    if constexpr (kHalf) {
      keep_in_range<kD>(d, dk, up);
      e[0] = operand<T>(d, 0);
      e[1] = operand<T>(d, 1);
    }
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      __builtin_amdgcn_sched_barrier(0);
      dk[x % (kD / 32)] = product<T>(f[x % kRing], e[x / (kD / 32)], dk[x % (kD / 32)]);
      read(3 * kX + x + kRing);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  const int which = (int)half;
  f32x16 sum[kD / 32];
  meet();  // the tiles are read out, and what was fetched behind the last one is there
  join_halves<T, kD>(sum, dk, dv, up, lds, lane, wave);
  if (kt.part(a, key) && there) {
    float* const out = kt.to_part(a, key, which);
#pragma unroll
    for (int dt = 0; dt < kD / 32; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 32 * dt + 8 * j + 4 * (int)h;
        if (col < a.D)
          *reinterpret_cast<f32x4*>(out + col) =
              f32x4{sum[dt][4 * j], sum[dt][4 * j + 1], sum[dt][4 * j + 2], sum[dt][4 * j + 3]};
      }
  }
  uint16_t* const mine = lds + wave * 32 * kD;
  put_rows<T, kD>(mine, sum, which ? 1.0f : a.scale, lane);
  const uint64_t redo = __ballot(there && !finite_rows<kD>(sum));
  const uint32_t bad = (uint32_t)redo | (uint32_t)(redo >> 32);
  between_lanes();
  if (!sinks) {
    const int done = kt.done(a);
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      const uint32_t x = (i * 64 + lane) / (kD / 8), col = (i * 64 + lane) % (kD / 8) * 8;
      const int j = key0 + (int)x;
      if (j >= done && j < length && (int)col < a.D) store16(kt.out(a, j, which) + col, load16(mine + place<kD>(x, col)));
    }
  }
  Again again;
  if (bad)
    again = keys_again<T, kD>(bad, mine, a, base, head, key0, which, [&](int j) { return kt.low(j); },
                              [&](int j) { return kt.high(j); });
  if (any_wave<kKeyWaves>(tiles, again.any())) make_keys_again<T, kD>(a, lds, lses[0], deltas[0], again);
}

// dk and dv of the sinks of sequences longer than the window: a wave for each
// sequence, key head, sink and gradient, a lane's values 2 lane and 2 lane + 1.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void window_sinks_kernel(WindowArgs a) {
  const int lane = threadIdx.x & 63;
  const int which = blockIdx.y & 1, j = (int)blockIdx.y >> 1;
  const int at = blockIdx.x * (kJoinThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = at % a.Hk, b = at / a.Hk;
  if (b >= a.B) return;
  const Sequences seqs{a.cu, a.N, a.B};
  const int64_t base = seqs.start(b), all = seqs.end(b) - base;
  if (all <= a.W || j >= all) return;
  const int length = (int)all, d = 2 * lane;
  const bool mine = d < a.D;
  const auto add = [&](float (&y)[2], int64_t piece) {
    const float* from = piece_sums(a, piece, head, which) + (int64_t)j * a.D + d;
    const f32x2 x = mine ? *reinterpret_cast<const f32x2*>(from) : f32x2{0, 0};
    y[0] += x[0];
    y[1] += x[1];
  };
  float y[2] = {0.0f, 0.0f};
  add(y, a.pieces + b);
  const int64_t first = first_tile(base, b, 1, (uint32_t)a.piece);
  for (int p = a.W / a.piece; p <= (length - 1) / a.piece; ++p) add(y, first + p);
  const float times = which ? 1.0f : a.scale;
  uint16_t* out = (which ? a.grad_v + (base + j) * a.ldgv : a.grad_k + (base + j) * a.ldgk) + (int64_t)head * a.D;
  if (mine) *reinterpret_cast<uint32_t*>(out + d) = pack2<T>(y[0] * times, y[1] * times);
}

struct WindowKernels {
  const void *fwd, *dq, *dkdv, *sinks;
};
template <typename T, int kD>
WindowKernels window_of() {
  return {(const void*)&window_fwd_kernel<T, kD>, (const void*)&window_dq_kernel<T, kD>,
          (const void*)&window_dkdv_kernel<T, kD>, (const void*)&window_sinks_kernel<T>};
}
WindowKernels window_kernels(int dtype, int D) {
  if (dtype == ENGRAM_BF16) return D <= 64 ? window_of<bf16_t, 64>() : window_of<bf16_t, 128>();
  return D <= 64 ? window_of<_Float16, 64>() : window_of<_Float16, 128>();
}

WindowArgs window_args(const WindowCall& w) {
  WindowArgs a{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
               nullptr, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.0f, Divide((uint32_t)(w.Hq / w.Hk))};
  a.q = w.q; a.k = w.k; a.v = w.v; a.cu = w.cu;
  a.N = w.N; a.ldq = w.ldq; a.ldk = w.ldk; a.ldv = w.ldv;
  a.B = (int)w.B; a.Hk = (int)w.Hk; a.G = (int)(w.Hq / w.Hk); a.D = (int)w.D;
  a.W = (int)(w.window < w.N ? w.window : w.N);
  a.S = (int)w.sinks;
  a.scale = w.scale;
  return a;
}
hipError_t launch_heads(const void* kernel, WindowArgs a, int64_t tiles, int threads, hipStream_t stream) {
  a.tiles = (int)tiles;
  void* args[] = {&a};
  return hipLaunchKernel(kernel, dim3((unsigned)(tiles * a.Hk + a.sink_blocks)), dim3((unsigned)threads), args, 0, stream);
}

// Tokens of a piece: some thousand workgroups in all, but pieces worth a launch.
int64_t piece_of(int64_t N, int64_t Hk) {
  const int64_t pieces = 1024 / Hk > 1 ? 1024 / Hk : 1, piece = (N + pieces - 1) / pieces;
  return piece < 256 ? 256 : piece;
}
int64_t delta_values(int64_t N, int64_t Hq) { return (N * Hq + 3) / 4 * 4; }

}  // namespace

size_t window_bwd_workspace(int64_t N, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks) {
  int64_t values = delta_values(N, Hq);
  if (sinks > 0 && window < N) values += (N / piece_of(N, Hk) + 2 * B) * Hk * 2 * sinks * D;
  return (size_t)values * sizeof(float);
}

hipError_t launch_window_fwd(const WindowCall& w, hipStream_t stream) {
  WindowArgs a = window_args(w);
  a.out = w.o; a.ldout = w.ldo; a.lse = w.lse;
  return launch_heads(window_kernels(w.dtype, a.D).fwd, a, a.N * a.G / kRows + a.B, kThreads, stream);
}

hipError_t launch_window_bwd(const WindowCall& w, hipStream_t stream) {
  WindowArgs a = window_args(w);
  const WindowKernels k = window_kernels(w.dtype, a.D);
  a.o = w.o_in; a.ldo = w.ldo; a.grad_o = w.grad_o; a.ldgo = w.ldgo; a.lse_in = w.lse_in;
  a.out = w.grad_q; a.ldout = w.ldgq; a.grad_k = w.grad_k; a.ldgk = w.ldgk; a.grad_v = w.grad_v; a.ldgv = w.ldgv;
  a.delta = static_cast<float*>(w.workspace);
  a.sums = a.delta + delta_values(w.N, w.Hq);
  a.piece = (int)piece_of(w.N, w.Hk);
  hipError_t e = launch_heads(k.dq, a, a.N * a.G / kRows + a.B, kThreads, stream);
  if (e != hipSuccess) return e;
  const bool sinks = a.S > 0 && a.W < a.N;
  a.pieces = (int)(a.N / a.piece) + a.B;
  if (sinks) a.sink_blocks = a.pieces * a.Hk;
  e = launch_heads(k.dkdv, a, a.N / kRows + a.B, kKeyThreads, stream);
  if (e != hipSuccess || !sinks) return e;
  void* args[] = {&a};
  return hipLaunchKernel(k.sinks, dim3((unsigned)((a.B * a.Hk * 64 + kJoinThreads - 1) / kJoinThreads), (unsigned)(2 * a.S)),
                         dim3(kJoinThreads), args, 0, stream);
}

}  // namespace engram
