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
// its joined state.
//
// Rounding.  bf16 operands enter the matrix cores as they are; sums are fp32.
// The scores (times their power of the decay) and X are rounded to bf16 where
// they become operands of the products that give y, which is rounded to bf16
// itself.  The products that update X, which all later chunks read and the
// caller gets in fp32, take c times its power of the decay as the sum of two
// bf16 values (relative error 2^-17), so X keeps fp32's standing.
#include "engram_device.h"
#include "engram_launch.h"

namespace engram {
namespace {

constexpr int kChunk = 64;
constexpr int kWalkThreads = 256;
constexpr int kPad = 16;  // 32 bytes: rows 8 banks apart for 16-byte and for transposing reads

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;


__device__ __forceinline__ bf16x8 join8(u32x2 lo, u32x2 hi) {
  const u32x4 r = {lo[0], lo[1], hi[0], hi[1]};
  return __builtin_bit_cast(bf16x8, r);
}

// Operand fragments of the 16x16x32 product: lane l holds row (or column)
// l % 16 and, with g = l / 16, the eight contraction indices 8g .. 8g+7.
// Here the row is a row of the tile.
template <int kStride>
__device__ __forceinline__ bf16x8 frag_rows(const uint16_t* tile, int row0, int k0, int lane) {
  return __builtin_bit_cast(bf16x8, load16(tile + (row0 + lane % 16) * kStride + k0 + 8 * (lane / 16)));
}
// The same, with the contraction indices in the order of an accumulator's
// rows: 4g .. 4g+3 of the first sixteen, then of the second.
template <int kStride>
__device__ __forceinline__ bf16x8 frag_rows_acc_order(const uint16_t* tile, int row0, int k0, int lane) {
  const uint16_t* p = tile + (row0 + lane % 16) * kStride + k0 + 4 * (lane / 16);
  return join8(*reinterpret_cast<const u32x2*>(p), *reinterpret_cast<const u32x2*>(p + 16));
}
// Here the row is a column of the tile and the contraction runs down the
// tile's rows, read through the transposing LDS load: the sixteen lanes of a
// group name four rows of sixteen values and get a column of four each.
template <int kStride>
__device__ __forceinline__ bf16x8 frag_cols(const uint16_t* tile, int k0, int col0, int lane) {
  const int l = lane % 16;
  const uint16_t* p = tile + (k0 + 8 * (lane / 16) + l / 4) * kStride + col0 + 4 * (l % 4);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * kStride));
  return join8(__builtin_bit_cast(u32x2, lo), __builtin_bit_cast(u32x2, hi));
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ u32x2 pack4(f32x4 v) {
  const u32x2 r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  return r;
}

// lam^steps for steps >= 0 (lam^0 is 1 also where lam is 0).
__device__ __forceinline__ float decay_power(float log_decay, int steps) {
  return steps == 0 ? 1.0f : expf(log_decay * (float)steps);
}

// The lane's number as a value the compiler knows nothing of: what is computed
// from it stays where it is used, instead of moving out of loops and being
// spilled.
__device__ __forceinline__ int afresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// A value that all lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const int32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | lo);
}

// Memory through a buffer descriptor: a base that all lanes share and a 32-bit
// offset each; loads from kBeyond give zero and stores to it are dropped.
constexpr uint32_t kBeyond = 0xf0000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0x80000000u, 0x00020000);
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
  static constexpr int kSa = kDa + kPad, kSc = kDc + kPad, kSp = kChunk + kPad;
  static constexpr int kDt = kDa / 16;            // tiles of state rows
  static constexpr int kNt = kDc / 64;            // tiles of state columns in a wave
  static constexpr int kVa = kDa * kChunk / 8 / kWalkThreads;  // 16-byte vectors a thread stages of a (and of b)
  static constexpr int kVc = kDc * kChunk / 8 / kWalkThreads;

  struct Lds {
    alignas(16) uint16_t a[kStateOnly ? 1 : kChunk * kSa];
    alignas(16) uint16_t b[kChunk * kSa];
    alignas(16) uint16_t c[kChunk * kSc];
    alignas(16) uint16_t p[kStateOnly ? 1 : kChunk * kSp];
    int bad[2];
  };

  // Rows pos .. pos + L - 1 of the head, the rest zero.
  template <int kV, int kD>
  static __device__ __forceinline__ void fetch(u32x4 (&r)[kV], const uint16_t* x, int64_t ld, int head, int d,
                                               int64_t pos, int L, const WalkArgs& w, int tid) {
    const __amdgpu_buffer_rsrc_t src = buffer_of(x + (w.turned ? w.N - pos - L : pos) * ld + (int64_t)head * d);
    const int row = tid / (kD / 8), col = tid % (kD / 8) * 8;
    constexpr int kRows = kWalkThreads / (kD / 8);
    const uint32_t line = (uint32_t)ld * 2;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int t = row + i * kRows;
      const uint32_t off = (uint32_t)(w.turned ? L - 1 - t : t) * line + (uint32_t)col * 2;
      r[i] = __builtin_amdgcn_raw_buffer_load_b128(src, (int)(t < L && col < d ? off : kBeyond), 0, 0);
    }
  }
  template <int kV, int kD, int kStride>
  static __device__ __forceinline__ void put(uint16_t* tile, const u32x4 (&r)[kV], int tid) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      constexpr int kRows = kWalkThreads / (kD / 8);
      store16(tile + (tid / (kD / 8) + i * kRows) * kStride + tid % (kD / 8) * 8, r[i]);
    }
  }
  template <int kV>
  static __device__ __forceinline__ bool not_finite(const u32x4 (&r)[kV]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bad |= (r[i][k] & 0x7f80u) == 0x7f80u || (r[i][k] & 0x7f800000u) == 0x7f800000u;
    return bad;
  }

  // X as accumulators: tile (dt, nt) of a wave holds rows 16 dt + 4 g + r and
  // column 16 (wave kNt + nt) + lane % 16.
  typedef f32x4 State[kDt][kNt];

  // kOut: X to p, else p to X (zero where p is null).
  template <bool kOut, bool kTransposed>
  static __device__ __forceinline__ void move_state(State& X, const float* p, const WalkArgs& w, int wave, int lane0) {
    const int lane = afresh(lane0);
    const __amdgpu_buffer_rsrc_t at = buffer_of(p);
    const int d = 4 * (lane / 16);
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      const int n = 16 * (wave * kNt + nt) + lane % 16;
      const uint32_t first = p && n < w.Dc ? 4u * (uint32_t)(kTransposed ? n * w.Da + d : d * w.Dc + n) : kBeyond;
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) {
        const int off = (int)(16 * dt + d < w.Da ? first : kBeyond);
        if constexpr (kTransposed && kOut) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, X[dt][nt]), at, off, 64 * dt, 0);
        } else if constexpr (kTransposed) {
          X[dt][nt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(at, off, 64 * dt, 0));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int line = 4 * (16 * dt + r) * w.Dc;
            if constexpr (kOut) {
              const float v = X[dt][nt][r];
              __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), at, off, line, 0);
            } else {
              X[dt][nt][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(at, off, line, 0));
            }
          }
        }
      }
    }
  }
  static __device__ __forceinline__ void load_state(State& X, const float* p, bool transposed, const WalkArgs& w, int wave,
                                                    int lane) {
    if (transposed) move_state<false, true>(X, p, w, wave, lane);
    else move_state<false, false>(X, p, w, wave, lane);
  }
  static __device__ __forceinline__ void store_state(State& X, float* p, bool transposed, const WalkArgs& w, int wave,
                                                     int lane) {
    if (transposed) move_state<true, true>(X, p, w, wave, lane);
    else move_state<true, false>(X, p, w, wave, lane);
  }

  // The powers of the decay that a lane needs, as products of a factor of its
  // own and one that all lanes share: scores lam^(t-s) with t = 16 wave + l and
  // s = 16 st + 4 g + r, the carried state lam^(t+e) with t = 16 tt + l, and the
  // rows of a full chunk lam^(64-e-s) with s = 32 kt + 8 g + i.
  struct Powers {
    float diagonal[4];   // s_intra lam^(l-4g-r), 0 above the diagonal
    float below[4];      // s_intra lam^(16+l-4g-r)
    float tiles[3];      // lam^(16 i)
    float in;            // s_inter lam^(l+e)
    float rows[2];       // s_upd lam^(57-e-32kt-8g)
    float eight[8];      // lam^i
    __device__ __forceinline__ void set(float ld, const WalkArgs& w, int lane) {
      const int g = lane / 16, l = lane % 16;
      for (int r = 0; r < 4; ++r) {
        const int steps = l - 4 * g - r;
        diagonal[r] = steps >= 0 ? w.s_intra * decay_power(ld, steps) : 0.0f;
        below[r] = w.s_intra * decay_power(ld, 16 + steps);
      }
      for (int i = 0; i < 3; ++i) tiles[i] = uniform(decay_power(ld, 16 * i));
      in = w.s_inter * decay_power(ld, l + w.e);
      for (int kt = 0; kt < 2; ++kt) rows[kt] = w.s_upd * decay_power(ld, kChunk - 7 - w.e - 32 * kt - 8 * g);
      for (int i = 0; i < 8; ++i) eight[i] = uniform(decay_power(ld, i));
    }
  };

  // Walk the rows [pos, stop) of one sequence, chunk by chunk.
  static __device__ __forceinline__ void rows(Lds& lds, State& X, int64_t pos, int64_t stop, int head, const float ld,
                                              const Powers& pw, int& parity, const WalkArgs& w, int wave, int lane0) {
    u32x4 ra[kStateOnly ? 1 : kVa], rb[kVa], rc[kVc];
    int64_t single = pos;  // rows before this one are walked one at a time
    int L = (int)(stop - pos < kChunk ? stop - pos : kChunk);
    auto get = [&](int64_t at, int n, int tid) {
      if constexpr (!kStateOnly) fetch<kVa, kDa>(ra, w.a, w.lda, head, w.Da, at, n, w, tid);
      fetch<kVa, kDa>(rb, w.b, w.ldb, head, w.Da, at, n, w, tid);
      fetch<kVc, kDc>(rc, w.c, w.ldc, head, w.Dc, at, n, w, tid);
    };
    get(pos, L, threadIdx.x);
    while (pos < stop) {
      const int lane = afresh(lane0);
      const int g = lane / 16, l = lane % 16, tid = wave * 64 + lane;
      if constexpr (!kStateOnly) put<kVa, kDa, kSa>(lds.a, ra, tid);
      put<kVa, kDa, kSa>(lds.b, rb, tid);
      put<kVc, kDc, kSc>(lds.c, rc, tid);
      if (not_finite<kVc>(rc)) lds.bad[parity] = 1;
      __syncthreads();
      // An infinity or NaN in a row of c would reach the rows before it too, as
      // 0 * c in the product with the scores: such a chunk is walked row by row.
      const bool bad = lds.bad[parity] != 0;
      if (bad && L > 1) {
        single = pos + L;
        L = 1;
        get(pos, L, tid);
        parity ^= 1;
        if (threadIdx.x == 0) lds.bad[parity] = 0;
        __syncthreads();
        continue;
      }
      if (threadIdx.x == 0) lds.bad[parity ^ 1] = 0;
      const int64_t next = pos + L;
      const int next_L = next < single ? 1 : (int)(stop - next < kChunk ? stop - next : kChunk);
      if (next < stop) get(next, next_L, tid);

      bf16x8 cf[2][kNt];
      if constexpr (!kStateOnly) {
        // scores of the wave's sixteen rows t, transposed: the lane has t = 16 wave + l and four neighbouring s
        bf16x8 at[kDa / 32];
#pragma unroll
        for (int kk = 0; kk < kDa / 32; ++kk) at[kk] = frag_rows<kSa>(lds.a, 16 * wave, 32 * kk, lane);
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          u32x2 packed = {0, 0};
          if (st <= wave) {
            f32x4 s = {0, 0, 0, 0};
            const float between = wave - st <= 1 ? 1.0f : wave - st == 2 ? pw.tiles[1] : pw.tiles[2];
#pragma unroll
            for (int kk = 0; kk < kDa / 32; ++kk) s = mfma(frag_rows<kSa>(lds.b, 16 * st, 32 * kk, lane), at[kk], s);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (st == wave) s[r] = 4 * g + r <= l ? s[r] * pw.diagonal[r] : 0.0f;
              else s[r] *= pw.below[r] * between;
            }
            packed = pack4(s);
          }
          *reinterpret_cast<u32x2*>(lds.p + (16 * wave + l) * kSp + 16 * st + 4 * g) = packed;
        }
      }
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) cf[kt][nt] = frag_cols<kSc>(lds.c, 32 * kt, 16 * (wave * kNt + nt), lane);
      if constexpr (!kStateOnly) {
        bf16x8 xf[kDa / 32][kNt];
#pragma unroll
        for (int kk = 0; kk < kDa / 32; ++kk)
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) xf[kk][nt] = join8(pack4(X[2 * kk][nt]), pack4(X[2 * kk + 1][nt]));
        const __amdgpu_buffer_rsrc_t dst =
            buffer_of(w.y + (w.turned ? w.N - pos - L : pos) * w.ldy + (int64_t)head * w.Dc);
        __syncthreads();  // the scores of all waves
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          __builtin_amdgcn_sched_barrier(0);
          f32x4 y[kNt];
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) y[nt] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int kk = 0; kk < kDa / 32; ++kk) {
            const bf16x8 af = frag_rows_acc_order<kSa>(lds.a, 16 * tt, 32 * kk, lane);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) y[nt] = mfma(xf[kk][nt], af, y[nt]);
          }
          const float in = pw.in * (tt < 3 ? pw.tiles[tt] : pw.tiles[1] * pw.tiles[2]);
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) y[nt] *= in;
#pragma unroll
          for (int kt = 0; kt <= tt / 2; ++kt) {
            const bf16x8 sf = frag_rows<kSp>(lds.p, 16 * tt, 32 * kt, lane);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) y[nt] = mfma(cf[kt][nt], sf, y[nt]);
          }
          const int t = 16 * tt + l;
          const uint32_t line = (uint32_t)(w.turned ? L - 1 - t : t) * (uint32_t)w.ldy * 2;
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            const int n = 16 * (wave * kNt + nt) + 4 * g;
            __builtin_amdgcn_raw_buffer_store_b64(pack4(y[nt]), dst, (int)(t < L && n < w.Dc ? line + 2 * n : kBeyond), 0, 0);
          }
        }
      }
      // X = lam^L X + s_upd sum_s lam^(L-e-s) b_s c_s^T
      __builtin_amdgcn_sched_barrier(0);
      const float less_one = uniform(expm1f(ld * (float)L));
      float up[2][8];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = 32 * kt + 8 * g + i;
          if (L == kChunk) up[kt][i] = pw.rows[kt] * pw.eight[7 - i];
          else up[kt][i] = s < L ? w.s_upd * decay_power(ld, L - w.e - s) : 0.0f;
        }
      bf16x8 hi[2][kNt], lo[2][kNt];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          const u32x4 raw = __builtin_bit_cast(u32x4, cf[kt][nt]);
          u32x4 h, q;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = bf_lo(raw[i]) * up[kt][2 * i], x1 = bf_hi(raw[i]) * up[kt][2 * i + 1];
            h[i] = pack_bf16x2(x0, x1);
            const float h0 = bf_lo(h[i]), h1 = bf_hi(h[i]);
            // an infinite value has no second part
            q[i] = pack_bf16x2(x0 == h0 ? 0.0f : x0 - h0, x1 == h1 ? 0.0f : x1 - h1);
          }
          hi[kt][nt] = __builtin_bit_cast(bf16x8, h);
          lo[kt][nt] = __builtin_bit_cast(bf16x8, q);
        }
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) {
        if (dt % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int r = 0; r < 4; ++r) X[dt][nt][r] = fmaf(X[dt][nt][r], less_one, X[dt][nt][r]);
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const bf16x8 bf = frag_cols<kSa>(lds.b, 32 * kt, 16 * dt, lane);
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            X[dt][nt] = mfma(bf, hi[kt][nt], X[dt][nt]);
            X[dt][nt] = mfma(bf, lo[kt][nt], X[dt][nt]);
          }
        }
      }
      parity ^= 1;
      pos = next;
      L = next_L;
      __syncthreads();  // the tiles are read out
    }
  }

  static __device__ __forceinline__ void run(const WalkArgs& w) {
    __shared__ __attribute__((aligned(16))) Lds lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % w.H;
    const int64_t seg = blockIdx.x / w.H;
    const float ld = uniform(w.log_decay[head]);
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
__global__ __launch_bounds__(kWalkThreads, 2) void decay_walk_kernel(WalkArgs w) {
  Walk<kDa, kDc, kStateOnly>::run(w);
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
  const float less_one = expm1f(w.log_decay[head] * (float)w.seg);
  const int64_t first = start / w.seg + 1, last = (end - 1) / w.seg;
  f32x4 x = {0, 0, 0, 0};
  for (int64_t j = first; j <= last; ++j) {
    f32x4* p = reinterpret_cast<f32x4*>(w.carry + (j * w.H + head) * state + at);
    f32x4 own = *p;
    if (j > first && (j - 1) * w.seg > start) {
#pragma unroll
      for (int r = 0; r < 4; ++r) own[r] += fmaf(x[r], less_one, x[r]);
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
    if (mine && d < Dk) *reinterpret_cast<f32x4*>(state + (int64_t)d * Dv) = S[i];
  }
}

template <bool kStateOnly>
const void* walk_kernel(int Da, int Dc) {
  if (Da <= 64)
    return Dc <= 64 ? (const void*)&decay_walk_kernel<64, 64, kStateOnly> : (const void*)&decay_walk_kernel<64, 128, kStateOnly>;
  return Dc <= 64 ? (const void*)&decay_walk_kernel<128, 64, kStateOnly> : (const void*)&decay_walk_kernel<128, 128, kStateOnly>;
}

int64_t segments(int64_t N, int64_t seg) { return (N + seg - 1) / seg; }

hipError_t launch_state_pass(WalkArgs w, hipStream_t stream) {
  void* args[] = {&w};
  return hipLaunchKernel(walk_kernel<true>(w.Da, w.Dc), dim3((unsigned)((segments(w.N, w.seg) - 1) * w.H)),
                         dim3(kWalkThreads), args, 0, stream);
}
hipError_t launch_join(WalkArgs w, hipStream_t stream) {
  void* args[] = {&w};
  const unsigned parts = (unsigned)((w.Da * w.Dc + 4 * kJoinThreads - 1) / (4 * kJoinThreads));
  return hipLaunchKernel(reinterpret_cast<const void*>(&decay_join_kernel), dim3((unsigned)(w.B * w.H), parts),
                         dim3(kJoinThreads), args, 0, stream);
}
hipError_t launch_walk(WalkArgs w, hipStream_t stream) {
  void* args[] = {&w};
  return hipLaunchKernel(walk_kernel<false>(w.Da, w.Dc), dim3((unsigned)(segments(w.N, w.seg) * w.H)),
                         dim3(kWalkThreads), args, 0, stream);
}
// The states of a cut axis, and the states of empty sequences.
hipError_t launch_carries(const WalkArgs& w, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (segments(w.N, w.seg) > 1) e = launch_state_pass(w, stream);
  if (e == hipSuccess && (segments(w.N, w.seg) > 1 || w.state_out)) e = launch_join(w, stream);
  return e;
}

}  // namespace

// Tokens of a segment: enough segments for about two workgroups a CU.
int64_t decay_segment(int64_t N, int64_t H) {
  constexpr int64_t kWant = 512;
  const int64_t want = (kWant + H - 1) / H;  // segments
  int64_t seg = (N + want - 1) / want;
  seg = (seg + kChunk - 1) / kChunk * kChunk;
  return seg < 2 * kChunk ? 2 * kChunk : seg;
}

size_t decay_workspace(int64_t N, int64_t H, int64_t Dk, int64_t Dv) {
  return (size_t)segments(N, decay_segment(N, H)) * (size_t)H * (size_t)Dk * (size_t)Dv * sizeof(float);
}

hipError_t launch_decay_fwd(const DecayCall& d, hipStream_t stream) {
  WalkArgs w{};
  w.a = d.q; w.b = d.k; w.c = d.v; w.y = d.o;
  w.lda = d.ldq; w.ldb = d.ldk; w.ldc = d.ldv; w.ldy = d.ldo;
  w.log_decay = d.log_decay; w.cu = d.cu; w.state_in = d.state_in; w.state_out = d.state_out;
  w.carry = static_cast<float*>(d.workspace);
  w.N = d.N; w.seg = decay_segment(d.N, d.H);
  w.B = (int)d.B; w.H = (int)d.H; w.Da = (int)d.Dk; w.Dc = (int)d.Dv;
  w.e = 1;
  w.s_intra = w.s_inter = d.scale;
  w.s_upd = 1.0f;
  hipError_t e = launch_carries(w, stream);
  return e == hipSuccess ? launch_walk(w, stream) : e;
}

hipError_t launch_decay_bwd(const DecayCall& d, hipStream_t stream) {
  // dq: forward in time, the state transposed
  WalkArgs w{};
  w.log_decay = d.log_decay; w.cu = d.cu;
  w.carry = static_cast<float*>(d.workspace);
  w.N = d.N; w.seg = decay_segment(d.N, d.H);
  w.B = (int)d.B; w.H = (int)d.H;
  w.a = d.grad_o; w.b = d.v; w.c = d.k; w.y = d.grad_q;
  w.lda = d.ldgo; w.ldb = d.ldv; w.ldc = d.ldk; w.ldy = d.ldgq;
  w.Da = (int)d.Dv; w.Dc = (int)d.Dk;
  w.state_in = d.state_in; w.state_t = true;
  w.e = 1;
  w.s_intra = w.s_inter = d.scale;
  w.s_upd = 1.0f;
  hipError_t e = launch_carries(w, stream);
  if (e == hipSuccess) e = launch_walk(w, stream);
  if (e != hipSuccess) return e;
  // dv: against time; this walk's last states are the gradients of state_in
  w.turned = true;
  w.a = d.k; w.b = d.q; w.c = d.grad_o; w.y = d.grad_v;
  w.lda = d.ldk; w.ldb = d.ldq; w.ldc = d.ldgo; w.ldy = d.ldgv;
  w.Da = (int)d.Dk; w.Dc = (int)d.Dv;
  w.state_in = d.grad_state_out; w.state_out = d.grad_state_in; w.state_t = false;
  w.e = 0;
  w.s_inter = 1.0f;
  w.s_upd = d.scale;
  e = launch_carries(w, stream);
  if (e == hipSuccess) e = launch_walk(w, stream);
  if (e != hipSuccess) return e;
  // dk: the same states, transposed
  w.a = d.v; w.b = d.grad_o; w.c = d.q; w.y = d.grad_k;
  w.lda = d.ldv; w.ldb = d.ldgo; w.ldc = d.ldq; w.ldy = d.ldgk;
  w.Da = (int)d.Dv; w.Dc = (int)d.Dk;
  w.state_out = nullptr; w.state_t = true; w.carry_t = true;
  return launch_walk(w, stream);
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
  // few states: a head's columns over up to four workgroups, so that more CUs take part
  const bool few = (int64_t)B * H < 512;
  const int cols = few ? 32 : 128;
  const void* kernel = few ? (const void*)&decay_step_kernel<32> : (const void*)&decay_step_kernel<128>;
  return hipLaunchKernel(kernel, dim3((unsigned)(B * H), (unsigned)((Dv + cols - 1) / cols)), dim3(kStepThreads), args, 0,
                         stream);
}

}  // namespace engram
