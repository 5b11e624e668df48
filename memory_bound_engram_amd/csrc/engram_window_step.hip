// engram_window_step.hip -- the window attention of single tokens over a pool of
// caches, and the caches' filling from a prompt (gfx950).
//
// A cache has a line for each of the first S tokens (the sinks) and a ring of
// R >= W lines: token j is in line j < S, or S + (j - S) % R.  The token at
// position p sees the sinks and the last W tokens; what it sees, as a list, is
//   the tokens 0 .. n_sinks - 1, then the tokens a .. p,  a = max(S, p - W + 1)
// whose lines follow each other round the ring.
//
// Mapping.  The lines seen are read once, which bounds the kernel, and past the
// caches, as nothing reads them again (64 rows, 8 key heads of 128, 1028 tokens seen:
// 48.3 us, 5.6 TB/s; 53.9 with plain loads).  A workgroup has
// one row of the batch, one key head and up to sixteen of its query heads, or a
// part of the list for these; its waves go through the list in tiles of 32 lines, each
// on its own: keys go from memory to registers as they are operands of the products
// that give the scores (16x16x32, transposed: a lane has one query head), the next
// tile's on their way; values through LDS of the wave's own, to be read
// transposed.  The waves' maxima, sums and outputs are joined through LDS at the
// end; where a list is split over workgroups, a second kernel joins theirs.
//
// Rows of one slot that are neighbours in the batch are tokens one behind the other:
// a row takes those before it from k and v instead of the cache, into which
// another workgroup may not have written them yet.
#include "engram_launch.h"
#include "engram_sequences.h"
#include "engram_values.h"

namespace engram {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kWaves = 4;    // of a workgroup
constexpr int kLines = 32;   // of a tile
constexpr int kHeads = 16;   // query heads of a workgroup
constexpr float kLog2e = 1.44269504f;

struct StepArgs {
  const uint16_t *q, *k, *v;
  uint16_t *cache_k, *cache_v, *o;
  const int64_t *slots, *positions;
  float* parts;  // [B][Hq][splits][D], then maximum and sum [B][Hq][splits][2]
  int64_t n_slots, ldq, ldk, ldv, ldo;
  int B, Hk, G, D, S, R, W, groups, splits;
  float scale;
};

template <typename T>
__device__ __forceinline__ f32x4 product16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (__is_same(T, bf16_t))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (__is_same(T, bf16_t)) {
    return pack_bf16x2(lo, hi);
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
}

// The maximum (sum) over the four lanes of a query head, in each.
__device__ __forceinline__ float head_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float head_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A tile of values in LDS: rows of kD values, the 16-byte pieces of row r in the
// order piece ^ turn(r), with which thirty-two lanes of a transposing read (eight
// rows of two neighbouring pieces) find their values in different banks.
template <int kD>
__device__ __forceinline__ uint32_t place(uint32_t row, uint32_t col) {
  const uint32_t turn = kD == 128 ? (row & 7) << 1 : (row >> 1 & 3) << 1;
  return row * kD + ((col >> 3) ^ turn) * 8 + (col & 7);
}

// a % b for a >= 0: 64-bit division takes hundreds of instructions.
__device__ __forceinline__ int rest_of(int64_t a, int b) {
  return a >> 32 == 0 ? (int)((uint32_t)a % (uint32_t)b) : (int)(a % b);
}
// The list of a row: which tokens its tile's lines hold, and where they lie.
struct Seen {
  int64_t p;       // the row's position
  int sinks, n;    // tokens that are sinks; of the list
  int start, R, S; // the ring's line of the first behind them
  int mates;       // rows of the same slot right before this one
  // the line of the i-th token of the list, and how far it is back
  __device__ __forceinline__ int line(int i, int64_t* back) const {
    const bool sink = i < sinks;
    *back = sink ? p - i : (int64_t)(n - 1 - i);
    const int at = start + (i - sinks);
    return sink ? i : S + (at >= R ? at - R : at);
  }
};

template <typename T, int kD>
__global__ __launch_bounds__(kWaves * 64) void window_step_kernel(StepArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t tiles[kWaves][kLines * kD];
  __shared__ float maxima[kWaves][kHeads], sums[kWaves][kHeads];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l = lane & 15, g = lane >> 4;
  int at = blockIdx.x;
  const int split = at % a.splits;
  at /= a.splits;
  const int group = at % a.groups;
  at /= a.groups;
  const int head = at % a.Hk, b = at / a.Hk;
  const int64_t slot = a.slots[b];
  Seen seen;
  seen.p = a.positions[b];
  if (slot < 0 || slot >= a.n_slots || seen.p < 0) return;
  {
    const int before = b - 1 - (int)lane, safe = before >= 0 ? before : 0;
    const uint64_t same = __ballot(before >= 0 && a.slots[safe] == slot && a.positions[safe] == seen.p - 1 - (int64_t)lane);
    seen.mates = ~same ? __builtin_ctzll(~same) : 64;
  }
  const int64_t p = seen.p;
  seen.R = a.R;
  seen.S = a.S;
  seen.sinks = p + 1 < a.S ? (int)(p + 1) : a.S;
  const int64_t first = p - a.W + 1 > a.S ? p - a.W + 1 : a.S;
  seen.n = seen.sinks + (int)(p >= first ? p - first + 1 : 0);
  seen.start = rest_of(first - a.S, a.R);
  const int64_t lines = (int64_t)a.S + a.R, cache = (slot * a.Hk + head) * lines * a.D;
  uint16_t *ck = a.cache_k + cache, *cv = a.cache_v + cache;
  const uint16_t *nk = a.k + (int64_t)head * a.D, *nv = a.v + (int64_t)head * a.D;

  // The token itself goes into its line, which no row of the call reads.
  if (split == 0 && group == 0 && (int)threadIdx.x < a.D / 4) {
    const int64_t line = p < a.S ? p : a.S + rest_of(p - a.S, a.R);
    const int d = (int)threadIdx.x % (a.D / 8) * 8;
    if ((int)threadIdx.x < a.D / 8) store16(ck + line * a.D + d, load16(nk + (int64_t)b * a.ldk + d));
    else store16(cv + line * a.D + d, load16(nv + (int64_t)b * a.ldv + d));
  }

  // Tiles of the list: split after split, wave after wave in turn.
  const int all = (seen.n + kLines - 1) / kLines, each = (all + a.splits - 1) / a.splits;
  const int from = split * each, to = from + each < all ? from + each : all;
  const u32x4 zero = {0, 0, 0, 0};
  u32x4 q[kD / 32];
  const int hq = group * kHeads + (int)l;
#pragma unroll
  for (int kk = 0; kk < kD / 32; ++kk) {
    const int d = 32 * kk + 8 * (int)g;
    q[kk] = hq < a.G && d < a.D ? load16(a.q + (int64_t)b * a.ldq + ((int64_t)head * a.G + hq) * a.D + d) : zero;
  }
  u32x4 kr[2][kD / 32];             // keys 16 u + l, values 32 kk + 8 g on
  constexpr int kMoves = kLines * kD / 512;
  u32x4 vr[kMoves];                 // pieces in order: row (64 i + lane) / (kD / 8)
  const auto fetch = [&](int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = tile * kLines + 16 * u + (int)l;
      int64_t back;
      const int line = seen.line(i, &back);
      const uint16_t* from = back <= seen.mates ? nk + (b - back) * a.ldk : ck + (int64_t)line * a.D;
#pragma unroll
      for (int kk = 0; kk < kD / 32; ++kk) {
        const int d = 32 * kk + 8 * (int)g;
        kr[u][kk] = i < seen.n && d < a.D ? load16_stream(from + d) : zero;
      }
    }
#pragma unroll
    for (int m = 0; m < kMoves; ++m) {
      const int i = tile * kLines + (64 * m + (int)lane) / (kD / 8), d = (int)lane % (kD / 8) * 8;
      int64_t back;
      const int line = seen.line(i, &back);
      const uint16_t* from = back <= seen.mates ? nv + (b - back) * a.ldv : cv + (int64_t)line * a.D;
      vr[m] = i < seen.n && d < a.D ? load16_stream(from + d) : zero;
    }
  };
  uint16_t* tv = tiles[wave];
  const float c = a.scale * kLog2e;
  f32x4 o[kD / 16];
#pragma unroll
  for (int dt = 0; dt < kD / 16; ++dt) o[dt] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, sum = 0.0f;
  int tile = from + (int)wave;
  if (tile < to) fetch(tile);
  for (; tile < to; tile += kWaves) {
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < kD / 32; ++kk) s[u] = product16<T>(kr[u][kk], q[kk], s[u]);
    }
#pragma unroll
    for (int i = 0; i < kMoves; ++i)
      store16(tv + place<kD>((64 * i + lane) / (kD / 8), lane % (kD / 8) * 8), vr[i]);
    if (tile + kWaves < to) fetch(tile + kWaves);
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (tile * kLines + 16 * u + 4 * (int)g + e >= seen.n) s[u][e] = -INFINITY;
        top = fmaxf(top, s[u][e]);
      }
    // (as in the forward: the terms may grow to 2^8 before they are scaled anew)
    if (__any((top - m) * c > 8.0f)) {
      top = fmaxf(m, head_max(top));
      const float keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * c);
      sum *= keep;
#pragma unroll
      for (int dt = 0; dt < kD / 16; ++dt) o[dt] *= keep;
      m = top;
    }
    float less = m == -INFINITY ? 0.0f : -m * c;
    // (fp16, whose steps below 2^-14 are all 2^-24: times 2^7, which leaves 2^15 at most)
    if constexpr (__is_same(T, _Float16)) less += 7.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[u][e] = __builtin_amdgcn_exp2f(fmaf(s[u][e], c, less));
        sum += s[u][e];
      }
    // contraction index 8 g + e: line 16 (e / 4) + 4 g + e % 4
    const u32x4 pw = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]), pack2<T>(s[1][0], s[1][1]),
                      pack2<T>(s[1][2], s[1][3])};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int dt = 0; dt < kD / 16; ++dt) {
      const uint32_t row = 4 * g + l / 4, col = 16 * dt + 4 * (l % 4);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(tv + place<kD>(row, col)));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(tv + place<kD>(row + 16, col)));
      const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
      o[dt] = product16<T>(u32x4{x[0], x[1], y[0], y[1]}, pw, o[dt]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  sum = head_sum(sum);

  // The waves' parts: maxima and sums, then the outputs in LDS, a head's values
  // (fp32) in the order they are there for each lane.
  if (g == 0) {
    maxima[wave][l] = m;
    sums[wave][l] = sum;
  }
  __syncthreads();  // all waves' tiles are read out
  f32x4(*outs)[kD / 16][64] = reinterpret_cast<f32x4(*)[kD / 16][64]>(&tiles[0][0]);  // one wave's: kD / 16 KB
  float top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, maxima[w][l]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    total += maxima[w][l] == -INFINITY ? sums[w][l] : sums[w][l] * __builtin_amdgcn_exp2f((maxima[w][l] - top) * c);
  const float keep = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c);
#pragma unroll
  for (int dt = 0; dt < kD / 16; ++dt) o[dt] *= keep;
  // in halves: what one half of the waves leaves, the other adds
#pragma unroll
  for (int half = kWaves / 2; half >= 1; half /= 2) {
    if ((int)wave >= half && (int)wave < 2 * half)
#pragma unroll
      for (int dt = 0; dt < kD / 16; ++dt) outs[wave - half][dt][lane] = o[dt];
    __syncthreads();
    if ((int)wave < half)
#pragma unroll
      for (int dt = 0; dt < kD / 16; ++dt) o[dt] += outs[wave][dt][lane];
    __syncthreads();
  }
  if (wave != 0 || hq >= a.G) return;
  const int64_t at_head = (int64_t)b * a.Hk * a.G + (int64_t)head * a.G + hq;
  if (a.splits == 1) {
    const float inverse = 1.0f / total;
    uint16_t* to_o = a.o + (int64_t)b * a.ldo + ((int64_t)head * a.G + hq) * a.D;
#pragma unroll
    for (int dt = 0; dt < kD / 16; ++dt) {
      const int d = 16 * dt + 4 * (int)g;
      if (d < a.D)
        *reinterpret_cast<u32x2*>(to_o + d) = u32x2{pack2<T>(o[dt][0] * inverse, o[dt][1] * inverse),
                                                    pack2<T>(o[dt][2] * inverse, o[dt][3] * inverse)};
    }
    return;
  }
  float* part = a.parts + (at_head * a.splits + split) * a.D;
#pragma unroll
  for (int dt = 0; dt < kD / 16; ++dt) {
    const int d = 16 * dt + 4 * (int)g;
    if (d < a.D) *reinterpret_cast<f32x4*>(part + d) = o[dt];
  }
  if (g == 0)
    *reinterpret_cast<f32x2*>(a.parts + (int64_t)a.B * a.Hk * a.G * a.splits * a.D + 2 * (at_head * a.splits + split)) =
        f32x2{top, total};
}

// The parts of a split list: a lane has four values of one query head.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void window_step_join_kernel(StepArgs a) {
  const int64_t at = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int Hq = a.Hk * a.G, quads = a.D / 4;
  const int64_t at_head = at / quads;
  const int d = (int)(at % quads) * 4, b = (int)(at_head / Hq), hq = (int)(at_head % Hq);
  if (b >= a.B) return;
  const int64_t slot = a.slots[b];
  if (slot < 0 || slot >= a.n_slots || a.positions[b] < 0) return;
  const float* state = a.parts + (int64_t)a.B * Hq * a.splits * a.D + 2 * at_head * a.splits;
  const float* part = a.parts + at_head * a.splits * a.D + d;
  const float c = a.scale * kLog2e;
  float top = -INFINITY, total = 0.0f;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, state[2 * s]);
  f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float m = state[2 * s], keep = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c);
    total += keep * state[2 * s + 1];
    o += keep * *reinterpret_cast<const f32x4*>(part + (int64_t)s * a.D);
  }
  o *= 1.0f / total;
  *reinterpret_cast<u32x2*>(a.o + (int64_t)b * a.ldo + (int64_t)hq * a.D + d) =
      u32x2{pack2<T>(o[0], o[1]), pack2<T>(o[2], o[3])};
}

// The filling: workgroups of a sequence and eight lines of its slot, a thread
// sixteen bytes of a line's head.  Of sequences with the same slot the last counts.
constexpr int kFillThreads = 256, kFillLines = 8;
struct FillArgs {
  const uint16_t *k, *v;
  uint16_t *cache_k, *cache_v;
  const int64_t *cu, *slots;
  int64_t N, n_slots, ldk, ldv;
  int B, Hk, D, S, R;
};
__global__ __launch_bounds__(kFillThreads) void window_fill_kernel(FillArgs a) {
  const int b = blockIdx.y, part = blockIdx.x;
  const int64_t slot = a.slots[b];
  if (slot < 0 || slot >= a.n_slots) return;
  bool later = false;
  for (int i = b + 1 + (int)threadIdx.x; i < a.B; i += kFillThreads) later |= a.slots[i] == slot;
  if (__syncthreads_or(later)) return;
  const Sequences seqs{a.cu, a.N, a.B};
  const int64_t base = seqs.start(b), n = seqs.end(b) - base, lines = (int64_t)a.S + a.R;
  const int pieces = a.Hk * (a.D / 8);
  for (int at = threadIdx.x; at < kFillLines * pieces; at += kFillThreads) {
    const int64_t line = (int64_t)part * kFillLines + at / pieces;
    const int head = at % pieces / (a.D / 8), d = at % pieces % (a.D / 8) * 8;
    if (line >= lines) continue;
    // the last token of the sequence that belongs into the line
    const int64_t back = line < a.S ? n - 1 - line : (n - 1 - line) % a.R, t = n - 1 - back;
    if (n - 1 < line || t < 0) continue;
    const int64_t to = ((slot * a.Hk + head) * lines + line) * a.D + d, from = (int64_t)head * a.D + d;
    store16(a.cache_k + to, load16(a.k + (base + t) * a.ldk + from));
    store16(a.cache_v + to, load16(a.v + (base + t) * a.ldv + from));
  }
}

struct StepKernels {
  const void *step, *join;
};
template <typename T>
StepKernels step_of(int D) {
  return {D <= 64 ? (const void*)&window_step_kernel<T, 64> : (const void*)&window_step_kernel<T, 128>,
          (const void*)&window_step_join_kernel<T>};
}

int64_t groups_of(int64_t Hq, int64_t Hk) { return (Hq / Hk + kHeads - 1) / kHeads; }

int64_t units_of(int64_t B, int64_t Hq, int64_t Hk) { return B * Hk * groups_of(Hq, Hk); }

// Into how many parts the lists are split, each a workgroup's (a second launch joins
// them): while there are two workgroups a CU, which is what the registers let in, but
// not into less than a tile for each wave.  (One row, 8 key heads, 1028 tokens seen:
// 12.6 us with 9 parts and the join, 16.2 with one part of eight waves.)
constexpr int64_t kPlaces = 512;
int64_t splits_of(int64_t B, int64_t Hq, int64_t Hk, int64_t seen) {
  const int64_t tiles = (seen + kLines - 1) / kLines, most = (tiles + kWaves - 1) / kWaves;
  const int64_t want = kPlaces / units_of(B, Hq, Hk), splits = want < most ? want : most;
  return splits > 1 ? splits : 1;
}

}  // namespace

size_t window_step_workspace(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t capacity) {
  const int64_t splits = splits_of(B, Hq, Hk, capacity);
  return splits > 1 ? (size_t)(B * Hq * splits * (D + 2)) * sizeof(float) : 0;
}

hipError_t launch_window_step(const WindowStepCall& w, hipStream_t stream) {
  StepArgs a{};
  a.q = w.q; a.k = w.k; a.v = w.v; a.cache_k = w.cache_k; a.cache_v = w.cache_v; a.o = w.o;
  a.slots = w.slots; a.positions = w.positions; a.parts = static_cast<float*>(w.workspace);
  a.n_slots = w.n_slots; a.ldq = w.ldq; a.ldk = w.ldk; a.ldv = w.ldv; a.ldo = w.ldo;
  a.B = (int)w.B; a.Hk = (int)w.Hk; a.G = (int)(w.Hq / w.Hk); a.D = (int)w.D;
  a.S = (int)w.sinks; a.R = (int)(w.capacity - w.sinks); a.W = (int)w.window;
  a.groups = (int)groups_of(w.Hq, w.Hk);
  a.splits = (int)splits_of(w.B, w.Hq, w.Hk, w.sinks + w.window);
  a.scale = w.scale;
  const StepKernels k = w.dtype == ENGRAM_BF16 ? step_of<bf16_t>(a.D) : step_of<_Float16>(a.D);
  void* args[] = {&a};
  const hipError_t e = hipLaunchKernel(k.step, dim3((unsigned)(units_of(w.B, w.Hq, w.Hk) * a.splits)), dim3(kWaves * 64), args,
                                       0, stream);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t threads = w.B * w.Hq * (w.D / 4);
  return hipLaunchKernel(k.join, dim3((unsigned)((threads + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), args, 0,
                         stream);
}

hipError_t launch_window_fill(const WindowStepCall& w, hipStream_t stream) {
  FillArgs a{};
  a.k = w.k; a.v = w.v; a.cache_k = w.cache_k; a.cache_v = w.cache_v; a.cu = w.cu; a.slots = w.slots;
  a.N = w.N; a.n_slots = w.n_slots; a.ldk = w.ldk; a.ldv = w.ldv;
  a.B = (int)w.B; a.Hk = (int)w.Hk; a.D = (int)w.D; a.S = (int)w.sinks; a.R = (int)(w.capacity - w.sinks);
  const int64_t lines = w.capacity < w.N ? w.capacity : w.N;  // no sequence reaches the others
  const int64_t parts = (lines + kFillLines - 1) / kFillLines;
  void* args[] = {&a};
  return hipLaunchKernel((const void*)&window_fill_kernel, dim3((unsigned)parts, (unsigned)w.B), dim3(kFillThreads), args, 0,
                         stream);
}

}  // namespace engram
