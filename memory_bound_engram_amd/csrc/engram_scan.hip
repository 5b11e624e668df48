// engram_scan.hip -- a gated recurrence over each channel: forward and backward
// over ragged sequences, and the step of single tokens (gfx950).
//
// For every sequence and channel, f = sigmoid(gate) and n = 1 - f = sigmoid(-gate):
//   h_t = f_t h_{t-1} + n_t u_t                       (h before the first: state_in)
// and with e the gradient that reaches the state before a token,
//   dh_t = grad_h_t + e_{t+1},  e_t = f_t dh_t        (e behind the last: grad_state_out)
//   du_t = n_t dh_t,  dgate_t = dh_t (h_{t-1} - u_t) f_t n_t,  dstate_in = e_first
//
// Digits.  Of f and n the smaller one, s = t / (1 + t) with t = exp(-|gate|), is exact
// relative to itself up to a few units (see Gate); the other is 1 - s.  f x is taken as x - s x where the gate is
// positive and as s x where it is not: a memory of 1 / n tokens needs n, not the
// 24 bits of a factor near 1 (which at n = 6e-6 would be off by half a percent of
// n), and a small f loses none either.
//
// Mapping.  One pass: each value is read once and written once, so HBM bounds the
// kernel.  The axis of time is cut into chunks; a workgroup takes one chunk of
// 256 channels, a lane four channels of kTokens tokens.  It walks its tokens from
// a state of zero, keeping x_t = local state and P_t = product of the factors in
// registers, so that the state that comes in, once known, is one fma a value.
// What a chunk does to the state, (P, x) at its end, goes to the other workgroups
// through memory, in two levels: the last of a group of eight chunks joins its
// group's and publishes that, and the last of eight groups the state behind them.
// A chunk's incoming state is the one behind the eight groups before its own,
// carried through the groups and then the chunks before it, always in the same
// order: one hop from workgroup to workgroup for every 64 chunks.
//
// What bounds it (29623 tokens of 5120 channels, bf16, forward: 231 us, 3.9 TB/s;
// backward of 8455: 130 us, 4.0 TB/s): a workgroup's stages follow each other (ticket,
// loads, walk, words, stores), two workgroups a CU overlap them only so far, and
// the vector units are at work most of the time too: an exponential, a reciprocal and some
// fifteen more instructions a value.  One level of words (a hop for every eight
// chunks) took 392.  Loads come back in order, so what the walk needs besides the values
// is asked for before them (261 without).  Slower: chunks of 32 tokens with
// three workgroups a CU (327), chunk and group words looked at together (249), workgroups that
// stay and take the next ticket, and ask for its values, before they are done with this
// one (432: others wait for a chunk that is held but not begun).
//
// Waiting.  A workgroup waits for words that others write.  Chunks are dealt by a
// ticket (a counter in the workspace), so all chunks before a workgroup's own
// belong to workgroups that run already.  A chunk's (P, x) is published before its
// workgroup waits for anything; a group's after waiting for chunks of lower
// tickets only; a state after waiting for those, groups of lower tickets and the
// state of a lower ticket.  So all chunks' words come, then all groups', then, by
// induction, all states: every wait ends.  A word is 8 bytes and says by itself
// whether it is there: all ones before (a launch of its own fills them), never all
// ones after (P is no NaN but the one below, and the state's second half is 0); no
// order of different words is assumed.
#include "engram_device.h"
#include "engram_launch.h"
#include "engram_sequences.h"
#include "engram_values.h"

namespace engram {
namespace {

constexpr int kWaves = 8;                    // of a workgroup
constexpr int kThreads = kWaves * 64;
constexpr int kCh = 4;                       // channels of a lane
constexpr int kTile = 64 * kCh;              // channels of a workgroup
constexpr int kGroup = 8;                    // chunks of a group, groups of a span: a wave looks at one of each
constexpr uint64_t kAbsent = ~0ull;
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;

// Tokens of a lane: as many as the registers of two workgroups a CU hold.
template <typename T>
constexpr int tokens_of() {
  return sizeof(T) == 4 ? 4 : 8;
}

// (P, x): what tokens do to a state y, x + P y; kFresh in P: a sequence begins
// among them, and the state behind them is x whatever it was before.
constexpr float kFresh = -1.0f;
__device__ __forceinline__ float through(f32x2 token, float y) {
  return token[0] == kFresh ? token[1] : fmaf(token[0], y, token[1]);
}
__device__ __forceinline__ f32x2 joined(f32x2 before, f32x2 after) {
  if (after[0] == kFresh) return after;
  return f32x2{before[0] == kFresh ? kFresh : after[0] * before[0], fmaf(after[0], before[1], after[1])};
}

// The exponent -|g| log2(e), rounded, is off by up to |g| 2^-24: for gates in fp32
// what it lacks, -|g| - x ln 2 by two fmas, is put back (without, s is off by up to 64 units of
// 2^-24 at |g| = 87, 16 at 12; with it by 7, as exp2, the reciprocal and three roundings are).
// For 16-bit gates, which are themselves off by 2^-12 or 2^-9 of |g|, it is not worth its
// four instructions a value (29623 tokens x 5120, bf16: 242 us, 236 without; 14811 in fp32: 189, 188).
template <typename T>
struct Gate {
  float s, n;   // the smaller of f and n, and n
  float a;      // -s, or s where that is f
  bool keeps;   // f is the larger
  __device__ __forceinline__ explicit Gate(float g) {
    const float m = __builtin_fabsf(g), x = -kLog2e * m;
    float t = __builtin_amdgcn_exp2f(x);
    // (an infinite gate's t is 0, whatever it is times; a NaN's is NaN)
    if constexpr (sizeof(T) == 4) t = fmaf(t, fminf(fmaf(-kLn2Low, x, fmaf(-kLn2, x, -m)), 1.0f), t);
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    s = t * r;
    keeps = g > 0.0f;
    n = keeps ? s : r;
    a = keeps ? -s : s;
  }
  // f P of a product of factors, and f x of any x: x - s x would make NaN of an infinity.
  __device__ __forceinline__ float f_of(float P) const { return fmaf(a, P, keeps ? P : 0.0f); }
  __device__ __forceinline__ float f_times(float x) const {
    const float most = 0x1.fffffep127f, bounded = __builtin_amdgcn_fmed3f(x, -most, most);
    return fmaf(a, keeps ? bounded : x, keeps ? x : 0.0f);
  }
};

struct ScanArgs {
  const void *gate, *u, *h_in, *grad_h;
  const int64_t* cu;
  const float* state_in;        // forward: before the first tokens; backward: the same, for h_{t-1}
  const float* state_end;       // backward: grad_state_out
  float* state_out;             // forward: behind the last tokens; backward: grad_state_in
  void *out, *out2;             // forward: h; backward: grad_gate, grad_u
  uint64_t* words;              // tickets, (P, x) of chunks, states of groups; null: one chunk is all
  int64_t N, ldg, ldu, ldh, ldgh, ldout, ldout2;
  int B, D, tiles, chunks, handing;  // handing: workgroups of a tile for empty sequences alone
};

// Words: the ticket in a line of its own; then, a tile's words for each, the chunks,
// the groups and the spans (the state before each).
constexpr int kTicketWords = 16;

__global__ void scan_clear_kernel(uint64_t* words, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 2;
  if (i >= n) return;  // n is even
  const uint32_t v = i < kTicketWords ? 0u : ~0u;
  store16(words + i, u32x4{v, v, v, v});
}

typedef uint64_t Words[kCh];
typedef f32x2 Ends[kCh];
// A lane's words, 64 apart, once they are there.
__device__ __forceinline__ void wait_words(const uint64_t* p, f32x2 (*to)[64], int lane) {
  Words v;
  for (;;) {
    bool there = true;
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      v[k] = __hip_atomic_load(p + 64 * k + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      there &= v[k] != kAbsent;
    }
    if (there) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int k = 0; k < kCh; ++k)
    to[k][lane] = f32x2{__uint_as_float((uint32_t)(v[k] >> 32)), __uint_as_float((uint32_t)v[k])};
}
__device__ __forceinline__ uint64_t word_of(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | (uint64_t)__float_as_uint(hi) << 32;
}

__device__ __forceinline__ void publish(uint64_t* p, const Ends& v, int lane) {
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    const float P = v[k][0] == v[k][0] ? v[k][0] : __uint_as_float(0x7fc00000u);  // no word is kAbsent
    __hip_atomic_store(p + 64 * k + lane, word_of(v[k][1], P), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

__device__ __forceinline__ void load_state(const float* p, bool mine, float (&v)[kCh]) {
  if (p && mine) unpack4(load_raw4(p), v);
  else unpack4(zero_raw4<float>(), v);
}

// The states of empty sequences go through unchanged: dealt out over the waves of all
// chunks, and of workgroups that are there for these alone where a wave would
// have more than kHanded of them (2^20 empty sequences behind one chunk).
constexpr int kHanded = 8;
template <bool kBack>
__device__ __forceinline__ void hand_on(const ScanArgs& a, const Sequences& seqs, int chunk, int wave, int ch) {
  const float* from = kBack ? a.state_end : a.state_in;
  const int64_t all = a.chunks + a.handing;
  for (int64_t b = chunk + all * wave; b < a.B; b += all * kWaves) {
    if (seqs.start((int)b) < seqs.end((int)b)) continue;
    float s[kCh];
    load_state(from ? from + b * a.D + ch : nullptr, true, s);
    store4<false>(a.state_out + b * a.D + ch, s);
  }
}

template <typename T, bool kBack>
__global__ __launch_bounds__(kThreads, 4) void scan_kernel(ScanArgs a) {
  constexpr int kTok = tokens_of<T>(), kChunk = kTok * kWaves;
  __shared__ f32x2 ends[kWaves][kCh][64];        // (P, x) of each wave's tokens
  __shared__ f32x2 looked[2][kGroup][kCh][64];   // of the chunks before this one in its group; of the groups before it
                                                 // in its span, and the state before the span as the last
  __shared__ uint32_t dealt;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t ticket = blockIdx.x;
  if (a.words) {
    if (threadIdx.x == 0)
      dealt = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.words), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    ticket = __builtin_amdgcn_readfirstlane(dealt);
  }
  const int chunk = (int)(ticket / a.tiles), tile = (int)(ticket % a.tiles), ch = tile * kTile + lane * kCh;
  const bool mine = ch < a.D;
  const Sequences seqs{a.cu, a.N, a.B};
  if (chunk >= a.chunks) {
    if (mine) hand_on<kBack>(a, seqs, chunk, wave, ch);
    return;
  }

  // The wave's tokens, in the order of the walk: step i is token first + i, or first - i.
  const int64_t walked = (int64_t)chunk * kChunk + wave * kTok;
  const int64_t first = kBack ? a.N - 1 - walked : walked;
  const auto token = [&](int i) { return kBack ? first - i : first + i; };
  const auto there = [&](int i) { return walked + i < a.N; };
  const auto get = [&](const void* p, int64_t ld, int64_t t, bool in) {
    return in && mine ? load_raw4<true>(static_cast<const T*>(p) + t * ld + ch) : zero_raw4<T>();
  };
  const int64_t asked = seqs.ask();  // before the values, as loads come back in order
  __builtin_amdgcn_sched_barrier(0);
  Raw4<T> gate[kTok], in[kTok];  // in: u, or the gradient of h
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    gate[i] = get(a.gate, a.ldg, token(i), there(i));
    in[i] = get(kBack ? a.grad_h : a.u, kBack ? a.ldgh : a.ldu, token(i), there(i));
  }

  // Whose tokens they are: the sequence of each, or -1; whether it is the first or the last.
  int seq[kTok];
  const int64_t low = kBack ? token(kTok - 1) : first;
  const auto start_of = [](int64_t at, int) { return at; };
  int64_t start, end;
  int b = seqs.last_at_most(low < 0 ? 0 : low, start_of, &start, &end, asked);
  uint32_t begins = 0, ends_here = 0;
#pragma unroll
  for (int i = 0; i < kTok; ++i) seq[i] = -1;
  // One sequence after the other, `t` the first token that none of them had (a test of each token's
  // own: 235 us for 231).
  for (int64_t t = low; t < low + kTok; t = end) {
    if (end <= t) {
      ++b;
      if (b < a.B) {
        start = seqs.start(b);
        end = seqs.end(b);
        // empty ones, of which there may be millions, are not walked through
        if (end <= t) b = seqs.last_at_most(t, start_of, &start, &end);
      }
      if (b >= a.B || end <= t) break;
    }
    const int from = (int)((start > t ? start : t) - low < kTok ? (start > t ? start : t) - low : kTok);
    const int to = (int)(end - low < kTok ? end - low : kTok);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const int i = kBack ? kTok - 1 - j : j;
      if (j < from || j >= to) continue;
      seq[i] = b;
      if (low + j == start) begins |= 1u << i;
      if (low + j == end - 1) ends_here |= 1u << i;
    }
  }
  const uint32_t enters = kBack ? ends_here : begins, leaves = kBack ? begins : ends_here;

  // The tokens from a state of zero.  Forward: x = h, and P behind the token.
  // Backward: x = dh; P, before the token in the walk (dh needs the e of the token
  // walked before), is made again with the gates below.
  float x[kTok][kCh], P[kBack ? 1 : kTok][kCh];
  f32x2 last[kCh];
#pragma unroll
  for (int k = 0; k < kCh; ++k) last[k] = f32x2{1.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    if (!there(i)) continue;  // a token that is not there leaves the state as it is
    if (enters >> i & 1) {
      const float* from = kBack ? a.state_end : a.state_in;
      float s[kCh];
      load_state(from ? from + (int64_t)seq[i] * a.D + ch : nullptr, mine, s);
#pragma unroll
      for (int k = 0; k < kCh; ++k) last[k] = f32x2{0.0f, s[k]};
    }
    float g[kCh], v[kCh];
    unpack4(gate[i], g);
    unpack4(in[i], v);
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const Gate<T> q(g[k]);
      if constexpr (kBack) {
        x[i][k] = v[k] + last[k][1];
        last[k] = f32x2{q.f_of(last[k][0]), q.f_times(x[i][k])};
      } else {
        last[k] = f32x2{q.f_of(last[k][0]), fmaf(q.n, v[k], q.f_times(last[k][1]))};
        x[i][k] = last[k][1];
        P[i][k] = last[k][0];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kCh; ++k) ends[wave][k][lane] = f32x2{enters ? kFresh : last[k][0], last[k][1]};
  __syncthreads();

  // What the waves before this one do; with the last one's, the chunk.
  Ends before;
#pragma unroll
  for (int k = 0; k < kCh; ++k) before[k] = f32x2{1.0f, 0.0f};
#pragma unroll 1
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int k = 0; k < kCh; ++k) before[k] = joined(before[k], ends[w][k][lane]);
  float carry[kCh];
#pragma unroll
  for (int k = 0; k < kCh; ++k) carry[k] = 0.0f;
  if (a.words) {
    const int group = chunk / kGroup, r = chunk % kGroup, span = group / kGroup, g = group % kGroup;
    const int groups = (a.chunks + kGroup - 1) / kGroup;
    const bool writer = wave == kWaves - 1;
    const auto words = [&](int i) { return a.words + kTicketWords + ((int64_t)i * a.tiles + tile) * kTile; };
    Ends all;
    if (writer) {
#pragma unroll
      for (int k = 0; k < kCh; ++k) all[k] = joined(before[k], ends[wave][k][lane]);
      publish(words(chunk), all, lane);
    }
    if (wave < r) wait_words(words(group * kGroup + wave), looked[0][wave], lane);
    __syncthreads();
    Ends chunks;
#pragma unroll
    for (int k = 0; k < kCh; ++k) chunks[k] = f32x2{1.0f, 0.0f};
#pragma unroll 1
    for (int j = 0; j < r; ++j)
#pragma unroll
      for (int k = 0; k < kCh; ++k) chunks[k] = joined(chunks[k], looked[0][j][k][lane]);
    if (writer && r == kGroup - 1) {
#pragma unroll
      for (int k = 0; k < kCh; ++k) all[k] = joined(chunks[k], all[k]);
      publish(words(a.chunks + group), all, lane);
    }
    if (writer ? span > 0 : wave < g)
      wait_words(words(writer ? a.chunks + groups + span : a.chunks + span * kGroup + wave), looked[1][wave], lane);
    __syncthreads();
    if (span > 0)
#pragma unroll
      for (int k = 0; k < kCh; ++k) carry[k] = looked[1][kGroup - 1][k][lane][1];
#pragma unroll 1
    for (int j = 0; j < g; ++j)
#pragma unroll
      for (int k = 0; k < kCh; ++k) carry[k] = through(looked[1][j][k][lane], carry[k]);
    if (writer && r == kGroup - 1 && g == kGroup - 1) {
#pragma unroll
      for (int k = 0; k < kCh; ++k) all[k] = f32x2{0.0f, through(all[k], carry[k])};
      publish(words(a.chunks + groups + span + 1), all, lane);
    }
#pragma unroll
    for (int k = 0; k < kCh; ++k) carry[k] = through(chunks[k], carry[k]);
  }
#pragma unroll
  for (int k = 0; k < kCh; ++k) carry[k] = through(before[k], carry[k]);

  // The state that comes in, applied, and the results.
  Raw4<T> us[2], hs[2];  // backward: of two tokens, the next two's on their way
  const auto fetch = [&](int i) {
    us[i % 2] = get(a.u, a.ldu, token(i), seq[i] >= 0);
    hs[i % 2] = get(a.h_in, a.ldh, token(i) - 1, seq[i] >= 0 && !(leaves >> i & 1));
  };
  if constexpr (kBack) {
    fetch(0);
    fetch(1);
  }
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    if (enters >> i & 1)
#pragma unroll
      for (int k = 0; k < kCh; ++k) carry[k] = 0.0f;
    float v[kCh];
#pragma unroll
    for (int k = 0; k < kCh; ++k) v[k] = kBack ? x[i][k] + carry[k] : fmaf(P[kBack ? 0 : i][k], carry[k], x[i][k]);
    const int64_t own = (int64_t)seq[i] * a.D + ch;
    const bool leaving = leaves >> i & 1;
    if constexpr (kBack) {
      float g[kCh], u[kCh], h[kCh], dg[kCh], du[kCh], e[kCh];
      unpack4(gate[i], g);
      unpack4(us[i % 2], u);
      if (leaving) load_state(a.state_in ? a.state_in + own : nullptr, mine, h);
      else unpack4(hs[i % 2], h);
      if (i + 2 < kTok) fetch(i + 2);
#pragma unroll
      for (int k = 0; k < kCh; ++k) {
        const Gate<T> q(g[k]);
        du[k] = q.n * v[k];
        dg[k] = du[k] * (h[k] - u[k]) * (q.keeps ? 1.0f - q.s : q.s);
        e[k] = q.f_times(v[k]);
        carry[k] = q.f_times(carry[k]);
      }
      if (seq[i] >= 0 && mine) {
        store4<true>(static_cast<T*>(a.out) + token(i) * a.ldout + ch, dg);
        store4<true>(static_cast<T*>(a.out2) + token(i) * a.ldout2 + ch, du);
        if (leaving && a.state_out) store4<false>(a.state_out + own, e);
      }
    } else if (seq[i] >= 0 && mine) {
      store4<true>(static_cast<T*>(a.out) + token(i) * a.ldout + ch, v);
      if (leaving && a.state_out) store4<false>(a.state_out + own, v);
    }
  }

  if (a.state_out && mine) hand_on<kBack>(a, seqs, chunk, wave, ch);
}

// The step: row i of the batch is one token of the sequence whose state is slot
// slots[i].  A thread has eight channels.  Rows with the same slot are taken in
// order by the workgroup of the first of them, which keeps the state in registers
// in between.
constexpr int kStepThreads = 256;
struct StepArgs {
  const void *gate, *u;
  float* pool;
  const int64_t* slots;
  void* h;
  int64_t n_slots, ldg, ldu, ldh;
  int B, D;
};

template <typename T>
__global__ __launch_bounds__(kStepThreads) void scan_step_kernel(StepArgs a) {
  __shared__ int next_row[2];
  int row = blockIdx.x;
  const int64_t slot = a.slots[row];
  if (slot < 0 || slot >= a.n_slots) return;
  const int ch = (blockIdx.y * kStepThreads + threadIdx.x) * 8;
  const bool mine = ch < a.D;
  float* state = a.pool + slot * a.D + ch;
  float s[8];
  if (mine) unpack8(load_raw<float>(state), s);
  if (threadIdx.x < 2) next_row[threadIdx.x] = a.B;
  __syncthreads();
  bool behind = false;
  int next = a.B;
  for (int i = threadIdx.x; i < a.B; i += kStepThreads)
    if (i != row && a.slots[i] == slot) {
      if (i < row) behind = true;
      else if (i < next) next = i;
    }
  if (behind) atomicMin(&next_row[1], 0);
  if (next < a.B) atomicMin(&next_row[0], next);
  __syncthreads();
  if (next_row[1] == 0) return;  // an earlier row's workgroup takes this one
  for (;;) {
    if (mine) {
      float g[8], u[8];
      unpack8(load_raw(static_cast<const T*>(a.gate) + (int64_t)row * a.ldg + ch), g);
      unpack8(load_raw(static_cast<const T*>(a.u) + (int64_t)row * a.ldu + ch), u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const Gate<T> q(g[k]);
        s[k] = fmaf(q.n, u[k], q.f_times(s[k]));
      }
      store8<false>(static_cast<T*>(a.h) + (int64_t)row * a.ldh + ch, s);
    }
    row = next_row[0];
    if (row >= a.B) break;
    __syncthreads();  // next_row is read
    if (threadIdx.x == 0) next_row[0] = a.B;
    __syncthreads();
    next = a.B;
    for (int i = row + 1 + threadIdx.x; i < a.B; i += kStepThreads)
      if (a.slots[i] == slot && i < next) next = i;
    if (next < a.B) atomicMin(&next_row[0], next);
    __syncthreads();
  }
  if (mine) store8<false>(state, s);
}

template <typename T>
const void* scan_of(bool back) {
  return back ? (const void*)&scan_kernel<T, true> : (const void*)&scan_kernel<T, false>;
}
int tokens_of_chunk(int dtype) { return (dtype == ENGRAM_FP32 ? tokens_of<float>() : tokens_of<bf16_t>()) * kWaves; }
int64_t tiles_of(int64_t D) { return (D + kTile - 1) / kTile; }
int64_t words_of(int64_t chunks, int64_t tiles) {
  const int64_t groups = (chunks + kGroup - 1) / kGroup, spans = groups / kGroup + 1;
  return kTicketWords + (chunks + groups + spans) * tiles * kTile;
}

// Workgroups up to which some are there for empty sequences: a launch counts its threads in 32 bits.
constexpr int kBlocksMost = 1 << 22;

hipError_t launch_scan(ScanArgs a, int dtype, bool back, void* workspace, hipStream_t stream) {
  const int64_t chunk = tokens_of_chunk(dtype);
  a.tiles = (int)tiles_of(a.D);
  a.chunks = (int)((a.N + chunk - 1) / chunk);
  a.words = a.chunks > 1 ? static_cast<uint64_t*>(workspace) : nullptr;
  const int most = a.state_out ? (a.B + kHanded * kWaves - 1) / (kHanded * kWaves) : 0;
  const int there = most < kBlocksMost / a.tiles ? most : kBlocksMost / a.tiles;  // (else each has more of them)
  a.handing = there > a.chunks ? there - a.chunks : 0;
  if (a.words) {
    uint64_t* words = a.words;
    int64_t n = words_of(a.chunks, a.tiles);
    void* args[] = {&words, &n};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&scan_clear_kernel), dim3((unsigned)((n + 511) / 512)),
                                         dim3(256), args, 0, stream);
    if (e != hipSuccess) return e;
  }
  const void* kernel = dtype == ENGRAM_BF16 ? scan_of<bf16_t>(back)
                       : dtype == ENGRAM_FP16 ? scan_of<_Float16>(back) : scan_of<float>(back);
  void* args[] = {&a};
  return hipLaunchKernel(kernel, dim3((unsigned)((int64_t)(a.chunks + a.handing) * a.tiles)), dim3(kThreads), args, 0, stream);
}

}  // namespace

// The words of the narrowest chunk, whatever the type.
size_t scan_workspace(int64_t N, int64_t D) {
  const int64_t chunk = tokens_of_chunk(ENGRAM_FP32);
  return (size_t)words_of((N + chunk - 1) / chunk, tiles_of(D)) * sizeof(uint64_t);
}

hipError_t launch_scan_fwd(const ScanCall& c, hipStream_t stream) {
  ScanArgs a{};
  a.gate = c.gate; a.u = c.u; a.cu = c.cu; a.state_in = c.state_in; a.state_out = c.state_out; a.out = c.h;
  a.N = c.N; a.B = (int)c.B; a.D = (int)c.D; a.ldg = c.ldg; a.ldu = c.ldu; a.ldout = c.ldh;
  return launch_scan(a, c.dtype, false, c.workspace, stream);
}

hipError_t launch_scan_bwd(const ScanCall& c, hipStream_t stream) {
  ScanArgs a{};
  a.gate = c.gate; a.u = c.u; a.h_in = c.h_in; a.grad_h = c.grad_h; a.cu = c.cu; a.state_in = c.state_in;
  a.state_end = c.grad_state_out; a.state_out = c.grad_state_in; a.out = c.grad_gate; a.out2 = c.grad_u;
  a.N = c.N; a.B = (int)c.B; a.D = (int)c.D; a.ldg = c.ldg; a.ldu = c.ldu; a.ldh = c.ldh; a.ldgh = c.ldgh;
  a.ldout = c.ldgg; a.ldout2 = c.ldgu;
  return launch_scan(a, c.dtype, true, c.workspace, stream);
}

hipError_t launch_scan_step(const ScanCall& c, hipStream_t stream) {
  StepArgs a{};
  a.gate = c.gate; a.u = c.u; a.pool = c.pool; a.slots = c.slots; a.h = c.h; a.n_slots = c.n_slots;
  a.ldg = c.ldg; a.ldu = c.ldu; a.ldh = c.ldh; a.B = (int)c.B; a.D = (int)c.D;
  const void* kernel = c.dtype == ENGRAM_BF16 ? (const void*)&scan_step_kernel<bf16_t>
                       : c.dtype == ENGRAM_FP16 ? (const void*)&scan_step_kernel<_Float16>
                                                : (const void*)&scan_step_kernel<float>;
  void* args[] = {&a};
  return hipLaunchKernel(kernel, dim3((unsigned)c.B, (unsigned)((c.D + 8 * kStepThreads - 1) / (8 * kStepThreads))),
                         dim3(kStepThreads), args, 0, stream);
}

}  // namespace engram
