// engram_scan.hip -- a gated recurrence over each channel: forward and backward
// over ragged sequences, and the step of single tokens (gfx950).
//
// For every sequence and channel, f = sigmoid(gate) and n = 1 - f = sigmoid(-gate):
//   h_t = f_t h_{t-1} + n_t u_t                       (h before the first: state_in)
// and with e the gradient that reaches the state before a token,
//   dh_t = grad_h_t + e_{t+1},  e_t = f_t dh_t        (e behind the last: grad_state_out)
//   du_t = n_t dh_t,  dgate_t = dh_t (h_{t-1} - u_t) f_t n_t,  dstate_in = e_first
//
// Digits.  Of f and n the smaller one, s = t / (1 + t) with t = exp(-|gate|), keeps
// all its digits; the other is 1 - s.  f x is taken as x - s x where the gate is
// positive and as s x where it is not: a memory of 1 / n tokens needs n, not the
// 24 bits of a factor near 1 (which at n = 6e-6 would be off by half a percent of
// n), and a small f loses none either.
//
// Mapping.  One pass: each value is read once and written once, so HBM bounds the
// kernel.  The axis of time is cut into chunks; a workgroup takes one chunk of
// 512 channels, a lane eight channels of kTokens tokens.  It walks its tokens from
// a state of zero, keeping x_t = local state and P_t = product of the factors in
// registers, so that the state that comes in, once known, is one fma a value.
// What a chunk does to the state, (P, x) at its end, goes to the other workgroups
// through memory: the chunks of a group of eight publish theirs; the group's last
// publishes the state behind it.  A chunk's incoming state is that behind the group before,
// carried through the chunks of its own group in order: eight hops for 4096
// tokens, and always the same sums in the same order.
//
// Waiting.  A workgroup waits for words that others write.  Chunks are dealt by a
// ticket (a counter in the workspace), so all chunks before a workgroup's own
// belong to workgroups that run already.  It publishes its own (P, x) before it
// waits for anything, and then waits for lower tickets only; so by induction over
// the tickets every wait ends.  A word is 8 bytes and says by itself whether it
// is there: all ones before (a launch of its own fills them), never all ones after (P
// is no NaN but the one below, and the state's second half is 0); no order of
// different words is assumed.
#include "engram_device.h"
#include "engram_launch.h"
#include "engram_sequences.h"
#include "engram_values.h"

namespace engram {
namespace {

constexpr int kWaves = 8;                    // of a workgroup
constexpr int kThreads = kWaves * 64;
constexpr int kTile = 64 * 8;                // channels of a workgroup
constexpr int kGroup = 8;                    // chunks of a group: a wave looks at one
constexpr uint64_t kAbsent = ~0ull;
constexpr float kLog2e = 1.44269504f;

// Tokens of a lane: as many as the registers of two workgroups a CU hold.
template <typename T>
constexpr int tokens_of() {
  return sizeof(T) == 4 ? 2 : 4;
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

struct Gate {
  float s, n;   // the smaller of f and n, and n
  float a;      // -s, or s where that is f
  bool keeps;   // f is the larger
  __device__ __forceinline__ explicit Gate(float g) {
    const float t = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(g));
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
  int B, D, tiles, chunks;
};

constexpr int kTicketWords = 16;  // a line of its own
__device__ __host__ __forceinline__ int64_t chunk_word(int chunk, int tile, int tiles) {
  return kTicketWords + ((int64_t)chunk * tiles + tile) * kTile;
}

__global__ void scan_clear_kernel(uint64_t* words, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 2;
  if (i >= n) return;  // n is even
  const uint32_t v = i < kTicketWords ? 0u : ~0u;
  store16(words + i, u32x4{v, v, v, v});
}

// Eight words of a lane, 64 apart, once they are there.
__device__ __forceinline__ void wait_words(const uint64_t* p, uint64_t (&v)[8]) {
  for (;;) {
    bool there = true;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = __hip_atomic_load(p + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      there &= v[k] != kAbsent;
    }
    if (there) return;
    __builtin_amdgcn_s_sleep(1);
  }
}
__device__ __forceinline__ uint64_t word_of(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | (uint64_t)__float_as_uint(hi) << 32;
}

__device__ __forceinline__ void load_state(const float* p, bool mine, float (&v)[8]) {
  if (p && mine) unpack8(load_raw(p), v);
  else unpack8(zero_raw<float>(), v);
}

template <typename T, bool kBack>
__global__ __launch_bounds__(kThreads, 4) void scan_kernel(ScanArgs a) {
  constexpr int kTok = tokens_of<T>(), kChunk = kTok * kWaves;
  __shared__ f32x2 ends[kWaves][8][64];   // (P, x) of each wave's tokens
  __shared__ f32x2 looked[kGroup][8][64];  // of the group's chunks before this one; last, the state behind the group before
  __shared__ uint32_t dealt;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t ticket = blockIdx.x;
  if (a.words) {
    if (threadIdx.x == 0)
      dealt = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.words), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    ticket = __builtin_amdgcn_readfirstlane(dealt);
  }
  const int chunk = (int)(ticket / a.tiles), tile = (int)(ticket % a.tiles), ch = tile * kTile + lane * 8;
  const bool mine = ch < a.D;

  // The wave's tokens, in the order of the walk: step i is token first + i, or first - i.
  const int64_t walked = (int64_t)chunk * kChunk + wave * kTok;
  const int64_t first = kBack ? a.N - 1 - walked : walked;
  const auto token = [&](int i) { return kBack ? first - i : first + i; };
  const auto there = [&](int i) { return walked + i < a.N; };
  const auto get = [&](const void* p, int64_t ld, int64_t t, bool in) {
    return in && mine ? load_raw(static_cast<const T*>(p) + t * ld + ch) : zero_raw<T>();
  };
  Raw<T> gate[kTok], in[kTok];  // in: u, or the gradient of h
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    gate[i] = get(a.gate, a.ldg, token(i), there(i));
    in[i] = get(kBack ? a.grad_h : a.u, kBack ? a.ldgh : a.ldu, token(i), there(i));
  }

  // Whose tokens they are: the sequence of each, or -1; whether it is the first or the last.
  const Sequences seqs{a.cu, a.N, a.B};
  int seq[kTok];
  uint32_t begins = 0, ends_here = 0;
  {
    const int64_t low = kBack ? token(kTok - 1) : first;
    int b = seqs.first_behind(low < 0 ? 0 : low);
    int64_t start = b < a.B ? seqs.start(b) : a.N, end = b < a.B ? seqs.end(b) : a.N;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const int i = kBack ? kTok - 1 - j : j;
      const int64_t t = low + j;
      while (b < a.B && end <= t) {
        ++b;
        start = b < a.B ? seqs.start(b) : a.N;
        end = b < a.B ? seqs.end(b) : a.N;
      }
      seq[i] = b < a.B && t >= start && t >= 0 && t < a.N ? b : -1;
      if (seq[i] >= 0 && t == start) begins |= 1u << i;
      if (seq[i] >= 0 && t == end - 1) ends_here |= 1u << i;
    }
  }
  const uint32_t enters = kBack ? ends_here : begins, leaves = kBack ? begins : ends_here;

  // The tokens from a state of zero.  Forward: x = h, and P behind the token.
  // Backward: x = dh; P, before the token in the walk (dh needs the e of the token
  // walked before), is made again with the gates below.
  float x[kTok][8], P[kBack ? 1 : kTok][8];
  f32x2 last[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) last[k] = f32x2{1.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    if (!there(i)) continue;  // a token that is not there leaves the state as it is
    if (enters >> i & 1) {
      const float* from = kBack ? a.state_end : a.state_in;
      float s[8];
      load_state(from ? from + (int64_t)seq[i] * a.D + ch : nullptr, mine, s);
#pragma unroll
      for (int k = 0; k < 8; ++k) last[k] = f32x2{0.0f, s[k]};
    }
    float g[8], v[8];
    unpack8(gate[i], g);
    unpack8(in[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Gate q(g[k]);
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
  for (int k = 0; k < 8; ++k) ends[wave][k][lane] = f32x2{enters ? kFresh : last[k][0], last[k][1]};
  __syncthreads();

  // What the chunk does, for the others; what theirs do, from them.
  if (a.words) {
    const int group = chunk / kGroup, r = chunk % kGroup;
    const bool state = wave == kWaves - 1;
    if (state) {
      uint64_t* to = a.words + chunk_word(chunk, tile, a.tiles) + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f32x2 all = ends[0][k][lane];
#pragma unroll 1
        for (int w = 1; w < kWaves; ++w) all = joined(all, ends[w][k][lane]);
        const float p = all[0] == all[0] ? all[0] : __uint_as_float(0x7fc00000u);  // no word is kAbsent
        __hip_atomic_store(to + 64 * k, word_of(all[1], p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (state ? group > 0 : wave < r) {
      uint64_t v[8];
      const int64_t word = state ? chunk_word(a.chunks + group, tile, a.tiles) : chunk_word(group * kGroup + wave, tile, a.tiles);
      wait_words(a.words + word + lane, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        looked[wave][k][lane] = f32x2{__uint_as_float((uint32_t)(v[k] >> 32)), __uint_as_float((uint32_t)v[k])};
    }
    __syncthreads();
  }
  float carry[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) carry[k] = 0.0f;
  if (a.words) {
    if (chunk >= kGroup)
#pragma unroll
      for (int k = 0; k < 8; ++k) carry[k] = looked[kGroup - 1][k][lane][1];
#pragma unroll 1
    for (int j = 0; j < chunk % kGroup; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) carry[k] = through(looked[j][k][lane], carry[k]);
  }
#pragma unroll 1
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int k = 0; k < 8; ++k) carry[k] = through(ends[w][k][lane], carry[k]);
  if (a.words && wave == kWaves - 1 && chunk % kGroup == kGroup - 1 && chunk + 1 < a.chunks) {
    uint64_t* to = a.words + chunk_word(a.chunks + chunk / kGroup + 1, tile, a.tiles) + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      __hip_atomic_store(to + 64 * k, word_of(through(ends[wave][k][lane], carry[k]), 0.0f), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
  }

  // The state that comes in, applied, and the results.
  Raw<T> us[2], hs[2];  // backward: of two tokens, the next two's on their way
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
      for (int k = 0; k < 8; ++k) carry[k] = 0.0f;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = kBack ? x[i][k] + carry[k] : fmaf(P[kBack ? 0 : i][k], carry[k], x[i][k]);
    const int64_t own = (int64_t)seq[i] * a.D + ch;
    const bool leaving = leaves >> i & 1;
    if constexpr (kBack) {
      float g[8], u[8], h[8], dg[8], du[8], e[8];
      unpack8(gate[i], g);
      unpack8(us[i % 2], u);
      if (leaving) load_state(a.state_in ? a.state_in + own : nullptr, mine, h);
      else unpack8(hs[i % 2], h);
      if (i + 2 < kTok) fetch(i + 2);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const Gate q(g[k]);
        du[k] = q.n * v[k];
        dg[k] = du[k] * (h[k] - u[k]) * (q.keeps ? 1.0f - q.s : q.s);
        e[k] = q.f_times(v[k]);
        carry[k] = q.f_times(carry[k]);
      }
      if (seq[i] >= 0 && mine) {
        store8<true>(static_cast<T*>(a.out) + token(i) * a.ldout + ch, dg);
        store8<true>(static_cast<T*>(a.out2) + token(i) * a.ldout2 + ch, du);
        if (leaving && a.state_out) store8<false>(a.state_out + own, e);
      }
    } else if (seq[i] >= 0 && mine) {
      store8<true>(static_cast<T*>(a.out) + token(i) * a.ldout + ch, v);
      if (leaving && a.state_out) store8<false>(a.state_out + own, v);
    }
  }

  // The states of empty sequences go through unchanged.
  if (a.state_out && mine) {
    const float* from = kBack ? a.state_end : a.state_in;
    for (int64_t b = chunk + (int64_t)a.chunks * wave; b < a.B; b += (int64_t)a.chunks * kWaves) {
      if (seqs.start((int)b) < seqs.end((int)b)) continue;
      float s[8];
      load_state(from ? from + b * a.D + ch : nullptr, true, s);
      store8<false>(a.state_out + b * a.D + ch, s);
    }
  }
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
  load_state(state, mine, s);
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
        const Gate q(g[k]);
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
  return kTicketWords + (chunks + (chunks + kGroup - 1) / kGroup) * tiles * kTile;
}

hipError_t launch_scan(ScanArgs a, int dtype, bool back, void* workspace, hipStream_t stream) {
  const int64_t chunk = tokens_of_chunk(dtype);
  a.tiles = (int)tiles_of(a.D);
  a.chunks = (int)((a.N + chunk - 1) / chunk);
  a.words = a.chunks > 1 ? static_cast<uint64_t*>(workspace) : nullptr;
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
  return hipLaunchKernel(kernel, dim3((unsigned)((int64_t)a.chunks * a.tiles)), dim3(kThreads), args, 0, stream);
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
