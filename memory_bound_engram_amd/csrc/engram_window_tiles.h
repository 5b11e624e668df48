// engram_window_tiles.h -- tiles and matrix products of the window attention's
// kernels (gfx950, internal).
//
// The 32x32x16 product.  Operands: lane l holds row (or column) l % 32 and, with
// h = l / 32, the eight contraction indices 8h .. 8h+7.  Accumulator: lane l has
// column l % 32, and its value i is row 8 (i / 4) + 4 h + i % 4.  Two neighbouring
// quarters of an accumulator, rounded, are so an operand of a product that
// contracts over its rows, with index 8h + e standing for row 8 (e / 4) + 4 h + e % 4;
// the other operand is read in that order.
#pragma once

#include "engram_layers_device.h"
#include "engram_values.h"
#include "engram_window_bounds.h"

namespace engram {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) const void* lds_ptr;

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

template <typename T>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (__is_same(T, bf16_t))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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
// Half m of an accumulator as an operand.
template <typename T>
__device__ __forceinline__ u32x4 operand(const f32x16& v, int m) {
  return u32x4{pack2<T>(v[8 * m], v[8 * m + 1]), pack2<T>(v[8 * m + 2], v[8 * m + 3]),
               pack2<T>(v[8 * m + 4], v[8 * m + 5]), pack2<T>(v[8 * m + 6], v[8 * m + 7])};
}

// Sum and maximum over the two lanes that share a column, in both.
__device__ __forceinline__ float column_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float column_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// A tile in LDS: rows of kD (64 or 128) values without gaps, the 16-byte pieces
// of row r in the order piece ^ turn(r).  LDS serves sixteen lanes of a 16-byte
// read at once, here sixteen rows that differ modulo 16, of one piece; and
// thirty-two of a transposing one, four rows of four neighbouring pieces.  With this
// order both find their values in different banks.
template <int kD>
__device__ __forceinline__ uint32_t turn(uint32_t row) {
  return kD == 128 ? (row & 3) << 2 | (row >> 2 & 3) : (row >> 1 & 1) << 2 | (row >> 2 & 3);
}
template <int kD>
__device__ __forceinline__ uint32_t place(uint32_t row, uint32_t col) {
  return row * kD + ((col >> 3) ^ turn<kD>(row)) * 8 + (col & 7);
}

// A tile's place as LDS sees it.
typedef __attribute__((address_space(3))) const char* lds_bytes;
__device__ __forceinline__ lds_bytes lds_of(const uint16_t* tile) { return (lds_bytes)(lds_ptr)tile; }
// What lies at a place of LDS; and through the transposing read, at two.
__device__ __forceinline__ u32x4 lds_read(uint32_t at) {
  typedef __attribute__((address_space(3))) const u32x4* words;
  return *(words)(lds_bytes)(uintptr_t)at;
}
__device__ __forceinline__ u32x4 lds_read_turned(uint32_t lo, uint32_t hi) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds_bytes)(uintptr_t)lo));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds_bytes)(uintptr_t)hi));
  return u32x4{a[0], a[1], b[0], b[1]};
}

// An operand whose rows are rows of the tile, row0 + l % 32 (row0 a multiple of
// 32), values 16 kk + 8 h on.
template <int kD>
struct RowReader {
  uint32_t at, swap;  // of row l % 32, in bytes
  __device__ __forceinline__ explicit RowReader(uint32_t lane)
      : at((lane & 31) * kD * 2), swap((turn<kD>(lane & 31) ^ (lane >> 5)) * 16) {}
  __device__ __forceinline__ u32x4 operator()(lds_bytes tile, int row0, int kk) const {
    return lds_read((uint32_t)(uintptr_t)tile + (at + ((32 * kk) ^ swap)) + row0 * kD * 2);
  }
};

// An operand whose rows are columns of the tile, 32 dt + l % 32, and whose
// contraction runs down the tile's rows row0 .. row0 + 15 in the order of an
// accumulator's rows, through the transposing LDS read: the sixteen lanes of a
// group name four rows of sixteen values and get a column of four each.
template <int kD>
struct ColumnReader {
  uint32_t at[2][kD / 32];  // of the rows' first eight and the second, in bytes
  __device__ __forceinline__ explicit ColumnReader(uint32_t lane) {
    const uint32_t l = lane % 16, row = 4 * (lane >> 5) + l / 4, col = 16 * (lane >> 4 & 1) + 4 * (l % 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int dt = 0; dt < kD / 32; ++dt) at[i][dt] = place<kD>(row + 8 * i, col + 32 * dt) * 2;
  }
};

// load_to_lds by some of the lanes (all are at work here); the others' places stay as they are.
__device__ __forceinline__ void load_some_to_lds(uint32_t to, u32x4 src, uint32_t off, uint64_t lanes) {
  uint64_t all;
  asm volatile("s_mov_b64 %0, exec\n\ts_mov_b32 m0, %1\n\ts_mov_b64 exec, %4\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
               "s_mov_b64 exec, %0"
               : "=&s"(all)
               : "s"(to), "v"(off), "s"(src), "s"(lanes)
               : "memory");
}

// The pieces of a tile that a lane of kThreads moves: the q-th lies at
// (q kThreads + thread) 16 bytes of the tile.
template <int kD, int kRows, int kThreads>
struct Pieces {
  static constexpr int kMoves = kRows * kD / 8 / kThreads;
  static constexpr int kStep = kThreads * 8 / kD;  // rows between a lane's pieces
  static_assert(kMoves * kThreads * 8 == kRows * kD, "");
  // the order of the pieces repeats every 16 rows: else a lane's column is another for each
  static constexpr bool kSame = kStep % 16 == 0;
  uint32_t row, col;  // of the first
  __device__ __forceinline__ explicit Pieces(uint32_t thread)
      : row(thread / (kD / 8)), col(((thread % (kD / 8)) ^ turn<kD>(thread / (kD / 8))) * 8) {}
  // The place of the first piece, in bytes from a tile's first row, where rows are
  // ld values apart.
  __device__ __forceinline__ uint32_t offset(int64_t ld, int D) const {
    static_assert(kSame, "one offset serves all of a lane's pieces");
    return col < (uint32_t)D ? row * (uint32_t)(ld * 2) + col * 2 : kBeyond;
  }
  // Of n rows (n may be more than the tile has; what is not there is zeros, the memory's
  // bound sees to it) from src on, ld apart, the q-th pieces; `at`: the above.  No vector
  // instruction but the load.
  __device__ __forceinline__ void move(int q, const uint16_t* tile, const uint16_t* src, int64_t ld, int n, int D, uint32_t at,
                                       uint32_t wave) const {
    load_to_lds(lds_place(q, tile, wave), words_of(q, src, ld, n, D), at);
  }
  // Those of the lanes in `some`.
  __device__ __forceinline__ void move_some(int q, const uint16_t* tile, const uint16_t* src, int64_t ld, int n, int D,
                                            uint32_t at, uint32_t wave, uint64_t some) const {
    load_some_to_lds(lds_place(q, tile, wave), words_of(q, src, ld, n, D), at, some);
  }
  static __device__ __forceinline__ uint32_t lds_place(int q, const uint16_t* tile, uint32_t wave) {
    return (uint32_t)(uintptr_t)(lds_ptr)tile + wave * 1024 + q * kThreads * 16;
  }
  static __device__ __forceinline__ u32x4 words_of(int q, const uint16_t* src, int64_t ld, int n, int D) {
    u32x4 words = buffer_words(src + (int64_t)(q * kStep) * ld);
    words[2] = readable_bytes(n - q * kStep, kStep, ld, D);
    return words;
  }
  __device__ __forceinline__ void fetch(const uint16_t* tile, const uint16_t* src, int64_t ld, int n, int D, uint32_t at,
                                        uint32_t wave) const {
#pragma unroll
    for (int q = 0; q < kMoves; ++q) move(q, tile, src, ld, n, D, at, wave);
  }
  // Rows wherever they are: `where(row)` in bytes from src, or kBeyond.
  template <typename F>
  __device__ __forceinline__ void gather(const uint16_t* tile, const void* src, int D, uint32_t wave, F where) const {
    const u32x4 words = buffer_words(src);
    const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr)tile + wave * 1024;
#pragma unroll
    for (int q = 0; q < kMoves; ++q) {
      const uint32_t from = where(row + q * kStep);
      const uint32_t c = kSame ? col : col ^ (turn<kD>(row) ^ turn<kD>(row + q * kStep)) * 8;
      load_to_lds(to + q * kThreads * 16, words, c < (uint32_t)D && from != kBeyond ? from + c * 2 : kBeyond);
    }
  }
};

// This wave's loads (into LDS too) and LDS accesses are done; then all waves'.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt 0, lgkmcnt 0
  __syncthreads();
}

// x / G for x < 2^22, without a branch.
struct Divide {
  uint32_t inverse, more;  // ceil(2^32 / G); for G = 1 (x + 1) (2^32 - 1) / 2^32 is x
  __device__ __host__ __forceinline__ explicit Divide(uint32_t G)
      : inverse(G > 1 ? (uint32_t)((0x100000000ull + G - 1) / G) : 0xffffffffu), more(G == 1) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return __umulhi(x + more, inverse); }
};

}  // namespace
}  // namespace engram
