// Shared parts of the experts' operators (gfx950): segments of receive rows,
// the tile plan over them, LDS tiles filled by asynchronous loads, and the
// matrix-core main loop.
//
// Every product is computed transposed, D[channel][row] = sum_k A[channel][k]
// B[row][k], so that a lane ends up with four consecutive channels of one
// row; the epilogue turns them around in LDS and stores eight as one 16-byte vector.
#pragma once

#include <type_traits>

#include "ep_device.hpp"
#include "ep_internal.hpp"
#include "experts_choice.hpp"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

#define EP_LDS __attribute__((address_space(3)))
typedef EP_LDS char lds_char;
typedef EP_LDS float lds_float;

// ---- activations -----------------------------------------------------------

// 1 / (1 + exp(-v)) by the hardware's exponential and reciprocal (one unit in
// the last place each): the epilogues have one wave per SIMD, where every
// instruction counts, and a correctly rounded division is ten of them.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

// Gaussian cumulative distribution, 0.5 erfc(-v / sqrt 2), with a relative
// error below 7e-7 for |v| <= 3, growing with the unit in the last place of
// v^2 / 2 beyond (2e-6 at 9, 4e-6 at 12; 1 + erf would cancel for negative v).  For
// x >= 0, erfc(x) = t exp(-x^2 + Q(t)) with t = 2 / (2 + x), the form of Press et al.,
// "Numerical Recipes", section 6.2; Q is a polynomial of our own fit
// to log(erfc(x) exp(x^2) / t) over t in [1/8, 1] (x <= 14, where erfc
// is far below the smallest float) with an error of 1.03e-7 at most.  An epilogue of 64
// values a lane is bound by instructions, and this is a third of erfcf's.
__device__ __forceinline__ float gauss_cdf(float v) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(v), 0.35355339059327376f, 1.0f));
  float q = 0.16099350154399872f;
  q = __builtin_fmaf(q, t, -0.7680159211158752f);
  q = __builtin_fmaf(q, t, 1.361040711402893f);
  q = __builtin_fmaf(q, t, -0.9666953086853027f);
  q = __builtin_fmaf(q, t, 0.14182044565677643f);
  q = __builtin_fmaf(q, t, -0.11564194411039352f);
  q = __builtin_fmaf(q, t, 0.07388374209403992f);
  q = __builtin_fmaf(q, t, 0.3785519301891327f);
  q = __builtin_fmaf(q, t, 0.9995550513267517f);
  q = __builtin_fmaf(q, t, -1.2654922008514404f);
  const float tail = 0.5f * t * __expf(__builtin_fmaf(-0.5f * v, v, q));
  return v < 0.0f ? tail : 1.0f - tail;
}

// one branch for all values
template <int B>
__device__ __forceinline__ void act_each(int act, float (&v)[B][8]) {
  if (act == EP_ACT_SILU) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c) v[b][c] = v[b][c] * sigmoid(v[b][c]);
  } else if (act == EP_ACT_GELU) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c) v[b][c] = v[b][c] * gauss_cdf(v[b][c]);
  } else if (act == EP_ACT_RELU) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c) v[b][c] = v[b][c] < 0.0f ? 0.0f : v[b][c];
  }
}

// act(v) and act'(v); relu's derivative at 0 is 0
__device__ __forceinline__ void act_both(int act, float v, float& value, float& slope) {
  switch (act) {
    case EP_ACT_RELU:
      value = v > 0.0f ? v : (v != v ? v : 0.0f);
      slope = v > 0.0f ? 1.0f : 0.0f;
      return;
    case EP_ACT_SILU: {
      const float t = sigmoid(v);
      value = v * t;
      slope = t * (1.0f + v * (1.0f - t));
      return;
    }
    case EP_ACT_GELU: {
      const float c = gauss_cdf(v);
      value = v * c;
      slope = c + v * __expf(-0.5f * v * v) * 0.39894228040143268f;  // 1 / sqrt(2 pi)
      return;
    }
    default:
      value = v;
      slope = 1.0f;
  }
}

// ---- bf16 ------------------------------------------------------------------

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// fp32 -> bf16 nearest even by v_cvt_pk_bf16_f32 (NaN stays NaN)
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = __builtin_bit_cast(
        uint32_t, __builtin_convertvector((f32x2){f[2 * q], f[2 * q + 1]}, bf16x2));
  return o;
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = bf16_lo(v[q]);
    f[2 * q + 1] = bf16_hi(v[q]);
  }
}

// ---- segments --------------------------------------------------------------

// What of a segment lies past the row buffers is left out and reported.
__device__ __forceinline__ void cut_segment(const Segments& s, int e, int64_t first, int64_t c,
                                            int64_t& start, int& count) {
  if (s.start) {
    start = first;
  } else {
    start = e * s.block_rows;
    c = min(c, s.block_rows);
  }
  if (c <= 0) c = 0;
  if (c > 0 && (start < 0 || start + c > s.cap)) {
    set_err(s.err, EP_DEVERR_CAPACITY);
    c = start < 0 || start >= s.cap ? 0 : s.cap - start;
  }
  count = (int)c;
}

__device__ __forceinline__ void segment_of(const Segments& s, int e, int64_t& start, int& count) {
  cut_segment(s, e, s.start ? s.start[e] : 0, s.count[e], start, count);
}

// The same for a uniform e.  The arrays do not change during the call, so the
// loads are scalar: a vector load would be waited for together with every
// asynchronous load issued before it.
__device__ __forceinline__ void segment_at(const Segments& s, int e, int64_t& start, int& count) {
  typedef const __attribute__((address_space(4))) int32_t* fixed;
  const int32_t c = ((fixed)s.count)[e], first = s.start ? ((fixed)s.start)[e] : 0;
  cut_segment(s, e, first, c, start, count);
}

// ---- tile plan -------------------------------------------------------------

// upto[e] = tiles of `step` rows of the experts up to e.  Every workgroup scans
// the counts itself (E <= 2048 of them, in the shadow of its own start), so a
// call is one launch and needs no workspace.
struct TilePlan {
  int upto[kMaxExperts];
  __device__ __forceinline__ int first(int e) const { return e == 0 ? 0 : upto[e - 1]; }
};

// sums: LDS for an int per wavefront, free afterwards
template <int THREADS>
__device__ void plan_tiles(const Segments& s, int step, TilePlan& p, int* sums) {
  constexpr int kPer = (kMaxExperts + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & 63;
  const int per = (s.E + THREADS - 1) / THREADS;
  int n[kPer], sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    n[i] = 0;
    if (e < s.E) {
      int64_t start;
      int count;
      segment_of(s, e, start, count);
      n[i] = (int)(((uint32_t)count + step - 1) / step);  // count + step may pass 2^31
    }
    sum += n[i];
  }
  int upto = sum;  // inclusive scan over the wavefront
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == kWave - 1) sums[tid / kWave] = upto;
  __syncthreads();
  int at = upto - sum;
  for (int w = 0; w < tid / kWave; ++w) at += sums[w];
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    at += n[i];
    if (e < s.E) p.upto[e] = at;
  }
  __syncthreads();
}

// Expert of tile t (first(e) <= t < upto[e]): two steps of 64 lanes each.
__device__ __forceinline__ int expert_of(const TilePlan& p, int E, int t) {
  const int lane = lane_id();
  const int stride = (E + kWave - 1) / kWave;  // <= 32
  const int far = (lane + 1) * stride - 1;     // the last expert of this lane's stride
  const int skip = __popcll(__ballot(far < E && p.upto[min(far, E - 1)] <= t));
  const int base = skip * stride;
  const int near = base + lane;
  const bool pass = lane < stride && near < E && p.upto[min(near, E - 1)] <= t;
  return uniform(base + __popcll(__ballot(pass)));
}

// ---- LDS tiles -------------------------------------------------------------

// A lane whose 16 bytes lie past the data reads these zeros instead.
static __device__ const uint4 k_zeros[4] = {};

// Asynchronous loads of 16 bytes a lane into LDS (lane i's at dst + 16 i of the
// wave's dst), completed by wait_loads.  They are written as assembly (they
// have no result register) because the compiler waits for every such load of
// its own before the next LDS read, whichever buffer that reads.  M0 holds the
// LDS address; nothing else in these kernels uses it.
__device__ __forceinline__ int lds_offset(const lds_char* p) {
  return uniform((int)(uintptr_t)p);
}

// The base is uniform and in scalar registers.  The compiler may have filled
// those with vector instructions (v_readlane) just before, and does not look
// into assembly for the five wait states that a vector-memory instruction
// needs after such a write; a scalar one needs none, so every block copies the
// base first.  The copy is also the wait state that M0 needs.

// from base + off
__device__ __forceinline__ void load_lds16(const char* base, uint32_t off, const lds_char* dst) {
  const char* from;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(from)
               : "s"(lds_offset(dst)), "v"(off), "s"(base)
               : "memory");
}

// The same of what is read once: past the caches, which other operands are read from.
__device__ __forceinline__ void stream_lds16(const char* base, uint32_t off, const lds_char* dst) {
  const char* from;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0 nt"
               : "=&s"(from)
               : "s"(lds_offset(dst)), "v"(off), "s"(base)
               : "memory");
}

// 4 bytes a lane, or one byte zero-extended to four
template <bool BYTE>
__device__ __forceinline__ void load_lds4(const char* base, uint32_t off, const lds_char* dst) {
  const char* from;
  if (BYTE)
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_ubyte %2, %0"
                 : "=&s"(from)
                 : "s"(lds_offset(dst)), "v"(off), "s"(base)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dword %2, %0"
                 : "=&s"(from)
                 : "s"(lds_offset(dst)), "v"(off), "s"(base)
                 : "memory");
}

// from an address of the lane's own
__device__ __forceinline__ void load_lds16(const char* src, const lds_char* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(lds_offset(dst)), "v"(src)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tile of ROWS rows x KB bytes whose rows are contiguous along the
// contraction.  An asynchronous load stores lane i's 16 bytes at the wave's
// LDS base + 16 i, so the order in LDS is fixed and the lanes choose what
// they fetch: slot j of row r holds chunk j ^ turn(r).  The 64 banks are 256
// bytes wide, 256 / KB rows; a 16-byte read is served 16 lanes at a time, and
// any 16 of them that are four runs of four consecutive rows with different
// row / 4 modulo 4, or sixteen consecutive rows, fall into sixteen different
// columns when turn counts those groups of rows.  (With r modulo 8 alone a
// 128-byte row's reads collided in pairs: 49% of the LDS's active cycles.)
template <int ROWS, int KB = 128>
struct RowTile {
  static constexpr int kBytes = ROWS * KB;
  static constexpr int kChunks = KB / 16;                     // of a row
  static constexpr int kPassRows = 4096 / KB;                 // rows the workgroup fetches at once
  static constexpr int kPasses = (ROWS + kPassRows - 1) / kPassRows;
  static constexpr int kWaveRows = kPassRows / 4;
  static __device__ __forceinline__ int turn(int r) {
    return kChunks >= 16 ? r & 15 : (r / (16 / (kChunks < 16 ? kChunks : 16))) & (kChunks - 1);
  }
  // the chunk that this lane fetches in pass p
  static __device__ __forceinline__ int chunk(int p) {
    const int tid = threadIdx.x;
    return (tid % kChunks) ^ turn(p * kPassRows + tid / kChunks);
  }
  uint32_t off[kPasses];

  // row_of(r): byte offset of tile row r from the tile's base
  template <class F>
  __device__ __forceinline__ void init(F row_of) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      off[p] = row_of((p * kPassRows + tid / kChunks) % ROWS) + chunk(p) * 16;
  }
  // Pass p's load.  base: the tile's first byte of this step; the second half
  // of every PERIOD rows comes from `other` (a gated block's ups).  ONCE: nobody else reads it.
  template <int PERIOD, bool ONCE = false>
  __device__ __forceinline__ void load(int p, const char* base, const char* other,
                                       lds_char* lds) const {
    const int wave = uniform(threadIdx.x >> 6);
    // a wave's rows of a pass are all in one half
    const int r = p * kPassRows + (PERIOD / 2 % kPassRows == 0 ? 0 : wave * kWaveRows);
    if constexpr (ONCE)
      stream_lds16(r % PERIOD >= PERIOD / 2 ? other : base, off[p],
                   lds + (p * 4096 + wave * 1024) % kBytes);
    else
      load_lds16(r % PERIOD >= PERIOD / 2 ? other : base, off[p],
                 lds + (p * 4096 + wave * 1024) % kBytes);
  }
  // the last step of rows with fewer than KB bytes left
  template <int PERIOD>
  __device__ __forceinline__ void load_tail(const char* base, const char* other, int left,
                                            lds_char* lds) const {
    const int wave = uniform(threadIdx.x >> 6);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const bool in = chunk(p) * 16 < left;
      const int r = p * kPassRows + wave * kWaveRows;
      const char* src = (r % PERIOD >= PERIOD / 2 ? other : base) + off[p];
      load_lds16(in ? src : (const char*)k_zeros, lds + (p * 4096 + wave * 1024) % kBytes);
    }
  }
};

// 16-byte chunk c of row r
template <class Tile>
__device__ __forceinline__ i32x4 row_chunk(const lds_char* lds, int r, int c) {
  return *(const EP_LDS i32x4*)(lds + r * (Tile::kChunks * 16) + ((c ^ Tile::turn(r)) << 4));
}

// Tile of KR contraction rows x COLS bf16 whose rows run across the
// contraction (the operand is read transposed).  Slot j of row k holds
// 16-byte chunk j ^ 4 (k & 3): a transposed read takes 32 columns (64 bytes)
// of four consecutive rows, which the exclusive-or sends to four different
// quarters of the banks.
template <int COLS, int KR = 64>
struct ColTile {
  static constexpr int kBytes = KR * COLS * 2;
  static constexpr int kSlots = COLS / 8;
  static constexpr int kPasses = kBytes / 4096;
  static constexpr int kRowsPerPass = kGemmThreads / kSlots;
  static_assert(COLS >= 128 && kRowsPerPass % 4 == 0, "a lane's rows agree modulo 4");
  uint32_t off[kPasses];
  int row;  // this lane's row in pass 0

  // cols: columns the operand has from the tile's first on (a multiple of 8)
  __device__ __forceinline__ void init(uint32_t row_bytes, int cols) {
    const int tid = threadIdx.x;
    row = tid / kSlots;
    const int chunk = (tid % kSlots) ^ ((row & 3) << 2);
#pragma unroll
    for (int p = 0; p < kPasses; ++p)  // past the last column: columns not stored
      off[p] = (row + p * kRowsPerPass) * row_bytes + min(chunk * 16, cols * 2 - 16);
  }
  __device__ __forceinline__ void load(int p, const char* base, lds_char* lds) const {
    load_lds16(base, off[p], lds + p * 4096 + uniform(threadIdx.x >> 6) * 1024);
  }
  // the last step, with fewer than KR contraction rows left
  __device__ __forceinline__ void load_tail(const char* base, int left, lds_char* lds) const {
    const int wave = uniform(threadIdx.x >> 6);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const char* src = base + off[p];
      load_lds16(row + p * kRowsPerPass < left ? src : (const char*)k_zeros,
                 lds + p * 4096 + wave * 1024);
    }
  }
};

__device__ __forceinline__ s16x4 read_tr(const lds_char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((EP_LDS s16x4*)p);
}

// ---- operand fragments -------------------------------------------------------
//
// v_mfma 32x32x16 (MF = 32): lane l holds index l % 32, contraction elements
// 8 (l / 32) .. + 7; 16x16x32 (MF = 16): index l % 16, elements 8 (l / 16) .. + 7.
// Step kk covers contraction elements kk * 512 / MF .. of the tile's 64.

template <int MF, int ROWS, int KB>
__device__ __forceinline__ bf16x8 fragment(const RowTile<ROWS, KB>&, const lds_char* lds, int first,
                                           int kk) {
  const int lane = lane_id();
  return __builtin_bit_cast(bf16x8, row_chunk<RowTile<ROWS, KB>>(
                                        lds, first + lane % MF, kk * (kWave / MF) + lane / MF));
}

// ds_read_b64_tr_b16: of each 16 lanes, lane s gives the address of four
// columns of one row and lane i receives column i of the four rows that lanes
// i / 4 + 4 j (j = 0..3) address: with lane s at row s / 4, columns
// 4 (s % 4), lane i gets rows 0..3 of column i.
template <int MF, int COLS, int KR>
__device__ __forceinline__ bf16x8 fragment(const ColTile<COLS, KR>&, const lds_char* lds, int first,
                                           int kk) {
  const int lane = lane_id();
  const int k = kk * (512 / MF) + 8 * (lane / MF) + (lane % 16) / 4;
  const int col = first + (lane % MF) / 16 * 16 + 4 * (lane % 4);
  const int slot = (col >> 3) ^ ((k & 3) << 2);
  const lds_char* at = lds + k * (COLS * 2) + slot * 16 + (col & 4) * 2;
  union {
    s16x4 half[2];
    bf16x8 all;
  } u;
  u.half[0] = read_tr(at);
  u.half[1] = read_tr(at + 4 * COLS * 2);  // rows k + 4 ..: same residue modulo 4
  return u.all;
}

// FP8: 128 contraction bytes a tile; 32x32x64 takes 32 bytes a lane, 16x16x128
// too.  Which contraction elements a lane takes is free as long as both
// operands agree.
template <int MF, int ROWS, int KB>
__device__ __forceinline__ i32x8 fragment8(const RowTile<ROWS, KB>&, const lds_char* lds, int first, int kk) {
  const int lane = lane_id();
  typedef RowTile<ROWS, KB> Tile;
  const int r = first + lane % MF, c = 2 * (kk * (kWave / MF) + lane / MF);
  const i32x4 a = row_chunk<Tile>(lds, r, c), b = row_chunk<Tile>(lds, r, c + 1);
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <int MF>
struct Mfma;
template <>
struct Mfma<32> {
  typedef f32x16 acc_t;
  static __device__ __forceinline__ acc_t bf16(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ acc_t fp8(i32x8 a, i32x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
  }
  static __device__ __forceinline__ acc_t int8(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_bit_cast(acc_t, __builtin_amdgcn_mfma_i32_32x32x32_i8(
                                         __builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                         __builtin_bit_cast(i32x16, c), 0, 0, 0));
  }
};
template <>
struct Mfma<16> {
  typedef f32x4 acc_t;
  static __device__ __forceinline__ acc_t bf16(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ acc_t fp8(i32x8 a, i32x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
  }
  static __device__ __forceinline__ acc_t int8(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_bit_cast(acc_t, __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                         __builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                         __builtin_bit_cast(i32x4, c), 0, 0, 0));
  }
};

// One product of 16-byte fragments.  8-bit integers take the places of half as many bf16:
// a lane's 16 consecutive ones of a row, 32x32x32 and 16x16x64.  Their sums are 32-bit
// integers (exact up to 2^17 channels), kept in the same registers as bits until
// sum_value converts them.
template <int MF, bool INT8>
__device__ __forceinline__ typename Mfma<MF>::acc_t product(bf16x8 a, bf16x8 b,
                                                            typename Mfma<MF>::acc_t c) {
  if constexpr (INT8) return Mfma<MF>::int8(a, b, c);
  else return Mfma<MF>::bf16(a, b, c);
}

template <bool INT8>
__device__ __forceinline__ float sum_value(float bits) {
  return INT8 ? (float)__float_as_int(bits) : bits;
}

// First of the four consecutive channels that accumulator registers 4 q .. 4 q + 3
// of a lane hold.
template <int MF>
__device__ __forceinline__ int channel_of(int q) {
  return MF == 32 ? 8 * q + 4 * (lane_id() / 32) : 4 * (lane_id() / 16);
}

// A tile's dimensions, and this wave's place in it.
template <class D>
struct Shape : D {
  static_assert(kWavefront == kWave, "");
  typedef typename Mfma<D::MF>::acc_t acc_t;
  int wc, wr, wk;
  __device__ __forceinline__ Shape() {
    const int wave = uniform(threadIdx.x >> 6);
    wc = wave % D::WC;
    wr = wave / D::WC % D::WT;
    wk = wave / (D::WC * D::WT);
  }
};

// Tile t of mt row tiles x nt channel tiles.  Row tiles are taken in groups
// of kGroup, a group's channel tiles one after another with its row tiles
// fastest, so the workgroups that run together share both operands; each
// die (block b runs on die b % kXcds) takes a run of them.
constexpr int kGroup = 8;

__device__ __forceinline__ void tile_at(int64_t t, int mt, int nt, int& m, int& n) {
  const int64_t per = (int64_t)kGroup * nt;
  const int g = (int)(t / per);
  const int in = (int)(t - g * per);
  const int rows = min(kGroup, mt - g * kGroup);
  n = uniform(in / rows);
  m = uniform(g * kGroup + in - n * rows);
}

// This workgroup's place among gridDim.x (a multiple of kXcds, or below it)
__device__ __forceinline__ int block_place() {
  const int g = gridDim.x, b = blockIdx.x;
  return g % kXcds == 0 ? (b % kXcds) * (g / kXcds) + b / kXcds : b;
}

// ---- main loop ---------------------------------------------------------------

template <class S>
__device__ __forceinline__ void clear(typename S::acc_t (&acc)[S::CT][S::TT]) {
#pragma unroll
  for (int i = 0; i < S::CT; ++i)
#pragma unroll
    for (int j = 0; j < S::TT; ++j)
#pragma unroll
      for (int q = 0; q < S::REGS; ++q) acc[i][j][q] = 0.0f;
}

// One tile after another with STAGES >= 3 buffers in a ring.  While stage k is
// multiplied, stage k + STAGES - 1 is loaded into the buffer that stage k - 1
// left; towards a tile's end those are the next tile's first stages, so the
// loads never stop and the epilogue (which turns its sums around in the last
// stage's buffer) runs while they arrive.  With 16 stages a tile (FP8, 2,048
// channels) a third of the time had gone into starting and ending tiles.
//
// Job: nk stages a tile, the first nfull of them full; setup(t) points the
//   loads at tile t and returns what its epilogue needs; load(k, slot, p) issues
//   pass p (of kPasses) of stage k's loads into a buffer, kLoads a wave in all;
//   tail(k, slot) a short last stage's; epilogue(tile, region) stores.
// Engine: first(slot) reads what the first stage begins with; stage(slot, next,
//   issue, mid) multiplies the stage in `slot`, calls issue(p) for p = 0 ..
//   kPasses - 1 spread between the products, and mid() once this stage's
//   buffer is read out and before it reads from buffer `next`.  By then it has
//   made kIssued of the issue calls.
template <class S, bool CHAIN, class Job, class Engine>
__device__ __forceinline__ void run_ring(Job& job, Engine& engine, lds_char* lds, int64_t t,
                                         int64_t tiles, bool may_chain) {
  constexpr int N = S::STAGES, kSlot = S::kSlotBytes;
  static_assert(N >= 3, "a stage is loaded while another one waits");
  if (t >= tiles) return;
  auto after = [](int slot) { return slot + 1 == N ? 0 : slot + 1; };
  auto before = [](int slot) { return slot == 0 ? N - 1 : slot - 1; };
  auto load_any = [&](int k, int slot) {
    if (k < job.nfull) {
#pragma unroll
      for (int p = 0; p < Job::kPasses; ++p) job.load(k, slot, p);
    } else {
      job.tail(k, slot);
    }
  };
  const bool chain = CHAIN && may_chain && job.nk >= N;
  auto tile = job.setup(t);
  bool fresh = true;
  int slot = 0;
  for (;;) {
    if (fresh) {
      barrier();  // the previous tile's epilogue
      slot = 0;
#pragma unroll
      for (int k = 0; k < N - 1; ++k)
        if (k < job.nk) load_any(k, k);
      if (N - 2 < job.nk) wait_loads<Job::kLoads*(N - 2)>();
      else wait_loads<0>();
      barrier();
      engine.first(slot);
    }
    engine.clear();
    const int64_t then = t + gridDim.x;
    const bool more = chain && then < tiles;
    auto next = tile;
    int k = 0;
    for (; k + N - 1 < job.nfull; ++k) {
      const int into = before(slot);
      engine.template stage<true>(
          slot, after(slot), [&](int p) { job.load(k + N - 1, into, p); },
          [&]() {
            // stage k + 1 has arrived; younger: the stages between and what
            // of stage k + N - 1 has been issued
            wait_loads<Job::kLoads*(N - 3) + Engine::kIssued>();
            barrier();
          });
      slot = after(slot);
    }
    for (; k < job.nk; ++k) {
      const int ahead = k + N - 1;
      if (ahead < job.nk) {
        job.tail(ahead, before(slot));
      } else if (more) {
        if (ahead == job.nk) next = job.setup(then);
        load_any(ahead - job.nk, before(slot));
      }
      engine.template stage<false>(
          slot, after(slot), [](int) {},
          [&]() {
            if (more) wait_loads<Job::kLoads*(N - 2)>();
            else wait_loads<0>();
            barrier();
          });
      slot = after(slot);
    }
    job.epilogue(tile, chain ? lds + before(slot) * kSlot : lds);
    t = then;
    if (t >= tiles) return;
    fresh = !chain;
    if (chain) {
      tile = next;
      barrier();  // the epilogue's buffer is loaded next
    } else {
      tile = job.setup(t);
    }
  }
}

// bf16.  The loads and the reads of the next step's fragments are spread evenly
// between the products and the order is pinned: a wave's loads issued together
// wait for each other, and left to itself the compiler moves the products
// before the barrier and the reads behind it, which leaves the matrix cores
// idle for a barrier and an LDS round trip per stage.  A stage's last products
// cover the barrier and the next stage's first reads.
template <class S, class Chan, class Row, bool INT8 = false>
struct RingEngine {
  static constexpr int CT = S::CT, TT = S::TT, KK = S::KK;
  static constexpr int kSlot = Chan::kBytes + Row::kBytes;
  static constexpr int kPasses = Chan::kPasses + Row::kPasses;
  static constexpr int kGroups = KK * CT;
  static constexpr int kIssued = (KK - 1) * CT * kPasses / kGroups;
  static_assert(KK % 2 == 0, "a stage ends on the fragments it began with");
  typename S::acc_t acc[CT][TT];
  bf16x8 fa[2][CT], fb[2][TT];
  lds_char* lds;
  S at;

  __device__ __forceinline__ explicit RingEngine(lds_char* l) : lds(l) {}
  __device__ __forceinline__ void read_chan(int slot, int kk, int to, int i) {
    fa[to][i] = fragment<S::MF>(Chan(), lds + slot * kSlot, (at.wc * CT + i) * S::MF,
                                at.wk * KK + kk);
  }
  __device__ __forceinline__ void read_row(int slot, int kk, int to, int j) {
    fb[to][j] = fragment<S::MF>(Row(), lds + slot * kSlot + Chan::kBytes, (at.wr * TT + j) * S::MF,
                                at.wk * KK + kk);
  }
  __device__ __forceinline__ void clear() { ep::clear<S>(acc); }
  __device__ __forceinline__ void first(int slot) {
#pragma unroll
    for (int i = 0; i < CT; ++i) read_chan(slot, 0, 0, i);
#pragma unroll
    for (int j = 0; j < TT; ++j) read_row(slot, 0, 0, j);
  }
  template <bool LOADS, class Issue, class Mid>
  __device__ __forceinline__ void stage(int slot, int next, Issue issue, Mid mid) {
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int from = kk & 1;
      if (kk == KK - 1) mid();
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        if constexpr (LOADS) {
          const int g = kk * CT + i;
#pragma unroll
          for (int p = g * kPasses / kGroups; p < (g + 1) * kPasses / kGroups; ++p) issue(p);
        }
        const int s = kk == KK - 1 ? next : slot, n = kk == KK - 1 ? 0 : kk + 1;
        read_chan(s, n, from ^ 1, i);
#pragma unroll
        for (int j = i * TT / CT; j < (i + 1) * TT / CT; ++j) read_row(s, n, from ^ 1, j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TT; ++j)
          acc[i][j] = product<S::MF, INT8>(fa[from][i], fb[from][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
};

// FP8: the products of a 128-channel group are summed on the matrix cores and
// added to the fp32 sums times the row's and the weight block's scale.  The matrix
// cores' FP8 instructions, scaled or not, add eight products at a time (of eight
// consecutive channels) and cut each off 13 bits below the largest of them; what they
// add these to has fp32's 24 bits.  On normally distributed rows and weights that
// leaves a relative error of 2^-16 (2-norm); the result's rounding to bf16 is 2^-9.
// Codes converted to bf16 would be summed without it, at half the rate (2.5
// against 5 PFLOP/s at peak) and with the conversion on top.
template <class S, class Chan, class Row, bool GATED, int Q>
struct RingEngine8 {
  static constexpr int CT = S::CT, TT = S::TT, MF = S::MF;
  static constexpr int kSlot = Chan::kBytes + Row::kBytes;
  static constexpr int kPasses = Chan::kPasses + Row::kPasses;
  static constexpr int GS = S::GS, kSteps = S::KK8 / GS;
  static constexpr int kScales = S::kScaleFloats;
  static constexpr int kIssued = kPasses + GS * S::SLOADS + 1;  // all loads
  typename S::acc_t acc[CT][TT];
  lds_char* lds;
  lds_float* scales;
  S at;

  __device__ __forceinline__ RingEngine8(lds_char* l, lds_float* s) : lds(l), scales(s) {}
  __device__ __forceinline__ void clear() { ep::clear<S>(acc); }
  __device__ __forceinline__ void first(int) {}
  template <bool LOADS, class Issue, class Mid>
  __device__ __forceinline__ void stage(int slot, int, Issue issue, Mid mid) {
    const lds_char* wl = lds + slot * kSlot;
    const lds_char* xl = wl + Chan::kBytes;
    const lds_float* sc = scales + (slot * 4 + uniform(threadIdx.x >> 6)) * kScales;
    const int lane = lane_id(), first = at.wk * GS;
#pragma unroll
    for (int g = 0; g < GS; ++g) {
      const float w0 = sc[GS * S::SLOADS * kWave + 2 * g];
      const float w1 = sc[GS * S::SLOADS * kWave + 2 * g + 1];
      float sx[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const float s = sc[g * S::SLOADS * kWave + j * MF + lane % MF];
        sx[j] = Q == EP_QUANT_FP8_F32 ? s : __builtin_ldexpf(1.0f, __float_as_int(s) - 127);
      }
      i32x8 fb[TT][kSteps];
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          fb[j][kk] = fragment8<MF>(Row(), xl, (at.wr * TT + j) * MF, (first + g) * kSteps + kk);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        if constexpr (LOADS) {
          constexpr int kGroups = GS * CT;
          const int u = g * CT + i;
#pragma unroll
          for (int p = u * kPasses / kGroups; p < (u + 1) * kPasses / kGroups; ++p) issue(p);
        }
        i32x8 fa[kSteps];
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          fa[kk] = fragment8<MF>(Chan(), wl, (at.wc * CT + i) * MF, (first + g) * kSteps + kk);
        const float w = GATED && i >= CT / 2 ? w1 : w0;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          typename S::acc_t part;
#pragma unroll
          for (int q = 0; q < S::REGS; ++q) part[q] = 0.0f;
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) part = Mfma<MF>::fp8(fa[kk], fb[j][kk], part);
          const float s = sx[j] * w;
#pragma unroll
          for (int q = 0; q < S::REGS; ++q)
            acc[i][j][q] = __builtin_fmaf(part[q], s, acc[i][j][q]);
        }
      }
    }
    mid();
  }
};

// acc += a tile's nk stages, for tiles so large that only two stages fit (256 x
// 256: their fragments, 128 registers a lane, are the third).  load(k, buf, p)
// issues pass p of stage k's loads into buffer buf (first the channel operand's
// passes, then the row operand's); tail(k, buf) all loads of a short last
// stage; the first nfull stages are full.  Fragment set s (the
// operands of step s, four steps a stage) is read one step after the products
// that used its registers:
//   step 0 of stage k:  reads set 3 of stage k; then buffer k is read out
//   barrier:            ... and stage k + 1 has arrived in the other one
//   steps 1, 2, 3:      read sets 0, 1, 2 of stage k + 1; steps 1 and 2 load
//                       stage k + 2 into buffer k
// so a load has two to four steps (16 products of 32 cycles a wave each) to
// arrive and rows are fetched as whole 128-byte lines.  64-byte stages, four
// of which fit, were tried first: their loads alone take 1.54 ms at 16
// experts x 2,048 rows x 7168 x 4096, those of 128 bytes 1.04 ms.
template <class S, bool INT8 = false, class Chan, class Row, class Load, class Tail>
__device__ __forceinline__ void products_deep(const Chan& ct, const Row& rt, lds_char* lds, int nk,
                                              int nfull, Load load, Tail tail,
                                              typename S::acc_t (&acc)[S::CT][S::TT]) {
  constexpr int kStage = Chan::kBytes + Row::kBytes;
  constexpr int kLoads = Chan::kPasses + Row::kPasses;
  constexpr int CT = S::CT, TT = S::TT;
  constexpr int KK = S::KK;
  static_assert(S::STAGES == 2 && KK % 2 == 0, "");
  const S at;
  const int wc = at.wc, wr = at.wr;
  auto load_any = [&](int k, lds_char* buf) {
    if (k < nfull) {
#pragma unroll
      for (int p = 0; p < kLoads; ++p) load(k, buf, p);
    } else if (k < nk) {
      tail(k, buf);
    }
  };
  if (nk == 0) return;
  barrier();  // the previous tile's reads
  load_any(0, lds);
  load_any(1, lds + kStage);
  if (nk > 1)
    wait_loads<kLoads>();
  else
    wait_loads<0>();
  barrier();
  bf16x8 fa[KK][CT], fb[KK][TT];
  auto read = [&](lds_char* buf, int set, int n) {  // the n-th fragment of a set
    if (n < CT)
      fa[set][n] = fragment<S::MF>(ct, buf, (wc * CT + n) * S::MF, set);
    else
      fb[set][n - CT] = fragment<S::MF>(rt, buf + Chan::kBytes, (wr * TT + n - CT) * S::MF, set);
  };
  constexpr int kFrags = CT + TT;
  // Step s's products, one at a time: before each at most one read of `set`
  // (all in the first half of step 0, whose barrier waits for them) or one of
  // stage k's loads.  With one wave per SIMD the few instructions between two
  // products have to fit into the time of one, 32 cycles.
  constexpr int kProducts = CT * TT, kStepLoads = kLoads / (KK / 2);
  static_assert(kLoads % (KK / 2) == 0 && kStepLoads <= kProducts, "");
  auto step = [&](int s, lds_char* buf, int set, auto loads, int k, lds_char* into) {
#pragma unroll
    for (int m = 0; m < kProducts; ++m) {
      const int i = m / TT, j = m % TT;
      const int span = s == 0 ? kProducts / 2 : kProducts;
#pragma unroll
      for (int n = 0; n < kFrags; ++n)
        if (n * span / kFrags == m) read(buf, set, n);
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int l = 0; l < kStepLoads; ++l)
          if ((2 * l + 1) * kProducts / (2 * kStepLoads) == m)
            load(k, into, (s - 1) * kStepLoads + l);
      }
      __builtin_amdgcn_sched_barrier(0);
      acc[i][j] = product<S::MF, INT8>(fa[s][i], fb[s][j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
#pragma unroll
  for (int set = 0; set < KK - 1; ++set)
#pragma unroll
    for (int n = 0; n < kFrags; ++n) read(lds, set, n);
  lds_char* buf = lds;
  lds_char* other = lds + kStage;
  int k = 0;
  for (; k + 2 < nfull; ++k) {
    step(0, buf, KK - 1, no, 0, nullptr);
    wait_loads<0>();
    barrier();
#pragma unroll
    for (int s = 1; s <= KK / 2; ++s) step(s, other, s - 1, yes, k + 2, buf);
#pragma unroll
    for (int s = KK / 2 + 1; s < KK; ++s) step(s, other, s - 1, no, 0, nullptr);
    lds_char* t = buf;
    buf = other;
    other = t;
  }
  for (; k < nk; ++k) {  // the last stages; past the last one the reads go unused
    step(0, buf, KK - 1, no, 0, nullptr);
    wait_loads<0>();
    barrier();
    if (k + 2 < nk) tail(k + 2, buf);
#pragma unroll
    for (int s = 1; s < KK; ++s) step(s, other, s - 1, no, 0, nullptr);
    lds_char* t = buf;
    buf = other;
    other = t;
  }
}

// Epilogue: a wave turns MF rows at a time around in its own part of the LDS,
// so that eight consecutive channels of one row meet in a lane and rows leave
// as whole 16-byte vectors.  A row's quads of channels lie in two halves, the
// even ones and the odd ones: both a lane's two reads and the writes then
// fall into all banks once.
template <class S>
struct Turned {
  static constexpr int kHalf = S::kHalfBytes;
  static constexpr int kRowBytes = S::kTurnRowBytes;  // 16 more than two halves: rows start four banks apart
  const lds_char* at;
  // eight channels, `further` channels on (a multiple of 8); the sum of the
  // waves' parts of the contraction, in their order
  __device__ __forceinline__ void get(int further, float (&f)[8]) const {
    f32x4 a = *(const EP_LDS f32x4*)(at + further * 2);
    f32x4 b = *(const EP_LDS f32x4*)(at + kHalf + further * 2);
#pragma unroll
    for (int w = 1; w < S::WK; ++w) {
      constexpr int kPart = S::WC * S::WT * S::MF * kRowBytes;  // the waves of one part
      a += *(const EP_LDS f32x4*)(at + w * kPart + further * 2);
      b += *(const EP_LDS f32x4*)(at + w * kPart + kHalf + further * 2);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = a[q], f[4 + q] = b[q];
  }
};

// What a lane of turn_out stores: channels from `channel` on of the first OUT channel
// tiles of the waves in column wc, the same for all its rows.
template <class S, int OUT>
struct TurnLane {
  static constexpr int kVecs = OUT * S::MF / 8;  // vectors of a row
  // threads that turn a region together: a wave, or those that share a tile
  static constexpr int kThreads = S::WK > 1 ? kGemmThreads / S::WC : kWave;
  static constexpr int kRows = kThreads / kVecs;  // rows at once
  static constexpr int kTurns = kRows >= S::MF ? 1 : S::MF / kRows;
  static constexpr int kBatch = kTurns < 4 ? kTurns : 4;  // rows that a lane stores together
  int wc, row, channel;
  __device__ __forceinline__ TurnLane() {
    const int id = threadIdx.x % kThreads;
    wc = S::WK > 1 ? uniform(threadIdx.x / kThreads) : S().wc;
    row = id / kVecs;
    channel = id % kVecs * 8;
  }
};

// Rows r, r + kRows, ..: fetch(r) loads what a row's result needs from memory, one turn
// ahead: a load behind a store waits for the store as well (linear product with
// residual, 64 experts x 2,048 rows, 2048 x 7168: 4.23 -> 3.72 ms).  put(r, turned,
// fetched) takes kBatch rows.
template <class S, int OUT, bool INT8 = false, class Fetch, class Put>
__device__ __forceinline__ void turn_out(lds_char* lds, const typename S::acc_t (&acc)[S::CT][S::TT],
                                         Fetch fetch, Put put) {
  typedef Turned<S> T;
  typedef TurnLane<S, OUT> Lane;
  constexpr int MF = S::MF, kTurns = Lane::kTurns, kBatch = Lane::kBatch;
  const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
  const S place;
  const Lane at;
  decltype(fetch(0)) fetched[2][kTurns];
  auto fetch_all = [&](int j) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
      fetched[j & 1][i] = fetch((place.wr * S::TT + j) * MF + at.row + i * Lane::kRows);
  };
  fetch_all(0);
  barrier();
  lds_char* mine = lds + wave * (MF * T::kRowBytes);
  const lds_char* from =
      (S::WK > 1 ? lds + at.wc * (MF * T::kRowBytes) : mine) + at.row * T::kRowBytes + at.channel * 2;
#pragma unroll
  for (int j = 0; j < S::TT; ++j) {
    if (j + 1 < S::TT) fetch_all(j + 1);
    lds_char* to = mine + (lane % MF) * T::kRowBytes;
#pragma unroll
    for (int i = 0; i < S::CT; ++i)
#pragma unroll
      for (int q = 0; q < S::REGS / 4; ++q) {
        const f32x4 v = {
            sum_value<INT8>(acc[i][j][4 * q]), sum_value<INT8>(acc[i][j][4 * q + 1]),
            sum_value<INT8>(acc[i][j][4 * q + 2]), sum_value<INT8>(acc[i][j][4 * q + 3])};
        const int quad = (i * MF + channel_of<MF>(q)) / 4;
        *(EP_LDS f32x4*)(to + (quad & 1) * T::kHalf + (quad >> 1) * 16) = v;
      }
    static_assert(S::WK == 1 || (S::WT == 1 && S::TT == 1), "one region for the waves of a tile");
    if (S::WK > 1) barrier();
    else wave_lds_sync();
    if (Lane::kRows <= MF || at.row < MF) {
#pragma unroll
      for (int i = 0; i < kTurns; i += kBatch) {
        T turned[kBatch];
        decltype(fetch(0)) own[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          turned[b].at = from + (i + b) * Lane::kRows * T::kRowBytes;
          own[b] = fetched[j & 1][i + b];
        }
        put((place.wr * S::TT + j) * MF + at.row + i * Lane::kRows, turned, own);
      }
    }
    if (S::WK == 1) wave_lds_sync();
  }
}

}  // namespace ep
