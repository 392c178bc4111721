// Matrix products grouped by expert on microscaled 4-bit weights (MXFP4: e2m1
// codes, one e8m0 scale per 32 values of a row), for rows in bf16 or in MXFP4.
//
//   out[r][n] = sum_d a(r)[d] * w_e[n][d],  r in expert e's span of offsets
//
// What bounds it.  Up to some 200 MXFP4 rows an expert (100 bf16 rows) the
// weights' 17/32 byte a value, past that the matrix cores.  So one block takes
// up to 192 (128) rows of one expert, and a weight byte is loaded once:
//   - a wave owns 16 CB weight rows and every row of the tile, so no two waves
//     load the same weights; they come as whole lines into registers, one
//     512-value chunk of each row ahead of its use, and pass through LDS of
//     the wave's own to become fragments;
//   - weights are the first operand, rows the second: a lane then holds 4
//     consecutive weight rows' products with one row, and the weight rows are
//     dealt to the instructions so that its outputs go out 16 bytes at a time,
//     next to its neighbour's;
//   - the rows go through LDS, in tiles of 256 bytes a row (512 4-bit values
//     or 128 bf16), two stages, the 16-byte pieces XOR-swizzled by the row;
//   - more than 16 rows: 32 x 32 instructions.  On registers alone and random
//     data this card does 5.6 PFLOP/s of MXFP4 with 16 x 16 and 7.4 with 32 x
//     32, in bf16 1.4 and 1.8.
// MXFP4 rows: v_mfma_scale_f32_*_f8f6f4, both scales applied by the instruction
// (a lane holds one 32-value block of its row, and its scale).  bf16 rows: the
// 32 codes of a lane become four 8-value fragments of v_mfma_f32_*_bf16 (exact:
// e2m1 times a power of two has two significant bits), the rows' fragments taken
// at the same values.  Sums are fp32 in both.
//
// Measured: 8146 rows of 6144 on 64 experts of 4096 x 6144 with SwiGLU (127 rows
// an expert), 212 us, 4.3 TB/s of what has to be moved; one row an expert, down
// weights of 6144 x 2048, 55 us with bf16 rows, 5.0 TB/s.
//
// A row length that is no multiple of 512 ends with the chunk [D - 512, D)
// whose part before the last whole multiple is skipped (bf16 rows) or meets
// zero codes (MXFP4 rows): every weight load stays a full one inside its row.
#pragma once

#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace mx {

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
// a 16-byte load at a 4-byte aligned address (scale rows)
typedef i32x4 __attribute__((aligned(4))) i32x4u;

constexpr int kThreads = 256;      // 4 waves
constexpr int kPitch = 256;        // bytes of a row in an LDS stage
constexpr int kChunk = 512;        // values of a weight row per load chunk
// Rows of an m-tile.  MXFP4 rows: one tile for nearly every expert that the
// weights bound; 256 rows' stages and the weights' LDS do not fit a CU's.  bf16
// rows: the matrix cores bound an expert of more than about 100 rows, and the
// accumulators of more next to the fragments in two forms spill.
template <bool A4> constexpr int kMaxRows = A4 ? 192 : 128;
constexpr int kFewRows = 16;       // rows of a decode m-tile
using Yes = std::true_type;
using No = std::false_type;
template <int I> using C = std::integral_constant<int, I>;
template <int N, int I = 0, class F> __device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(C<I>{});
    each<N, I + 1>(f);
  }
}
template <class F> __device__ __forceinline__ void each4(F&& f) { each<4>(f); }
constexpr int kFp4 = 4;            // the instruction's operand format code for e2m1

struct GemmArgs {
  const void* a;                   // bf16 [.][D] or codes [.][D / 2]
  const uint8_t* a_scales;         // [.][D / 32], MXFP4 rows only
  const int32_t* row_src;          // row r reads a[row_src[r] / K]; NULL: a[r]
  int K, T;
  const int32_t* offsets;
  int rows_cap, n_experts, D, N;
  const uint8_t* w;                // [E][N][D / 2]
  const uint8_t* w_scales;         // [E][N][D / 32]
  void* out;                       // [.][N] or, SwiGLU, [.][N / 2]
  // list mode: m-tiles tiles[0] .. tiles[*count - 1]; direct mode (count NULL):
  // the rows of each expert that has any
  const int4* tiles;
  const int* count;
  int NT;                          // column tiles
};

__device__ __forceinline__ int swz16(int row, int at) { return at ^ (row & 15); }

// g / (1 + exp(-g)).  exp(-g) = 2^t with t = -g log2(e) in two parts, 2^hi times
// 1 + lo ln 2: a far g costs no digits, and the hardware's 2^x and 1/x are good
// to a unit in the last place.  (With expf and a division the outputs of a
// 128 x 128 tile took 4 us, with this 2.)
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269504f, kLog2eLo = 1.9259630e-8f, kLn2 = 0.693147181f;
  const float hi = -g * kLog2e;
  const float lo = fmaf(-g, kLog2eLo, fmaf(-g, kLog2e, -hi));
  float x = __builtin_amdgcn_exp2f(hi);
  // past that 2^hi is or nears 0 or infinity (whose product with lo is no number)
  x = fabsf(hi) < 126.0f ? fmaf(x, lo * kLn2, x) : x;
  return g * __builtin_amdgcn_rcpf(1.0f + x);
}

template <typename OutT, int C>
__device__ __forceinline__ void store_cols(OutT* o, const float* v) {
  if constexpr (sizeof(OutT) == 2) {
    if constexpr (C % 8 == 0) {
#pragma unroll
      for (int i = 0; i < C; i += 8) {
        bf16x8 p;
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = (bf16)v[i + k];
        *(bf16x8*)(o + i) = p;
      }
    } else {
      typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
      bf16x4 p;
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = (bf16)v[k];
      *(bf16x4*)o = p;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; i += 4) *(f32x4*)(o + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  }
}

// LDS of a tile of 16 R rows: two stages of rows; for MXFP4 rows two stages of
// their scales (one dword a row and 32-value group of a slice: byte j is slice
// j's); and for every wave 256 values of its 16 CB weight rows, with a chunk's
// scales in the same form.
template <int CB> constexpr int kWaveLds = 16 * CB * (128 + 16);
// (R: rows / 16)
template <int R, int CB, bool A4>
constexpr int lds_bytes() {
  return 2 * 16 * R * kPitch + (A4 ? 2 * 16 * R * 16 : 0) + 4 * kWaveLds<CB>;
}

// One block of matrix instructions of MS x MS outputs: 16 or 32.  Lane l holds
// row l % MS of either operand and one 32-value block of it, number l / MS of
// the instruction's 4 (MS = 16) or 2; a slice of 128 values is kU instructions.
template <int MS> struct Mma;
template <> struct Mma<16> {
  typedef f32x4 Acc;
  static constexpr int kU = 1;
  static __device__ __forceinline__ Acc bf16_(bf16x8 w, bf16x8 a, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, a, c, 0, 0, 0);
  }
  template <int B>
  static __device__ __forceinline__ Acc fp4(i32x8 w, i32x8 a, Acc c, int sw, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, kFp4, kFp4, B, sw, B, sa);
  }
};
template <> struct Mma<32> {
  typedef f32x16 Acc;
  static constexpr int kU = 2;
  static __device__ __forceinline__ Acc bf16_(bf16x8 w, bf16x8 a, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, a, c, 0, 0, 0);
  }
  template <int B>
  static __device__ __forceinline__ Acc fp4(i32x8 w, i32x8 a, Acc c, int sw, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, kFp4, kFp4, B, sw, B, sa);
  }
};

// One tile: RB blocks of MS rows times 4 waves of 16 CB weight rows.
// NT: the weights are loaded past the caches (no other m-tile reads them).
template <int MS, int RB, int CB, bool A4, bool SW, bool NT, typename OutT>
__device__ __forceinline__ void tile(char* smem, const GemmArgs& p, int e, int row0, int rows,
                                     int nt) {
  using M = Mma<MS>;
  constexpr int BM = MS * RB;                   // rows
  constexpr int NB = 16 * CB / MS;              // weight blocks of a wave
  constexpr int U = M::kU, G = 64 / MS;         // instructions of a slice; 32-value blocks of one
  constexpr int SL = 16 * CB / G;               // outputs of a lane per row
  constexpr int kAcc = MS * MS / 64;
  constexpr int WC = SW ? 8 * CB : 16 * CB;     // output columns of a wave
  static_assert(NB >= 1 && (!SW || SL % 8 == 0), "gate and up in one lane, 4 at a time");
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int m = lane & (MS - 1), g = lane / MS;
  const int D = p.D, N = p.N;
  const int width = SW ? N / 2 : N;             // output columns
  const int code_pitch = D >> 1, scale_pitch = D >> 5;
  const bool small = D < kChunk;                // one chunk, shorter than 512
  const int KC = (D + kChunk - 1) / kChunk;
  // first value of chunk c
  auto window = [&](int c) { return small ? 0 : min(c * kChunk, D - kChunk); };

  // ---- weights.  Row r = MS b + i of the wave's 16 CB is row i of block b.  An
  // instruction leaves a lane rows 4 g + (0..3) of its 16, or rows 8 q + 4 g +
  // (0..3) of its 32; which weight row each is makes a lane's outputs OW
  // consecutive columns, 16 bytes, and the lanes of a row neighbours, with
  // SwiGLU its first half the gates and its second the ups of the same columns.
  // (One run of SL columns a lane: each store writes a piece of every line,
  // the fp32 outputs of a 192 x 256 tile took 11 us.)
  constexpr int OC = SW ? SL / 2 : SL;
  constexpr int OW = OC < 16 / (int)sizeof(OutT) ? OC : 16 / (int)sizeof(OutT);
  const int col0 = nt * (4 * WC) + wave * WC;   // first output column of the wave
  const char* wbase = (const char*)p.w + (size_t)e * N * code_pitch;
  const char* sbase = (const char*)p.w_scales + (size_t)e * N * scale_pitch;
  auto weight_row = [&](int r) {
    const int b = r / MS, i = r % MS;
    const int gi = MS == 16 ? i >> 2 : (i >> 2) & 1;
    const int slot = MS == 16 ? 4 * b + (i & 3) : 16 * b + 4 * (i >> 3) + (i & 3);
    const int k = slot % OC;
    const int j = min(col0 + k / OW * (G * OW) + gi * OW + k % OW, width - 1);
    return (uint32_t)(j + (slot >= OC ? width : 0));
  };
  // Codes come in steps of 256 values (half a chunk), 8 rows x 128 bytes a
  // load: whole lines.  (Loads in the fragments' own layout, 16 rows x 64
  // bytes with neighbouring lanes in different rows, take the address unit 58
  // cycles each instead of 17: 4.2 TB/s.)  Two steps are in flight in
  // registers; they pass through LDS, the wave's own part, where 16-byte
  // pieces are XOR-swizzled by the row, to become fragments.
  constexpr int NL = 2 * CB;                    // loads of a step
  uint32_t woff[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i)
    woff[i] = weight_row(8 * i + (lane >> 3)) * (uint32_t)code_pitch;
  constexpr int NS = (16 * CB + 63) / 64;       // scale rows of a lane
  uint32_t soff[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
    soff[i] = weight_row((lane & (16 * CB - 1)) + 64 * i) * (uint32_t)scale_pitch;
  // Loads in front of the loop also take rows shorter than a chunk (FIRST): the
  // same places again instead of bytes past the row.  Loads inside the loop do
  // not branch, so that the waits for them stay exact.
  const int last_j = small ? scale_pitch / 4 - 1 : 3;     // last slice of a chunk
  auto load_scales = [&](auto FIRST, const char* s, int k0) -> i32x4 {
    if constexpr (!decltype(FIRST)::value) return *(const i32x4u*)(s + (k0 >> 5));
    i32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *(const int*)(s + 4 * min(j, last_j));
    return v;
  };
  i32x4 wr[2][NL], wsr[NS];                      // steps in flight; the next chunk's scales
  auto load_w = [&](auto FIRST, auto B, int step) {
    constexpr int b = decltype(B)::value;        // step & 1
    const int at = 128 * b + 16 * (lane & 7);    // in the chunk
    const char* wc = wbase + (window(step >> 1) >> 1) +
                     (decltype(FIRST)::value ? min(at, 64 * last_j + 48) : at);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const i32x4* src = (const i32x4*)(wc + woff[i]);
      wr[b][i] = NT ? __builtin_nontemporal_load(src) : *src;
    }
  };
  auto load_ws = [&](auto FIRST, int c) {
#pragma unroll
    for (int i = 0; i < NS; ++i) wsr[i] = load_scales(FIRST, sbase + soff[i], window(c));
  };
  char* wlds = smem + 2 * BM * kPitch + (A4 ? 2 * BM * 16 : 0) + wave * kWaveLds<CB>;
  char* slds = wlds + 16 * CB * 128;
  auto write_w = [&](auto B) {
    constexpr int b = decltype(B)::value;
    char* d = wlds + (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 3)) * 16;
    wave_lds_order();                            // behind the reads of the step before
#pragma unroll
    for (int i = 0; i < NL; ++i) *(i32x4*)(d + i * 1024) = wr[b][i];
    wave_lds_order();                            // in front of other lanes' reads
  };
  i32x4 fw[2][NB][U];                            // codes of a slice, by its parity
  auto read_w = [&](auto T) {                    // slice T of the step in LDS
    constexpr int t = decltype(T)::value;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u)
        fw[t][b][u] = *(const i32x4*)(wlds + (MS * b + m) * 128 +
                                      ((4 * t + G * u + g) ^ (m & 7)) * 16);
  };
  // A row's 16 scales of a chunk (dword j: slice j) as the lanes use them: MS =
  // 16: dword g holds group g of the 4 slices; MS = 32: dwords 2 g + w hold
  // groups g and 2 + g of slices 2 w and 2 w + 1.
  auto scale_dwords = [&](const i32x4& v) {
    if constexpr (MS == 16) {
      i32x4 t;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int sel = s | ((4 + s) << 8) | 0x0c0c0000;
        t[s] = (int)__builtin_amdgcn_perm(__builtin_amdgcn_perm(v[3], v[2], sel),
                                          __builtin_amdgcn_perm(v[1], v[0], sel), 0x05040100);
      }
      return t;
    } else {
      return i32x4{(int)__builtin_amdgcn_perm(v[1], v[0], 0x06040200),
                   (int)__builtin_amdgcn_perm(v[3], v[2], 0x06040200),
                   (int)__builtin_amdgcn_perm(v[1], v[0], 0x07050301),
                   (int)__builtin_amdgcn_perm(v[3], v[2], 0x07050301)};
    }
  };
  // byte kByte(j, u) of dword kDword(j): the scale of a lane's block in
  // instruction u of slice j
  constexpr auto kByte = [](int j, int u) { return MS == 16 ? j : 2 * (j & 1) + u; };
  constexpr auto kDword = [](int j) { return MS == 16 ? 0 : j >> 1; };
  auto read_scales = [&](const char* s, int* d) {
#pragma unroll
    for (int w = 0; w < U; ++w) d[w] = *(const int*)(s + (U * g + w) * 4);
  };
  int sw[NB][U];
  auto pass_scales = [&] {
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (16 * CB >= 64 || lane < 16 * CB)
        *(i32x4*)(slds + (lane + 64 * i) * 16) = scale_dwords(wsr[i]);
    wave_lds_order();
#pragma unroll
    for (int b = 0; b < NB; ++b) read_scales(slds + (MS * b + m) * 16, sw[b]);
  };

  // ---- rows: thread t stages 16-byte chunk t % 16 of rows t / 16 + 16 i;
  // rows past the tile's are its last one again (never stored)
  constexpr int R = BM / 16;
  const int sr = tid >> 4, sc = tid & 15;
  const int a_pitch = A4 ? code_pitch : 2 * D;
  constexpr int NQ = A4 ? R + 1 : R;
  int src[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i)
    src[i] = row0 + min(i < R ? sr + 16 * i : min(tid, BM - 1), rows - 1);
  if (p.row_src) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) src[i] = p.row_src[src[i]];
  }
  // the first weights are on their way while the row indices arrive
  load_ws(Yes{}, 0);
  load_w(Yes{}, C<0>{}, 0);
  load_w(Yes{}, C<1>{}, 1);
  if (p.row_src) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) src[i] = min(max(src[i], 0) / p.K, p.T - 1);
  }
  // A row's address in 32 bits: in units of 128 values, which a row is a whole
  // number of (2^39 values at most, the host checks)
  constexpr int kUnit = A4 ? 6 : 8;              // log2 of a unit's bytes
  uint32_t arow[R];
#pragma unroll
  for (int i = 0; i < R; ++i) arow[i] = (uint32_t)(((size_t)src[i] * a_pitch) >> kUnit);
  auto row_ptr = [&](int i) { return (const char*)p.a + ((size_t)arow[i] << kUnit); };

  typename M::Acc acc[RB][NB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < kAcc; ++k) acc[i][j][k] = 0.0f;
  constexpr int stage_bytes = BM * kPitch;
  // A lane's pieces of a row: MXFP4 4 j + b for block b of slice j; bf16 4 b + q
  // for fragment q of block b, kept at place 4 q + b, so that the lanes of
  // either read, which are served in an order that mixes rows of neighbouring
  // groups, meet different banks.
  const int place = A4 ? sc : 4 * (sc & 3) + (sc >> 2);
  auto write_rows = [&](char* st, const i32x4* v) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = sr + 16 * i;
      *(i32x4*)(st + r * kPitch + swz16(r, place) * 16) = v[i];
    }
  };
  auto frag = [&](const char* st, int rb, int at) {
    const int r = MS * rb + m;
    return *(const i32x4*)(st + r * kPitch + swz16(r, at) * 16);
  };
  // Multiplications run in groups of RG row blocks (RG * NB matrix
  // instructions); a group's row fragments are read from LDS before the group
  // in front of it is multiplied, a slice's weight fragments a slice before.
  // Each group is a basic block of its own, behind a branch on a value the
  // compiler cannot see through: matrix instructions have no side effects, and
  // without the branches they are all moved behind the waits for the next
  // chunk's loads, which then hide behind nothing.
  constexpr int RG = RB <= 5 ? RB : RB / 2;
  constexpr int NH = RB / RG;                    // groups per instruction step
  static_assert(RB % RG == 0, "whole groups");
  i32x4 fr[2][RG];
  auto opaque = [&](int v) {
    v = __builtin_amdgcn_readfirstlane(v);
    asm volatile("" : "+s"(v));
    return v != 0;
  };
  // The weights' part of slice J of chunk c, between its groups: the next
  // slice's fragments, and at the end of a step the next step's codes into LDS
  // and the loads of the step two further on.  AHEAD: chunks that follow c, as
  // far as 2.
  auto advance_w = [&](auto AHEAD, auto J, int c) {
    constexpr int ahead = decltype(AHEAD)::value, j = decltype(J)::value;
    if constexpr (j % 2 == 0) {
      read_w(C<1>{});
    } else if constexpr (j == 1 || ahead > 0) {
      write_w(C<(j + 1) / 2 % 2>{});
      // j = 1: step 2c + 3 of the next chunk; j = 3: step 2c + 4 of the one after
      if constexpr (ahead > j / 2) load_w(No{}, C<(j + 1) / 2 % 2>{}, 2 * c + (j + 5) / 2);
      read_w(C<0>{});
    }
  };
  // Chunks in order, told how many follow.
  auto sweep = [&](auto&& chunk) {
    for (int c = 0; c + 2 < KC; ++c) chunk(C<2>{}, c);
    if (KC >= 2) chunk(C<1>{}, KC - 2);
    chunk(C<0>{}, KC - 1);
  };
  // In front of the sweep: step 0 in LDS, its first fragments, step 2 on its way.
  auto first_w = [&] {
    write_w(C<0>{});
    if (KC >= 2) load_w(No{}, C<0>{}, 2);
    pass_scales();
    read_w(C<0>{});
  };

  if constexpr (A4) {
    constexpr int NG = U * NH;                   // groups per slice
    char* scl = smem + 2 * stage_bytes;
    const char* as_ptr = (const char*)p.a_scales + (size_t)src[R] * scale_pitch;
    i32x4 av[R], as;
    auto load_a = [&](auto FIRST, int c) {
      const int kb = (window(c) >> 1) +
                     (decltype(FIRST)::value ? min(16 * sc, 64 * last_j + 48) : 16 * sc);
#pragma unroll
      for (int i = 0; i < R; ++i) av[i] = *(const i32x4*)(row_ptr(i) + kb);
      as = load_scales(FIRST, as_ptr, window(c));
    };
    auto write_a = [&](int c) {
      // values before c * 512 were multiplied in the chunk before, values
      // past D do not exist: zero codes
      const int k = window(c) + 32 * sc;
      const bool live = k >= c * kChunk && k < D;
      const int b = c & 1;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) av[i][q] = live ? av[i][q] : 0;
      write_rows(smem + b * stage_bytes, av);
      const i32x4 t = scale_dwords(as);
      if (BM == kThreads || tid < BM) *(i32x4*)(scl + (b * BM + tid) * 16) = t;
    };
    auto chunk = [&](auto AHEAD, int c) {
      constexpr bool more = decltype(AHEAD)::value > 0;
      const int b = c & 1;
      const char* st = smem + b * stage_bytes;
      int sa[RB][U];
#pragma unroll
      for (int r = 0; r < RG; ++r) fr[0][r] = frag(st, r, g);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) read_scales(scl + (b * BM + MS * rb + m) * 16, sa[rb]);
      if constexpr (more) {
        load_ws(No{}, c + 1);     // before the codes: the waits for these leave them in flight
        load_a(No{}, c + 1);
      }
      each4([&](auto J) {
        constexpr int j = decltype(J)::value;
        // with several groups a slice the writes to LDS come behind its first
        if constexpr (NG == 1 || j % 2 == 0) advance_w(AHEAD, J, c);
        each<NG>([&](auto I) {
          constexpr int u = decltype(I)::value / NH, h = decltype(I)::value % NH;
          constexpr int n = j * NG + decltype(I)::value;
          if constexpr (decltype(I)::value == 1) {
            if constexpr (j % 2 == 1) advance_w(AHEAD, J, c);
            if constexpr (more && j == 3) write_a(c + 1);
          }
          if (opaque(1)) {
            if constexpr (n + 1 < 4 * NG) {
              constexpr int j1 = (n + 1) / NG, u1 = (n + 1) % NG / NH, h1 = (n + 1) % NH;
#pragma unroll
              for (int r = 0; r < RG; ++r)
                fr[(n + 1) & 1][r] = frag(st, h1 * RG + r, 4 * j1 + G * u1 + g);
            }
#pragma unroll
            for (int r = 0; r < RG; ++r) {
              const i32x4 f = fr[n & 1][r];
              const i32x8 fa = {f[0], f[1], f[2], f[3], 0, 0, 0, 0};
              constexpr int w0 = kDword(j);
              const int rb = h * RG + r;
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                const i32x4 w = fw[j & 1][b][u];
                const i32x8 fb = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
                acc[rb][b] = M::template fp4<kByte(j, u)>(fb, fa, acc[rb][b], sw[b][w0], sa[rb][w0]);
              }
            }
          }
        });
      });
      if constexpr (more) {
        if constexpr (NG == 1) write_a(c + 1);
        pass_scales();
      }
      lds_barrier();
    };
    load_a(Yes{}, 0);
    first_w();
    write_a(0);
    lds_barrier();
    sweep(chunk);
  } else {
    constexpr int NG = 4 * U * NH;       // groups per slice
    constexpr int PA = 2;                // row stages in flight in registers
    i32x4 av[PA][R];
    const int S = 4 * KC;
    auto load_a = [&](i32x4* v, int s) {
      const int kb = 2 * min(window(s >> 2) + 128 * (s & 3), D - 128) + 16 * sc;
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] = *(const i32x4*)(row_ptr(i) + kb);
    };
    // slice J; between(n) runs behind group n.  !live: only those
    auto compute = [&](auto J, int live, auto&& between) {
      constexpr int j = decltype(J)::value;
      const char* st = smem + (j & 1) * stage_bytes;
      bf16x8 fb[2][NB];
      // codes of fragment q in instruction u as bf16, scaled (0xFF: NaN)
      auto unpack = [&](auto Q) {
        constexpr int u = decltype(Q)::value / 4, q = decltype(Q)::value % 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float s2 = __uint_as_float(
              __builtin_amdgcn_ubfe((unsigned)sw[b][kDword(j)], 8 * kByte(j, u), 8) << 23);
          const unsigned c = (unsigned)fw[j & 1][b][u][q];
          const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s2, 0);
          const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s2, 1);
          const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s2, 2);
          const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s2, 3);
          fb[q & 1][b] = bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
        }
      };
#pragma unroll
      for (int r = 0; r < RG; ++r) fr[0][r] = frag(st, r, g);
      unpack(C<0>{});
      each<NG>([&](auto I) {
        constexpr int n = decltype(I)::value, uq = n / NH, q = uq % 4, h = n % NH;
        if (opaque(live)) {
          if constexpr (n + 1 < NG) {
            constexpr int u1 = (n + 1) / NH / 4, q1 = (n + 1) / NH % 4, h1 = (n + 1) % NH;
#pragma unroll
            for (int r = 0; r < RG; ++r)
              fr[(n + 1) & 1][r] = frag(st, h1 * RG + r, 4 * q1 + G * u1 + g);
          }
          if constexpr (h == NH - 1 && uq + 1 < 4 * U) unpack(C<uq + 1>{});
#pragma unroll
          for (int r = 0; r < RG; ++r) {
            const bf16x8 fa = __builtin_bit_cast(bf16x8, fr[n & 1][r]);
            const int rb = h * RG + r;
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[rb][b] = M::bf16_(fb[q & 1][b], fa, acc[rb][b]);
          }
        }
        between(I);
      });
    };
    auto chunk = [&](auto AHEAD, int c) {
      constexpr bool more = decltype(AHEAD)::value > 0;
      const int k0 = window(c);
      if constexpr (more) load_ws(No{}, c + 1);
      each4([&](auto J) {
        constexpr int j = decltype(J)::value;
        const int s = 4 * c + j;
        auto rows_on = [&] {
          if constexpr (more || j < 3) {
            i32x4* v = av[(j + 1) % PA];
            write_rows(smem + ((j + 1) & 1) * stage_bytes, v);
            if constexpr (more || j + 1 + PA < 4) load_a(v, min(s + 1 + PA, S - 1));
          }
        };
        if constexpr (RB == 1) {
          rows_on();
          advance_w(AHEAD, J, c);
        }
        // not the slices that the chunk before holds, nor those past a short row
        const int k = k0 + 128 * j;
        compute(J, k >= c * kChunk && k < D ? 1 : 0, [&](auto I) {
          if constexpr (RB > 1 && decltype(I)::value == 0) rows_on();
          if constexpr (RB > 1 && decltype(I)::value == 1) advance_w(AHEAD, J, c);
        });
        if constexpr (more && j == 3) pass_scales();
        lds_barrier();
      });
    };
    // stage 0's rows, then stages 1 .. PA in registers
    load_a(av[0], 0);
    first_w();
    write_rows(smem, av[0]);
#pragma unroll
    for (int i = 1; i <= PA; ++i) load_a(av[i % PA], min(i, S - 1));
    lds_barrier();
    sweep(chunk);
  }

  // ---- lane l: row MS rb + l % MS, OW columns at a time
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = MS * rb + m;
    if (r >= rows) continue;
    auto at = [&](int slot) { return acc[rb][slot / kAcc][slot % kAcc]; };
#pragma unroll
    for (int i = 0; i < OC; i += OW) {
      float v[OW];
#pragma unroll
      for (int k = 0; k < OW; ++k) v[k] = SW ? silu(at(i + k)) * at(OC + i + k) : at(i + k);
      // widths are multiples of 8, so no piece is split
      const int n = col0 + i * G + OW * g;
      if (n < width) store_cols<OutT, OW>((OutT*)p.out + (size_t)(row0 + r) * width + n, v);
    }
  }
}

// Block -> (m-tile, column tile).  Consecutive blocks land on the 8 XCDs in
// turn, so all column tiles of one m-tile run on one XCD and share its rows in
// that XCD's L2.
__device__ __forceinline__ bool find_tile(const GemmArgs& p, int4& t, int& nt) {
  const int b = blockIdx.x, slot = b >> 3;
  const int mt = (slot / p.NT) * 8 + (b & 7);
  nt = slot % p.NT;
  if (p.count) {
    if (mt >= *p.count) return false;
    t = p.tiles[mt];
    return true;
  }
  // the mt-th of the experts that have rows, 64 experts a turn (numbered
  // without the others, m-tiles spread over the XCDs evenly)
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < p.n_experts; e0 += 64) {
    const int e = e0 + lane;
    int r0 = 0, m = 0;
    if (e < p.n_experts) {
      r0 = min(max(p.offsets[e], 0), p.rows_cap);
      m = min(max(p.offsets[e + 1], r0), p.rows_cap) - r0;
    }
    const unsigned long long hit = __ballot(m > 0);
    const int k = mt - before;
    before += __popcll(hit);
    if (mt < before) {
      const bool mine = m > 0 && __popcll(hit & ((1ull << lane) - 1)) == k;
      const int src = __ffsll((long long)__ballot(mine)) - 1;
      t = make_int4(e0 + src, __builtin_amdgcn_readlane(r0, src),
                    __builtin_amdgcn_readlane(m, src), 0);
      return true;
    }
  }
  return false;
}

// Two kernels, since a kernel's registers are those of its largest tile.
//
// Few rows an expert (decode): every m-tile is one of at most 16 rows, two
// blocks to a CU.  An expert that has more is taken 16 rows at a time.
template <int CB, bool A4, bool SW, typename OutT>
__global__ __launch_bounds__(kThreads, 2) void gemm_few(GemmArgs p) {
  __shared__ __attribute__((aligned(16))) char smem[lds_bytes<1, CB, A4>()];
  int4 t;
  int nt;
  if (!find_tile(p, t, nt)) return;
  int r = 0;
  do {
    // nothing of a turn is kept in registers for the next
    int e = __builtin_amdgcn_readfirstlane(t.x), n = __builtin_amdgcn_readfirstlane(nt);
    asm volatile("" : "+s"(e), "+s"(n));
    tile<16, 1, CB, A4, SW, true, OutT>(smem, p, e, t.y + r, min(kFewRows, t.z - r), n);
    r += kFewRows;
  } while (r < t.z);
}

// m-tiles of any size up to kMaxRows, one block to a CU.  One launch for all of
// them: with one each for up to 16, up to 64 and more rows, the few m-tiles of
// the rarer sizes held the chip by themselves (50 rows an expert: FFN 462 us).
template <bool A4, bool SW, typename OutT>
__global__ __launch_bounds__(kThreads, 1) void gemm_any(GemmArgs p) {
  __shared__ __attribute__((aligned(16))) char smem[lds_bytes<kMaxRows<A4> / 16, 4, A4>()];
  int4 t;
  int nt;
  if (!find_tile(p, t, nt)) return;
  if (t.z <= 16)
    tile<16, 1, 4, A4, SW, true, OutT>(smem, p, t.x, t.y, t.z, nt);
  else if (t.z <= 32)
    tile<32, 1, 4, A4, SW, true, OutT>(smem, p, t.x, t.y, t.z, nt);
  else if (t.z <= 64)
    tile<32, 2, 4, A4, SW, true, OutT>(smem, p, t.x, t.y, t.z, nt);
  else if (t.z <= 96)
    tile<32, 3, 4, A4, SW, false, OutT>(smem, p, t.x, t.y, t.z, nt);
  else if (!A4 || t.z <= 128)
    tile<32, 4, 4, A4, SW, false, OutT>(smem, p, t.x, t.y, t.z, nt);
  else if constexpr (A4) {
    if (t.z <= 160)
      tile<32, 5, 4, A4, SW, false, OutT>(smem, p, t.x, t.y, t.z, nt);
    else
      tile<32, 6, 4, A4, SW, false, OutT>(smem, p, t.x, t.y, t.z, nt);
  }
}

// Launches of one form of rows.  few_cb: 0, gemm_any over the m-tile list; 2 or
// (without SwiGLU) 1, gemm_few with so many column blocks a wave.
template <bool A4>
hipError_t launch_gemm(GemmArgs p, int few_cb, bool swiglu, int out_dtype, unsigned mtiles,
                       hipStream_t s);

template <bool A4, bool SW, typename OutT>
void launch_gemm_t(GemmArgs& p, int few_cb, unsigned mtiles, hipStream_t s) {
  const int width = SW ? p.N / 2 : p.N, cb = few_cb ? few_cb : 4;
  p.NT = (int)ceil_div(width, SW ? 32 * cb : 64 * cb);
  const unsigned grid = ceil_div(mtiles, 8) * 8 * p.NT;
  if (few_cb == 0) {
    MOE_LAUNCH(A4 ? "mx_gemm_any_fp4" : "mx_gemm_any_bf16", s,
               gemm_any<A4, SW, OutT><<<grid, kThreads, 0, s>>>(p));
  } else if (few_cb == 2) {
    MOE_LAUNCH(A4 ? "mx_gemm_few_fp4" : "mx_gemm_few_bf16", s,
               gemm_few<2, A4, SW, OutT><<<grid, kThreads, 0, s>>>(p));
  } else if constexpr (!SW) {
    MOE_LAUNCH(A4 ? "mx_gemm_few_fp4" : "mx_gemm_few_bf16", s,
               gemm_few<1, A4, SW, OutT><<<grid, kThreads, 0, s>>>(p));
  }
}

#define MX_INSTANTIATE(A4)                                                                       \
  template <>                                                                                    \
  hipError_t launch_gemm<A4>(GemmArgs p, int few_cb, bool swiglu, int out_dtype,                 \
                             unsigned mtiles, hipStream_t s) {                                   \
    if (out_dtype == MOE_BF16)                                                                   \
      swiglu ? launch_gemm_t<A4, true, bf16>(p, few_cb, mtiles, s)                               \
             : launch_gemm_t<A4, false, bf16>(p, few_cb, mtiles, s);                             \
    else                                                                                         \
      swiglu ? launch_gemm_t<A4, true, float>(p, few_cb, mtiles, s)                              \
             : launch_gemm_t<A4, false, float>(p, few_cb, mtiles, s);                            \
    return hipGetLastError();                                                                    \
  }

}  // namespace mx
}  // namespace moe
