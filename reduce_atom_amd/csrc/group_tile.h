// One output tile of a grouped product on the matrix units, by one workgroup of four
// waves: BM rows by BN columns, the contraction in steps of 128 bytes (64 elements of 16
// bits, 128 of 8).
//
// Operands. R gives the output's rows, C its columns. Each is staged by asynchronous
// global -> LDS copies of 16 bytes a lane, in one of two layouts that follow its memory:
//   rows:   memory rows run along the contraction. LDS [rows][128 bytes], 16-byte chunk c
//           of row r at slot c ^ ((r >> 1) & 7): the 32 rows that a fragment's lanes read
//           at one chunk then lie on all banks evenly.
//   steps:  memory rows run across it (the operand is transposed). LDS [64][columns],
//           chunk c of row s at slot c ^ ((s & 3) << 2); fragments are read with the
//           transposing LDS read, 4 contraction rows by 16 columns at a time.
// A fragment (32 rows or columns by half a step) is 32 bytes of a lane. The matrix
// instruction takes C's fragment first, so a lane ends with one output row and 16 columns
// of a 32 x 32 tile; C's columns are dealt to the fragment's rows such that these 16 lie
// side by side (column 16 ((r >> 2) & 1) + 4 (r >> 3) + (r & 3) at fragment row r) and a
// lane stores whole 16-byte vectors.
//
// Pipeline. LDS has two slots for R's steps and DEPTH for C's. Half 0 of step t is multiplied
// while half 1 is read from LDS into registers; then every wave has read step t whole, one
// barrier passes (step t + 1 has landed by then), and while half 1 is multiplied, the copies
// of R's step t + 2 and C's step t + DEPTH are issued into the slots just freed and half 0 of
// step t + 1 is read. Each wave alone so keeps its matrix unit fed. C is the weights, which
// come from HBM where a group has few row tiles; a third slot gives them one step more.
// Where a workgroup goes from tile to tile, the first steps of the next are copied once the
// last step of one has been read from LDS, while its last half is multiplied and stored (8 x
// 512 rows by 4096 x 4096: 180 -> 177 us in bf16, 90 -> 82 us in 8 bits).
#pragma once

#include "device_common.h"
#include "moe.h"

namespace plr {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// What a contraction row or chunk past the end is read from.
__device__ const u32x4 g_zeros = {0, 0, 0, 0};

// 16 bytes per lane from p into LDS at `lds` (wave-uniform) + 16 * lane, asynchronously. In
// assembly, so that the compiler does not hold every LDS read back until all copies have
// landed; the waits are in step_barrier. Nothing is written to a vector register; m0 is
// written here and nowhere else (it is reserved: the compiler keeps no value in it).
__device__ __forceinline__ void dma16(const char* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(p));
}

// Every wave's LDS reads are done and all but its last N copies have landed.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile(
      "s_waitcnt vmcnt(%0) lgkmcnt(0)\n\t"
      "s_barrier" ::"n"(N)
      : "memory");
}

// Layouts of a lane's fragment: two 16-byte parts, part s holding contraction elements
// of instruction s (16-bit types) or of one instruction (8-bit).
struct Frag {
  u32x4 part[2];
};

template <int DT>
__device__ __forceinline__ f32x16 mfma32(const Frag& c, const Frag& r, f32x16 acc, int s) {
  if constexpr (DT == PLR_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, c.part[s]),
                                                   __builtin_bit_cast(bf16x8, r.part[s]), acc, 0, 0, 0);
  else if constexpr (DT == PLR_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, c.part[s]),
                                                  __builtin_bit_cast(f16x8, r.part[s]), acc, 0, 0, 0);
  else {
    // e4m3 by e4m3, block scales of one. The instruction adds the products of 8 neighbouring
    // elements with the bits below 2^-13 of the largest cut off (measured: a product of 4 beside
    // one of 65536 is lost within 8 elements and kept outside), the rest in binary32: 1.5e-5 of
    // random sums (2-norm), half a unit in the last place of bfloat16 being 3.9e-3. Accepted: the
    // 16-bit instructions on converted operands would be exact at half the rate (8192 x 8192 x
    // 8192: 400-427 us against 797-871).
    const i32x8 cv = {(int)c.part[0].x, (int)c.part[0].y, (int)c.part[0].z, (int)c.part[0].w,
                      (int)c.part[1].x, (int)c.part[1].y, (int)c.part[1].z, (int)c.part[1].w};
    const i32x8 rv = {(int)r.part[0].x, (int)r.part[0].y, (int)r.part[0].z, (int)r.part[0].w,
                      (int)r.part[1].x, (int)r.part[1].y, (int)r.part[1].z, (int)r.part[1].w};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(cv, rv, acc, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
  }
}

// Wave tiles of RT x CT matrices of 32 x 32, waves WR x WC.
template <int RT_, int CT_, int WR_, int WC_>
struct Shape {
  static constexpr int RT = RT_, CT = CT_, WR = WR_, WC = WC_;
  static constexpr int BM = WR * RT * 32, BN = WC * CT * 32;
  static_assert(WR * WC == 4, "four waves");
};

// Bytes of a row of contraction elements in one step.
constexpr int kStepBytes = 128;

// LDS of TILE x TILE tiles.
template <int TILE, int DEPTH_>
struct Slots {
  static constexpr int DEPTH = DEPTH_;
  static constexpr int SLOT = TILE * kStepBytes;  // one operand's step
  static constexpr int LDS = (2 + DEPTH) * SLOT;
  __device__ static __forceinline__ int r(int slot) { return slot * SLOT; }
  __device__ static __forceinline__ int c(int slot) { return (2 + slot) * SLOT; }
};

// One operand of a tile: where its copies come from and how its fragments are read.
//   SPAN  rows (or columns) of the tile; STEPS  the layout; PERM  the dealing of columns
//   described above; ES  bytes of an element; WAVES  waves that share the copies.
template <int SPAN, bool STEPS, bool PERM, int ES, int WAVES = 4>
struct Operand {
  static constexpr int N = SPAN / 8 / WAVES;             // copies per wave and step
  static constexpr int RPI = STEPS ? 512 / SPAN : 8;     // memory rows per copy of a wave
  static_assert(!STEPS || SPAN == 256 || SPAN == 128, "whole memory rows per copy, and room for their swizzle");
  static constexpr int LANES = 64 / RPI;                 // lanes (16-byte chunks) per memory row
  static constexpr int STEP = kStepBytes / ES;           // contraction elements per step
  const char* p[N];
  int chunk;       // rows: this lane's 16-byte chunk of the step in the wave's even copies
  uint32_t at[4];  // LDS offsets of this lane's reads

  __device__ __forceinline__ int chunk_of(int n) const { return WAVES & 1 ? chunk ^ (4 * (n & 1)) : chunk; }

  // Rows layout: `row(r)` gives the address of tile row r's first contraction element.
  template <typename F>
  __device__ __forceinline__ void rows_copies(int wave, int lane, F row) {
    chunk = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
#pragma unroll
    for (int n = 0; n < N; ++n) p[n] = row(8 * (wave + WAVES * n) + (lane >> 3)) + chunk_of(n) * 16;
  }
  __device__ __forceinline__ void rows_reads(int lane, int first) {
    const int r = lane & 31, g = lane >> 5;
    const int m = PERM ? 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3) : r;
    const int slot = g ^ ((m >> 1) & 7);
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = (first + m) * kStepBytes + ((slot ^ (2 * q)) << 4);
  }

  // Steps layout: `base` is the address of column 0 of the tile at contraction row 0.
  // Column chunks past `cols` re-read chunk 0; what they give is not stored.
  __device__ __forceinline__ int step_of(int wave, int lane, int n) const {
    return RPI * (wave + WAVES * n) + lane / LANES;
  }
  __device__ __forceinline__ int64_t col_bytes(int wave, int lane, int64_t cols) const {
    const int s = step_of(wave, lane, 0);  // the same modulo 4 for every n
    const int c = (lane % LANES) ^ ((s & 3) << 2);
    return c * 8 < cols ? c * 16 : 0;
  }
  __device__ __forceinline__ void steps_reads(int lane, int first) {
    const int h = (lane >> 4) & 1, g = lane >> 5, q = (lane & 15) >> 2, e = lane & 3;
    const int c = PERM ? 2 * (e & 1) + h : 2 * h + (e >> 1), half = PERM ? e >> 1 : e & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      at[i] = (8 * g + q) * (SPAN * 2) + ((((first >> 3) + 4 * i + c) ^ (q << 2)) << 4) + half * 8;
  }

  // Fragment i's part s of half h of the buffer at `lds`.
  __device__ __forceinline__ u32x4 read(PLR_LDS char* lds, int i, int h, int s) const {
    if constexpr (!STEPS) {
      return *(PLR_LDS u32x4*)(lds + at[2 * h + s] + i * (32 * kStepBytes));
    } else {
      PLR_LDS char* b = lds + at[i] + (32 * h + 16 * s) * (SPAN * 2);
      union {
        s16x4 v[2];
        u32x4 u;
      } x;
      x.v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((PLR_LDS s16x4*)b);
      x.v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((PLR_LDS s16x4*)(b + 4 * SPAN * 2));
      return x.u;
    }
  }
};

}  // namespace plr
