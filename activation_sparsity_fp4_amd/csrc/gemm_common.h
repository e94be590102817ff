// Pieces shared by the MXFP4 GEMMs (two-path and plain): the LDS swizzle, the
// rows and columns behind an output tile, buffer loads into LDS and their
// waits, the order of the tiles and the tile lookup of grouped launches.
#pragma once

#include "sharq_device.h"

namespace sharq {

constexpr int kRowBytes = 64;            // 128 FP4 codes
constexpr int kLdsBytes = 160 * 1024;    // LDS of one CU
constexpr uint32_t kOOB = 0x80000000u;   // buffer offset past every bound: reads as 0

// LDS chunk swizzle. gfx950 LDS has 64 four-byte banks; a ds_read_b128 of an
// MFMA fragment serves 16 lanes (16 consecutive rows, one 16-byte chunk each)
// per pass, and rows r and r + 4 start on the same bank. XOR-ing the chunk
// index with bits 2..3 of the row spreads those 16 rows over all 64 banks
// (measured: zero SQ_LDS_BANK_CONFLICT cycles).
__device__ __forceinline__ int swz_part(int row) { return (row >> 2) & 3; }
__device__ __forceinline__ int swz(int row, int part) {
  return row * kRowBytes + ((part ^ swz_part(row)) << 4);
}

// An MFMA operand fragment from LDS. The FP4 form of the scaled MFMA reads
// only the low 4 of its 8 operand registers, so the upper half is left
// undefined (no registers are spent on it).
typedef int v4i __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v8i frag(const uint8_t* p) {
  const v4i v = *reinterpret_cast<const v4i*>(p);
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Row sources of one output tile: which activation row feeds tile row r, or
// -1 (the row then reads as zeros). A gathered index outside [0, src_rows)
// is -1 as well, so malformed gather contents never address memory outside
// the activation buffers.
struct TileRows {
  int64_t m0;          // first output row of the tile
  int64_t rows_valid;  // output rows of the tile that exist (<= the tile height)
  const int32_t* gather;  // activation row of each output row, or nullptr (identity)
  int64_t src_rows;    // rows of the activation buffers (bound of a gathered index)
  __device__ __forceinline__ int64_t src(int r) const {
    if (r >= rows_valid) return -1;
    const int64_t p = m0 + r;
    if (!gather) return p;
    const int64_t g = gather[p];
    return g >= 0 && g < src_rows ? g : -1;
  }
};

// Weight rows of one output tile: the weight row behind tile column c.
// Plain tiles take rows n0 + c. A fused gate|up tile over h columns
// from h0 on, of a weight whose rows are [gate (I rows); up (I rows)],
// alternates blocks of 2^shift rows: block b holds the gate (b even) or up
// (b odd) rows of h columns h0 + 2^shift (b / 2) + c % 2^shift, so that half of
// each wave's 32-column MFMA tiles (four with shift 6, two with 5) are gate and
// half up columns of the same h columns.
struct TileCols {
  int64_t n0;    // first output column (plain) or first h column (gate|up)
  int64_t half;  // 0 for a plain tile, else I
  int shift = 6;
  __device__ __forceinline__ int64_t w_row(int c) const {
    if (half == 0) return n0 + c;
    const int b = c >> shift;
    return ((b & 1) ? half : 0) + n0 + ((int64_t)(b >> 1) << shift) + (c & ((1 << shift) - 1));
  }
};

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Buffer resource (gfx9 layout): base address, no stride, `bytes` records; a
// load at an offset past `bytes` returns zeros.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  i32x4 r = {(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)bytes, 0x00020000};
  return r;
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}

// Buffer loads that write straight into LDS: lane i of the wave stores its
// BYTES at lds + BYTES * i. They are written as inline assembly so that the
// compiler does not treat every later LDS read as dependent on them (it would
// otherwise wait for all loads in flight before each stage); completion is
// awaited explicitly with wait_vmcnt before the stage barrier. M0 carries the
// LDS base; gfx950 wants one wait state between writing M0 and the load.
__device__ __forceinline__ void buffer_to_lds16(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void buffer_to_lds4(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(lds) : "memory", "m0");
}

// s_waitcnt with only the vector-memory counter bounded (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// Barrier for the LDS ring. The vector-memory wait for the stage about to be
// read is issued separately (wait_vmcnt); a fenced __syncthreads() would wait
// for every buffer->LDS load in flight, including the stages being prefetched.
// The "memory" clobber keeps the compiler from moving LDS accesses across it.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Tile order. Workgroups are dispatched round-robin over the 8 XCDs, each
// with its own L2; block b is remapped so that each XCD receives a contiguous
// range of tile indices. Inside a range, tiles go in groups of 4 row tiles:
// the group's column tiles are walked with the 4 row tiles innermost, so the
// tiles in flight on one XCD share 4 activation row tiles and a few weight
// column tiles (measured 2-6% faster than row tiles innermost over all rows).
struct TileIndex {
  int tm, tn;
};
// Tile t of tiles_total in walking order: groups of 4 row tiles walk the
// column tiles with the row tiles innermost.
__device__ __forceinline__ TileIndex tile_order(int tile, int tiles_m, int tiles_total) {
  constexpr int kGroup = 4;
  const int tiles_n = tiles_total / tiles_m;
  const int group = tile / (kGroup * tiles_n);
  const int first_m = group * kGroup;
  const int gsize = min(tiles_m - first_m, kGroup);
  const int in_group = tile - group * kGroup * tiles_n;
  return TileIndex{first_m + in_group % gsize, in_group / gsize};
}

// Workgroups are dispatched round-robin over the 8 XCDs: block b of a grid
// of n (n % 8 == 0) becomes item (b % 8) (n / 8) + b / 8, so that each XCD
// takes a contiguous range of items.
__device__ __forceinline__ int xcd_item(int b, int n) {
  return (n & 7) == 0 ? (b & 7) * (n >> 3) + (b >> 3) : b;
}

__device__ __forceinline__ TileIndex tile_index(int b, int tiles_m, int tiles_total) {
  return tile_order(xcd_item(b, tiles_total), tiles_m, tiles_total);
}

// Tile of a grouped launch. The grid is one-dimensional over (row slot,
// column tile) pairs, column tiles innermost. With kXcdRanges the pairs are
// remapped so that each XCD (to which workgroups are dealt round-robin)
// receives a contiguous range: the column tiles of one row tile then share
// its activation rows, and the row tiles of one expert its weight tiles, in
// that XCD's L2. The A real tiles are dealt over the first A rounded up to 8
// workgroups, so the grid must be a multiple of 8 (a smaller one leaves tiles
// to no workgroup). Without it, pair b runs on XCD b mod 8, which for 8 column
// tiles gives each XCD a fixed column slice of every weight. The row slot is
// a linear index over all (expert, row-tile) pairs, expert e holding
// ceil(count_e / BM) row tiles in expert order; the expert is found by a wave-wide prefix sum of the
// per-expert tile counts. Returns e = -1 (uniform over the workgroup) for the
// surplus indices of the grid's upper bound. Segment bounds are clamped to
// [0, P], so malformed offsets never address rows outside the output.
struct GroupedTile {
  int e, col;
  TileRows tr;
};
__device__ __forceinline__ int64_t seg_bound(const int32_t* __restrict__ seg, int e, int64_t lo, int64_t P) {
  const int64_t v = seg[e];
  return v < lo ? lo : v > P ? P : v;
}

// Row tiles of 64 experts, one a lane, and their prefix sums.
struct ExpertTiles {
  int64_t lo, hi;  // the expert's rows
  int incl, excl;  // row tiles up to and before it
};
template <class C>
__device__ __forceinline__ ExpertTiles expert_tiles(const int32_t* __restrict__ seg, int e, int E, int64_t P) {
  ExpertTiles t;
  const int at = e < E ? e : E - 1;
  t.lo = seg_bound(seg, at, 0, P);
  t.hi = e < E ? seg_bound(seg, at + 1, t.lo, P) : t.lo;
  const int tiles = (int)((t.hi - t.lo + C::BM - 1) / C::BM);
  t.incl = wave_inclusive_scan(tiles);
  t.excl = t.incl - tiles;
  return t;
}

template <class C, bool kXcdRanges>
__device__ __forceinline__ GroupedTile grouped_tile(const int32_t* __restrict__ seg, int E, int64_t P,
                                                    const int32_t* __restrict__ a_rows, int64_t src_rows,
                                                    int tiles_n) {
  __shared__ int64_t s_rows[2];
  __shared__ int s_info[2];
  const int tid = threadIdx.x;
  if (tid == 0) s_info[0] = -1;
  __syncthreads();
  if (tid < 64) {
    // Experts 0 .. 127 are read once, in one round trip to memory; later ones
    // by the passes that need them.
    constexpr int kHeld = 2;
    ExpertTiles held[kHeld];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) held[c] = expert_tiles<C>(seg, 64 * c + tid, E, P);
    // With kXcdRanges, the real tiles A are counted; the first A (rounded up
    // to 8) workgroups take the work, so that every XCD gets an equal share,
    // XCD x the logical range [x A8 / 8, (x + 1) A8 / 8).
    const int b = blockIdx.x;
    int logical = b, target = b / tiles_n;  // slots past the last tile find no expert
    if constexpr (kXcdRanges) {
      int rows_total = 0;
#pragma unroll
      for (int c = 0; c < kHeld; ++c) rows_total += __builtin_amdgcn_readlane(held[c].incl, 63);
      for (int e0 = 64 * kHeld; e0 < E; e0 += 64)
        rows_total += __builtin_amdgcn_readlane(expert_tiles<C>(seg, e0 + tid, E, P).incl, 63);
      const int A = rows_total * tiles_n, A8 = (A + 7) & ~7;
      logical = b < A8 ? (b & 7) * (A8 >> 3) + (b >> 3) : A;
      target = logical < A ? logical / tiles_n : -1;
    }
    // The expert holding row slot target.
    int base = 0;
    auto find = [&](int e, const ExpertTiles& t) {
      if (target >= base + t.excl && target < base + t.incl) {
        s_info[0] = e;
        s_info[1] = logical - (logical / tiles_n) * tiles_n;
        s_rows[0] = t.lo + (int64_t)(target - base - t.excl) * C::BM;
        s_rows[1] = t.hi;
      }
      base += __builtin_amdgcn_readlane(t.incl, 63);
    };
#pragma unroll
    for (int c = 0; c < kHeld; ++c) find(64 * c + tid, held[c]);
    for (int e0 = 64 * kHeld; e0 < E && target >= base; e0 += 64) find(e0 + tid, expert_tiles<C>(seg, e0 + tid, E, P));
  }
  __syncthreads();
  GroupedTile g;
  g.e = s_info[0];
  if (g.e >= 0) {
    g.col = s_info[1];
    g.tr.m0 = s_rows[0];
    const int64_t hi = s_rows[1];
    g.tr.rows_valid = hi - g.tr.m0 < C::BM ? hi - g.tr.m0 : C::BM;
    g.tr.gather = a_rows;
    g.tr.src_rows = src_rows;
  }
  return g;
}

}  // namespace sharq
