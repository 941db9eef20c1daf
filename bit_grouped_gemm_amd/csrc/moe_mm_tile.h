// moe_mm_tile.h -- what the kernels of the row-major products share: loads
// straight into LDS, barriers between their stages, the search for a
// workgroup's tile among ragged groups, and the rounding of results.
#pragma once

#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr double kCUs = 256;
constexpr uint32_t kOutside = 0x80000000u;  // a byte offset no descriptor reaches

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// Direct-to-LDS load of 16 bytes per lane: lane l's land at lds + 16 l (lds
// wave-uniform).  `off` counts from `base`; from `span` on it reads zeros.
// STREAM: read once, so not kept in the caches (non-temporal).
template <bool STREAM>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t span, uint32_t off, uint8_t* lds) {
  auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, span, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0,
                                           STREAM ? 2 : 0);
}

// Barrier after this wave's LDS accesses and loads have completed; nothing is
// scheduled across it.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The same, but for this wave's last N loads.
template <int N>
__device__ __forceinline__ void stage_barrier_but() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Barrier after this wave's LDS accesses; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes per lane to base + off, past the caches; nothing for kOutside.
__device__ __forceinline__ void store16(uint8_t* base, const v4i& v, uint32_t off) {
  auto r = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7FFFFFFF, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);
}

// A group's rows and the tile's place in it.
struct Place {
  int e;      // group; E and E + 1: the rows behind the last and before the first one (clear_rest)
  int row0;   // first row of the tile
  int rows;   // rows of the tile (<= BM)
};

// Row range of group e (E: the rows behind the last group, E + 1: those before
// the first): the offsets clamped to [0, R], so a wrong offset array reads and
// writes nothing outside the tensors.
__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int e, int E, int R) {
  if (!offsets) return make_int2(e ? R : 0, R);
  if (e > E) return make_int2(0, min(max(offsets[0], 0), R));
  const int a = min(max(offsets[e], 0), R);
  const int b = e < E ? min(max(offsets[e + 1], a), R) : R;
  return make_int2(a, b);
}

// The sums of the lanes up to each one, saturating: within 16 lanes, then the rows of 16
// before it (lane moves inside the vector unit: each is some ten cycles, a shuffle through
// LDS a hundred).
__device__ __forceinline__ int wave_scan_sat(int v) {
#define MOE_SCAN(CTRL, ROWS) \
  v = __builtin_elementwise_add_sat(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false))
  MOE_SCAN(0x111, 0xF);  // row_shr:1
  MOE_SCAN(0x112, 0xF);
  MOE_SCAN(0x114, 0xF);
  MOE_SCAN(0x118, 0xF);
  MOE_SCAN(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  MOE_SCAN(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef MOE_SCAN
  return v;
}

// Tile `t` of the launch: every wave scans the groups' tile counts (64 lanes
// at a time), so nothing has to be prepared on the host.  `id` runs over this
// launch's workgroups; workgroup ids are dealt round-robin over the 8 XCDs,
// and XCD x takes tiles [x per, (x + 1) per): neighbouring tiles, which share
// rows or weights, share an L2.  Tiles run over all columns of four row tiles
// before the next four, of eight where there are eight columns or more
// (measured with 6, 8 and 16 columns: 4 and 8 are within 2 % of the best of 2,
// 4, 8 and 16).  BY_GROUP: of the row tiles of one group only, so that its weights come
// into an L2 once.  Returns false where the id has no tile.
template <bool BY_GROUP = false>
__device__ __forceinline__ bool find_tile(const MmArgs& a, int BM, int ncol, int id, Place& pl, int& col) {
  const int lane = threadIdx.x & 63;
  const int G = a.E + (a.clear_rest ? 2 : 0);
  // inclusive scan of 64 groups' tile counts, from group e0 on
  int2 r;
  int n, incl;
  auto scan = [&](int e0) __attribute__((always_inline)) {
    n = 0;
    r = make_int2(0, 0);
    if (e0 + lane < G) {
      r = group_rows(a.offsets, e0 + lane, a.E, a.R);
      n = (r.y - r.x + BM - 1) / BM;
    }
    incl = wave_scan_sat(n);
  };
  int total = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    scan(e0);
    total = __builtin_elementwise_add_sat(total, __builtin_amdgcn_readlane(incl, 63));
  }
  // A launch has fewer than 2^24 tiles (see plan).  Offsets that decrease can name
  // rows many times over, and their tiles pass 32 bits: then there is none.
  if (uint64_t(uint32_t(total)) * uint32_t(ncol) >= 0x7FFFFFFFu) return false;
  const uint32_t tiles = uint32_t(total) * uint32_t(ncol), per = (tiles + 7) / 8;
  const uint32_t t = (id & 7) * per + (id >> 3);
  if (uint32_t(id >> 3) >= per || t >= tiles) return false;
  const uint32_t high = ncol < 8 ? 4 : 8;
  int want = int(t / uint32_t(ncol));  // BY_GROUP: a row tile of the same group
  auto place = [&](uint32_t t, int total) __attribute__((always_inline)) {  // t's column and row tile, of `total` row tiles
    const uint32_t block = t / (high * ncol), in = t - block * high * ncol;
    const uint32_t wide = min(high, uint32_t(total) - block * high);  // row tiles of this block of columns
    col = int(in / wide);
    return int(block * high + in % wide);
  };
  if (!BY_GROUP) want = place(t, total);
  int before = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    if (G > 64) scan(e0);  // else as it stands
    const uint64_t past = __ballot(before + incl > want);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1, tiles = __builtin_amdgcn_readlane(n, l);
      const int first = before + __builtin_amdgcn_readlane(incl, l) - tiles;
      const int at = BY_GROUP ? place(t - uint32_t(first) * ncol, tiles) : want - first;
      pl.e = e0 + l;
      pl.row0 = __builtin_amdgcn_readlane(r.x, l) + at * BM;
      pl.rows = min(BM, __builtin_amdgcn_readlane(r.y, l) - pl.row0);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// four fp32 results in a 16-bit type, rounded once (to nearest even; NaN and
// infinity stay)
__device__ __forceinline__ uint2 round4(const v4f& v, int ty) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  typedef __bf16 b4 __attribute__((ext_vector_type(4)));
  return ty == kFp16 ? __builtin_bit_cast(uint2, __builtin_convertvector(v, h4))
                     : __builtin_bit_cast(uint2, __builtin_convertvector(v, b4));
}
__device__ __forceinline__ void store4(void* out, long at, const v4f& v, int ty) {
  if (ty == kFp32) *reinterpret_cast<v4f*>(static_cast<float*>(out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = round4(v, ty);
}

// Row tiles of a launch: sum over non-empty groups (and the rows outside them) of ceil(n / rows) at most.
inline long row_tiles(const MmArgs& a, int rows) {
  const long G = (a.E < a.R ? a.E : a.R) + (a.clear_rest ? 2 : 0);
  const long most = (long(a.R) + G * (rows - 1)) / rows;
  return most < a.R ? most : a.R;
}

}  // namespace moe
