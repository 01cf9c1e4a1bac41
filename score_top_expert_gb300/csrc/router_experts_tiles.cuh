// Tiles of the expert products on the tensor cores, shared by their kernels: the
// expert and ragged rows of a tile, bounded waits, and the small arithmetic around
// them.
#pragma once

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_tcgen.cuh"

namespace moe_router {

constexpr int kDeep = 64;     // contraction indices per stage: 128 bytes
constexpr int kSegment = 15;  // most stages per accumulator of a fp32 output

struct TcArgs {
  const int32_t* offsets;
  const int32_t* p2u;
  void* out;
  int* status;
  int T, P, E, N, D;
  int x_rows;  // rows of the gathered x
  uint32_t inv_T;  // floor(2^32 / T), at most 2^32 - 1
};

// S gives a kernel's tile: kTileA values of A's dimension, at most kTileB of B's,
// rounded up to kRound.
struct Tile {
  int e;
  int start, cnt;  // ragged rows (weight grad: the expert's)
  int a0, b0;      // first value of A's dimension; weight grad: of B's
};

template <int FORM, typename S>
__device__ __forceinline__ Tile find_tile(const TcArgs& g, const int* prefix, const int* offs,
                                          int tile) {
  Tile t;
  if constexpr (FORM == EX_WGRAD) {
    const int ta = (g.N + S::kTileA - 1) / S::kTileA, tb = (g.D + S::kTileB - 1) / S::kTileB;
    t.e = tile / (ta * tb);
    const int r = tile - t.e * ta * tb;
    t.a0 = r / tb * S::kTileA;
    t.b0 = r % tb * S::kTileB;
    t.start = offs[t.e];
    t.cnt = max(offs[t.e + 1] - t.start, 0);
  } else {
    const int ta = ((FORM == EX_FWD ? g.N : g.D) + S::kTileA - 1) / S::kTileA;
    t.e = expert_of_tile(prefix, g.E, tile / ta);
    const int first = prefix[t.e], tiles = prefix[t.e + 1] - first;
    const int r = tile - first * ta;
    const int a = r / tiles;  // one slice of the weight, all row tiles, then the next
    const int lo = offs[t.e], hi = max(offs[t.e + 1], lo);
    const int each = ((hi - lo + tiles - 1) / tiles + S::kRound - 1) / S::kRound * S::kRound;
    t.a0 = a * S::kTileA;
    t.start = lo + (r - a * tiles) * each;
    t.cnt = min(each, hi - t.start);
    t.b0 = 0;
  }
  return t;
}

// Waits that give up set the CTA's flag and the device's status word.
struct Waiter {
  int* gave_up;
  int* status;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (mbar_wait_bounded(bar, parity)) return true;
    *reinterpret_cast<volatile int*>(gave_up) = 1;
    atomicExch(status, kDeviceWaitTimeout);
    return false;
  }
};

// Tile *i, or the first one after it in this CTA's sequence that has products
// (weight grad: an expert without rows has none).
template <int FORM, typename S>
__device__ __forceinline__ Tile next_tile(const TcArgs& g, const int* prefix, const int* offs,
                                          int tiles, int step, int* i) {
  Tile t{};
  while (*i < tiles) {
    t = find_tile<FORM, S>(g, prefix, offs, *i);
    if (FORM != EX_WGRAD || t.cnt > 0) break;
    *i += step;
  }
  return t;
}

// floor(2^32 / T), at most 2^32 - 1.
inline uint32_t inverse_of(int T) {
  return T > 1 ? static_cast<uint32_t>((1ull << 32) / T) : 0xffffffffu;
}

// u mod T.  u inv_T / 2^32 is below u / T by less than 1, so its floor is the
// quotient or one less.
__device__ __forceinline__ int token_of(const TcArgs& g, int u) {
  const int r = u - static_cast<int>(__umulhi(static_cast<uint32_t>(u), g.inv_T)) * g.T;
  return r >= g.T ? r - g.T : r;
}

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Adds v to *p without reading it back.
__device__ __forceinline__ void red_add(float* p, float v) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}

// Stages per accumulator of a tile: all of them, or for a fp32 output near-equal
// shares of at most `most`.
template <bool F32>
__device__ __forceinline__ int segment_of(int slices, int most = kSegment) {
  if (!F32 || slices <= most) return slices;
  const int parts = (slices + most - 1) / most;
  return (slices + parts - 1) / parts;
}

}  // namespace moe_router
