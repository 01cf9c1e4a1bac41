// Shared parts of the expert-side operators: the products of each expert's
// weight with its rows (forward, both gradients, 4-bit weights) and the
// weighted combination of the experts' outputs.
//
// The routed rows lie in the maps' order: expert e owns the permuted rows
// [offset[e], offset[e + 1]).  The offsets are on the device and the host
// launches without reading them, so each kernel finds its tiles itself: a
// block adds up the row tiles of all experts once (one pass over E offsets)
// and looks its tiles up by bisection in shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_router.h"

namespace moe_router {

// Arguments of the three products; which of a, b, out is what:
//   forward       a = x [T or P, D], b = weight [E, N, D], out [P, N]
//   input grad    a = grad_out [P, N], b = weight [E, N, D], out [P, D]
//   weight grad   a = grad_out [P, N], b = x [T or P, D], out [E, N, D]
struct ExpertArgs {
  const void* a;
  const void* b;
  const int32_t* offsets;  // [E + 1]
  const int32_t* p2u;      // [P] or NULL: rows of x are permuted rows
  void* out;
  int T;  // rows of x when p2u is given
  int P, E, N, D;
  int dtype, out_dtype;
};

enum { EX_FWD = 0, EX_DGRAD = 1, EX_WGRAD = 2 };

struct W4Args {
  const void* x;  // bf16 [T or P, D]
  const uint8_t* q;
  const void* scales;  // bf16 [E, N, D / group]
  const uint8_t* zeros;
  const int32_t* offsets;
  const int32_t* p2u;
  void* out;
  int T, P, E, N, D, group, out_dtype;
};

struct CombineArgs {
  const void* z;         // expert outputs [T K, D]
  const void* gy;        // grad of the sums [T, D]
  const int32_t* u2p;    // [T K]
  const float* weights;  // [T, ld_w] or NULL
  void* out;             // forward [T, D]; backward grad of z [T K, D]
  float* grad_weights;   // [T, K] or NULL
  long long ld_w;
  int T, K, D, dtype;
};

// SMs of the current device, and its status word (router_api.cu).
int device_sm_count();
int* device_status_word();

// Each returns an MR_* status; arguments already checked.
bool expert_matmul_tc_ok(int form, const ExpertArgs& a);  // types and alignment qualify
int launch_expert_matmul_tc(int form, const ExpertArgs& a, cudaStream_t st);
bool expert_matmul_few_ok(const ExpertArgs& a);
int launch_expert_matmul_few(const ExpertArgs& a, cudaStream_t st);  // forward only
int launch_expert_matmul_split(int form, const ExpertArgs& a, cudaStream_t st);  // any operands
int launch_expert_matmul_w4(const W4Args& a, cudaStream_t st);
int launch_combine_fwd(const CombineArgs& a, cudaStream_t st);
int launch_combine_bwd(const CombineArgs& a, cudaStream_t st);

// ---------------------------------------------------------------------------
// device side
// ---------------------------------------------------------------------------

// Expert e's permuted rows [lo, hi).  Offsets outside [0, P] or out of order
// are clamped, so no kernel leaves its buffers whatever the map holds.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int P, int* lo,
                                            int* hi) {
  const int a = min(max(offsets[e], 0), P);
  *lo = a;
  *hi = min(max(offsets[e + 1], a), P);
}

// prefix[e] = row tiles of the experts before e (prefix[E]: of all), where an
// expert of n rows has ceil(n / rows_per_tile).  Every thread of the block (a
// multiple of 32 threads, at most 1024) calls it; prefix (E + 1 ints) and tmp
// (33 ints) are in shared memory.  Thread i adds up a contiguous run of
// experts; the runs' sums are scanned by warp shuffles.
__device__ __forceinline__ int expert_tile_prefix(const int32_t* __restrict__ offsets, int E,
                                                  int P, int rows_per_tile, int* prefix,
                                                  int* tmp) {
  const int nthreads = blockDim.x;
  const int per = (E + nthreads - 1) / nthreads;
  const int b0 = threadIdx.x * per;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int local = 0;
  if (b0 < E) {
    const int b1 = min(b0 + per, E);
    int lo = min(max(offsets[b0], 0), P);
    for (int e = b0; e < b1; ++e) {
      // the expert's own range, clamped as in expert_rows
      const int hi = min(max(offsets[e + 1], 0), P);
      prefix[e] = local;
      local += (max(hi - lo, 0) + rows_per_tile - 1) / rows_per_tile;
      lo = hi;
    }
  }
  int x = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = x - local;
  for (int w = 0; w < warp; ++w) before += tmp[w];
  for (int e = b0; e < min(b0 + per, E); ++e) prefix[e] += before;
  if (threadIdx.x == nthreads - 1) prefix[E] = before + local;
  __syncthreads();
  return prefix[E];
}

// The expert whose row tiles contain tile q: prefix[e] <= q < prefix[e + 1].
__device__ __forceinline__ int expert_of_tile(const int* prefix, int E, int q) {
  int lo = 0, hi = E;  // prefix[lo] <= q < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= q) lo = mid; else hi = mid;
  }
  return lo;
}

// Row of x behind permuted row p: token u mod T of its expanded row u = t +
// k T, or p itself without a map; -1 for a map entry below zero.
__device__ __forceinline__ int source_row(const int32_t* __restrict__ p2u, int T, int p) {
  if (p2u == nullptr) return p;
  const int u = p2u[p];
  return u < 0 ? -1 : u % T;
}

}  // namespace moe_router
