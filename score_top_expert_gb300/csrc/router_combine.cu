// Weighted combination of the experts' outputs and its gradients.
//
//   forward   y[t] = sum_k w[t, k] z[p(t, k)],      p(t, k) = u2p[t + k T]
//   backward  gz[p(t, k)] = w[t, k] gy[t],   gw[t, k] = gy[t] . z[p(t, k)]
//
// Both stream rows once and are bound by HBM; the sums are fp32 in a fixed
// order (k ascending; for the dots lanes, then warps), so results repeat bit
// for bit.  A choice without a permuted row (-1, or outside [0, T K)) is left
// out of the sum and gets the gradient 0.
#include "router_common.cuh"
#include "router_experts.cuh"

namespace moe_router {
namespace {

// What a lane holds of a stretch of 32 kN columns of a row, as it was loaded (so
// that rows in flight take few registers), widened to fp32 when used.  BYTES is
// what one access takes: 16 where every row is 16-byte aligned, else 4 or 2, in
// four accesses 32 lanes apart, so that each is contiguous over the warp.
template <int DT, int BYTES>
struct Piece {
  static constexpr int kSize = DT == DT_F32 ? 4 : 2;
  static constexpr int kEach = BYTES / kSize;                          // columns per access
  static constexpr int kAccesses = BYTES == 16 ? 1 : 4;
  static constexpr int kN = kEach * kAccesses;
  static constexpr int kWords = BYTES == 16 ? 4 : kAccesses;
  uint32_t w[kWords];

  __device__ __forceinline__ static int column(int col0, int q, int lane) {
    return col0 + (q * 32 + lane) * kEach;
  }

  // The row starts at element `row` of base and has D columns.  STREAM: not kept
  // in L1 (the forward's rows; it costs the backward 2 to 6 %).
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* base, size_t row, int col0, int lane, int D) {
    const uint8_t* at = static_cast<const uint8_t*>(base) + row * kSize;
#pragma unroll
    for (int q = 0; q < kAccesses; ++q) {
      const int c = column(col0, q, lane);
      if (BYTES != 16) w[q] = 0u;
      if (c >= D) continue;
      if constexpr (BYTES == 16) {
        const uint4 t = get<STREAM>(reinterpret_cast<const uint4*>(at + c * kSize));
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      } else if constexpr (BYTES == 4) {
        w[q] = get<STREAM>(reinterpret_cast<const unsigned int*>(at + c * kSize));
      } else {
        w[q] = get<STREAM>(reinterpret_cast<const unsigned short*>(at + c * kSize));
      }
    }
  }

  template <bool STREAM, typename W>
  __device__ __forceinline__ static W get(const W* p) {
    return STREAM ? __ldcs(p) : __ldg(p);
  }

  // value j is column (j / kEach, j % kEach)
  __device__ __forceinline__ void widen(float (&v)[kN]) const {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = __uint_as_float(w[j]);
    } else if constexpr (BYTES == 2) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = bf16_bits_to_f32(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }

  __device__ __forceinline__ static void store(void* base, size_t row, int col0, int lane, int D,
                                               const float (&v)[kN]) {
    uint8_t* at = static_cast<uint8_t*>(base) + row * kSize;
    uint32_t u[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (DT == DT_F32) {
        u[j] = __float_as_uint(v[j]);
      } else if constexpr (BYTES == 2) {
        u[j] = f32_to_bf16_bits(v[j]);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
#pragma unroll
    for (int q = 0; q < kAccesses; ++q) {
      const int c = column(col0, q, lane);
      if (c >= D) continue;
      if constexpr (BYTES == 16)
        __stcs(reinterpret_cast<uint4*>(at + c * kSize), make_uint4(u[0], u[1], u[2], u[3]));
      else if constexpr (BYTES == 4)
        __stcs(reinterpret_cast<unsigned int*>(at + c * kSize), u[q]);
      else
        __stcs(reinterpret_cast<unsigned short*>(at + c * kSize), static_cast<unsigned short>(u[q]));
    }
  }
};

constexpr int kUnroll = 4;  // backward: rows in flight per thread

// A warp sums one stretch of one token's row: its lanes hold the token's choices
// (two each for K > 32), handed round by shuffles, and load UNROLL rows ahead of
// the sum.  Eight rows in flight and four blocks an SM (8192 tokens, 8 choices,
// 2048 bf16: 57 us, 61 with three blocks, 59 with four rows and five blocks),
// four rows for K <= 4 (4096 columns: 72 us against 80).
template <int DT, int BYTES, int UNROLL>
__global__ __launch_bounds__(256, UNROLL == 8 ? 4 : BYTES != 16 ? 5 : 1) void combine_fwd_kernel(
    CombineArgs a, int stretches) {
  pdl_enter();
  using P = Piece<DT, BYTES>;
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / stretches);
  if (t >= a.T) return;
  const int col0 = static_cast<int>(unit - static_cast<long long>(t) * stretches) * 32 * P::kN;
  const unsigned rows = static_cast<unsigned>(a.T) * static_cast<unsigned>(a.K);
  int p0 = -1, p1 = -1;
  float w0 = 0.0f, w1 = 0.0f;
  if (lane < a.K) {
    p0 = a.u2p[t + static_cast<size_t>(lane) * a.T];
    w0 = a.weights != nullptr ? a.weights[t * a.ld_w + lane] : 1.0f;
  }
  if (lane + 32 < a.K) {
    p1 = a.u2p[t + static_cast<size_t>(lane + 32) * a.T];
    w1 = a.weights != nullptr ? a.weights[t * a.ld_w + lane + 32] : 1.0f;
  }
  if (static_cast<unsigned>(p0) >= rows) p0 = -1;
  if (static_cast<unsigned>(p1) >= rows) p1 = -1;
  float acc[P::kN];
#pragma unroll
  for (int j = 0; j < P::kN; ++j) acc[j] = 0.0f;
  for (int k0 = 0; k0 < a.K; k0 += UNROLL) {
    int p[UNROLL];
    float w[UNROLL];
    P z[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int k = k0 + u;  // the same for all lanes; past K the lane's own choice is empty
      p[u] = __shfl_sync(0xffffffffu, k < 32 ? p0 : p1, k & 31);
      w[u] = __shfl_sync(0xffffffffu, k < 32 ? w0 : w1, k & 31);
      if (p[u] >= 0)
        z[u].template load<true>(a.z, static_cast<size_t>(p[u]) * a.D, col0, lane, a.D);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (p[u] < 0) continue;
      float v[P::kN];
      z[u].widen(v);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) acc[j] = fmaf(w[u], v[j], acc[j]);
    }
  }
  P::store(a.out, static_cast<size_t>(t) * a.D, col0, lane, a.D, acc);
}

// A block takes one token: kUnroll choices at a time, each warp its stretches of
// the row, every z row read and every gz row written once; the token's own row
// comes from L1 after its first reading.
template <int DT, int BYTES>
__global__ __launch_bounds__(256) void combine_bwd_kernel(CombineArgs a) {
  __shared__ float part[MR_MAX_TOPK][8];
  pdl_enter();
  using P = Piece<DT, BYTES>;
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const unsigned rows = static_cast<unsigned>(a.T) * static_cast<unsigned>(a.K);
  const size_t gy_row = static_cast<size_t>(t) * a.D;
  const bool dots = a.grad_weights != nullptr;
  for (int k0 = 0; k0 < a.K; k0 += kUnroll) {
    int p[kUnroll];
    float w[kUnroll], dot[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u;
      p[u] = k < a.K ? a.u2p[t + static_cast<size_t>(k) * a.T] : -1;
      if (static_cast<unsigned>(p[u]) >= rows) p[u] = -1;
      w[u] = (k < a.K && a.weights != nullptr) ? a.weights[t * a.ld_w + k] : 1.0f;
      dot[u] = 0.0f;
    }
    for (int col0 = warp * 32 * P::kN; col0 < a.D; col0 += warps * 32 * P::kN) {
      P g, z[kUnroll];
      float gy[P::kN];
      g.template load<false>(a.gy, gy_row, col0, lane, a.D);
      if (dots) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (p[u] >= 0)
            z[u].template load<false>(a.z, static_cast<size_t>(p[u]) * a.D, col0, lane, a.D);
      }
      g.widen(gy);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p[u] < 0) continue;
        float gz[P::kN], v[P::kN];
        if (dots) {
          z[u].widen(v);
          // columns past the row are not loaded (16-byte pieces) or zero
          if (BYTES != 16 || P::column(col0, 0, lane) < a.D) {
#pragma unroll
            for (int j = 0; j < P::kN; ++j) dot[u] = fmaf(gy[j], v[j], dot[u]);
          }
        }
#pragma unroll
        for (int j = 0; j < P::kN; ++j) gz[j] = w[u] * gy[j];
        P::store(a.out, static_cast<size_t>(p[u]) * a.D, col0, lane, a.D, gz);
      }
    }
    if (dots) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float d = seg_sum<32>(dot[u]);
        if (lane == 0 && k0 + u < a.K) part[k0 + u][warp] = d;
      }
    }
  }
  if (!dots) return;
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    float d = 0.0f;
    for (int w = 0; w < warps; ++w) d += part[k][w];
    a.grad_weights[static_cast<size_t>(t) * a.K + k] = d;
  }
}

// Bytes of one access: what every row of the three tensors is aligned to.
int access_bytes(const CombineArgs& a) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.gy) |
                        reinterpret_cast<uintptr_t>(a.out) |
                        static_cast<uintptr_t>(a.D) * (a.dtype == DT_F32 ? 4 : 2);
  return (all & 15u) == 0 ? 16 : (all & 3u) == 0 ? 4 : 2;
}

template <int DT, int BYTES>
int fwd_typed(const CombineArgs& a, cudaStream_t st) {
  constexpr int width = 32 * Piece<DT, BYTES>::kN;
  const int stretches = (a.D + width - 1) / width;
  const long long blocks = (static_cast<long long>(a.T) * stretches + 7) / 8;
  if (blocks > 0x7fffffffll) return MR_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaError_t e =
      a.K <= 4 || BYTES != 16
          ? launch_kernel(combine_fwd_kernel<DT, BYTES, 4>, grid, dim3(256), 0, st, a, stretches)
          : launch_kernel(combine_fwd_kernel<DT, 16, 8>, grid, dim3(256), 0, st, a, stretches);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int DT, int BYTES>
int bwd_typed(const CombineArgs& a, cudaStream_t st) {
  constexpr int width = 32 * Piece<DT, BYTES>::kN;
  const int warps = (a.D + width - 1) / width;
  const cudaError_t e = launch_kernel(combine_bwd_kernel<DT, BYTES>, dim3(a.T),
                                      dim3(32 * (warps < 8 ? warps : 8)), 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

}  // namespace

int launch_combine_fwd(const CombineArgs& a, cudaStream_t st) {
  const int bytes = access_bytes(a);
  if (a.dtype == DT_F32)
    return bytes == 16 ? fwd_typed<DT_F32, 16>(a, st) : fwd_typed<DT_F32, 4>(a, st);
  return bytes == 16  ? fwd_typed<DT_BF16, 16>(a, st)
         : bytes == 4 ? fwd_typed<DT_BF16, 4>(a, st)
                      : fwd_typed<DT_BF16, 2>(a, st);
}

int launch_combine_bwd(const CombineArgs& a, cudaStream_t st) {
  const int bytes = access_bytes(a);
  if (a.dtype == DT_F32)
    return bytes == 16 ? bwd_typed<DT_F32, 16>(a, st) : bwd_typed<DT_F32, 4>(a, st);
  return bytes == 16  ? bwd_typed<DT_BF16, 16>(a, st)
         : bytes == 4 ? bwd_typed<DT_BF16, 4>(a, st)
                      : bwd_typed<DT_BF16, 2>(a, st);
}

}  // namespace moe_router
