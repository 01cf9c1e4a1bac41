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

// One 16-byte vector (VEC) or one element of a row, held as it was loaded (so
// that rows in flight take four registers) and widened to fp32 when used.
template <int DT, bool VEC>
struct Piece {
  static constexpr int kN = !VEC ? 1 : DT == DT_F32 ? 4 : 8;
  static constexpr int kWords = VEC ? 4 : 1;
  uint32_t w[kWords];

  // STREAM: not kept in L1 (the forward's rows; it costs the backward 2 to 6 %)
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* base, size_t i) {
    const uint8_t* at = static_cast<const uint8_t*>(base) + i * (DT == DT_F32 ? 4 : 2);
    if constexpr (!VEC) {
      if (DT == DT_F32) w[0] = get<STREAM>(reinterpret_cast<const unsigned int*>(at));
      else w[0] = get<STREAM>(reinterpret_cast<const unsigned short*>(at));
    } else {
      const uint4 t = get<STREAM>(reinterpret_cast<const uint4*>(at));
      w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    }
  }

  template <bool STREAM, typename W>
  __device__ __forceinline__ static W get(const W* p) {
    return STREAM ? __ldcs(p) : __ldg(p);
  }

  __device__ __forceinline__ void widen(float (&v)[kN]) const {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = __uint_as_float(w[j]);
    } else if constexpr (!VEC) {
      v[0] = bf16_bits_to_f32(w[0]);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }

  __device__ __forceinline__ static void store(void* base, size_t i, const float (&v)[kN]) {
    if constexpr (!VEC) {
      if (DT == DT_F32) __stcs(static_cast<float*>(base) + i, v[0]);
      else __stcs(static_cast<unsigned short*>(base) + i,
                  static_cast<unsigned short>(f32_to_bf16_bits(v[0])));
    } else if constexpr (DT == DT_F32) {
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(base) + i),
             make_float4(v[0], v[1], v[2], v[3]));
    } else {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      __stcs(reinterpret_cast<uint4*>(static_cast<unsigned short*>(base) + i),
             make_uint4(u[0], u[1], u[2], u[3]));
    }
  }
};

constexpr int kUnroll = 4;  // backward: rows in flight per thread

// A warp sums one stretch of 32 pieces of one token's row: its lanes hold the
// token's choices (two each for K > 32), handed round by shuffles, and load
// UNROLL rows ahead of the sum.
// Eight rows in flight and four blocks an SM (8192 tokens, 8 choices, 2048 bf16:
// 57 us, 61 with three blocks, 59 with four rows and five blocks), four rows for
// K <= 4 (4096 columns: 72 us against 80).
template <int DT, bool VEC, int UNROLL>
__global__ __launch_bounds__(256, UNROLL == 8 ? 4 : 1) void combine_fwd_kernel(CombineArgs a, int stretches) {
  pdl_enter();
  constexpr int N = Piece<DT, VEC>::kN;
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / stretches);
  if (t >= a.T) return;
  const int col = (static_cast<int>(unit - static_cast<long long>(t) * stretches) * 32 + lane) * N;
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
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  for (int k0 = 0; k0 < a.K; k0 += UNROLL) {
    int p[UNROLL];
    float w[UNROLL];
    Piece<DT, VEC> z[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int k = k0 + u;  // the same for all lanes; past K the lane's own choice is empty
      p[u] = __shfl_sync(0xffffffffu, k < 32 ? p0 : p1, k & 31);
      w[u] = __shfl_sync(0xffffffffu, k < 32 ? w0 : w1, k & 31);
      if (p[u] >= 0 && col < a.D) z[u].template load<true>(a.z, static_cast<size_t>(p[u]) * a.D + col);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (p[u] < 0 || col >= a.D) continue;
      float v[N];
      z[u].widen(v);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(w[u], v[j], acc[j]);
    }
  }
  if (col < a.D) Piece<DT, VEC>::store(a.out, static_cast<size_t>(t) * a.D + col, acc);
}

// A block takes one token: kUnroll choices at a time, each thread its pieces
// of the row, every z row read and every gz row written once; the token's own
// row comes from L1 after its first reading.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void combine_bwd_kernel(CombineArgs a) {
  __shared__ float part[MR_MAX_TOPK][8];
  pdl_enter();
  constexpr int N = Piece<DT, VEC>::kN;
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const unsigned rows = static_cast<unsigned>(a.T) * static_cast<unsigned>(a.K);
  const size_t gy0 = static_cast<size_t>(t) * a.D;
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
    for (int col = threadIdx.x * N; col < a.D; col += blockDim.x * N) {
      Piece<DT, VEC> g, z[kUnroll];
      float gy[N];
      g.template load<false>(a.gy, gy0 + col);
      if (dots) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (p[u] >= 0) z[u].template load<false>(a.z, static_cast<size_t>(p[u]) * a.D + col);
      }
      g.widen(gy);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p[u] < 0) continue;
        float gz[N], v[N];
        if (dots) z[u].widen(v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (dots) dot[u] = fmaf(gy[j], v[j], dot[u]);
          gz[j] = w[u] * gy[j];
        }
        Piece<DT, VEC>::store(a.out, static_cast<size_t>(p[u]) * a.D + col, gz);
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows that can be read in 16-byte pieces.
bool vector_rows(const CombineArgs& a) {
  return a.D % (a.dtype == DT_F32 ? 4 : 8) == 0 && aligned16(a.z) && aligned16(a.gy) &&
         aligned16(a.out);
}

template <int DT, bool VEC>
int fwd_typed(const CombineArgs& a, cudaStream_t st) {
  constexpr int N = Piece<DT, VEC>::kN;
  const int stretches = (a.D + 32 * N - 1) / (32 * N);
  const long long blocks = (static_cast<long long>(a.T) * stretches + 7) / 8;
  if (blocks > 0x7fffffffll) return MR_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaError_t e =
      a.K <= 4 ? launch_kernel(combine_fwd_kernel<DT, VEC, 4>, grid, dim3(256), 0, st, a, stretches)
               : launch_kernel(combine_fwd_kernel<DT, VEC, 8>, grid, dim3(256), 0, st, a, stretches);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int DT, bool VEC>
int bwd_typed(const CombineArgs& a, cudaStream_t st) {
  constexpr int N = Piece<DT, VEC>::kN;
  const int warps = (a.D + 32 * N - 1) / (32 * N);
  const cudaError_t e = launch_kernel(combine_bwd_kernel<DT, VEC>, dim3(a.T),
                                      dim3(32 * (warps < 8 ? warps : 8)), 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

}  // namespace

int launch_combine_fwd(const CombineArgs& a, cudaStream_t st) {
  const bool vec = vector_rows(a);
  if (a.dtype == DT_F32) return vec ? fwd_typed<DT_F32, true>(a, st) : fwd_typed<DT_F32, false>(a, st);
  return vec ? fwd_typed<DT_BF16, true>(a, st) : fwd_typed<DT_BF16, false>(a, st);
}

int launch_combine_bwd(const CombineArgs& a, cudaStream_t st) {
  const bool vec = vector_rows(a);
  if (a.dtype == DT_F32) return vec ? bwd_typed<DT_F32, true>(a, st) : bwd_typed<DT_F32, false>(a, st);
  return vec ? bwd_typed<DT_BF16, true>(a, st) : bwd_typed<DT_BF16, false>(a, st);
}

}  // namespace moe_router
