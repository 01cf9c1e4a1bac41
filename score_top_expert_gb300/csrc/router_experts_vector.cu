// Products grouped by expert on the vector units: fp32 operands, and bf16
// operands whose rows are not 16-byte aligned.  Products and sums are fp32.
//
// A block of 256 threads computes a 64 x 64 tile of one expert's output, 4 x 4
// values a thread, from 16-deep slices of both operands that it stages in
// shared memory as fp32, indexed contraction-first so that the inner loop
// reads both fragments as float4.  Elements are loaded one by one (any
// alignment), neighbouring threads along whichever index is contiguous.
#include "router_common.cuh"
#include "router_experts.cuh"

namespace moe_router {
namespace {

constexpr int kTile = 64;   // rows and columns of an output tile
constexpr int kDeep = 16;   // contraction slice
constexpr int kThreads = 256;
constexpr int kPad = 4;     // keeps float4 rows aligned, spreads the transposed stores

template <typename T>
__device__ __forceinline__ float as_f32(T v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<unsigned short>(unsigned short v) {
  return bf16_bits_to_f32(v);
}

__device__ __forceinline__ void store_out(void* out, int dtype, size_t i, float v) {
  if (dtype == DT_F32) static_cast<float*>(out)[i] = v;
  else static_cast<unsigned short*>(out)[i] = static_cast<unsigned short>(f32_to_bf16_bits(v));
}

template <typename TIn, int FORM>
__global__ __launch_bounds__(kThreads) void expert_matmul_vector_kernel(ExpertArgs g) {
  __shared__ int prefix[MR_MAX_EXPERTS + 1];
  __shared__ int tmp[33];
  __shared__ __align__(16) float sa[kDeep][kTile + kPad];
  __shared__ __align__(16) float sb[kDeep][kTile + kPad];
  __shared__ int row_of[kTile];  // forward: x rows of the tile; weight grad: of the slice

  pdl_enter();
  const TIn* __restrict__ A = static_cast<const TIn*>(g.a);
  const TIn* __restrict__ B = static_cast<const TIn*>(g.b);
  const int cols = FORM == EX_FWD ? g.N : g.D;  // columns of the output
  const int col_tiles = (cols + kTile - 1) / kTile;
  long long tiles;
  if (FORM == EX_WGRAD) {
    tiles = static_cast<long long>(g.E) * ((g.N + kTile - 1) / kTile) * col_tiles;
  } else {
    tiles = static_cast<long long>(expert_tile_prefix(g.offsets, g.E, g.P, kTile, prefix, tmp)) *
            col_tiles;
  }
  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;  // 4 columns, 4 rows each

  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int ct = static_cast<int>(tile % col_tiles);
    const int q = static_cast<int>(tile / col_tiles);
    int e, lo, hi, row0, rows;
    if (FORM == EX_WGRAD) {
      const int row_tiles = (g.N + kTile - 1) / kTile;
      e = q / row_tiles;
      row0 = (q - e * row_tiles) * kTile;
      rows = min(kTile, g.N - row0);
      expert_rows(g.offsets, e, g.P, &lo, &hi);
    } else {
      e = expert_of_tile(prefix, g.E, q);
      expert_rows(g.offsets, e, g.P, &lo, &hi);
      row0 = lo + (q - prefix[e]) * kTile;
      rows = min(kTile, hi - row0);
    }
    const int col0 = ct * kTile;
    const int ncols = min(kTile, cols - col0);
    const int depth = FORM == EX_FWD ? g.D : FORM == EX_DGRAD ? g.N : hi - lo;
    if (FORM == EX_FWD) {
      __syncthreads();  // the previous tile's readers of row_of
      if (tid < kTile) row_of[tid] = tid < rows ? source_row(g.p2u, g.T, row0 + tid) : -1;
      __syncthreads();
    }
    float acc[4][4] = {};
    for (int k0 = 0; k0 < depth; k0 += kDeep) {
      const int deep = min(kDeep, depth - k0);
      if (FORM == EX_WGRAD) {
        __syncthreads();
        if (tid < kDeep) row_of[tid] = tid < deep ? source_row(g.p2u, g.T, lo + k0 + tid) : -1;
      }
      __syncthreads();  // the previous slice has been read
      for (int i = tid; i < kTile * kDeep; i += kThreads) {
        {
          // rows of the output.  Contraction contiguous except in the weight grad
          const int m = FORM == EX_WGRAD ? i % kTile : i / kDeep;
          const int k = FORM == EX_WGRAD ? i / kTile : i % kDeep;
          float v = 0.0f;
          if (m < rows && k < deep) {
            if (FORM == EX_FWD) {
              const int r = row_of[m];
              if (r >= 0) v = as_f32(A[static_cast<size_t>(r) * g.D + k0 + k]);
            } else if (FORM == EX_DGRAD) {
              v = as_f32(A[static_cast<size_t>(row0 + m) * g.N + k0 + k]);
            } else if (row_of[k] >= 0) {  // a row without a source counts in neither operand
              v = as_f32(A[static_cast<size_t>(lo + k0 + k) * g.N + row0 + m]);
            }
          }
          sa[k][m] = v;
        }
        {
          // columns of the output.  Contraction contiguous in the forward
          const int n = FORM == EX_FWD ? i / kDeep : i % kTile;
          const int k = FORM == EX_FWD ? i % kDeep : i / kTile;
          float v = 0.0f;
          if (n < ncols && k < deep) {
            if (FORM == EX_FWD)
              v = as_f32(B[(static_cast<size_t>(e) * g.N + col0 + n) * g.D + k0 + k]);
            else if (FORM == EX_DGRAD)
              v = as_f32(B[(static_cast<size_t>(e) * g.N + k0 + k) * g.D + col0 + n]);
            else if (row_of[k] >= 0)
              v = as_f32(B[static_cast<size_t>(row_of[k]) * g.D + col0 + n]);
          }
          sb[k][n] = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const float4 a4 = *reinterpret_cast<const float4*>(&sa[k][ty * 4]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[k][tx * 4]);
        const float av[4] = {a4.x, a4.y, a4.z, a4.w};
        const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = ty * 4 + i;
      if (m >= rows) continue;
      const size_t base = (FORM == EX_WGRAD ? static_cast<size_t>(e) * g.N + row0 + m
                                            : static_cast<size_t>(row0 + m)) * cols + col0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tx * 4 + j < ncols) store_out(g.out, g.out_dtype, base + tx * 4 + j, acc[i][j]);
    }
  }
}

template <typename TIn, int FORM>
int launch_typed(const ExpertArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MR_ERR_CUDA;
  const long long cols = ((FORM == EX_FWD ? a.N : a.D) + kTile - 1) / kTile;
  const long long rows = FORM == EX_WGRAD
                             ? static_cast<long long>(a.E) * ((a.N + kTile - 1) / kTile)
                             : static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / kTile;
  const long long most = 6ll * sms;
  const int grid = static_cast<int>(rows * cols < most ? rows * cols : most);
  const cudaError_t e = launch_kernel(expert_matmul_vector_kernel<TIn, FORM>, dim3(grid),
                                      dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

}  // namespace

int launch_expert_matmul_vector(int form, const ExpertArgs& a, cudaStream_t st) {
  if (a.dtype == DT_F32)
    return form == EX_FWD     ? launch_typed<float, EX_FWD>(a, st)
           : form == EX_DGRAD ? launch_typed<float, EX_DGRAD>(a, st)
                              : launch_typed<float, EX_WGRAD>(a, st);
  return form == EX_FWD     ? launch_typed<unsigned short, EX_FWD>(a, st)
         : form == EX_DGRAD ? launch_typed<unsigned short, EX_DGRAD>(a, st)
                            : launch_typed<unsigned short, EX_WGRAD>(a, st);
}

}  // namespace moe_router
