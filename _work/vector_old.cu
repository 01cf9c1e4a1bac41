// Products grouped by expert on the vector units: fp32 operands, and bf16
// operands whose rows are not 16-byte aligned.  Products and sums are fp32.
//
// A block of 128 threads computes a ROWS x 64 tile of one expert's output, ROWS
// / 8 x 4 values a thread, from 16-deep slices of both operands that it stages
// in shared memory as fp32, indexed contraction-first so that the inner loop
// reads both fragments as float4 (the rows' fragment is the same address for
// half a warp).  Two slices are staged: the next one is read from global memory
// into registers while the present one is multiplied, one barrier a slice.
// Elements are loaded one by one (any alignment), neighbouring threads along
// whichever index is contiguous.
#include "router_common.cuh"
#include "router_experts.cuh"

namespace moe_router {
namespace {

constexpr int kCols = 64;    // columns of an output tile
constexpr int kDeep = 16;    // contraction slice
constexpr int kThreads = 128;
constexpr int kPad = 4;      // keeps float4 rows aligned, spreads the transposed stores

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

template <typename TIn, int FORM, int ROWS>
__global__ __launch_bounds__(kThreads) void expert_matmul_vector_kernel(ExpertArgs g) {
  constexpr int kOwn = ROWS / 8;              // rows per thread
  constexpr int kLoadA = ROWS * kDeep / kThreads, kLoadB = kCols * kDeep / kThreads;
  // Elements a thread loads: kLoadA of the rows' operand at (row, deep), with
  // one of the two fixed.  Along the contraction: deep = tid % 16, rows 8 apart;
  // along the rows: row = tid % ROWS, deep kThreads / ROWS apart.  Same for B.
  constexpr bool kDeepA = FORM != EX_WGRAD, kDeepB = FORM == EX_FWD;
  __shared__ int prefix[FORM == EX_WGRAD ? 1 : MR_MAX_EXPERTS + 1];
  __shared__ int tmp[33];
  __shared__ __align__(16) float sa[2][kDeep][ROWS + kPad];
  __shared__ __align__(16) float sb[2][kDeep][kCols + kPad];

  pdl_enter();
  const TIn* __restrict__ A = static_cast<const TIn*>(g.a);
  const TIn* __restrict__ B = static_cast<const TIn*>(g.b);
  const int cols = FORM == EX_FWD ? g.N : g.D;  // columns of the output
  const int col_tiles = (cols + kCols - 1) / kCols;
  const int w_tiles = (g.N + ROWS - 1) / ROWS;  // weight grad: row tiles of an expert
  long long tiles;
  if (FORM == EX_WGRAD)
    tiles = static_cast<long long>(g.E) * w_tiles * col_tiles;
  else
    tiles = static_cast<long long>(expert_tile_prefix(g.offsets, g.E, g.P, ROWS, prefix, tmp)) *
            col_tiles;
  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;  // 4 columns, kOwn rows each

  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int ct = static_cast<int>(tile % col_tiles);
    const int q = static_cast<int>(tile / col_tiles);
    int e, lo, hi, row0, rows;
    if (FORM == EX_WGRAD) {
      e = q / w_tiles;
      row0 = (q - e * w_tiles) * ROWS;
      rows = min(ROWS, g.N - row0);
      expert_rows(g.offsets, e, g.P, &lo, &hi);
    } else {
      e = expert_of_tile(prefix, g.E, q);
      expert_rows(g.offsets, e, g.P, &lo, &hi);
      row0 = lo + (q - prefix[e]) * ROWS;
      rows = min(ROWS, hi - row0);
    }
    const int col0 = ct * kCols;
    const int ncols = min(kCols, cols - col0);
    const int depth = FORM == EX_FWD ? g.D : FORM == EX_DGRAD ? g.N : hi - lo;

    // this thread's elements of slice 0
    const int ka = kDeepA ? tid % kDeep : tid / ROWS, ma = kDeepA ? tid / kDeep : tid % ROWS;
    const int kb = kDeepB ? tid % kDeep : tid / kCols, nb = kDeepB ? tid / kDeep : tid % kCols;
    const TIn* pa[kDeepA ? kLoadA : 1];
    bool va[kDeepA ? kLoadA : 1];
    if constexpr (kDeepA) {
#pragma unroll
      for (int j = 0; j < kLoadA; ++j) {
        const int m = ma + j * (kThreads / kDeep);
        int r = row0 + min(m, rows - 1);
        if (FORM == EX_FWD) r = source_row(g.p2u, g.T, r);
        va[j] = m < rows && r >= 0;
        pa[j] = A + static_cast<size_t>(max(r, 0)) * depth + ka;
      }
    } else {
      va[0] = ma < rows;
      pa[0] = A + static_cast<size_t>(lo) * g.N + row0 + ma;
    }
    const TIn* pb;
    size_t step_b;  // between this thread's elements of one slice
    if (FORM == EX_FWD) {
      pb = B + (static_cast<size_t>(e) * g.N + col0 + nb) * g.D + kb;
      step_b = static_cast<size_t>(kThreads / kDeep) * g.D;
    } else {
      pb = FORM == EX_DGRAD ? B + (static_cast<size_t>(e) * g.N + kb) * g.D + col0 + nb
                            : B + col0 + nb;
      step_b = static_cast<size_t>(kThreads / kCols) * g.D;
    }

    float ra[kLoadA], rb[kLoadB];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int j = 0; j < kLoadA; ++j) {
        if constexpr (kDeepA) {
          ra[j] = va[j] && k0 + ka < depth ? as_f32(pa[j][k0]) : 0.0f;
        } else {
          const int k = k0 + ka + j * (kThreads / ROWS);
          ra[j] = va[0] && k < depth ? as_f32(pa[0][static_cast<size_t>(k) * g.N]) : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < kLoadB; ++j) {
        if constexpr (FORM == EX_FWD) {
          rb[j] = nb + j * (kThreads / kDeep) < ncols && k0 + kb < depth
                      ? as_f32(pb[j * step_b + k0]) : 0.0f;
        } else {
          const int k = k0 + kb + j * (kThreads / kCols);
          const bool ok = nb < ncols && k < depth;
          if (FORM == EX_DGRAD) {
            rb[j] = ok ? as_f32(pb[static_cast<size_t>(k0) * g.D + j * step_b]) : 0.0f;
          } else {
            const int r = ok ? source_row(g.p2u, g.T, lo + k) : -1;
            rb[j] = r >= 0 ? as_f32(pb[static_cast<size_t>(r) * g.D]) : 0.0f;
          }
        }
      }
    };
    auto stage = [&](int buf) {
#pragma unroll
      for (int j = 0; j < kLoadA; ++j) {
        if constexpr (kDeepA) sa[buf][ka][ma + j * (kThreads / kDeep)] = ra[j];
        else sa[buf][ka + j * (kThreads / ROWS)][ma] = ra[j];
      }
#pragma unroll
      for (int j = 0; j < kLoadB; ++j) {
        if constexpr (kDeepB) sb[buf][kb][nb + j * (kThreads / kDeep)] = rb[j];
        else sb[buf][kb + j * (kThreads / kCols)][nb] = rb[j];
      }
    };

    float acc[kOwn][4] = {};
    if (depth > 0) {
      fetch(0);
      __syncthreads();  // the previous tile's last slice has been read
      stage(0);
    }
    int buf = 0;
    for (int k0 = 0; k0 < depth; k0 += kDeep) {
      __syncthreads();  // this slice is staged, and the other buffer has been read
      const bool more = k0 + kDeep < depth;
      if (more) fetch(k0 + kDeep);
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        float av[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; i += 4)
          *reinterpret_cast<float4*>(&av[i]) =
              *reinterpret_cast<const float4*>(&sa[buf][k][ty * kOwn + i]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[buf][k][tx * 4]);
        const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      buf ^= 1;
      if (more) stage(buf);
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int m = ty * kOwn + i;
      if (m >= rows) continue;
      const size_t base = (FORM == EX_WGRAD ? static_cast<size_t>(e) * g.N + row0 + m
                                            : static_cast<size_t>(row0 + m)) * cols + col0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tx * 4 + j < ncols) store_out(g.out, g.out_dtype, base + tx * 4 + j, acc[i][j]);
    }
  }
}

template <typename TIn, int FORM, int ROWS>
int launch_rows(const ExpertArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MR_ERR_CUDA;
  const long long cols = ((FORM == EX_FWD ? a.N : a.D) + kCols - 1) / kCols;
  const long long rows = FORM == EX_WGRAD
                             ? static_cast<long long>(a.E) * ((a.N + ROWS - 1) / ROWS)
                             : static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / ROWS;
  const long long most = 8ll * sms;
  const int grid = static_cast<int>(rows * cols < most ? rows * cols : most);
  const cudaError_t e = launch_kernel(expert_matmul_vector_kernel<TIn, FORM, ROWS>, dim3(grid),
                                      dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

// Tiles of 32 rows where the experts have few: half as many rows are padding.
template <typename TIn, int FORM>
int launch_typed(const ExpertArgs& a, cudaStream_t st) {
  if (FORM != EX_WGRAD && a.P <= 48ll * a.E) return launch_rows<TIn, FORM, 32>(a, st);
  return launch_rows<TIn, FORM, 64>(a, st);
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
