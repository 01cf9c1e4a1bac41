// Rows in 8 bits, with a scale for each:
//
//   scale = max |x| / 127,   q = x / scale to the nearest integer, ties to even
//
// Bound by HBM: a row is read once, held in the registers of the 1 to 16 warps of its
// team (what goes beyond 16 warps' pieces is read again), and written once; a team's next
// row is asked for before the present one is done.  8192 x 2048 bf16: 12.5 us, 4.0 TB/s;
// 22066 x 504 9.1 us.
//
// The quotient is the exact one's rounding.  x (1 / scale) is off by 2^-23 of itself, 1.6e-5
// at 127, which matters only beside a half.
//   fp32: where it lies within 2e-5 of one, the remainder x - q scale decides, which one
//   multiply-add gives exactly: a multiple of the smaller operand's last bit and at most
//   scale / 2.
//   bf16: 127 x / max is k + 1/2 only for 254 x = (2 k + 1) max, so (127 is a prime) for
//   k = 63, |x| = max / 2, which is frequent, or for a max of 127 2^i, whose scale is a
//   power of two and all quotients exact; else it is 2^-16 of itself away at least, as
//   numbers of eight bits are.  So a row needs one decision, and 1 / scale is moved
//   by the few last places that it takes for |x| = max / 2 to come out right.
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_rows.cuh"

namespace moe_router {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kBlockWarps = 8;
constexpr int kFewRows = 608;  // four blocks an SM
constexpr float kMagic = 12582912.0f;     // 1.5 2^23: adding it rounds to an integer
constexpr float kSmallest = 1.17549435e-38f;  // 2^-126

// kMagic + q put right where the quotient is next to a half.
__device__ __forceinline__ float decided(float x, float scale, float r) {
  float q = r - kMagic;
  const float d = fmaf(-q, scale, x);
  const float twice = 2.0f * fabsf(d);
  const bool odd = (__float_as_int(r) & 1) != 0;
  if (twice > scale || (twice == scale && odd)) q += copysignf(1.0f, d);
  return q + kMagic;
}

// bf16 rows: 1 / scale, such that max / 2 is rounded as its quotient is.  (Two or three steps
// at most: both are within 2^-22 of the exact one.)
__device__ __forceinline__ float decided_inverse(float top, float scale, float inv) {
  const float half = 0.5f * top;
  const float want = decided(half, scale, fmaf(half, inv, kMagic));
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float r = fmaf(half, inv, kMagic);
    if (r == want) break;
    inv = __uint_as_float(__float_as_uint(inv) + (r < want ? 1u : 0xffffffffu));
  }
  return inv;
}

template <int DT, int N>
__device__ __forceinline__ void quantize(const float (&x)[N], float scale, float inv,
                                         uint32_t (&bytes)[N / 4]) {
  float r[N], far = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    r[j] = fmaf(x[j], inv, kMagic);
    if constexpr (DT == DT_F32) far = fmaxf(far, fabsf(fmaf(x[j], inv, kMagic - r[j])));
  }
  if (DT == DT_F32 && far > 0.49998f) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (fabsf(fmaf(x[j], inv, kMagic - r[j])) > 0.49998f) r[j] = decided(x[j], scale, r[j]);
  }
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const uint32_t lo = __byte_perm(__float_as_uint(r[4 * j]), __float_as_uint(r[4 * j + 1]), 0x0040);
    const uint32_t hi =
        __byte_perm(__float_as_uint(r[4 * j + 2]), __float_as_uint(r[4 * j + 3]), 0x0040);
    bytes[j] = __byte_perm(lo, hi, 0x5410);
  }
}

template <typename P, int BYTES>
__device__ __forceinline__ void store_bytes(int8_t* row, int col0, int lane, int D,
                                            const uint32_t (&b)[P::kN / 4]) {
  if constexpr (BYTES == 16) {
    const int c = P::column(col0, 0, lane);
    if (c >= D) return;
    if constexpr (P::kN == 8) __stcs(reinterpret_cast<uint2*>(row + c), make_uint2(b[0], b[1]));
    else __stcs(reinterpret_cast<unsigned int*>(row + c), b[0]);
  } else {
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int c = P::column(col0, j / P::kEach, lane) + j % P::kEach;
      if (c < D) row[c] = static_cast<int8_t>(b[j >> 2] >> (8 * (j & 3)));
    }
  }
}

struct QuantizeArgs {
  const void* x;
  int8_t* q;
  float* scales;
  int R, D, warps;
};

template <int DT, int BYTES, int U>
__global__ __launch_bounds__(32 * kMaxWarps) void quantize_kernel(const QuantizeArgs a) {
  using P = Piece<DT, BYTES>;
  __shared__ unsigned cells[2][kMaxWarps];
  pdl_enter();
  const int lane = threadIdx.x & 31, block_warp = threadIdx.x >> 5;
  const int team = block_warp / a.warps, warp = block_warp - team * a.warps;
  const int teams = (blockDim.x >> 5) / a.warps;
  const long long step = static_cast<long long>(gridDim.x) * teams;
  const int stride = a.warps * 32 * P::kN;
  const int col0 = warp * 32 * P::kN;
  P held[U], next[U];
  auto load = [&](P(&p)[U], long long row) {
#pragma unroll
    for (int q = 0; q < U; ++q)
      p[q].template load<true>(a.x, static_cast<size_t>(row) * a.D, col0 + q * stride, lane, a.D);
  };
  long long row = static_cast<long long>(blockIdx.x) * teams + team;
  if (row < a.R) load(next, row);
  for (int flip = 0; row < a.R; row += step, flip ^= 1) {
    const size_t at = static_cast<size_t>(row) * a.D;
#pragma unroll
    for (int q = 0; q < U; ++q) held[q] = next[q];
    if (row + step < a.R) load(next, row + step);
    unsigned top = 0;  // |x| as bits: a NaN is above an infinity, which is above all else
    auto largest = [&](const P& p, int col) {
      if (P::column(col, 0, lane) >= a.D) return;
      float v[P::kN];
      p.widen(v);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    };
#pragma unroll
    for (int q = 0; q < U; ++q) largest(held[q], col0 + q * stride);
    for (int col = col0 + U * stride; col < a.D; col += stride) {
      P p;
      p.template load<false>(a.x, at, col, lane, a.D);
      largest(p, col);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (a.warps > 1) {  // two sets of cells in turn: one barrier a row
      if (lane == 0) cells[flip][block_warp] = top;
      if (teams == 1) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(a.warps * 32) : "memory");
      for (int w = 0; w < a.warps; ++w) top = max(top, cells[flip][team * a.warps + w]);
    }
    float scale = __fdiv_rn(__uint_as_float(top), 127.0f);
    if (top != 0 && scale < kSmallest) scale = kSmallest;  // (whose inverse is a number)
    float inv = __fdiv_rn(1.0f, scale);
    // without a finite scale above zero all integers are zero
    const bool number = top - 1u < 0x7f7fffffu;
    if (DT == DT_BF16 && number) inv = decided_inverse(__uint_as_float(top), scale, inv);
    int8_t* const out = a.q + at;
    auto finish = [&](const P& p, int col) {
      if (P::column(col, 0, lane) >= a.D) return;
      float v[P::kN];
      p.widen(v);
      uint32_t b[P::kN / 4];
      if (number) {
        quantize<DT, P::kN>(v, scale, inv, b);
      } else {
#pragma unroll
        for (int j = 0; j < P::kN / 4; ++j) b[j] = 0u;
      }
      store_bytes<P, BYTES>(out, col, lane, a.D, b);
    };
#pragma unroll
    for (int q = 0; q < U; ++q) finish(held[q], col0 + q * stride);
    for (int col = col0 + U * stride; col < a.D; col += stride) {
      P p;
      p.template load<false>(a.x, at, col, lane, a.D);
      finish(p, col);
    }
    if (warp == 0 && lane == 0) a.scales[row] = scale;
  }
}

template <int DT, int BYTES, int U>
int launch_pieces(QuantizeArgs a, int stretches, cudaStream_t st) {
  const int needed = (stretches + U - 1) / U;
  a.warps = needed < kMaxWarps ? needed : kMaxWarps;
  const int teams = a.warps >= kBlockWarps ? 1 : kBlockWarps / a.warps;
  const int threads = 32 * a.warps * teams;
  const long long most = (static_cast<long long>(a.R) + teams - 1) / teams;
  // what is resident, by registers
  const long long resident = 152ll * (65536 / (threads * (U == 1 ? 64 : U == 2 ? 80 : 128)));
  const cudaError_t e =
      launch_kernel(quantize_kernel<DT, BYTES, U>,
                    dim3(static_cast<unsigned>(most < resident ? most : resident)), dim3(threads),
                    0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

// Few rows: a piece to a lane, up to 16 warps to a row, for the latency (one row of 2048 bf16
// 2.4 us against 3.8 with eight pieces to a lane of one warp).  Many: more pieces to
// a lane, so fewer barriers and divisions (8192 rows: one piece 27 us).
template <int DT, int BYTES>
int launch_typed(const QuantizeArgs& a, cudaStream_t st) {
  constexpr int columns = 32 * Piece<DT, BYTES>::kN;
  const int stretches = (a.D + columns - 1) / columns;
  if (stretches == 1 || a.R <= kFewRows) return launch_pieces<DT, BYTES, 1>(a, stretches, st);
  return stretches <= 3 ? launch_pieces<DT, BYTES, 2>(a, stretches, st)
                        : launch_pieces<DT, BYTES, 4>(a, stretches, st);
}

}  // namespace
}  // namespace moe_router

using namespace moe_router;

extern "C" int router_quantize_rows(const void* x, mr_dtype dtype, int R, int D, int8_t* q,
                                    float* scales, mr_stream_t stream) {
  if ((dtype != MR_F32 && dtype != MR_BF16) || R < 0 || D < 1) return MR_ERR_INVALID;
  if (D > MR_MAX_FEATURES) return MR_ERR_UNSUPPORTED;
  if (R == 0) return MR_OK;
  if (x == nullptr || q == nullptr || scales == nullptr) return MR_ERR_INVALID;
  const QuantizeArgs a{x, q, scales, R, D, 0};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // wide accesses: rows of x in whole aligned 16 bytes, those of q as many values' bytes
  const uintptr_t wide = reinterpret_cast<uintptr_t>(x) |
                         static_cast<uintptr_t>(D) * (dtype == MR_F32 ? 4 : 2);
  const bool aligned = (wide & 15u) == 0 &&
                       (reinterpret_cast<uintptr_t>(q) & (dtype == MR_F32 ? 3u : 7u)) == 0;
  if (dtype == MR_F32)
    return aligned ? launch_typed<DT_F32, 16>(a, st) : launch_typed<DT_F32, 4>(a, st);
  return aligned           ? launch_typed<DT_BF16, 16>(a, st)
         : (wide & 3u) == 0 ? launch_typed<DT_BF16, 4>(a, st)
                            : launch_typed<DT_BF16, 2>(a, st);
}
