// Products grouped by expert on 4-bit weights, for decoding:
//
//   out[p, n] = sum_g s[e, n, g] sum_{d in g} (q[e, n, d] - z[e, n, g]) x[row(p), d]
//
// An expert has few rows then, so the weights are the traffic: N (D / 2 + the
// groups' scales) bytes per expert, read once for up to 8 of its rows.  A
// block of 4 warps takes 16 weight rows; each warp a quarter of D, and the
// four partial sums are added in shared memory in a fixed order.
//
// Arithmetic.  A nibble q becomes the bf16 128 + q by placing it in the low
// mantissa bits of 128 (one and/or for two nibbles), and a bf16 subtraction
// of 128 + z leaves q - z, both exact.  mma.sync m16n8k16 multiplies them with
// the bf16 activations, exactly, and adds in fp32; each group's sum is then
// scaled in fp32.  No weight is rounded on the way.
//
// Layout.  A 32-bit word holds the nibbles of d .. d + 7; masking it after a
// shift by 4 i leaves nibbles i and i + 4 in the two halves, so the pairs
// that meet in a fragment are (i, i + 4).  Which columns of x meet which
// nibbles is free as long as both fragments agree: thread t of a quad takes
// the words t * V .. t * V + V - 1 of each 4 V-word step (V = group / 32, so a
// step is one group and its loads are 4 V bytes wide) and the 8 activations
// under each word.
#include "router_common.cuh"
#include "router_experts.cuh"

namespace moe_router {
namespace {

constexpr int kRows = 16;    // weight rows per block
constexpr int kTokens = 8;   // permuted rows per pass over the weights
constexpr int kWarps = 4;    // quarters of the contraction

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// nibbles i and i + 4 of w as the bf16 pair (q - z, q - z); zp = 128 + z twice
__device__ __forceinline__ uint32_t nibbles(uint32_t w, int i, __nv_bfloat162 zp) {
  const uint32_t q = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q), zp);
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {
  const uint32_t v = (0x4300u | z) * 0x00010001u;
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}

// V consecutive words
template <int V>
struct Words {
  uint32_t w[V];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (V == 4) {
      const uint4 t = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else if constexpr (V == 2) {
      const uint2 t = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = t.x; w[1] = t.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const unsigned int*>(p));
    }
  }
};

template <int V, bool ZEROS>
__global__ __launch_bounds__(32 * kWarps) void expert_matmul_w4_kernel(W4Args g) {
  constexpr int kGroup = 32 * V;
  __shared__ int prefix[MR_MAX_EXPERTS + 1];
  __shared__ int tmp[33];
  __shared__ float part[kWarps][kTokens][kRows + 1];

  pdl_enter();
  const int row_tiles = (g.N + kRows - 1) / kRows;
  const long long tiles =
      static_cast<long long>(expert_tile_prefix(g.offsets, g.E, g.P, kTokens, prefix, tmp)) *
      row_tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;  // fragment row (and token), place in the quad
  const int groups = g.D / kGroup;
  const int per = (groups + kWarps - 1) / kWarps;
  const int g0 = warp * per, g1 = min(g0 + per, groups);
  const unsigned short* __restrict__ x = static_cast<const unsigned short*>(g.x);
  const unsigned short* __restrict__ scales = static_cast<const unsigned short*>(g.scales);

  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int q = static_cast<int>(tile / row_tiles);
    const int n0 = static_cast<int>(tile - static_cast<long long>(q) * row_tiles) * kRows;
    const int e = expert_of_tile(prefix, g.E, q);
    int lo, hi;
    expert_rows(g.offsets, e, g.P, &lo, &hi);
    const int p0 = lo + (q - prefix[e]) * kTokens;
    const int cnt = min(kTokens, hi - p0);
    // tokens and weight rows past the end repeat the last one; their results
    // are not stored
    const int src = max(source_row(g.p2u, g.T, p0 + min(gq, cnt - 1)), 0);
    const unsigned short* xr = x + static_cast<size_t>(src) * g.D;
    const size_t ra = static_cast<size_t>(e) * g.N + min(n0 + gq, g.N - 1);
    const size_t rb = static_cast<size_t>(e) * g.N + min(n0 + gq + 8, g.N - 1);
    const uint8_t* qa = g.q + ra * (g.D / 2);
    const uint8_t* qb = g.q + rb * (g.D / 2);

    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int gi = g0; gi < g1; ++gi) {
      Words<V> wa, wb;
      const int byte = gi * (kGroup / 2) + t * (4 * V);
      wa.load(qa + byte);
      wb.load(qb + byte);
      const float sa = bf16_bits_to_f32(scales[ra * groups + gi]);
      const float sb = bf16_bits_to_f32(scales[rb * groups + gi]);
      const __nv_bfloat162 za = zero_pair(ZEROS ? (g.zeros[ra * groups + gi] & 15u) : 8u);
      const __nv_bfloat162 zb = zero_pair(ZEROS ? (g.zeros[rb * groups + gi] & 15u) : 8u);
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint4 xv =
            *reinterpret_cast<const uint4*>(xr + gi * kGroup + t * (8 * V) + v * 8);
        // (x[0], x[4]), (x[1], x[5]), (x[2], x[6]), (x[3], x[7])
        const uint32_t b0 = __byte_perm(xv.x, xv.z, 0x5410), b1 = __byte_perm(xv.x, xv.z, 0x7632);
        const uint32_t b2 = __byte_perm(xv.y, xv.w, 0x5410), b3 = __byte_perm(xv.y, xv.w, 0x7632);
        mma_16816(c, nibbles(wa.w[v], 0, za), nibbles(wb.w[v], 0, zb), nibbles(wa.w[v], 1, za),
                  nibbles(wb.w[v], 1, zb), b0, b1);
        mma_16816(c, nibbles(wa.w[v], 2, za), nibbles(wb.w[v], 2, zb), nibbles(wa.w[v], 3, za),
                  nibbles(wb.w[v], 3, zb), b2, b3);
      }
      acc[0] = fmaf(sa, c[0], acc[0]);
      acc[1] = fmaf(sa, c[1], acc[1]);
      acc[2] = fmaf(sb, c[2], acc[2]);
      acc[3] = fmaf(sb, c[3], acc[3]);
    }
    // fragment: rows gq and gq + 8, tokens 2 t and 2 t + 1
    part[warp][2 * t][gq] = acc[0];
    part[warp][2 * t + 1][gq] = acc[1];
    part[warp][2 * t][gq + 8] = acc[2];
    part[warp][2 * t + 1][gq + 8] = acc[3];
    __syncthreads();
    const int token = threadIdx.x / kRows, n = threadIdx.x % kRows;
    if (token < cnt && n0 + n < g.N) {
      float s = part[0][token][n];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += part[w][token][n];
      const size_t o = static_cast<size_t>(p0 + token) * g.N + n0 + n;
      if (g.out_dtype == DT_F32) static_cast<float*>(g.out)[o] = s;
      else static_cast<unsigned short*>(g.out)[o] = static_cast<unsigned short>(f32_to_bf16_bits(s));
    }
    __syncthreads();
  }
}

template <int V>
int launch_group(const W4Args& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MR_ERR_CUDA;
  const long long tasks = (static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / kTokens) *
                          ((a.N + kRows - 1) / kRows);
  const long long most = 8ll * sms;
  const dim3 grid(static_cast<unsigned>(tasks < most ? tasks : most));
  const cudaError_t e =
      a.zeros != nullptr
          ? launch_kernel(expert_matmul_w4_kernel<V, true>, grid, dim3(32 * kWarps), 0, st, a)
          : launch_kernel(expert_matmul_w4_kernel<V, false>, grid, dim3(32 * kWarps), 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

}  // namespace

int launch_expert_matmul_w4(const W4Args& a, cudaStream_t st) {
  return a.group == 32   ? launch_group<1>(a, st)
         : a.group == 64 ? launch_group<2>(a, st)
                         : launch_group<4>(a, st);
}

}  // namespace moe_router
