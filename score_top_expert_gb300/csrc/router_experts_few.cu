// Products grouped by expert for few rows per expert (decoding), on bf16 or
// 4-bit weights:
//
//   out[p, n] = sum_d w[e, n, d] x[row(p), d]
//   4-bit: w[e, n, d] = s[e, n, g] (q[e, n, d] - z[e, n, g]),  d in group g
//
// The weights of the experts that have rows are the traffic and are read once
// for up to 8 of an expert's rows.  A warp takes 16 weight rows at a time
// through a ring of shared-memory stages of its own, 256 bytes of each row a
// stage, filled by asynchronous copies three stages ahead, across tasks: no
// warp waits for another, and 12 warps an SM keep about 147 KB in flight.  With
// fewer tasks than warps the four warps of a block take a quarter of the
// contraction each and add up in shared memory in a fixed order.
//
// mma.sync m16n8k16 (16 weight rows, 8 permuted rows, fp32 sums) suits the
// shape: a tcgen05 product would be 128 weight rows wide and needs the operand
// pipeline that costs the latency here; neither is near its peak rate.  Which
// columns of x meet which of w is free as long as both fragments agree, so a
// thread takes 16 consecutive bytes of a row.
//
// 4-bit arithmetic.  A nibble q becomes the bf16 128 + q by placing it in the
// low mantissa bits of 128 (one and/or for two nibbles), and a bf16
// subtraction of 128 + z leaves q - z, both exact.  The products with the bf16
// activations are exact, each group's fp32 sum is scaled in fp32: no weight is
// rounded on the way.  A 32-bit word holds the nibbles of d .. d + 7; masking it
// after a shift by 4 i leaves nibbles i and i + 4 in the two halves, so the
// pairs that meet in a fragment are (i, i + 4).  Thread t of a quad takes the
// words t V .. t V + V - 1 of each group (V = group / 32), so that a product's 16
// columns lie in one group.
#include <atomic>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_launch.cuh"

namespace moe_router {
namespace {

constexpr int kRows = 16;         // weight rows per task
constexpr int kTokens = 8;        // permuted rows per task
constexpr int kWarps = 4;         // per block
constexpr int kChunk = 256;       // bytes of a weight row per stage
constexpr int kStages = 4;
constexpr int kBlocksPerSm = 3;

// V: 32-bit words a thread takes of each step; 0: bf16 weights.
template <int V>
struct Layout {
  static constexpr int kPerChunk = V == 0 ? kChunk / 2 : kChunk * 2;  // columns per stage
  static constexpr int kStep = V == 0 ? 32 : 32 * V;                  // columns per step
  static constexpr int kSteps = kPerChunk / kStep;
  // Row r's 16-byte piece p lies at piece p ^ swizzle(r) of its 256 bytes, so
  // that the rows one load reads at the same column fall into different banks.
  static constexpr int kSwizzle = V == 1 ? 1 : V == 2 ? 2 : 4;
  static __device__ __forceinline__ int swizzle(int row) { return (row * kSwizzle) & 7; }
};

constexpr int kStageBytes = kRows * kChunk;

// Dynamic shared memory: the rings, then the experts' prefix.
constexpr int few_smem(int E) { return kWarps * kStages * kStageBytes + (E + 1) * 4; }

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

// The bf16 pair 128 + z, z in bits 16-19 of m.
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t m) {
  const uint32_t v = __byte_perm(m | 0x43000000u, 0u, 0x3232);
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}

__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int V>
__device__ __forceinline__ void load_words(uint32_t at, uint32_t (&w)[V == 0 ? 4 : V]) {
  if constexpr (V == 0 || V == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
  else if constexpr (V == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
}

struct FewArgs {
  const void* x;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  const int32_t* offsets;
  const int32_t* p2u;
  void* out;
  int T, P, E, N, D, out_dtype;
};

// A task: up to 8 permuted rows of an expert and 16 of its weight rows.
struct Task {
  int e, p0, cnt, n0;
};

__device__ __forceinline__ Task task_of(const FewArgs& g, const int* prefix, long long i,
                                        int row_tiles) {
  // an expert's 8-row groups follow one another for the same weight rows
  Task t;
  t.e = expert_of_tile(prefix, g.E, static_cast<int>(i / row_tiles));
  const int first = prefix[t.e], groups = prefix[t.e + 1] - first;
  const int r = static_cast<int>(i - static_cast<long long>(first) * row_tiles);
  t.n0 = r / groups * kRows;
  int lo, hi;
  expert_rows(g.offsets, t.e, g.P, &lo, &hi);
  t.p0 = lo + (r % groups) * kTokens;
  t.cnt = min(kTokens, hi - t.p0);
  return t;
}

template <int V, bool ZEROS, bool SPLIT>
__global__ __launch_bounds__(32 * kWarps, kBlocksPerSm) void expert_matmul_few_kernel(FewArgs g) {
  using L = Layout<V>;
  extern __shared__ __align__(16) uint8_t ring[];
  int* prefix = reinterpret_cast<int*>(ring + kWarps * kStages * kStageBytes);
  __shared__ int tmp[33];
  __shared__ float part[SPLIT ? kWarps : 1][kTokens][kRows + 1];

  pdl_enter();
  const int row_tiles = (g.N + kRows - 1) / kRows;
  const long long tasks =
      static_cast<long long>(expert_tile_prefix(g.offsets, g.E, g.P, kTokens, prefix, tmp)) *
      row_tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;  // fragment row (and token), place in the quad
  const long long row_bytes = V == 0 ? 2ll * g.D : g.D / 2;
  const int groups = V == 0 ? 0 : g.D / L::kStep;
  const int chunks = (g.D + L::kPerChunk - 1) / L::kPerChunk;
  // this warp's chunks of each task
  const int per = (chunks + kWarps - 1) / kWarps;
  const int c0 = SPLIT ? min(warp * per, chunks) : 0;
  const int c1 = SPLIT ? min(c0 + per, chunks) : chunks;
  const long long first = SPLIT ? blockIdx.x : static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long step = SPLIT ? gridDim.x : static_cast<long long>(gridDim.x) * kWarps;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                           warp * kStages * kStageBytes;

  // ---- copies: a cursor kStages - 1 stages ahead of the products -----------------
  long long li = first;  // task and chunk the next copy belongs to
  int lc = c0, lstage = 0;
  const uint8_t* lsrc = nullptr;  // this lane's piece of the first row it copies
  int lrows = 0;                  // weight rows of the task that exist
  const int piece = (lane & 15) * 16, half = lane >> 4;  // 16 lanes copy a row, two rows at a time
  auto begin_copies = [&]() {
    if (li < tasks) {
      const Task k = task_of(g, prefix, li, row_tiles);
      lsrc = g.w + (static_cast<long long>(k.e) * g.N + k.n0 + half) * row_bytes + piece;
      lrows = g.N - k.n0;
    }
  };
  auto copy_stage = [&]() {
    if (li < tasks && c0 < c1) {
      const long long col = static_cast<long long>(lc) * kChunk;
      const bool inside = col + piece < row_bytes;
      const uint32_t dst = ring_at + lstage * kStageBytes;
#pragma unroll
      for (int j = 0; j < kRows / 2; ++j) {
        // rows past the last and columns past the row are filled with zeros
        const int row = 2 * j + half;
        const bool ok = inside && row < lrows;
        copy_16(dst + row * kChunk + (((lane & 15) ^ L::swizzle(row)) << 4), ok ? lsrc + 2 * j * row_bytes + col : g.w, ok);
      }
      if (++lc == c1) {
        lc = c0;
        li += step;
        begin_copies();
      }
    }
    if (++lstage == kStages) lstage = 0;
    copies_commit();
  };
  begin_copies();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_stage();

  const unsigned short* __restrict__ x = static_cast<const unsigned short*>(g.x);
  const unsigned short* __restrict__ scales = static_cast<const unsigned short*>(g.scales);
  int stage = 0;
  for (long long i = first; i < tasks; i += step) {
    const Task k = task_of(g, prefix, i, row_tiles);
    // tokens past the last repeat it; their results are not stored
    const int src = max(source_row(g.p2u, g.T, k.p0 + min(gq, k.cnt - 1)), 0);
    const unsigned short* xr = x + static_cast<size_t>(src) * g.D;
    const size_t ra = (static_cast<size_t>(k.e) * g.N + min(k.n0 + gq, g.N - 1)) * groups;
    const size_t rb = (static_cast<size_t>(k.e) * g.N + min(k.n0 + gq + 8, g.N - 1)) * groups;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = c0; c < c1; ++c) {
      copy_stage();
      // Scales (low half) and zero points of this chunk: the quad's lanes hold
      // every fourth group of both rows and hand them round.
      constexpr int kHeld = V == 0 ? 1 : (L::kSteps + 3) / 4;
      uint32_t ma[kHeld], mb[kHeld];
      if constexpr (V > 0) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          const int gi = c * L::kSteps + 4 * j + t;
          ma[j] = mb[j] = 8u << 16;
          if (gi < groups) {
            const uint32_t za = ZEROS ? g.zeros[ra + gi] & 15u : 8u;
            const uint32_t zb = ZEROS ? g.zeros[rb + gi] & 15u : 8u;
            ma[j] = scales[ra + gi] | (za << 16);
            mb[j] = scales[rb + gi] | (zb << 16);
          }
        }
      }
      // This chunk's activations, all loads in flight before the wait for the
      // weights: left to the steps, each waited for its own (the statements
      // that read shared memory keep their order), 2.5 times the chunk's time.
      const int col = c * L::kPerChunk;
      constexpr int kLoads = L::kPerChunk / 32;
      uint4 xs[kLoads];
#pragma unroll
      for (int s = 0; s < L::kSteps; ++s)
#pragma unroll
        for (int v = 0; v < kLoads / L::kSteps; ++v) {
          const int d = col + s * L::kStep + (V == 0 ? t * 8 : t * (8 * V) + v * 8);
          uint4& q = xs[s * (kLoads / L::kSteps) + v];
          q = make_uint4(0u, 0u, 0u, 0u);
          if (d < g.D) q = *reinterpret_cast<const uint4*>(xr + d);
        }
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint32_t at = ring_at + stage * kStageBytes + gq * kChunk;
      const int sw = L::swizzle(gq);  // and of row gq + 8
#pragma unroll
      for (int s = 0; s < L::kSteps; ++s) {
        const int d = col + s * L::kStep;
        if (d >= g.D) break;
        if constexpr (V == 0) {
          uint32_t wa[4], wb[4];
          const uint32_t from = at + (((4 * s + t) ^ sw) << 4);
          load_words<V>(from, wa);
          load_words<V>(from + 8 * kChunk, wb);
          const uint4 xv = xs[s];
          mma_16816(acc, wa[0], wb[0], wa[1], wb[1], xv.x, xv.y);
          mma_16816(acc, wa[2], wb[2], wa[3], wb[3], xv.z, xv.w);
        } else {
          uint32_t wa[V], wb[V];
          const int byte = s * (16 * V) + t * (4 * V);
          const uint32_t from = at + (((byte >> 4) ^ sw) << 4) + (byte & 15);
          load_words<V>(from, wa);
          load_words<V>(from + 8 * kChunk, wb);
          const int holder = (lane & 28) | (s & 3);
          const uint32_t a = __shfl_sync(0xffffffffu, ma[s >> 2], holder);
          const uint32_t b = __shfl_sync(0xffffffffu, mb[s >> 2], holder);
          const __nv_bfloat162 za = zero_pair(a & 0xf0000u), zb = zero_pair(b & 0xf0000u);
          float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const uint4 xv = xs[s * V + v];
            // (x[0], x[4]), (x[1], x[5]), (x[2], x[6]), (x[3], x[7])
            const uint32_t b0 = __byte_perm(xv.x, xv.z, 0x5410);
            const uint32_t b1 = __byte_perm(xv.x, xv.z, 0x7632);
            const uint32_t b2 = __byte_perm(xv.y, xv.w, 0x5410);
            const uint32_t b3 = __byte_perm(xv.y, xv.w, 0x7632);
            mma_16816(p, nibbles(wa[v], 0, za), nibbles(wb[v], 0, zb), nibbles(wa[v], 1, za),
                      nibbles(wb[v], 1, zb), b0, b1);
            mma_16816(p, nibbles(wa[v], 2, za), nibbles(wb[v], 2, zb), nibbles(wa[v], 3, za),
                      nibbles(wb[v], 3, zb), b2, b3);
          }
          const float sa = __uint_as_float(a << 16), sb = __uint_as_float(b << 16);
          acc[0] = fmaf(sa, p[0], acc[0]);
          acc[1] = fmaf(sa, p[1], acc[1]);
          acc[2] = fmaf(sb, p[2], acc[2]);
          acc[3] = fmaf(sb, p[3], acc[3]);
        }
      }
      __syncwarp();  // all lanes have read the stage before it is filled again
      if (++stage == kStages) stage = 0;
    }
    // fragment: weight rows gq and gq + 8, tokens 2 t and 2 t + 1
    if constexpr (SPLIT) {
      part[warp][2 * t][gq] = acc[0];
      part[warp][2 * t + 1][gq] = acc[1];
      part[warp][2 * t][gq + 8] = acc[2];
      part[warp][2 * t + 1][gq + 8] = acc[3];
      __syncthreads();
      const int token = threadIdx.x / kRows, n = threadIdx.x % kRows;
      if (token < k.cnt && k.n0 + n < g.N) {
        float s = part[0][token][n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += part[w][token][n];
        const size_t o = static_cast<size_t>(k.p0 + token) * g.N + k.n0 + n;
        if (g.out_dtype == DT_F32) static_cast<float*>(g.out)[o] = s;
        else static_cast<unsigned short*>(g.out)[o] = static_cast<unsigned short>(f32_to_bf16_bits(s));
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int token = 2 * t + (j & 1), n = k.n0 + gq + (j >> 1) * 8;
        if (token < k.cnt && n < g.N) {
          const size_t o = static_cast<size_t>(k.p0 + token) * g.N + n;
          if (g.out_dtype == DT_F32) static_cast<float*>(g.out)[o] = acc[j];
          else static_cast<unsigned short*>(g.out)[o] =
              static_cast<unsigned short>(f32_to_bf16_bits(acc[j]));
        }
      }
    }
  }
}

template <int V, bool ZEROS, bool SPLIT>
int launch_split(const FewArgs& a, long long tasks, int sms, cudaStream_t st) {
  static std::atomic<int> granted[kSmemDevs];
  const auto kern = expert_matmul_few_kernel<V, ZEROS, SPLIT>;
  cudaError_t e = allow_smem(kern, few_smem(a.E), granted);
  if (e != cudaSuccess) return MR_ERR_CUDA;
  const long long blocks = SPLIT ? tasks : (tasks + kWarps - 1) / kWarps;
  const long long most = static_cast<long long>(kBlocksPerSm) * sms;
  e = launch_kernel(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                    dim3(32 * kWarps), few_smem(a.E), st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int V, bool ZEROS>
int launch_typed(const FewArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MR_ERR_CUDA;
  // tasks at most (the host does not know which experts have rows)
  const long long tasks = (static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / kTokens) *
                          ((a.N + kRows - 1) / kRows);
  const bool split = tasks <= 2ll * kBlocksPerSm * sms * kWarps;
  return split ? launch_split<V, ZEROS, true>(a, tasks, sms, st)
               : launch_split<V, ZEROS, false>(a, tasks, sms, st);
}

}  // namespace

bool expert_matmul_few_ok(const ExpertArgs& a) {
  const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  return a.dtype == DT_BF16 && a.D % 8 == 0 && aligned(a.a) && aligned(a.b);
}

int launch_expert_matmul_few(const ExpertArgs& a, cudaStream_t st) {
  const FewArgs g{a.a, static_cast<const uint8_t*>(a.b), nullptr, nullptr, a.offsets, a.p2u,
                  a.out, a.T, a.P, a.E, a.N, a.D, a.out_dtype};
  return launch_typed<0, false>(g, st);
}

int launch_expert_matmul_w4(const W4Args& a, cudaStream_t st) {
  const FewArgs g{a.x, a.q, a.scales, a.zeros, a.offsets, a.p2u, a.out, a.T, a.P, a.E, a.N, a.D,
                  a.out_dtype};
  if (a.group == 32) return a.zeros ? launch_typed<1, true>(g, st) : launch_typed<1, false>(g, st);
  if (a.group == 64) return a.zeros ? launch_typed<2, true>(g, st) : launch_typed<2, false>(g, st);
  return a.zeros ? launch_typed<4, true>(g, st) : launch_typed<4, false>(g, st);
}

}  // namespace moe_router
