// Products grouped by expert for few rows per expert (decoding), on bf16 or
// 4-bit weights:
//
//   out[p, n] = sum_d w[e, n, d] x[row(p), d]
//   4-bit: w[e, n, d] = s[e, n, g] (q[e, n, d] - z[e, n, g]),  d in group g
//
// The weights of the experts that have rows are the traffic and are read once
// for up to 8 of an expert's rows.  A block's task is such a group of rows and a
// span of the expert's weight rows: the rows of x are staged in shared memory in
// the order the fragments want, then each of the 16 warps takes 16 weight rows
// through two shared-memory stages of its own, 256 bytes of each row a stage,
// filled by asynchronous copies a stage ahead, across tasks: 64 KB in flight on
// an SM while the block changes its x.  With few tasks four warps share 16 weight
// rows, a quarter of the contraction each, and add up in shared memory in a fixed
// order.
//
// What bounds it (4 bits): latency at four warps a scheduler.  33 tokens, 512
// experts, 22 choices, 1024 x 1024 in groups of 128: 98 us with 8 warps, 78 with 12,
// 64 with 16 (2.5 TB/s of weights), a third of HBM and 55 % of the issue slots; a
// warp waits 7.3 cycles from one instruction to the next, for the one before it, the
// arithmetic pipe and its turn most, at the barriers around x and for memory a
// quarter.  Eight weights of a lane take about 30 instructions, 11 of them to unpack
// the nibbles.  Groups of 32 with zero points at 1056 x 1000: 103 us, with three
// times the waits for global memory (scales).
//
// The tensor cores add the products of 16 columns to their accumulator by
// truncation (see router_experts_tc.cu), so a sum starts from zero for each chunk
// of 128 columns of bf16 weights, or each group of 4-bit weights, and is added to
// the tile's in round-to-nearest: one sum over the whole row was off by 2.1e-6 of
// its value at 8192 columns and 1.9e-5 at 65536.
//
// mma.sync m16n8k16 (16 weight rows, 8 permuted rows, fp32 sums) suits the
// shape: a tcgen05 product would be 128 weight rows wide and needs the operand
// pipeline that costs the latency here; neither is near its peak rate.  Which
// columns of x meet which of w is free as long as both fragments agree, so a
// thread takes 16 consecutive bytes of a weight row.
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
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_launch.cuh"

namespace moe_router {
namespace {

constexpr int kRows = 16;         // weight rows per tile
constexpr int kTokens = 8;        // permuted rows per task
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kShare = 4;         // warps that share a tile when there are few
constexpr int kChunk = 256;       // bytes of a weight row per stage
constexpr int kStages = 2;
constexpr int kStageBytes = kRows * kChunk;
constexpr int kPanel = 4096;      // columns of x staged at a time

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

// Bytes between staged rows of x: eight 16-byte reads of two neighbouring rows
// fall into different banks.
__host__ __device__ constexpr int x_pitch(int D) {
  return ((D < kPanel ? D : kPanel) * 2 + 127) / 128 * 128 + 64;
}

// Dynamic shared memory: the rings, x, the experts' prefix.
constexpr int few_smem(int E, int D) {
  return kWarps * kStages * kStageBytes + kTokens * x_pitch(D) + (E + 1) * 4;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with sums that start at zero.
__device__ __forceinline__ void mma_16816_from_zero(float (&c)[4], uint32_t a0, uint32_t a1,
                                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// V consecutive words of shared memory.
template <int V>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[V]) {
  if constexpr (V == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (V == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
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

__device__ __forceinline__ void store_value(const FewArgs& g, size_t i, float v) {
  if (g.out_dtype == DT_F32) static_cast<float*>(g.out)[i] = v;
  else static_cast<unsigned short*>(g.out)[i] = static_cast<unsigned short>(f32_to_bf16_bits(v));
}

// The four warps of a team.
__device__ __forceinline__ void team_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * kShare) : "memory");
}

// A task: up to 8 permuted rows of an expert and a span of its weight tiles.
struct Task {
  int e, p0, cnt;
  int first, last;  // weight tiles
};

__device__ __forceinline__ Task task_of(const FewArgs& g, const int* prefix, int i, int spans,
                                        int span, int row_tiles) {
  // an expert's 8-row groups follow one another for the same weights
  Task t;
  t.e = expert_of_tile(prefix, g.E, i / spans);
  const int first = prefix[t.e], groups = prefix[t.e + 1] - first;
  const int r = i - first * spans;
  const int s = groups == 1 ? r : r / groups;
  t.first = s * span;
  t.last = min(t.first + span, row_tiles);
  int lo, hi;
  expert_rows(g.offsets, t.e, g.P, &lo, &hi);
  t.p0 = lo + (r - s * groups) * kTokens;
  t.cnt = min(kTokens, hi - t.p0);
  return t;
}

// Scales (low half) and zero points of one chunk of 16 weight rows: the quad's
// lanes hold every fourth group of both of its rows and hand them round.
template <int V>
struct Meta {
  static constexpr int kHeld = V == 0 ? 1 : (Layout<V>::kSteps + 3) / 4;
  uint32_t a[kHeld], b[kHeld];

  // ra, rb: the rows' first group
  template <bool ZEROS>
  __device__ __forceinline__ void load(const FewArgs& g, size_t ra, size_t rb, int c, int groups,
                                       int t) {
    if constexpr (V > 0) {
      const unsigned short* scales = static_cast<const unsigned short*>(g.scales);
      const int g0 = c * Layout<V>::kSteps + t;
      const unsigned short *sa = scales + ra + g0, *sb = scales + rb + g0;
      const uint8_t *za = g.zeros + ra + g0, *zb = g.zeros + rb + g0;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        a[j] = b[j] = 0u;
        if (g0 + 4 * j < groups) {
          a[j] = sa[4 * j];
          b[j] = sb[4 * j];
          if (ZEROS) {
            a[j] |= (za[4 * j] & 15u) << 16;
            b[j] |= (zb[4 * j] & 15u) << 16;
          }
        }
      }
    }
  }
};

template <int V, bool ZEROS, bool SHARED>
__global__ __launch_bounds__(kThreads, 1) void expert_matmul_few_kernel(FewArgs g) {
  using L = Layout<V>;
  constexpr int kTeams = SHARED ? kWarps / kShare : kWarps;  // of warps with a tile of their own
  constexpr int span = kTeams;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* xs = smem + kWarps * kStages * kStageBytes;
  const int pitch = x_pitch(g.D);
  int* prefix = reinterpret_cast<int*>(xs + kTokens * pitch);
  __shared__ int tmp[33];
  __shared__ float part[SHARED ? kWarps : 1][kTokens][kRows + 1];

  pdl_enter();
  const int row_tiles = (g.N + kRows - 1) / kRows;
  const int spans = (row_tiles + span - 1) / span;
  const int tasks = expert_tile_prefix(g.offsets, g.E, g.P, kTokens, prefix, tmp) * spans;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int team = SHARED ? warp / kShare : warp, member = SHARED ? warp % kShare : 0;
  const int gq = lane >> 2, t = lane & 3;  // fragment row (and token), place in the quad
  const int row_bytes = V == 0 ? 2 * g.D : g.D / 2;
  const int groups = V == 0 ? 0 : g.D / L::kStep;
  const int chunks = (g.D + L::kPerChunk - 1) / L::kPerChunk;
  // this warp's chunks of each tile
  const int per = SHARED ? (chunks + kShare - 1) / kShare : chunks;
  const int c0 = min(member * per, chunks), c1 = min(c0 + per, chunks);
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                           warp * kStages * kStageBytes;

  // ---- copies: a cursor kStages - 1 stages ahead of the products -----------------
  int li = blockIdx.x, ltile = 0, llast = 0, le = 0, lc = c0, lstage = 0;
  const int half = lane >> 4;  // 16 lanes copy a row, two rows at a time
  const int piece = (lane & 15) * 16;
  const uint8_t* lsrc = nullptr;  // this lane's piece of the first row it copies, at chunk c0
  auto next_tile = [&](bool fresh) {  // the cursor's tile: in its task, or the first of a later one
    if (!fresh) ltile += kTeams;
    while (li < tasks && (fresh || ltile >= llast)) {
      if (!fresh) li += gridDim.x;
      fresh = false;
      if (li >= tasks) break;
      const Task k = task_of(g, prefix, li, spans, span, row_tiles);
      le = k.e;
      ltile = k.first + team;
      llast = k.last;
    }
    lsrc = g.w + (static_cast<size_t>(le) * g.N + ltile * kRows + half) * row_bytes +
           c0 * kChunk + piece;
  };
  auto copy_stage = [&]() {
    if (li < tasks) {
      const uint32_t dst = ring_at + lstage * kStageBytes + half * kChunk;
      if (ltile * kRows + kRows <= g.N && lc * kChunk + kChunk <= row_bytes) {
#pragma unroll
        for (int j = 0; j < kRows / 2; ++j)
          copy_16(dst + 2 * j * kChunk + (((lane & 15) ^ L::swizzle(2 * j + half)) << 4),
                  lsrc + 2 * j * row_bytes, true);
      } else {
        // rows past the last and columns past the row are filled with zeros
        const bool inside = lc * kChunk + piece < row_bytes;
#pragma unroll 1
        for (int j = 0; j < kRows / 2; ++j) {
          const bool ok = inside && ltile * kRows + half + 2 * j < g.N;
          copy_16(dst + 2 * j * kChunk + (((lane & 15) ^ L::swizzle(2 * j + half)) << 4),
                  ok ? lsrc + 2 * j * row_bytes : g.w, ok);
        }
      }
      lsrc += kChunk;
      if (++lc == c1) {
        lc = c0;
        next_tile(false);
      }
    }
    if (++lstage == kStages) lstage = 0;
    copies_commit();
  };
  if (c0 < c1) next_tile(true);
  else li = tasks;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_stage();

  const unsigned short* __restrict__ x = static_cast<const unsigned short*>(g.x);
  const uint8_t* const x_at = xs + gq * pitch + t * 16;
  int stage = 0;
  for (int i = blockIdx.x; i < tasks; i += gridDim.x) {
    const Task k = task_of(g, prefix, i, spans, span, row_tiles);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    Meta<V> meta, coming;
    // this warp's tile: a span has one for each team, so that a tile's sums stay
    // in registers over all panels of x
    const int tile = k.first + team;
    const size_t row = static_cast<size_t>(k.e) * g.N;
    const size_t ra = (row + min(tile * kRows + gq, g.N - 1)) * groups;
    const size_t rb = (row + min(tile * kRows + gq + 8, g.N - 1)) * groups;
    if (tile < k.last && c0 < c1) meta.template load<ZEROS>(g, ra, rb, c0, groups, t);
    for (int d0 = 0; d0 < g.D; d0 += kPanel) {
      // ---- this panel of x ---------------------------------------------------------
      const int cols = min(kPanel, g.D - d0);
      const int pieces = (cols + 31) / 32 * 4;  // of 8 columns, whole steps of 32
      __syncthreads();  // the panel before has been read
      for (int q = threadIdx.x; q < k.cnt * pieces; q += kThreads) {
        const int token = q / pieces, at = q - token * pieces;
        const int src = source_row(g.p2u, g.T, k.p0 + token);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (src >= 0 && at * 8 < cols)
          v = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(src) * g.D + d0 + at * 8);
        int place = at;
        if constexpr (V > 0) {
          // word i of a step goes to thread i / V as its word i % V; columns
          // (0, 4), (1, 5), (2, 6), (3, 7) of a word pair up as the nibbles do
          constexpr int kWords = 4 * V;
          const int step = at / kWords, w = at - step * kWords;
          place = step * kWords + (w % V) * 4 + w / V;
          v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                         __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
        *reinterpret_cast<uint4*>(xs + token * pitch + place * 16) = v;
      }
      __syncthreads();

      // ---- products ------------------------------------------------------------------
      const int b0 = max(c0, d0 / L::kPerChunk);
      const int b1 = min(c1, (d0 + cols + L::kPerChunk - 1) / L::kPerChunk);
      if (tile < k.last) {
        for (int c = b0; c < b1; ++c) {
          copy_stage();
          if (c + 1 < c1) coming.template load<ZEROS>(g, ra, rb, c + 1, groups, t);
          copies_wait<kStages - 1>();
          __syncwarp();
          const uint8_t* const at = smem + (warp * kStages + stage) * kStageBytes + gq * kChunk;
          const int sw = L::swizzle(gq);  // and of row gq + 8
          const int col = c * L::kPerChunk - d0;
          const uint8_t* const xa = x_at + col * 2;
          [[maybe_unused]] float sum[4];  // bf16 weights: this chunk's
#pragma unroll
          for (int s = 0; s < L::kSteps; ++s) {
            if (col + s * L::kStep >= cols) break;
            if constexpr (V == 0) {
              uint32_t wa[4], wb[4], xv[4];
              const uint8_t* const from = at + (((4 * s + t) ^ sw) << 4);
              load_words<4>(from, wa);
              load_words<4>(from + 8 * kChunk, wb);
              load_words<4>(xa + s * 64, xv);
              if (s == 0)
                mma_16816_from_zero(sum, wa[0], wb[0], wa[1], wb[1], xv[0], xv[1]);
              else
                mma_16816(sum, wa[0], wb[0], wa[1], wb[1], xv[0], xv[1]);
              mma_16816(sum, wa[2], wb[2], wa[3], wb[3], xv[2], xv[3]);
            } else {
              uint32_t wa[V], wb[V];
              const int byte = s * (16 * V) + t * (4 * V);
              const uint8_t* const from = at + (((byte >> 4) ^ sw) << 4) + (byte & 15);
              load_words<V>(from, wa);
              load_words<V>(from + 8 * kChunk, wb);
              const int holder = (lane & 28) | (s & 3);
              const uint32_t a = __shfl_sync(0xffffffffu, meta.a[s >> 2], holder);
              const uint32_t b = __shfl_sync(0xffffffffu, meta.b[s >> 2], holder);
              const __nv_bfloat162 za = zero_pair(ZEROS ? a & 0xf0000u : 8u << 16);
              const __nv_bfloat162 zb = zero_pair(ZEROS ? b & 0xf0000u : 8u << 16);
              float p[4];
#pragma unroll
              for (int v = 0; v < V; ++v) {
                uint32_t xv[4];
                load_words<4>(xa + s * (64 * V) + v * 64, xv);
                if (v == 0)
                  mma_16816_from_zero(p, nibbles(wa[v], 0, za), nibbles(wb[v], 0, zb),
                                      nibbles(wa[v], 1, za), nibbles(wb[v], 1, zb), xv[0], xv[1]);
                else
                  mma_16816(p, nibbles(wa[v], 0, za), nibbles(wb[v], 0, zb), nibbles(wa[v], 1, za),
                            nibbles(wb[v], 1, zb), xv[0], xv[1]);
                mma_16816(p, nibbles(wa[v], 2, za), nibbles(wb[v], 2, zb), nibbles(wa[v], 3, za),
                          nibbles(wb[v], 3, zb), xv[2], xv[3]);
              }
              const float sa = __uint_as_float(a << 16), sb = __uint_as_float(b << 16);
              acc[0] = fmaf(sa, p[0], acc[0]);
              acc[1] = fmaf(sa, p[1], acc[1]);
              acc[2] = fmaf(sb, p[2], acc[2]);
              acc[3] = fmaf(sb, p[3], acc[3]);
            }
          }
          if constexpr (V == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += sum[j];
          }
          __syncwarp();  // all lanes have read the stage before it is filled again
          if (++stage == kStages) stage = 0;
          meta = coming;
        }
        if (d0 + kPanel < g.D) continue;  // more panels: the sums go on
        // fragment: weight rows gq and gq + 8, tokens 2 t and 2 t + 1
        const int n0 = tile * kRows;
        if constexpr (SHARED) {
          float(*sums)[kTokens][kRows + 1] = part + team * kShare;
          sums[member][2 * t][gq] = acc[0];
          sums[member][2 * t + 1][gq] = acc[1];
          sums[member][2 * t][gq + 8] = acc[2];
          sums[member][2 * t + 1][gq + 8] = acc[3];
          team_sync(team + 1);
          const int token = member * 2 + (lane >> 4), n = lane & 15;
          if (token < k.cnt && n0 + n < g.N) {
            float v = sums[0][token][n];
#pragma unroll
            for (int w = 1; w < kShare; ++w) v += sums[w][token][n];
            store_value(g, static_cast<size_t>(k.p0 + token) * g.N + n0 + n, v);
          }
          team_sync(team + 1);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int token = 2 * t + (j & 1), n = n0 + gq + (j >> 1) * 8;
            if (token < k.cnt && n < g.N)
              store_value(g, static_cast<size_t>(k.p0 + token) * g.N + n, acc[j]);
          }
        }
      }
    }
  }
}

template <int V, bool ZEROS, bool SHARED>
int launch_shared(const FewArgs& a, long long groups, int sms, cudaStream_t st) {
  constexpr int span = SHARED ? kWarps / kShare : kWarps;
  static std::atomic<int> granted[kSmemDevs];
  const auto kern = expert_matmul_few_kernel<V, ZEROS, SHARED>;
  const int smem = few_smem(a.E, a.D);
  cudaError_t e = allow_smem(kern, smem, granted);
  if (e != cudaSuccess) return MR_ERR_CUDA;
  const int row_tiles = (a.N + kRows - 1) / kRows;
  const long long tasks = groups * ((row_tiles + span - 1) / span);
  if (tasks > INT_MAX / 2) return MR_ERR_UNSUPPORTED;  // a block's next task stays an int
  e = launch_kernel(kern, dim3(static_cast<unsigned>(tasks < sms ? tasks : sms)), dim3(kThreads),
                    smem, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int V, bool ZEROS>
int launch_typed(const FewArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MR_ERR_CUDA;
  // row groups at most (the host does not know which experts have rows)
  const long long groups = static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / kTokens;
  const int row_tiles = (a.N + kRows - 1) / kRows;
  // Fewer tiles than twice the warps of the GPU: four warps to a tile.
  if (groups * row_tiles <= 2ll * sms * kWarps)
    return launch_shared<V, ZEROS, true>(a, groups, sms, st);
  return launch_shared<V, ZEROS, false>(a, groups, sms, st);
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
