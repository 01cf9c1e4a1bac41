// The end of an expert block and the beginning of the next one, on token rows:
//
//   y    = sum_k w_k z[p_k]                      (or z's own row without a map)
//   h    = y r_post post_weight,   r_post = 1 / sqrt(mean y^2 + eps)
//   x    = residual + scale gate h
//   n    = x r_pre pre_weight,     r_pre = 1 / sqrt(mean x^2 + eps)
//
// and its gradients.  With g_x the whole gradient of x, xh = x r_pre, yh = y r_post:
//
//   u   = grad_normed pre_weight;   g_x = grad_sum + r_pre (u - xh mean(u xh))
//   c   = gate post_weight yh;      v = scale gate post_weight g_x
//   g_y = r_post (v - yh mean(v yh))
//   grad_gate = scale g_x h,  grad_pre_weight = sum_t grad_normed xh,
//   grad_post_weight = sum_t scale gate g_x yh
//
// Bound by HBM: every row is read once, held by the 1 to 16 warps of its team, and written
// once; all sums and both factors stay fp32, and x is normed before it is rounded.
//
// The forward (registers, of which rows of one piece to a lane spill 12 to 48 bytes a thread at 64; 8192
// tokens, 8 choices, 2048 bf16: 73 us, 5.1 TB/s, in every split tried, three to five blocks an SM
// alike; fp32 4096 columns 5.5 TB/s) needs one sum over a row behind the other.  The backward's second sum,
// mean(v yh), is over g_x, which holds the first; but it is linear in it:
//   sum c g_x = sum c (grad_sum + r_pre u) - r_pre mean(u xh) sum c xh,
// so all sums of a row are taken together behind one barrier.  A team keeps the
// columns' sums for the weights' gradients of all its rows, a block leaves its teams' as one
// row; a second kernel adds those up in order: repeated calls give the same bits.  Rows
// come through shared memory, several ahead; the instructions bound bf16 rows nearly as HBM
// does (8192 x 2048 39 us, 5.1 TB/s; 8192 x 4096 74, 5.4 TB/s; fp32 4096 x 4096 69, 5.8 TB/s).
// Two pieces to a lane and four warps to 2048 columns: with one piece and eight warps 62 us.
#include <atomic>
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_launch.cuh"
#include "router_rows.cuh"

namespace moe_router {
namespace {

constexpr int kMaxWarps = 16;     // of a row
constexpr int kBlockWarps = 8;    // of a block whose rows take fewer
constexpr int kFwdWarps = 8;      // most warps of a row whose lanes hold one or two pieces
constexpr int kSumThreads = 1024;

enum { GATE_NONE = 0, GATE_TOKEN = 1, GATE_VALUE = 2 };

struct NormArgs {
  const void* z;             // [T K, D], or [T, D] without a map
  const int32_t* u2p;        // [T K] or NULL
  const float* weights;      // [T, ld_w] or NULL
  const void* residual;      // [T, D]
  const float* post_weight;  // [D] or NULL
  const float* pre_weight;   // [D] or NULL
  const void* gate;          // by gate_kind
  void* sum;                 // x [T, D]
  void* normed;              // [T, D]
  void* block;               // y [T, D] or NULL
  float2* rstd;              // [T]: r_post, r_pre; NULL in a forward that keeps nothing
  const void* grad_sum;      // [T, D] or NULL
  const void* grad_normed;   // [T, D]
  void* grad_block;          // [T, D]
  void* grad_residual;       // [T, D]
  void* grad_gate;           // like gate
  float* partial;            // [blocks, 2, D]
  float* grad_post;          // [D]
  float* grad_pre;           // [D]
  long long ld_w;
  int T, K, D, gate_kind, warps;
  float scale, eps;
};

// A row's team of warps, and sums over it.
struct RowTeam {
  int warps, team, teams, warp, lane;

  __device__ __forceinline__ void sync() const {
    if (teams == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
  }

  // Three values (below: one) summed over the team, with cells [3][kMaxWarps] of its own, 16-byte
  // aligned and zero behind its warps: four warps' a read.
  __device__ __forceinline__ void sum3(float* mine, float (&v)[3]) const {
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = seg_sum<32>(v[i]);
    if (warps == 1) return;
    if (lane < 3) mine[lane * kMaxWarps + warp] = lane == 0 ? v[0] : lane == 1 ? v[1] : v[2];
    sync();
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = 0.0f;
    for (int w = 0; w < warps; w += 4) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const float4 c = *reinterpret_cast<const float4*>(mine + i * kMaxWarps + w);
        v[i] += (c.x + c.y) + (c.z + c.w);
      }
    }
  }

  // A value summed over the team, the same in all its threads; cells: one for each warp of the
  // block.  With two sets of cells in turn one barrier is enough: who writes a set has
  // passed the barrier behind its last reading.
  __device__ __forceinline__ float sum(float* cells, float v) const {
    v = seg_sum<32>(v);
    if (warps == 1) return v;
    float* const mine = cells + team * warps;
    if (lane == 0) mine[warp] = v;
    sync();
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += mine[w];
    return v;
  }
};

__device__ __forceinline__ RowTeam row_team(int warps) {
  RowTeam r;
  const int warp = threadIdx.x >> 5;
  r.warps = warps;
  r.team = warp / warps;
  r.teams = (blockDim.x >> 5) / warps;
  r.warp = warp - r.team * warps;
  r.lane = threadIdx.x & 31;
  return r;
}

// A lane's values of a [D] fp32 vector at the columns of its piece; `none` outside.
template <typename P, int BYTES>
__device__ __forceinline__ void vector_at(const float* __restrict__ w, int col0, int lane, int D,
                                          float (&v)[P::kN]) {
  if constexpr (BYTES == 16) {
    const int c = P::column(col0, 0, lane);
    if (c < D) {
#pragma unroll
      for (int j = 0; j < P::kN; j += 4) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(w + c + j));
        v[j] = t.x; v[j + 1] = t.y; v[j + 2] = t.z; v[j + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < P::kN; ++j) v[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int c = P::column(col0, j / P::kEach, lane) + j % P::kEach;
      v[j] = c < D ? __ldg(w + c) : 0.0f;
    }
  }
}

// Is the piece's access q inside the row?  (kEach columns that are all in or all out)
template <typename P>
__device__ __forceinline__ bool any_inside(int col0, int lane, int D) {
  return P::column(col0, 0, lane) < D;
}

// A piece's row, widened; zeros outside it.
template <typename P, bool STREAM>
__device__ __forceinline__ void load_wide(const void* base, int row, int col0, int lane, int D,
                                          float (&v)[P::kN]) {
  P p;
  if (any_inside<P>(col0, lane, D)) {
    p.template load<STREAM>(base, static_cast<size_t>(row) * D, col0, lane, D);
    p.widen(v);
  } else {
#pragma unroll
    for (int j = 0; j < P::kN; ++j) v[j] = 0.0f;
  }
}

// ONE: a block is one team (and has one barrier: sixteen a block, which barriers of teams
// take, leave room for four blocks on an SM).
template <int DT, int BYTES, int U, bool ONE>
__global__ __launch_bounds__(32 * (U == 4 ? kMaxWarps : kFwdWarps), U == 1 ? 4 : U == 2 ? 3 : 1)
    void norm_fwd_kernel(const NormArgs a) {
  using P = Piece<DT, BYTES>;
  constexpr int kAhead = 8 / U;  // rows of z in flight
  __shared__ float cells[2][kMaxWarps];
  pdl_enter();
  RowTeam r = row_team(a.warps);
  if (ONE) {
    r.team = 0;
    r.teams = 1;
  }
  const int lane = r.lane, t = blockIdx.x * r.teams + r.team;
  if (t >= a.T) return;  // whole teams, with barriers of their own
  const size_t at = static_cast<size_t>(t) * a.D;
  int col[U];
#pragma unroll
  for (int q = 0; q < U; ++q) col[q] = (r.warp + q * a.warps) * 32 * P::kN;

  // ---- the block's output, the residual's row (and the gate's) on the way ---------------
  float y[U][P::kN];
  P res[U], gates[U];
  int p0 = -1, p1 = -1;  // the row's choices and their weights, two to a lane
  float w0 = 1.0f, w1 = 1.0f;
  if (a.u2p != nullptr) {
    const unsigned rows = static_cast<unsigned>(a.T) * static_cast<unsigned>(a.K);
    if (lane < a.K) {
      p0 = a.u2p[t + static_cast<size_t>(lane) * a.T];
      if (a.weights != nullptr) w0 = a.weights[t * a.ld_w + lane];
    }
    if (lane + 32 < a.K) {
      p1 = a.u2p[t + static_cast<size_t>(lane + 32) * a.T];
      if (a.weights != nullptr) w1 = a.weights[t * a.ld_w + lane + 32];
    }
    if (static_cast<unsigned>(p0) >= rows) p0 = -1;
    if (static_cast<unsigned>(p1) >= rows) p1 = -1;
  }
#pragma unroll
  for (int q = 0; q < U; ++q) {
    res[q].template load<true>(a.residual, at, col[q], lane, a.D);
    if (a.gate_kind == GATE_VALUE) gates[q].template load<true>(a.gate, at, col[q], lane, a.D);
  }
  if (a.u2p != nullptr) {
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int j = 0; j < P::kN; ++j) y[q][j] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kAhead) {
      int p[kAhead];
      float w[kAhead];
      P z[kAhead][U];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u;  // past K the lane's own choice is empty
        p[u] = __shfl_sync(0xffffffffu, k < 32 ? p0 : p1, k & 31);
        w[u] = __shfl_sync(0xffffffffu, k < 32 ? w0 : w1, k & 31);
        if (p[u] < 0) continue;
#pragma unroll
        for (int q = 0; q < U; ++q)
          z[u][q].template load<true>(a.z, static_cast<size_t>(p[u]) * a.D, col[q], lane, a.D);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (p[u] < 0) continue;
#pragma unroll
        for (int q = 0; q < U; ++q) {
          if (!any_inside<P>(col[q], lane, a.D)) continue;
          float v[P::kN];
          z[u][q].widen(v);
#pragma unroll
          for (int j = 0; j < P::kN; ++j) y[q][j] = fmaf(w[u], v[j], y[q][j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < U; ++q) load_wide<P, true>(a.z, t, col[q], lane, a.D, y[q]);
  }
  if (a.block != nullptr) {
#pragma unroll
    for (int q = 0; q < U; ++q) P::store(a.block, at, col[q], lane, a.D, y[q]);
  }

  // ---- the norm behind the block, gate, residual (weights asked for before the barriers) --
  float r_post = 1.0f, r_pre = 1.0f;
  float by = a.scale;
  if (a.gate_kind == GATE_TOKEN) by *= static_cast<const float*>(a.gate)[t];
  if (a.post_weight != nullptr) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float w[P::kN];
      vector_at<P, BYTES>(a.post_weight, col[q], lane, a.D, w);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        s = fmaf(y[q][j], y[q][j], s);
        y[q][j] *= w[j];
      }
    }
    r_post = __frsqrt_rn(r.sum(cells[0], s) / a.D + a.eps);
  }
  by *= r_post;
  float x[U][P::kN];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    if (!any_inside<P>(col[q], lane, a.D)) {
#pragma unroll
      for (int j = 0; j < P::kN; ++j) x[q][j] = 0.0f;
      continue;
    }
    if (a.gate_kind == GATE_VALUE) {
      float g[P::kN];
      gates[q].widen(g);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) y[q][j] *= g[j];
    }
    res[q].widen(x[q]);
#pragma unroll
    for (int j = 0; j < P::kN; ++j) x[q][j] = fmaf(by, y[q][j], x[q][j]);
    P::store(a.sum, at, col[q], lane, a.D, x[q]);
  }

  // ---- the norm before the next block -----------------------------------------------------
  if (a.pre_weight != nullptr) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float w[P::kN];
      vector_at<P, BYTES>(a.pre_weight, col[q], lane, a.D, w);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        s = fmaf(x[q][j], x[q][j], s);
        x[q][j] *= w[j];
      }
    }
    r_pre = __frsqrt_rn(r.sum(cells[1], s) / a.D + a.eps);
#pragma unroll
    for (int q = 0; q < U; ++q) {
#pragma unroll
      for (int j = 0; j < P::kN; ++j) x[q][j] *= r_pre;
      P::store(a.normed, at, col[q], lane, a.D, x[q]);
    }
  }
  if (a.rstd != nullptr && r.warp == 0 && lane == 0) a.rstd[t] = make_float2(r_post, r_pre);
}

// The rows of a backward on their way through shared memory: a thread's pieces go to places
// of its own, so that it waits for its own copies and no barrier is needed; each warp's
// first lane brings the row's factors and gate.  Both weights lie behind the ring, in the order
// in which a warp reads them.
enum { ROW_GS = 0, ROW_GN = 1, ROW_X = 2, ROW_Y = 3, ROW_GATE = 4 };

// Places for 256 threads (512 in the blocks of long rows) whatever a block has, so that a
// thread's places lie at fixed distances.
__host__ __device__ constexpr int places_of(bool is_long) { return 32 * (is_long ? kMaxWarps : kBlockWarps); }
__host__ __device__ constexpr int stage_bytes(bool is_long, int pieces, bool value) {
  return places_of(is_long) * 16 * pieces * (4 + value) + places_of(is_long) / 32 * 16;
}

// Both weights are kept in shared memory for 16-byte accesses (long rows fill it).
__host__ __device__ constexpr bool weights_kept(int bytes, bool is_long) {
  return bytes == 16 && !is_long;
}

template <typename P, int U, bool VALUE, bool LONG>
struct Ring {
  static constexpr int kPitch = places_of(LONG) * 16;
  static constexpr int kStage = stage_bytes(LONG, U, VALUE);
  static constexpr bool kWeights = weights_kept(P::kBytes, LONG);  // in shared memory
  uint32_t base, factors, weights;  // the thread's, its warp's, and its weights' places
  int lane;

  __device__ __forceinline__ uint32_t at(int stage, int array, int q) const {
    return base + stage * kStage + (array * U + q) * kPitch;
  }
  __device__ __forceinline__ uint32_t factors_at(int stage) const { return factors + stage * kStage; }
  __device__ __forceinline__ uint32_t weight_at(int which, int q, int h) const {
    return weights + ((which * U + q) * (P::kN / 4) + h) * kPitch;
  }

  template <bool FULL>
  __device__ __forceinline__ void load(const NormArgs& a, int t, int stage, const int (&col)[U]) const {
    const size_t row = static_cast<size_t>(t) * a.D;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!any_inside<P>(col[q], lane, a.D)) continue;
      if (FULL || a.grad_sum != nullptr)
        P::load_async(at(stage, ROW_GS, q), a.grad_sum, row, col[q], lane, a.D);
      if (FULL || a.pre_weight != nullptr) {
        P::load_async(at(stage, ROW_GN, q), a.grad_normed, row, col[q], lane, a.D);
        P::load_async(at(stage, ROW_X, q), a.sum, row, col[q], lane, a.D);
      }
      if (FULL || a.block != nullptr)
        P::load_async(at(stage, ROW_Y, q), a.block, row, col[q], lane, a.D);
      if constexpr (VALUE)
        P::load_async(at(stage, ROW_GATE, q), a.gate, row, col[q], lane, a.D);
    }
    if (lane == 0) {
      if (a.rstd != nullptr) copy_async<8>(factors_at(stage), a.rstd + t);
      if (a.gate_kind == GATE_TOKEN)
        copy_async<4>(factors_at(stage) + 8, static_cast<const float*>(a.gate) + t);
    }
  }

  __device__ __forceinline__ float factor(int stage, int i) const {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(factors_at(stage) + 4 * i) : "memory");
    return v;
  }

  __device__ __forceinline__ void widened(int stage, int array, int q, float (&v)[P::kN]) const {
    P p;
    p.read(at(stage, array, q));
    p.widen(v);
  }

  template <int BYTES>
  __device__ __forceinline__ void weight(const float* w, int which, int q, int col, int D,
                                         float (&v)[P::kN]) const {
    if constexpr (kWeights) {
#pragma unroll
      for (int h = 0; h < P::kN / 4; ++h)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                     : "r"(weight_at(which, q, h)));
    } else {
      vector_at<P, BYTES>(w, col, lane, D, v);
    }
  }
};

// With raw rows x and y (xh = r_pre x, yh = r_post y), u = grad_normed pre_weight and
// c = gate post_weight y, a lane's share of the row's sums is
//   s0 = sum u x,  s1 = sum c (grad_sum + r_pre u),  s2 = sum c x,
// and then, with m = r_pre^2 mean(u x) and f = scale gate_token r_post,
//   g_x = grad_sum + r_pre u - r_pre m x,  g_y = (f g_x) gate post_weight - y r_post mean_v r_post,
//   the weights' sums take (r_pre grad_normed) x and (f g_x gate) y.
// FULL: both norms, grad_sum given, known when the kernel is built (which saves a seventh of its
// instructions; they bound it with bf16 rows).
template <int DT, int BYTES, int U, bool VALUE, bool LONG, bool FULL>
__global__ __launch_bounds__(32 * (LONG ? kMaxWarps : kBlockWarps), U <= 2 ? 2 : 1)
    void norm_bwd_kernel(const NormArgs a, int stages) {
  using P = Piece<DT, BYTES>;
  extern __shared__ __align__(16) uint8_t dynamic_smem[];
  __shared__ __align__(16) float cells[2][kBlockWarps][3 * kMaxWarps];  // [.][team]
  pdl_enter();
  const RowTeam r = row_team(a.warps);
  const int first = blockIdx.x * r.teams + r.team, step = gridDim.x * r.teams;
  const int lane = r.lane;
  const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(dynamic_smem));
  using R = Ring<P, U, VALUE, LONG>;
  const R ring{smem + threadIdx.x * 16, smem + R::kStage - (places_of(LONG) / 32 - (threadIdx.x >> 5)) * 16,
               smem + stages * R::kStage + (r.warp * 32 + lane) * 16, lane};
  for (int i = threadIdx.x; i < 2 * kBlockWarps * 3 * kMaxWarps; i += blockDim.x) cells[0][0][i] = 0.0f;
  __syncthreads();
  int col[U];
#pragma unroll
  for (int q = 0; q < U; ++q) col[q] = (r.warp + q * a.warps) * 32 * P::kN;
  const bool pre = FULL || a.pre_weight != nullptr, post = FULL || a.post_weight != nullptr;
  const bool summed = FULL || a.grad_sum != nullptr, block = FULL || a.block != nullptr;
  const float by_columns = 1.0f / static_cast<float>(a.D);
  int ahead = first;  // the next row to ask for
  for (int s = 0; s < stages - 1; ++s, ahead += step) {
    if (ahead < a.T) ring.template load<FULL>(a, ahead, s, col);
    copies_commit_group();
  }
  if constexpr (R::kWeights) {
    if (r.team == 0) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const float* const w = which == 0 ? a.post_weight : a.pre_weight;
#pragma unroll
        for (int q = 0; q < U; ++q) {
          float v[P::kN];
#pragma unroll
          for (int j = 0; j < P::kN; ++j) v[j] = 1.0f;
          if (w != nullptr) vector_at<P, BYTES>(w, col[q], lane, a.D, v);
#pragma unroll
          for (int h = 0; h < P::kN / 4; ++h)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(ring.weight_at(which, q, h)),
                         "f"(v[4 * h]), "f"(v[4 * h + 1]), "f"(v[4 * h + 2]), "f"(v[4 * h + 3])
                         : "memory");
        }
      }
    }
    __syncthreads();
  }
  float by_post[U][P::kN], by_pre[U][P::kN];  // the weights' gradients
#pragma unroll
  for (int q = 0; q < U; ++q)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) by_post[q][j] = by_pre[q][j] = 0.0f;
  int stage = 0, flip = 0;
  for (int t = first; t < a.T; t += step, flip ^= 1) {
    __syncwarp();  // the lanes have read the factors of the stage that is filled again
    if (ahead < a.T) ring.template load<FULL>(a, ahead, stage == 0 ? stages - 1 : stage - 1, col);
    ahead += step;
    copies_commit_group();
    if (stages == 4) copies_wait_group<3>();
    else if (stages == 3) copies_wait_group<2>();
    else if (stages == 2) copies_wait_group<1>();
    else copies_wait_group<0>();
    __syncwarp();
    const float r_post = a.rstd != nullptr ? ring.factor(stage, 0) : 1.0f;
    const float r_pre = a.rstd != nullptr ? ring.factor(stage, 1) : 1.0f;
    float s[3] = {0.0f, 0.0f, 0.0f};
    float g[U][P::kN];  // grad_sum + r_pre u
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!any_inside<P>(col[q], lane, a.D)) continue;
      float x[P::kN], v[P::kN], w[P::kN];
      if (!FULL) {
#pragma unroll
        for (int j = 0; j < P::kN; ++j) g[q][j] = x[j] = 0.0f;
      }
      if (summed) ring.widened(stage, ROW_GS, q, g[q]);
      if (pre) {
        ring.widened(stage, ROW_X, q, x);
        ring.widened(stage, ROW_GN, q, v);
        ring.template weight<BYTES>(a.pre_weight, 1, q, col[q], a.D, w);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          const float gn = r_pre * v[j], u = gn * w[j];
          by_pre[q][j] = fmaf(gn, x[j], by_pre[q][j]);
          s[0] = fmaf(u, x[j], s[0]);
          g[q][j] += u;
        }
      }
      if (block) {
        ring.widened(stage, ROW_Y, q, v);
        if constexpr (VALUE) {
          ring.widened(stage, ROW_GATE, q, w);
#pragma unroll
          for (int j = 0; j < P::kN; ++j) v[j] *= w[j];
        }
        if (post) {
          ring.template weight<BYTES>(a.post_weight, 0, q, col[q], a.D, w);
#pragma unroll
          for (int j = 0; j < P::kN; ++j) v[j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          s[1] = fmaf(v[j], g[q][j], s[1]);
          s[2] = fmaf(v[j], x[j], s[2]);
        }
      }
    }
    if (pre || post || a.gate_kind == GATE_TOKEN) r.sum3(cells[flip][r.team], s);
    // s[0] = r_pre sum u x;  g_x = g - k x
    const float k = pre ? r_pre * r_pre * (s[0] * by_columns) : 0.0f;
    const float whole = r_post * fmaf(-k, s[2], s[1]);  // sum c g_x, of yh
    const float by = a.gate_kind == GATE_TOKEN ? a.scale * ring.factor(stage, 2) : a.scale;
    const float f = by * r_post;
    const float back = post ? r_post * r_post * (by * whole * by_columns) : 0.0f;
    if (a.gate_kind == GATE_TOKEN && r.warp == 0 && lane == 0)
      static_cast<float*>(a.grad_gate)[t] = a.scale * whole;
    const size_t at = static_cast<size_t>(t) * a.D;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!any_inside<P>(col[q], lane, a.D)) continue;
      float v[P::kN], w[P::kN];
      if (pre) {
        ring.widened(stage, ROW_X, q, v);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) g[q][j] = fmaf(-k, v[j], g[q][j]);
      }
      P::store(a.grad_residual, at, col[q], lane, a.D, g[q]);
      if (block) ring.widened(stage, ROW_Y, q, v);
      if (post) ring.template weight<BYTES>(a.post_weight, 0, q, col[q], a.D, w);
      if constexpr (VALUE) {
        float gate[P::kN], gg[P::kN];
        ring.widened(stage, ROW_GATE, q, gate);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          gg[j] = f * g[q][j] * v[j];
          if (post) gg[j] *= w[j];
          g[q][j] *= gate[j];
        }
        P::store(a.grad_gate, at, col[q], lane, a.D, gg);
      }
      if (post) {
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          const float gh = f * g[q][j];
          by_post[q][j] = fmaf(gh, v[j], by_post[q][j]);
          g[q][j] = fmaf(gh, w[j], -back * v[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < P::kN; ++j) g[q][j] *= by;
      }
      P::store(a.grad_block, at, col[q], lane, a.D, g[q]);
    }
    if (++stage == stages) stage = 0;
  }
  if (a.partial == nullptr) return;
  // one row of sums a block: the teams' added up in the place of the rows under way
  float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.D;
  float* const part = reinterpret_cast<float*>(dynamic_smem);
  if (r.teams > 1) {
    __syncthreads();
    out = part + r.team * 2 * a.D;
  }
#pragma unroll
  for (int q = 0; q < U; ++q)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int c = P::column(col[q], j / P::kEach, lane) + j % P::kEach;
      if (c < a.D) {
        out[c] = by_post[q][j];
        out[a.D + c] = by_pre[q][j];
      }
    }
  if (r.teams > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += blockDim.x) {
      float v = part[c];
      for (int w = 1; w < r.teams; ++w) v += part[w * 2 * a.D + c];
      a.partial[static_cast<size_t>(blockIdx.x) * 2 * a.D + c] = v;
    }
  }
}

// The blocks' rows added up: 32 columns of one of the two a block, 32 warps on every
// 32nd row each.
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(const float* __restrict__ partial,
                                                               int rows, int D, float* post,
                                                               float* pre) {
  __shared__ float part[kSumThreads / 32][33];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* const out = blockIdx.y == 0 ? post : pre;
  if (out == nullptr) return;
  float s = 0.0f;
  if (c < D) {
    const float* at = partial + static_cast<size_t>(blockIdx.y) * D + c;
#pragma unroll 8
    for (int i = warp; i < rows; i += kSumThreads / 32)
      s += __ldcg(at + static_cast<size_t>(i) * 2 * D);
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) s += part[w][lane];
    out[c] = s;
  }
}

// ---- host ------------------------------------------------------------------------
// Bytes of one access: what every row of the call's [., D] tensors and its weights
// are aligned to.
int access_bytes(const NormArgs& a, int dtype) {
  uintptr_t all = static_cast<uintptr_t>(a.D) * (dtype == DT_F32 ? 4 : 2);
  for (const void* p : {a.z, a.residual, static_cast<const void*>(a.sum),
                        static_cast<const void*>(a.normed), static_cast<const void*>(a.block),
                        a.grad_sum, a.grad_normed, static_cast<const void*>(a.grad_block),
                        static_cast<const void*>(a.grad_residual),
                        static_cast<const void*>(a.post_weight),
                        static_cast<const void*>(a.pre_weight)})
    all |= reinterpret_cast<uintptr_t>(p);
  if (a.gate_kind == GATE_VALUE)
    all |= reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.grad_gate);
  return (all & 15u) == 0 ? 16 : (all & 3u) == 0 ? 4 : 2;
}

// Warps of a row and pieces of a lane.  Forward: one piece up to 8 warps, two up to 16
// pieces, else four.  Backward: as few pieces as 16 warps allow.
struct Split {
  int warps, pieces, teams;
};

Split split_of(int D, int columns, bool forward) {
  const int stretches = (D + columns - 1) / columns;
  int pieces;
  if (forward) pieces = stretches <= kFwdWarps ? 1 : stretches <= 2 * kFwdWarps ? 2 : 4;
  else pieces = stretches == 1 ? 1 : stretches <= 2 * kBlockWarps ? 2 : 4;
  const int warps = (stretches + pieces - 1) / pieces;
  return Split{warps, pieces, warps >= kBlockWarps ? 1 : kBlockWarps / warps};
}

// Blocks of a backward: what is resident, two on each SM for up to two pieces to a lane and one
// for longer rows.  From the sizes alone, so that sums have the same order on every GPU.
constexpr int kBwdBlocks = 2 * 152;

int bwd_blocks(int T, const Split& s) {
  const int most = (T + s.teams - 1) / s.teams;
  const int resident = s.pieces > 2 ? kBwdBlocks / 2 : kBwdBlocks;
  return most < resident ? most : resident;
}

// Rows of partial sums: a block's each, at any alignment (and so any number of teams).
size_t partial_rows(int T) { return T < kBwdBlocks ? T : kBwdBlocks; }

template <int DT, int BYTES, int U>
cudaError_t launch_fwd_pieces(const NormArgs& a, const Split& s, cudaStream_t st) {
  const dim3 grid((a.T + s.teams - 1) / s.teams), block(32 * s.warps * s.teams);
  return s.teams == 1 ? launch_kernel(norm_fwd_kernel<DT, BYTES, U, true>, grid, block, 0, st, a)
                      : launch_kernel(norm_fwd_kernel<DT, BYTES, U, false>, grid, block, 0, st, a);
}

template <int DT, int BYTES>
int launch_fwd(NormArgs a, cudaStream_t st) {
  const Split s = split_of(a.D, 32 * Piece<DT, BYTES>::kN, true);
  a.warps = s.warps;
  const cudaError_t e = s.pieces == 1   ? launch_fwd_pieces<DT, BYTES, 1>(a, s, st)
                        : s.pieces == 2 ? launch_fwd_pieces<DT, BYTES, 2>(a, s, st)
                                        : launch_fwd_pieces<DT, BYTES, 4>(a, s, st);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

// Rows on their way: as many as the blocks' shares of shared memory hold, four at most.
template <int DT, int BYTES, int U, bool VALUE, bool LONG, bool FULL>
cudaError_t launch_bwd_kernel(const NormArgs& a, const Split& s, int blocks, cudaStream_t st) {
  static std::atomic<int> granted[kSmemDevs];
  constexpr int size = stage_bytes(LONG, U, VALUE);
  constexpr int weights = weights_kept(BYTES, LONG) ? 2 * U * (Piece<DT, BYTES>::kN / 4) * places_of(LONG) * 16 : 0;
  constexpr int fit = ((U <= 2 ? 110 : 222) * 1024 - weights) / size;
  constexpr int stages = fit > 4 ? 4 : fit < 1 ? 1 : fit;
  constexpr size_t smem = static_cast<size_t>(stages) * size + weights;
  static_assert(smem > 48 * 1024 && smem <= 222 * 1024, "opted in, and within an SM's");
  const auto kern = norm_bwd_kernel<DT, BYTES, U, VALUE, LONG, FULL>;
  const cudaError_t e = allow_smem(kern, smem, granted);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(blocks), dim3(32 * s.warps * s.teams), smem, st, a, stages);
}

template <int DT, int BYTES, int U, bool VALUE, bool LONG>
cudaError_t launch_bwd_pieces(const NormArgs& a, const Split& s, int blocks, cudaStream_t st) {
  if constexpr (BYTES == 16) {
    if (a.pre_weight != nullptr && a.post_weight != nullptr && a.grad_sum != nullptr)
      return launch_bwd_kernel<DT, BYTES, U, VALUE, LONG, true>(a, s, blocks, st);
  }
  return launch_bwd_kernel<DT, BYTES, U, VALUE, LONG, false>(a, s, blocks, st);
}

template <int DT, int BYTES, bool VALUE>
cudaError_t launch_bwd_rows(const NormArgs& a, const Split& s, int blocks, cudaStream_t st) {
  if (s.pieces == 1) return launch_bwd_pieces<DT, BYTES, 1, VALUE, false>(a, s, blocks, st);
  if (s.pieces == 2) return launch_bwd_pieces<DT, BYTES, 2, VALUE, false>(a, s, blocks, st);
  // (8192 bf16 columns are 32 stretches of 256, or 64 of 128 as fp32 and by single values)
  if constexpr (Piece<DT, BYTES>::kN == 4) {
    if (s.warps > kBlockWarps) return launch_bwd_pieces<DT, BYTES, 4, VALUE, true>(a, s, blocks, st);
  }
  return launch_bwd_pieces<DT, BYTES, 4, VALUE, false>(a, s, blocks, st);
}

template <int DT, int BYTES>
int launch_bwd(NormArgs a, cudaStream_t st) {
  const Split s = split_of(a.D, 32 * Piece<DT, BYTES>::kN, false);
  a.warps = s.warps;
  const int blocks = bwd_blocks(a.T, s);
  cudaError_t e = a.gate_kind == GATE_VALUE ? launch_bwd_rows<DT, BYTES, true>(a, s, blocks, st)
                                            : launch_bwd_rows<DT, BYTES, false>(a, s, blocks, st);
  if (e == cudaSuccess && a.partial != nullptr)
    e = launch_kernel(norm_sum_kernel, dim3((a.D + 31) / 32, 2), dim3(kSumThreads), 0, st,
                      static_cast<const float*>(a.partial), blocks, a.D, a.grad_post,
                      a.grad_pre);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int check(int dtype, int T, int K, int D, float eps) {
  if (dtype != MR_F32 && dtype != MR_BF16) return MR_ERR_INVALID;
  if (T < 0 || K < 1 || D < 1 || static_cast<long long>(T) * K > INT_MAX) return MR_ERR_INVALID;
  if (!(eps > 0.0f)) return MR_ERR_INVALID;
  if (K > MR_MAX_TOPK || D > MR_MAX_NORM_FEATURES) return MR_ERR_UNSUPPORTED;
  if (T > MR_MAX_ROWS) return MR_ERR_UNSUPPORTED;  // (rows are stepped past T as ints)
  return MR_OK;
}

bool known_gate(int kind, const void* gate) {
  return (kind == MR_GATE_NONE && gate == nullptr) ||
         ((kind == MR_GATE_TOKEN || kind == MR_GATE_VALUE) && gate != nullptr);
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace moe_router

using namespace moe_router;

extern "C" {

int router_combine_norm_fwd(const void* expert_out, mr_dtype dtype,
                            const int32_t* unpermuted_to_permuted, const float* topk_weights,
                            int ld_weights, const void* residual, const float* post_weight,
                            const void* gate, mr_gate gate_kind, float residual_scale,
                            const float* pre_weight, float eps, int T, int K, int D, void* sum,
                            void* normed, void* block_out, float* rstd, mr_stream_t stream) {
  const int rc = check(dtype, T, K, D, eps);
  if (rc != MR_OK) return rc;
  if (unpermuted_to_permuted == nullptr && (K != 1 || topk_weights != nullptr))
    return MR_ERR_INVALID;
  if (topk_weights != nullptr && ld_weights < K) return MR_ERR_INVALID;
  if (gate_kind < MR_GATE_NONE || gate_kind > MR_GATE_VALUE) return MR_ERR_INVALID;
  if (T == 0) return MR_OK;
  if (!known_gate(gate_kind, gate) || expert_out == nullptr || residual == nullptr ||
      sum == nullptr || (pre_weight != nullptr && normed == nullptr) || !aligned(rstd, 8))
    return MR_ERR_INVALID;
  NormArgs a{};
  a.z = expert_out;
  a.u2p = unpermuted_to_permuted;
  a.weights = topk_weights;
  a.residual = residual;
  a.post_weight = post_weight;
  a.pre_weight = pre_weight;
  a.gate = gate;
  a.sum = sum;
  a.normed = pre_weight != nullptr ? normed : nullptr;
  a.block = block_out;
  a.rstd = reinterpret_cast<float2*>(rstd);
  a.ld_w = ld_weights;
  a.T = T; a.K = K; a.D = D;
  a.gate_kind = gate_kind;
  a.scale = residual_scale;
  a.eps = eps;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int bytes = access_bytes(a, dtype);
  if (dtype == MR_F32)
    return bytes == 16 ? launch_fwd<DT_F32, 16>(a, st) : launch_fwd<DT_F32, 4>(a, st);
  return bytes == 16  ? launch_fwd<DT_BF16, 16>(a, st)
         : bytes == 4 ? launch_fwd<DT_BF16, 4>(a, st)
                      : launch_fwd<DT_BF16, 2>(a, st);
}

size_t router_combine_norm_bwd_workspace_bytes(int T, int D) {
  if (T <= 0 || T > MR_MAX_ROWS || D < 1 || D > MR_MAX_NORM_FEATURES) return 0;
  return partial_rows(T) * 2 * D * sizeof(float);
}

int router_combine_norm_bwd(const void* grad_sum, const void* grad_normed, mr_dtype dtype,
                            const void* block_out, const void* sum, const float* rstd,
                            const float* post_weight, const void* gate, mr_gate gate_kind,
                            float residual_scale, const float* pre_weight, int T, int D,
                            void* grad_block, void* grad_residual, void* grad_gate,
                            float* grad_post_weight, float* grad_pre_weight, void* workspace,
                            size_t workspace_bytes, mr_stream_t stream) {
  const int rc = check(dtype, T, 1, D, 1.0f);
  if (rc != MR_OK) return rc;
  if (gate_kind < MR_GATE_NONE || gate_kind > MR_GATE_VALUE) return MR_ERR_INVALID;
  const bool pre = pre_weight != nullptr, post = post_weight != nullptr;
  if ((pre && grad_pre_weight == nullptr) || (post && grad_post_weight == nullptr))
    return MR_ERR_INVALID;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows: the weights' gradients are zero
    if (!pre && !post) return MR_OK;
    return launch_kernel(norm_sum_kernel, dim3((D + 31) / 32, 2), dim3(kSumThreads), 0, st,
                         static_cast<const float*>(nullptr), 0, D,
                         post ? grad_post_weight : static_cast<float*>(nullptr),
                         pre ? grad_pre_weight : static_cast<float*>(nullptr)) == cudaSuccess
               ? MR_OK
               : MR_ERR_CUDA;
  }
  const bool gated = gate_kind != MR_GATE_NONE;
  if (!known_gate(gate_kind, gate) || (gated && grad_gate == nullptr) ||
      (grad_sum == nullptr && !pre) || grad_block == nullptr || grad_residual == nullptr ||
      (pre && (grad_normed == nullptr || sum == nullptr)) ||
      ((post || gated) && block_out == nullptr) || ((pre || post) && rstd == nullptr) ||
      !aligned(rstd, 8))
    return MR_ERR_INVALID;
  if ((pre || post) &&
      (workspace == nullptr || !aligned(workspace, 16) ||
       workspace_bytes < router_combine_norm_bwd_workspace_bytes(T, D)))
    return MR_ERR_INVALID;
  NormArgs a{};
  a.grad_sum = grad_sum;
  a.grad_normed = pre ? grad_normed : nullptr;
  a.block = post || gated ? const_cast<void*>(block_out) : nullptr;
  a.sum = pre ? const_cast<void*>(sum) : nullptr;
  a.rstd = pre || post ? reinterpret_cast<float2*>(const_cast<float*>(rstd)) : nullptr;
  a.post_weight = post_weight;
  a.pre_weight = pre_weight;
  a.gate = gate;
  a.grad_block = grad_block;
  a.grad_residual = grad_residual;
  a.grad_gate = gated ? grad_gate : nullptr;
  a.partial = pre || post ? static_cast<float*>(workspace) : nullptr;
  a.grad_post = post ? grad_post_weight : nullptr;
  a.grad_pre = pre ? grad_pre_weight : nullptr;
  a.T = T; a.K = 1; a.D = D;
  a.gate_kind = gate_kind;
  a.scale = residual_scale;
  const int bytes = access_bytes(a, dtype);
  if (dtype == MR_F32)
    return bytes == 16 ? launch_bwd<DT_F32, 16>(a, st) : launch_bwd<DT_F32, 4>(a, st);
  return bytes == 16  ? launch_bwd<DT_BF16, 16>(a, st)
         : bytes == 4 ? launch_bwd<DT_BF16, 4>(a, st)
                      : launch_bwd<DT_BF16, 2>(a, st);
}

}  // extern "C"
