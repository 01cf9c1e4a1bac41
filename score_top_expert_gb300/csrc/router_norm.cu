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
// Bound by HBM: every row is read once, held in the registers of the 1 to 16 warps of
// its team, and written once; all sums and both factors stay fp32, and x is normed
// before it is rounded.
//
// The forward needs one sum over a row behind the other.  The backward's second sum,
// mean(v yh), is over g_x, which holds the first; but it is linear in it:
//   sum c g_x = sum c (grad_sum + r_pre u) - r_pre mean(u xh) sum c xh,
// so all sums of a row are taken together behind one barrier.  A team keeps the
// columns' sums for the weights' gradients of all its rows and leaves them as one row;
// a second kernel adds those up in order: repeated calls give the same bits.
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_rows.cuh"

namespace moe_router {
namespace {

constexpr int kMaxWarps = 16;     // of a row
constexpr int kBlockWarps = 8;    // of a block whose rows take fewer
constexpr int kAhead = 4;         // forward: rows of z in flight
constexpr int kSumThreads = 512;

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
  float* partial;            // [teams, 2, D]
  float* grad_post;          // [D]
  float* grad_pre;           // [D]
  long long ld_w;
  int T, K, D, gate_kind, warps;
  float scale, eps;
};

// A row's team of warps, and sums over it.
struct RowTeam {
  int warps, team, teams, warp, lane;
  float* cells;  // [teams, warps, kSums]

  __device__ __forceinline__ void sync() const {
    if (warps == static_cast<int>(blockDim.x >> 5)) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
  }

  // N values summed over the team, the same in all its threads.  The cells must not
  // be in use by an earlier call.
  template <int N>
  __device__ __forceinline__ void sum(float* cells_at, float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = seg_sum<32>(v[i]);
    if (warps == 1) return;
    float* const mine = cells_at + team * warps * N;
    if (lane < N) {
      float mineth = v[0];
#pragma unroll
      for (int i = 1; i < N; ++i) mineth = lane == i ? v[i] : mineth;
      mine[warp * N + lane] = mineth;
    }
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
      for (int w = 0; w < warps; ++w) s += mine[w * N + i];
      v[i] = s;
    }
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

template <int DT, int BYTES, int U>
__global__ __launch_bounds__(32 * kMaxWarps, 1) void norm_fwd_kernel(const NormArgs a) {
  using P = Piece<DT, BYTES>;
  __shared__ float cells[2][kMaxWarps];
  pdl_enter();
  const RowTeam r = row_team(a.warps);
  const int t = blockIdx.x * r.teams + r.team;
  if (t >= a.T) return;  // whole teams, with barriers of their own
  const int lane = r.lane;
  int col[U];
#pragma unroll
  for (int q = 0; q < U; ++q) col[q] = (r.warp + q * a.warps) * 32 * P::kN;

  // ---- the block's output -----------------------------------------------------------
  float y[U][P::kN];
  if (a.u2p != nullptr) {
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
    for (int q = 0; q < U; ++q)
      P::store(a.block, static_cast<size_t>(t) * a.D, col[q], lane, a.D, y[q]);
  }

  // ---- the norm behind the block, gate, residual ---------------------------------------
  float x[U][P::kN];
#pragma unroll
  for (int q = 0; q < U; ++q) load_wide<P, true>(a.residual, t, col[q], lane, a.D, x[q]);
  float r_post = 1.0f, r_pre = 1.0f;
  if (a.post_weight != nullptr) {
    float s[1] = {0.0f};
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int j = 0; j < P::kN; ++j) s[0] = fmaf(y[q][j], y[q][j], s[0]);
    r.sum(cells[0], s);
    r_post = __frsqrt_rn(s[0] / a.D + a.eps);
  }
  float by = a.scale * r_post;
  if (a.gate_kind == GATE_TOKEN) by *= static_cast<const float*>(a.gate)[t];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    if (a.post_weight != nullptr) {
      float w[P::kN];
      vector_at<P, BYTES>(a.post_weight, col[q], lane, a.D, w);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) y[q][j] *= w[j];
    }
    if (a.gate_kind == GATE_VALUE) {
      float g[P::kN];
      load_wide<P, true>(a.gate, t, col[q], lane, a.D, g);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) y[q][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < P::kN; ++j) x[q][j] = fmaf(by, y[q][j], x[q][j]);
    P::store(a.sum, static_cast<size_t>(t) * a.D, col[q], lane, a.D, x[q]);
  }

  // ---- the norm before the next block -----------------------------------------------------
  if (a.pre_weight != nullptr) {
    float s[1] = {0.0f};
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int j = 0; j < P::kN; ++j) s[0] = fmaf(x[q][j], x[q][j], s[0]);
    r.sum(cells[1], s);
    r_pre = __frsqrt_rn(s[0] / a.D + a.eps);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float w[P::kN];
      vector_at<P, BYTES>(a.pre_weight, col[q], lane, a.D, w);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) x[q][j] *= r_pre * w[j];
      P::store(a.normed, static_cast<size_t>(t) * a.D, col[q], lane, a.D, x[q]);
    }
  }
  if (a.rstd != nullptr && r.warp == 0 && lane == 0) a.rstd[t] = make_float2(r_post, r_pre);
}

// The rows of a backward that a lane holds, as they were loaded.
template <typename P, int U>
struct Held {
  P gs[U], gn[U], x[U], y[U], gate[U];
  float2 rstd;
  float token_gate;

  __device__ __forceinline__ void load(const NormArgs& a, int t, const int (&col)[U], int lane) {
    const size_t at = static_cast<size_t>(t) * a.D;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (a.grad_sum != nullptr) gs[q].template load<true>(a.grad_sum, at, col[q], lane, a.D);
      if (a.pre_weight != nullptr) {
        gn[q].template load<true>(a.grad_normed, at, col[q], lane, a.D);
        x[q].template load<true>(a.sum, at, col[q], lane, a.D);
      }
      if (a.block != nullptr) y[q].template load<true>(a.block, at, col[q], lane, a.D);
      if (a.gate_kind == GATE_VALUE) gate[q].template load<true>(a.gate, at, col[q], lane, a.D);
    }
    rstd = a.rstd != nullptr ? a.rstd[t] : make_float2(1.0f, 1.0f);
    token_gate = a.gate_kind == GATE_TOKEN ? static_cast<const float*>(a.gate)[t] : 1.0f;
  }
};

template <int DT, int BYTES, int U>
__global__ __launch_bounds__(32 * kMaxWarps, 1) void norm_bwd_kernel(const NormArgs a) {
  using P = Piece<DT, BYTES>;
  __shared__ float cells[2][3 * kMaxWarps];
  pdl_enter();
  const RowTeam r = row_team(a.warps);
  const int first = blockIdx.x * r.teams + r.team, step = gridDim.x * r.teams;
  const int lane = r.lane;
  int col[U];
#pragma unroll
  for (int q = 0; q < U; ++q) col[q] = (r.warp + q * a.warps) * 32 * P::kN;
  const bool pre = a.pre_weight != nullptr, post = a.post_weight != nullptr;
  float by_post[U][P::kN], by_pre[U][P::kN];  // the weights' gradients
#pragma unroll
  for (int q = 0; q < U; ++q)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) by_post[q][j] = by_pre[q][j] = 0.0f;
  Held<P, U> next;
  if (first < a.T) next.load(a, first, col, lane);
  int flip = 0;
  for (int t = first; t < a.T; t += step, flip ^= 1) {
    const Held<P, U> h = next;
    if (t + step < a.T) next.load(a, t + step, col, lane);
    const float r_post = h.rstd.x, r_pre = h.rstd.y;
    // sum u xh;  sum c (grad_sum + r_pre u);  sum c xh   (c without the token's gate)
    float s[3] = {0.0f, 0.0f, 0.0f};
    float g[U][P::kN], xh[U][P::kN], yh[U][P::kN], c[U][P::kN];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const bool in = any_inside<P>(col[q], lane, a.D);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) g[q][j] = xh[q][j] = yh[q][j] = c[q][j] = 0.0f;
      if (!in) continue;
      if (a.grad_sum != nullptr) h.gs[q].widen(g[q]);
      if (pre) {
        float w[P::kN], gn[P::kN];
        vector_at<P, BYTES>(a.pre_weight, col[q], lane, a.D, w);
        h.gn[q].widen(gn);
        h.x[q].widen(xh[q]);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          xh[q][j] *= r_pre;
          by_pre[q][j] = fmaf(gn[j], xh[q][j], by_pre[q][j]);
          const float u = gn[j] * w[j];
          s[0] = fmaf(u, xh[q][j], s[0]);
          g[q][j] = fmaf(r_pre, u, g[q][j]);
        }
      }
      if (a.block != nullptr) {
        h.y[q].widen(yh[q]);
        float w[P::kN];
        if (post) {
          vector_at<P, BYTES>(a.post_weight, col[q], lane, a.D, w);
        } else {
#pragma unroll
          for (int j = 0; j < P::kN; ++j) w[j] = 1.0f;
        }
        float gate[P::kN];
        if (a.gate_kind == GATE_VALUE) {
          h.gate[q].widen(gate);
        } else {
#pragma unroll
          for (int j = 0; j < P::kN; ++j) gate[j] = 1.0f;
        }
#pragma unroll
        for (int j = 0; j < P::kN; ++j) {
          yh[q][j] *= r_post;
          c[q][j] = gate[j] * w[j] * yh[q][j];
          s[1] = fmaf(c[q][j], g[q][j], s[1]);
          s[2] = fmaf(c[q][j], xh[q][j], s[2]);
        }
      }
    }
    if (pre || post || a.gate_kind == GATE_TOKEN) r.sum(cells[flip], s);
    const float mean = pre ? s[0] / a.D : 0.0f;
    const float whole = s[1] - r_pre * mean * s[2];  // sum c g_x
    const float by = a.scale * h.token_gate;
    const float mean_v = post ? by * whole / a.D : 0.0f;
    if (a.gate_kind == GATE_TOKEN && r.warp == 0 && lane == 0)
      static_cast<float*>(a.grad_gate)[t] = a.scale * whole;
    const size_t at = static_cast<size_t>(t) * a.D;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!any_inside<P>(col[q], lane, a.D)) continue;
#pragma unroll
      for (int j = 0; j < P::kN; ++j) g[q][j] = fmaf(-r_pre * mean, xh[q][j], g[q][j]);
      P::store(a.grad_residual, at, col[q], lane, a.D, g[q]);
      float w[P::kN], gate[P::kN], v[P::kN];
#pragma unroll
      for (int j = 0; j < P::kN; ++j) w[j] = gate[j] = 1.0f;
      if (post) vector_at<P, BYTES>(a.post_weight, col[q], lane, a.D, w);
      if (a.gate_kind == GATE_VALUE) {
        h.gate[q].widen(gate);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) v[j] = a.scale * g[q][j] * w[j] * yh[q][j];
        P::store(a.grad_gate, at, col[q], lane, a.D, v);
      }
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        const float gh = by * gate[j] * g[q][j];
        if (post) {
          by_post[q][j] = fmaf(gh, yh[q][j], by_post[q][j]);
          v[j] = r_post * (gh * w[j] - yh[q][j] * mean_v);
        } else {
          v[j] = gh;
        }
      }
      P::store(a.grad_block, at, col[q], lane, a.D, v);
    }
  }
  if (a.partial == nullptr) return;
  float* const mine = a.partial + static_cast<size_t>(first) * 2 * a.D;
#pragma unroll
  for (int q = 0; q < U; ++q)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int c = P::column(col[q], j / P::kEach, lane) + j % P::kEach;
      if (c < a.D) {
        if (post) mine[c] = by_post[q][j];
        if (pre) mine[a.D + c] = by_pre[q][j];
      }
    }
}

// The teams' rows added up: 32 columns of one of the two a block, 16 warps on every
// 16th row each.
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(const float* __restrict__ partial,
                                                               int teams, int D, float* post,
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
    for (int i = warp; i < teams; i += kSumThreads / 32)
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

// Warps of a row and pieces of a lane: as few pieces as 16 warps allow.
struct Split {
  int warps, pieces, teams;
};

Split split_of(int D, int columns) {
  const int stretches = (D + columns - 1) / columns;
  const int pieces = stretches <= kMaxWarps ? 1 : stretches <= 2 * kMaxWarps ? 2 : 4;
  const int warps = (stretches + pieces - 1) / pieces;
  return Split{warps, pieces, warps >= kBlockWarps ? 1 : kBlockWarps / warps};
}

// Teams of a backward: eight rows each at least, and no more than about two blocks of
// each SM hold.  From the sizes alone, so that sums have the same order on every GPU.
constexpr int kBwdBlocks = 2 * 152;

int bwd_blocks(int T, const Split& s) {
  const int most = (T + s.teams - 1) / s.teams;
  return most < kBwdBlocks ? most : kBwdBlocks;
}

// Rows of partial sums for any alignment (narrow accesses take more warps a row, so
// fewer teams).
size_t partial_rows(int T) {
  const size_t most = static_cast<size_t>(kBwdBlocks) * kBlockWarps;
  return static_cast<size_t>(T) + kBlockWarps < most ? static_cast<size_t>(T) + kBlockWarps : most;
}

template <int DT, int BYTES>
int launch_fwd(NormArgs a, cudaStream_t st) {
  const Split s = split_of(a.D, 32 * Piece<DT, BYTES>::kN);
  a.warps = s.warps;
  const dim3 grid((a.T + s.teams - 1) / s.teams), block(32 * s.warps * s.teams);
  const cudaError_t e =
      s.pieces == 1   ? launch_kernel(norm_fwd_kernel<DT, BYTES, 1>, grid, block, 0, st, a)
      : s.pieces == 2 ? launch_kernel(norm_fwd_kernel<DT, BYTES, 2>, grid, block, 0, st, a)
                      : launch_kernel(norm_fwd_kernel<DT, BYTES, 4>, grid, block, 0, st, a);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int DT, int BYTES>
int launch_bwd(NormArgs a, cudaStream_t st) {
  const Split s = split_of(a.D, 32 * Piece<DT, BYTES>::kN);
  a.warps = s.warps;
  const int blocks = bwd_blocks(a.T, s);
  const dim3 grid(blocks), block(32 * s.warps * s.teams);
  cudaError_t e =
      s.pieces == 1   ? launch_kernel(norm_bwd_kernel<DT, BYTES, 1>, grid, block, 0, st, a)
      : s.pieces == 2 ? launch_kernel(norm_bwd_kernel<DT, BYTES, 2>, grid, block, 0, st, a)
                      : launch_kernel(norm_bwd_kernel<DT, BYTES, 4>, grid, block, 0, st, a);
  if (e == cudaSuccess && a.partial != nullptr)
    e = launch_kernel(norm_sum_kernel, dim3((a.D + 31) / 32, 2), dim3(kSumThreads), 0, st,
                      static_cast<const float*>(a.partial), blocks * s.teams, a.D, a.grad_post,
                      a.grad_pre);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int check(int dtype, int T, int K, int D, float eps) {
  if (dtype != MR_F32 && dtype != MR_BF16) return MR_ERR_INVALID;
  if (T < 0 || K < 1 || D < 1 || static_cast<long long>(T) * K > INT_MAX) return MR_ERR_INVALID;
  if (!(eps > 0.0f)) return MR_ERR_INVALID;
  if (K > MR_MAX_TOPK || D > MR_MAX_NORM_FEATURES) return MR_ERR_UNSUPPORTED;
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
  if (T <= 0 || D < 1 || D > MR_MAX_NORM_FEATURES) return 0;
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
