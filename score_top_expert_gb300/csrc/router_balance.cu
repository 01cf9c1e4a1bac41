// Load-balancing loss of each sequence of a packed batch, the tokens per expert, the
// z loss, and the gradient of both by the logits.
//
//   sequence s owns tokens [o_s, o_{s+1}), n_s of them;  q = softmax(x) or
//   sigma(x) / sum sigma(x);  c_se = choices of e in s;  P_se = sum_{t in s} q_te
//   balance = coeff / S sum_s a_s sum_e c_se P_se,  a_s = E / (K n_s^2)
//   z       = z_coeff / n sum_t lse(x_t)^2,         n = tokens of all sequences
//   d/dx_tj = g0 coeff / S a_s w_tj (c_sj - sum_e c_se q_te)
//             + g1 z_coeff 2 lse_t / n softmax(x_t)_j,
//   w = q (softmax) or sigma (1 - sigma) / sum sigma (sigmoid)
//
// Bound by HBM: the forward reads the logits and the choices, the backward reads
// the logits and writes the gradient; no [T, E] score, map or score gradient exists.  8192 x
// 2304 fp32: forward 29 us (rows 21, of which a plain read of as many bytes takes 15; its second
// kernel 8), backward 30 (5.0 TB/s); 65536 x 512 bf16 34 and 29: there a row takes a warp 237
// instructions (284 backward), which fill two thirds of the issue slots, and the 21 warps of an SM
// do not cover each other's waits (for a fixed latency, shuffles and shared memory, the copies) in the
// rest; HBM is at 41 (54) %.
//
// Forward: a block takes a contiguous range of tokens, a warp a row at a time (two warps
// above 1152 experts).  A lane holds up to 36 logits, the next rows on their way, and the
// column sums of q of the rows that its team has seen; so a block leaves one row of column
// sums and one of counts for each sequence that its range touches ("slot": block + sequence,
// which rises by one or more from each to the next, so no two share one).  A
// second kernel adds a sequence's slots up in order; its last block to finish adds the
// blocks' shares.  No floating-point atomics: repeated calls give the same bits.  All sums are fp32:
// a team's rows (256 at most, one after the other) and a block's teams plain; a warp's slots with
// what each addition leaves over; then plain again, in trees, 32 warps' partial sums, the shares
// (a thread's one after the other) and the ranges' z.  Remainders carried through those as well cost
// 0.4 to 1.6 us and moved no result by a step that a test could see.
//
// Few warps to a row: what a row costs beside its values (two reductions, a barrier, its
// copies' addresses) is paid once a warp.  8192 x 2304 with six warps a row and 12 logits to a
// lane took 242 instructions a warp and row, 29 us.
//
// Backward: the same ranges; a team keeps its sequence's counts in registers.  They
// enter less the whole part of K n_s / E: a constant less changes nothing, since q sums to one,
// and leaves the difference c_sj - sum c q without the cancellation of two large numbers (in
// integers: a count above 2^24 is no fp32 number).
#include <atomic>
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"
#include "router_launch.cuh"
#include "router_rows.cuh"

namespace moe_router {
namespace {

constexpr int kMostWarps = 8;  // of a block

// By a lane's four-column pieces: a block's threads; the rows of a team under way (about 8 KB a
// warp, three rows at least: with one row ahead of 9 KB a team waited 2.4 us for each); registers a
// thread, which fix the blocks of an SM.
__host__ __device__ constexpr int threads_of(int nv) { return nv <= 6 ? 256 : 192; }
__host__ __device__ constexpr int ring_rows(int nv, int bytes) {
  const int n = 8192 / (nv * 32 * bytes);
  return n < 3 ? 3 : n > 8 ? 8 : n;
}
constexpr int registers_of(int nv) { return nv <= 4 ? 80 : nv <= 6 ? 128 : 168; }

// Shared memory of the rows under way.
__host__ __device__ constexpr int ring_bytes(bool vec, int nv, int bytes) {
  return vec ? ring_rows(nv, bytes) * nv * threads_of(nv) * bytes : 0;
}

struct BalanceArgs {
  const void* logits;
  const int32_t* choices;     // [T, ld_choices]
  const int32_t* seq;         // [S + 1] or NULL: one sequence of all T
  float* loss;                // [2]
  int32_t* counts;            // [S, E]
  float2* stats;              // [T] softmax: max, sum exp; sigmoid: sum sigma, lse
  float* slot_sums;           // [blocks + S, E]
  int32_t* slot_counts;       // [blocks + S, E]
  float* z_parts;             // [blocks]
  float* parts;               // [finish blocks]
  int* ticket;
  const float* grad_loss;     // [2]
  void* grad;                 // [T, E]
  long long ld_choices;
  int T, E, K, S;
  int rows;                   // tokens of a block
  int blocks;
  float coeff, z_coeff;
};

// Tokens [lo, hi) of sequence s, kept within [0, T].
__device__ __forceinline__ void sequence_range(const BalanceArgs& a, int s, int* lo, int* hi) {
  if (a.seq == nullptr) {
    *lo = 0;
    *hi = a.T;
    return;
  }
  *lo = min(max(a.seq[s], 0), a.T);
  *hi = min(max(a.seq[s + 1], *lo), a.T);
}

// The first sequence that ends behind token t (S: none), by one warp: 32 ends at a
// time.  Ends that are out of order give some sequence in [0, S].
__device__ __forceinline__ int first_sequence(const BalanceArgs& a, int t) {
  if (a.seq == nullptr) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.S;  // the answer is in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step + step - 1;  // the lane's last candidate
    const bool before = at < hi && a.seq[at + 1] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, before));
    const int next = lo + n * step;
    hi = min(hi, next + step - 1);
    lo = min(next, hi);
  }
  return lo;
}

// exp(x - max) of a row as 2^(x by - max by).  Where max log2 e could leave fp32's range no other
// logit lies within 2^76 of the largest: 1 for it and 0 for the others then is exp by any factor.
struct Shifted {
  float by, shift;
  __device__ __forceinline__ explicit Shifted(float top)
      : by(fabsf(top) < 0x1p100f ? kLog2e : 1.0f), shift(top * by) {}
  __device__ __forceinline__ float exp(float x) const { return ex2_approx(fmaf(x, by, -shift)); }
};

// Largest of a warp's values, in one instruction.
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Threads of a team of `warps` warps.
__device__ __forceinline__ void team_sync(int team, int warps) {
  if (warps > 1)
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

struct Team {
  int warps, team, teams, warp, lane;
  float* xch;  // [2][teams, warps][2]
  int flip;

  // A value summed over the team's warps (at most eight), in the same order in each.  Two
  // sets of cells in turn, so that one barrier a row is enough.
  __device__ __forceinline__ float sum(float x) {
    if (warps == 1) return x;
    float* const mine = xch + (flip * teams + team) * warps * 2;
    flip ^= 1;
    if (lane == 0) mine[warp] = x;
    team_sync(team, warps);
    const int w = lane & 7;
    return seg_sum<8>(w < warps ? mine[w] : 0.0f);
  }

  // Maxima and sums of exponentials relative to them, of the team's warps, as one.
  __device__ __forceinline__ void softmax_stats(float* m, float* s) {
    if (warps == 1) return;
    float* const mine = xch + (flip * teams + team) * warps * 2;
    flip ^= 1;
    if (lane == 0) {
      mine[2 * warp] = *m;
      mine[2 * warp + 1] = *s;
    }
    team_sync(team, warps);
    const int w = lane & 7;
    const bool in = w < warps;
    const float own = in ? mine[2 * w] : -INFINITY;
    const float top = warp_max(own);
    const float part = in ? mine[2 * w + 1] * ex2_approx((own - top) * kLog2e) : 0.0f;
    *m = top;
    *s = seg_sum<8>(part);
  }
};

__device__ __forceinline__ Team make_team(int warps, float* xch) {
  Team t;
  const int warp = threadIdx.x >> 5;
  t.warps = warps;
  t.team = warp / warps;
  t.teams = blockDim.x / (32 * warps);
  t.warp = warp - t.team * warps;
  t.lane = threadIdx.x & 31;
  t.xch = xch;
  t.flip = 0;
  return t;
}

// A lane's NV times four logits of a row: columns 4 (lane + 32 (warp + warps j)).
template <int NV>
struct Row {
  float v[NV][4];
};

__device__ __forceinline__ int column_of(const Team& t, int j) {
  return 4 * (t.lane + 32 * (t.warp + t.warps * j));
}

template <int DT, bool VEC, int NV>
__device__ __forceinline__ void load_row(const BalanceArgs& a, const Team& t, int row,
                                         Row<NV>* r) {
  const size_t at = static_cast<size_t>(row) * a.E;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column_of(t, j);
    if (c < a.E) load4<DT, VEC>(a.logits, at, c, a.E, r->v[j]);
  }
}

// Columns outside the row as minus infinity: their exponentials and sigmoids are zero and
// no maximum is theirs.
template <bool VEC, int NV>
__device__ __forceinline__ void blank_outside(const Team& t, int E, Row<NV>* r) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column_of(t, j);
    if (VEC ? c >= E : c + 4 > E) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (VEC || c + u >= E) r->v[j][u] = -INFINITY;
    }
  }
}

// The rows of the block's range on their way to the team, through places in shared memory
// that belong to the thread: the thread waits for its own copies, no barrier is needed,
// and several rows are under way where registers held one.  They are asked for before it
// is known which sequences they belong to.  (Rows that are not aligned are loaded when
// they are needed.)
template <int DT, bool VEC, int NV>
struct RowRing {
  static constexpr int kBytes = DT == DT_F32 ? 16 : 8;  // of four logits
  static constexpr int kRing = ring_rows(NV, kBytes);
  uint32_t base;          // the thread's first place
  int taken, asked;       // of the next row to take and to ask for, in rows
  const uint8_t* from;    // the thread's first four logits of the latter
  size_t stride;          // from one row of the team to the next, in bytes
  int row, hi;            // the latter's number

  __device__ __forceinline__ void request(const BalanceArgs& a, const Team& t) {
    if constexpr (VEC) {
      constexpr uint32_t kWidth = threads_of(NV) * kBytes;  // of a block's pieces j
      if (row < hi) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (column_of(t, j) < a.E)
            copy_async<kBytes>(base + (asked * NV + j) * kWidth, from + j * t.warps * (32 * kBytes));
      }
      row += t.teams;
      from += stride;
      if (++asked == kRing) asked = 0;
      copies_commit_group();
    }
  }

  __device__ __forceinline__ void begin(const BalanceArgs& a, const Team& t, void* smem, int lo,
                                        int stop) {
    base = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * kBytes;
    row = lo + t.team;
    hi = stop;
    stride = static_cast<size_t>(t.teams) * a.E * (kBytes / 4);
    from = static_cast<const uint8_t*>(a.logits) +
           (static_cast<size_t>(row) * a.E + column_of(t, 0)) * (kBytes / 4);
    taken = asked = 0;
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) request(a, t);
  }

  // The team's next row is one of padding.  Its copy is waited for like any other: the next
  // request goes to its place, and nothing orders two copies to one place that are both under way.
  __device__ __forceinline__ void skip(const BalanceArgs& a, const Team& t) {
    request(a, t);
    if constexpr (VEC) copies_wait_group<kRing - 1>();
    if (++taken == kRing) taken = 0;
  }

  // Row `at_row`, the team's next.
  __device__ __forceinline__ void take(const BalanceArgs& a, const Team& t, int at_row, Row<NV>* r) {
    if constexpr (VEC) {
      constexpr uint32_t kWidth = threads_of(NV) * kBytes;
      request(a, t);
      copies_wait_group<kRing - 1>();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t at = base + (taken * NV + j) * kWidth;
        if constexpr (DT == DT_F32) {
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(r->v[j][0]), "=f"(r->v[j][1]), "=f"(r->v[j][2]), "=f"(r->v[j][3])
                       : "r"(at) : "memory");
        } else {
          uint32_t x, y;
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at) : "memory");
          r->v[j][0] = __uint_as_float(x << 16);
          r->v[j][1] = __uint_as_float(x & 0xffff0000u);
          r->v[j][2] = __uint_as_float(y << 16);
          r->v[j][3] = __uint_as_float(y & 0xffff0000u);
        }
      }
      if (++taken == kRing) taken = 0;
    } else {
      load_row<DT, false>(a, t, at_row, r);
    }
    if (a.E < 128 * NV * t.warps) blank_outside<VEC>(t, a.E, r);
  }
};

template <int DT, bool VEC, int NV, int SF>
__global__ __launch_bounds__(threads_of(NV), NV <= 4 ? 3 : 2) void balance_fwd_kernel(
    const BalanceArgs a, int warps) {
  // the rows under way; [E] column sums; [E] counts
  extern __shared__ __align__(16) uint8_t dynamic_smem[];
  __shared__ float xch[2 * kMostWarps * 2];
  __shared__ float z_warp[kMostWarps];
  __shared__ int first_s;
  pdl_enter();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  Team t = make_team(warps, xch);
  const int t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  RowRing<DT, VEC, NV> ring;
  ring.begin(a, t, dynamic_smem, t0, t1);
  float* const block_sums = reinterpret_cast<float*>(
      dynamic_smem + ring_bytes(VEC, NV, ring.kBytes));
  int* const hist = reinterpret_cast<int*>(block_sums + a.E);
  if (threadIdx.x < 32) {
    const int s = first_sequence(a, t0);
    if (threadIdx.x == 0) first_s = s;
  }
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const bool want_z = a.z_coeff != 0.0f;
  float z = 0.0f;
  int row = t0 + t.team;  // the team's next
  for (int s = first_s, p = t0; s < a.S && p < t1; ++s) {
    int lo, hi;
    sequence_range(a, s, &lo, &hi);
    lo = max(lo, p);
    hi = min(hi, t1);
    if (lo >= t1) break;
    if (hi <= lo) continue;
    p = hi;
    for (; row < lo; row += t.teams) ring.skip(a, t);
    // ---- counts: the choices of the range's tokens, while the rows are on their way ---------
    const int32_t* const chosen = a.choices + lo * a.ld_choices;
    const int n = (hi - lo) * a.K;
    auto count = [&](int e) {
      if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) atomicAdd(hist + e, 1);
    };
    if (a.ld_choices == a.K) {
      constexpr int kAtOnce = 8;
      int i = threadIdx.x;
      for (; i + (kAtOnce - 1) * static_cast<int>(blockDim.x) < n; i += kAtOnce * blockDim.x) {
        int e[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) e[u] = __ldcs(chosen + i + u * blockDim.x);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) count(e[u]);
      }
#pragma unroll 4
      for (; i < n; i += blockDim.x) count(__ldcs(chosen + i));
    } else {
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int at = i / a.K;
        count(chosen[at * a.ld_choices + (i - at * a.K)]);
      }
    }
    // ---- column sums of q ------------------------------------------------------------------
    Row<NV> sums{};
    for (; row < hi; row += t.teams) {
      Row<NV> r;
      ring.take(a, t, row, &r);
      float top = -INFINITY, total = 0.0f, factor;
      if (SF == SF_SOFTMAX || want_z) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) top = fmaxf(top, r.v[j][u]);
        top = warp_max(top);
      }
      // (a warp without columns: its maximum is minus infinity, its sum zero)
      const float own = top;
      const Shifted from(top == -INFINITY ? 0.0f : top);
      if constexpr (SF == SF_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            r.v[j][u] = from.exp(r.v[j][u]);
            total += r.v[j][u];
          }
        total = seg_sum<32>(total);
        t.softmax_stats(&top, &total);
        factor = rcp_approx(total);
        if (t.warps > 1) factor *= ex2_approx((own - top) * kLog2e);
        if (t.warp == 0) {
          if (want_z) {
            const float lse = top + logf(total);
            z = fmaf(lse, lse, z);
          }
          if (t.lane == 0) a.stats[row] = make_float2(top, total);
        }
      } else {
        float lse = 0.0f;
        if (want_z) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) total += from.exp(r.v[j][u]);
          total = seg_sum<32>(total);
          t.softmax_stats(&top, &total);
          lse = top + logf(total);
          z = fmaf(lse, lse, z);
        }
        float norm = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            r.v[j][u] = sigmoid_f32(r.v[j][u]);
            norm += r.v[j][u];
          }
        norm = t.sum(seg_sum<32>(norm));
        factor = rcp_approx(norm);
        if (t.warp == 0 && t.lane == 0) a.stats[row] = make_float2(norm, lse);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) sums.v[j][u] = fmaf(r.v[j][u], factor, sums.v[j][u]);
    }
    // ---- the slot of this block and sequence: the sums of the teams that had a row of it, one
    // after the other from the first row's ----------------------------------------------------
    const int adding = min(hi - lo, t.teams);
    const int place = (t.team + t.teams - (lo - t0) % t.teams) % t.teams;
    for (int w = 0; w < adding; ++w) {
      if (place == w) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = column_of(t, j);
          if constexpr (VEC) {
            float4* const to = reinterpret_cast<float4*>(block_sums + c);
            if (c < a.E) {
              const float4 v = w == 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *to;
              *to = make_float4(v.x + sums.v[j][0], v.y + sums.v[j][1], v.z + sums.v[j][2],
                                v.w + sums.v[j][3]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (c + u < a.E)
                block_sums[c + u] = (w == 0 ? 0.0f : block_sums[c + u]) + sums.v[j][u];
          }
        }
      }
      __syncthreads();
    }
    const size_t slot = (static_cast<size_t>(blockIdx.x) + s) * a.E;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
      a.slot_sums[slot + e] = block_sums[e];
      a.slot_counts[slot + e] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
  }
  copies_wait_group<0>();  // (rows of padding that nobody took)
  // every lane of a team has its rows' z: the first of each counts
  if (t.lane == 0) z_warp[threadIdx.x >> 5] = t.warp == 0 ? z : 0.0f;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) v += z_warp[w];
    a.z_parts[blockIdx.x] = v;
  }
}

// Slots above which a sequence's are added up by all warps of a block.
constexpr int kLongSlots = 32;

// Adds up each sequence's slots, then counts times sums, and the last block the whole.  An item is
// a sequence and 32 WIDE columns: GROUPS warps take every GROUPS-th slot each.  With few
// slots to a sequence on average a warp takes an item by itself, 128 columns wide, and the block's
// warps together those of a sequence of many: by one warp a forward of 65536 tokens, 64 experts, one
// long sequence among 63 short ones took 99 us, together 42 (64 equal ones 17.6 and 18.2).
template <int GROUPS, int WIDE, int WARPS>
__global__ __launch_bounds__(32 * WARPS) void balance_finish_kernel(const BalanceArgs a) {
  constexpr int kCols = 32 * WIDE, kItems = WARPS / GROUPS;
  static_assert(GROUPS == 1 || (GROUPS == 32 && WARPS == 32 && WIDE == 1), "a warp a column");
  constexpr int kParts = GROUPS == 1 ? WARPS : GROUPS;
  __shared__ float sums[kParts][kCols + 1], left[GROUPS == 1 ? WARPS : 1][kCols + 1];
  __shared__ int counts[kParts][kCols + 1];
  __shared__ int many[2][WARPS];  // GROUPS 1: is the warp's item one of many slots?
  __shared__ float shared[2][WARPS];
  __shared__ int last;
  pdl_enter();
  const int tiles = (a.E + kCols - 1) / kCols;
  const long long items = static_cast<long long>(tiles) * a.S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp % GROUPS;
  const bool vec = WIDE == 4 && (a.E & 3) == 0;
  float share = 0.0f;
  struct Item {
    int s, c, tokens, b0, b1;  // the lane's first column; the sequence's slots
  };
  auto item_of = [&](long long item) {
    Item t;
    t.s = static_cast<int>(item / tiles);
    t.c = static_cast<int>(item - static_cast<long long>(t.s) * tiles) * kCols + WIDE * lane;
    int lo, hi;
    sequence_range(a, t.s, &lo, &hi);
    t.tokens = hi - lo;
    t.b0 = lo / a.rows;
    t.b1 = hi > lo ? (hi - 1) / a.rows : t.b0 - 1;
    return t;
  };
  // fp32 sums with what each addition left over (a long batch has 100000 slots)
  float v[WIDE], rest[WIDE];
  int n[WIDE];
  auto add = [&](int u, float x, int k) {
    const float y = x - rest[u], next = v[u] + y;
    rest[u] = (next - v[u]) - y;
    v[u] = next;
    n[u] += k;
  };
  // every step-th slot of an item from slot `from`
  auto add_slots = [&](const Item& t, int from, int step) {
#pragma unroll
    for (int u = 0; u < WIDE; ++u) {
      v[u] = rest[u] = 0.0f;
      n[u] = 0;
    }
    if (vec) {
      if (t.c < a.E) {
#pragma unroll 4
        for (int b = from; b <= t.b1; b += step) {
          const size_t at = (static_cast<size_t>(b) + t.s) * a.E + t.c;
          const float4 x = __ldcg(reinterpret_cast<const float4*>(a.slot_sums + at));
          const int4 k = __ldcg(reinterpret_cast<const int4*>(a.slot_counts + at));
          add(0, x.x, k.x);
          if constexpr (WIDE == 4) {
            add(1, x.y, k.y);
            add(2, x.z, k.z);
            add(3, x.w, k.w);
          }
        }
      }
    } else {
#pragma unroll 8
      for (int b = from; b <= t.b1; b += step) {
        const size_t at = (static_cast<size_t>(b) + t.s) * a.E + t.c;
#pragma unroll
        for (int u = 0; u < WIDE; ++u)
          if (t.c + u < a.E) add(u, __ldcg(a.slot_sums + at + u), __ldcg(a.slot_counts + at + u));
      }
    }
  };
  // c_se P_se / n_s^2 (the factors that all share come last)
  auto finish = [&](const Item& t, int e, float p, int k) {
    const float by_tokens = 1.0f / static_cast<float>(max(t.tokens, 1));
    a.counts[static_cast<size_t>(t.s) * a.E + e] = k;
    share = fmaf(static_cast<float>(k) * by_tokens, p * by_tokens, share);
  };
  int flip = 0;
  const bool any_long = a.blocks > kLongSlots;
  // (neighbours in different blocks: a long sequence's columns)
  for (long long first = blockIdx.x; first < items;
       first += static_cast<long long>(gridDim.x) * kItems, flip ^= 1) {
    if constexpr (GROUPS > 1) {  // warp w adds up column w of the item
      const Item t = item_of(first);
      add_slots(t, t.b0 + group, GROUPS);
      sums[group][lane] = v[0];
      counts[group][lane] = n[0];
      __syncthreads();
      const float p = seg_sum<32>(sums[lane][warp]);
      const int k = __reduce_add_sync(0xffffffffu, counts[lane][warp]);
      const int e = t.c - lane + warp;
      if (lane == 0 && e < a.E) finish(t, e, p, k);
      __syncthreads();
    } else {
      Item t{};
      const auto item = [&](int w) { return first + static_cast<long long>(gridDim.x) * w; };
      const bool mine = item(warp) < items;
      if (mine) t = item_of(item(warp));
      const bool long_one = mine && t.b1 - t.b0 >= kLongSlots;
      if (lane == 0 && any_long) many[flip][warp] = long_one;
      if (mine && !long_one) {
        add_slots(t, t.b0, 1);
#pragma unroll
        for (int u = 0; u < WIDE; ++u)
          if (t.c + u < a.E) finish(t, t.c + u, v[u], n[u]);
      }
      if (!any_long) continue;
      __syncthreads();  // (two sets of flags in turn: one barrier a round)
      unsigned waiting = __ballot_sync(0xffffffffu, lane < WARPS && many[flip][lane % WARPS]);
      for (; waiting != 0; waiting &= waiting - 1) {  // the same in all threads
        const int w = __ffs(waiting) - 1;
        const Item whole = item_of(item(w));
        add_slots(whole, whole.b0 + warp, WARPS);
#pragma unroll
        for (int u = 0; u < WIDE; ++u) {
          sums[warp][WIDE * lane + u] = v[u];
          left[warp][WIDE * lane + u] = rest[u];
          counts[warp][WIDE * lane + u] = n[u];
        }
        __syncthreads();
        if (warp == w) {
          for (int g = 0; g < WARPS; ++g) {
            if (g == warp) continue;
#pragma unroll
            for (int u = 0; u < WIDE; ++u) {
              add(u, sums[g][WIDE * lane + u], counts[g][WIDE * lane + u]);
              add(u, -left[g][WIDE * lane + u], 0);
            }
          }
#pragma unroll
          for (int u = 0; u < WIDE; ++u)
            if (whole.c + u < a.E) finish(whole, whole.c + u, v[u], n[u]);
        }
        __syncthreads();
      }
    }
  }
  share = seg_sum<32>(share);
  if (lane == 0) shared[0][warp] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < WARPS; ++w) share += shared[0][w];
    a.parts[blockIdx.x] = share;
    __threadfence();
    last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // the blocks' shares and the ranges' z: each thread its own few, then in a fixed order
  float balance = 0.0f, z = 0.0f;
  for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += 32 * WARPS)
    balance += __ldcg(a.parts + b);
  if (a.z_coeff != 0.0f)
    for (int b = threadIdx.x; b < a.blocks; b += 32 * WARPS) z += __ldcg(a.z_parts + b);
  balance = seg_sum<32>(balance);
  z = seg_sum<32>(z);
  if (lane == 0) {
    shared[0][warp] = balance;
    shared[1][warp] = z;
  }
  __syncthreads();
  if (warp == 0) {
    balance = seg_sum<32>(lane < WARPS ? shared[0][lane] : 0.0f);
    z = seg_sum<32>(lane < WARPS ? shared[1][lane] : 0.0f);
    int lo, hi, unused;
    sequence_range(a, 0, &lo, &unused);
    sequence_range(a, a.S - 1, &unused, &hi);
    if (lane == 0) {
      a.loss[0] = balance * (a.coeff * a.E / a.K / a.S);
      a.loss[1] = a.z_coeff == 0.0f ? 0.0f : z * (a.z_coeff / max(hi - lo, 1));
    }
  }
}

template <int DT, bool VEC, int NV, int SF>
__global__ __launch_bounds__(threads_of(NV), NV <= 4 ? 3 : 2) void balance_bwd_kernel(
    const BalanceArgs a, int warps) {
  extern __shared__ __align__(16) uint8_t dynamic_smem[];  // the rows under way
  __shared__ float xch[2 * kMostWarps * 2];
  __shared__ int first_s;
  pdl_enter();
  Team t = make_team(warps, xch);
  const int t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  RowRing<DT, VEC, NV> ring;
  ring.begin(a, t, dynamic_smem, t0, t1);
  if (threadIdx.x < 32) {
    const int s = first_sequence(a, t0);
    if (threadIdx.x == 0) first_s = s;
  }
  __syncthreads();
  int whole_lo, whole_hi, unused;
  sequence_range(a, 0, &whole_lo, &unused);
  sequence_range(a, a.S - 1, &unused, &whole_hi);
  const float by_balance = a.grad_loss[0] * a.coeff / static_cast<float>(a.S);
  const float by_z = a.z_coeff == 0.0f
                         ? 0.0f
                         : a.grad_loss[1] * a.z_coeff * 2.0f /
                               static_cast<float>(max(whole_hi - whole_lo, 1));
  int row = t0 + t.team;  // the team's next
  // rows of no sequence: zeros
  auto clear = [&](int to) {
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (; row < to; row += t.teams) {
      ring.skip(a, t);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column_of(t, j);
        if (c < a.E) store4<DT, VEC>(a.grad, static_cast<size_t>(row) * a.E, c, a.E, none);
      }
    }
  };
  for (int s = first_s, p = t0; s < a.S && p < t1; ++s) {
    int lo, hi;
    sequence_range(a, s, &lo, &hi);
    const int all = hi - lo;
    const float tokens = static_cast<float>(all);
    lo = max(lo, p);
    hi = min(hi, t1);
    if (lo >= t1) break;
    if (hi <= lo) continue;
    p = hi;
    clear(lo);
    const float scale = by_balance * (static_cast<float>(a.E) / a.K) / tokens / tokens;
    const int mean = static_cast<int>(static_cast<long long>(all) * a.K / a.E);
    Row<NV> c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = column_of(t, j);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        c.v[j][u] = col + u < a.E
                        ? static_cast<float>(a.counts[static_cast<size_t>(s) * a.E + col + u] - mean)
                        : 0.0f;
    }
    float2 next_st = row < hi ? a.stats[row] : make_float2(0.0f, 1.0f);
    for (; row < hi; row += t.teams) {
      const float2 st = next_st;
      if (row + t.teams < hi) next_st = a.stats[row + t.teams];
      Row<NV> r;
      ring.take(a, t, row, &r);
      const float inv = rcp_approx(SF == SF_SOFTMAX ? st.y : st.x);
      const Shifted from(SF == SF_SOFTMAX ? st.x : st.y);
      float z = 0.0f;
      if (by_z != 0.0f) z = by_z * (SF == SF_SOFTMAX ? st.x + logf(st.y) : st.y);
      // r becomes exp(x - max), q times the row's sum; sigmoid: sigma(-|x|) with the sign of
      // x, so that sigma and 1 - sigma are both without cancellation (x by itself for z)
      Row<NV> x;
      if (SF != SF_SOFTMAX) x = r;
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if constexpr (SF == SF_SOFTMAX) {
            r.v[j][u] = from.exp(r.v[j][u]);
            dot = fmaf(c.v[j][u], r.v[j][u], dot);
          } else {
            const float e = ex2_approx(-fabsf(r.v[j][u]) * kLog2e);
            const float small = e * rcp_approx(1.0f + e);
            dot = fmaf(c.v[j][u], r.v[j][u] < 0.0f ? small : 1.0f - small, dot);
            r.v[j][u] = small;
          }
        }
      dot = t.sum(seg_sum<32>(dot)) * inv;
      // softmax: q (scale (c - dot) + z) = exp (by c + less); sigmoid alike, z apart
      const float by = scale * inv, less = SF == SF_SOFTMAX ? inv * (z - scale * dot) : -by * dot;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = column_of(t, j);
        float g[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float w = SF == SF_SOFTMAX ? r.v[j][u] : fmaf(-r.v[j][u], r.v[j][u], r.v[j][u]);
          g[u] = w * fmaf(by, c.v[j][u], less);
          if (SF != SF_SOFTMAX && by_z != 0.0f) g[u] = fmaf(z, from.exp(x.v[j][u]), g[u]);
        }
        if (col < a.E) store4<DT, VEC>(a.grad, static_cast<size_t>(row) * a.E, col, a.E, g);
      }
    }
  }
  clear(t1);
  copies_wait_group<0>();
}

// ---- host ------------------------------------------------------------------------
// Warps of a row and times four columns of a lane: the fewest warps, then the fewest pieces
// that are built.
struct Shape {
  int warps, nv, teams;
};

Shape shape_of(int E) {
  const int pieces = (E + 127) / 128;  // at most 18
  const int warps = pieces <= 9 ? 1 : 2, least = (pieces + warps - 1) / warps;
  const int nv = least <= 2 ? least : least <= 4 ? 4 : least <= 6 ? 6 : 9;
  return Shape{warps, nv, threads_of(nv) / 32 / warps};
}

size_t smem_of(int E, const Shape& sh, bool vec, int bytes, bool forward) {
  const size_t ring = ring_bytes(vec, sh.nv, bytes);
  return forward ? ring + static_cast<size_t>(E) * 8 : ring;
}

// Blocks that an SM holds, by registers and shared memory: a block more than that would run
// by itself behind the others.
constexpr int kMostPerSm = 3;

int blocks_per_sm(const Shape& sh, size_t smem) {
  const int by_registers = 65536 / (registers_of(sh.nv) * threads_of(sh.nv));
  const int by_memory = static_cast<int>(227 * 1024 / (smem + 2048));
  const int n = by_registers < by_memory ? by_registers : by_memory;
  return n < 1 ? 1 : n > kMostPerSm ? kMostPerSm : n;
}

// Tokens of a block: `per_sm` blocks on each of 152 SMs, two rows a team at least, and 256 at
// most, since a team adds its rows up one after the other in fp32.  A function of the
// sizes alone, so that sums have the same order on every GPU.
constexpr int kMostRows = 256;

int rows_of(int T, int teams, int per_sm) {
  const int blocks = 152 * per_sm;
  const int each = ((T + blocks - 1) / blocks + teams - 1) / teams;  // of a team
  return teams * (each < 2 ? 2 : each > kMostRows ? kMostRows : each);
}

constexpr int kFinishBlocks = 608;

int blocks_of(int T, int rows) { return T == 0 ? 1 : (T + rows - 1) / rows; }

struct Workspace {
  size_t slots, z, parts, ticket, bytes;
};

Workspace workspace_of(int T, int E, int S) {
  const Shape sh = shape_of(E);
  const int blocks = blocks_of(T, rows_of(T, sh.teams, kMostPerSm));
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  Workspace w;
  w.slots = up((static_cast<size_t>(blocks) + S) * E * 4);
  w.z = 2 * w.slots;
  w.parts = w.z + up(static_cast<size_t>(blocks) * 4);
  w.ticket = w.parts + up(kFinishBlocks * 4);
  w.bytes = w.ticket + 256;
  return w;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check(int dtype, int T, int E, int K, int S, bool packed, int score_func) {
  if (dtype != MR_F32 && dtype != MR_BF16) return MR_ERR_INVALID;
  if (score_func != MR_SOFTMAX && score_func != MR_SIGMOID) return MR_ERR_INVALID;
  if (T < 0 || E < 1 || K < 1 || K > E || S < 1) return MR_ERR_INVALID;
  if (S > (T > 1 ? T : 1) || (!packed && S != 1)) return MR_ERR_INVALID;
  if (static_cast<long long>(T) * E > INT_MAX || static_cast<long long>(T) * K > INT_MAX)
    return MR_ERR_INVALID;
  if (E > MR_MAX_EXPERTS || K > MR_MAX_TOPK) return MR_ERR_UNSUPPORTED;
  if (T > MR_MAX_ROWS) return MR_ERR_UNSUPPORTED;  // (a block's rows end behind T, still as an int)
  return MR_OK;
}

template <int DT, bool VEC, int NV, int SF, bool FWD>
cudaError_t launch_rows(const BalanceArgs& a, dim3 grid, dim3 block, size_t smem, int warps,
                        cudaStream_t st) {
  static std::atomic<int> granted[kSmemDevs];
  const auto kern = FWD ? balance_fwd_kernel<DT, VEC, NV, SF> : balance_bwd_kernel<DT, VEC, NV, SF>;
  // above 40 KB the kernel's own arrays may take it past the default of 48 KB
  const size_t limit = smem > 40 * 1024 && smem <= 48 * 1024 ? 48 * 1024 + 16 : smem;
  const cudaError_t e = allow_smem(kern, limit, granted);
  return e == cudaSuccess ? launch_kernel(kern, grid, block, smem, st, a, warps) : e;
}

template <int DT, bool VEC, int SF, bool FWD>
cudaError_t launch_nv(const BalanceArgs& a, const Shape& sh, cudaStream_t st) {
  const dim3 grid(a.blocks), block(threads_of(sh.nv));
  const size_t smem = smem_of(a.E, sh, VEC, DT == DT_F32 ? 16 : 8, FWD);
  switch (sh.nv) {
    case 1: return launch_rows<DT, VEC, 1, SF, FWD>(a, grid, block, smem, sh.warps, st);
    case 2: return launch_rows<DT, VEC, 2, SF, FWD>(a, grid, block, smem, sh.warps, st);
    case 4: return launch_rows<DT, VEC, 4, SF, FWD>(a, grid, block, smem, sh.warps, st);
    case 6: return launch_rows<DT, VEC, 6, SF, FWD>(a, grid, block, smem, sh.warps, st);
    default: return launch_rows<DT, VEC, 9, SF, FWD>(a, grid, block, smem, sh.warps, st);
  }
}

// Slots to a sequence up to which a warp adds them up by itself (512 sequences of 16 tokens, 2304
// experts: 32 warps to each took 100 us).
constexpr int kFewSlots = 8;

cudaError_t launch_finish(const BalanceArgs& a, cudaStream_t st) {
  const auto grid = [](long long items, int each, int most) {
    const long long n = (items + each - 1) / each;
    return dim3(static_cast<unsigned>(n < most ? n : most));
  };
  if (a.blocks / a.S + 1 <= kFewSlots)
    return launch_kernel(balance_finish_kernel<1, 4, 8>,
                         grid(static_cast<long long>((a.E + 127) / 128) * a.S, 8, kFinishBlocks),
                         dim3(256), 0, st, a);
  return launch_kernel(balance_finish_kernel<32, 1, 32>,
                       grid(static_cast<long long>((a.E + 31) / 32) * a.S, 1, kFinishBlocks),
                       dim3(1024), 0, st, a);
}

template <bool FWD>
cudaError_t launch_balance(const BalanceArgs& a, int dtype, int sf, bool vec, const Shape& sh,
                           cudaStream_t st) {
  if (dtype == MR_F32) {
    if (sf == MR_SOFTMAX)
      return vec ? launch_nv<DT_F32, true, SF_SOFTMAX, FWD>(a, sh, st)
                 : launch_nv<DT_F32, false, SF_SOFTMAX, FWD>(a, sh, st);
    return vec ? launch_nv<DT_F32, true, SF_SIGMOID, FWD>(a, sh, st)
               : launch_nv<DT_F32, false, SF_SIGMOID, FWD>(a, sh, st);
  }
  if (sf == MR_SOFTMAX)
    return vec ? launch_nv<DT_BF16, true, SF_SOFTMAX, FWD>(a, sh, st)
               : launch_nv<DT_BF16, false, SF_SOFTMAX, FWD>(a, sh, st);
  return vec ? launch_nv<DT_BF16, true, SF_SIGMOID, FWD>(a, sh, st)
             : launch_nv<DT_BF16, false, SF_SIGMOID, FWD>(a, sh, st);
}

}  // namespace
}  // namespace moe_router

using namespace moe_router;

extern "C" {

size_t router_balance_loss_workspace_bytes(int T, int E, int S) {
  if (T < 0 || T > MR_MAX_ROWS || E < 1 || E > MR_MAX_EXPERTS || S < 1) return 0;
  return workspace_of(T, E, S).bytes;
}

int router_balance_loss_fwd(const void* logits, mr_dtype dtype, const int32_t* topk_indices,
                            int ld_indices, const int32_t* seq_offsets, int T, int E, int K, int S,
                            mr_score_func score_func, float coeff, float z_coeff, float* loss,
                            int32_t* tokens_per_expert, float* row_stats, void* workspace,
                            size_t workspace_bytes, mr_stream_t stream) {
  const int rc = check(dtype, T, E, K, S, seq_offsets != nullptr, score_func);
  if (rc != MR_OK) return rc;
  if (ld_indices < K || loss == nullptr || tokens_per_expert == nullptr) return MR_ERR_INVALID;
  if (T > 0 && (logits == nullptr || topk_indices == nullptr || row_stats == nullptr))
    return MR_ERR_INVALID;
  const Workspace w = workspace_of(T, E, S);
  if (workspace == nullptr || workspace_bytes < w.bytes || !aligned(workspace, 16) ||
      !aligned(row_stats, 8))
    return MR_ERR_INVALID;
  const Shape sh = shape_of(E);
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  BalanceArgs a{};
  a.logits = logits;
  a.choices = topk_indices;
  a.seq = seq_offsets;
  a.loss = loss;
  a.counts = tokens_per_expert;
  a.stats = reinterpret_cast<float2*>(row_stats);
  a.slot_sums = reinterpret_cast<float*>(base);
  a.slot_counts = reinterpret_cast<int32_t*>(base + w.slots);
  a.z_parts = reinterpret_cast<float*>(base + w.z);
  a.parts = reinterpret_cast<float*>(base + w.parts);
  a.ticket = reinterpret_cast<int*>(base + w.ticket);
  a.ld_choices = ld_indices;
  a.T = T; a.E = E; a.K = K; a.S = S;
  const int piece = dtype == MR_F32 ? 16 : 8;
  const bool vec = E % 4 == 0 && aligned(logits, piece);
  a.rows = rows_of(T, sh.teams, blocks_per_sm(sh, smem_of(E, sh, vec, piece, true)));
  a.blocks = blocks_of(T, a.rows);
  a.coeff = coeff;
  a.z_coeff = z_coeff;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_balance<true>(a, dtype, score_func, vec, sh, st) != cudaSuccess) return MR_ERR_CUDA;
  return launch_finish(a, st) == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int router_balance_loss_bwd(const float* grad_loss, const void* logits, mr_dtype dtype,
                            const int32_t* tokens_per_expert, const float* row_stats,
                            const int32_t* seq_offsets, int T, int E, int K, int S,
                            mr_score_func score_func, float coeff, float z_coeff,
                            void* grad_logits, mr_stream_t stream) {
  const int rc = check(dtype, T, E, K, S, seq_offsets != nullptr, score_func);
  if (rc != MR_OK) return rc;
  if (T == 0) return MR_OK;
  if (grad_loss == nullptr || logits == nullptr || tokens_per_expert == nullptr ||
      row_stats == nullptr || grad_logits == nullptr || !aligned(row_stats, 8))
    return MR_ERR_INVALID;
  const Shape sh = shape_of(E);
  BalanceArgs a{};
  a.logits = logits;
  a.seq = seq_offsets;
  a.counts = const_cast<int32_t*>(tokens_per_expert);
  a.stats = reinterpret_cast<float2*>(const_cast<float*>(row_stats));
  a.grad_loss = grad_loss;
  a.grad = grad_logits;
  a.T = T; a.E = E; a.K = K; a.S = S;
  const int piece = dtype == MR_F32 ? 16 : 8;
  const bool vec = E % 4 == 0 && aligned(logits, piece) && aligned(grad_logits, piece);
  a.rows = rows_of(T, sh.teams, blocks_per_sm(sh, smem_of(E, sh, vec, piece, false)));
  a.blocks = blocks_of(T, a.rows);
  a.coeff = coeff;
  a.z_coeff = z_coeff;
  return launch_balance<false>(a, dtype, score_func, vec, sh,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MR_OK
             : MR_ERR_CUDA;
}

}  // extern "C"
