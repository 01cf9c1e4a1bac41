// Products grouped by expert on 8-bit integers with a scale for each row and each
// output channel, on the tensor cores:
//
//   out[p, n] = x_scales[row(p)] weight_scales[e, n] sum_d weight[e, n, d] x[row(p), d]
//
// sm_103a's tcgen05 has no integer products.  An 8-bit integer is exact in fp16, a product
// of two in fp32, and a sum of 896 of them (seven stages) stays below 2^24: so the operands are
// widened to fp16 on their way to shared memory and multiplied at the 16-bit rate.  A fp32 output
// is summed in segments of at most 896 terms, each exact; a bf16 output is one sum, exact
// while it stays below 2^24 (and off by about 2^-30 of its value a term above that).
//
// The tiles and their order are those of router_experts_tc.cu's forward: 128 or 256 weight
// rows by up to 128 or 256 of the expert's rows, one CTA or a pair.  Stages hold 128 columns;
// two groups of eight warps load alternate ones: eight lanes a row (whole lines: a request of
// 64-byte pieces took 11 wavefronts of the load pipe), four rows of both operands a thread, each
// piece asked for two stages ahead in the registers that its predecessor has just left, widened
// and stored in the layout that the tensor cores read.  One group's stores (half of the
// shared memory's time) pass while the other fetches and waits: with all sixteen warps on
// each stage, 8192 tokens, 8 experts, 4096 x 4096 took 390 us where this took 365.
//
// In a pair each CTA's loading warps arrive on its own barrier, and a warp of the second CTA that
// waits there passes that on to the leader's by an arrival with release semantics of cluster
// scope: what it has seen is then ordered before the products.  Such an arrival holds its warp for
// about 1500 cycles, so each stage has a warp of its own.  (The completion of an asynchronous store
// is ordered behind that store alone, not behind what its thread has seen: 8192 tokens, 8 experts
// took 355 us that way, and would not have been sound.)  The second CTA's storing warps hand
// their accumulators back in the same way, through a fourth.
//
// A tile's lookup and its scales' loads are made a tile ahead: made where they were needed they
// took 5000 of the 10400 cycles of a tile with 43 rows and four stages.
//
// Bound by the load pipe and shared memory: a stage's loads, widened stores and the tensor
// cores' reads are 1280 cycles of its 128 bytes a cycle, the products 1024; a stage takes 1750 (1600
// without the second CTA's arrivals, whose latency three stages do not hide).
// 8192 tokens, 8 experts, 4096 x 4096 388 us (1417 TFLOP/s), 64 experts of 2048 x 2048 241, 256
// experts of 2048 -> 1024 294; 1003 tokens, 512 experts, 504 -> 1000, fp32 out 118 (3.1 TB/s).
#include <atomic>

#include "router_experts_tiles.cuh"
#include "router_widen.cuh"

namespace moe_router {
namespace {

constexpr int kLoaders = 8;  // warps of each of the two groups
constexpr int kThreads = 32 * (8 + 2 * kLoaders);
constexpr int kStages = 3;
constexpr int kWide = 128;   // columns of a stage: two of the layout's 128-byte rows in fp16
constexpr int kOwn = 4;      // rows of each operand that a thread loads, 32 apart
constexpr int kMostStages = 7;  // of a fp32 output's sum
constexpr int kRowsA = 128;  // weight rows of a CTA
constexpr int kRowsB = 128;  // most rows of x of a CTA
constexpr int kHalf = 128 * 128;  // 64 columns of an operand
constexpr int kBytesA = 2 * kHalf;
constexpr int kBytesB = 2 * kHalf;
constexpr int kStageBytes = kBytesA + kBytesB;
constexpr int kSmem = kStages * kStageBytes + 1024;  // stages start on 1024 bytes

template <int CG>
struct Shape {
  static constexpr int kTileA = kRowsA * CG;
  static constexpr int kTileB = kRowsB * CG;
  static constexpr int kRound = 16 * CG;
  static constexpr uint32_t kColumns = 2 * kTileB;  // two accumulators
};

struct W8TcArgs {
  TcArgs t;
  const int8_t* x;
  const int8_t* w;
  const float* x_scales;
  const float* w_scales;
  uint32_t inv_a;  // inverse_of the weight's slices
  int least;       // rows of an expert, below which it is left to the few-rows kernel
};

// 16 consecutive bytes of a row, VB bytes an access, of which `left` (a multiple of VB, or
// more than 16) exist; zeros behind them.
template <int VB>
__device__ __forceinline__ uint4 load_piece(const int8_t* p, int left) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (VB == 16) {
    if (left > 0) v = __ldg(reinterpret_cast<const uint4*>(p));
  } else if constexpr (VB == 8) {
    if (left > 0) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
      v.x = a.x;
      v.y = a.y;
    }
    if (left > 8) {
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(p) + 1);
      v.z = b.x;
      v.w = b.y;
    }
  } else if constexpr (VB == 4) {
    const unsigned* q = reinterpret_cast<const unsigned*>(p);
    if (left > 0) v.x = __ldg(q);
    if (left > 4) v.y = __ldg(q + 1);
    if (left > 8) v.z = __ldg(q + 2);
    if (left > 12) v.w = __ldg(q + 3);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const uint8_t* q = reinterpret_cast<const uint8_t*>(p);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) w[i >> 2] |= static_cast<uint32_t>(__ldg(q + i)) << (8 * (i & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Eight bytes, widened, to one 16-byte piece of shared memory.
__device__ __forceinline__ void store_wide(uint32_t at, uint32_t a, uint32_t b) {
  const uint4 v = widen_eight(a, b);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w) : "memory");
}

// Waits for data that the other CTA of the pair has published.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait_cluster(const Waiter& w, uint64_t* bar, uint32_t parity) {
  if (try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (try_wait_cluster(bar, parity)) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) break;
  }
  *reinterpret_cast<volatile int*>(w.gave_up) = 1;
  atomicExch(w.status, kDeviceWaitTimeout);
  return false;
}

// find_tile by a whole warp: 32 probes at a time, and divisions only for an expert of
// several row tiles.
template <typename S>
__device__ __forceinline__ Tile find_tile_by_warp(const TcArgs& g, const int* prefix,
                                                  const int* offs, int tile, int slices_a,
                                                  uint32_t inv_a) {
  const int lane = threadIdx.x & 31;
  int q = static_cast<int>(__umulhi(static_cast<uint32_t>(tile), inv_a));  // tile / slices_a, or one less
  if (tile - q * slices_a >= slices_a) ++q;
  int lo = 0, width = g.E;  // prefix[lo] <= q < prefix[lo + width]
  while (width > 1) {
    const int step = (width + 31) / 32;
    const bool below = lane * step < width && prefix[lo + lane * step] <= q;
    const int n = __popc(__ballot_sync(0xffffffffu, below)) - 1;
    lo += n * step;
    width = min(step, width - n * step);
  }
  Tile t;
  t.e = lo;
  t.b0 = 0;
  const int first = prefix[lo], of = prefix[lo + 1] - first;
  const int from = offs[lo], to = max(offs[lo + 1], from);
  int a = tile - first * slices_a, r = 0, each = to - from;
  if (of > 1) {
    const int at = a;
    a = at / of;  // one slice of the weight, all row tiles, then the next
    r = at - a * of;
    each = (each + of - 1) / of;
  }
  each = (each + S::kRound - 1) / S::kRound * S::kRound;
  t.a0 = a * S::kTileA;
  t.start = from + r * each;
  t.cnt = min(each, to - t.start);
  return t;
}

template <int CG, int VB, bool F32>
__global__ __launch_bounds__(kThreads, 1) void expert_matmul_w8_kernel(const W8TcArgs args) {
  using S = Shape<CG>;
  const TcArgs& g = args.t;
  extern __shared__ uint8_t dynamic_smem[];
  __shared__ __align__(8) uint64_t full[kStages], peer[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t done[2], drained[2], read[2];
  __shared__ uint32_t tmem_at;
  __shared__ int gave_up;
  __shared__ int tmp[33];
  __shared__ int prefix[MR_MAX_EXPERTS + 1];
  __shared__ int offs[MR_MAX_EXPERTS + 1];  // the offsets, clamped to [0, P]
  __shared__ __align__(16) float row_scales[4][S::kTileB];  // of each storing warp

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const uint32_t stages_at = (smem_addr(dynamic_smem) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&peer[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&drained[i], 4 + (CG - 1));  // one arrival per storing warp, one for the second CTA's
      mbar_init(&read[i], 4);                // the second CTA's storing warps
    }
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<CG>(&tmem_at, S::kColumns);
  pdl_enter();
  for (int e = threadIdx.x; e <= g.E; e += blockDim.x) offs[e] = min(max(g.offsets[e], 0), g.P);
  const int slices_a = (g.N + S::kTileA - 1) / S::kTileA;
  const int tiles =
      expert_tile_prefix(g.offsets, g.E, g.P, S::kTileB, prefix, tmp, args.least) * slices_a;
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const Waiter wait{&gave_up, g.status};
  const int first = static_cast<int>(blockIdx.x) / CG, step = static_cast<int>(gridDim.x) / CG;
  const auto find = [&](int tile) {
    return find_tile_by_warp<S>(g, prefix, offs, tile, slices_a, args.inv_a);
  };
  const int slices = (g.D + kWide - 1) / kWide;

  if (warp >= 8) {
    // ---- loads -----------------------------------------------------------------
    const int group = (warp - 8) / kLoaders;
    const int row = ((static_cast<int>(threadIdx.x) - 256) & (32 * kLoaders - 1)) >> 3;
    const int piece = threadIdx.x & 7;  // of the eight of a row and stage
    const size_t far = static_cast<size_t>(32) * g.D;
    // the cursor: tile li, stage ls of it, this thread's rows row + 32 h of both operands
    int li = first, ls = group;
    const int8_t* pa = nullptr;
    int source[kOwn];     // rows of x, -1: none
    uint32_t has_a = 0, wanted = 0;  // by h: the weight has the row; the tile has (rounded up)
    auto enter = [&]() {
      const Tile t = find(li);
      const int n = t.a0 + static_cast<int>(rank) * kRowsA + row;
      pa = args.w + (static_cast<size_t>(t.e) * g.N + n) * g.D + piece * 16;
      const int half = (t.cnt + S::kRound - 1) / S::kRound * S::kRound / CG;
      has_a = wanted = 0;
#pragma unroll
      for (int h = 0; h < kOwn; ++h) {
        const int r = row + 32 * h, b = static_cast<int>(rank) * half + r;
        if (n + 32 * h < g.N) has_a |= 1u << h;
        source[h] = -1;
        if (r < half) {
          wanted |= 1u << h;
          if (b < t.cnt) source[h] = g.p2u == nullptr ? t.start + b : g.p2u[t.start + b];
        }
      }
      if (g.p2u != nullptr) {
#pragma unroll
        for (int h = 0; h < kOwn; ++h)
          if (source[h] >= 0) source[h] = token_of(g, source[h]);
      }
    };
    auto settle = [&]() {  // the cursor behind its tile's last stage: on to the tile that has it
      if (ls < slices) return;
      do {
        ls -= slices;
        li += step;
      } while (ls >= slices && li < tiles);
      if (li < tiles) enter();
    };
    uint4 a[kOwn], b[kOwn];
    auto load_a = [&](int h) {
      const int at = ls * kWide;
      a[h] = load_piece<VB>(pa + at + h * far, has_a >> h & 1u ? g.D - piece * 16 - at : 0);
    };
    auto load_b = [&](int h) {
      const int at = piece * 16 + ls * kWide;
      b[h] = load_piece<VB>(args.x + static_cast<size_t>(max(source[h], 0)) * g.D + at,
                            source[h] >= 0 ? g.D - at : 0);
    };
    if (ls >= slices) settle();
    else if (li < tiles) enter();
    if (li < tiles) {
#pragma unroll
      for (int h = 0; h < kOwn; ++h) {
        load_a(h);
        load_b(h);
      }
    }
    int stage = group;
    uint32_t parity = 1;  // the first pass finds the stages empty
    // The piece is two of the eight in a row of the 128-byte swizzle, rows 32 apart alike.  The
    // lanes of a row's second half store the second first: the eight of a row then meet
    // all banks.
    const uint32_t half_at = row * 128 + (piece >> 2) * kHalf;
    const uint32_t even = half_at + ((((2 * piece) & 7) ^ (row & 7)) << 4);
    const uint32_t odd = half_at + ((((2 * piece + 1) & 7) ^ (row & 7)) << 4);
    const bool swap = piece >= 4;
    const uint32_t to0 = swap ? odd : even, to1 = swap ? even : odd;
    auto store_piece = [&](uint32_t at, const uint4& v) {
      store_wide(at + to0, swap ? v.z : v.x, swap ? v.w : v.y);
      store_wide(at + to1, swap ? v.x : v.z, swap ? v.y : v.w);
    };
    while (li < tiles) {
      const uint32_t keep = wanted;
      ls += 2;
      settle();
      const bool more = li < tiles;
      if (!__all_sync(0xffffffffu, wait(&empty[stage], parity))) break;
      const uint32_t at = stages_at + stage * kStageBytes;
      // An operand's stores before its next loads, one after the other: with each load right
      // behind its own piece's stores 8192 tokens and 256 experts took 285 us instead of 278 and
      // 8 experts of 4096 x 4096 368 instead of 355 (1003 tokens of 504 columns 116 instead of 118);
      // all loads behind all stores 305 and more (with the asynchronous store between the CTAs).
#pragma unroll
      for (int h = 0; h < kOwn; ++h) store_piece(at + h * 4096, a[h]);
      if (more) {
#pragma unroll
        for (int h = 0; h < kOwn; ++h) load_a(h);
      }
#pragma unroll
      for (int h = 0; h < kOwn; ++h)
        if (keep >> h & 1u) store_piece(at + kBytesA + h * 4096, b[h]);
      if (more) {
#pragma unroll
        for (int h = 0; h < kOwn; ++h) load_b(h);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
      // Three stages, two groups: a group's next use of a stage lies two phases on, the other
      // group's between them; its wait for the stage in between has seen the earlier phase end.
      stage += 2;
      if (stage >= kStages) {
        stage -= kStages;
        parity ^= 1;
      }
    }
  } else if (CG == 2 && rank == 1 && warp != 2 && warp < 4) {
    // ---- the second CTA's stages, announced to the leader, by a warp each -------------
    const int own = warp == 3 ? 2 : warp;
    int stage = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int i = first; i < tiles && ok; i += step)
      for (int s = 0; s < slices && ok; ++s) {
        if (stage == own) {
          ok = __all_sync(0xffffffffu, wait(&full[stage], parity));
          if (ok && lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&peer[stage]), 0));
          __syncwarp();
        }
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
  } else if (CG == 2 && rank == 1 && warp == 2) {
    // ---- its accumulators that have been read ---------------------------------------
    int n = 0;
    bool ok = true;
    const int segment = segment_of<F32>(slices, kMostStages);
    for (int i = first; i < tiles && ok; i += step)
      for (int s0 = 0; s0 < slices && ok; s0 += segment, ++n) {
        ok = __all_sync(0xffffffffu, wait(&read[n & 1], (n >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        tc_fence_before();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&drained[n & 1]), 0));
        __syncwarp();
      }
  } else if (warp == 1 && rank == 0) {
    // ---- products ----------------------------------------------------------------
    int stage = 0, n = 0;  // n: accumulators filled
    uint32_t parity = 0;
    bool ok = true;
    const int segment = segment_of<F32>(slices, kMostStages);
    Tile t{};
    if (first < tiles) t = find(first);
    for (int i = first; i < tiles && ok; i += step) {
      Tile nt = t;
      const int cols = (t.cnt + S::kRound - 1) / S::kRound * S::kRound;
      const uint32_t desc = half_product_desc(S::kTileA, cols);
      for (int s0 = 0; s0 < slices && ok; s0 += segment) {
        const int end = min(s0 + segment, slices);
        const int buf = n & 1;
        // an accumulator that the storing warps are done with
        ok = __all_sync(0xffffffffu, CG == 2 ? wait_cluster(wait, &drained[buf], ((n >> 1) & 1) ^ 1)
                                             : wait(&drained[buf], ((n >> 1) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * S::kTileB;
        for (int s = s0; s < end; ++s) {
          ok = __all_sync(0xffffffffu, wait(&full[stage], parity) &&
                                           (CG == 1 || wait_cluster(wait, &peer[stage], parity)));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = stages_at + stage * kStageBytes;
          const uint64_t da = operand_desc(at, 0, 1024);
          const uint64_t db = operand_desc(at + kBytesA, 0, 1024);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kWide / 16; ++k) {
              const uint64_t by = (k >> 2) * (kHalf >> 4) + (k & 3) * 2;
              if (16 * k < g.D - s * kWide)
                tc_product<CG>(d, da + by, db + by, desc, s > s0 || k > 0);
            }
            tc_commit<CG>(&empty[stage]);
            if (s == end - 1) tc_commit<CG>(&done[buf]);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
          // the next tile is looked up while this stage is computed
          if (s == 0 && i + step < tiles) nt = find(i + step);
        }
        ++n;
      }
      t = nt;
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- stores --------------------------------------------------------------------
    const int quad = warp - 4;
    int n = 0;
    bool ok = true;
    const int segment = segment_of<F32>(slices, kMostStages);
    // a tile's scales are asked for a tile ahead; each warp has its own copy of the rows', so
    // that one that gives up leaves none waiting
    float* const by_row = row_scales[quad];
    float scale[S::kTileB / 32], next_channel = 0.0f;
    Tile nt{};
    auto look = [&](int tile) {
      nt = find(tile);
      int source[S::kTileB / 32];
#pragma unroll
      for (int j = 0; j < S::kTileB / 32; ++j) {
        const int b = lane + 32 * j;
        source[j] = b >= nt.cnt ? -1 : g.p2u == nullptr ? nt.start + b : g.p2u[nt.start + b];
      }
      const int row = nt.a0 + static_cast<int>(rank) * kRowsA + quad * 32 + lane;
      next_channel = row < g.N ? args.w_scales[static_cast<size_t>(nt.e) * g.N + row] : 0.0f;
#pragma unroll
      for (int j = 0; j < S::kTileB / 32; ++j) {
        if (g.p2u != nullptr && source[j] >= 0) source[j] = token_of(g, source[j]);
        scale[j] = source[j] >= 0 ? args.x_scales[source[j]] : 0.0f;
      }
    };
    if (first < tiles) look(first);
    for (int i = first; i < tiles && ok; i += step) {
      const Tile t = nt;
      const float channel = next_channel;
      __syncwarp();  // all lanes have used the rows' scales of the tile before
#pragma unroll
      for (int j = 0; j < S::kTileB / 32; ++j) by_row[lane + 32 * j] = scale[j];
      __syncwarp();
      const int row = t.a0 + static_cast<int>(rank) * kRowsA + quad * 32 + lane;
      if (i + step < tiles) look(i + step);
      for (int first_slice = 0; first_slice == 0 || first_slice < slices;) {
        const bool add = first_slice > 0;  // fp32 only: to what this thread stored before
        const int buf = n & 1;
        ok = __all_sync(0xffffffffu, wait(&done[buf], (n >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc =
            tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * S::kTileB;
        for (int c = 0; c < t.cnt; c += 32) {
          uint32_t v[32];
          tmem_load_32(acc + c, v);
          if (c + 32 >= t.cnt) {  // the accumulator is free before the last stores
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(CG == 2 && rank == 1 ? &read[buf] : &drained[buf]);
          }
          // scaled in place first: reads of the rows' scales between the stores wait for one
          // another (110 cycles a store)
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(by_row + c + j);
            v[j] = __float_as_uint(scaled_sum(__uint_as_float(v[j]), channel, f.x));
            v[j + 1] = __float_as_uint(scaled_sum(__uint_as_float(v[j + 1]), channel, f.y));
            v[j + 2] = __float_as_uint(scaled_sum(__uint_as_float(v[j + 2]), channel, f.z));
            v[j + 3] = __float_as_uint(scaled_sum(__uint_as_float(v[j + 3]), channel, f.w));
          }
          const size_t o = static_cast<size_t>(t.start + c) * g.N + row;
          const bool whole = c + 32 <= t.cnt;
          if (row < g.N) {
            if constexpr (F32) {
              float* out = static_cast<float*>(g.out) + o;
              if (add) {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += g.N)
                  if (c + j < t.cnt) red_add(out, __uint_as_float(v[j]));
              } else if (whole) {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += g.N) *out = __uint_as_float(v[j]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += g.N)
                  if (c + j < t.cnt) *out = __uint_as_float(v[j]);
              }
            } else {
              unsigned short* out = static_cast<unsigned short*>(g.out) + o;
              if (whole) {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += g.N)
                  *out = static_cast<unsigned short>(f32_to_bf16_bits(__uint_as_float(v[j])));
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += g.N)
                  if (c + j < t.cnt)
                    *out = static_cast<unsigned short>(f32_to_bf16_bits(__uint_as_float(v[j])));
              }
            }
          }
          __syncwarp();
        }
        ++n;
        first_slice += max(segment, 1);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  // After a wait that gave up: leave products in flight another millisecond
  // before the shared and tensor memory is given back.
  if (*reinterpret_cast<volatile int*>(&gave_up))
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem, S::kColumns);
  }
}

// ---- host ------------------------------------------------------------------------
// Clusters of the kernel that run at once, asked once per device and kernel.
constexpr int kDevices = 64;
template <typename Kern>
int resident_clusters(Kern kern, int cg, std::atomic<int>* known) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
      cudaSuccess)
    return 0;
  n = device_sm_count();
  if (cg == 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  }
  if (n > 0) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int CG, int VB, bool F32>
int launch_typed(const W8Args& a, cudaStream_t st) {
  using S = Shape<CG>;
  static std::atomic<int> known[kDevices];
  const auto kern = expert_matmul_w8_kernel<CG, VB, F32>;
  const int resident = resident_clusters(kern, CG, known);
  W8TcArgs g{};
  g.t = TcArgs{a.offsets, a.p2u, a.out, device_status_word(), a.T, a.P, a.E, a.N, a.D,
               a.p2u == nullptr ? a.P : a.T, inverse_of(a.T)};
  if (resident <= 0 || g.t.status == nullptr) return MR_ERR_CUDA;
  g.x = a.x;
  g.w = a.w;
  g.x_scales = a.x_scales;
  g.w_scales = a.w_scales;
  g.least = a.least;
  const long long ta = (a.N + S::kTileA - 1) / S::kTileA;
  g.inv_a = inverse_of(static_cast<int>(ta));
  const long long tb = static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / S::kTileB;
  const long long clusters = ta * tb < resident ? ta * tb : resident;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, g) == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int VB>
int launch_width(const W8Args& a, cudaStream_t st) {
  const bool pair = a.P >= 40ll * a.E;
  if (a.out_dtype == DT_F32)
    return pair ? launch_typed<2, VB, true>(a, st) : launch_typed<1, VB, true>(a, st);
  return pair ? launch_typed<2, VB, false>(a, st) : launch_typed<1, VB, false>(a, st);
}

}  // namespace

int launch_expert_matmul_w8_tc(const W8Args& a, cudaStream_t st) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w) |
                        static_cast<uintptr_t>(a.D);
  return (all & 15u) == 0  ? launch_width<16>(a, st)
         : (all & 7u) == 0 ? launch_width<8>(a, st)
         : (all & 3u) == 0 ? launch_width<4>(a, st)
                           : launch_width<1>(a, st);
}

}  // namespace moe_router
