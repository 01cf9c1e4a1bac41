// Products grouped by expert on the tensor cores (bf16 operands, fp32 sums).
//
// The ragged dimension is the number of an expert's rows.  The tensor cores
// take 128 or 256 values of one dimension at a time and any multiple of 16 of
// the other, so the expert's weight rows (forward) or columns (input gradient)
// go to the first and its ragged rows to the second: out^T = W x^T.  An expert
// with n rows takes ceil(n / most) near-equal tiles, each rounded up to 16 (32
// for a pair of CTAs), and one with two rows costs a product of 16.
//
//   forward       A = W[e] rows n, K-major (d);       B = x rows p, K-major (d)
//   input grad    A = W[e] columns d, MN-major (n);   B = grad_out rows p, K-major (n)
//   weight grad   A = grad_out columns n, MN-major;   B = x columns d, MN-major; both
//                 over the expert's rows p, in slices of 64 from its first one
//
// Rows that lie in order come in boxes of 16 rows.  Rows of x behind the expert
// map, and the last rows of an expert in the weight gradient, come by gathering
// copies of four rows, each with its own index; an index behind the expert's
// last row points one past the tensor, which reads as zero.  So no row of
// another expert enters a product (the boxes of the forward and the input
// gradient may hold some: they fill columns that are not stored).
//
// Block: 24 warps.  Warps 0 and 3 load A, warps 8-23 load B, 16 rows (weight
// grad: of A and B, 16 rows x 64 columns) each: two groups of nine that take
// alternate slices, since one warp needs 500 to 1200 cycles from one slice to the
// next (four gathers are 400), and the products 350 to 500.  One elected thread
// of warp 1 issues the products, warp 2 owns the tensor memory, warps 4-7 store
// finished tiles while the next one is computed into the other half of the
// accumulator columns.  A stage holds 64 contraction indices: 16 KB of A and up to
// 16 KB of B.  Every loading warp arrives on its stages' barriers even with
// nothing to load, so none falls behind by a phase.  CG = 2: two CTAs share a
// tile of 256 x (up to 256), each holding half of A and of B, which halves the
// shared-memory and L2 traffic per product.  The grid is persistent; tile i goes
// to CTA (pair) i mod the grid.
//
// fp32 outputs.  The tensor cores add each 16-deep product to the accumulator
// by truncation, so a sum of n of them is off by about n 2^-26 of its value
// (measured: 4.7e-7 at n = 32), where a bf16 output's rounding is up to 2^-8.  A fp32
// output's contraction is therefore cut into segments of at most 960: each is
// an accumulator of its own and is added to the output, rounding to nearest, by
// the threads (weight grad: the copy engine) that stored the one before, in
// order, so results repeat bit for bit.  It costs a quarter of the compute-bound
// forward (8192 tokens, 64 experts, 2048 x 2048: 205 to 268 us; adding through
// staged boxes took 285 us).
//
// What bounded it on the way (forward, 8192 tokens, 64 experts, 4 choices,
// 2048 x 2048): the issue of copies and products.  Under a lane test each cost
// 60 to 100 cycles; 32 gathers a stage from one warp ran at 430 TFLOP/s, from
// eight warps at 1060, and with operands in uniform registers (elect_one) the
// kernel ran at 1250 through the map and 1310 in order, with two groups of loading
// warps at 1400 and 1430; 4096 x 4096 over 8 experts at 1770 and 1800 (input
// gradient).  A slice takes 640 to 700 cycles (29 to 32 KB for each SM) at 172, 210
// and 242 rows a tile alike, with L2 at 51 to 55 % of its rate and the tensor pipe at
// 67 to 71 %; which part of its way sets that is not separated.
#include <atomic>

#include "router_experts_tiles.cuh"

namespace moe_router {
namespace {

constexpr int kLoaders = 8;               // warps that load a slice of B (weight grad: A and B)
constexpr int kThreads = 32 * (8 + 2 * kLoaders);
constexpr int kMaxStages = 6;
constexpr int kRowsA = 128;               // values of A's dimension per CTA
constexpr int kRowsB = 128;               // most values of B's dimension per CTA
constexpr int kBytesA = kRowsA * 128;
constexpr int kBytesB = kRowsB * 128;
constexpr int kStageBytes = kBytesA + kBytesB;
constexpr int kBoxes = 4;  // weight grad: 32 x 128-byte boxes per storing warp

// Stages, and dynamic shared memory: stages and boxes start on 1024 bytes.  Stages
// are even in number: each belongs to one of the two groups of loading warps.
constexpr int stages_of(int form) { return form == EX_WGRAD ? 4 : kMaxStages; }
constexpr int smem_bytes(int form) {
  return stages_of(form) * kStageBytes + (form == EX_WGRAD ? 4 * kBoxes * 4096 : 0) + 1024;
}

template <int FORM, int CG>
struct Shape {
  static constexpr int kTileA = kRowsA * CG;
  static constexpr int kTileB = kRowsB * CG;
  static constexpr int kRound = 16 * CG;
  static constexpr int kStages = stages_of(FORM);
  static constexpr uint32_t kColumns = 2 * kTileB;  // two accumulators
};

// First row, within tile t, that loading warp w brings for slice s.
template <int FORM, int CG>
__device__ __forceinline__ int loader_row(const Tile& t, uint32_t rank, int w, int s) {
  if (FORM == EX_WGRAD) return s * kDeep + 16 * (w >> 1);
  constexpr int round = Shape<FORM, CG>::kRound;
  return static_cast<int>(rank) * ((t.cnt + round - 1) / round * round / CG) + 16 * w;
}

// Map entries of tile rows b0 + 4 l .. + 3, l = lane mod 4 (the loads are
// issued here and used a slice later).
__device__ __forceinline__ void fetch_rows(const TcArgs& g, const Tile& t, int b0, int lane,
                                           int (&u)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = b0 + 4 * (lane & 3) + j;
    u[j] = b >= t.cnt ? -1 : g.p2u == nullptr ? t.start + b : g.p2u[t.start + b];
  }
}

// Their rows of x: `none` for rows behind the tile's last.
__device__ __forceinline__ void source_rows(const TcArgs& g, const int (&u)[4], int none,
                                            int (&r)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = u[j] < 0 ? none : g.p2u == nullptr ? u[j] : token_of(g, u[j]);
}

// 16 rows of 64 columns: lanes 0-3 hold four row indices each.
template <int CG>
__device__ __forceinline__ void issue_gather(uint32_t dst, const CUtensorMap* map, int col,
                                             const int (&r)[4], bool one, uint32_t bar) {
  int q[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) q[j] = __shfl_sync(0xffffffffu, r[j & 3], j >> 2);
  if (one) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tma_gather4<CG>(dst + j * 512, map, col, q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3],
                      bar);
  }
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int FORM, int CG, bool F32>
__global__ __launch_bounds__(kThreads, 1) void expert_matmul_tc_kernel(
    const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
    const __grid_constant__ CUtensorMap box_a, const __grid_constant__ CUtensorMap box_b,
    const __grid_constant__ CUtensorMap map_out, const TcArgs g) {
  using S = Shape<FORM, CG>;
  extern __shared__ uint8_t dynamic_smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], done[2], drained[2];
  __shared__ uint32_t tmem_at;
  __shared__ int gave_up;
  __shared__ int tmp[33];
  __shared__ int prefix[FORM == EX_WGRAD ? 1 : MR_MAX_EXPERTS + 1];
  __shared__ int offs[MR_MAX_EXPERTS + 1];  // the offsets, clamped to [0, P]

  // the same value in all lanes, and known to be
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const uint32_t stages_at = (smem_addr(dynamic_smem) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], CG * (kLoaders + 1));
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&drained[i], 4 * CG);  // one arrival per storing warp
    }
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<CG>(&tmem_at, S::kColumns);
  pdl_enter();
  for (int e = threadIdx.x; e <= g.E; e += blockDim.x) offs[e] = min(max(g.offsets[e], 0), g.P);
  int tiles;
  if constexpr (FORM == EX_WGRAD) {
    tiles = g.E * ((g.N + S::kTileA - 1) / S::kTileA) * ((g.D + S::kTileB - 1) / S::kTileB);
  } else {
    tiles = expert_tile_prefix(g.offsets, g.E, g.P, S::kTileB, prefix, tmp) *
            (((FORM == EX_FWD ? g.N : g.D) + S::kTileA - 1) / S::kTileA);
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const Waiter wait{&gave_up, g.status};
  const int first = static_cast<int>(blockIdx.x) / CG, step = static_cast<int>(gridDim.x) / CG;
  // contraction slices of a tile
  const int fixed_slices = ((FORM == EX_FWD ? g.D : g.N) + kDeep - 1) / kDeep;

  if (warp >= 8 || warp == 0 || warp == 3) {
    // ---- loads -----------------------------------------------------------------
    // Two groups of warps load alternate slices.  A group's next slice, its tile
    // and its map entries are fetched before the present slice's copies are
    // issued, so their latency passes behind the issue.
    const int group = warp >= 8 ? (warp - 8) / kLoaders : warp == 3;
    const int w = warp >= 8 ? (warp - 8) % kLoaders : -1;  // -1: the warps that load A
    const bool mapped = w >= 0 && (FORM == EX_WGRAD || g.p2u != nullptr);
    int stage = group;
    uint32_t parity = 1;  // the first pass finds the stages empty
    int i = first, s = 0;
    Tile t = next_tile<FORM, S>(g, prefix, offs, tiles, step, &i);
    auto advance = [&](int* i, int* s, Tile* t) {
      const int slices = FORM == EX_WGRAD ? (t->cnt + kDeep - 1) / kDeep : fixed_slices;
      if (++*s == slices) {
        *i += step;
        *s = 0;
        *t = next_tile<FORM, S>(g, prefix, offs, tiles, step, i);
      }
    };
    if (group == 1 && i < tiles) advance(&i, &s, &t);
    int u[4], r[4];
    bool fresh = true;  // the map entries in u are not yet rows in r
    if (mapped && i < tiles) fetch_rows(g, t, loader_row<FORM, CG>(t, rank, w, s), lane, u);
    while (i < tiles) {
      if (mapped && (FORM == EX_WGRAD || fresh)) source_rows(g, u, g.x_rows, r);
      int ni = i, ns = s;
      Tile nt = t;
      advance(&ni, &ns, &nt);
      if (ni < tiles) advance(&ni, &ns, &nt);
      fresh = ni != i;
      if (mapped && ni < tiles && (FORM == EX_WGRAD || fresh))
        fetch_rows(g, nt, loader_row<FORM, CG>(nt, rank, w, ns), lane, u);

      const int row = loader_row<FORM, CG>(t, rank, w, s);
      const int a0 = t.a0 + static_cast<int>(rank) * kRowsA;
      // weight grad: a slice inside the expert comes as whole boxes of A; the
      // last one in pieces by the warps that load B
      const bool all_a = FORM != EX_WGRAD || s * kDeep + kDeep <= t.cnt;
      const bool whole = row + 16 <= t.cnt;
      uint32_t bytes;
      if (w < 0) {
        bytes = all_a ? kBytesA : 0;
      } else if (FORM == EX_WGRAD) {
        bytes = row < t.cnt ? (all_a ? 2048 : 4096) : 0;
      } else {
        const int rows = (t.cnt + S::kRound - 1) / S::kRound * S::kRound / CG;
        bytes = 16 * w < rows ? 2048 : 0;
      }
      if (!__all_sync(0xffffffffu, wait(&empty[stage], parity))) break;
      const uint32_t at = stages_at + stage * kStageBytes;
      const uint32_t bar =
          CG == 2 ? map_to_rank(smem_addr(&full[stage]), 0) : smem_addr(&full[stage]);
      const bool one = elect_one();
      if (one) mbar_expect_tx_cluster(bar, bytes);
      if (bytes == 0) {
      } else if (w < 0) {
        if (one) {
          if constexpr (FORM == EX_FWD) {
            tma_load_3d<CG>(at, &map_a, s * kDeep, a0, t.e, bar);
          } else if constexpr (FORM == EX_DGRAD) {
            tma_load_3d<CG>(at, &map_a, a0, s * kDeep, t.e, bar);
            tma_load_3d<CG>(at + 8192, &map_a, a0 + 64, s * kDeep, t.e, bar);
          } else {
            tma_load_2d<CG>(at, &box_a, a0, t.start + s * kDeep, bar);
            tma_load_2d<CG>(at + 8192, &box_a, a0 + 64, t.start + s * kDeep, bar);
          }
        }
      } else if constexpr (FORM == EX_WGRAD) {
        const uint32_t piece = at + (w & 1) * 8192 + (w >> 1) * 2048;
        const int cb = t.b0 + static_cast<int>(rank) * kRowsB + 64 * (w & 1);
        if (g.p2u != nullptr || !whole) {
          issue_gather<CG>(piece + kBytesA, &map_b, cb, r, one, bar);
        } else if (one) {
          tma_load_2d<CG>(piece + kBytesA, &box_b, cb, t.start + row, bar);
        }
        if (!all_a) {
          int p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int b = row + 4 * (lane & 3) + j;
            p[j] = b < t.cnt ? t.start + b : g.P;
          }
          issue_gather<CG>(piece, &map_a, a0 + 64 * (w & 1), p, one, bar);
        }
      } else {
        const uint32_t piece = at + kBytesA + w * 2048;
        if (mapped) {
          issue_gather<CG>(piece, &map_b, s * kDeep, r, one, bar);
        } else if (one) {
          tma_load_2d<CG>(piece, &box_b, s * kDeep, t.start + row, bar);
        }
      }
      stage += 2;
      if (stage >= S::kStages) {
        stage = group;
        parity ^= 1;
      }
      i = ni;
      t = nt;
      s = ns;
    }
  } else if (warp == 1 && rank == 0) {
    // ---- products ----------------------------------------------------------------
    int stage = 0, n = 0;  // n: accumulators filled
    uint32_t parity = 0;
    bool ok = true;
    int i = first;
    Tile t = next_tile<FORM, S>(g, prefix, offs, tiles, step, &i);
    while (i < tiles && ok) {
      const int slices = FORM == EX_WGRAD ? (t.cnt + kDeep - 1) / kDeep : fixed_slices;
      const int cols = FORM == EX_WGRAD ? S::kTileB
                                        : (t.cnt + S::kRound - 1) / S::kRound * S::kRound;
      const uint32_t desc =
          product_desc(S::kTileA, cols, FORM != EX_FWD, FORM == EX_WGRAD);
      int ni = i + step;
      Tile nt = t;
      const int segment = segment_of<F32>(slices);
      for (int s0 = 0; s0 < slices && ok; s0 += segment) {
        const int end = min(s0 + segment, slices);
        const int buf = n & 1;
        // an accumulator that the storing warps are done with
        ok = __all_sync(0xffffffffu, wait(&drained[buf], ((n >> 1) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * S::kTileB;
        for (int s = s0; s < end; ++s) {
          ok = __all_sync(0xffffffffu, wait(&full[stage], parity));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = stages_at + stage * kStageBytes;
          // 16 contraction indices are 32 bytes of a K-major row, 16 rows of an
          // MN-major slice
          const uint64_t da = FORM == EX_FWD ? operand_desc(at, 0, 1024)
                                             : operand_desc(at, 8192, 1024);
          const uint64_t db = FORM == EX_WGRAD ? operand_desc(at + kBytesA, 8192, 1024)
                                               : operand_desc(at + kBytesA, 0, 1024);
          constexpr uint64_t ka = FORM == EX_FWD ? 2 : 128, kb = FORM == EX_WGRAD ? 128 : 2;
          const int depth = FORM == EX_WGRAD ? min(kDeep, t.cnt - s * kDeep) : kDeep;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kDeep / 16; ++k)
              if (16 * k < depth)
                tc_product<CG>(d, da + k * ka, db + k * kb, desc, s > s0 || k > 0);
            tc_commit<CG>(&empty[stage]);
            if (s == end - 1) tc_commit<CG>(&done[buf]);
          }
          __syncwarp();
          if (++stage == S::kStages) {
            stage = 0;
            parity ^= 1;
          }
          // the next tile is looked up while this slice is computed
          if (s == 0) nt = next_tile<FORM, S>(g, prefix, offs, tiles, step, &ni);
        }
        ++n;
      }
      i = ni;
      t = nt;
    }
  } else if (warp >= 4) {
    // ---- stores --------------------------------------------------------------------
    const int quad = warp - 4;
    [[maybe_unused]] const uint32_t boxes_at =
        stages_at + S::kStages * kStageBytes +
        quad * (kBoxes * 4096);
    // the lane that issues copies: their groups are its own to wait for
    [[maybe_unused]] const bool one = elect_one();
    int n = 0;
    bool ok = true;
    Tile nt{};
    if (first < tiles) nt = find_tile<FORM, S>(g, prefix, offs, first);
    for (int i = first; i < tiles && ok; i += step) {
      const Tile t = nt;
      if (i + step < tiles) nt = find_tile<FORM, S>(g, prefix, offs, i + step);
      const bool none = FORM == EX_WGRAD && t.cnt == 0;  // an expert without rows: zeros
      const int slices = FORM == EX_WGRAD ? (t.cnt + kDeep - 1) / kDeep : fixed_slices;
      // one accumulator after the other: the first is stored, the others added
      const int segment = segment_of<F32>(slices);
      for (int first_slice = 0; first_slice == 0 || first_slice < slices;) {
        const bool add = first_slice > 0;
        const int buf = n & 1;
        if (!none) {
          ok = __all_sync(0xffffffffu, wait(&done[buf], (n >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t acc =
            tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * S::kTileB;
        const int row0 = t.a0 + static_cast<int>(rank) * kRowsA + quad * 32;  // of A's dimension
        if constexpr (FORM == EX_WGRAD) {
          // a lane holds one row of the gradient: 128 bytes of it at a time go to
          // shared memory (16-byte pieces swizzled, so that neither side meets a
          // bank conflict) and leave as a box of 32 rows.  Storing each lane's
          // piece directly touched 32 lines per instruction and ran at 2.9 TB/s.
          constexpr int wide = F32 ? 32 : 64;
          const int cols = row0 < g.N ? min(S::kTileB, g.D - t.b0) : 0;
          if (none && cols > 0) {  // one box of zeros for the whole tile
            const uint32_t box = boxes_at;
            if (one) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) st_shared_v4(box + (j * 32 + lane) * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (one) {
              for (int c = 0; c < cols; c += wide) tma_store_3d(&map_out, box, t.b0 + c, row0, t.e);
              bulk_commit();
            }
          }
          if (add && one) bulk_wait_all();  // what it is added to has arrived
          for (int c0 = 0; c0 < cols && !none; c0 += kBoxes * wide) {
            if (one) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kBoxes; ++q) {
              const int c = c0 + q * wide;
              if (c >= cols) break;
              const uint32_t box = boxes_at + q * 4096;
              uint32_t v[32];
              if constexpr (F32) {
                tmem_load_32(acc + c, v);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t u[32];
                  tmem_load_32(acc + c + 32 * h, u);
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    v[16 * h + j] =
                        bf16_pair(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
                }
              }
#pragma unroll
              for (int j = 0; j < 8; ++j)
                st_shared_v4(box + lane * 128 + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1],
                             v[4 * j + 2], v[4 * j + 3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (one) {
              for (int q = 0; q < kBoxes && c0 + q * wide < cols; ++q) {
                if (add) tma_add_3d(&map_out, boxes_at + q * 4096, t.b0 + c0 + q * wide, row0, t.e);
                else tma_store_3d(&map_out, boxes_at + q * 4096, t.b0 + c0 + q * wide, row0, t.e);
              }
              bulk_commit();
            }
          }
        } else {
          const int row = row0 + lane;
          const int rows = FORM == EX_DGRAD ? g.D : g.N;
          for (int c = 0; c < t.cnt; c += 32) {
            uint32_t v[32];
            tmem_load_32(acc + c, v);
            // a warp holds 32 neighbours of 32 output rows
            const size_t o = static_cast<size_t>(t.start + c) * rows + row;
            if constexpr (F32) {
              if (row < rows) {
                float* out = static_cast<float*>(g.out) + o;
                if (add) {
#pragma unroll
                  for (int j = 0; j < 32; ++j, out += rows)
                    if (c + j < t.cnt) red_add(out, __uint_as_float(v[j]));
                } else if (c + 32 <= t.cnt) {
#pragma unroll
                  for (int j = 0; j < 32; ++j, out += rows) *out = __uint_as_float(v[j]);
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j, out += rows)
                    if (c + j < t.cnt) *out = __uint_as_float(v[j]);
                }
              }
            } else if (row < rows) {
              unsigned short* out = static_cast<unsigned short*>(g.out) + o;
              if (c + 32 <= t.cnt) {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += rows)
                  *out = static_cast<unsigned short>(f32_to_bf16_bits(__uint_as_float(v[j])));
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += rows)
                  if (c + j < t.cnt)
                    *out = static_cast<unsigned short>(f32_to_bf16_bits(__uint_as_float(v[j])));
              }
            }
            __syncwarp();
          }
        }
        if (!none) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0)
            mbar_arrive_cluster(CG == 2 ? map_to_rank(smem_addr(&drained[buf]), 0)
                                        : smem_addr(&drained[buf]));
          ++n;
        }
        first_slice += max(segment, 1);
      }
    }
    if (FORM == EX_WGRAD && one) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  // After a wait that gave up: leave copies and products in flight another
  // millisecond before the shared and tensor memory is given back.
  if (*reinterpret_cast<volatile int*>(&gave_up))
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem, S::kColumns);
  }
}

// ---- host ------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up through the runtime.
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Tensor of `rank` dimensions, innermost first, dense; boxes 128 bytes wide,
// 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
              const cuuint32_t* box, bool f32 = false) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t strides[2];
  strides[0] = dims[0] * (f32 ? 4 : 2);
  if (rank == 3) strides[1] = strides[0] * dims[1];
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            static_cast<cuuint32_t>(rank),
            const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows_map(CUtensorMap* map, const void* base, int rows, int cols, cuuint32_t high) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[2] = {64, high};
  return make_map(map, base, 2, dims, box);
}

bool weight_map(CUtensorMap* map, const void* base, const ExpertArgs& a, int box_rows,
                bool f32 = false) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.N),
                              static_cast<cuuint64_t>(a.E)};
  const cuuint32_t box[3] = {f32 ? 32u : 64u, static_cast<cuuint32_t>(box_rows), 1};
  return make_map(map, base, 3, dims, box, f32);
}

// Clusters of the kernel that run at once, asked once per device and kernel.
constexpr int kDevices = 64;
template <typename Kern>
int resident_clusters(Kern kern, int cg, int smem, std::atomic<int>* known) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return 0;
  n = device_sm_count();
  if (cg == 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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

template <int FORM, int CG, bool F32>
int launch_typed(const ExpertArgs& a, cudaStream_t st) {
  using S = Shape<FORM, CG>;
  static std::atomic<int> known[kDevices];
  const auto kern = expert_matmul_tc_kernel<FORM, CG, F32>;
  const int resident = resident_clusters(kern, CG, smem_bytes(FORM), known);
  TcArgs g{a.offsets, a.p2u, a.out, device_status_word(), a.T, a.P, a.E, a.N, a.D,
           FORM == EX_DGRAD || a.p2u == nullptr ? a.P : a.T,
           inverse_of(a.T)};
  if (resident <= 0 || g.status == nullptr) return MR_ERR_CUDA;
  // a and b: weights, or single rows for gathering; the boxes: 16 rows in order
  CUtensorMap ma, mb, ba, bb, out;
  bool maps;
  if (FORM == EX_WGRAD) {
    maps = rows_map(&ma, a.a, a.P, a.N, 1) && rows_map(&ba, a.a, a.P, a.N, kDeep) &&
           rows_map(&mb, a.b, g.x_rows, a.D, 1) && rows_map(&bb, a.b, g.x_rows, a.D, 16) &&
           weight_map(&out, a.out, a, 32, F32);
  } else {
    const int cols = FORM == EX_FWD ? a.D : a.N;
    maps = weight_map(&ma, a.b, a, FORM == EX_FWD ? kRowsA : kDeep) &&
           rows_map(&mb, a.a, g.x_rows, cols, 1) && rows_map(&bb, a.a, g.x_rows, cols, 16);
    ba = out = ma;  // not used
  }
  if (!maps) return MR_ERR_CUDA;
  const long long ta = ((FORM == EX_DGRAD ? a.D : a.N) + S::kTileA - 1) / S::kTileA;
  const long long tb = FORM == EX_WGRAD
                           ? static_cast<long long>(a.E) * ((a.D + S::kTileB - 1) / S::kTileB)
                           : static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / S::kTileB;
  const long long clusters = ta * tb < resident ? ta * tb : resident;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(FORM);
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
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, ba, bb, out, g) == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <int FORM>
int launch_form(const ExpertArgs& a, cudaStream_t st) {
  const bool pair = FORM == EX_WGRAD ? a.N > kRowsA : a.P >= 40ll * a.E;
  if (a.out_dtype == DT_F32)
    return pair ? launch_typed<FORM, 2, true>(a, st) : launch_typed<FORM, 1, true>(a, st);
  return pair ? launch_typed<FORM, 2, false>(a, st) : launch_typed<FORM, 1, false>(a, st);
}

}  // namespace

bool expert_matmul_tc_ok(int form, const ExpertArgs& a) {
  const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (a.dtype != DT_BF16 || a.P < 1 || !aligned(a.a) || !aligned(a.b) || !aligned(a.out))
    return false;
  if (a.D % 8 != 0) return false;
  return form == EX_FWD || a.N % 8 == 0;
}

int launch_expert_matmul_tc(int form, const ExpertArgs& a, cudaStream_t st) {
  return form == EX_FWD     ? launch_form<EX_FWD>(a, st)
         : form == EX_DGRAD ? launch_form<EX_DGRAD>(a, st)
                            : launch_form<EX_WGRAD>(a, st);
}

}  // namespace moe_router
