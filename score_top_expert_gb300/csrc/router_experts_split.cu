// Products grouped by expert on the tensor cores for operands that the copy
// engine cannot bring: fp32, and bf16 rows that are not 16-byte aligned.
//
// fp32.  A value's 24 significant bits are cut into three bf16 parts of 8,
// x = h + m + l, exactly (each part is the upper half of what is left).  Of the
// nine products of two values all but the smallest, l l, are computed, each exact
// in fp32; what is left out is below 2^-28 of the product, and what of a value lies
// below 2^-133, the smallest bf16 number.  The first, h h, has an
// accumulator of its own and the seven small ones share another, so that the
// truncation of the tensor cores' sums (see router_experts_tc.cu) acts on as few
// additions of large terms as in a bf16 product; a contraction is cut into
// segments of at most 512 the same way, and a segment's two sums are added in
// round-to-nearest: 2.7e-7 of the value at 515 terms and 4.9e-7 at 3900, where
// fp32 multiply-add loops leave 4e-7 and 1.1e-6.
// In the small products an infinity meets empty parts (NaN), so a first sum that
// is not finite is the result by itself (1 % of the kernel).
//
// The tiles, their order and which operand is A are those of
// router_experts_tc.cu with one CTA to a tile (128 x up to 128).  A stage holds 64
// contraction indices of all parts.  Sixteen warps load: 64 neighbouring elements
// of a row a warp at a time, two per lane, element loads at any alignment, the next
// slice's rows of one operand in flight while the other's parts are stored; the
// parts go to shared memory in the layout that the tensor cores read.
//
// Bound by the slices, 1.9 to 2.3 us each whether a CTA has few or many: shared
// memory, which the 32 instructions of a slice read 8 KB of operands each from and
// the parts are written to, and the loading warps' instructions (issue slots at 56 to
// 66 %, tensor pipe 30 to 42 %).  8192 tokens, 64 experts, 4 choices, 1024 x 1024 fp32
// take 573 us forward (120 TFLOP/s of fp32 products), 500 us and 660 us the gradients;
// the vector units reach 75 at most.  517 tokens of 515 x 333, two tiles of nine
// slices on most SMs: 46 us.
#include <atomic>

#include "router_experts_tiles.cuh"

namespace moe_router {
namespace {

constexpr int kLoaders = 16;
constexpr int kThreads = 32 * (8 + kLoaders);
constexpr int kTileRows = 128;               // of A and (at most) of B
constexpr int kPartBytes = kTileRows * 128;  // one part of one operand
constexpr int kOwn = kTileRows / kLoaders;   // rows of each operand that a warp loads
constexpr int kStages = 2;
// Stages per accumulator of fp32 operands (15 left 9e-7 of the value at 3900 terms).
constexpr int kSplitSegment = 8;
constexpr int kPadded = 33;                  // weight grad: staging row, in words

struct SplitShape {
  static constexpr int kTileA = kTileRows;
  static constexpr int kTileB = kTileRows;
  static constexpr int kRound = 16;
};

// Parts of an element, and accumulators of a tile.
template <typename TIn> struct Parts;
template <> struct Parts<float> { static constexpr int kN = 3, kSums = 2; };
template <> struct Parts<unsigned short> { static constexpr int kN = 1, kSums = 1; };

constexpr int smem_of(int parts, int form) {
  return kStages * 2 * parts * kPartBytes + (form == EX_WGRAD ? 4 * 32 * kPadded * 4 : 0) + 1024;
}

struct SplitArgs {
  TcArgs t;
  const void* a;
  const void* b;
  int out_f32;
};

// x minus its upper half; nothing of an infinity or NaN, which is its own first part.
__device__ __forceinline__ uint32_t rest_of(uint32_t x) {
  const float r = __uint_as_float(x) - __uint_as_float(x & 0xffff0000u);
  return r == r ? __float_as_uint(r) : 0u;
}

// x minus its rest, which is its upper half; of a NaN, whose bits may all lie in the
// lower half, the NaN of any arithmetic (2 % of the kernel; comparing and marking it
// instead took 17 %).
__device__ __forceinline__ uint32_t without_rest(uint32_t x, uint32_t rest) {
  return __float_as_uint(__uint_as_float(x) - __uint_as_float(rest));
}

__device__ __forceinline__ uint32_t rest_of_finite(uint32_t x) {
  return __float_as_uint(__uint_as_float(x) - __uint_as_float(x & 0xffff0000u));
}

// A tile's two sums: the first alone where it is infinite or NaN, since an infinity
// has met empty parts in the second.
__device__ __forceinline__ uint32_t with_small(uint32_t big, uint32_t small) {
  const bool finite = (big & 0x7f800000u) != 0x7f800000u;
  return finite ? __float_as_uint(__uint_as_float(big) + __uint_as_float(small)) : big;
}

// The upper halves of x0 and x1 as a bf16 pair.
__device__ __forceinline__ uint32_t upper_halves(uint32_t x0, uint32_t x1) {
  return __byte_perm(x0, x1, 0x7632);
}

__device__ __forceinline__ void st_word(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Element i as its bits, for bf16 in the low half.
__device__ __forceinline__ uint32_t load_bits(const float* p) { return __float_as_uint(__ldg(p)); }
__device__ __forceinline__ uint32_t load_bits(const unsigned short* p) { return __ldg(p); }

// Two elements of a row from column 2 * lane, zero behind `cols`.
template <typename TIn>
__device__ __forceinline__ void load_two(const TIn* p, int cols, int lane, uint32_t (&v)[2]) {
  v[0] = 2 * lane < cols ? load_bits(p + 2 * lane) : 0u;
  v[1] = 2 * lane + 1 < cols ? load_bits(p + 2 * lane + 1) : 0u;
}

// A warp's rows of a stage, row index w + 16 j.  Flat: rows of 64 columns, j = 0
// .. 7.  Else 64 rows of 128 columns as two halves, j & 3 and j >> 2.  p: row w,
// stride: 16 rows; `rows` of the 128 (64) and `cols` exist, the others are zero.
template <bool FLAT, typename TIn>
__device__ __forceinline__ void load_rows(const TIn* p, size_t stride, int rows, int cols, int w,
                                          int lane, uint32_t (&v)[kOwn][2]) {
  if (rows >= (FLAT ? 128 : 64) && cols >= (FLAT ? 64 : 128)) {
    p += 2 * lane;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const TIn* q = FLAT ? p + j * stride : p + (j & 3) * stride + (j >> 2) * 64;
      v[j][0] = load_bits(q);
      v[j][1] = load_bits(q + 1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int r = w + 16 * (FLAT ? j : j & 3);
      load_two(FLAT ? p + j * stride : p + (j & 3) * stride + (j >> 2) * 64,
               r < rows ? cols - (FLAT ? 0 : (j >> 2) * 64) : 0, lane, v[j]);
    }
  }
}

// Row r of a part, two elements per lane, in the 128-byte swizzle.
template <typename TIn>
__device__ __forceinline__ void store_parts(uint32_t at, int r, int lane, uint32_t (&v)[2]) {
  const uint32_t to = at + r * 128 + ((((lane >> 2) ^ r) & 7) << 4) + (lane & 3) * 4;
  if constexpr (Parts<TIn>::kN == 1) {
    st_word(to, v[0] | (v[1] << 16));
  } else {
    const uint32_t m0 = rest_of(v[0]), m1 = rest_of(v[1]);
    st_word(to, upper_halves(without_rest(v[0], m0), without_rest(v[1], m1)));
    st_word(to + kPartBytes, upper_halves(m0, m1));
    st_word(to + 2 * kPartBytes, upper_halves(rest_of_finite(m0), rest_of_finite(m1)));
  }
}

template <typename TIn, int FORM>
__global__ __launch_bounds__(kThreads, 1) void expert_matmul_split_kernel(const SplitArgs args) {
  using S = SplitShape;
  constexpr int kN = Parts<TIn>::kN, kSums = Parts<TIn>::kSums;
  constexpr int kStageBytes = 2 * kN * kPartBytes;
  constexpr uint32_t kColumns = 2 * kSums * kTileRows;  // two accumulators
  const TcArgs& g = args.t;
  extern __shared__ uint8_t dynamic_smem[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done[2], drained[2];
  __shared__ uint32_t tmem_at;
  __shared__ int gave_up;
  __shared__ int tmp[33];
  __shared__ int prefix[FORM == EX_WGRAD ? 1 : MR_MAX_EXPERTS + 1];
  __shared__ int offs[MR_MAX_EXPERTS + 1];  // the offsets, clamped to [0, P]

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t stages_at = (smem_addr(dynamic_smem) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&drained[i], 4);
    }
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<1>(&tmem_at, kColumns);
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
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const Waiter wait{&gave_up, g.status};
  const int first = blockIdx.x, step = gridDim.x;
  const int fixed_slices = ((FORM == EX_FWD ? g.D : g.N) + kDeep - 1) / kDeep;

  if (warp >= 8) {
    // ---- loads -----------------------------------------------------------------
    const int w = warp - 8;
    const TIn* __restrict__ A = static_cast<const TIn*>(args.a);
    const TIn* __restrict__ B = static_cast<const TIn*>(args.b);
    // Element loads of a slice's rows of one operand.  A's are in flight while B's
    // parts of the slice before are stored and the other way round.
    auto load_a = [&](const Tile& t, int s, uint32_t (&v)[kOwn][2]) {
      const int k = s * kDeep;
      if constexpr (FORM == EX_FWD)
        load_rows<true>(A + (static_cast<size_t>(t.e) * g.N + t.a0 + w) * g.D + k,
                        static_cast<size_t>(16) * g.D, g.N - t.a0, g.D - k, w, lane, v);
      else if constexpr (FORM == EX_DGRAD)
        load_rows<false>(A + (static_cast<size_t>(t.e) * g.N + k + w) * g.D + t.a0,
                         static_cast<size_t>(16) * g.D, g.N - k, g.D - t.a0, w, lane, v);
      else
        load_rows<false>(A + static_cast<size_t>(t.start + k + w) * g.N + t.a0,
                         static_cast<size_t>(16) * g.N, t.cnt - k, g.N - t.a0, w, lane, v);
    };
    [[maybe_unused]] const TIn* source[kOwn];  // forward: the tokens behind this warp's rows of B
    auto load_b = [&](const Tile& t, int s, bool fresh, uint32_t (&v)[kOwn][2]) {
      const int k = s * kDeep;
      if constexpr (FORM == EX_FWD) {
        if (fresh) {
          int token[kOwn];
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            const int r = w + j * kLoaders;
            token[j] = r < t.cnt ? (g.p2u == nullptr ? t.start + r : g.p2u[t.start + r]) : -1;
          }
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            if (g.p2u != nullptr && token[j] >= 0) token[j] = token_of(g, token[j]);
            source[j] = token[j] < 0 ? nullptr : B + static_cast<size_t>(token[j]) * g.D;
          }
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
          load_two(source[j] + k, source[j] == nullptr ? 0 : g.D - k, lane, v[j]);
      } else if constexpr (FORM == EX_DGRAD) {
        load_rows<true>(B + static_cast<size_t>(t.start + w) * g.N + k,
                        static_cast<size_t>(16) * g.N, t.cnt, g.N - k, w, lane, v);
      } else if (g.p2u == nullptr) {
        load_rows<false>(B + static_cast<size_t>(t.start + k + w) * g.D + t.b0,
                         static_cast<size_t>(16) * g.D, t.cnt - k, g.D - t.b0, w, lane, v);
      } else {
        int u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = k + w + 16 * j;
          u[j] = r < t.cnt ? g.p2u[t.start + r] : -1;
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int row = u[j & 3];
          const TIn* p = B + static_cast<size_t>(row < 0 ? 0 : token_of(g, row)) * g.D + t.b0 +
                         (j >> 2) * 64;
          load_two(p, row < 0 ? 0 : g.D - t.b0 - (j >> 2) * 64, lane, v[j]);
        }
      }
    };
    int stage = 0;
    uint32_t parity = 1;  // the first pass finds the stages empty
    int i = first, s = 0;
    Tile t = next_tile<FORM, S>(g, prefix, offs, tiles, step, &i);
    uint32_t va[kOwn][2], vb[kOwn][2];
    if (i < tiles) {
      load_a(t, 0, va);
      load_b(t, 0, true, vb);
    }
    while (i < tiles) {
      const int slices = FORM == EX_WGRAD ? (t.cnt + kDeep - 1) / kDeep : fixed_slices;
      const int rows_b = FORM == EX_WGRAD ? kTileRows : (t.cnt + 15) / 16 * 16;
      if (++s == slices) {  // t and s: the slice after the one that is stored
        s = 0;
        i += step;
        t = next_tile<FORM, S>(g, prefix, offs, tiles, step, &i);
      }
      if (!__all_sync(0xffffffffu, wait(&empty[stage], parity))) break;
      const uint32_t at = stages_at + stage * kStageBytes;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) store_parts<TIn>(at, w + j * kLoaders, lane, va[j]);
      if (i < tiles) load_a(t, s, va);
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (w + j * kLoaders < rows_b)
          store_parts<TIn>(at + kN * kPartBytes, w + j * kLoaders, lane, vb[j]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
      if (i < tiles) load_b(t, s, s == 0, vb);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
  } else if (warp == 1) {
    // ---- products ----------------------------------------------------------------
    int stage = 0, n = 0;  // n: accumulators filled
    uint32_t parity = 0;
    bool ok = true;
    int i = first;
    Tile t = next_tile<FORM, S>(g, prefix, offs, tiles, step, &i);
    while (i < tiles && ok) {
      const int slices = FORM == EX_WGRAD ? (t.cnt + kDeep - 1) / kDeep : fixed_slices;
      const int cols = FORM == EX_WGRAD ? kTileRows : (t.cnt + 15) / 16 * 16;
      const uint32_t desc = product_desc(kTileRows, cols, FORM != EX_FWD, FORM == EX_WGRAD);
      const int segment = args.out_f32 ? segment_of<true>(slices, kN == 3 ? kSplitSegment : kSegment) : slices;
      int ni = i + step;
      Tile nt = t;
      for (int s0 = 0; s0 < slices && ok; s0 += segment) {
        const int end = min(s0 + segment, slices);
        const int buf = n & 1;
        ok = __all_sync(0xffffffffu, wait(&drained[buf], ((n >> 1) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * (kSums * kTileRows);
        for (int s = s0; s < end; ++s) {
          ok = __all_sync(0xffffffffu, wait(&full[stage], parity));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = stages_at + stage * kStageBytes;
          constexpr uint64_t ka = FORM == EX_FWD ? 2 : 128, kb = FORM == EX_WGRAD ? 128 : 2;
          constexpr uint64_t part = kPartBytes >> 4;
          const uint64_t da = FORM == EX_FWD ? operand_desc(at, 0, 1024)
                                             : operand_desc(at, 8192, 1024);
          const uint32_t at_b = at + kN * kPartBytes;
          const uint64_t db = FORM == EX_WGRAD ? operand_desc(at_b, 8192, 1024)
                                               : operand_desc(at_b, 0, 1024);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kDeep / 16; ++k) {
              const uint64_t a = da + k * ka, b = db + k * kb;
              const bool more = s > s0 || k > 0;
              tc_product<1>(d, a, b, desc, more);
              if constexpr (kN == 3) {
                const uint32_t small = d + kTileRows;
                tc_product<1>(small, a, b + part, desc, more);
                tc_product<1>(small, a + part, b, desc, true);
                tc_product<1>(small, a + part, b + part, desc, true);
                tc_product<1>(small, a, b + 2 * part, desc, true);
                tc_product<1>(small, a + 2 * part, b, desc, true);
                tc_product<1>(small, a + part, b + 2 * part, desc, true);
                tc_product<1>(small, a + 2 * part, b + part, desc, true);
              }
            }
            tc_commit<1>(&empty[stage]);
            if (s == end - 1) tc_commit<1>(&done[buf]);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
          if (s == 0) nt = next_tile<FORM, S>(g, prefix, offs, tiles, step, &ni);
        }
        ++n;
      }
      i = ni;
      t = nt;
    }
  } else if (warp >= 4) {
    // ---- stores --------------------------------------------------------------------
    const int quad = warp & 3;
    [[maybe_unused]] const uint32_t staged =
        stages_at + kStages * kStageBytes + quad * (32 * kPadded * 4);
    int n = 0;
    bool ok = true;
    Tile nt{};
    if (first < tiles) nt = find_tile<FORM, S>(g, prefix, offs, first);
    for (int i = first; i < tiles && ok; i += step) {
      const Tile t = nt;
      if (i + step < tiles) nt = find_tile<FORM, S>(g, prefix, offs, i + step);
      const bool none = FORM == EX_WGRAD && t.cnt == 0;  // an expert without rows: zeros
      const int slices = FORM == EX_WGRAD ? (t.cnt + kDeep - 1) / kDeep : fixed_slices;
      const int segment = args.out_f32 ? segment_of<true>(slices, kN == 3 ? kSplitSegment : kSegment) : slices;
      for (int first_slice = 0; first_slice == 0 || first_slice < slices;) {
        const bool add = first_slice > 0;  // fp32 only: to what this thread stored before
        const int buf = n & 1;
        if (!none) {
          ok = __all_sync(0xffffffffu, wait(&done[buf], (n >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t acc =
            tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * (kSums * kTileRows);
        const int row0 = t.a0 + quad * 32;  // of A's dimension
        const int rows = FORM == EX_DGRAD ? g.D : g.N;
        const int cols = FORM == EX_WGRAD ? min(kTileRows, g.D - t.b0) : t.cnt;
        for (int c = 0; c < cols; c += 32) {
          uint32_t v[32];
          if (none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          } else {
            tmem_load_32(acc + c, v);
            if constexpr (kSums == 2) {
              uint32_t u[32];
              tmem_load_32(acc + kTileRows + c, u);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                v[j] = with_small(v[j], u[j]);
            }
          }
          // a lane's 32 values go to 32 rows of the output (its own column of
          // them); the weight gradient's are 32 columns of one row: turned
          size_t o, pitch;
          int last;  // rows of the output here
          bool mine;
          if constexpr (FORM == EX_WGRAD) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j) st_word(staged + (lane * kPadded + j) * 4, v[j]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              asm volatile("ld.shared.b32 %0, [%1];"
                           : "=r"(v[j]) : "r"(staged + (j * kPadded + lane) * 4) : "memory");
            o = (static_cast<size_t>(t.e) * g.N + row0) * g.D + t.b0 + c + lane;
            pitch = g.D;
            last = min(32, g.N - row0);
            mine = c + lane < cols;
          } else {
            o = static_cast<size_t>(t.start + c) * rows + row0 + lane;
            pitch = rows;
            last = min(32, cols - c);
            mine = row0 + lane < rows;
          }
          if (mine) {
            if (args.out_f32) {
              float* out = static_cast<float*>(g.out) + o;
              if (add) {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += pitch)
                  if (j < last) red_add(out, __uint_as_float(v[j]));
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j, out += pitch)
                  if (j < last) *out = __uint_as_float(v[j]);
              }
            } else {
              unsigned short* out = static_cast<unsigned short*>(g.out) + o;
#pragma unroll
              for (int j = 0; j < 32; ++j, out += pitch)
                if (j < last)
                  *out = static_cast<unsigned short>(f32_to_bf16_bits(__uint_as_float(v[j])));
            }
          }
          __syncwarp();
        }
        if (!none) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&drained[buf]);
          ++n;
        }
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
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, kColumns);
  }
}

template <typename TIn, int FORM>
int launch_typed(const ExpertArgs& a, cudaStream_t st) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  const int sms = device_sm_count();
  if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MR_ERR_CUDA;
  const auto kern = expert_matmul_split_kernel<TIn, FORM>;
  constexpr int smem = smem_of(Parts<TIn>::kN, FORM);
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return MR_ERR_CUDA;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  const bool mapped = FORM != EX_DGRAD && a.p2u != nullptr;
  SplitArgs g{};
  g.t = TcArgs{a.offsets, mapped ? a.p2u : nullptr, a.out, device_status_word(), a.T, a.P, a.E,
               a.N, a.D, mapped ? a.T : a.P, inverse_of(a.T)};
  if (g.t.status == nullptr) return MR_ERR_CUDA;
  g.a = FORM == EX_WGRAD ? a.a : a.b;
  g.b = FORM == EX_WGRAD ? a.b : a.a;
  g.out_f32 = a.out_dtype == DT_F32;
  const long long ta = ((FORM == EX_DGRAD ? a.D : a.N) + kTileRows - 1) / kTileRows;
  const long long tb = FORM == EX_WGRAD
                           ? static_cast<long long>(a.E) * ((a.D + kTileRows - 1) / kTileRows)
                           : static_cast<long long>(a.E < a.P ? a.E : a.P) + a.P / kTileRows;
  const long long most = ta * tb < sms ? ta * tb : sms;
  const cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(most)), dim3(kThreads),
                                      smem, st, g);
  return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

template <typename TIn>
int launch_type(int form, const ExpertArgs& a, cudaStream_t st) {
  return form == EX_FWD     ? launch_typed<TIn, EX_FWD>(a, st)
         : form == EX_DGRAD ? launch_typed<TIn, EX_DGRAD>(a, st)
                            : launch_typed<TIn, EX_WGRAD>(a, st);
}

}  // namespace

int launch_expert_matmul_split(int form, const ExpertArgs& a, cudaStream_t st) {
  return a.dtype == DT_F32 ? launch_type<float>(form, a, st)
                           : launch_type<unsigned short>(form, a, st);
}

}  // namespace moe_router
