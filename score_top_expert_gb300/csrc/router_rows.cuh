// A warp's share of a token's row, for the kernels that stream rows of [T, D] and
// [T K, D] tensors: the combination and the norms around a block.
#pragma once

#include "router_common.cuh"

namespace moe_router {

// N bytes (4, 8 or 16) from global to the thread's own place in shared memory, on their way
// until the thread waits for the group; zeros instead when not `valid`.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool valid = true) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                 "r"(valid ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(N),
                 "r"(valid ? N : 0) : "memory");
}

__device__ __forceinline__ void copies_commit_group() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Until at most PENDING of the thread's groups are on their way.
template <int PENDING>
__device__ __forceinline__ void copies_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// What a lane holds of a stretch of 32 kN columns of a row, as it was loaded (so
// that rows in flight take few registers), widened to fp32 when used.  BYTES is
// what one access takes: 16 where every row is 16-byte aligned, else 4 or 2, in
// four accesses 32 lanes apart, so that each is contiguous over the warp.
template <int DT, int BYTES>
struct Piece {
  static constexpr int kBytes = BYTES;
  static constexpr int kSize = DT == DT_F32 ? 4 : 2;
  static constexpr int kEach = BYTES / kSize;                          // columns per access
  static constexpr int kAccesses = BYTES == 16 ? 1 : 4;
  static constexpr int kN = kEach * kAccesses;
  static constexpr int kWords = BYTES == 16 ? 4 : kAccesses;
  uint32_t w[kWords];

  __device__ __forceinline__ static int column(int col0, int q, int lane) {
    return col0 + (q * 32 + lane) * kEach;
  }

  // The row starts at element `row` of base and has D columns.  STREAM: not kept
  // in L1 (the forward's rows; it costs the backward 2 to 6 %).
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* base, size_t row, int col0, int lane, int D) {
    const uint8_t* at = static_cast<const uint8_t*>(base) + row * kSize;
#pragma unroll
    for (int q = 0; q < kAccesses; ++q) {
      const int c = column(col0, q, lane);
      if (BYTES != 16) w[q] = 0u;
      if (c >= D) continue;
      if constexpr (BYTES == 16) {
        const uint4 t = get<STREAM>(reinterpret_cast<const uint4*>(at + c * kSize));
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      } else if constexpr (BYTES == 4) {
        w[q] = get<STREAM>(reinterpret_cast<const unsigned int*>(at + c * kSize));
      } else {
        w[q] = get<STREAM>(reinterpret_cast<const unsigned short*>(at + c * kSize));
      }
    }
  }

  // The same 16 bytes of the lane, to its place in shared memory and back.  (Two-byte
  // accesses have no asynchronous copy: they are stored there.)
  __device__ __forceinline__ static void load_async(uint32_t to, const void* base, size_t row,
                                                    int col0, int lane, int D) {
    const uint8_t* at = static_cast<const uint8_t*>(base) + row * kSize;
    if constexpr (BYTES == 16) {
      copy_async<16>(to, at + column(col0, 0, lane) * kSize);
    } else if constexpr (BYTES == 4) {
#pragma unroll
      for (int q = 0; q < kAccesses; ++q) {
        const int c = column(col0, q, lane);
        copy_async<4>(to + 4 * q, c < D ? at + c * kSize : at, c < D);
      }
    } else {
      Piece p;
      p.template load<true>(base, row, col0, lane, D);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(p.w[0]), "r"(p.w[1]),
                   "r"(p.w[2]), "r"(p.w[3]) : "memory");
    }
  }

  __device__ __forceinline__ void read(uint32_t from) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
  }

  template <bool STREAM, typename W>
  __device__ __forceinline__ static W get(const W* p) {
    return STREAM ? __ldcs(p) : __ldg(p);
  }

  // value j is column (j / kEach, j % kEach)
  __device__ __forceinline__ void widen(float (&v)[kN]) const {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = __uint_as_float(w[j]);
    } else if constexpr (BYTES == 2) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = bf16_bits_to_f32(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }

  __device__ __forceinline__ static void store(void* base, size_t row, int col0, int lane, int D,
                                               const float (&v)[kN]) {
    uint8_t* at = static_cast<uint8_t*>(base) + row * kSize;
    uint32_t u[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (DT == DT_F32) {
        u[j] = __float_as_uint(v[j]);
      } else if constexpr (BYTES == 2) {
        u[j] = f32_to_bf16_bits(v[j]);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
#pragma unroll
    for (int q = 0; q < kAccesses; ++q) {
      const int c = column(col0, q, lane);
      if (c >= D) continue;
      if constexpr (BYTES == 16)
        __stcs(reinterpret_cast<uint4*>(at + c * kSize), make_uint4(u[0], u[1], u[2], u[3]));
      else if constexpr (BYTES == 4)
        __stcs(reinterpret_cast<unsigned int*>(at + c * kSize), u[q]);
      else
        __stcs(reinterpret_cast<unsigned short*>(at + c * kSize), static_cast<unsigned short>(u[q]));
    }
  }
};

}  // namespace moe_router
