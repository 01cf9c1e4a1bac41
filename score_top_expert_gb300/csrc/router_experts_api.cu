// C ABI of the expert-side operators: argument checks and the choice of
// kernel.  Declarations and contracts are in moe_router.h.
#include <climits>

#include "router_common.cuh"
#include "router_experts.cuh"

using namespace moe_router;

namespace {

bool known_dtype(int dtype) { return dtype == MR_F32 || dtype == MR_BF16; }

// Sizes shared by the products.  P rows, x rows by a map (T) or directly.
int check_product(int T, int P, int E, int N, int D, bool mapped) {
  if (P < 0 || E < 1 || N < 1 || D < 1) return MR_ERR_INVALID;
  if (mapped && (T < 0 || (T == 0 && P > 0))) return MR_ERR_INVALID;
  if (E > MR_MAX_EXPERTS || N > MR_MAX_FEATURES || D > MR_MAX_FEATURES)
    return MR_ERR_UNSUPPORTED;
  // an expert's rows and its row tiles are added up as ints
  if (P > MR_MAX_ROWS) return MR_ERR_UNSUPPORTED;
  return MR_OK;
}

// Rows up to which, and columns from which, the forward of bf16 operands takes
// the few-rows kernel.
constexpr int kFewRows = 36;
constexpr int kFewColumns = 512;

// Rows an expert, on average, up to which 8-bit operands take the few-rows kernel: 2.3 rows of
// 2048 -> 1024 take 56 us there and 70 in the tensor-core pipeline, 8 rows 124 and 128, of 4096
// -> 1024 115 and 131.
constexpr int kFewRowsW8 = 8;

// The few-rows kernel reads an expert's weights again for every eight of its rows.  In calls of
// more than 2^31 multiply-adds, where all rows in one expert would cost it 43 us or more, experts
// of more rows than a tile holds are left to the tensor-core pipeline, in a launch of its own.
// 16384 rows, 2304 experts of 1024 x 1024, us by both, the few-rows kernel alone, the pipeline alone:
// evenly 536, 532, 595; by a power law 455, 563, 509; half of them in one expert 443, 580, 601; all
// of them 57, 331, 54.  1024 rows, 128 experts of 4096 -> 1024, where a long tile has nothing beside
// it, by both and the few-rows kernel: 109, 107; 132, 124; 125, 127; 29, 74.  From 32 rows instead:
// 411 by the power law at 2304 experts, but 123 for 107 with slightly uneven ones at 4096 -> 1024.
constexpr int kHotRowsW8 = 128;
constexpr double kHotWorkW8 = 2147483648.0;

int run_product(int form, const ExpertArgs& a, mr_stream_t stream) {
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // One token's rows: 4 experts of 1024 x 1024 take 10 us here and 14 us in the
  // tensor-core pipeline, 2 of 4096 x 4096 22 and 29; 28 or more experts of 1024
  // x 1024 the same in both.  Rows too short to pay for the staging of x take
  // longer: 28 experts of 1736 x 88 22 us against 16.
  if (form == EX_FWD && a.P <= kFewRows && a.D >= kFewColumns && expert_matmul_few_ok(a))
    return launch_expert_matmul_few(a, st);
  return expert_matmul_tc_ok(form, a) ? launch_expert_matmul_tc(form, a, st)
                                      : launch_expert_matmul_split(form, a, st);
}

}  // namespace

extern "C" {

int router_expert_matmul(const void* x, mr_dtype dtype, const void* weight,
                         const int32_t* expert_first_token_offset,
                         const int32_t* permuted_to_unpermuted, int T, int P, int E, int N, int D,
                         void* out, mr_dtype out_dtype, mr_stream_t stream) {
  if (!known_dtype(dtype) || !known_dtype(out_dtype)) return MR_ERR_INVALID;
  const int rc = check_product(T, P, E, N, D, permuted_to_unpermuted != nullptr);
  if (rc != MR_OK) return rc;
  if (P == 0) return MR_OK;
  if (x == nullptr || weight == nullptr || expert_first_token_offset == nullptr ||
      out == nullptr)
    return MR_ERR_INVALID;
  const ExpertArgs a{x, weight, expert_first_token_offset, permuted_to_unpermuted, out, T, P, E,
                     N, D, dtype, out_dtype};
  return run_product(EX_FWD, a, stream);
}

int router_expert_matmul_bwd_input(const void* grad_out, mr_dtype dtype, const void* weight,
                                   const int32_t* expert_first_token_offset, int P, int E, int N,
                                   int D, void* grad_x, mr_dtype out_dtype, mr_stream_t stream) {
  if (!known_dtype(dtype) || !known_dtype(out_dtype)) return MR_ERR_INVALID;
  const int rc = check_product(0, P, E, N, D, false);
  if (rc != MR_OK) return rc;
  if (P == 0) return MR_OK;
  if (grad_out == nullptr || weight == nullptr || expert_first_token_offset == nullptr ||
      grad_x == nullptr)
    return MR_ERR_INVALID;
  const ExpertArgs a{grad_out, weight, expert_first_token_offset, nullptr, grad_x, 0, P, E, N, D,
                     dtype, out_dtype};
  return run_product(EX_DGRAD, a, stream);
}

int router_expert_matmul_bwd_weight(const void* grad_out, mr_dtype dtype, const void* x,
                                    const int32_t* expert_first_token_offset,
                                    const int32_t* permuted_to_unpermuted, int T, int P, int E,
                                    int N, int D, void* grad_weight, mr_dtype out_dtype,
                                    mr_stream_t stream) {
  if (!known_dtype(dtype) || !known_dtype(out_dtype)) return MR_ERR_INVALID;
  const int rc = check_product(T, P, E, N, D, permuted_to_unpermuted != nullptr);
  if (rc != MR_OK) return rc;
  if (grad_weight == nullptr || expert_first_token_offset == nullptr) return MR_ERR_INVALID;
  if (P > 0 && (grad_out == nullptr || x == nullptr)) return MR_ERR_INVALID;
  const ExpertArgs a{grad_out, x, expert_first_token_offset, permuted_to_unpermuted, grad_weight,
                     T, P, E, N, D, dtype, out_dtype};
  return run_product(EX_WGRAD, a, stream);
}

int router_expert_matmul_w4(const void* x, const uint8_t* qweight, const void* scales,
                            const uint8_t* zeros, int group_size,
                            const int32_t* expert_first_token_offset,
                            const int32_t* permuted_to_unpermuted, int T, int P, int E, int N,
                            int D, void* out, mr_dtype out_dtype, mr_stream_t stream) {
  if (!known_dtype(out_dtype)) return MR_ERR_INVALID;
  const int rc = check_product(T, P, E, N, D, permuted_to_unpermuted != nullptr);
  if (rc != MR_OK) return rc;
  if (group_size < 1 || D % group_size != 0) return MR_ERR_INVALID;
  if (group_size != 32 && group_size != 64 && group_size != 128) return MR_ERR_UNSUPPORTED;
  if (P == 0) return MR_OK;
  if (x == nullptr || qweight == nullptr || scales == nullptr ||
      expert_first_token_offset == nullptr || out == nullptr)
    return MR_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(qweight)) & 15u) != 0)
    return MR_ERR_INVALID;
  const W4Args a{x, qweight, scales, zeros, expert_first_token_offset, permuted_to_unpermuted,
                 out, T, P, E, N, D, group_size, out_dtype};
  return launch_expert_matmul_w4(a, reinterpret_cast<cudaStream_t>(stream));
}

int router_expert_matmul_w8(const int8_t* x, const float* x_scales, const int8_t* weight,
                            const float* weight_scales, const int32_t* expert_first_token_offset,
                            const int32_t* permuted_to_unpermuted, int T, int P, int E, int N,
                            int D, void* out, mr_dtype out_dtype, mr_stream_t stream) {
  if (!known_dtype(out_dtype)) return MR_ERR_INVALID;
  const int rc = check_product(T, P, E, N, D, permuted_to_unpermuted != nullptr);
  if (rc != MR_OK) return rc;
  if (P == 0) return MR_OK;
  if (x == nullptr || x_scales == nullptr || weight == nullptr || weight_scales == nullptr ||
      expert_first_token_offset == nullptr || out == nullptr)
    return MR_ERR_INVALID;
  const W8Args a{x, x_scales, weight, weight_scales, expert_first_token_offset,
                 permuted_to_unpermuted, out, T, P, E, N, D, out_dtype, 0, INT_MAX};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (P > kFewRowsW8 * static_cast<long long>(E) || !expert_matmul_w8_few_ok(a))
    return launch_expert_matmul_w8_tc(a, st);
  if (P > kHotRowsW8 && 1.0 * P * N * D > kHotWorkW8) {
    W8Args hot = a, rest = a;
    hot.least = kHotRowsW8 + 1;
    rest.most = kHotRowsW8;
    const int code = launch_expert_matmul_w8_tc(hot, st);
    return code != MR_OK ? code : launch_expert_matmul_w8_few(rest, st);
  }
  return launch_expert_matmul_w8_few(a, st);
}

// Sizes of the combination: every row index stays below 2^31.
static int check_combine(int dtype, int T, int K, int D) {
  if (!known_dtype(dtype)) return MR_ERR_INVALID;
  if (T < 0 || K < 1 || D < 1 || static_cast<long long>(T) * K > INT_MAX) return MR_ERR_INVALID;
  if (K > MR_MAX_TOPK || D > MR_MAX_FEATURES) return MR_ERR_UNSUPPORTED;
  return MR_OK;
}

int router_combine_fwd(const void* expert_out, mr_dtype dtype,
                       const int32_t* unpermuted_to_permuted, const float* topk_weights,
                       int ld_weights, int T, int K, int D, void* out, mr_stream_t stream) {
  const int rc = check_combine(dtype, T, K, D);
  if (rc != MR_OK) return rc;
  if (topk_weights != nullptr && ld_weights < K) return MR_ERR_INVALID;
  if (T == 0) return MR_OK;
  if (expert_out == nullptr || unpermuted_to_permuted == nullptr || out == nullptr)
    return MR_ERR_INVALID;
  CombineArgs a{};
  a.z = expert_out;
  a.u2p = unpermuted_to_permuted;
  a.weights = topk_weights;
  a.out = out;
  a.ld_w = ld_weights;
  a.T = T; a.K = K; a.D = D;
  a.dtype = dtype;
  return launch_combine_fwd(a, reinterpret_cast<cudaStream_t>(stream));
}

int router_combine_bwd(const void* grad_out, mr_dtype dtype,
                       const int32_t* unpermuted_to_permuted, const void* expert_out,
                       const float* topk_weights, int ld_weights, int T, int K, int D,
                       void* grad_expert_out, float* grad_weights, mr_stream_t stream) {
  const int rc = check_combine(dtype, T, K, D);
  if (rc != MR_OK) return rc;
  if (topk_weights != nullptr && ld_weights < K) return MR_ERR_INVALID;
  if (T == 0) return MR_OK;
  if (grad_out == nullptr || unpermuted_to_permuted == nullptr || grad_expert_out == nullptr ||
      (grad_weights != nullptr && expert_out == nullptr))
    return MR_ERR_INVALID;
  CombineArgs a{};
  a.z = expert_out;
  a.gy = grad_out;
  a.u2p = unpermuted_to_permuted;
  a.weights = topk_weights;
  a.out = grad_expert_out;
  a.grad_weights = grad_weights;
  a.ld_w = ld_weights;
  a.T = T; a.K = K; a.D = D;
  a.dtype = dtype;
  return launch_combine_bwd(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
