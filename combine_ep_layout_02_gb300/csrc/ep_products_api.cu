// ep_products_api.cu -- C entry points of the BF16 products, the dense layer
// and the gradient of the combine: argument checks on the host, then the
// launches.  Every check that can fail happens before anything is enqueued.
#include "ep_products.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return EP_OK;
    ep::record_cuda_error((int)e);
    return EP_ERR_CUDA;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline const uint16_t* bf16(const void* p) { return static_cast<const uint16_t*>(p); }

// A tile's last row and channel still have 32-bit coordinates.
constexpr int64_t kMaxRows = INT32_MAX - 256, kMaxWidth = 1 << 30;

// Sizes, segments and the word that the experts' products have in common.
// `weight_rows` per expert, `width` of every operand a multiple of 8.
int check_group(int64_t rows, int64_t weight_rows, int64_t width, int E, const int32_t* counts,
                const int32_t* offsets, int kind, int capacity, const uint32_t* status) {
    if (rows < 0 || rows > kMaxRows || weight_rows < 1 || weight_rows > kMaxWidth || width < 1 ||
        width > kMaxWidth || E < 1 || E > EP_MAX_EXPERTS || weight_rows > INT32_MAX / E)
        return EP_ERR_INVALID_ARG;
    if (kind != EP_LAYOUT_CONTIGUOUS && kind != EP_LAYOUT_MASKED) return EP_ERR_INVALID_ARG;
    if (kind == EP_LAYOUT_MASKED && (capacity < 0 || (int64_t)E * capacity > rows)) return EP_ERR_INVALID_ARG;
    if (weight_rows % 8 != 0 || width % 8 != 0) return EP_ERR_ALIGNMENT;
    if (!counts || (kind == EP_LAYOUT_CONTIGUOUS && !offsets)) return EP_ERR_INVALID_ARG;
    if (!aligned(counts, 4) || !aligned(offsets, 4) || !aligned(status, 4)) return EP_ERR_ALIGNMENT;
    return EP_OK;
}

bool known_type(int t) { return t == EP_TYPE_F32 || t == EP_TYPE_BF16; }

// Sizes and pointers that ep_linear and ep_linear_backward have in common.
int check_linear(int64_t M, int64_t K, int64_t N, int activation) {
    if (M < 0 || M > kMaxRows || K < 1 || K > kMaxWidth || N < 1 || activation < EP_ACT_NONE ||
        activation > EP_ACT_SWIGLU || N > kMaxWidth / (activation == EP_ACT_SWIGLU ? 2 : 1))
        return EP_ERR_INVALID_ARG;
    if (K % 8 != 0 || N % (activation == EP_ACT_SWIGLU ? 16 : 8) != 0) return EP_ERR_ALIGNMENT;
    return EP_OK;
}

ep::ProductArgs group_args(const void* a, const void* b, int64_t rows, int64_t N, int64_t K, int E,
                           const int32_t* counts, const int32_t* offsets, int kind, int capacity,
                           uint32_t* status) {
    ep::ProductArgs p = {};
    p.a = bf16(a);
    p.b = bf16(b);
    p.rows = rows;
    p.N = N;
    p.K = K;
    p.E = E;
    p.counts = counts;
    p.offsets = offsets;
    p.kind = kind;
    p.capacity = capacity;
    p.out_type = EP_TYPE_BF16;
    p.status = status;
    p.splits = 1;
    return p;
}

}  // namespace

extern "C" {

int ep_group_gemm(const void* a, int64_t rows, int64_t K, const void* w, int64_t N, int E,
                  const int32_t* expert_counts, const int32_t* expert_offsets, int kind,
                  int capacity, void* out, uint32_t* status, void* stream) {
    const int rc = check_group(rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    if (rc != EP_OK) return rc;
    if (rows == 0) return EP_OK;
    if (!a || !w || !out) return EP_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16)) return EP_ERR_ALIGNMENT;
    ep::ProductArgs p = group_args(a, w, rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    p.out = out;
    return cuda_status(ep::launch_product(p, ep::kForward, as_stream(stream)));
}

int ep_group_gemm_swiglu(const void* a, int64_t rows, int64_t K, const void* w13, int64_t I, int E,
                         const int32_t* expert_counts, const int32_t* expert_offsets, int kind,
                         int capacity, void* out, void* z, uint32_t* status, void* stream) {
    if (I < 1 || I > kMaxWidth / 2) return EP_ERR_INVALID_ARG;
    const int rc = check_group(rows, 2 * I, K, E, expert_counts, expert_offsets, kind, capacity, status);
    if (rc != EP_OK) return rc;
    if (I % 16 != 0) return EP_ERR_ALIGNMENT;
    if (rows == 0) return EP_OK;
    if (!a || !w13 || !out) return EP_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w13, 16) || !aligned(out, 16) || !aligned(z, 16)) return EP_ERR_ALIGNMENT;
    ep::ProductArgs p =
        group_args(a, w13, rows, 2 * I, K, E, expert_counts, expert_offsets, kind, capacity, status);
    p.activation = EP_ACT_SWIGLU;
    p.out = out;
    p.z = static_cast<uint16_t*>(z);
    return cuda_status(ep::launch_product(p, ep::kForward, as_stream(stream)));
}

int ep_group_gemm_dgrad(const void* dy, int64_t rows, int64_t N, const void* w, int64_t K, int E,
                        const int32_t* expert_counts, const int32_t* expert_offsets, int kind,
                        int capacity, void* dx, uint32_t* status, void* stream) {
    const int rc = check_group(rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    if (rc != EP_OK) return rc;
    if (rows == 0) return EP_OK;
    if (!dy || !w || !dx) return EP_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16)) return EP_ERR_ALIGNMENT;
    ep::ProductArgs p = group_args(dy, w, rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    p.out = dx;
    return cuda_status(ep::launch_product(p, ep::kInput, as_stream(stream)));
}

int ep_group_gemm_swiglu_dgrad(const void* dy, int64_t rows, int64_t H, const void* w2, int64_t I,
                               int E, const void* z, const int32_t* expert_counts,
                               const int32_t* expert_offsets, int kind, int capacity, void* dz,
                               uint32_t* status, void* stream) {
    if (I > kMaxWidth / 2) return EP_ERR_INVALID_ARG;
    const int rc = check_group(rows, H, I, E, expert_counts, expert_offsets, kind, capacity, status);
    if (rc != EP_OK) return rc;
    if (I % 16 != 0) return EP_ERR_ALIGNMENT;
    if (rows == 0) return EP_OK;
    if (!dy || !w2 || !z || !dz) return EP_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(w2, 16) || !aligned(z, 16) || !aligned(dz, 16)) return EP_ERR_ALIGNMENT;
    ep::ProductArgs p = group_args(dy, w2, rows, H, I, E, expert_counts, expert_offsets, kind, capacity, status);
    p.activation = EP_ACT_SWIGLU;
    p.out = dz;
    p.z = const_cast<uint16_t*>(bf16(z));
    return cuda_status(ep::launch_product(p, ep::kInput, as_stream(stream)));
}

int ep_group_gemm_wgrad(const void* dy, const void* x, int64_t rows, int64_t N, int64_t K, int E,
                        const int32_t* expert_counts, const int32_t* expert_offsets, int kind,
                        int capacity, const void* add, void* dw, int dw_type, uint32_t* status,
                        void* stream) {
    const int rc = check_group(rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    if (rc != EP_OK) return rc;
    if (!known_type(dw_type) || !dw || (rows > 0 && (!dy || !x))) return EP_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(add, 16)) return EP_ERR_ALIGNMENT;
    ep::ProductArgs p = group_args(dy, x, rows, N, K, E, expert_counts, expert_offsets, kind, capacity, status);
    p.add = add;
    p.out = dw;
    p.out_type = dw_type;
    if (E == 1) p.most = ep::weight_plan(rows, N, K, false).most;
    return cuda_status(ep::launch_product(p, ep::kWeight, as_stream(stream)));
}

size_t ep_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, int activation) {
    if (M <= EP_LINEAR_FEW_TOKENS || check_linear(M, K, N, activation) != EP_OK) return 0;
    const int64_t wide = activation == EP_ACT_SWIGLU ? 2 * N : N;
    const int splits = ep::dense_plan(M, K, N, activation == EP_ACT_SWIGLU, true).splits;
    return splits > 1 ? (size_t)splits * M * wide * 4 : 0;
}

int ep_linear(const void* x, int64_t M, int64_t K, const void* w, int64_t N, const void* bias,
              int bias_type, int activation, const void* residual, void* out, int out_type, void* z,
              uint32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_linear(M, K, N, activation);
    if (rc != EP_OK) return rc;
    const bool gated = activation == EP_ACT_SWIGLU;
    if (!known_type(out_type) || !known_type(bias_type) || (gated && out_type != EP_TYPE_BF16))
        return EP_ERR_INVALID_ARG;
    if (M == 0) return EP_OK;
    if (!x || !w || !out) return EP_ERR_INVALID_ARG;
    const size_t need = ep_linear_workspace_bytes(M, K, N, activation);
    if (need > 0 && (!workspace || workspace_bytes < need)) return EP_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(z, 16) || !aligned(residual, 16) ||
        !aligned(bias, bias_type == EP_TYPE_F32 ? 4 : 2) || !aligned(status, 4) || (need > 0 && !aligned(workspace, 16)))
        return EP_ERR_ALIGNMENT;
    ep::ProductArgs p = group_args(x, w, M, gated ? 2 * N : N, K, 1, nullptr, nullptr, 0, 0, status);
    p.activation = activation;
    p.bias = bias;
    p.bias_type = bias_type;
    p.residual = residual;
    p.out = out;
    p.out_type = out_type;
    p.z = static_cast<uint16_t*>(z);
    if (M <= EP_LINEAR_FEW_TOKENS) return cuda_status(ep::launch_linear_few(p, as_stream(stream)));
    const ep::DensePlan plan = ep::dense_plan(M, K, N, gated, true);
    p.most = plan.most;
    if (plan.splits == 1) return cuda_status(ep::launch_product(p, ep::kForward, as_stream(stream)));
    // the parts' sums as they are, all rows of w alike, then everything that follows a sum
    ep::ProductArgs part = group_args(x, w, M, p.N, K, 1, nullptr, nullptr, 0, 0, status);
    part.most = plan.most;
    part.splits = plan.splits;
    part.out = workspace;
    part.out_type = EP_TYPE_F32;
    cudaError_t err = ep::launch_product(part, ep::kForward, as_stream(stream));
    if (err == cudaSuccess)
        err = ep::launch_linear_finish(p, static_cast<const float*>(workspace), plan.splits, as_stream(stream));
    return cuda_status(err);
}

size_t ep_linear_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int activation) {
    if (check_linear(M, K, N, activation) != EP_OK) return 0;
    const int64_t wide = activation == EP_ACT_SWIGLU ? 2 * N : N;
    const int splits = ep::weight_plan(M, wide, K, true).splits;
    return splits > 1 ? (size_t)splits * wide * K * 4 : 0;
}

int ep_linear_backward(const void* dy, const void* x, const void* w, const void* z, int64_t M,
                       int64_t K, int64_t N, int activation, void* dz, void* dx, const void* add,
                       void* dw, int dw_type, float* dbias, uint32_t* status, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const int rc = check_linear(M, K, N, activation);
    if (rc != EP_OK) return rc;
    if (!known_type(dw_type)) return EP_ERR_INVALID_ARG;
    const bool act = activation != EP_ACT_NONE;
    if (act != (z != nullptr) || act != (dz != nullptr)) {
        if (M > 0 || !act) return EP_ERR_INVALID_ARG;
    }
    if (M > 0 && (!dy || (dx && !w) || (dw && !x))) return EP_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(dz, 16) ||
        !aligned(dx, 16) || !aligned(add, 16) || !aligned(dw, 16) || !aligned(dbias, 4) || !aligned(status, 4))
        return EP_ERR_ALIGNMENT;
    const int64_t wide = activation == EP_ACT_SWIGLU ? 2 * N : N;
    const size_t need = dw ? ep_linear_backward_workspace_bytes(M, K, N, activation) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return EP_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return EP_ERR_ALIGNMENT;
    cudaError_t err = cudaSuccess;
    if ((act && M > 0) || dbias)
        err = ep::launch_act_backward(bf16(dy), bf16(z), M, N, activation, static_cast<uint16_t*>(dz), dbias,
                                      as_stream(stream));
    const void* g = act ? dz : dy;
    if (err == cudaSuccess && dx && M > 0) {
        ep::ProductArgs p = group_args(g, w, M, wide, K, 1, nullptr, nullptr, 0, 0, status);
        p.out = dx;
        p.most = ep::dense_plan(M, wide, K, false, false).most;
        err = ep::launch_product(p, ep::kInput, as_stream(stream));
    }
    if (err == cudaSuccess && dw) {
        const ep::DensePlan plan = ep::weight_plan(M, wide, K, true);
        const bool split = plan.splits > 1;
        ep::ProductArgs p = group_args(g, x, M, wide, K, plan.splits, nullptr, nullptr, 0, 0, status);
        p.most = plan.most;
        p.add = split ? nullptr : add;
        p.out = split ? workspace : dw;
        p.out_type = split ? EP_TYPE_F32 : dw_type;
        if (split) p.part_rows = ((M + 63) / 64 + plan.splits - 1) / plan.splits * 64;  // whole blocks of the summed index
        err = ep::launch_product(p, ep::kWeight, as_stream(stream));
        if (err == cudaSuccess && split)
            err = ep::launch_weight_finish(static_cast<const float*>(workspace), plan.splits, wide * K, add, dw, dw_type,
                                           as_stream(stream));
    }
    return cuda_status(err);
}

int ep_combine_backward(const void* dout, const void* y, const float* topk_w, const int32_t* dst_row,
                        int64_t T, int64_t H, int k, int64_t rows, void* dy, float* dw,
                        uint32_t* status, void* stream) {
    if (T < 0 || H <= 0 || k < 1 || k > EP_MAX_TOPK || rows < 0 || rows > (int64_t)INT32_MAX + 1 ||
        T > (int64_t)INT32_MAX / k)
        return EP_ERR_INVALID_ARG;
    if (H % 8 != 0) return EP_ERR_ALIGNMENT;
    if (T == 0) return EP_OK;
    if (!dout || !topk_w || !dst_row || (rows > 0 && (!dy || (dw && !y)))) return EP_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(topk_w, 4) || !aligned(dw, 4) ||
        !aligned(dst_row, 4) || !aligned(status, 4))
        return EP_ERR_ALIGNMENT;
    return cuda_status(ep::launch_combine_backward(dout, y, topk_w, dst_row, T, H, k, rows, dy, dw, status,
                                                   as_stream(stream)));
}

}  // extern "C"
