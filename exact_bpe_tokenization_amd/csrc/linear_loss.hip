// linear_loss.hip -- next-token cross entropy straight from hidden states: entry points and their checks (linear_loss.h).
#include "linear_loss.h"

namespace tt {
template <> void linear_loss<float>(const Call &c, const Sizes &z, uint8_t *ws, hipStream_t s) { enqueue<float>(c, z, ws, s); }
extern template void linear_loss<_Float16>(const Call &, const Sizes &, uint8_t *, hipStream_t);
extern template void linear_loss<__bf16>(const Call &, const Sizes &, uint8_t *, hipStream_t);

namespace {

constexpr uint32_t MAX_ROWS = TOKTIER_MAX_LINEAR_ROWS, MAX_DIM = TOKTIER_MAX_LINEAR_DIM;

int run(const Call &c, void *workspace, uint64_t workspace_bytes, void *stream)
{
    const bool forward = !c.lse_in, grads = c.grad_hidden || c.grad_weight;
    if (!elem_size(c.type) || c.n_vocab == 0 || c.n_vocab > TOKTIER_MAX_VOCAB || c.dim == 0 || c.dim > MAX_DIM || c.n_rows > MAX_ROWS)
        return TOKTIER_E_INVALID_ARG;
    if (c.grad_weight && c.grad_weight_type != c.type && c.grad_weight_type != TOKTIER_F32) return TOKTIER_E_INVALID_ARG;
    if (c.n_rows == 0 && (!c.grad_weight || c.accumulate)) return TOKTIER_OK;
    const Sizes z = sizes_of(c.n_rows, c.n_vocab, c.dim, c.type, grads);
    struct Area {
        const void *p;
        uint64_t n;
    };
    Area in[8], out[8];
    int n_in = 0, n_out = 0;
    auto matrix = [&](const void *p, int type, uint64_t r, uint64_t cols, uint64_t stride, Area *list, int &k) {
        if (r == 0) return true;
        list[k++] = Area{p, extent(type, r, cols, stride)};
        return matrix_ok(p, type, r, cols, stride);
    };
    auto vector = [&](const void *p, bool needed, Area *list, int &k) {
        if (c.n_rows == 0) return true;
        if (p) list[k++] = Area{p, 4ull * c.n_rows};
        return (p || !needed) && aligned4(p);
    };
    if (!matrix(c.hidden, c.type, c.n_rows, c.dim, c.hidden_stride, in, n_in) ||
        !matrix(c.weight, c.type, c.n_vocab, c.dim, c.weight_stride, in, n_in) || !vector(c.targets, true, in, n_in) ||
        !vector(c.grad_loss, false, in, n_in))
        return TOKTIER_E_INVALID_ARG;
    if (forward ? !vector(c.loss, true, out, n_out) || !vector(c.lse, true, out, n_out) : !vector(c.lse_in, true, in, n_in))
        return TOKTIER_E_INVALID_ARG;
    if (c.grad_hidden && !matrix(c.grad_hidden, c.type, c.n_rows, c.dim, c.grad_hidden_stride, out, n_out)) return TOKTIER_E_INVALID_ARG;
    if (c.grad_weight && !matrix(c.grad_weight, c.grad_weight_type, c.n_vocab, c.dim, c.grad_weight_stride, out, n_out)) return TOKTIER_E_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u)) return TOKTIER_E_INVALID_ARG;
    if (workspace_bytes < z.total) return TOKTIER_E_CAPACITY;
    out[n_out++] = Area{workspace, z.total};
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (!apart(out[i].p, out[i].n, in[k].p, in[k].n)) return TOKTIER_E_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (!apart(out[i].p, out[i].n, out[k].p, out[k].n)) return TOKTIER_E_INVALID_ARG;
    }
    with_type(c.type, [&](auto t) { linear_loss<decltype(t)>(c, z, (uint8_t *)workspace, (hipStream_t)stream); });
    return hip_status(hipGetLastError());
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int toktier_linear_cross_entropy_workspace_bytes(uint32_t n_rows, uint32_t n_vocab, uint32_t dim, int type, int grads,
                                                            uint64_t *out_bytes)
{
    if (!out_bytes || !elem_size(type) || n_vocab == 0 || n_vocab > TOKTIER_MAX_VOCAB || dim == 0 || dim > MAX_DIM || n_rows > MAX_ROWS)
        return TOKTIER_E_INVALID_ARG;
    *out_bytes = sizes_of(n_rows, n_vocab, dim, type, grads != 0).total;
    return TOKTIER_OK;
}

extern "C" int toktier_linear_cross_entropy(const void *hidden, int type, uint32_t n_rows, uint32_t dim, uint64_t hidden_stride,
                                            const void *weight, uint32_t n_vocab, uint64_t weight_stride, const uint32_t *targets, float *loss,
                                            float *lse, const float *grad_loss, float grad_scale, void *grad_hidden,
                                            uint64_t grad_hidden_stride, void *grad_weight, int grad_weight_type, uint64_t grad_weight_stride,
                                            int accumulate, void *workspace, uint64_t workspace_bytes, void *stream)
{
    return run(Call{hidden, weight, type, n_rows, n_vocab, dim, hidden_stride, weight_stride, targets, loss, lse, nullptr, grad_loss, grad_scale,
                    grad_hidden, grad_hidden_stride, grad_weight, grad_weight_type, grad_weight_stride, accumulate},
               workspace, workspace_bytes, stream);
}

extern "C" int toktier_linear_cross_entropy_backward(const void *hidden, int type, uint32_t n_rows, uint32_t dim, uint64_t hidden_stride,
                                                     const void *weight, uint32_t n_vocab, uint64_t weight_stride, const uint32_t *targets,
                                                     const float *lse, const float *grad_loss, float grad_scale, void *grad_hidden,
                                                     uint64_t grad_hidden_stride, void *grad_weight, int grad_weight_type,
                                                     uint64_t grad_weight_stride, int accumulate, void *workspace, uint64_t workspace_bytes,
                                                     void *stream)
{
    if (!lse && n_rows) return TOKTIER_E_INVALID_ARG;
    static const float nothing = 0.f;   // of no rows
    return run(Call{hidden, weight, type, n_rows, n_vocab, dim, hidden_stride, weight_stride, targets, nullptr, nullptr, lse ? lse : &nothing,
                    grad_loss, grad_scale, grad_hidden, grad_hidden_stride, grad_weight, grad_weight_type, grad_weight_stride, accumulate},
               workspace, workspace_bytes, stream);
}
