// Tiled products of the linear layer, f16: y = act(x w^T + bias) + residual.

#include "ag_linear_device.h"

namespace ag {
namespace {

template <class C> LinearGemmFn pick(int act)
{
    switch (act) {
    case AG_ACT_NONE: return ag_linear_gemm_kernel<false, kFormNT, AG_ACT_NONE, C>;
    case AG_ACT_RELU: return ag_linear_gemm_kernel<false, kFormNT, AG_ACT_RELU, C>;
    case AG_ACT_GELU: return ag_linear_gemm_kernel<false, kFormNT, AG_ACT_GELU, C>;
    case AG_ACT_GELU_TANH: return ag_linear_gemm_kernel<false, kFormNT, AG_ACT_GELU_TANH, C>;
    case AG_ACT_SILU: return ag_linear_gemm_kernel<false, kFormNT, AG_ACT_SILU, C>;
    default: return nullptr;
    }
}

}  // namespace

LinearGemmFn linear_forward_f16(int act, int tile)
{
    switch (tile) {
    case kLinearTile256: return pick<Cfg256>(act);
    case kLinearTile128: return pick<Cfg128>(act);
    case kLinearTile256x128: return pick<Cfg256x128>(act);
    default: return nullptr;
    }
}

}  // namespace ag
