// Tiled products of the linear layer's gradients, f16: dx = dz w, dw = dz^T x, alone and in one launch.

#include "ag_linear_device.h"

namespace ag {
namespace {

template <class C> LinearGemmFn pick(int form)
{
    switch (form) {
    case kFormNN: return ag_linear_gemm_kernel<false, kFormNN, AG_ACT_NONE, C>;
    case kFormTN: return ag_linear_gemm_kernel<false, kFormTN, AG_ACT_NONE, C>;
    default: return nullptr;
    }
}

}  // namespace

LinearGemmFn linear_gradient_f16(int form, int tile)
{
    switch (tile) {
    case kLinearTile256: return pick<Cfg256>(form);
    case kLinearTile128: return pick<Cfg128>(form);
    case kLinearTile256x128: return pick<Cfg256x128>(form);
    default: return nullptr;
    }
}

LinearInTurnFn linear_in_turn_f16(bool dx_first)
{
    return dx_first ? ag_linear_grads_in_turn_kernel<false, true, Cfg256> : ag_linear_grads_in_turn_kernel<false, false, Cfg256>;
}

LinearSideBySideFn linear_side_by_side_f16() { return ag_linear_grads_kernel<false, Cfg128>; }

}  // namespace ag
