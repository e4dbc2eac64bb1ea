// Internal interface between the linear layer's host code (ag_linear_host.cpp)
// and its kernels (ag_linear.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ag {

// What happens to a product's fp32 element before it is stored.
struct LinearEpilogue {
    const uint16_t* bias;       // per column, or null
    const uint16_t* residual;   // or null
    uint16_t* z;                // pre-activation output, or null
    void* out;
    int64_t ldr, ldz, ldo;
    int32_t act;                // ag_act_t
    int32_t out_f32;            // out holds fp32, else the operands' type
    int32_t accumulate;         // out += instead of out =
    int32_t reserved;
};

// db(n) (+)= sum over parts of sums(part, n).
struct LinearBiasGradArgs {
    const float* sums;
    void* db;
    int64_t parts, N;
    int32_t kind;               // of db: 0 f16, 1 bf16, 2 f32
    int32_t accumulate;
};

// out(i, j) = epilogue(sum_r A(i, r) B(j, r)).
struct LinearGemmArgs {
    const uint16_t* A;          // element (i, r) at A[i*lda + r], or A[r*lda + i] (transposed kernels)
    const uint16_t* B;          // element (j, r) at B[j*ldb + r], or B[r*ldb + j]
    int64_t lda, ldb;
    int64_t I, J, R;
    int32_t tiles_i, tiles_j;
    int32_t stages;             // 64-wide steps of the reduction, at least 1
    int32_t full_tiles;         // tiles that one workgroup computes whole, the first of the order
    int32_t splits;             // parts of the other tiles' reductions, split_stages steps each (the last may be shorter)
    int32_t split_stages;
    int32_t heavy;              // > 0: whole tiles, common_rounds rounds on all workgroups and the rest on those from
    int32_t common_rounds;      //   number `heavy` on
    float* partial;             // fp32 tile (part, tail tile)
    LinearEpilogue epi;
    LinearBiasGradArgs db;      // gradient kernels: the bias gradient's sum on the side (db.db null: none)
};

enum LinearTile { kLinearTile256 = 0, kLinearTile128 = 1, kLinearTile256x128 = 2, kLinearTiles = 3 };
enum LinearForm { kFormNT = 0, kFormNN = 1, kFormTN = 2 };   // y, dx, dw

hipError_t launch_linear_gemm(const LinearGemmArgs& a, int bf16, int form, int tile, int programs, hipStream_t stream);
// The tiled kernels, by type (each in a source of its own); null where there is none.
using LinearGemmFn = void (*)(LinearGemmArgs);
LinearGemmFn linear_forward_f16(int act, int tile);
LinearGemmFn linear_forward_bf16(int act, int tile);
LinearGemmFn linear_gradient_f16(int form, int tile);
LinearGemmFn linear_gradient_bf16(int form, int tile);

// Joins the parts of the cut tiles in order and applies the epilogue.
hipError_t launch_linear_join(const LinearGemmArgs& a, int bf16, int form, int tile, hipStream_t stream);

// Row streaming: out(m, n) for few rows m of x (I = N, J = M <= kLinearStreamRows).
constexpr int kLinearStreamRows = 32;
struct LinearStreamArgs {
    const uint16_t* x;
    const uint16_t* w;
    int64_t ldx, ldw;
    int64_t M, N, K;
    LinearEpilogue epi;
};
hipError_t launch_linear_stream(const LinearStreamArgs& a, int bf16, int cus, hipStream_t stream);

// Copies rows to aligned rows (ld_dst a multiple of 8).
hipError_t launch_linear_pack(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                              int64_t cols, hipStream_t stream);

// dz = dy * act'(z), rounded, what the rounding leaves, and the column sums of the unrounded dz over row blocks.
struct LinearSlopeArgs {
    const uint16_t* dy;
    const uint16_t* z;          // null when act is none
    uint16_t* dz;               // null: not stored
    uint16_t* dz_rest;          // dz's second term, dz - (its rounded value), rounded; or null
    float* sums;                // ceil(M / rows) rows of N, or null
    int64_t lddy, ldz, lddz;
    int64_t M, N;
    int32_t act;
    int32_t rows;               // of one workgroup and partial column sum
};
hipError_t launch_linear_slope(const LinearSlopeArgs& a, int bf16, hipStream_t stream);
hipError_t launch_linear_bias_grad(const LinearBiasGradArgs& a, hipStream_t stream);

using LinearInTurnFn = void (*)(LinearGemmArgs, LinearGemmArgs, LinearBiasGradArgs);
LinearInTurnFn linear_in_turn_f16(bool dx_first);
LinearInTurnFn linear_in_turn_bf16(bool dx_first);
using LinearSideBySideFn = void (*)(LinearGemmArgs, LinearGemmArgs, int, int, LinearBiasGradArgs);
LinearSideBySideFn linear_side_by_side_f16();
LinearSideBySideFn linear_side_by_side_bf16();

// dx, dw and (db.db set) db in turn on `programs` workgroups, in 256 x 256 tiles, none cut.
hipError_t launch_linear_grads_in_turn(const LinearGemmArgs& dx, const LinearGemmArgs& dw, bool dx_first, int programs,
                                       const LinearBiasGradArgs& db, int bf16, hipStream_t stream);

// dx, dw and (db.db set) db in one launch of 128 x 128 tiles, none cut.
hipError_t launch_linear_grads(const LinearGemmArgs& dx, const LinearGemmArgs& dw, int dx_programs, int dw_programs,
                               const LinearBiasGradArgs& db, int bf16, hipStream_t stream);

// Tile shape and threads of a tile configuration (host-only).
void linear_tile_shape(int tile, int* tm, int* tn, int* threads);

}  // namespace ag
