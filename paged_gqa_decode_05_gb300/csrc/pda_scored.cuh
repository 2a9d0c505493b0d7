// pda_scored.cuh -- the scored instances of the split kernels, bf16 and 8-bit
// (Scoring in pda_params.h).
#pragma once

#include <type_traits>

#include "pda_quant.cuh"
#include "pda_scored.h"

namespace pda {

// visit(rows of a stage, mode) for a bf16 form, visit(mode, fine) for an 8-bit one, or `none`.
template <int N>
using Int = std::integral_constant<int, N>;
template <int D, class R, class Visit>
R visit_scored_bf16(const ScoredForm& f, R none, const Visit& visit) {
    if (f.st == 64) {
        if (f.rows == 1) return visit(Int<64>(), Int<kScored>());
        if (f.rows == 8) return visit(Int<64>(), Int<kScoredMulti>());
        if constexpr (D <= 128) return f.rows == 16 ? visit(Int<64>(), Int<kScoredRows16>()) : visit(Int<64>(), Int<kScoredRows32>());
    }
    if constexpr (D == 256) {
        if (f.st == 32 && f.rows == 1) return visit(Int<32>(), Int<kScored>());
        if (f.st == 32 && f.rows == 8) return visit(Int<32>(), Int<kScoredMulti>());
    }
    return none;
}
template <class R, class Visit>
R visit_scored_quant(const ScoredForm& f, const Visit& visit) {
    if (f.fine) return f.rows > 1 ? visit(Int<kScoredMulti>(), std::true_type()) : visit(Int<kScored>(), std::true_type());
    return f.rows > 1 ? visit(Int<kScoredMulti>(), std::false_type()) : visit(Int<kScored>(), std::false_type());
}

template <int D>
ScoredShape scored_shape_bf16(const ScoredForm& f) {
    return visit_scored_bf16<D>(f, ScoredShape{}, [](auto rows, auto mode) -> ScoredShape {
        using C = Cfg<D, rows(), mode()>;
        return {reinterpret_cast<const void*>(&split_kernel<D, rows(), mode()>), C::kThreads, C::kST, C::kStages,
                (uint32_t)C::kStageBytes, max_launch_rows(mode())};
    });
}
template <int D>
cudaError_t launch_scored_bf16(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return visit_scored_bf16<D>(f, cudaErrorInvalidValue, [&](auto rows, auto mode) -> cudaError_t {
        return launch_split_mode<D, rows(), mode()>(p, grid, smem, stream);
    });
}

template <int D, int FMT>
ScoredShape scored_shape_quant(const ScoredForm& f) {
    return visit_scored_quant<ScoredShape>(f, [](auto mode, auto fine) -> ScoredShape {
        using C = QuantCfg<D, 1>;
        return {reinterpret_cast<const void*>(&quant_split_kernel<D, FMT, 1, mode(), fine()>), C::kThreads, C::kST,
                C::kStages, (uint32_t)C::kStageBytes, max_launch_rows(mode())};
    });
}
template <int D, int FMT>
cudaError_t launch_scored_quant(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return visit_scored_quant<cudaError_t>(f, [&](auto mode, auto fine) -> cudaError_t {
        return launch_quant_as<D, FMT, 1, mode(), fine()>(p, grid, smem, stream);
    });
}

}  // namespace pda
