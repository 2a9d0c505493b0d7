// pda_scored.cuh -- kScored instances of the split kernels, bf16 and 8-bit:
// the n8 forms with the score changes, score outputs and the join of a shared
// prefix's state (Scoring in pda_params.h).
#pragma once

#include "pda_quant.cuh"
#include "pda_scored.h"

namespace pda {

// visit(kernel instance) or `none`.
template <int D, class R, class Visit>
R visit_scored(int st, int format, bool fine, R none, const Visit& visit) {
    switch (format) {
        case kBf16:
            if (st == 64) return visit(std::integral_constant<int, 64>(), std::integral_constant<int, kBf16>(), std::false_type());
            if constexpr (D == 256)
                if (st == 32) return visit(std::integral_constant<int, 32>(), std::integral_constant<int, kBf16>(), std::false_type());
            return none;
        case kE4m3:
            return fine ? visit(std::integral_constant<int, 0>(), std::integral_constant<int, kE4m3>(), std::true_type())
                        : visit(std::integral_constant<int, 0>(), std::integral_constant<int, kE4m3>(), std::false_type());
        case kInt8:
            return fine ? visit(std::integral_constant<int, 0>(), std::integral_constant<int, kInt8>(), std::true_type())
                        : visit(std::integral_constant<int, 0>(), std::integral_constant<int, kInt8>(), std::false_type());
        default: return none;
    }
}

template <int D>
ScoredShape scored_shape_of(int st, int format, bool fine) {
    return visit_scored<D>(st, format, fine, ScoredShape{}, [](auto rows, auto fmt, auto f) -> ScoredShape {
        if constexpr (fmt() == kBf16) {
            using C = Cfg<D, rows(), kScored>;
            return {reinterpret_cast<const void*>(&split_kernel<D, rows(), kScored>), C::kThreads, C::kST, C::kStages,
                    (uint32_t)C::kStageBytes};
        } else {
            using C = QuantCfg<D, 1>;
            return {reinterpret_cast<const void*>(&quant_split_kernel<D, fmt(), 1, kScored, f()>), C::kThreads, C::kST,
                    C::kStages, (uint32_t)C::kStageBytes};
        }
    });
}

template <int D>
cudaError_t launch_scored_of(int st, int format, bool fine, const QuantParams& p, int grid, size_t smem,
                             cudaStream_t stream) {
    return visit_scored<D>(st, format, fine, cudaErrorInvalidValue, [&](auto rows, auto fmt, auto f) -> cudaError_t {
        if constexpr (fmt() == kBf16) return launch_split_mode<D, rows(), kScored>(p, grid, smem, stream);
        else return launch_quant_as<D, fmt(), 1, kScored, f()>(p, grid, smem, stream);
    });
}

}  // namespace pda
