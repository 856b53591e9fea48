// What the gated norm's two directions share (norm_gated.hip has the formulas).
#pragma once

#include <type_traits>

#include "block_internal.h"
#include "norm_rows.h"

namespace ssm {

enum Gate { kNone, kBefore, kAfter };

// Host: calls f(io element, gate, whether the stores pass by the caches) for a
// call over so many matrices.  The last is taken for whole pieces where the
// matrices pass the last-level cache together.  (16384 x 5120 in 8 groups with
// two checkpoints: forward 139 -> 123 us, backward 137 -> 133; 32768 x 5120:
// 176 -> 168.  Nontemporal loads took that backward from 138 to 216 us; the
// residual norm gained nothing by either.)
template <typename RS, typename F>
void for_gate(const NormShape& s, bool gated, int matrices, F&& f) {
    const bool past = s.M * s.W * (s.io == SSM_BF16 ? 2 : 4) * matrices > kStreamBytes;
    auto typed = [&](auto t) {
        auto streamed = [&](auto gate) {
            if constexpr (RS::NC == 1 && RS::RAGGED == kWhole && gate.value != kNone)
                if (past) return f(t, gate, std::true_type());
            f(t, gate, std::false_type());
        };
        if (!gated) streamed(std::integral_constant<Gate, kNone>());
        else if (s.after) streamed(std::integral_constant<Gate, kAfter>());
        else streamed(std::integral_constant<Gate, kBefore>());
    };
    if (s.io == SSM_BF16) typed(bf16_t());
    else typed(float());
}

}  // namespace ssm
