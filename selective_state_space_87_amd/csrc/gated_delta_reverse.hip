// Gated delta rule backward: launches of the walk back over the chunks.
#include "gated_delta_reverse.h"

namespace ssm {

int launch_gdr_reverse(const GatedDeltaBwdArgs& a, const GdrWork& ws, int64_t chunks, bool vec, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int n = static_cast<int>(chunks);
  const auto types = [&](auto np, auto bf16) {
    constexpr int NP = decltype(np)::value;
    constexpr bool BF16 = decltype(bf16)::value;
    vec ? gdr_launch_reverse_nw<NP, BF16, true>(a, ws, n, st) : gdr_launch_reverse_nw<NP, BF16, false>(a, ws, n, st);
  };
  const auto width = [&](auto np) {
    a.f.in_bf16 ? types(np, std::true_type{}) : types(np, std::false_type{});
  };
  if (a.f.dstate <= 64) {
    width(std::integral_constant<int, 64>{});
  } else {
    width(std::integral_constant<int, 128>{});
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace ssm
