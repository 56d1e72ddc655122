// adamw32.hip - the AdamW step's kernel instances with states of 32 bits.
#include "adamw_launch.hpp"

namespace dytb {

void adamw_launch32(const AdamArgs& a, int pdt, int gdt, bool master, unsigned grid, hipStream_t s) {
    adamw_types(pdt, gdt, [&](auto* p, auto* g) {
        using TP = std::remove_pointer_t<decltype(p)>;
        using TG = std::remove_pointer_t<decltype(g)>;
        if constexpr (!std::is_same_v<TP, float>) {
            if (master) return adamw_kernel<TP, TG, true><<<grid, kAdamThreads, 0, s>>>(a);
        }
        adamw_kernel<TP, TG, false><<<grid, kAdamThreads, 0, s>>>(a);
    });
}

}  // namespace dytb
