// adamw8.hip - the AdamW step's kernel instances with states of 8 bits.
#include "adamw_launch.hpp"

namespace dytb {

void adamw_launch8(const AdamArgs& a, int pdt, int gdt, bool master, unsigned grid, hipStream_t s) {
    adamw_types(pdt, gdt, [&](auto* p, auto* g) {
        using TP = std::remove_pointer_t<decltype(p)>;
        using TG = std::remove_pointer_t<decltype(g)>;
        const auto run = [&](auto with_master) {
            constexpr bool MASTER = decltype(with_master)::value;
            if (a.seeded) adamw8_kernel<TP, TG, MASTER, true><<<grid, kAdamThreads, 0, s>>>(a);
            else adamw8_kernel<TP, TG, MASTER, false><<<grid, kAdamThreads, 0, s>>>(a);
        };
        if constexpr (!std::is_same_v<TP, float>) {
            if (master) return run(std::true_type{});
        }
        run(std::false_type{});
    });
}

}  // namespace dytb
