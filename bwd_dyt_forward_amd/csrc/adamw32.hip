// adamw32.hip - the AdamW step's kernel instances with states of 32 bits.
#include "adamw_launch.hpp"

namespace dytb {

void adamw_launch32(const AdamArgs& a, int pdt, int gdt, bool master, bool stream_past, unsigned grid, hipStream_t s) {
    adamw_types(pdt, gdt, [&](auto* p, auto* g) {
        using TP = std::remove_pointer_t<decltype(p)>;
        using TG = std::remove_pointer_t<decltype(g)>;
        const auto run = [&](auto with_master) {
            constexpr bool MASTER = decltype(with_master)::value;
            if (stream_past) adamw_kernel<TP, TG, MASTER, true><<<grid, kAdamThreads, 0, s>>>(a);
            else adamw_kernel<TP, TG, MASTER, false><<<grid, kAdamThreads, 0, s>>>(a);
        };
        if constexpr (!std::is_same_v<TP, float>) {
            if (master) return run(std::true_type{});
        }
        run(std::false_type{});
    });
}

}  // namespace dytb
