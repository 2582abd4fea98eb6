// Workspace sizes of softmax attention. Host code only.
#include <algorithm>

#include "attention_kernels.hpp"
#include "op_layout.hpp"

namespace muir {

size_t attention_bwd_workspace_bytes(int N, int H) { return 2 * up256(static_cast<size_t>(N) * H * 4); }

int attention_step_parts(int B, int H, int Hk, int d, int capacity, bool bf16) {
    (void)d, (void)bf16;
    const long long groups = static_cast<long long>(B) * Hk * ((H / Hk + 15) / 16), room = 512;
    const long long most = std::max(1, capacity / 256);
    return static_cast<int>(std::min<long long>(most, std::max<long long>(1, room / groups)));
}

size_t attention_step_workspace_bytes(int B, int H, int Hk, int d, int capacity, bool bf16) {
    const int parts = attention_step_parts(B, H, Hk, d, capacity, bf16);
    return parts == 1 ? 0 : static_cast<size_t>(B) * H * parts * (d + 2) * 4;
}

}  // namespace muir
