// Workspace sizes of softmax attention. Host code only.
#include <algorithm>

#include "attention_kernels.hpp"
#include "op_layout.hpp"

namespace muir {

// Where 128 rows to a workgroup make fewer than two of them to a compute unit, blocks of 32 rows whose wavefronts share the keys (or the queries) fill the
// card better: forward and backward of bf16 B1 T2048 H12 d128, 216 such workgroups, 31 and 89 us against 52 and 138 with 128 rows; at T4096 H16 (544) both
// 104 us; at B4 T1024 H16 (592) 46 and 133 against 43 and 101. In float32 the products take so long that rows are never too few for it: d64 is
// faster at every size measured (B1 T128 H12 7.3 and 20 us against 15 and 43, B8 T4096 H16 2.24 and 7.38 ms against 2.38 and 7.82), d128 up to
// B4 T1024 H16 (201 and 666 us against 218 and 830), and at B8 T4096 H16 7 and 3 % slower.
bool attention_split(int N, int S, int heads) { return attention_blocks(N, S, 128) * heads <= 400; }

size_t attention_bwd_workspace_bytes(int N, int H) { return 2 * up256(static_cast<size_t>(N) * H * 4); }

// One workgroup to a compute unit, by its LDS: B1 T32768 H16 Hk4 d128 bf16 (page 64) 17.1 us with room for 256 workgroups, 20.7 with 512 (the parts then cost
// more than they gain), 18.8 with half as many wavefronts. bf16 heads of 64 take half of the LDS; where the parts stay long, room for 512 pays:
// B64 T8000 H16 Hk4 66 us against 74, while B16 T1000 H12 (192 workgroups) has 9.0 unsplit and 10.8 in two. A part has 256 keys at least, a tile for
// each wavefront.
int attention_step_parts(int B, int H, int Hk, int d, int capacity, bool bf16) {
    const long long groups = static_cast<long long>(B) * Hk * ((H / Hk + 15) / 16), most = capacity / 256;
    long long parts = std::min(most, 256 / groups);
    if (bf16 && d == 64) parts = std::max(parts, std::min<long long>(512 / groups, capacity / 2048));
    return static_cast<int>(std::max<long long>(parts, 1));
}

size_t attention_step_workspace_bytes(int B, int H, int Hk, int d, int capacity, bool bf16) {
    const int parts = attention_step_parts(B, H, Hk, d, capacity, bf16);
    return parts == 1 ? 0 : static_cast<size_t>(B) * H * parts * (d + 2) * 4;
}

}  // namespace muir
