// Workspace sizes of the layer operators. Host code only.
#include "op_kernels.hpp"
#include "op_layout.hpp"

namespace muir {

int head_decay_segments(int B, int T, int H, bool bf16) {
    // 512 workgroups in bf16 and 256 in float32, of at least two chunks each: a segment costs a second reading of its keys and
    // values and a state written and read. At dk = dv = 128 that many run at once (LDS: two to a compute unit, one); narrower
    // heads admit more, which the rule does not use.
    const long long heads = static_cast<long long>(B) * H, room = bf16 ? 512 : 256;
    const int n = hd::chunks_of(T);
    const int want = static_cast<int>(std::min<long long>(room / std::min(heads, room), n / 2));
    if (want <= 1) return 1;
    const int per = (n + want - 1) / want;
    return (n + per - 1) / per;
}

size_t head_decay_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, bool bf16) {
    const int nseg = head_decay_segments(B, T, H, bf16);
    if (nseg == 1) return 0;
    const size_t bhs = static_cast<size_t>(B) * H * nseg;
    return up256(bhs * dk * dv * 4) + up256(bhs * 8);
}

size_t head_decay_bwd_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv, bool bf16) {
    const int nseg = head_decay_segments(B, T, H, bf16);
    const size_t bh = static_cast<size_t>(B) * H, tok = bh * T, groups = hd::groups_of(T);
    size_t n = 2 * up256(tok * 4) + up256(bh * groups * dk * dv * 4) + up256(bh * groups * (dk / 16) * 4) + up256(bh * groups * 8);
    if (nseg > 1) n += 2 * up256(bh * nseg * dk * dv * 4) + 2 * up256(bh * nseg * 8);
    if (Hk != H) n += 2 * up256(tok * dk * 4);
    return n;
}

size_t rms_norm_bwd_workspace_bytes(int rows, int D) {
    return rows > 0 ? static_cast<size_t>(norm_bwd_blocks(rows, D)) * D * 4 : 0;
}

}  // namespace muir
