// Workspace sizes of softmax attention. Host code only.
#include <algorithm>

#include "attention_kernels.hpp"
#include "op_layout.hpp"

namespace muir {

// bf16: 128 rows to a workgroup, or blocks of 32 whose four wavefronts share the keys (or the queries). The first reads each key a quarter as often; the
// second fills the card with few rows, and does not wait for the workgroup with the most keys, which without a window has twice the mean. Measured,
// forward and backward in us, of blocks of 32 and of 128 rows, by the number W of the latter:
//   d128, T <= 1024:      W 300 (T1024 H30) 24.8, 76 and 29.4, 84     W 400 (T1024 H40) 30.9, 96 and 30.7, 90
//   d128, T >= 2048:      W 544 (T4096 H16) 108, 308 and 119, 345     W 680 (T4096 H20) 135, 401 and 152, 390
//   d128, a short window: W 136 (T4096 H4, 512) 13.3, 41 and 21.2, 57 W 204 (T4096 H6, 512) 23.6, 68 and 22.3, 59
//   d64, a quarter more:  W 400 (T1024 H40) 16.6, 53 and 20.7, 59     W 720 (T2048 H40) 45.1, 133 and 45.8, 138
//                         W 136 (T4096 H4, 512) 9.3, 25 and 13.9, 38  W 272 (T4096 H8, 512) 13.5, 43 and 14.5, 39
// Lengths are taken for equal, as they lie on the device.
// float32: the same in the forward (d64 B4 T1024 H16, W 592, 77 and 80, B8 T4096 H16 1728 and 1600; d128 163 and 146, 3856 and 3199). The backward has
// blocks of 32 only: d64 233 and 260, 5570 and 5728; d128 546 and 643, and only the largest gains by 128 (13036 and 12467).
bool attention_split(int N, int S, int heads, int d, int window) {
    const int most = attention_even(N, S, window) ? 160 : N / S < 2048 ? 350 : 600;
    return attention_blocks(N, S, 128) * heads <= (d == 64 ? most * 5 / 4 : most);
}

bool attention_even(int N, int S, int window) { return window && window <= N / S / 2; }

// Whether the blocks with the most to do go first. Without a window, in us, sequence after sequence and by place: bf16 B8 T4096 H16 d128 forward 580 and
// 550, dq 870 and 851, dkv 1020 and 966; 24 packed sequences up to 4001, H16 Hk4, 425 and 397: the last sequence's largest blocks began when the card was
// running empty. With a short window packed sequences are taken one after another, which keeps neighbours' keys in the caches: 9 up to 4096, H16
// Hk4, window 512, dq 127 and 136, dkv 131 and 138; of a batch they are as near either way (B8 T4096 H12 d64 window 1024 129 and 126).
bool attention_by_place(const int *offsets, int N, int S, int window) { return !offsets || !attention_even(N, S, window); }

// Whether dk and dv of a block of 32 keys take eight wavefronts instead of four: where four would all run at once (two workgroups to a compute unit), the
// one with the most tiles is what is waited for, and it has the queries of every head that shares the key. The backward in us with four and with eight:
// bf16 d128 B1 T2048 H16 Hk4 (256 workgroups, 256 tiles) 141 and 114, B1 T512 H16 Hk4 (64, 64) 41.5 and 35.4, B1 T4096 H16 Hk4 (512, 512) 347 and 302,
// B1 T2048 H16 Hk16 (1024, 64) 98.7 and 112.6, B1 T128 H16 Hk16 (64, 4) 17.9 and 18.5; float32 d64 B3 T777 H12 Hk6 (432, 48) 108.8 and 101.7.
bool attention_far(int N, int S, int H, int Hk, int window) {
    const long long length = N / S, seen = window && window < length ? window : length;
    return static_cast<long long>(N / 32) * Hk <= 512 && H / Hk * seen >= 12 * 32;
}

size_t attention_bwd_workspace_bytes(int N, int H) { return 2 * up256(static_cast<size_t>(N) * H * 4); }

// One workgroup to a compute unit, by its LDS: B1 T32768 H16 Hk4 d128 bf16 (page 64) 17.1 us with room for 256 workgroups, 20.7 with 512 (the parts then cost
// more than they gain), 18.8 with half as many wavefronts. bf16 heads of 64 take half of the LDS; where the parts stay long, room for 512 pays:
// B64 T8000 H16 Hk4 66 us against 74, while B16 T1000 H12 (192 workgroups) has 9.0 unsplit and 10.8 in two. A part has 256 keys at least, a tile for
// each wavefront. Up to 128 KB of keys a second launch costs more than it saves: B4 H16 Hk4 by calls, and in a graph, whole and in parts, bf16 d128 T511 7.9
// and 11.0, 7.3 and 8.3; d64 T1023 8.0 and 11.6, 8.4 and 8.0; float32 d64 T511 9.3 and 11.6, 9.9 and 9.7; beyond, bf16 d128 T1023 9.5 and 11.3, 10.1 and
// 8.3, T2047 15.6 and 11.1, 16.3 and 8.5.
int attention_step_parts(int B, int H, int Hk, int d, int capacity, bool bf16) {
    if (static_cast<long long>(capacity) * d * (bf16 ? 2 : 4) <= 128 << 10) return 1;
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
