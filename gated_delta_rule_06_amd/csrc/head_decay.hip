// Linear attention with one decay per head: chunked forward and backward (head_decay.hpp has the
// formulas). Four kernels:
//   pass, LOCAL             each segment's own contribution to the state at its end, and its decay
//   join_kernel             the state at each segment's start from those, in order
//   pass                    one walk over a segment's chunks: outputs (or one gradient) with the state in registers
//   dla_kernel, *_sum       the decay's gradient from the row sums of two passes; sums over shared heads
// Where B * H workgroups fill the card there is one segment per head and the pass is the only launch of a forward.
//
// Measured in bf16, 128/128, 8192 chunks (fastest of 20, us): forward of B1 T32768 H16 65 local pass, 17 join, 149 pass; backward of
// B8 T4096 H16 97 for both local passes, 18 both joins, 237 dq, 245 dk, 150 dv, 11 the decay's gradient. The local pass reads k and v
// at 4.1 TB/s; in the others instructions issue in up to 72 to 86 % of the cycles, vector ones in 49 to 57 %, and the matrix cores
// are busy for 26 to 37 %. dq and dk keep three bf16 terms where the forward and dv keep two, and write and read the states between groups
// (268 MB each): 877 and 906 vector instructions a wavefront and chunk against 590.
#include <algorithm>

#include "head_decay.hpp"
#include "launch.hpp"
#include "op_kernels.hpp"

namespace muir {
namespace {

using namespace hd;

struct PassArgs {
    const void *x, *y, *z;  // [B, T, h*, D*]
    int hx, hy, hz;
    const float *a;         // [B, T, H], or [H]
    bool a_fixed;
    const int *lens;        // [B] or NULL
    const float *start;     // [B*H, nseg] states [DX, DZ] at the segments' starts, or NULL for zeros
    bool start_t;           // the states are stored [DZ, DX]
    void *out;              // [B, T, H, DZ] in the element type, or float32 with out_f32
    bool out_f32;
    float *s_out;           // state after the last token, [DX, DZ], or NULL; LOCAL: [B*H, nseg] states
    f32x2_t *dec;           // LOCAL: [B*H, nseg] decays, as a float32 and what it leaves
    const void *w;          // KEEP: [B, T, hw, DZ], dots [B, T, H] = out . w but for the token's own z in out
    int hw;
    float *dots;
    float *anchors;         // KEEP: [B*H, groups] states, written in order and read reversed
    float *edges;           // KEEP, reversed: [B*H, groups, DZ / 16] parts of <S, A>
    int B, T, H, nseg, seg_chunks, nchunks;
};

// A tile of 64 rows of one head on its way from memory to LDS.
template <typename T, int D, int THREADS> struct Tile {
    static constexpr int VEC = 16 / sizeof(T);
    static constexpr int PER = D / VEC, N = C * PER / THREADS;  // 16-byte vectors of a row, of a thread
    u32x4_t r[N];
    // Rows from `rows` on are zeros and are not read: the buffer ends there.
    __device__ __forceinline__ void load(const unsigned char *base, int stride, int rows, int tid) {
        const rsrc_t b = make_rsrc(base, static_cast<unsigned>(rows) * stride);
        const int off = tid / PER * stride + tid % PER * 16;
#pragma unroll
        for (int j = 0; j < N; ++j) r[j] = __builtin_amdgcn_raw_buffer_load_b128(b, off, j * (THREADS / PER) * stride, 0);
    }
    __device__ __forceinline__ void put(unsigned char *lds, int tid) const {
#pragma unroll
        for (int j = 0; j < N; ++j) Op<T>::template put16<D>(lds, (tid + THREADS * j) / PER, (tid + THREADS * j) % PER, r[j]);
    }
};

template <typename T, int DX, int DZ, bool LOCAL, int NTP> struct PassLds {
    using O = Op<T>;
    static constexpr int THREADS = 4 * DZ, NW = DZ / 16;  // one wavefront for 16 columns
    static constexpr int Y = 0, Z = Y + O::template tile_bytes<DX>(), X = Z + O::template tile_bytes<DZ>();
    static constexpr int P = X + (LOCAL ? 0 : O::template tile_bytes<DX>());
    static constexpr int TAIL = P + (LOCAL ? 0 : NTP * O::template tile_bytes<C>());
    static constexpr int BYTES = TAIL + C * 8 + C * 4 * 2 + 16 + (LOCAL ? 0 : NW * C * 4 + C * 4);
};

// One wavefront owns 16 columns of the state and of the output; see head_decay.hpp for the operand order.
// Rounding, for bf16 inputs: the products x.y are exact in float32; D (x.y) and the state go into the second
// products as NTP and NTS bf16 terms, the decayed z into the state's update as three, so states, and the
// row sums that the decay's gradient is made of, keep float32 accuracy.
template <typename T_, int DX_, int DZ_, bool REV_, bool LOCAL_, bool KEEP_, int NTP_, int NTS_, int NTU_> struct Pass {
    using T = T_;
    static constexpr int DX = DX_, DZ = DZ_, NTP = NTP_, NTS = NTS_, NTU = NTU_;
    static constexpr bool REV = REV_, LOCAL = LOCAL_, KEEP = KEEP_;
    static constexpr int BYTES = PassLds<T, DX, DZ, LOCAL, NTP>::BYTES;
};

template <typename K> __device__ __forceinline__ void pass(const PassArgs &p, int block) {
    using T = typename K::T;
    constexpr int DX = K::DX, DZ = K::DZ, NTP = K::NTP, NTS = K::NTS, NTU = K::NTU;
    constexpr bool REV = K::REV, LOCAL = K::LOCAL, KEEP = K::KEEP;
    using O = Op<T>;
    using L = PassLds<T, DX, DZ, LOCAL, NTP>;
    using frag = typename O::frag;
    constexpr int RT = DX / 16, ES = sizeof(T), THREADS = L::THREADS, NW = L::NW;
    // LOCAL walks against the order of the pass that follows it, which then finds what was read last in the caches.
    constexpr bool DOWN = REV != LOCAL;
    constexpr int SIDE = KEEP ? 2 : 4;  // sums that are added to in turn, so that a product does not wait for the one before
    constexpr int PAIRS = ES == 4 ? 2 : 1;  // blocks of 32 tokens that the state takes at once
    constexpr int OSIDE = NTS > 1 ? 2 : 4;  // in the products with the state, whose terms take registers too
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char *const ly = smem + L::Y, *const lz = smem + L::Z, *const lx = smem + L::X, *const lp = smem + L::P;
    // Sums of log2 a from the chunk's start, each as a float32 and what it leaves of the 64-bit sum. A difference of the two parts
    // is rounded like the float32 it becomes, also where the sums are far from zero (a decay of zero adds -200 to each).
    f32x2_t *const sh_L = reinterpret_cast<f32x2_t *>(smem + L::TAIL);
    float *const sh_out = reinterpret_cast<float *>(sh_L + C);        // decay between a token and the start state
    float *const sh_upd = sh_out + C;                                 // decay of a token's z in the update
    float *const sh_carry = sh_upd + C;                               // decay of the state over the chunk, and what it owes the next
    float *const sh_dot = sh_carry + 4;                               // [NW][C]
    float *const sh_diag = sh_dot + NW * C;                           // KEEP: x_i . y_i

    int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, m = lane & 15, g = lane >> 4;
    // Quotients and clamped values are made in vector registers; they are the same in every lane, and a buffer's
    // description has to be known to be.
    auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    // LOCAL: the last segment in the order of the walk is not needed.
    const int per = LOCAL ? p.nseg - 1 : p.nseg;
    const int bh = uniform(block / per), seg = block - bh * per + (LOCAL && REV ? 1 : 0), b = uniform(bh / p.H), h = bh - b * p.H;
    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);
    const int end = uniform(p.lens ? min(max(p.lens[b], 0), p.T) : p.T);
    const int live = end / C + (end % C != 0), steps = max(min(c1, live) - c0, 0);  // chunks that hold a token
    const int col0 = wv * 16;
    const size_t bT = static_cast<size_t>(b) * p.T;
    // Row strides in bytes, and the head's first row in each tensor.
    const int sx = p.hx * DX * ES, sy = p.hy * DX * ES, sz = p.hz * DZ * ES, sw = p.hw * DZ * ES;
    const int so = p.H * DZ * (p.out_f32 ? 4 : ES);
    auto head = [&](const void *t, int heads, int D) {
        return static_cast<const unsigned char *>(t) + (bT * heads + uniform(h / (p.H / heads))) * (D * ES);
    };
    const unsigned char *gx = LOCAL ? nullptr : head(p.x, p.hx, DX), *gy = head(p.y, p.hy, DX), *gz = head(p.z, p.hz, DZ);
    const unsigned char *gw = KEEP ? head(p.w, p.hw, DZ) : nullptr;
    unsigned char *go = LOCAL ? nullptr : static_cast<unsigned char *>(p.out) + (bT * p.H + h) * (DZ * (p.out_f32 ? 4 : ES));
    const int groups = (p.nchunks + ANCHOR - 1) / ANCHOR;
    constexpr int DUMP = DX * DZ;

    // The state: tile rt holds rows 16 rt + 4 g .. + 3 of column col0 + m.
    f32x4_t S[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) S[rt] = zero4();
    if (!LOCAL && p.start) {
        const float *s = p.start + static_cast<size_t>(bh * static_cast<size_t>(p.nseg) + seg) * DUMP;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int row = 16 * rt + 4 * g, col = col0 + m;
            if (p.start_t) {
                S[rt] = *reinterpret_cast<const f32x4_t *>(s + col * DX + row);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) S[rt][i] = s[(row + i) * DZ + col];
            }
        }
    }
    const float a_h = p.a_fixed && p.nchunks > 0 ? p.a[h] : 1.f;
    double seg_log = 0.0;
    if (!LOCAL && tid == 0) sh_carry[1] = 0.f;

    struct Chunk {
        Tile<T, DX, THREADS> x, y;
        Tile<T, DZ, THREADS> z;
        float a;
    };
    Chunk f;
    // The wavefronts take turns at a chunk's decays.
    auto fetch = [&](int it) {
        const int t0 = (DOWN ? c0 + steps - 1 - it : c0 + it) * C, rows = uniform(min(max(end - t0, 0), C));
        if constexpr (!LOCAL) f.x.load(gx + static_cast<size_t>(t0) * sx, sx, rows, tid);
        f.y.load(gy + static_cast<size_t>(t0) * sy, sy, rows, tid);
        f.z.load(gz + static_cast<size_t>(t0) * sz, sz, rows, tid);
        if (wv == it % NW) f.a = lane >= rows ? 1.f : p.a_fixed ? a_h : p.a[(bT + t0 + lane) * p.H + h];
    };
    // KEEP: <S, A> at the end of every ANCHOR-th chunk. The pass in order leaves S there before it takes the next chunk,
    // the reversed one takes the product.
    auto anchor = [&](int c) {
        if (REV ? (c + 1) % ANCHOR == 0 || c + 1 == p.nchunks : c % ANCHOR == 0 && c > 0) {
            const int entry = REV ? c / ANCHOR : c / ANCHOR - 1;
            f32x4_t *at = reinterpret_cast<f32x4_t *>(p.anchors + (static_cast<size_t>(bh) * groups + entry) * DUMP) +
                          wv * (RT * 64) + lane;
            f32x4_t sum = zero4();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if constexpr (REV) {
                    sum += S[rt] * at[rt * 64];
                    if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // four loads at a time: registers
                } else {
                    at[rt * 64] = S[rt];
                }
            }
            if constexpr (REV) {
                const float e = wave_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
                if (lane == 0) p.edges[(static_cast<size_t>(bh) * groups + entry) * NW + wv] = e;
            }
        }
    };
    // Chunks behind the sequence's end leave the state as it is, and their outputs are zeros.
    auto behind = [&] {
        if constexpr (LOCAL) return;
        for (int i = max(c0, live); i < c1; ++i) {
            const int c = REV ? c1 - 1 - (i - max(c0, live)) : i, t0 = c * C;
            if constexpr (KEEP) anchor(c);
            const rsrc_t bo = make_rsrc(go + static_cast<size_t>(t0) * so, static_cast<unsigned>(uniform(min(p.T - t0, C))) * so);
            const int off = m * so + (col0 + 4 * g) * (p.out_f32 ? 4 : ES);
            for (int tb = 0; tb < 4; ++tb) {
                if (ES == 4 || p.out_f32) buf_store16(bo, off + 16 * tb * so, u32x4_t{0, 0, 0, 0});
                else __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{0, 0}, bo, off, 16 * tb * so, 0);
            }
            if constexpr (KEEP) {
                if (tid < C && t0 + tid < p.T) p.dots[(bT + t0 + tid) * p.H + h] = 0.f;
            }
        }
    };
    if (steps > 0) fetch(0);
    if constexpr (REV) behind();

    for (int it = 0; it < steps; ++it) {
        const int c = DOWN ? c0 + steps - 1 - it : c0 + it, t0 = c * C;
        // Addresses that follow from the lane are made anew in each chunk: kept over the loop they would take some forty
        // registers that the state and the tiles need.
        asm volatile("" : "+v"(lane), "+v"(m), "+v"(g));
        if constexpr (KEEP) asm volatile("" : "+v"(tid));
        if constexpr (!LOCAL) f.x.put(lx, tid);
        f.y.put(ly, tid);
        f.z.put(lz, tid);
        if (wv == it % NW) {
            const double Lt = scan64(log2_decay(f.a));
            // LOCAL: decayed up to the segment's end at once, over the chunks walked before.
            const double far = LOCAL ? seg_log : 0.0;
            const float to_start = exp2_pair(Lt + far), to_end = exp2_pair(lane_value(Lt, 63) - Lt + far);
            sh_L[lane] = f32x2_t{static_cast<float>(Lt), static_cast<float>(Lt - static_cast<float>(Lt))};
            sh_out[lane] = REV ? to_end : to_start;
            sh_upd[lane] = REV ? to_start : to_end;
        }
        if constexpr (KEEP) anchor(c);
        if (it + 1 < steps) fetch(it + 1);
        lds_barrier();
        const f32x2_t Lc = sh_L[C - 1];
        if constexpr (LOCAL) seg_log += static_cast<double>(Lc[0]) + Lc[1];
        frag zf[2];
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) zf[pr] = O::template col<DZ>(lz, 32 * pr, col0, lane);

        if constexpr (!LOCAL) {
            // P[i][j] = D (x_i . y_j) for a block of 16 tokens i and one of 32 tokens j: the six blocks that are not all
            // zero, one to a wavefront (with four wavefronts, two to some). The product's rows are j, so a lane
            // stores four consecutive j.
#pragma unroll
            for (int q = 0; q < 8 / NW; ++q) {
                const int ib = NW == 8 ? wv >> 1 : wv, pr = NW == 8 ? wv & 1 : q;
                if (REV ? pr < ib / 2 : pr > ib / 2) continue;
                const int i = 16 * ib + m;
                f32x4_t acc[2] = {zero4(), zero4()};
#pragma unroll
                for (int k0 = 0; k0 < DX; k0 += 32) {
                    const frag fx = O::template row<DX>(lx, 16 * ib, k0, lane);
#pragma unroll
                    for (int u = 0; u < 2; ++u) acc[u] = O::mma(O::template row<DX>(ly, 32 * pr + 16 * u, k0, lane), fx, acc[u]);
                    // Not all operands at once: next to the state and the chunk on its way there are not the registers.
                    if (ES == 2 && k0 % 64 == 32) __builtin_amdgcn_sched_barrier(0);
                }
                // KEEP: the diagonal is added to the outputs by itself, behind their dots. A token's own product is in q.dq and in k.dk
                // alike; where the decay is strong it is far above what is left of their difference, and so were its roundings.
                if constexpr (KEEP) {
                    if (pr == ib / 2 && m >> 2 == g) {
                        const f32x4_t own = ib & 1 ? acc[1] : acc[0];
                        sh_diag[i] = m & 2 ? (m & 1 ? own[3] : own[2]) : (m & 1 ? own[1] : own[0]);
                    }
                }
                const f32x2_t Li = sh_L[i];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j0 = 32 * pr + 16 * u + 4 * g;
                    f32x4_t v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x2_t d = REV ? sh_L[j0 + e] - Li : Li - sh_L[j0 + e];
                        const float w = acc[u][e] * exp2_f(d[0] + d[1]);
                        v[e] = (KEEP ? REV ? j0 + e > i : j0 + e < i : REV ? j0 + e >= i : j0 + e <= i) ? w : 0.f;
                    }
                    O::template put4<C, NTP>(lp, i, j0 / 4, v);
                }
            }
            // A wavefront with less to do here makes the state's decay over the chunk. A float32 near exp2(L) is off by up to
            // 2^-24, and a fixed decay's by the same amount in every chunk, which adds up in a state that lives long. So what a chunk's
            // factor leaves of L goes into the next one's, and the product of the factors stays within one rounding. Float32 state, H16 d64: 5.0e-7 off
            // after 262144 tokens of half-life 1e5 against 5.6e-6 without, 2.4e-7 against 7.6e-7 after 32768, 1.9e-7 against 3.9e-7 there at
            // half-life 1000; nothing in time.
            if (wv == (REV ? NW / 8 * 4 + NW / 4 % 2 * 3 : NW / 8)) {
                const float rest = Lc[1] + sh_carry[1], factor = exp2_pair(Lc[0], rest);
                const float n = rintf(Lc[0]);
                // 2^(L - n) in 64 bits by the exponential's series (|L - n| ln 2 < 0.35: eleven terms leave 2^-42).
                const double y = (static_cast<double>(Lc[0] - n) + rest) * 0.6931471805599453;
                double e = 1.0;
#pragma unroll
                for (int k = 10; k >= 1; --k) e = fma(e * y, 1.0 / k, 1.0);
                const float off = static_cast<float>(ldexp(static_cast<double>(factor), -static_cast<int>(n)) - e) / static_cast<float>(e);
                if (lane == 0) {
                    sh_carry[0] = factor;
                    // log2 of what the rounding took. Only of a normal factor: below that range the rounding is percents of it, up to
                    // all, and the next factor also decays what this chunk itself added. (a = 0.2, 65 tokens: +27 % in the state.)
                    sh_carry[1] = factor >= 1.17549435e-38f ? -1.44269504f * off : 0.f;
                }
            }
            lds_barrier();

            // Output tiles with a token in each lane's column: decayed state . x, then P z.
            f32x4_t acc[4];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) acc[tb] = zero4();
#pragma unroll
            for (int k = 0; k < RT / 2; ++k) {
                frag sf[NTS];
                float s8[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s8[e] = S[2 * k][e];
                    s8[4 + e] = S[2 * k + 1][e];
                }
                // (Loads moved across here cost the dk pass of 128/64 a tile's vector, spilled while on its way.)
                if constexpr (KEEP && ES == 2 && DX < DZ) __builtin_amdgcn_sched_barrier(0);
                O::template split<NTS>(s8, sf);
#pragma unroll
                for (int t0b = 0; t0b < 4; t0b += OSIDE) {
                    frag fx[OSIDE];
#pragma unroll
                    for (int r = 0; r < OSIDE; ++r) fx[r] = O::template row<DX>(lx, 16 * (t0b + r), 32 * k, lane);
#pragma unroll
                    for (int n = 0; n < NTS; ++n)
#pragma unroll
                        for (int r = 0; r < OSIDE; ++r) acc[t0b + r] = O::mma(sf[n], fx[r], acc[t0b + r]);
                }
            }
            // KEEP: the rows that this chunk's outputs are multiplied with, in the accumulators' layout. Fetched only here: over
            // the products with the state there is no register left for them.
            using pack4_t = std::conditional_t<ES == 2, u32x2_t, u32x4_t>;
            pack4_t w4[KEEP ? 4 : 1];
            if constexpr (KEEP) {
                const rsrc_t bw = make_rsrc(gw + static_cast<size_t>(t0) * sw, static_cast<unsigned>(uniform(min(max(end - t0, 0), C))) * sw);
                const int off = m * sw + (col0 + 4 * g) * ES;
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) {
                    if constexpr (ES == 2) w4[tb] = __builtin_amdgcn_raw_buffer_load_b64(bw, off, 16 * tb * sw, 0);
                    else w4[tb] = __builtin_amdgcn_raw_buffer_load_b128(bw, off, 16 * tb * sw, 0);
                }
            }
            const rsrc_t bo = make_rsrc(go + static_cast<size_t>(t0) * so, static_cast<unsigned>(uniform(min(p.T - t0, C))) * so);
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                acc[tb] *= sh_out[16 * tb + m];
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                    if (REV ? pr < tb / 2 : pr > tb / 2) continue;
#pragma unroll
                    for (int n = 0; n < NTP; ++n)
                        acc[tb] = O::mma(zf[pr], O::template row<C>(lp + n * O::template tile_bytes<C>(), 16 * tb, 32 * pr, lane), acc[tb]);
                }
                const int t = 16 * tb + m, col = col0 + 4 * g;
                if (t0 + C > end && t0 + t >= end) acc[tb] = zero4();
                if constexpr (KEEP) {
                    float dot = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float w;
                        if constexpr (ES == 2) w = bf16_to_f32(static_cast<uint16_t>(w4[tb][e / 2] >> (16 * (e % 2))));
                        else w = __uint_as_float(w4[tb][e]);
                        dot = fmaf(w, acc[tb][e], dot);
                    }
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (g == 0) sh_dot[wv * C + t] = dot;
                    const f32x4_t z4 = O::template quad<DZ>(lz, t, col / 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[tb][e] = fmaf(sh_diag[t], z4[e], acc[tb][e]);
                }
                if (ES == 4 || p.out_f32) {
                    buf_store16(bo, (16 * tb + m) * so + 4 * col, __builtin_bit_cast(u32x4_t, acc[tb]));
                } else {
                    u16x4_t u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] = f32_to_bf16(acc[tb][e]);
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, u), bo, m * so + 2 * col, 16 * tb * so, 0);
                }
            }
        }

        // The state: decayed over the chunk, plus y^T (decayed z). In float32 the chunk's own sum is made first, so that the state is
        // rounded once a chunk and not with each product of four tokens: 3.8e-6 -> 5e-7 off after 262144 tokens of half-life 1e5, in the same
        // time. bf16 adds straight to the state, three times for 32 tokens: the same there took 748 -> 976 us for the backward of
        // B8 T4096 H16 d128 (registers), where ds0 is 4.5e-7 off.
        const float carry = LOCAL ? 1.f : *sh_carry;
        if constexpr (!LOCAL && ES == 2) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) S[rt] *= carry;
        }
#pragma unroll
        for (int p0 = 0; p0 < 2; p0 += PAIRS) {
            frag zs[PAIRS][NTU];
#pragma unroll
            for (int u = 0; u < PAIRS; ++u) {
                const int j0 = 32 * (p0 + u) + 4 * g;
                const f32x4_t ulo = *reinterpret_cast<const f32x4_t *>(sh_upd + j0);
                const f32x4_t uhi = *reinterpret_cast<const f32x4_t *>(sh_upd + j0 + 16);
                float z8[8];
                O::floats(zf[p0 + u], z8);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z8[e] *= ulo[e];
                    z8[4 + e] *= uhi[e];
                }
                O::template split<NTU>(z8, zs[u]);
            }
#pragma unroll
            for (int r0 = 0; r0 < RT; r0 += SIDE) {
                f32x4_t sum[SIDE];
#pragma unroll
                for (int r = 0; r < SIDE; ++r) sum[r] = ES == 2 ? S[r0 + r] : zero4();
#pragma unroll
                for (int u = 0; u < PAIRS; ++u) {
                    frag fy[SIDE];
#pragma unroll
                    for (int r = 0; r < SIDE; ++r) fy[r] = O::template col<DX>(ly, 32 * (p0 + u), 16 * (r0 + r), lane);
#pragma unroll
                    for (int n = NTU - 1; n >= 0; --n)
#pragma unroll
                        for (int r = 0; r < SIDE; ++r) sum[r] = O::mma(fy[r], zs[u][n], sum[r]);
                }
#pragma unroll
                for (int r = 0; r < SIDE; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[r0 + r][e] = ES == 2 ? sum[r][e] : fmaf(carry, S[r0 + r][e], sum[r][e]);
            }
        }
        lds_barrier();
        if constexpr (KEEP) {
            if (tid < C && t0 + tid < p.T) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) x += sh_dot[w * C + tid];
                p.dots[(bT + t0 + tid) * p.H + h] = x;
            }
        }
    }

    if constexpr (!REV) behind();
    if constexpr (KEEP && !REV) {
        if (seg == p.nseg - 1 && p.nchunks > 0) {
            f32x4_t *at = reinterpret_cast<f32x4_t *>(p.anchors + (static_cast<size_t>(bh) * groups + groups - 1) * DUMP) +
                          wv * (RT * 64) + lane;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) at[rt * 64] = S[rt];
        }
    }
    float *st = nullptr;
    if (LOCAL) {
        st = p.s_out + static_cast<size_t>(bh * static_cast<size_t>(p.nseg) + seg) * DUMP;
        if (tid == 0) {
            const double d = exp2(seg_log);
            p.dec[static_cast<size_t>(bh) * p.nseg + seg] = f32x2_t{static_cast<float>(d), static_cast<float>(d - static_cast<float>(d))};
        }
    } else if (p.s_out && seg == (REV ? 0 : p.nseg - 1)) {
        st = p.s_out + static_cast<size_t>(bh) * DUMP;
    }
    if (st) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) st[(16 * rt + 4 * g + i) * DZ + col0 + m] = S[rt][i];
    }
}

// bf16: two workgroups of eight (or four of four) wavefronts to a compute unit.
template <typename K> constexpr int pass_waves() { return K::DZ / 64 * (sizeof(typename K::T) == 2 ? 2 : 1); }

template <typename K>
__global__ __launch_bounds__(4 * K::DZ, pass_waves<K>()) void pass_kernel(PassArgs p) {
    pass<K>(p, blockIdx.x);
}

// Two passes over the same segments in one launch, `n` workgroups each. Workgroups go to the eight dies in turn: the two
// of one segment are eight apart, so the second finds in its die's cache what the first has read.
template <typename K, typename M>
__global__ __launch_bounds__(4 * K::DZ, pass_waves<K>()) void pair_kernel(PassArgs p, PassArgs q, int n) {
    const int unit = (blockIdx.x >> 4 << 3) | (blockIdx.x & 7);
    if (unit >= n) return;
    if (blockIdx.x & 8) pass<M>(q, unit);
    else pass<K>(p, unit);
}

// The state at each segment's start (reversed: end), in place of the segments' own contributions:
// x <- s0 (or zeros); segment by segment: start = x, x <- dec x + contribution.
struct JoinArgs {
    const float *s0;
    float *seg;
    const f32x2_t *dec;
    bool rev;
};
__global__ __launch_bounds__(256) void join_kernel(JoinArgs first, JoinArgs second, int nseg, int n4) {
    const JoinArgs p = blockIdx.y ? second : first;
    const int blocks = (n4 + 255) / 256, bh = blockIdx.x / blocks, i = blockIdx.x % blocks * 256 + threadIdx.x;
    if (i >= n4) return;
    f32x4_t x = p.s0 ? reinterpret_cast<const f32x4_t *>(p.s0)[static_cast<size_t>(bh) * n4 + i] : zero4();
    f32x4_t *at = reinterpret_cast<f32x4_t *>(p.seg) + static_cast<size_t>(bh) * nseg * n4 + i;
    const f32x2_t *d = p.dec + static_cast<size_t>(bh) * nseg;
#pragma unroll 4
    for (int s = 0; s < nseg; ++s) {
        const int k = p.rev ? nseg - 1 - s : s;
        f32x4_t own = zero4();
        if (s + 1 < nseg) own = at[static_cast<size_t>(k) * n4];  // the last one's is not made: no segment starts behind it
        at[static_cast<size_t>(k) * n4] = x;
        if (s + 1 < nseg) x = x * d[k][0] + (x * d[k][1] + own);
    }
}

// dla of one group of ANCHOR chunks, from the nearer of its two ends: <S, A> at its end plus the sum of q.dq - k.dk from the token on, or
// <S, A> at its start less the sum over the tokens before. In 64 bits: the terms cancel where the decay is strong. What q.dq and k.dk
// were rounded by adds up with the distance; a fixed decay's gradient sums it over all tokens.
__global__ __launch_bounds__(ANCHOR *C) void dla_kernel(const float *rows, const float *cols, const float *edges,
                                                        const int *lens, float *dla, double *part, int T, int H,
                                                        int groups, int parts, bool zero_start) {
    __shared__ double sh[ANCHOR];
    const int grp = blockIdx.x % groups, bh = blockIdx.x / groups, b = bh / H, h = bh % H;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t = grp * (ANCHOR * C) + ANCHOR * C - 1 - static_cast<int>(threadIdx.x);
    const int end = lens ? min(max(lens[b], 0), T) : T;
    const size_t at = (static_cast<size_t>(b) * T + t) * H + h;
    double x = t < end ? static_cast<double>(rows[at]) - static_cast<double>(cols[at]) : 0.0;
    x = scan64(x);
    if (lane == 63) sh[wv] = x;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < ANCHOR; ++w) {
        if (w < wv) x += sh[w];
        total += sh[w];
    }
    // The first group's start: zero where the state there is, else its end serves all.
    const bool from_start = static_cast<int>(threadIdx.x) >= ANCHOR * C / 2 && (grp > 0 || zero_start);
    if (from_start) x -= total;
    if (!from_start || grp > 0) {
        const float *e = edges + (static_cast<size_t>(bh) * groups + grp - (from_start ? 1 : 0)) * parts;
        for (int i = 0; i < parts; ++i) x += e[i];
    }
    if (t >= end) x = 0.0;
    if (dla) {
        if (t < T) dla[at] = static_cast<float>(x);
        return;
    }
    __syncthreads();
    for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
    if (lane == 0) sh[wv] = x;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < ANCHOR; ++w) x += sh[w];
    part[static_cast<size_t>(bh) * groups + grp] = x;
}

// A fixed decay's gradient: one wavefront per head sums its groups over the batch, in a fixed order.
__global__ __launch_bounds__(64) void dla_sum_kernel(const double *part, float *dla, int B, int H, int groups) {
    const int h = blockIdx.x;
    double x = 0.0;
    for (int i = threadIdx.x; i < B * groups; i += 64)
        x += part[(static_cast<size_t>(i / groups) * H + h) * groups + i % groups];
    for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
    if (threadIdx.x == 0) dla[h] = static_cast<float>(x);
}

// Gradients of shared heads: out [rows, Hk, d] = sum over the rep value heads of part [rows, Hk * rep, d].
template <typename T>
__global__ __launch_bounds__(256) void head_sum_kernel(const float *part, T *out, size_t n4, int rep, int d4) {
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n4) return;
    const size_t head = i / d4, c = i % d4;
    const f32x4_t *p = reinterpret_cast<const f32x4_t *>(part) + head * rep * d4 + c;
    f32x4_t x = p[0];
    for (int r = 1; r < rep; ++r) x += p[static_cast<size_t>(r) * d4];
    store4(out + 4 * i, x);
}

// The passes, by what their results need of each operand. P and the state go into the forward and dv as two terms each, which leaves 2^-16
// of them: the outputs are as exact as their own rounding to bf16. (The state as one term: 1.92e-3 off in the 2-norm against 1.66e-3, and 225
// against 234 us for the forward of B1 T32768 H16 d128, 698 against 711 for the backward of B8 T4096.)
template <typename T, int DK, int DV> struct Kinds {
    static constexpr int N2 = sizeof(T) == 2 ? 2 : 1, N3 = sizeof(T) == 2 ? 3 : 1;
    using Forward = Pass<T, DK, DV, false, false, false, N2, N2, N3>;
    using LocalFwd = Pass<T, DK, DV, false, true, false, 1, 1, N3>;
    using LocalRev = Pass<T, DK, DV, true, true, false, 1, 1, N3>;
    using Dq = Pass<T, DV, DK, false, false, true, N3, N3, N3>;
    using Dk = Pass<T, DV, DK, true, false, true, N3, N3, N3>;
    using Dv = Pass<T, DK, DV, true, false, false, N2, N2, N3>;
};

template <typename K> unsigned pass_blocks(const PassArgs &p) {
    return static_cast<unsigned>(p.B) * p.H * (K::LOCAL ? p.nseg - 1 : p.nseg);
}

template <typename K> hipError_t launch_pass(const PassArgs &p, hipStream_t s) {
    const hipError_t err = allow_lds<pass_kernel<K>>(K::BYTES);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(pass_kernel<K>, dim3(pass_blocks<K>(p)), dim3(4 * K::DZ), K::BYTES, s, p);
    return hipGetLastError();
}

template <typename K, typename M> hipError_t launch_pair(const PassArgs &p, const PassArgs &q, hipStream_t s) {
    if constexpr (K::DZ != M::DZ) {  // another number of threads
        const hipError_t err = launch_pass<K>(p, s);
        return err != hipSuccess ? err : launch_pass<M>(q, s);
    } else {
        constexpr int bytes = K::BYTES > M::BYTES ? K::BYTES : M::BYTES;
        const hipError_t err = allow_lds<pair_kernel<K, M>>(bytes);
        if (err != hipSuccess) return err;
        const unsigned n = pass_blocks<K>(p);
        hipLaunchKernelGGL((pair_kernel<K, M>), dim3((n + 7) / 8 * 16), dim3(4 * K::DZ), bytes, s, p, q, static_cast<int>(n));
        return hipGetLastError();
    }
}

hipError_t launch_join(const JoinArgs &first, const JoinArgs *second, int bh, int nseg, int n, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>((n / 4 + 255) / 256) * bh, second ? 2 : 1);
    hipLaunchKernelGGL(join_kernel, grid, dim3(256), 0, s, first, second ? *second : first, nseg, n / 4);
    return hipGetLastError();
}

struct Carver {
    unsigned char *base;
    size_t at = 0;
    template <typename V> V *take(size_t n) {
        V *p = reinterpret_cast<V *>(base + at);
        at += up256(n * sizeof(V));
        return p;
    }
};

PassArgs pass_args(const HeadDecayCall &c) {
    PassArgs p{};
    p.a = c.a;
    p.a_fixed = c.a_fixed;
    p.lens = c.lens;
    p.B = c.B;
    p.T = c.T;
    p.H = c.H;
    p.nchunks = chunks_of(c.T);
    p.nseg = head_decay_segments(c.B, c.T, c.H, c.bf16);
    p.seg_chunks = (p.nchunks + p.nseg - 1) / p.nseg;
    return p;
}

template <typename T, int DK, int DV>
hipError_t forward(const HeadDecayCall &c, void *o, float *s_out, void *workspace, hipStream_t stream) {
    using Kind = Kinds<T, DK, DV>;
    PassArgs p = pass_args(c);
    p.x = c.q;
    p.y = c.k;
    p.z = c.v;
    p.hx = p.hy = c.Hk;
    p.hz = c.H;
    p.start = c.s0;
    if (p.nseg > 1) {
        Carver w{static_cast<unsigned char *>(workspace)};
        const size_t bhs = static_cast<size_t>(c.B) * c.H * p.nseg;
        float *seg = w.take<float>(bhs * DK * DV);
        f32x2_t *dec = w.take<f32x2_t>(bhs);
        p.s_out = seg;
        p.dec = dec;
        hipError_t err = launch_pass<typename Kind::LocalFwd>(p, stream);
        if (err != hipSuccess) return err;
        err = launch_join(JoinArgs{c.s0, seg, dec, false}, nullptr, c.B * c.H, p.nseg, DK * DV, stream);
        if (err != hipSuccess) return err;
        p.start = seg;
    }
    p.out = o;
    p.s_out = s_out;
    return launch_pass<typename Kind::Forward>(p, stream);
}

template <typename T>
hipError_t sum_heads(const float *part, void *out, size_t n4, int rep, int d4, hipStream_t stream) {
    hipLaunchKernelGGL(head_sum_kernel<T>, dim3(static_cast<unsigned>((n4 + 255) / 256)), dim3(256), 0, stream, part,
                       static_cast<T *>(out), n4, rep, d4);
    return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t backward(const HeadDecayCall &c, const HeadDecayGrads &g, void *workspace, hipStream_t stream) {
    using Kind = Kinds<T, DK, DV>;
    const PassArgs p0 = pass_args(c);
    const int groups = groups_of(c.T), BH = c.B * c.H, rep = c.H / c.Hk;
    const size_t bh = BH, tok = bh * c.T, st = static_cast<size_t>(DK) * DV;
    Carver w{static_cast<unsigned char *>(workspace)};
    float *rows = w.take<float>(tok), *cols = w.take<float>(tok);
    float *anchors = w.take<float>(bh * groups * st), *edges = w.take<float>(bh * groups * (DK / 16));
    double *part = w.take<double>(bh * groups);
    const float *s_start = c.s0, *a_start = g.ds_out;
    hipError_t err;
    if (p0.nseg > 1) {
        float *seg[2] = {w.take<float>(bh * p0.nseg * st), w.take<float>(bh * p0.nseg * st)};
        f32x2_t *dec[2] = {w.take<f32x2_t>(bh * p0.nseg), w.take<f32x2_t>(bh * p0.nseg)};
        PassArgs p[2] = {p0, p0};
        for (int rev = 0; rev < 2; ++rev) {
            p[rev].y = rev ? c.q : c.k;
            p[rev].z = rev ? g.dout : c.v;
            p[rev].hx = p[rev].hy = c.Hk;
            p[rev].hz = c.H;
            p[rev].s_out = seg[rev];
            p[rev].dec = dec[rev];
        }
        err = launch_pair<typename Kind::LocalFwd, typename Kind::LocalRev>(p[0], p[1], stream);
        if (err != hipSuccess) return err;
        const JoinArgs rev{g.ds_out, seg[1], dec[1], true};
        err = launch_join(JoinArgs{c.s0, seg[0], dec[0], false}, &rev, BH, p0.nseg, DK * DV, stream);
        if (err != hipSuccess) return err;
        s_start = seg[0];
        a_start = seg[1];
    }
    float *shared[2] = {nullptr, nullptr};  // dq and dk of every value head, where key heads are shared
    if (rep > 1)
        for (float *&x : shared) x = w.take<float>(tok * DK);
    PassArgs p[2] = {p0, p0};  // dq in order, dk reversed
    for (int pass = 0; pass < 2; ++pass) {
        p[pass].x = pass ? c.v : g.dout;
        p[pass].y = pass ? g.dout : c.v;
        p[pass].z = pass ? c.q : c.k;
        p[pass].hx = p[pass].hy = c.H;
        p[pass].hz = c.Hk;
        p[pass].start = pass ? a_start : s_start;
        p[pass].start_t = true;
        p[pass].out = shared[pass] ? shared[pass] : pass ? g.dk : g.dq;
        p[pass].out_f32 = shared[pass] != nullptr;
        p[pass].w = pass ? c.k : c.q;
        p[pass].hw = c.Hk;
        p[pass].dots = pass ? cols : rows;
        p[pass].anchors = anchors;
        p[pass].edges = edges;
    }
    PassArgs pv = p0;
    pv.x = c.k;
    pv.y = c.q;
    pv.z = g.dout;
    pv.hx = pv.hy = c.Hk;
    pv.hz = c.H;
    pv.start = a_start;
    pv.out = g.dv;
    pv.s_out = g.ds0;
    if (c.T == 0) {  // ds0 = ds_out, and no token's gradient
        err = launch_pass<typename Kind::Dv>(pv, stream);
        if (err != hipSuccess) return err;
    } else {
        // dv and dq together where both fit the card at once: B3 T777 H12 d64, float32, 252 workgroups each, 34 us against
        // 23 and 21 (measured on dk and dv). Where they do not, they get in each other's way: 418 us against 226 and 135 for
        // dk and dv of B8 T4096 H16 d128, 512 each. In turn, each walks against the one before, whose last tokens the caches hold.
        const unsigned room = 256 * std::max(1, 163840 / Kind::Dq::BYTES);
        if (2 * pass_blocks<typename Kind::Dq>(p[0]) <= room) {
            err = launch_pair<typename Kind::Dq, typename Kind::Dv>(p[0], pv, stream);
        } else {
            err = launch_pass<typename Kind::Dv>(pv, stream);
            if (err == hipSuccess) err = launch_pass<typename Kind::Dq>(p[0], stream);
        }
        if (err == hipSuccess) err = launch_pass<typename Kind::Dk>(p[1], stream);
        if (err != hipSuccess) return err;
        if (rep > 1) {
            const size_t n4 = tok / rep * DK / 4;
            err = sum_heads<T>(shared[0], g.dq, n4, rep, DK / 4, stream);
            if (err != hipSuccess) return err;
            err = sum_heads<T>(shared[1], g.dk, n4, rep, DK / 4, stream);
            if (err != hipSuccess) return err;
        }
        hipLaunchKernelGGL(dla_kernel, dim3(static_cast<unsigned>(groups) * BH), dim3(ANCHOR * C), 0, stream, rows, cols, edges,
                           c.lens, c.a_fixed ? nullptr : g.dla, part, c.T, c.H, groups, DK / 16, c.s0 == nullptr);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (c.a_fixed) {
        hipLaunchKernelGGL(dla_sum_kernel, dim3(c.H), dim3(64), 0, stream, part, g.dla, c.B, c.H, groups);
        err = hipGetLastError();
    }
    return err;
}

}  // namespace

#define MUIR_HD(K, V, F)                                                     \
    if (c.dk == K && c.dv == V) return c.bf16 ? F(bf16_t, K, V) : F(float, K, V);

hipError_t launch_head_decay_fwd(const HeadDecayCall &c, void *o, float *s_out, void *workspace, hipStream_t stream) {
#define MUIR_F(T, K, V) forward<T, K, V>(c, o, s_out, workspace, stream)
    MUIR_HD(64, 64, MUIR_F) MUIR_HD(64, 128, MUIR_F) MUIR_HD(128, 64, MUIR_F) MUIR_HD(128, 128, MUIR_F)
#undef MUIR_F
    return hipErrorInvalidValue;
}

hipError_t launch_head_decay_bwd(const HeadDecayCall &c, const HeadDecayGrads &g, void *workspace, hipStream_t stream) {
#define MUIR_F(T, K, V) backward<T, K, V>(c, g, workspace, stream)
    MUIR_HD(64, 64, MUIR_F) MUIR_HD(64, 128, MUIR_F) MUIR_HD(128, 64, MUIR_F) MUIR_HD(128, 128, MUIR_F)
#undef MUIR_F
    return hipErrorInvalidValue;
}

#undef MUIR_HD

}  // namespace muir
