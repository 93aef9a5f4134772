// chunk_decode.cu -- attention of few query rows (decode steps) to a paged
// e4m3 cache, 8 or 16 packed rows of a (sequence, KV head) at a time,
//   o = sum_j 2^{x_j} v_j / sum_j 2^{x_j},  x_j = scale * log2(e) * q.k_j.
//
// Bound by memory: a key's K and V are 2 (D + 1) bytes, read once, and want
// few instructions per byte.  Tensor-core tiles of 128 rows would be mostly
// padding here and need every code rewritten as f16 in shared memory first
// (chunk_tc.cu on one sequence of 256k keys: 179 us).  Here codes go from
// shared memory to registers and become exact f16 pairs in one conversion
// each (e4m3 values fit f16), the operands of warp-level MMAs; the
// row scales, powers of two, are applied to the scores and to the weights,
// of which there are D times fewer.
//
// One CTA per SM takes its range of the schedule (chunk_plan.cuh, items of
// up to 8, or at D = 64 up to 16, rows).  A producer warp keeps five (D = 64:
// eight) 128-key stages of codes and scale bytes on their way by TMA; four warps
// take the even tiles and four the odd ones, 32 keys each, every warp with a
// running maximum, sum and output of its own, joined once per item.
//
// Both products put the long side on the MMA's 16 (keys, then d) and the
// query rows on its 8:  S^T = K Q^T,  O^T += V^T P^T.  With rows on the 16,
// decode's four to eight rows left most of each MMA empty, and the warp-level
// MMA, 18 cycles each, was two thirds busy (256k keys: 137 us).  Fragments
// without transposing loads: the contraction order of an MMA is free as long
// as both operands follow it, so a lane's four bytes of K stand for the four
// d its fragment of Q holds, and for V a lane loads D/8 bytes of four keys and
// pairs the bytes of neighbouring keys itself.  P^T is turned by movmatrix.
//
// Precision.  Q is scaled per row by a power of two into f16's range, which
// holds bf16's 8 bits exactly down to 2^-28 of the row's maximum.  Weights
// enter the second product as f16 relative to the running maximum of
// x_j + log2(scale of v_j), so that a large weight on a small V row is not
// lost beside a small weight on a large one; rounding them moves a weight by
// 2^-11.  Sums, maxima and outputs are fp32.
#include "chunk_plan.cuh"

namespace hta {

namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = (kDecWarps + 1) * 32;

template <int D, int NR>                                    // NR: groups of 8 rows
struct DecCfg {
    static constexpr int ROWS = 8 * NR;
    static constexpr int NS = D == 64 ? 8 : 5;              // stages
    static constexpr int RAW = 128 * D;
    static constexpr int STAGE = 2 * RAW + 256;             // K, V, scale bytes of K and of V
    static constexpr int OFF_STAGE = 0;                     // (codes at multiples of 1024: NS * 2 * RAW first)
    static constexpr int OFF_SCALE = NS * 2 * RAW;
    static constexpr int ROW = D + 4;                       // floats of an output row in the join
    static constexpr int OFF_JOIN = OFF_SCALE + NS * 256;   // [warp][row][ROW]
    static constexpr int OFF_STAT = OFF_JOIN + kDecWarps * ROWS * ROW * 4;   // [warp][row][m, l, M, bad]
    static constexpr int OFF_BAR = OFF_STAT + kDecWarps * ROWS * 16;
    static constexpr int OFF_MISC = OFF_BAR + 2 * NS * 8;   // abort; Start
    static constexpr int SMEM = OFF_MISC + 16 + 80;
    static_assert(sizeof(Start) <= 80, "room of the plan's result");
    static constexpr int SMEM_ALLOC = SMEM + 1024;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(kPlanUnits * 8 <= OFF_SCALE, "the plan's scratch lies in the stages");
};

// two e4m3 codes to an f16 pair, exactly (0x7f, 0xff: NaN)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}
// d += a (16 x 16, rows) * b (16 x 8)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// over the lanes of one t (lane % 4): the keys of a warp
__device__ __forceinline__ float keys_max(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 16-byte piece of a row of codes as TMA's swizzle left it: 128-byte rows in
// the 128-byte pattern, 64-byte rows in the 64-byte one
template <int D>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int D, int NR>
__global__ void __launch_bounds__(kDecThreads, 1)
chunk_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ ChunkParams p) {
    using C = DecCfg<D, NR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *empty = full + C::NS;
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
    Start *s_start = reinterpret_cast<Start *>(smem + C::OFF_MISC + 16);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) { mbar_init(full + i, 1); mbar_init(empty + i, kDecWarps); }
        *s_abort = 0;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    plan_start(p, reinterpret_cast<long long *>(smem + C::OFF_STAGE), s_start);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");     // the plan's scratch becomes a stage
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort, p.status));
    };
    Walk w;
    w.start(p, s_start);
    const int bs = p.cache.block_size, bsh = __ffs(bs) - 1;

    if (warp == kDecWarps) {
        // ----------------------------------------------------- TMA producer
        if (lane == 0) { tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
        const int nb = 128 >> bsh;
        int st = 0, ph = 1, issued = 0;
        bool ok = true;
        while (ok && w.next(p)) {
            const int32_t *row = p.cache.block_table + static_cast<size_t>(w.cur_b) * p.cache.max_blocks;
            const int first = w.it.lo >> bsh, last = (w.it.hi - 1) >> bsh;
            // (blocks outside the item's keys are not looked up: one inside is repeated and masked)
            auto fetch = [&](int j) {
                return lane < nb && w.it.hi > 0 && j < w.j1 ? row[min(max((w.key0(j) >> bsh) + lane, first), last)] : 0;
            };
            int id = fetch(w.j0);
            for (int j = w.j0; j < w.j1; ++j) {
                if (!warp_wait(empty + st, ph)) { ok = false; break; }
                if (w.it.hi == 0) {                     // nothing to read: a wholly masked tile
                    if (lane == 0) mbar_arrive(full + st);
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(full + st, C::STAGE);
                    __syncwarp();
                    if (lane < nb) {
                        int n = id;
                        if (n < 0 || n >= p.cache.num_blocks) {
                            raise_status(p.status, kStatusBadBlock);
                            n = 0;
                        }
                        const int y = (n * p.Hkv + w.cur_kvh) << bsh, at = lane << bsh;
                        uint8_t *stage = smem + C::OFF_STAGE + st * 2 * C::RAW, *sc = smem + C::OFF_SCALE + st * 256 + at;
                        tma_load_2d(stage + at * D, &tm_k, full + st, 0, y);
                        bulk_load(sc, p.cache.k_scale + y, bs, full + st);
                        tma_load_2d(stage + C::RAW + at * D, &tm_v, full + st, 0, y);
                        bulk_load(sc + 128, p.cache.v_scale + y, bs, full + st);
                    }
                }
                id = fetch(j + 1);
                ++issued;
                if (++st == C::NS) { st = 0; ph ^= 1; }
            }
        }
        if (blockIdx.x == 0) check_ranges(p.q_start, p.B, p.N, p.status);
        __syncwarp();
        if (lane == 0 && *s_abort)                      // let the copies in flight land
            for (int i = max(0, issued - C::NS); i < issued; ++i) mbar_wait(full + i % C::NS, (i / C::NS) & 1);
        return;
    }

    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, t = lane & 3;
    const float nan = __int_as_float(0x7fc00000);
    constexpr int KI = D / 64;                          // 16-byte pieces of a K row per lane
    constexpr int MT = D / 16;                          // m16 tiles of the output
    float *join = reinterpret_cast<float *>(smem + C::OFF_JOIN);
    float4 *stat = reinterpret_cast<float4 *>(smem + C::OFF_STAT);
    int st = 0, ph = 0;
    bool ok = true;
    int head_first = -1, head_last = -1;
    while (w.next(p)) {
        if (w.s.bad && threadIdx.x == 0) raise_status(p.status, kStatusPrefixLenRange);
        // ---- Q: row 8n + g, the lane's d = [D/4 * t, D/4 * (t + 1)), as f16 fragments
        uint32_t qf[NR][KI * 4][2];
        float up_of[NR];                                // scale * log2(e) * 2^-(the row's shift)
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = 8 * n + g;
            const bool valid = row < w.it.rows;
            const int pr = w.it.r0 + (valid ? row : 0), tok = div_g(p, pr);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + (w.s.s0 + tok) * p.q_stride + static_cast<size_t>(w.cur_kvh * p.G + pr - tok * p.G) * D + t * (D / 4));
            uint4 u[KI * 2];
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < KI * 2; ++i) {
                u[i] = valid ? src[i] : make_uint4(0u, 0u, 0u, 0u);
                big = __vmaxu2(__vmaxu2(big, u[i].x & 0x7fff7fffu), __vmaxu2(u[i].y & 0x7fff7fffu, u[i].z & 0x7fff7fffu));
                big = __vmaxu2(big, u[i].w & 0x7fff7fffu);
            }
            big = max(big & 0xffffu, big >> 16);
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // largest magnitude into [2^14, 2^15)
            const int up = min(14 - (static_cast<int>(big >> 7) - 127), 100);
            const float mul = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
            up_of[n] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int i = 0; i < KI * 2; ++i) {
                const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)             // pair i*4+k of the lane: k-step (i*4+k)/2, half k&1
                    qf[n][(i * 4 + k) / 2][k & 1] = pack_f16x2(bf16_lo(x[k]) * mul, bf16_hi(x[k]) * mul);
            }
        }
        // ---- the rows of this lane's scores: 8n + 2t + r, index 2n + r
        float qs[2 * NR], m[2 * NR], M[2 * NR], l[2 * NR], f[2 * NR];   // f = 2^(m - M)
        int row_lo[2 * NR], row_hi[2 * NR];
        bool bad[2 * NR];
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) {
            const int row = 8 * (i >> 1) + 2 * t + (i & 1);
            qs[i] = __shfl_sync(0xffffffffu, up_of[i >> 1], (2 * t + (i & 1)) * 4);
            row_hi[i] = w.s.bad ? 0 : w.s.L + div_g(p, w.it.r0 + min(row, w.it.rows - 1)) + 1;
            row_lo[i] = p.window > 0 ? max(0, row_hi[i] - p.window) : 0;
            m[i] = M[i] = -INFINITY;
            l[i] = 0.f;
            f[i] = 1.f;
            bad[i] = w.s.bad;
        }
        float acc[NR][MT][4];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;

        for (int j = w.j0; j < w.j1; ++j, st = st + 1 == C::NS ? 0 : st + 1, ph ^= st == 0 ? 1 : 0) {
            // Every warp sees every phase of a stage and gives it back, whether the
            // tile is its own or not: a wait by parity that skipped a phase would
            // take the one before the last for the one it waits for.
            if (ok) ok = warp_wait(full + st, ph);
            if (((j - w.j0) & 1) != (warp >> 2)) {
                if (lane == 0) mbar_arrive(empty + st);
                continue;
            }
            const uint8_t *ks = smem + C::OFF_STAGE + st * 2 * C::RAW, *vs = ks + C::RAW;
            const uint8_t *sc = smem + C::OFF_SCALE + st * 256;
            const int r0 = (warp & 3) * 32;
            // ---- scores of 32 keys: m16 tile h holds keys r0 + 16h + g (values 0, 1: rows 2t, 2t + 1)
            //      and r0 + 16h + 8 + g (values 2, 3); u = 2h + (key + 8)
            float x[NR][2][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[n][h][0] = x[n][h][1] = x[n][h][2] = x[n][h][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                uint4 c[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) c[u] = *reinterpret_cast<const uint4 *>(ks + piece<D>(r0 + 8 * u + g, KI * t + i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 c0 = c[2 * h], c1 = c[2 * h + 1];
                        const uint32_t w0 = k == 0 ? c0.x : k == 1 ? c0.y : k == 2 ? c0.z : c0.w;
                        const uint32_t w1 = k == 0 ? c1.x : k == 1 ? c1.y : k == 2 ? c1.z : c1.w;
                        const uint32_t a[4] = {e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w1), e4m3x2_to_f16x2(w0 >> 16),
                                               e4m3x2_to_f16x2(w1 >> 16)};
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816(x[n][h], a, qf[n][i * 4 + k][0], qf[n][i * 4 + k][1]);
                    }
            }
            // ---- scales of the lane's four keys, K's as 2^(e - 127), V's as bytes
            int ev[4];
            bool nan_key = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float s = __uint_as_float(static_cast<uint32_t>(sc[r0 + 8 * u + g]) << 23);
                ev[u] = sc[128 + r0 + 8 * u + g];
                nan_key |= ev[u] == kScaleNan;
#pragma unroll
                for (int i = 0; i < 2 * NR; ++i) x[i >> 1][u >> 1][2 * (u & 1) + (i & 1)] *= qs[i] * s;
            }
            const bool special = __any_sync(0xffffffffu, nan_key) || w.partial(j);
            if (special) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int key = w.key0(j) + r0 + 8 * u + g;
                    const bool live = key >= w.it.lo && key < w.it.hi;
#pragma unroll
                    for (int i = 0; i < 2 * NR; ++i) {
                        const bool see = live && key >= row_lo[i] && key < row_hi[i];
                        if (!see) x[i >> 1][u >> 1][2 * (u & 1) + (i & 1)] = -INFINITY;
                        bad[i] |= see && ev[u] == kScaleNan;
                    }
                    if (!live || ev[u] == kScaleNan) ev[u] = 127;
                }
                __syncwarp();
            }
            // ---- weights, P^T turned into the second product's fragments
            uint32_t pb[NR][2][2];
            float M_up[2 * NR];
            bool grew = false;
#pragma unroll
            for (int i = 0; i < 2 * NR; ++i) {
                M_up[i] = 1.f;
                float mt = -INFINITY, Mt = -INFINITY;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float xv = x[i >> 1][u >> 1][2 * (u & 1) + (i & 1)];
                    mt = fmaxf(mt, xv);
                    // (2^23 + e) - (2^23 + 127): the conversion without the slow unit
                    Mt = fmaxf(Mt, xv + (__uint_as_float(0x4b000000u | ev[u]) - 8388735.f));
                }
                mt = keys_max(mt);
                Mt = keys_max(Mt);
                if (mt > m[i] + 8.f || Mt > M[i] + 8.f) {
                    if (mt > m[i] + 8.f) {
                        l[i] *= ex2(m[i] - mt);
                        m[i] = mt;
                    }
                    if (Mt > M[i] + 8.f) {
                        M_up[i] = ex2(M[i] - Mt);
                        M[i] = Mt;
                        grew = true;
                    }
                    f[i] = ex2(m[i] - M[i]);
                }
                const float mu = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float &xv = x[i >> 1][u >> 1][2 * (u & 1) + (i & 1)];
                    const float w1 = ex2(xv - mu);
                    l[i] += w1;
                    xv = w1 * (__uint_as_float(static_cast<uint32_t>(ev[u]) << 23) * f[i]);
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    pb[n][h][0] = transpose8x8(pack_f16x2(x[n][h][0], x[n][h][1]));
                    pb[n][h][1] = transpose8x8(pack_f16x2(x[n][h][2], x[n][h][3]));
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[n][i][0] *= M_up[2 * n]; acc[n][i][1] *= M_up[2 * n + 1];
                        acc[n][i][2] *= M_up[2 * n]; acc[n][i][3] *= M_up[2 * n + 1];
                    }
            }
            // ---- O^T += V^T P^T, 16 keys at a time: keys 2t, 2t + 1, 2t + 8, 2t + 9 of them, the lane's
            //      columns (D/8) g + c; m16 tile i holds c = 2i (row g) and 2i + 1 (row g + 8)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t vc[4][D / 32];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = r0 + 16 * h + 2 * t + (k & 1) + 8 * (k >> 1);
                    if constexpr (D == 128) {
                        const uint4 c = *reinterpret_cast<const uint4 *>(vs + piece<D>(r, g));
                        vc[k][0] = c.x; vc[k][1] = c.y; vc[k][2] = c.z; vc[k][3] = c.w;
                    } else {
                        const uint2 c = *reinterpret_cast<const uint2 *>(vs + piece<D>(r, g >> 1) + (g & 1) * 8);
                        vc[k][0] = c.x; vc[k][1] = c.y;
                    }
                    if (special) {
                        // what no row may see, or holds NaN, must not meet a weight of 0
                        const int key = w.key0(j) + r;
                        if (key < w.it.lo || key >= w.it.hi || sc[128 + r] == kScaleNan)
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) vc[k][i] = 0;
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t lo01 = __byte_perm(vc[0][i], vc[1][i], 0x5140), hi01 = __byte_perm(vc[0][i], vc[1][i], 0x7362);
                    const uint32_t lo23 = __byte_perm(vc[2][i], vc[3][i], 0x5140), hi23 = __byte_perm(vc[2][i], vc[3][i], 0x7362);
                    const uint32_t a[4] = {e4m3x2_to_f16x2(lo01), e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo23),
                                           e4m3x2_to_f16x2(lo23 >> 16)};
                    const uint32_t b[4] = {e4m3x2_to_f16x2(hi01), e4m3x2_to_f16x2(hi01 >> 16), e4m3x2_to_f16x2(hi23),
                                           e4m3x2_to_f16x2(hi23 >> 16)};
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        mma16816(acc[n][2 * i], a, pb[n][h][0], pb[n][h][1]);
                        mma16816(acc[n][2 * i + 1], b, pb[n][h][0], pb[n][h][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
        }

        // ---- the eight warps' parts joined: row by row, m = max m_i,
        //      l = sum l_i 2^(m_i - m), o = sum O_i 2^(M_i - m) / l
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) {
            const int n = i >> 1, row = 8 * n + 2 * t + (i & 1);
            int b = bad[i] || !ok;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
                b |= __shfl_xor_sync(0xffffffffu, b, o);
            }
            if (row < w.it.rows) {
                float *dst = join + (warp * C::ROWS + row) * C::ROW + g * (D / 8);
#pragma unroll
                for (int c = 0; c < MT; c += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * c) = make_float4(acc[n][c][i & 1], acc[n][c][2 + (i & 1)],
                                                                           acc[n][c + 1][i & 1], acc[n][c + 1][2 + (i & 1)]);
                if (g == 0) stat[warp * C::ROWS + row] = make_float4(m[i], l[i], M[i], b ? 1.f : 0.f);
            }
        }
        bar_sync(1, kDecWarps * 32);
        const bool whole = w.j0 == 0 && w.j1 == w.it.nt;
        const int which = w.j0 > 0 ? 0 : 1;
        {
            constexpr int TPR = 256 / C::ROWS, PER = D / TPR > 4 ? D / TPR : 4;   // threads of a row, values of a thread
            const int row = threadIdx.x / (D / PER), col = threadIdx.x % (D / PER) * PER;
            if (row < w.it.rows) {
                float ms = -INFINITY, ls = 0.f, o[PER];
                bool nan_row = false;
#pragma unroll
                for (int i = 0; i < kDecWarps; ++i) ms = fmaxf(ms, stat[i * C::ROWS + row].x);
#pragma unroll
                for (int k = 0; k < PER; ++k) o[k] = 0.f;
#pragma unroll
                for (int i = 0; i < kDecWarps; ++i) {
                    const float4 s = stat[i * C::ROWS + row];
                    nan_row |= s.w != 0.f || s.y != s.y;
                    if (s.x == -INFINITY) continue;     // the warp saw none of the row's keys
                    ls += s.y * ex2(s.x - ms);
                    const float f = ex2(s.z - ms);
                    const float *src = join + (i * C::ROWS + row) * C::ROW + col;
#pragma unroll
                    for (int k = 0; k < PER; k += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(src + k);
                        o[k] = fmaf(f, v.x, o[k]);
                        o[k + 1] = fmaf(f, v.y, o[k + 1]);
                        o[k + 2] = fmaf(f, v.z, o[k + 2]);
                        o[k + 3] = fmaf(f, v.w, o[k + 3]);
                    }
                }
                const float inv = nan_row ? nan : ls > 0.f ? 1.f / ls : 0.f;
                const float lse = nan_row ? nan : ls > 0.f ? (ms + lg2(ls)) * kLn2 : -INFINITY;
#pragma unroll
                for (int k = 0; k < PER; ++k) o[k] *= inv;
                if (whole) {
                    const int pr = w.it.r0 + row, tok = div_g(p, pr);
                    const size_t orow = static_cast<size_t>(w.s.s0 + tok) * p.Hq + w.cur_kvh * p.G + pr - tok * p.G;
#pragma unroll
                    for (int k = 0; k < PER; k += 4)
                        *reinterpret_cast<uint2 *>(p.out + orow * D + col + k) =
                            make_uint2(pack_bf16x2(o[k], o[k + 1]), pack_bf16x2(o[k + 2], o[k + 3]));
                    if (col == 0) p.lse[orow] = lse;
                } else {
                    const long long prow = slot_row(p, blockIdx.x, which) + row;
#pragma unroll
                    for (int k = 0; k < PER; k += 4)
                        *reinterpret_cast<float4 *>(p.o_part + prow * D + col + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    if (col == 0) p.lse_part[prow] = lse;
                }
            }
        }
        if (!whole && threadIdx.x == 0) {
            write_head(p, w, s_start, which);
            if (which == 0) head_first = 1; else head_last = 1;
        }
        bar_sync(1, kDecWarps * 32);                    // the join's buffers are free again
    }
    if (threadIdx.x == 0) {
        if (head_first < 0) p.heads[2 * blockIdx.x].rows = 0;
        if (head_last < 0) p.heads[2 * blockIdx.x + 1].rows = 0;
    }
}

template <int D, int NR>
cudaError_t launch(const ChunkParams &p, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    using C = DecCfg<D, NR>;
    constexpr int kMaxDev = 64;
    static bool attr_set[kMaxDev] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_decode_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDev) attr_set[dev] = true;
    }
    OverlappedLaunch l(dim3(p.grid), dim3(kDecThreads), C::SMEM_ALLOC, stream);
    e = cudaLaunchKernelEx(&l.cfg, chunk_decode_kernel<D, NR>, tm[0], tm[1], p);
    return e != cudaSuccess ? e : launch_chunk_merge(p, stream);
}

}  // namespace

cudaError_t launch_chunk_decode(const ChunkParams &p0, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    ChunkParams p = p0;
    // 8 rows at a time; at D = 64 up to 16 where a KV head has more than 8 query heads,
    // the second group of 8 sharing the codes' loads and conversions (32 x 8k keys: 67
    // against 93 us).  At D = 128 two groups do not fit the registers: 199 against 108.
    const bool wide = p.D == 64 && p.G > 8;
    p.item_rows = wide ? 16 : 8;
    p.slot_rows = p.slot_rows < p.item_rows ? p.slot_rows : p.item_rows;
    p.c0 = 4;
    p.c1 = p.c2 = 4;
    p.min_share = 8;
    if (p.D == 128) return launch<128, 1>(p, tm, stream);
    return wide ? launch<64, 2>(p, tm, stream) : launch<64, 1>(p, tm, stream);
}

}  // namespace hta
