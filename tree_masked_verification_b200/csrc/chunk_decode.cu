// chunk_decode.cu -- attention of few query rows (decode steps) to a paged
// e4m3 cache: up to 16 packed rows of a (sequence, KV head) at a time,
//   o = sum_j 2^{x_j} v_j / sum_j 2^{x_j},  x_j = scale * log2(e) * q.k_j.
//
// Bound by memory: a key's K and V are 2 (D + 1) bytes, read once, and want
// few instructions per byte.  Tensor-core tiles of 128 rows would be mostly
// padding here and need every code rewritten as bf16 in shared memory first
// (chunk_tc.cu on one sequence of 256k keys: 218 us).  Here codes go from
// shared memory to registers and become exact f16 pairs in one conversion
// each (e4m3 values fit f16), the operands of 16-row warp-level MMAs; the
// row scales, powers of two, are applied to the scores and to the weights,
// of which there are D times fewer.
//
// One CTA per SM takes its range of the schedule (chunk_plan.cuh, items of
// up to 16 rows).  A producer warp keeps four 128-key stages of codes and
// scale bytes on their way by TMA; four warps take the even tiles and four the
// odd ones, 32 keys each, every warp with a running maximum, sum and output
// of its own, joined once per item.  (16 keys of every tile a warp took 158
// us for 256k keys: the chain from the codes to the second product is a
// latency, and two key groups in it hide each other's.)  Fragments without transposing loads: the contraction order of an
// MMA is free as long as both operands follow it, so a lane's four bytes of
// K stand for the four d its A fragment (Q) holds, and for V a lane loads 16
// bytes of four keys and pairs the bytes of neighbouring keys itself.
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

constexpr int kDecRows = 16;
constexpr int kDecWarps = 8;
constexpr int kDecThreads = (kDecWarps + 1) * 32;

template <int D>
struct DecCfg {
    static constexpr int NS = D == 128 ? 4 : 8;             // stages
    static constexpr int RAW = 128 * D;
    static constexpr int STAGE = 2 * RAW + 256;             // K, V, scale bytes of K and of V
    static constexpr int OFF_STAGE = 0;                     // (codes at multiples of 1024: NS * 2 * RAW first)
    static constexpr int OFF_SCALE = NS * 2 * RAW;
    static constexpr int ROW = D + 4;                       // floats of an output row in the join
    static constexpr int OFF_JOIN = OFF_SCALE + NS * 256;   // [warp][row][ROW]
    static constexpr int OFF_STAT = OFF_JOIN + kDecWarps * kDecRows * ROW * 4;   // [warp][row][m, l, M, bad]
    static constexpr int OFF_BAR = OFF_STAT + kDecWarps * kDecRows * 16;
    static constexpr int OFF_MISC = OFF_BAR + 2 * NS * 8;   // abort; Start
    static constexpr int SMEM = OFF_MISC + 64;
    static constexpr int SMEM_ALLOC = SMEM + 1024;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(kPlanUnits * 8 <= OFF_SCALE, "the plan's scratch lies in the stages");
};

__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// two e4m3 codes to an f16 pair, exactly (0x7f, 0xff: NaN)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// d += a (16 x 16, rows) * b (16 x 8)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// 16-byte piece of a row of codes as TMA's swizzle left it: 128-byte rows in
// the 128-byte pattern, 64-byte rows in the 64-byte one
template <int D>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 1)
chunk_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ ChunkParams p) {
    using C = DecCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *empty = full + C::NS;
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
    Start *s_start = reinterpret_cast<Start *>(smem + C::OFF_MISC + 16);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) { mbar_init(full + i, 1); mbar_init(empty + i, kDecWarps / 2); }
        *s_abort = 0;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && warp == 0) check_ranges(p.q_start, p.B, p.N, p.status);
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
        __syncwarp();
        if (lane == 0 && *s_abort)                      // let the copies in flight land
            for (int i = max(0, issued - C::NS); i < issued; ++i) mbar_wait(full + i % C::NS, (i / C::NS) & 1);
        return;
    }

    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, t = lane & 3;
    const float nan = __int_as_float(0x7fc00000);
    constexpr int KI = D / 64;                          // 16-byte pieces of a K row per lane
    constexpr int NT = D / 8;                           // n8 tiles of the output
    float *join = reinterpret_cast<float *>(smem + C::OFF_JOIN);
    float4 *stat = reinterpret_cast<float4 *>(smem + C::OFF_STAT);
    int st = 0, ph = 0;
    bool ok = true;
    int head_first = -1, head_last = -1;
    while (w.next(p)) {
        if (w.s.bad && threadIdx.x == 0) raise_status(p.status, kStatusPrefixLenRange);
        // ---- Q: rows g and g + 8, the lane's d = [D/4 * t, D/4 * (t + 1)), as f16 fragments
        uint32_t qf[KI * 4][4];
        float qs[2];
        int row_lo[2], row_hi[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            const bool valid = row < w.it.rows;
            const int pr = w.it.r0 + (valid ? row : 0), tok = div_g(p, pr);
            row_hi[r] = w.s.bad ? 0 : w.s.L + tok + 1;
            row_lo[r] = p.window > 0 ? max(0, row_hi[r] - p.window) : 0;
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
            qs[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int i = 0; i < KI * 2; ++i) {
                const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)     // bf16 pair i*4+k of the lane: k-step (i*4+k)/2, half k&1
                    qf[(i * 4 + k) / 2][r + 2 * (k & 1)] = pack_f16x2(bf16_lo(x[k]) * mul, bf16_hi(x[k]) * mul);
            }
        }
        float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        bool bad[2] = {w.s.bad, w.s.bad};
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

        float f[2] = {1.f, 1.f};                        // 2^(m - M)
        for (int j = w.j0; j < w.j1; ++j, st = st + 1 == C::NS ? 0 : st + 1, ph ^= st == 0 ? 1 : 0) {
            if (((j - w.j0) & 1) != (warp >> 2)) continue;
            if (ok) ok = warp_wait(full + st, ph);
            const uint8_t *ks = smem + C::OFF_STAGE + st * 2 * C::RAW, *vs = ks + C::RAW;
            const uint8_t *sc = smem + C::OFF_SCALE + st * 256;
            const int r0 = (warp & 3) * 32;
            // ---- scores of 16 rows x 32 keys: key r0 + 8u + 2t (+1), rows g (values 0, 1) and g + 8 (2, 3)
            float x[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                uint4 c[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) c[u] = *reinterpret_cast<const uint4 *>(ks + piece<D>(r0 + 8 * u + g, KI * t + i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t cw = k == 0 ? c[u].x : k == 1 ? c[u].y : k == 2 ? c[u].z : c[u].w;
                        mma16816(x[u], qf[i * 4 + k], e4m3x2_to_f16x2(cw), e4m3x2_to_f16x2(cw >> 16));
                    }
            }
            // ---- scales: bytes of the lane's eight keys, K's as 2^(e - 127), V's as bytes
            int ev[8];
            bool nan_key = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t a = *reinterpret_cast<const uint16_t *>(sc + r0 + 8 * u + 2 * t);
                const uint32_t b = *reinterpret_cast<const uint16_t *>(sc + 128 + r0 + 8 * u + 2 * t);
                ev[2 * u] = b & 255;
                ev[2 * u + 1] = b >> 8;
                nan_key |= ev[2 * u] == kScaleNan || ev[2 * u + 1] == kScaleNan;
                const float s0 = __uint_as_float((a & 255) << 23), s1 = __uint_as_float((a >> 8) << 23);
                x[u][0] *= qs[0] * s0;
                x[u][1] *= qs[0] * s1;
                x[u][2] *= qs[1] * s0;
                x[u][3] *= qs[1] * s1;
            }
            uint32_t dead = 0;                          // V rows (bit per key of the lane) to be read as zeros
            if (__any_sync(0xffffffffu, nan_key) || w.partial(j)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int key = w.key0(j) + r0 + 8 * (k >> 1) + 2 * t + (k & 1);
                    const bool live = key >= w.it.lo && key < w.it.hi;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool see = live && key >= row_lo[r] && key < row_hi[r];
                        if (!see) x[k >> 1][2 * r + (k & 1)] = -INFINITY;
                        bad[r] |= see && ev[k] == kScaleNan;
                    }
                    // what no row may see, or holds NaN, must not meet a weight of 0
                    if (!live || ev[k] == kScaleNan) {
                        ev[k] = 127;
                        dead |= 1u << k;
                    }
                }
                __syncwarp();
            }
            // ---- weights
            uint32_t a[2][4];
            float M_up[2] = {1.f, 1.f};
            bool grew = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mt = -INFINITY, Mt = -INFINITY;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float xv = x[k >> 1][2 * r + (k & 1)];
                    mt = fmaxf(mt, xv);
                    // (2^23 + e) - (2^23 + 127), the conversion without the slow unit
                    Mt = fmaxf(Mt, xv + (__uint_as_float(0x4b000000u | ev[k]) - 8388735.f));
                }
                mt = quad_max(mt);
                Mt = quad_max(Mt);
                if (mt > m[r] + 8.f || Mt > M[r] + 8.f) {
                    if (mt > m[r] + 8.f) {
                        l[r] *= ex2(m[r] - mt);
                        m[r] = mt;
                    }
                    if (Mt > M[r] + 8.f) {
                        M_up[r] = ex2(M[r] - Mt);
                        M[r] = Mt;
                        grew = true;
                    }
                    f[r] = ex2(m[r] - M[r]);
                }
                const float mu = m[r] == -INFINITY ? 0.f : m[r];
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float w1 = ex2(x[k >> 1][2 * r + (k & 1)] - mu);
                    l[r] += w1;
                    y[k] = w1 * (__uint_as_float(static_cast<uint32_t>(ev[k]) << 23) * f[r]);
                }
                a[0][r] = pack_f16x2(y[0], y[1]);
                a[0][2 + r] = pack_f16x2(y[2], y[3]);
                a[1][r] = pack_f16x2(y[4], y[5]);
                a[1][2 + r] = pack_f16x2(y[6], y[7]);
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][0] *= M_up[0]; acc[i][1] *= M_up[0];
                    acc[i][2] *= M_up[1]; acc[i][3] *= M_up[1];
                }
            }
            // ---- O += P V, 16 keys at a time; n8 tile i: column (D/8) * n + i
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
                }
                if (__any_sync(0xffffffffu, dead)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            if ((dead >> (4 * h + k)) & 1u) vc[k][i] = 0;
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t lo01 = __byte_perm(vc[0][i], vc[1][i], 0x5140), hi01 = __byte_perm(vc[0][i], vc[1][i], 0x7362);
                    const uint32_t lo23 = __byte_perm(vc[2][i], vc[3][i], 0x5140), hi23 = __byte_perm(vc[2][i], vc[3][i], 0x7362);
                    mma16816(acc[4 * i + 0], a[h], e4m3x2_to_f16x2(lo01), e4m3x2_to_f16x2(lo23));
                    mma16816(acc[4 * i + 1], a[h], e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo23 >> 16));
                    mma16816(acc[4 * i + 2], a[h], e4m3x2_to_f16x2(hi01), e4m3x2_to_f16x2(hi23));
                    mma16816(acc[4 * i + 3], a[h], e4m3x2_to_f16x2(hi01 >> 16), e4m3x2_to_f16x2(hi23 >> 16));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
        }

        // ---- the eight warps' parts joined: row by row, m = max m_i,
        //      l = sum l_i 2^(m_i - m), o = sum O_i 2^(M_i - m) / l
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            int b = bad[r] || !ok;
            b |= __shfl_xor_sync(0xffffffffu, b, 1);
            b |= __shfl_xor_sync(0xffffffffu, b, 2);
            if (row < w.it.rows) {
                float *dst = join + (warp * kDecRows + row) * C::ROW + t * (D / 4);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < NT; i += 4)
                        *reinterpret_cast<float4 *>(dst + h * NT + i) =
                            make_float4(acc[i][2 * r + h], acc[i + 1][2 * r + h], acc[i + 2][2 * r + h], acc[i + 3][2 * r + h]);
                if (t == 0) stat[warp * kDecRows + row] = make_float4(m[r], l[r], M[r], b ? 1.f : 0.f);
            }
        }
        bar_sync(1, kDecWarps * 32);
        const bool whole = w.j0 == 0 && w.j1 == w.it.nt;
        const int which = w.j0 > 0 ? 0 : 1;
        {
            constexpr int PER = D / 16;                 // values of a thread
            const int row = threadIdx.x >> 4, col = (threadIdx.x & 15) * PER;
            if (row < w.it.rows) {
                float ms = -INFINITY, ls = 0.f, o[PER];
                bool nan_row = false;
#pragma unroll
                for (int i = 0; i < kDecWarps; ++i) ms = fmaxf(ms, stat[i * kDecRows + row].x);
#pragma unroll
                for (int k = 0; k < PER; ++k) o[k] = 0.f;
#pragma unroll
                for (int i = 0; i < kDecWarps; ++i) {
                    const float4 s = stat[i * kDecRows + row];
                    nan_row |= s.w != 0.f || s.y != s.y;
                    if (s.x == -INFINITY) continue;     // the warp saw none of the row's keys
                    ls += s.y * ex2(s.x - ms);
                    const float f = ex2(s.z - ms);
                    const float *src = join + (i * kDecRows + row) * C::ROW + col;
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

template <int D>
cudaError_t launch(const ChunkParams &p, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    using C = DecCfg<D>;
    constexpr int kMaxDev = 64;
    static bool attr_set[kMaxDev] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDev) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = C::SMEM_ALLOC;
    e = cudaLaunchKernelEx(&cfg, chunk_decode_kernel<D>, tm[0], tm[1], p);
    return e != cudaSuccess ? e : launch_chunk_merge(p, stream);
}

}  // namespace

cudaError_t launch_chunk_decode(const ChunkParams &p0, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    ChunkParams p = p0;
    p.item_rows = kDecRows;
    p.slot_rows = p.slot_rows < kDecRows ? p.slot_rows : kDecRows;
    p.c0 = 4;
    p.c1 = p.c2 = 4;
    p.min_share = 8;
    return p.D == 128 ? launch<128>(p, tm, stream) : launch<64>(p, tm, stream);
}

}  // namespace hta
